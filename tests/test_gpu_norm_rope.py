"""spla_qk_norm_rope against the 64-bit form.

Bound per element: with u = 2^-24 and y = a cos t - b sin t, the norm is off by at most
20 u (its sum of 16 products a lane and three shuffles, halved by the root; the root's
2 steps, gamma and the product), the sine and cosine by 8 u (their 2 steps and the
rounding of the reduced angle, 2^-24 of at most a whole turn), the products and the sum
by 3 u: 32 u (|a| + |b|), and half a step of the stored type.
"""
import pytest
import torch

from block_sparse_linear_b200 import SplaConfig, SplaError, SplaPagedKV, _lib, qk_norm_rope

from . import paged_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def cfg_of(hq, hkv, d, dtype, block=64):
    return SplaConfig(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=block, top_k=1,
                      dtype=dtype)


def freqs(rot, base=1e4):
    return base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)


def check(got, x, gamma, positions, inv, rot, inter, eps, dtype, left):
    """Rows with a position match; the others still hold `left`."""
    want, size = ref.norm_rope(x.double(), None if gamma is None else gamma.double(), positions,
                               inv, rot, inter, eps)
    tol = 32 * ref.U32 * size + ref.half_step(dtype) * want.abs() + 1e-30
    live = positions >= 0
    err = (got.double() - want).abs()[live]
    assert (err <= tol[live]).all(), float((err / tol[live]).max())
    assert (got[~live].float() == left).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (8, 8, 64), (32, 8, 128), (2, 1, 128)])
@pytest.mark.parametrize("rows,rot,inter", [(1, 64, False), (5, 64, True), (37, 16, False),
                                            (64, 48, True), (1300, 32, False), (3, 0, False)])
def test_rows_match(dtype, hq, hkv, d, rows, rot, inter):
    g = torch.Generator("cuda").manual_seed(rows * d + rot)
    dt = DT[dtype]
    cfg = cfg_of(hq, hkv, d, dtype)
    pad = 16 * (rows % 3)                                   # row strides beyond the heads'
    w = (hq + 2 * hkv) * d + pad
    qkv = (3 * torch.randn((rows, w), device="cuda", generator=g)).to(dt)
    q = qkv[:, :hq * d].unflatten(1, (hq, d))
    k = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    v = qkv[:, (hq + hkv) * d:(hq + 2 * hkv) * d].unflatten(1, (hkv, d))
    pos = torch.randint(0, 1 << 20, (rows,), device="cuda", generator=g, dtype=torch.int32)
    pos[2::5] = -1
    qg = 1 + 0.3 * torch.randn(d, device="cuda", generator=g)
    kg = -qg if rows % 2 else None
    inv = freqs(rot) if rot else None
    out = [torch.full((rows, h, d), 7.0, device="cuda", dtype=dt) for h in (hq, hkv, hkv)]
    qk_norm_rope(cfg, q, k, v, pos, inv, qg, kg, 1e-5, inter, *out)
    check(out[0], q, qg, pos, inv, rot, inter, 1e-5, dt, 7.0)
    check(out[1], k, kg, pos, inv, rot, inter, 1e-5, dt, 7.0)
    live = pos >= 0
    assert torch.equal(out[2][live], v[live]) and (out[2][~live] == 7).all()


@pytest.mark.parametrize("d,block", [(64, 128), (128, 64)])
def test_pages_by_slot(d, block):
    """Keys and values land at their slots; other slots, and rows without one, are left."""
    g = torch.Generator("cuda").manual_seed(d)
    hq, hkv, rows, phys = 8, 2, 203, 7
    cfg = cfg_of(hq, hkv, d, "bf16", block)
    mk = lambda h: torch.randn((rows, h, d), device="cuda", generator=g).bfloat16()
    q, k, v = mk(hq), mk(hkv), mk(hkv)
    pos = torch.randint(0, 4096, (rows,), device="cuda", generator=g, dtype=torch.int32)
    slots = torch.randperm(phys * block, device="cuda", generator=g)[:rows]
    pos[0], slots[1], slots[2] = -1, -1, phys * block        # padding, no slot, past the pool
    inv, ones = freqs(d), torch.ones(d, device="cuda")
    shape = (phys, hkv, block, d)
    kv = SplaPagedKV(cfg, torch.full(shape, 9.0, device="cuda", dtype=torch.bfloat16),
                     torch.full(shape, 9.0, device="cuda", dtype=torch.bfloat16))
    qo = qk_norm_rope(cfg, q, k, v, pos, inv, ones, ones, kv=kv, slots=slots)
    check(qo, q, ones, pos, inv, d, False, 1e-6, torch.bfloat16, 0.0)
    assert kv.status() == _lib.SPLA_DEV_BAD_BLOCK_TABLE
    keep = torch.arange(3, rows, device="cuda")
    flat = lambda p: p.transpose(1, 2).reshape(-1, hkv, d)
    check(flat(kv.k_pool)[slots[keep]], k[keep], ones, pos[keep], inv, d, False, 1e-6,
          torch.bfloat16, 0.0)
    assert torch.equal(flat(kv.v_pool)[slots[keep]], v[keep])
    rest = torch.ones(phys * block, dtype=torch.bool, device="cuda")
    rest[slots[keep]] = False
    assert (flat(kv.k_pool)[rest] == 9).all() and (flat(kv.v_pool)[rest] == 9).all()


def test_slots_past_32_bits_of_elements():
    """A pool of more than 2^31 elements, written in its last block."""
    hkv, d, block = 8, 128, 128
    phys = 2 ** 31 // (hkv * d * block) + 2
    cfg = cfg_of(8, hkv, d, "bf16", block)
    kp = torch.zeros((phys, hkv, block, d), device="cuda", dtype=torch.bfloat16)
    vp = torch.zeros_like(kp)
    kv = SplaPagedKV(cfg, kp, vp)
    x = torch.randn((2, 8, d), device="cuda").bfloat16()
    slots = torch.tensor([phys * block - 1, (phys - 1) * block], device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    qk_norm_rope(cfg, x, x, x, pos, kv=kv, slots=slots)
    assert torch.equal(kp[-1, :, block - 1], x[0]) and torch.equal(vp[-1, :, 0], x[1])
    assert int((kp != 0).sum()) == int((x != 0).sum())


def test_nan_stays_in_its_head_and_zero_rows_are_zero():
    cfg = cfg_of(4, 1, 64, "f32")
    q = torch.randn((3, 4, 64), device="cuda")
    q[1, 2, 5] = float("nan")
    q[2, 3] = 0
    k = torch.zeros((3, 1, 64), device="cuda")
    pos = torch.arange(3, dtype=torch.int32, device="cuda")
    qo, ko, vo = qk_norm_rope(cfg, q, k, None, pos, freqs(64), torch.ones(64, device="cuda"),
                              torch.ones(64, device="cuda"))
    assert vo is None and torch.isnan(qo[1, 2]).all() and int(torch.isnan(qo).sum()) == 64
    assert (qo[2, 3] == 0).all() and (ko == 0).all()


def test_no_rows_and_another_stream():
    cfg = cfg_of(4, 1, 64, "bf16")
    z = torch.zeros((0, 4, 64), device="cuda", dtype=torch.bfloat16)
    zk = torch.zeros((0, 1, 64), device="cuda", dtype=torch.bfloat16)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert qk_norm_rope(cfg, z, zk, zk, none, freqs(64))[0].shape == (0, 4, 64)
    q = torch.randn((50, 4, 64), device="cuda").bfloat16()
    k = torch.randn((50, 1, 64), device="cuda").bfloat16()
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    want = qk_norm_rope(cfg, q, k, k, pos, freqs(64))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = qk_norm_rope(cfg, q, k, k, pos, freqs(64))
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_overlapping_outputs_are_refused():
    cfg = cfg_of(4, 1, 64, "bf16")
    buf = torch.zeros((4, 6, 64), device="cuda", dtype=torch.bfloat16)
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    q, k, v = buf[:, :4], buf[:, 4:5], buf[:, 5:]
    with pytest.raises(SplaError):
        qk_norm_rope(cfg, q, k, v, pos, q_out=buf.view(-1)[:4 * 4 * 64])


def test_one_row_of_any_stride_and_a_named_stream():
    """A single row's stride says nothing; tensors made by a call on a named stream belong to
    it."""
    cfg = cfg_of(4, 1, 64, "bf16")
    base = torch.randn(2000, device="cuda").bfloat16()
    q = base.as_strided((1, 4, 64), (3, 64, 1))
    k = base.as_strided((1, 1, 64), (7, 5, 1), 512)
    pos = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    want = qk_norm_rope(cfg, q.contiguous(), k.contiguous(), None, pos, freqs(64))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = qk_norm_rope(cfg, q, k, None, pos, freqs(64), stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
