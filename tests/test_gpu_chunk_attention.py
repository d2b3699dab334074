"""spla_chunk_attention against the 64-bit form, every sequence, query and head, with the
bounds that paged_ref.chunk derives."""
import math

import pytest
import torch

from block_sparse_linear_b200 import SplaConfig, SplaDecodeCache, SplaPagedKV, _lib

from . import paged_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAN, INF = math.nan, math.inf


def build(seed, lens, max_new, hq, hkv, d, block, dtype, spare=3, mbp=None, spread=1.0):
    """Random pages behind a shuffled table; every slot past a length, and every page no
    sequence holds, is NaN."""
    g = torch.Generator("cuda").manual_seed(seed)
    dt, batch = DT[dtype], len(lens)
    nb = [-(-n // block) for n in lens]
    mbp = mbp or max(max(nb), 1)
    phys = sum(nb) + spare
    perm = torch.randperm(phys, device="cuda", generator=g).to(torch.int32)
    table = torch.full((batch, mbp), -1, dtype=torch.int32, device="cuda")
    pools = [(spread * torch.randn((phys, hkv, block, d), device="cuda", generator=g)).to(dt)
             for _ in range(2)]
    at = 0
    for b, k in enumerate(nb):
        table[b, :k] = perm[at:at + k]
        if lens[b] % block:
            for p in pools:
                p[perm[at + k - 1].long(), :, lens[b] % block:] = NAN
        at += k
    for p in pools:
        p[perm[at:].long()] = NAN
    cfg = SplaConfig(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=block, top_k=1,
                     dtype=dtype)
    kv = SplaPagedKV(cfg, *pools, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    q = (spread * torch.randn((batch, max_new, hq, d), device="cuda", generator=g)).to(dt)
    return kv, q


def run(kv, q, n_new, lens=None):
    out = torch.full_like(q, 5.0)
    lse = torch.full(q.shape[:3], 5.0, dtype=torch.float32, device="cuda")
    n = torch.tensor(n_new, dtype=torch.int32, device="cuda")
    kv.chunk_attention(q, n, out=out, lse=lse, lens=lens)
    return out, lse


def check(kv, q, n_new, lens, out, lse, skip=()):
    cfg = kv.cfg
    g = cfg.num_q_heads // cfg.num_kv_heads
    scale = cfg.softmax_scale if cfg.softmax_scale > 0 else 1 / math.sqrt(cfg.head_dim)
    for b, (n, L) in enumerate(zip(n_new, lens)):
        assert (out[b, n:] == 5).all() and (lse[b, n:] == 5).all(), b
        if n == 0 or b in skip:
            continue
        for h in range(cfg.num_kv_heads):
            K = ref.tokens(kv.k_pool, kv.block_table[b], L, h)
            V = ref.tokens(kv.v_pool, kv.block_table[b], L, h)
            for e in range(h * g, (h + 1) * g):
                o, z, to, tz = ref.chunk(q[b, :n, e].double(), K, V, L, scale, q.dtype)
                got, gz = out[b, :n, e].double(), lse[b, :n, e].double()
                fin = torch.isfinite(o)
                assert torch.equal(got[~fin].nan_to_num(1.5), o[~fin].nan_to_num(1.5)), (b, e)
                err = (got - o).abs()[fin]
                assert (err <= to[fin]).all(), (b, e, float((err / to[fin]).max()))
                ez = (gz - z).abs()
                assert (ez <= tz).all(), (b, e, float((ez / tz).max()))


CASES = [
    # lens, n_new, max_new
    ([1], [1], 1),
    ([1, 63, 64, 65, 0, 127, 128, 129], [1, 1, 1, 1, 0, 1, 1, 1], 1),
    ([300, 700, 64, 5], [1, 3, 64, 5], 64),
    ([33, 257, 513], [33, 30, 17], 33),
    ([400, 129, 1, 128], [400, 129, 0, 128], 400),
    ([1000, 300], [259, 300], 300),
    ([2100], [2], 7),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d,block", [(4, 1, 64, 64), (4, 2, 128, 64), (2, 2, 128, 128),
                                            (8, 2, 128, 64), (2, 1, 64, 128), (3, 3, 64, 64)])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_chunk_matches(dtype, hq, hkv, d, block, case):
    lens, n_new, max_new = CASES[case]
    kv, q = build(case, lens, max_new, hq, hkv, d, block, dtype)
    out, lse = run(kv, q, n_new)
    check(kv, q, n_new, lens, out, lse)
    assert kv.status() == 0


@pytest.mark.parametrize("dtype,n_new", [("bf16", 1), ("bf16", 9), ("bf16", 150), ("f32", 2)])
def test_long_and_ragged(dtype, n_new):
    """Work split over the cache and joined: thousands of tokens, lengths far apart."""
    lens = [20011, 1500, 9000 + n_new, max(n_new, 40)]
    kv, q = build(7, lens, n_new, 8, 2, 128, 64, dtype)
    out, lse = run(kv, q, [n_new] * 4)
    check(kv, q, [n_new] * 4, lens, out, lse)


@pytest.mark.parametrize("dtype,L", [("bf16", 200003), ("f32", 60001)])
@pytest.mark.parametrize("n_new", [1, 40])
def test_one_long_sequence(dtype, L, n_new):
    """Every thread block takes many steps in a row of one sequence."""
    kv, q = build(30, [L], n_new, 4, 1, 64, 64, dtype)
    out, lse = run(kv, q, [n_new])
    check(kv, q, [n_new], [L], out, lse)
    assert kv.status() == 0


@pytest.mark.parametrize("dtype,lens", [("bf16", [200003, 90, 130001]), ("f32", [100001, 90, 65003])])
@pytest.mark.parametrize("n_new", [1, 17])
def test_long_runs_over_few_sequences(dtype, lens, n_new):
    """Runs of more than 16 steps with fewer units than thread blocks: the units' starts count
    in the split there, and a run may end one unit and begin the next."""
    kv, q = build(32, lens, n_new, 4, 1, 64, 64, dtype)
    out, lse = run(kv, q, [n_new] * 3)
    check(kv, q, [n_new] * 3, lens, out, lse)
    assert kv.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("max_new", [9, 140])
def test_queries_past_the_counts_have_no_part(dtype, max_new):
    """Rows of q past a sequence's count may hold anything."""
    lens, n_new = [700, 150, 3000, 64], [5, 0, max_new, 1]
    kv, q = build(33, lens, max_new, 8, 2, 128, 64, dtype)
    q[0, 5:] = NAN
    q[1] = INF
    q[3, 1:] = -INF
    out, lse = run(kv, q, n_new)
    check(kv, q, n_new, lens, out, lse)
    assert kv.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,block", [(64, 64), (128, 128)])
def test_decodes_and_chunks_in_one_batch(dtype, d, block):
    """Single tokens, drafts and chunks of several tiles side by side, so that units of one
    tile and of two follow one another within a thread block."""
    lens = [5000, 9000, 300, 4000, 1, 777, 2500, 90]
    n_new = [1, 200, 40, 33, 1, 129, 0, 65]
    kv, q = build(31, lens, 200, 8, 2, d, block, dtype)
    out, lse = run(kv, q, n_new)
    check(kv, q, n_new, lens, out, lse)
    assert kv.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_short_sequences(dtype):
    """More sequences than SMs, several whole ones a thread block."""
    lens = [1 + (37 * i) % 200 for i in range(180)]
    n_new = [min(n, 1 + i % 4) for i, n in enumerate(lens)]
    kv, q = build(8, lens, 4, 4, 2, 64, 64, dtype)
    out, lse = run(kv, q, n_new)
    check(kv, q, n_new, lens, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_new", [5, 200])
def test_large_logits_move_the_maximum(dtype, n_new):
    """Keys that grow along the sequence: the running maximum rises in almost every tile, by
    far more than a few powers of two."""
    L = 900
    kv, q = build(9, [L], n_new, 4, 1, 128, 64, dtype)
    ramp = torch.linspace(0.1, 12, L, device="cuda")
    for i, page in enumerate(kv.block_table[0].long()):
        kv.k_pool[page, :, :] *= torch.nn.functional.pad(ramp, (0, 64))[i * 64:(i + 1) * 64, None].to(q.dtype)
    q.mul_(3)
    out, lse = run(kv, q, [n_new])
    check(kv, q, [n_new], [L], out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 4])
def test_values_after_a_query_have_no_part_in_it(dtype, G):
    """Infinities and NaN among the chunk's own keys and values: rows before them are as if
    they were not there, rows from them on have them."""
    L, n = 330, 290
    kv, q = build(10, [L], n, G, 1, 64, 64, dtype)

    def put(pool, s, i, x):
        pool[kv.block_table[0, s // 64].long(), 0, s % 64, i] = x

    put(kv.v_pool, 150, 3, INF)
    put(kv.v_pool, 200, 3, -INF)
    put(kv.v_pool, 201, 9, -INF)
    put(kv.v_pool, 300, 10, NAN)
    put(kv.v_pool, 329, 11, INF)
    out, lse = run(kv, q, [n])
    check(kv, q, [n], [L], out, lse)
    # a NaN key: its own and later rows are NaN, the rows before it are not
    kv, q = build(11, [L], n, G, 1, 64, 64, dtype)
    put(kv.k_pool, 250, 5, NAN)
    out, lse = run(kv, q, [n])
    first = 250 - (L - n)
    assert torch.isfinite(out[0, :first]).all() and torch.isfinite(lse[0, :first]).all()
    assert torch.isnan(out[0, first:]).all() and torch.isnan(lse[0, first:]).all()
    put(kv.k_pool, 250, 5, 0.0)
    want, wz = run(kv, q, [n])
    assert torch.equal(out[0, :first], want[0, :first]) and torch.equal(lse[0, :first], wz[0, :first])


def test_softmax_scale_and_own_lengths():
    lens = [500, 90]
    kv, q = build(12, lens, 20, 4, 1, 128, 64, "bf16")
    kv.params.softmax_scale = 0.3
    kv.cfg.softmax_scale = 0.3
    # the first 400 and 70 tokens only, by lengths of the call's own
    cut = torch.tensor([400, 70], dtype=torch.int32, device="cuda")
    out, lse = run(kv, q, [20, 7], lens=cut)
    check(kv, q, [20, 7], [400, 70], out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_sequences_are_flagged_and_left(dtype):
    lens = [200, 130, 100, 90, 64]
    kv, q = build(13, lens, 8, 4, 1, 64, 64, dtype)
    kv.context_lens.copy_(torch.tensor([200, 64 * kv.c.max_blocks_per_seq + 1, 100, 5, 64]))
    out, lse = run(kv, q, [8, 8, 9, 6, -1])
    assert kv.status() == _lib.SPLA_DEV_CAPACITY | _lib.SPLA_DEV_BAD_COUNT
    check(kv, q, [8, 0, 0, 0, 0], [200, 0, 0, 0, 0], out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [3, 120])
def test_bad_table_entries_count_as_zero_tokens(dtype, n):
    lens = [260, 400]
    kv, q = build(14, lens, n, 4, 1, 64, 64, dtype)
    kv.block_table[0, 1] = -1
    kv.block_table[1, 6] = kv.num_phys_blocks
    out, lse = run(kv, q, [n, n])
    assert kv.status() == _lib.SPLA_DEV_BAD_BLOCK_TABLE
    check(kv, q, [n, n], lens, out, lse)


@pytest.mark.parametrize("n", [2, 140])
def test_pool_past_32_bits_of_elements(n):
    """Pages whose elements lie past 2^31."""
    hkv, d, block, L = 8, 128, 128, 500
    phys = 2 ** 31 // (hkv * d * block) + 6
    cfg = SplaConfig(num_q_heads=8, num_kv_heads=hkv, head_dim=d, block_size=block, top_k=1)
    kp = torch.full((phys, hkv, block, d), NAN, device="cuda", dtype=torch.bfloat16)
    vp = torch.full_like(kp, NAN)
    kp[-4:] = torch.randn((4, hkv, block, d), device="cuda").bfloat16()
    vp[-4:] = torch.randn((4, hkv, block, d), device="cuda").bfloat16()
    table = torch.arange(phys - 1, phys - 5, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    kv = SplaPagedKV(cfg, kp, vp, table, torch.tensor([L], dtype=torch.int32, device="cuda"))
    q = torch.randn((1, n, 8, d), device="cuda").bfloat16()
    out, lse = run(kv, q, [n])
    check(kv, q, [n], [L], out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_repeats_are_the_same_bits_and_without_lse(dtype):
    lens = [5000, 77, 1300]
    kv, q = build(15, lens, 70, 8, 2, 128, 64, dtype)
    a, az = run(kv, q, [70, 70, 12])
    b, bz = run(kv, q, [70, 70, 12])
    assert torch.equal(a, b) and torch.equal(az, bz)
    n = torch.tensor([70, 70, 12], dtype=torch.int32, device="cuda")
    c = kv.chunk_attention(q, n)
    assert torch.equal(c[0], a[0]) and (c[2, 12:] == 0).all()


def test_captured_call_follows_lengths_counts_and_queries():
    """One graph, replayed after the lengths, counts and queries in its buffers changed, with
    larger eager calls of the same cache between."""
    lens = [900, 2000]
    kv, q = build(16, lens, 6, 8, 2, 128, 64, "bf16")
    n = torch.tensor([6, 1], dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(q, 5.0), torch.full(q.shape[:3], 5.0, device="cuda")
    kv.chunk_attention(q, n, out=out, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.chunk_attention(q, n, out=out, lse=lse)
    for new_lens, counts in (([900, 2000], [6, 1]), ([3, 1999], [2, 6]), ([900, 0], [0, 0])):
        kv.context_lens.copy_(torch.tensor(new_lens, dtype=torch.int32))
        n.copy_(torch.tensor(counts, dtype=torch.int32))
        q.copy_(torch.randn(q.shape, device="cuda"))
        out.fill_(5.0)
        lse.fill_(5.0)
        big = torch.randn((2, 300, 8, 128), device="cuda").bfloat16()
        kv.chunk_attention(big, torch.zeros_like(n))
        graph.replay()
        check(kv, q, counts, new_lens, out, lse)


def test_two_caches_on_two_streams():
    sets = [build(20 + i, [3000 + i, 700], 40, 8, 2, 128, 64, "bf16") for i in range(2)]
    n = torch.tensor([40, 40], dtype=torch.int32, device="cuda")
    want = [kv.chunk_attention(q, n) for kv, q in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[kv.chunk_attention(q, n, stream=s) for _ in range(5)]
           for (kv, q), s in zip(sets, streams)]
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        for g in many:
            assert torch.equal(g, w)


def test_one_token_of_a_sparse_cache_with_every_block_kept():
    """On a SplaDecodeCache, one token's chunk attention is the sparse branch of a decode that
    keeps every block."""
    torch.manual_seed(3)
    batch, hq, hkv, d, block, L = 2, 8, 2, 128, 64, 300
    cfg = SplaConfig(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=block, top_k=8)
    table = torch.randperm(10, dtype=torch.int32).view(2, 5)
    cache = SplaDecodeCache(cfg, batch, table, 10)
    k, v = (torch.randn((batch, L, hkv, d), device="cuda").bfloat16() for _ in range(2))
    cache.append(k, v)
    q = torch.randn((batch, hq, d), device="cuda").bfloat16()
    out, sel, osp, orl = cache.new_outputs()
    cache.decode(q, None, out, sel, osp, orl)
    one = torch.ones(batch, dtype=torch.int32, device="cuda")
    got = cache.chunk_attention(q.view(batch, 1, hq, d), one)[:, 0]
    # both are within their own bounds of the same numbers: twice the bound apart at most
    for b in range(batch):
        for e in range(hq):
            K, V = (ref.tokens(p, cache.block_table[b], L, e // 4) for p in (cache.k_pool, cache.v_pool))
            o, _, to, _ = ref.chunk(q[b, e][None].double(), K, V, L, 1 / math.sqrt(d), torch.bfloat16)
            assert ((got[b, e].double() - o[0]).abs() <= to[0]).all()
            assert ((osp[b, e].double() - got[b, e].double()).abs() <= 2 * to[0]).all()
    assert cache.status() == 0
