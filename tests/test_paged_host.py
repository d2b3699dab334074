"""The paged serving calls reject bad arguments on the host, before any CUDA call: the C
entry points with addresses that are never dereferenced, the Python ones with CPU tensors."""
import ctypes

import pytest
import torch

from block_sparse_linear_b200 import (SplaBlockPool, SplaConfig, SplaPagedKV, _lib, qk_norm_rope)

from .test_abi_host import FAKE, _cache, _params

B = ctypes.byref
INVALID, UNSUPPORTED, WORKSPACE, CAPACITY = (_lib.SPLA_ERR_INVALID_ARG, _lib.SPLA_ERR_UNSUPPORTED,
                                             _lib.SPLA_ERR_WORKSPACE, _lib.SPLA_ERR_CAPACITY)


def _pool(**kw):
    base = dict(block_table=FAKE, free_list=FAKE, free_count=FAKE, batch=4, max_blocks_per_seq=100,
                num_phys_blocks=500, block_size=64)
    base.update(kw)
    return _lib.spla_block_pool(**base)


PLAN = dict(context_lens=FAKE, n_new=2 * FAKE, max_new=8, n_granted=3 * FAKE, lens_after=4 * FAKE,
            positions=5 * FAKE, slots=6 * FAKE, free_out=FAKE)


@pytest.mark.parametrize("pool,args,code", [
    (dict(block_table=None), {}, INVALID), (dict(free_list=None), {}, INVALID),
    (dict(free_count=None), {}, INVALID), (dict(batch=0), {}, INVALID),
    (dict(max_blocks_per_seq=0), {}, INVALID), (dict(num_phys_blocks=0), {}, INVALID),
    (dict(block_size=32), {}, UNSUPPORTED),
    (dict(batch=_lib.SPLA_MAX_PLAN_BATCH + 1), {}, CAPACITY),
    (dict(max_blocks_per_seq=_lib.SPLA_MAX_BLOCKS_PER_SEQ + 1), {}, CAPACITY),
    ({}, dict(context_lens=None), INVALID), ({}, dict(n_new=None), INVALID),
    ({}, dict(n_granted=None), INVALID), ({}, dict(free_out=None), INVALID),
    ({}, dict(max_new=-1), INVALID), ({}, dict(lens_after=FAKE), INVALID),
    ({}, dict(n_granted=FAKE), INVALID), ({}, dict(max_new=2 ** 30), CAPACITY),
])
def test_plan_refuses(lib, pool, args, code):
    a = {**PLAN, **args}
    assert lib.spla_block_plan(B(_pool(**pool)), *a.values(), None, None) == code


def test_release_refuses(lib):
    assert lib.spla_block_release(B(_pool(batch=-1)), FAKE, 2 * FAKE, None, None) == INVALID
    assert lib.spla_block_release(B(_pool()), None, FAKE, None, None) == INVALID
    assert lib.spla_block_release(B(_pool()), FAKE, None, None, None) == INVALID
    assert lib.spla_block_release(B(_pool()), FAKE, FAKE, None, None) == INVALID


BIG = 1 << 40                                   # outputs far from the inputs
ROPE = dict(q=FAKE, q_stride=6144, k=FAKE + 8192, k_stride=6144, v=FAKE + 10240, v_stride=6144,
            rows=10, positions=FAKE, inv_freq=FAKE, rot_dim=128, interleaved=0, q_gamma=None,
            k_gamma=None, eps=1e-6, q_out=BIG, k_out=2 * BIG, v_out=3 * BIG, slots=None,
            num_phys_blocks=0)


@pytest.mark.parametrize("args,code", [
    (dict(rows=-1), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(positions=None), INVALID), (dict(inv_freq=None), INVALID), (dict(q_out=None), INVALID),
    (dict(k_out=None), INVALID), (dict(v_out=None), INVALID),
    (dict(rot_dim=-16), INVALID), (dict(rot_dim=144), UNSUPPORTED), (dict(rot_dim=24), UNSUPPORTED),
    (dict(q_stride=4095), INVALID), (dict(q_stride=6148), INVALID), (dict(k_stride=1000), INVALID),
    (dict(v_stride=6145), INVALID), (dict(q=FAKE + 2), INVALID), (dict(k_out=2 * BIG + 8), INVALID),
    (dict(slots=FAKE), INVALID),                                  # no pool size
    (dict(rows=1 << 32), CAPACITY), (dict(q_stride=1 << 32), CAPACITY),
    (dict(q_out=FAKE + 16), INVALID),                             # over its own inputs
    (dict(k_out=BIG + 1024), INVALID),                            # over q_out
    (dict(slots=FAKE, num_phys_blocks=64, v_out=2 * BIG + 4096), INVALID),   # the two pools
])
def test_norm_rope_refuses(lib, args, code):
    a = {**ROPE, **args}
    assert lib.spla_qk_norm_rope(B(_params()), *a.values(), None, None) == code


def test_norm_rope_refuses_params_and_takes_no_rows(lib):
    assert lib.spla_qk_norm_rope(B(_params(head_dim=96)), *ROPE.values(), None, None) == UNSUPPORTED
    assert lib.spla_qk_norm_rope(None, *ROPE.values(), None, None) == INVALID
    a = {**ROPE, "rows": 0, "q": None}
    assert lib.spla_qk_norm_rope(B(_params()), *a.values(), None, None) == _lib.SPLA_OK


CHUNK = dict(q=FAKE, n_new=FAKE, max_new=8, out=BIG, lse=None, workspace=FAKE, workspace_bytes=BIG)


@pytest.mark.parametrize("cache,args,code", [
    (dict(k_pool=None), {}, INVALID), (dict(v_pool=None), {}, INVALID),
    (dict(block_table=None), {}, INVALID), (dict(context_lens=None), {}, INVALID),
    (dict(batch=0), {}, INVALID), (dict(max_blocks_per_seq=0), {}, INVALID),
    (dict(num_phys_blocks=0), {}, INVALID),
    (dict(max_blocks_per_seq=_lib.SPLA_MAX_BLOCKS_PER_SEQ + 1), {}, CAPACITY),
    (dict(num_phys_blocks=2 ** 23), {}, CAPACITY),
    (dict(k_pool=FAKE + 8), {}, INVALID), (dict(v_pool=FAKE + 2), {}, INVALID),
    ({}, dict(q=None), INVALID), ({}, dict(out=None), INVALID), ({}, dict(n_new=None), INVALID),
    ({}, dict(max_new=-1), INVALID), ({}, dict(q=FAKE + 4), INVALID),
    ({}, dict(out=BIG + 2), INVALID), ({}, dict(out=FAKE + 64), INVALID),
    ({}, dict(max_new=2 ** 28), CAPACITY), (dict(batch=2 ** 22 + 1), dict(max_new=1), CAPACITY),
    ({}, dict(workspace=None), WORKSPACE), ({}, dict(workspace=FAKE + 16), WORKSPACE),
    ({}, dict(workspace_bytes=0), WORKSPACE),
])
def test_chunk_attention_refuses(lib, cache, args, code):
    a = {**CHUNK, **args}
    assert lib.spla_chunk_attention(B(_params()), B(_cache(**cache)), *a.values(), None, None) == code


def test_chunk_attention_needs_no_state_and_takes_no_tokens(lib):
    c = _cache(blk_stats=None, S=None, z=None, m=None)
    a = {**CHUNK, "max_new": 0, "q": None}
    assert lib.spla_chunk_attention(B(_params()), B(c), *a.values(), None, None) == _lib.SPLA_OK
    a = {**CHUNK, "workspace": None}
    assert lib.spla_chunk_attention(B(_params()), B(c), *a.values(), None, None) == WORKSPACE


def test_chunk_workspace_size(lib):
    for d in (64, 128):
        for dtype in (_lib.SPLA_BF16, _lib.SPLA_F32):
            p = _params(head_dim=d, dtype=dtype)
            sizes = {_lib.spla_chunk_attention_workspace_size(p, b, n)
                     for b, n in ((1, 1), (64, 1), (1, 4096), (300, 70))}
            assert len(sizes) == 1 and sizes.pop() > 0     # one size: callers keep one workspace
    n = ctypes.c_size_t()
    assert lib.spla_chunk_attention_workspace_size(B(_params()), 0, 1, B(n)) == INVALID
    assert lib.spla_chunk_attention_workspace_size(B(_params()), 1, 1, None) == INVALID


def _cfg(**kw):
    base = dict(num_q_heads=4, num_kv_heads=1, head_dim=64, block_size=64, top_k=1)
    return SplaConfig(**{**base, **kw})


def _kv(cfg=None, batch=2):
    cfg = cfg or _cfg()
    shape = (5, cfg.num_kv_heads, cfg.block_size, cfg.head_dim)
    return SplaPagedKV(cfg, torch.zeros(shape, dtype=cfg.torch_dtype),
                       torch.zeros(shape, dtype=cfg.torch_dtype),
                       torch.zeros((batch, 3), dtype=torch.int32),
                       torch.zeros(batch, dtype=torch.int32))


def test_python_calls_check_types_shapes_and_layout():
    kv = _kv()
    q = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16)
    n = torch.zeros(2, dtype=torch.int32)
    for bad_q, bad_n in ((q.float(), n), (q[:, :, :2], n), (q[0], n), (q, n.long()), (q, n[:1]),
                         (q.transpose(1, 2), n)):
        with pytest.raises(ValueError):
            kv.chunk_attention(bad_q, bad_n)
    with pytest.raises(ValueError):
        kv.chunk_attention(q, n, lse=torch.zeros((2, 3, 4), dtype=torch.float64))
    with pytest.raises(ValueError):
        kv.chunk_attention(q, n, lens=n.long())
    cfg = _cfg()
    rows = torch.zeros((6, 4, 64), dtype=torch.bfloat16)
    one = torch.zeros((6, 1, 64), dtype=torch.bfloat16)
    pos = torch.zeros(6, dtype=torch.int32)
    for args in ((rows[:, :3], one, one, pos), (rows, one[:5], one, pos), (rows, one, one[:5], pos),
                 (rows, one, one, pos.long()), (rows, one, one, pos[:3]),
                 (rows.float(), one, one, pos), (rows.transpose(0, 1), one, one, pos)):
        with pytest.raises(ValueError):
            qk_norm_rope(cfg, *args)
    with pytest.raises(ValueError):
        qk_norm_rope(cfg, rows, one, one, pos, inv_freq=torch.zeros(32))          # not float64
    with pytest.raises(ValueError):
        qk_norm_rope(cfg, rows, one, one, pos, q_gamma=torch.zeros(63))
    with pytest.raises(ValueError):
        SplaPagedKV(cfg, kv.k_pool.float(), kv.v_pool)
    with pytest.raises(ValueError):
        SplaPagedKV(cfg, kv.k_pool[:, :, :32], kv.v_pool)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ValueError):
        SplaBlockPool(i(2, 3), i(5).long(), i(1), 64)
    with pytest.raises(ValueError):
        SplaBlockPool(i(2, 3), i(5), i(2), 64)
    with pytest.raises(ValueError):
        SplaBlockPool(i(6), i(5), i(1), 64)
    pool = SplaBlockPool(i(2, 3), i(5), i(1), 64)
    with pytest.raises(ValueError):
        pool.plan(i(3), i(2), 1)
    with pytest.raises(ValueError):
        pool.plan(i(2), i(2).long(), 1)
    with pytest.raises(ValueError):
        pool.release(i(1), i(2))
