"""Block planning and release at their limits, and the paged calls on several streams."""
import numpy as np
import pytest
import torch

from block_sparse_linear_b200 import SplaBlockPool, SplaConfig, SplaDecodeCache, _lib

from .test_gpu_block_plan import dev, make
from .test_gpu_chunk_attention import build

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("at", [3, 1000, 1023, 1024, 2047])
def test_release_past_the_pool_leaves_every_later_sequence(at):
    """Blocks given back twice: the first sequence that would push the stack past the pool, and
    every later one that gives blocks back, stays as it is, however many sequences there are."""
    batch, block = 2100, 64
    rng = np.random.default_rng(at)
    lens = np.full(batch, 60, np.int32)
    lens[at] = 4 * block
    table, free, count = make(rng, lens, block, 4, 5)
    # what the sequences before `at` give back, and then room for two blocks more
    count[0] = len(free) - at - 2
    pool = SplaBlockPool(dev(table), dev(free), dev(count), block)
    d = dev(lens)
    keep = np.zeros(batch, np.int32)
    keep[-1] = 10                                      # gives no block back
    pool.release(dev(keep), d)
    want = lens.copy()
    want[:at] = 0
    want[-1] = 10
    np.testing.assert_array_equal(d.cpu().numpy(), want)
    assert pool.status() == _lib.SPLA_DEV_CAPACITY
    assert int(pool.free_count) == len(free) - 2
    t = pool.block_table.cpu().numpy()
    np.testing.assert_array_equal(t[at:], table[at:])
    assert (t[:at] == -1).all()
    np.testing.assert_array_equal(pool.free_list.cpu().numpy()[count[0]:count[0] + at], table[:at, 0])


def test_bulk_append_takes_the_counts_of_the_plan_before_it():
    """A plan and the bulk append that reads its counts, back to back: whatever the buffer held
    before, the append sees what the plan granted, and the state and pages are those of an append
    with counts that were there from the start."""
    cfg = SplaConfig(num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=64, top_k=4)
    batch, mbp, max_new = 3, 40, 600
    rng = np.random.default_rng(8)
    g = torch.Generator("cuda").manual_seed(8)
    pool = SplaBlockPool.empty(batch, mbp, batch * mbp, 64)
    caches = [SplaDecodeCache(cfg, batch, pool.block_table, batch * mbp) for _ in range(2)]
    for c in caches:
        c.k_pool.zero_()
        c.v_pool.zero_()
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    after, granted = torch.zeros_like(lens), torch.zeros_like(lens)
    stream = torch.cuda.current_stream().cuda_stream
    for step in range(12):
        n = dev(rng.integers(1, 200, batch) if step else [max_new, 1, 300])
        k, v = (torch.randn((batch, max_new, 2, 128), device="cuda", generator=g).bfloat16()
                for _ in "kv")
        granted.fill_((0, max_new, max_new + 1)[step % 3])
        torch.cuda.synchronize()
        _lib.spla_block_plan(pool.c, lens.data_ptr(), n.data_ptr(), max_new, granted.data_ptr(),
                             after.data_ptr(), 0, 0, pool.free_count.data_ptr(),
                             pool.dev_status.data_ptr(), stream)
        caches[1].append(k, v, granted, bulk=True)
        lens.copy_(after)
        torch.cuda.synchronize()
        caches[0].append(k, v, n, bulk=True)
        for name in ("k_pool", "v_pool", "blk_stats", "S", "z", "m", "context_lens"):
            assert torch.equal(getattr(caches[0], name), getattr(caches[1], name)), (step, name)
        assert torch.equal(caches[1].context_lens, lens)
    assert pool.status() == 0 and [c.status() for c in caches] == [0, 0]


def test_plan_of_the_widest_rows():
    """max_new up to 2^31 - 1 (batch 1): the row tiles are counted past 32 bits."""
    max_new = 2 ** 31 - 1
    pool = SplaBlockPool.empty(1, 8, 8, 64)
    lens, n = dev([5]), dev([300])
    granted, after = torch.zeros_like(n), torch.zeros_like(n)
    pos = torch.full((max_new,), 7, dtype=torch.int32, device="cuda")
    _lib.spla_block_plan(pool.c, lens.data_ptr(), n.data_ptr(), max_new, granted.data_ptr(),
                         after.data_ptr(), pos.data_ptr(), 0, pool.free_count.data_ptr(),
                         pool.dev_status.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert granted.tolist() == [300] and after.tolist() == [305] and pool.status() == 0
    assert torch.equal(pos[:300], torch.arange(5, 305, dtype=torch.int32, device="cuda"))
    assert int(pos[300:].max()) == int(pos[300:].min()) == -1


def test_workspace_outlives_its_object_on_every_stream_it_was_used_on():
    """The workspace a first call made on one stream, used on another: when the object goes while
    that stream is still busy, nobody else gets the memory."""
    kv, q = build(50, [3000], 4, 8, 2, 128, 64, "bf16")
    n = dev([4])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = kv.chunk_attention(q, n, stream=side)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                     # 0.1 s of clocks on the current stream
    got = kv.chunk_attention(q, n)
    ws, size = kv._chunk_ws.data_ptr(), kv._chunk_ws.numel()
    del kv
    with torch.cuda.stream(side):
        others = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
    assert not torch.cuda.current_stream().query()     # the call is still to come
    assert all(ws not in range(t.data_ptr(), t.data_ptr() + size) for t in others)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
