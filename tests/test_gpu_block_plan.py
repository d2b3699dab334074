"""spla_block_plan and spla_block_release against the sequence-by-sequence form, equal in
every entry."""
import numpy as np
import pytest
import torch

from block_sparse_linear_b200 import SplaBlockPool, _lib

from . import paged_ref as ref

pytestmark = pytest.mark.gpu


def dev(a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a)).to(device="cuda", dtype=dtype)


def make(rng, lens, block, mbp, spare):
    """A pool whose sequences hold `lens` tokens in random blocks, `spare` blocks free."""
    lens = np.asarray(lens, np.int32)
    nb = np.clip(-(-lens // block), 0, mbp)
    phys = int(nb.sum()) + spare
    perm = rng.permutation(phys).astype(np.int32)
    table = np.full((len(lens), mbp), -1, np.int32)
    at = 0
    for b, k in enumerate(nb):
        table[b, :k] = perm[at:at + k]
        at += k
    free = np.full(phys, -7, np.int32)
    free[:spare] = perm[at:]
    return table, free, np.array([spare], np.int32)


def check_plan(table, free, count, block, lens, n_new, max_new, commit=True):
    want = ref.plan(table, free, count[0], block, np.asarray(lens), np.asarray(n_new), max_new)
    pool = SplaBlockPool(dev(table), dev(free), dev(count), block)
    got = pool.plan(dev(lens), dev(n_new), max_new, commit=commit)
    assert pool.status() == want["status"]
    for k in ("n_granted", "lens_after", "positions", "slots"):
        np.testing.assert_array_equal(getattr(got, k).cpu().numpy(), want[k], err_msg=k)
    np.testing.assert_array_equal(pool.block_table.cpu().numpy(), want["block_table"])
    assert int(got.free_count) == want["free_count"]
    assert int(pool.free_count) == (want["free_count"] if commit else count[0])
    return pool, want


@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("batch,max_new", [(1, 1), (3, 1), (7, 130), (40, 1000), (300, 5),
                                           (1025, 3), (2100, 65)])
def test_plan_matches_plain_form(block, batch, max_new):
    rng = np.random.default_rng(batch + max_new + block)
    lens = rng.integers(0, 6 * block, batch)
    lens[::3] = lens[::3] // block * block                 # whole blocks: the next token opens one
    n = rng.integers(0, max_new + 1, batch)
    n[-1] = max_new
    mbp = int(max(-(-(lens + n) // block)))
    need = int((-(-(lens + n) // block) - -(-lens // block)).sum())
    for spare in {need, max(need - 1, 0), need // 2, 0, need + 9}:
        check_plan(*make(rng, lens, block, mbp, max(spare, 1)), block, lens, n, max_new)


def test_refused_requests_are_not_overtaken():
    lens, n = [0, 0, 10, 64], [65, 65, 3, 1]               # need 2, 2, 1 held already: 0, 1
    rng = np.random.default_rng(0)
    pool, want = check_plan(*make(rng, lens, 64, 4, 3), 64, lens, n, 65)
    assert want["n_granted"].tolist() == [65, 0, 3, 0] and want["status"] == _lib.SPLA_DEV_NO_BLOCKS


def test_bad_counts_and_lengths_are_flagged_and_granted_nothing():
    rng = np.random.default_rng(1)
    lens = [5, 5, -3, 300, 250, 7]
    table, free, count = make(rng, [5, 5, 0, 256, 250, 7], 64, 4, 9)
    check_plan(table, free, count, 64, lens, [4, -1, 2, 0, 7, 9], 8)


def test_free_count_outside_the_pool_counts_as_none():
    rng = np.random.default_rng(2)
    table, free, _ = make(rng, [5, 64], 64, 4, 6)
    for bad in (len(free) + 1, -1):
        check_plan(table, free, np.array([bad], np.int32), 64, [5, 64], [1, 1], 8)


def test_entry_outside_the_pool_gives_no_slot():
    rng = np.random.default_rng(3)
    table, free, count = make(rng, [70, 70], 64, 4, 6)
    table[1, 1] = 10 ** 6
    check_plan(table, free, count, 64, [70, 70], [3, 3], 3)


def test_look_ahead_leaves_the_blocks_and_repeats():
    rng = np.random.default_rng(4)
    lens, n = [0, 63, 64, 200], [64, 2, 1, 0]
    table, free, count = make(rng, lens, 64, 6, 12)
    pool, want = check_plan(table, free, count, 64, lens, n, 64, commit=False)
    again = pool.plan(dev(lens), dev(n), 64)
    np.testing.assert_array_equal(again.slots.cpu().numpy(), want["slots"])
    assert int(pool.free_count) == want["free_count"]


def test_without_rows_and_in_place_counts():
    rng = np.random.default_rng(5)
    lens, n = np.array([0, 63, 64], np.int32), np.array([64, 2, 1], np.int32)
    table, free, count = make(rng, lens, 64, 6, 2)
    want = ref.plan(table, free, 2, 64, lens, n, 64)
    pool = SplaBlockPool(dev(table), dev(free), dev(count), 64)
    d_lens, d_n = dev(lens), dev(n)
    p = pool.plan(d_lens, d_n, 64, rows=False, commit=False)
    assert p.positions is None and p.slots is None
    # n_granted over n_new
    _lib.spla_block_plan(pool.c, d_lens.data_ptr(), d_n.data_ptr(), 64, d_n.data_ptr(), 0, 0, 0,
                         pool.free_count.data_ptr(), 0, torch.cuda.current_stream().cuda_stream)
    np.testing.assert_array_equal(d_n.cpu().numpy(), want["n_granted"])
    assert int(pool.free_count) == want["free_count"]


@pytest.mark.parametrize("batch", [1, 5, 1500])
def test_release_gives_back_what_plan_took(batch):
    block, mbp = 64, 12
    rng = np.random.default_rng(batch)
    pool = SplaBlockPool.empty(batch, mbp, batch * mbp, block)
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    for _ in range(4):
        room = mbp * block - lens.cpu().numpy()
        n = rng.integers(0, np.minimum(room, 300) + 1)
        p = pool.plan(lens, dev(n), 300)
        lens = p.lens_after.clone()
        L = lens.cpu().numpy()
        keep = np.where(rng.random(batch) < 0.3, 0, rng.integers(0, L + 20))
        before, table = int(pool.free_count), pool.block_table.cpu().numpy()
        pool.release(dev(keep), lens)
        after = np.minimum(keep, L)
        np.testing.assert_array_equal(lens.cpu().numpy(), after)
        back = []
        for b in range(batch):
            back += table[b, -(-after[b] // block):-(-L[b] // block)].tolist()
        assert int(pool.free_count) == before + len(back)
        stack = pool.free_list.cpu().numpy()
        np.testing.assert_array_equal(stack[before:before + len(back)], back)
        # every block is held or free, once
        t = pool.block_table.cpu().numpy()
        held = t[t >= 0]
        everyone = np.concatenate([held, stack[:int(pool.free_count)]])
        np.testing.assert_array_equal(np.sort(everyone), np.arange(batch * mbp))
        assert all((t[b, -(-after[b] // block):] == -1).all() for b in range(batch))
    assert pool.status() == 0


def test_release_refuses_bad_sequences_alone():
    rng = np.random.default_rng(6)
    lens = np.array([130, 130, 130, 5], np.int32)
    table, free, count = make(rng, lens, 64, 4, 3)
    table[1, 2] = -1                                        # its last block is not one
    pool = SplaBlockPool(dev(table), dev(free), dev(count), 64)
    d = dev(lens)
    pool.release(dev([0, 0, -1, 0]), d)
    assert pool.status() == _lib.SPLA_DEV_BAD_BLOCK_TABLE | _lib.SPLA_DEV_BAD_COUNT
    assert d.tolist() == [0, 130, 130, 0] and int(pool.free_count) == 3 + 3 + 1
    np.testing.assert_array_equal(pool.block_table[1].cpu().numpy(), table[1])
    # a stack that would grow past the pool: blocks given back twice
    pool.dev_status.zero_()
    pool.block_table.copy_(dev(table))
    pool.block_table[1] = pool.block_table[2]
    pool.free_count.fill_(len(free) - 2)
    d.copy_(dev([0, 130, 130, 0]))
    pool.release(dev([0, 0, 0, 0]), d)
    assert pool.status() == _lib.SPLA_DEV_CAPACITY
    assert d.tolist() == [0, 130, 130, 0] and int(pool.free_count) == len(free) - 2


def test_named_stream_and_replayed_graph():
    """plan and release on a stream of their own, and captured: every replay takes the next
    blocks and follows the lengths in place."""
    batch, mbp, block = 5, 6, 64
    side = torch.cuda.Stream()
    pool = SplaBlockPool.empty(batch, mbp, batch * mbp, block)
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    n = dev([64, 1, 0, 63, 65])
    torch.cuda.synchronize()
    want = ref.plan(pool.block_table.cpu().numpy(), pool.free_list.cpu().numpy(), batch * mbp, block,
                    lens.cpu().numpy(), n.cpu().numpy(), 65)
    p = pool.plan(lens, n, 65, stream=side)
    side.synchronize()
    for key in ("n_granted", "lens_after", "positions", "slots"):
        np.testing.assert_array_equal(getattr(p, key).cpu().numpy(), want[key])
    pool.release(torch.zeros_like(lens), p.lens_after, stream=side)
    side.synchronize()
    assert int(pool.free_count) == batch * mbp and (p.lens_after == 0).all()
    one = torch.full((batch,), 40, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        p = pool.plan(lens, one, 40)
        lens.copy_(p.lens_after)
    torch.cuda.synchronize()
    table, free, top = pool.block_table.cpu().numpy(), pool.free_list.cpu().numpy(), batch * mbp
    L = np.zeros(batch, np.int32)
    for _ in range(10):                                     # 400 tokens: more than the table holds
        want = ref.plan(table, free, top, block, L, np.full(batch, 40), 40)
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(p.slots.cpu().numpy(), want["slots"])
        np.testing.assert_array_equal(lens.cpu().numpy(), want["lens_after"])
        table, top, L = want["block_table"], want["free_count"], want["lens_after"]
        assert int(pool.free_count) == top
    assert pool.status() == _lib.SPLA_DEV_CAPACITY
