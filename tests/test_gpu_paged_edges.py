"""Block planning and release at their limits, and the paged calls on several streams."""
import numpy as np
import pytest
import torch

from block_sparse_linear_b200 import SplaBlockPool, _lib

from .test_gpu_block_plan import dev, make

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
