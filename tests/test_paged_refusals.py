"""What the paged serving calls refuse beside bad types and shapes, on the host."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

from block_sparse_linear_b200 import SplaDecodeCache, paged, qk_norm_rope

from .test_paged_host import INVALID, PLAN, _cfg, _kv, _pool


def test_norm_rope_writes_no_pages_of_a_sparse_cache():
    """A SplaDecodeCache's pages go with statistics and a state that a write by slot would leave
    behind: refused before anything is launched."""
    kv, cfg = _kv(), _cfg()
    cache = SplaDecodeCache.__new__(SplaDecodeCache)      # no device here: the attributes it has
    cache.__dict__.update(cfg=cfg, k_pool=kv.k_pool, v_pool=kv.v_pool, num_phys_blocks=5,
                          dev_status=torch.zeros(1, dtype=torch.int32))
    rows = torch.zeros((6, 4, 64), dtype=torch.bfloat16)
    one = torch.zeros((6, 1, 64), dtype=torch.bfloat16)
    pos, slots = torch.zeros(6, dtype=torch.int32), torch.arange(6)
    with pytest.raises(ValueError, match="SplaPagedKV"):
        qk_norm_rope(cfg, rows, one, one, pos, kv=cache, slots=slots)


def test_a_stream_of_another_device_is_refused():
    """It cannot run work on these tensors; the call does not go to some other stream instead."""
    here, other = torch.device("cuda", 0), torch.device("cuda", 1)
    with pytest.raises(ValueError, match="stream"):
        paged._at(here, SimpleNamespace(device=other))


def test_plan_refuses_one_buffer_for_counts_and_lengths(lib):
    """n_granted and lens_after in one buffer: the rows would follow the wrong one of them."""
    a = {**PLAN, "lens_after": PLAN["n_granted"]}
    assert lib.spla_block_plan(ctypes.byref(_pool()), *a.values(), None, None) == INVALID
