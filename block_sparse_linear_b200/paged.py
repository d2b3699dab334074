"""Paged serving around the decode cache: block tables grown on the device
(``SplaBlockPool``), q/k norm with rotation in one pass (``qk_norm_rope``), and exact
chunk attention over paged K and V (``SplaPagedKV``, and ``chunk_attention`` of
``SplaDecodeCache``). Arguments are checked and marshalled here; all work runs in the
library's kernels, on the stream given or the current one of the tensors' device.

One serving step of a model whose layers share a block table:

    plan = pool.plan(lens, n_new, max_new)                  # blocks, positions, slots
    # a layer of full attention
    q = qk_norm_rope(cfg, q, k, v, plan.positions, inv_freq, kv=kv, slots=plan.slots)
    out = kv.chunk_attention(q.view(batch, max_new, Hq, d), plan.n_granted, lens=plan.lens_after)
    # a sparse layer: rows out, then the append that keeps statistics and state current
    q = qk_norm_rope(cfg, q, k, v, plan.positions, inv_freq, k_out=k_new, v_out=v_new)
    cache.append(k_new, v_new, plan.n_granted)
    out = cache.decode(q)
"""
import contextlib
from collections import namedtuple

import torch

from . import _lib

BlockPlan = namedtuple("BlockPlan", "n_granted lens_after positions slots free_count")

_NO_GUARD = contextlib.nullcontext()


def _on(device):
    """Makes `device` current for the launches of one call, where it is not already."""
    return _NO_GUARD if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _stream(device, stream):
    return (stream if stream is not None else torch.cuda.current_stream(device)).cuda_stream


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _need(t, name, dtype, shape, device):
    """A contiguous tensor of this type and shape on this device, or ValueError."""
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or t.device != device \
            or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} "
                         f"on {device}, got {t.dtype} {tuple(t.shape)} on {t.device}")


class SplaBlockPool:
    """The free blocks of a paged pool and the block table they are handed out through
    (include/spla.h's ``spla_block_pool``), kept on the device.

    block_table: [batch][max_blocks_per_seq] int32; free_list: [num_phys_blocks] int32, a
    stack whose first free_count entries are free; free_count: [1] int32. The table may be
    the one a SplaDecodeCache or SplaPagedKV was made with: both keep the tensor itself."""

    def __init__(self, block_table, free_list, free_count, block_size: int):
        _lib.load()
        dev = block_table.device
        if block_table.dim() != 2 or free_list.dim() != 1:
            raise ValueError("block_table is [batch][max_blocks_per_seq], free_list [num_phys_blocks]")
        _need(block_table, "block_table", torch.int32, block_table.shape, dev)
        _need(free_list, "free_list", torch.int32, free_list.shape, dev)
        _need(free_count, "free_count", torch.int32, (1,), dev)
        self.device = dev
        self.block_table, self.free_list, self.free_count = block_table, free_list, free_count
        self.batch, self.max_blocks_per_seq = map(int, block_table.shape)
        self.num_phys_blocks = int(free_list.shape[0])
        self.block_size = int(block_size)
        self.dev_status = torch.zeros((1,), dtype=torch.int32, device=dev)
        self.c = _lib.spla_block_pool(block_table.data_ptr(), free_list.data_ptr(),
                                      free_count.data_ptr(), self.batch, self.max_blocks_per_seq,
                                      self.num_phys_blocks, self.block_size)

    @classmethod
    def empty(cls, batch: int, max_blocks_per_seq: int, num_phys_blocks: int, block_size: int,
              device="cuda"):
        """A pool all of whose blocks are free (block 0 is handed out first) and a table of
        -1: every sequence starts without tokens."""
        i32 = dict(dtype=torch.int32, device=device)
        return cls(torch.full((batch, max_blocks_per_seq), -1, **i32),
                   torch.arange(num_phys_blocks - 1, -1, -1, **i32),
                   torch.full((1,), num_phys_blocks, **i32), block_size)

    def plan(self, context_lens, n_new, max_new: int, rows: bool = True, commit: bool = True,
             stream=None) -> BlockPlan:
        """Gives every sequence the blocks for its n_new tokens (spla_block_plan). Returns
        n_granted and lens_after [batch], positions and slots [batch][max_new] (None without
        rows) and free_count [1]. commit=False looks ahead: table rows and outputs are written,
        the blocks stay free."""
        dev, b = self.device, self.batch
        _need(context_lens, "context_lens", torch.int32, (b,), dev)
        _need(n_new, "n_new", torch.int32, (b,), dev)
        with _on(dev):
            i32 = dict(dtype=torch.int32, device=dev)
            granted, after = torch.empty((2, b), **i32)
            pos = torch.empty((b, max_new), **i32) if rows else None
            slots = torch.empty((b, max_new), dtype=torch.int64, device=dev) if rows else None
            left = self.free_count if commit else torch.empty((1,), **i32)
            _lib.spla_block_plan(self.c, context_lens.data_ptr(), n_new.data_ptr(), max_new,
                                 granted.data_ptr(), after.data_ptr(), _ptr(pos), _ptr(slots),
                                 left.data_ptr(), self.dev_status.data_ptr(),
                                 _stream(dev, stream))
        return BlockPlan(granted, after, pos, slots, left)

    def release(self, keep_lens, context_lens, stream=None) -> None:
        """Shortens sequences to keep_lens tokens (0: done) and takes their blocks back;
        context_lens is updated in place (spla_block_release)."""
        dev = self.device
        _need(keep_lens, "keep_lens", torch.int32, (self.batch,), dev)
        _need(context_lens, "context_lens", torch.int32, (self.batch,), dev)
        with _on(dev):
            _lib.spla_block_release(self.c, keep_lens.data_ptr(), context_lens.data_ptr(),
                                    self.dev_status.data_ptr(), _stream(dev, stream))

    def status(self) -> int:
        """Device-detected fault bits (synchronises)."""
        return int(self.dev_status.item())


def chunk_attention(owner, q, n_new, out=None, lse=None, lens=None, stream=None):
    """spla_chunk_attention over an owner's cache struct (SplaDecodeCache, SplaPagedKV)."""
    cfg, dev = owner.cfg, owner.k_pool.device
    if q.dim() != 4:
        raise ValueError("q is [batch][max_new][Hq][d]")
    b, T = owner.c.batch, int(q.shape[1])
    _need(q, "q", cfg.torch_dtype, (b, T, cfg.num_q_heads, cfg.head_dim), dev)
    _need(n_new, "n_new", torch.int32, (b,), dev)
    if lse is not None:
        _need(lse, "lse", torch.float32, (b, T, cfg.num_q_heads), dev)
    c = owner.c
    if lens is not None:
        _need(lens, "lens", torch.int32, (b,), dev)
        c = _lib.spla_cache.from_buffer_copy(c)
        c.context_lens = lens.data_ptr()
    with _on(dev):
        if out is None:
            out = torch.zeros_like(q)
        else:
            _need(out, "out", q.dtype, q.shape, dev)
        # one size whatever the chunk, so that a captured call and later eager ones never
        # see it replaced
        if owner._chunk_ws is None:
            need = _lib.spla_chunk_attention_workspace_size(owner.params, b, T)
            owner._chunk_ws = torch.empty((need + 255) // 256 * 256, dtype=torch.uint8, device=dev)
        ws = owner._chunk_ws
        _lib.spla_chunk_attention(owner.params, c, q.data_ptr(), n_new.data_ptr(), T,
                                  out.data_ptr(), _ptr(lse), ws.data_ptr(), ws.numel(),
                                  owner.dev_status.data_ptr(), _stream(dev, stream))
    return out


class SplaPagedKV:
    """Paged K and V of one full-attention layer: pools [num_phys_blocks][Hkv][B][d], the
    block table and the lengths, without the sparse path's statistics and state. The tensors
    are the caller's and are kept, not copied. block_table and context_lens may be left out
    where only qk_norm_rope writes through it."""

    def __init__(self, cfg, k_pool, v_pool, block_table=None, context_lens=None):
        _lib.load()
        dev = k_pool.device
        n = int(k_pool.shape[0])
        shape = (n, cfg.num_kv_heads, cfg.block_size, cfg.head_dim)
        _need(k_pool, "k_pool", cfg.torch_dtype, shape, dev)
        _need(v_pool, "v_pool", cfg.torch_dtype, shape, dev)
        if block_table is not None:
            _need(block_table, "block_table", torch.int32, block_table.shape, dev)
        batch, mbp = map(int, block_table.shape) if block_table is not None else (0, 0)
        if context_lens is not None:
            _need(context_lens, "context_lens", torch.int32, (batch,), dev)
        self.cfg, self.device, self.num_phys_blocks = cfg, dev, n
        self.k_pool, self.v_pool = k_pool, v_pool
        self.block_table, self.context_lens = block_table, context_lens
        self.params = cfg.params()
        self.c = _lib.spla_cache(k_pool.data_ptr(), v_pool.data_ptr(), None, None, None, None,
                                 _ptr(block_table), _ptr(context_lens), batch, mbp, n)
        self.dev_status = torch.zeros((1,), dtype=torch.int32, device=dev)
        self._chunk_ws = None

    def chunk_attention(self, q, n_new, out=None, lse=None, lens=None, stream=None):
        """Exact causal attention of each sequence's last n_new tokens over all it holds.
        q: [batch][max_new][Hq][d]; n_new: [batch] int32; lens: [batch] int32 lengths with the
        chunk included (default: context_lens). Returns out (q's layout; rows past n_new are
        left as they are, zeros in a tensor made here); lse: [batch][max_new][Hq] fp32, filled
        when given."""
        return chunk_attention(self, q, n_new, out, lse, lens, stream)

    def status(self) -> int:
        """Device-detected fault bits (synchronises)."""
        return int(self.dev_status.item())


def _flat(t, name, dtype, n, device):
    """A contiguous tensor of n elements, whatever its shape, or ValueError."""
    if t.numel() != n:
        raise ValueError(f"{name}: expected {n} elements, got {t.numel()}")
    _need(t, name, dtype, t.shape, device)


def _rows(t, name, heads, d, dtype, device):
    """Row stride of a [rows][heads][d] view whose heads lie side by side."""
    if t.dim() != 3 or t.shape[1:] != (heads, d) or t.dtype != dtype or t.device != device \
            or t.stride(2) != 1 or (heads > 1 and t.stride(1) != d):
        raise ValueError(f"{name}: expected a {dtype} [rows][{heads}][{d}] tensor on {device} "
                         "whose heads lie side by side")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), heads * d)


def qk_norm_rope(cfg, q, k, v, positions, inv_freq=None, q_gamma=None, k_gamma=None, eps=1e-6,
                 interleaved=False, q_out=None, k_out=None, v_out=None, kv=None, slots=None,
                 dev_status=None, stream=None):
    """RMSNorm of the query and key heads and the rotary position in one pass
    (spla_qk_norm_rope). q: [rows][Hq][d], k and v: [rows][Hkv][d], slices of a fused
    projection or tensors of their own (v may be None); positions: [rows] int32, negative:
    row skipped; inv_freq: [rot_dim / 2] float64. Outputs, positions and slots may have any shape
    of that many elements. Keys and values go to k_out, v_out
    [rows][Hkv][d] (made here when not given), or with slots ([rows] int64) into the pools of
    kv (a SplaPagedKV or SplaDecodeCache). Returns q_out, or (q_out, k_out, v_out) without
    slots; tensors made here hold zeros in skipped rows."""
    hq, hkv, d, dt, dev = (cfg.num_q_heads, cfg.num_kv_heads, cfg.head_dim, cfg.torch_dtype,
                           q.device)
    rows = int(q.shape[0])
    qs, ks = _rows(q, "q", hq, d, dt, dev), _rows(k, "k", hkv, d, dt, dev)
    vs = _rows(v, "v", hkv, d, dt, dev) if v is not None else 0
    if k.shape[0] != rows or (v is not None and v.shape[0] != rows):
        raise ValueError("q, k and v have different numbers of rows")
    _flat(positions, "positions", torch.int32, rows, dev)
    rot = 0
    if inv_freq is not None:
        _need(inv_freq, "inv_freq", torch.float64, (inv_freq.numel(),), dev)
        rot = 2 * inv_freq.numel()
    for g, name in ((q_gamma, "q_gamma"), (k_gamma, "k_gamma")):
        if g is not None:
            _need(g, name, torch.float32, (d,), dev)
    with _on(dev):
        if q_out is None:
            q_out = torch.zeros((rows, hq, d), dtype=dt, device=dev)
        else:
            _flat(q_out, "q_out", dt, rows * hq * d, dev)
        phys = 0
        if slots is not None:
            if kv is None or k_out is not None or v_out is not None:
                raise ValueError("slots go with kv, and without k_out and v_out")
            _flat(slots, "slots", torch.int64, rows, dev)
            pool = (kv.num_phys_blocks, hkv, cfg.block_size, d)
            _need(kv.k_pool, "kv.k_pool", dt, pool, dev)
            kp, vp, phys = kv.k_pool, kv.v_pool, kv.num_phys_blocks
        else:
            if kv is not None:
                raise ValueError("kv goes with slots")
            if k_out is None:
                k_out = torch.zeros((rows, hkv, d), dtype=dt, device=dev)
            if v_out is None and v is not None:
                v_out = torch.zeros((rows, hkv, d), dtype=dt, device=dev)
            _flat(k_out, "k_out", dt, rows * hkv * d, dev)
            if v_out is not None:
                _flat(v_out, "v_out", dt, rows * hkv * d, dev)
            kp, vp = k_out, v_out
        status = dev_status if dev_status is not None else getattr(kv, "dev_status", None)
        _lib.spla_qk_norm_rope(cfg.params(), q.data_ptr(), qs, k.data_ptr(), ks, _ptr(v), vs, rows,
                               positions.data_ptr(), _ptr(inv_freq), rot, int(interleaved),
                               _ptr(q_gamma), _ptr(k_gamma), eps, q_out.data_ptr(), kp.data_ptr(),
                               _ptr(vp), _ptr(slots), phys, _ptr(status), _stream(dev, stream))
    return q_out if slots is not None else (q_out, k_out, v_out)
