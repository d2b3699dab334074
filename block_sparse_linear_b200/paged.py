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
from collections import namedtuple

import torch

from . import _lib

BlockPlan = namedtuple("BlockPlan", "n_granted lens_after positions slots free_count")

def _elsewhere(device, stream):
    """Whether the call has to be made within _at: another device is current than the tensors'
    (launches go to the current one), or a stream is named (tensors made here are to be
    allocated and filled on it)."""
    return stream is not None or torch.cuda.current_device() != device.index


def _at(device, stream):
    if stream is not None and stream.device != device:
        raise ValueError(f"stream: one of {stream.device}, the tensors are on {device}")
    return torch.cuda.stream(stream) if stream is not None else torch.cuda.device(device)


def _stream(device):
    return torch._C._cuda_getCurrentRawStream(device.index)   # the handle without an object


def _ptr(t):
    return None if t is None else t.data_ptr()


def _bad(t, name, dtype, shape, device):
    raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} "
                     f"on {device}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _need(t, name, dtype, shape, device):
    """A contiguous tensor of this type and shape on this device, or ValueError."""
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        _bad(t, name, dtype, shape, device)


class SplaBlockPool:
    """The free blocks of a paged pool and the block table they are handed out through
    (include/spla.h's ``spla_block_pool``), kept on the device.

    block_table: [batch][max_blocks_per_seq] int32; free_list: [num_phys_blocks] int32, a
    stack whose first free_count entries are free; free_count: [1] int32. The table may be
    the one a SplaDecodeCache or SplaPagedKV was made with: both keep the tensor itself.
    Calls on one pool are made on one stream or ordered by events."""

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
        self._rows_like = None                  # shape and type of the row outputs
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
        shape = (b,)
        _need(context_lens, "context_lens", torch.int32, shape, dev)
        _need(n_new, "n_new", torch.int32, shape, dev)
        if _elsewhere(dev, stream):
            with _at(dev, stream):
                return self.plan(context_lens, n_new, max_new, rows, commit)
        like = torch.empty_like                 # (half the host time of naming shape and type)
        granted, after = like(n_new), like(n_new)
        left = self.free_count if commit else like(self.free_count)
        pos = slots = None
        if rows:
            if self._rows_like is None or self._rows_like[0].shape[1] != max_new:
                self._rows_like = tuple(
                    torch.empty(1, dtype=dt, device=dev).expand(b, max_new)
                    for dt in (torch.int32, torch.int64))
            fmt = torch.contiguous_format
            pos = like(self._rows_like[0], memory_format=fmt)
            slots = like(self._rows_like[1], memory_format=fmt)
        _lib.spla_block_plan(self.c, context_lens.data_ptr(), n_new.data_ptr(), max_new,
                             granted.data_ptr(), after.data_ptr(), _ptr(pos), _ptr(slots),
                             left.data_ptr(), self.dev_status.data_ptr(), _stream(dev))
        return BlockPlan(granted, after, pos, slots, left)

    def release(self, keep_lens, context_lens, stream=None) -> None:
        """Shortens sequences to keep_lens tokens (0: done) and takes their blocks back;
        context_lens is updated in place (spla_block_release). A SplaDecodeCache's sequence
        that ends also has its own context_lens and S, z set to 0 and m to -inf before the
        index is used again: its state still holds what was appended."""
        dev = self.device
        _need(keep_lens, "keep_lens", torch.int32, (self.batch,), dev)
        _need(context_lens, "context_lens", torch.int32, (self.batch,), dev)
        if _elsewhere(dev, stream):
            with _at(dev, stream):
                return self.release(keep_lens, context_lens)
        _lib.spla_block_release(self.c, keep_lens.data_ptr(), context_lens.data_ptr(),
                                self.dev_status.data_ptr(), _stream(dev))

    def status(self) -> int:
        """Device-detected fault bits (synchronises)."""
        return int(self.dev_status.item())


def chunk_attention(owner, q, n_new, out=None, lse=None, lens=None, stream=None):
    """spla_chunk_attention over an owner's cache struct (SplaDecodeCache, SplaPagedKV)."""
    p, dev = owner.params, owner.k_pool.device
    if q.dim() != 4:
        raise ValueError("q is [batch][max_new][Hq][d]")
    b, T, hq = owner.c.batch, q.shape[1], p.num_q_heads
    _need(q, "q", owner.k_pool.dtype, (b, T, hq, p.head_dim), dev)
    _need(n_new, "n_new", torch.int32, (b,), dev)
    if lse is not None:
        _need(lse, "lse", torch.float32, (b, T, hq), dev)
    c = owner.c
    if lens is not None:
        _need(lens, "lens", torch.int32, (b,), dev)
        c = _lib.spla_cache.from_buffer_copy(c)
        c.context_lens = lens.data_ptr()
    if _elsewhere(dev, stream):
        with _at(dev, stream):
            return chunk_attention(owner, q, n_new, out, lse, lens)
    if out is None:
        out = torch.zeros_like(q)
    else:
        _need(out, "out", q.dtype, q.shape, dev)
    # one size whatever the chunk, so that a captured call and later eager ones never see it
    # replaced
    if owner._chunk_ws is None:
        need = _lib.spla_chunk_attention_workspace_size(p, b, T)
        owner._chunk_ws = torch.empty((need + 255) // 256 * 256, dtype=torch.uint8, device=dev)
        owner._chunk_ws_stream = _stream(dev)
    ws, at = owner._chunk_ws, _stream(dev)
    if at != owner._chunk_ws_stream:            # its memory is reused when this stream is done too
        ws.record_stream(torch.cuda.current_stream(dev))
    _lib.spla_chunk_attention(p, c, q.data_ptr(), n_new.data_ptr(), T, out.data_ptr(),
                              _ptr(lse), ws.data_ptr(), ws.numel(), owner.dev_status.data_ptr(),
                              at)
    return out


class SplaPagedKV:
    """Paged K and V of one full-attention layer: pools [num_phys_blocks][Hkv][B][d], the
    block table and the lengths, without the sparse path's statistics and state. The tensors
    are the caller's and are kept, not copied. block_table and context_lens may be left out
    where only qk_norm_rope writes through it. Chunk-attention calls of one object share its
    workspace (39 MB for heads of 128, 20 MB for 64, made by the first call): they are made on
    one stream or ordered by events; layers that run side by side have an object each."""

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
    if t.numel() != n or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of {n} elements on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _rows(t, name, heads, d, dtype, device):
    """Row stride of a [rows][heads][d] view whose heads lie side by side."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != d or t.dtype is not dtype \
            or t.device != device or stride[2] != 1 or (heads > 1 and stride[1] != d):
        raise ValueError(f"{name}: expected a {dtype} [rows][{heads}][{d}] tensor on {device} "
                         "whose heads lie side by side")
    return stride[0] if shape[0] > 1 else heads * d


def qk_norm_rope(cfg, q, k, v, positions, inv_freq=None, q_gamma=None, k_gamma=None, eps=1e-6,
                 interleaved=False, q_out=None, k_out=None, v_out=None, kv=None, slots=None,
                 dev_status=None, stream=None):
    """RMSNorm of the query and key heads and the rotary position in one pass
    (spla_qk_norm_rope). q: [rows][Hq][d], k and v: [rows][Hkv][d], slices of a fused
    projection or tensors of their own (v may be None); positions: [rows] int32, negative:
    row skipped; inv_freq: [rot_dim / 2] float64. Outputs, positions and slots may have any shape
    of that many elements. Keys and values go to k_out, v_out
    [rows][Hkv][d] (made here when not given), or with slots ([rows] int64) into the pools of
    kv, a SplaPagedKV. (A SplaDecodeCache is refused: its pages are written by append, which
    keeps the statistics, state and lengths in step with them.) Returns q_out, or (q_out, k_out,
    v_out) without slots; tensors made here hold zeros in skipped rows."""
    hq, hkv, d, dt, dev = (cfg.num_q_heads, cfg.num_kv_heads, cfg.head_dim, cfg.torch_dtype,
                           q.device)
    rows = q.shape[0]
    qs, ks = _rows(q, "q", hq, d, dt, dev), _rows(k, "k", hkv, d, dt, dev)
    vs = _rows(v, "v", hkv, d, dt, dev) if v is not None else 0
    if k.shape[0] != rows or (v is not None and v.shape[0] != rows):
        raise ValueError("q, k and v have different numbers of rows")
    _flat(positions, "positions", torch.int32, rows, dev)
    rot = 0
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        _flat(inv_freq, "inv_freq", torch.float64, rot // 2, dev)
    if q_gamma is not None:
        _need(q_gamma, "q_gamma", torch.float32, (d,), dev)
    if k_gamma is not None:
        _need(k_gamma, "k_gamma", torch.float32, (d,), dev)
    if (slots is None) != (kv is None) or (kv is not None and (k_out is not None or v_out is not None)):
        raise ValueError("kv and slots go together, and without k_out and v_out")
    if kv is not None and not isinstance(kv, SplaPagedKV):
        raise ValueError(f"kv: expected a SplaPagedKV, got {type(kv).__name__} (a SplaDecodeCache "
                         "takes keys and values by append)")
    if _elsewhere(dev, stream):
        with _at(dev, stream):
            return qk_norm_rope(cfg, q, k, v, positions, inv_freq, q_gamma, k_gamma, eps, interleaved,
                                q_out, k_out, v_out, kv, slots, dev_status)
    if q_out is None:
        q_out = torch.zeros((rows, hq, d), dtype=dt, device=dev)
    else:
        _flat(q_out, "q_out", dt, rows * hq * d, dev)
    if kv is not None:
        _flat(slots, "slots", torch.int64, rows, dev)
        kp, vp, phys = kv.k_pool, kv.v_pool, kv.num_phys_blocks
        _need(kp, "kv.k_pool", dt, (phys, hkv, cfg.block_size, d), dev)
        if dev_status is None:
            dev_status = kv.dev_status
    else:
        phys = 0
        if k_out is None:
            k_out = torch.zeros((rows, hkv, d), dtype=dt, device=dev)
        else:
            _flat(k_out, "k_out", dt, rows * hkv * d, dev)
        if v_out is not None:
            _flat(v_out, "v_out", dt, rows * hkv * d, dev)
        elif v is not None:
            v_out = torch.zeros((rows, hkv, d), dtype=dt, device=dev)
        kp, vp = k_out, v_out
    _lib.spla_qk_norm_rope(cfg.params(), q.data_ptr(), qs, k.data_ptr(), ks, _ptr(v), vs, rows,
                           positions.data_ptr(), _ptr(inv_freq), rot, interleaved, _ptr(q_gamma),
                           _ptr(k_gamma), eps, q_out.data_ptr(), kp.data_ptr(), _ptr(vp),
                           _ptr(slots), phys, _ptr(dev_status), _stream(dev))
    return q_out if kv is not None else (q_out, k_out, v_out)
