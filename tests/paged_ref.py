"""Plain 64-bit forms of the paged serving operators, for the tests."""
import math

import numpy as np
import torch

U32 = 2.0 ** -24                                   # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def plan(table, free_list, free_count, block, lens, n_new, max_new):
    """One sequence after another, as the header words it. Returns a dict of arrays."""
    table = table.copy()
    batch, mbp = table.shape
    phys = len(free_list)
    status, top, full = 0, int(free_count), False
    if not 0 <= top <= phys:
        status, top = status | 0x2, 0
    granted = np.zeros(batch, np.int32)
    for b in range(batch):
        n, L = int(n_new[b]), int(lens[b])
        if n < 0 or n > max_new:
            status |= 0x8
            continue
        if L < 0 or L + n > mbp * block:
            status |= 0x2
            continue
        have, want = -(-L // block), -(-(L + n) // block)
        need = want - have
        if need and (full or need > top):
            full, status = True, status | 0x20
            continue
        for j in range(have, want):
            top -= 1
            table[b, j] = free_list[top]
        granted[b] = n
    pos = np.full((batch, max_new), -1, np.int32)
    slots = np.full((batch, max_new), -1, np.int64)
    for b in range(batch):
        for t in range(granted[b]):
            p = int(lens[b]) + t
            pos[b, t] = p
            page = int(table[b, p // block])
            if 0 <= page < phys:
                slots[b, t] = page * block + p % block
            else:
                status |= 0x1
    return dict(block_table=table, n_granted=granted, lens_after=(lens + granted).astype(np.int32),
                positions=pos, slots=slots, free_count=top, status=status)


def norm_rope(x, gamma, positions, inv_freq, rot, interleaved, eps):
    """(result, |a| + |b| per element): x [rows][heads][d] float64 on any device."""
    y = x
    if gamma is not None:
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma
    out, size = y.clone(), y.abs()
    if rot:
        ang = positions.double()[:, None, None] * inv_freq
        c, s = torch.cos(ang), torch.sin(ang)
        i = torch.arange(rot // 2, device=x.device)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        a, b = y[..., ia], y[..., ib]
        out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
        size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return out, size


def tokens(pool, table_row, L, h):
    """[L][d] float64 of one sequence and KV head; entries outside the pool count as zeros."""
    block = pool.shape[2]
    nb = -(-L // block)
    rows = table_row[:nb].long()
    ok = (rows >= 0) & (rows < pool.shape[0])
    x = pool[rows.clamp(0, pool.shape[0] - 1), h].double()
    return torch.where(ok[:, None, None], x, torch.zeros_like(x)).reshape(-1, pool.shape[3])[:L]


def chunk(q, K, V, L, scale, dtype):
    """One query head's chunk: q [n][d], K, V [L][d] float64. Returns out, lse and the
    bounds of their errors for kernels that keep logits, statistics and sums in fp32 and
    round p (to `dtype`) and out once.

    A row's logit x = scale q.k is off by dx <= (d + 4) u scale sum|q_i k_i| + 2 u |x - m|
    (d products and sums, the scaling, the subtraction of the maximum) plus 4 u for the
    exponential; the sums over L tokens add (L + 8) u of the absolute sum, whatever their
    order. With e = max dx + (L + 12) u: |d out| <= 2 e' sum p|v| / l, e' = exp(e) - 1, plus
    half a step of p for each product (16-bit types) and half a step of out."""
    n, d = q.shape
    pos = L - n + torch.arange(n, device=q.device)
    seen = torch.arange(L, device=q.device)[None] <= pos[:, None]
    x = (q @ K.T) * scale
    size = (q.abs() @ K.abs().T) * scale
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - lse[:, None])
    Vz, pv = V, None
    # tokens a row does not see have no part in it, finite or not: sum only what is seen
    if not torch.isfinite(V).all():
        rows = [p[i, :int(pos[i]) + 1] @ V[:int(pos[i]) + 1] for i in range(n)]
        out = torch.stack(rows)
        Vz = torch.nan_to_num(V, 0.0, 0.0, 0.0)
    else:
        out = p @ V
    pv = p @ Vz.abs()
    m = torch.where(seen, x, torch.full_like(x, -math.inf)).amax(1, keepdim=True)
    dx = ((d + 4) * U32 * size + 2 * U32 * (m - x).abs().nan_to_num(0.0, 0.0, 0.0))
    dx = torch.where(seen & (p > 0), dx, torch.zeros_like(dx)).amax(1)
    e = torch.expm1(dx + (L + 12) * U32)
    hs = half_step(dtype)
    p_step = hs if dtype != torch.float32 else 0.0
    out_tol = ((2 * e + p_step)[:, None] * pv) * (1 + hs) + hs * out.abs() + 1e-30
    lse_tol = dx + (L + 12) * U32 + 4 * U32 * lse.abs() + 4 * U32 * m[:, 0].abs()
    return out, lse, out_tol, lse_tol
