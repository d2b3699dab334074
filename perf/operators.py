"""Cases and plain forms of the paged serving operators.

Three operators that a serving step runs in a row around the paged cache:

  plan   block-table rows, positions and slots of the step's new tokens, from the requests'
         lengths and a stack of free blocks (spla_block_plan);
  rope   RMSNorm of every query and key head and the rotary position in one pass, with the
         keys and values written into the pages by slot, or out as rows (spla_qk_norm_rope);
  attn   exact causal attention of a chunk of new tokens (one token included) over the paged
         cache (spla_chunk_attention).

A case is a dict of plain values; lengths come from the case alone, values from the seed.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ROPE_BASE = 500000.0
EPS = 1e-6


# ------------------------------------------------------------------------------- the cases
def _plan(name, batch, past, new, block, spare):
    return {"name": name, "op": "plan", "batch": batch, "past_lo": past[0], "past_hi": past[1],
            "new_lo": new[0], "new_hi": new[1], "block": block, "spare": spare}


def _rope(name, rows, heads, d, dtype, rot, interleaved, pages, pad, far):
    return {"name": name, "op": "rope", "rows": rows, "hq": heads[0], "hkv": heads[1], "d": d,
            "dtype": dtype, "rot": rot, "interleaved": interleaved, "pages": pages, "pad": pad,
            "far": far, "block": 64}


def _attn(name, batch, past, new, heads, d, block, dtype):
    return {"name": name, "op": "attn", "batch": batch, "past_lo": past[0], "past_hi": past[1],
            "new_lo": new[0], "new_hi": new[1], "hq": heads[0], "hkv": heads[1], "d": d,
            "block": block, "dtype": dtype}


def listed():
    return [
        # one decode step of the ragged 16-sequence workload: a token each, mostly no new block
        _plan("plan_decode_16", 16, (4096, 262144), (1, 1), 64, 1.0),
        # a scheduler's prefill wave: 256 prompts of up to 8192 tokens, the pool nearly used up
        # (the last requests in line are refused)
        _plan("plan_prefill_256", 256, (0, 4096), (1, 8192), 64, 0.9),
        # one decode step of the 32K workload: 8 tokens, K and V into their pages
        _rope("rope_decode_8", 8, (32, 8), 128, "bf16", 128, False, True, 0, 32768),
        # a 4096-token fp32 prompt of the 4K workload's heads, interleaved pairs, half of the
        # dimensions rotated, rows out for the append call, some padding rows
        _rope("rope_chunk_f32", 4096, (4, 1), 64, "f32", 32, True, False, 33, 4096),
        # a 65536-token prefill chunk at far positions of a 1M-token context, into the pages
        _rope("rope_prefill_64k", 65536, (32, 8), 128, "bf16", 128, False, True, 0, 1048576),
        # one token for each sequence of the 32K workload
        _attn("attn_decode_8x32k", 8, (32768, 32768), (1, 1), (32, 8), 128, 64, "bf16"),
        # verification of five drafted tokens over the 128K workload
        _attn("attn_verify_4x128k", 4, (130000, 131067), (5, 5), (32, 8), 128, 64, "bf16"),
        # the ragged workload, decodes and short chunks in one batch
        _attn("attn_ragged_16", 16, (4096, 262111), (1, 33), (32, 8), 128, 64, "bf16"),
        # one token over the 1M-token context, 128-token pages
        _attn("attn_decode_1m", 1, (1048500, 1048500), (1, 1), (32, 8), 128, 128, "bf16"),
        # a 2048-token chunk of a long prompt: 65536 tokens held before it
        _attn("attn_prefill_2k_over_64k", 1, (65536, 65536), (2048, 2048), (32, 8), 128, 64, "bf16"),
        # a wave of prompts of unequal lengths from nothing, 64-wide heads, two queries a KV head
        _attn("attn_prompts_24", 24, (0, 0), (61, 1500), (16, 8), 64, 64, "bf16"),
        # a 512-token fp32 chunk over the 4K workload
        _attn("attn_chunk_f32", 1, (3584, 3584), (512, 512), (4, 1), 64, 64, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("plan", "rope", "attn", "attn"))
    if op == "plan":
        batch = _log(rng, 1, 512)
        new = _log(rng, 1, min(8192, 2097152 // batch))
        c = _plan("", batch, (_log(rng, 1, 64) - 1, _log(rng, 64, 262144 if batch <= 64 else 16384)),
                  (rng.choice((0, 1)) if new > 1 else 1, new), rng.choice((64, 128)),
                  rng.choice((0.8, 0.95, 1.0)))
    elif op == "rope":
        d, dtype = rng.choice((64, 128)), rng.choice(("bf16", "bf16", "f32"))
        hkv = rng.choice((1, 2, 4, 8))
        pages = rng.random() < 0.5
        rows = _log(rng, 1, 65536 if dtype == "bf16" else 32768)
        c = _rope("", rows, (hkv * rng.choice((1, 2, 4)), hkv), d, dtype,
                  16 * rng.randint(1, d // 16), rng.random() < 0.5, pages,
                  0 if pages else rng.randint(0, rows // 8), _log(rng, 64, 1048576))
        c["block"] = rng.choice((64, 128))
    else:
        d, dtype = rng.choice((64, 128)), rng.choice(("bf16", "bf16", "bf16", "f32"))
        hkv, g = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4))
        batch = _log(rng, 1, 32)
        new = rng.choice((1, _log(rng, 2, 64), _log(rng, 2, 2048)))
        # score elements and cached bytes within what the largest listed cases have
        most = (4.0e9 if dtype == "bf16" else 1.0e8) / (batch * hkv * g * new)
        most = int(min(most, 2.0e9 / (batch * hkv * d * 4), 1000000))
        hi = _log(rng, 2, max(3, most))
        lo = _log(rng, 1, hi) - 1
        c = _attn("", batch, (lo, hi), (rng.choice((1, new)), new), (hkv * g, hkv), d,
                  rng.choice((64, 128)), dtype)
    del c["name"]
    return c


def _spread(lo, hi, n, salt):
    """n whole numbers evenly spread over the logarithm of [lo, hi], in a fixed shuffled order."""
    a, b = math.log(lo + 1), math.log(hi + 1)
    v = [hi] if n == 1 else [int(round(math.exp(a + (b - a) * i / (n - 1)) - 1)) for i in range(n)]
    random.Random(salt).shuffle(v)
    return [min(max(x, lo), hi) for x in v]


def _lengths(c):
    """(tokens held before the step, new tokens) of every sequence."""
    return (_spread(c["past_lo"], c["past_hi"], c["batch"], 1),
            _spread(c["new_lo"], c["new_hi"], c["batch"], 2))


def _blocks(n, block):
    return (n + block - 1) // block


# ------------------------------------------------------------------------------- inputs
def _paged(c, held, width, spare_blocks, gen):
    """A block table over randomly placed physical blocks for `held` tokens a sequence, and the
    blocks left over."""
    nb = [_blocks(n, c["block"]) for n in held]
    total = sum(nb)
    perm = torch.randperm(total + spare_blocks, device="cuda", generator=gen).to(torch.int32)
    nbt = torch.tensor(nb, device="cuda")
    start = torch.cumsum(nbt, 0) - nbt
    j = torch.arange(width, device="cuda")[None]
    table = torch.where(j < nbt[:, None], perm[(start[:, None] + j).clamp(max=total + spare_blocks - 1)],
                        torch.full((), -1, dtype=torch.int32, device="cuda")).contiguous()
    return table, perm[total:].contiguous(), total + spare_blocks


def prepare(case, seed):
    c = case
    gen = torch.Generator("cuda").manual_seed(seed)
    s = {"case": c}
    i32 = dict(dtype=torch.int32, device="cuda")
    if c["op"] == "plan":
        past, new = _lengths(c)
        B = c["block"]
        need = sum(_blocks(p + n, B) - _blocks(p, B) for p, n in zip(past, new))
        spare = max(1, int(need * c["spare"])) if c["spare"] < 1 else need + 64
        width = max(_blocks(p + n, B) for p, n in zip(past, new))
        s["table"], free, s["phys"] = _paged(c, past, max(1, width), spare, gen)
        s["free_list"] = torch.zeros(s["phys"], **i32)
        s["free_list"][:spare] = free
        s["free_count"] = torch.tensor([spare], **i32)
        s["lens"] = torch.tensor(past, **i32)
        s["n_new"] = torch.tensor(new, **i32)
        s["max_new"] = max(1, max(new))
    elif c["op"] == "rope":
        dt, rows, hq, hkv, d = DT[c["dtype"]], c["rows"], c["hq"], c["hkv"], c["d"]
        # the fused projection's output: q, k and v heads of a token side by side
        s["qkv"] = torch.randn((rows, (hq + 2 * hkv) * d), device="cuda", generator=gen).to(dt)
        s["positions"] = torch.randint(0, c["far"], (rows,), device="cuda", generator=gen,
                                       dtype=torch.int32)
        if c["pad"]:
            s["positions"][rows - c["pad"]:] = -1
        s["q_gamma"] = 1 + 0.2 * torch.randn(d, device="cuda", generator=gen)
        s["k_gamma"] = 1 + 0.2 * torch.randn(d, device="cuda", generator=gen)
        i = torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda")
        s["inv_freq"] = ROPE_BASE ** (-2.0 * i / c["rot"])
        s["q_out"] = torch.zeros((rows, hq, d), dtype=dt, device="cuda")
        if c["pages"]:
            blocks = _blocks(rows, c["block"]) + 1
            shape = (blocks, hkv, c["block"], d)
            s["slots"] = torch.randperm(blocks * c["block"], device="cuda", generator=gen)[:rows]
            s["k_pool"] = torch.zeros(shape, dtype=dt, device="cuda")
            s["v_pool"] = torch.zeros(shape, dtype=dt, device="cuda")
        else:
            s["k_out"] = torch.zeros((rows, hkv, d), dtype=dt, device="cuda")
            s["v_out"] = torch.zeros((rows, hkv, d), dtype=dt, device="cuda")
    else:
        dt, hq, hkv, d, B = DT[c["dtype"]], c["hq"], c["hkv"], c["d"], c["block"]
        past, new = _lengths(c)
        held = [p + n for p, n in zip(past, new)]
        s["table"], _, phys = _paged(c, held, max(_blocks(n, B) for n in held), 1, gen)
        # keys and values: unit normal with an offset of their own for each page and head
        for name in ("k_pool", "v_pool"):
            x = torch.randn((phys, hkv, B, d), device="cuda", generator=gen, dtype=dt)
            x += 0.5 * torch.randn((phys, hkv, 1, d), device="cuda", generator=gen, dtype=dt)
            s[name] = x
        T = max(new)
        s["q"] = torch.randn((c["batch"], T, hq, d), device="cuda", generator=gen, dtype=dt)
        s["lens"] = torch.tensor(held, **i32)
        s["n_new"] = torch.tensor(new, **i32)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((c["batch"], T, hq), dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------------------- plain forms
def _plain_plan(s):
    B, T = s["case"]["block"], s["max_new"]
    lens, n, table = s["lens"].long(), s["n_new"].long(), s["table"]
    have = (lens + B - 1) // B
    need = (lens + n + B - 1) // B - have
    upto = torch.cumsum(need, 0)
    fits = (need == 0) | (upto <= s["free_count"])
    granted = torch.where(fits, n, 0)
    taken = torch.where(fits, need, 0)
    j = torch.arange(table.shape[1], device="cuda")[None]
    fresh = (j >= have[:, None]) & (j < (have + taken)[:, None])
    at = s["free_count"] - 1 - (upto - need)[:, None] - (j - have[:, None])
    table = torch.where(fresh, s["free_list"][at.clamp(0, s["phys"] - 1)], table)
    t = torch.arange(T, device="cuda")[None]
    live = t < granted[:, None]
    pos = torch.where(live, lens[:, None] + t, -1)
    page = torch.gather(table, 1, (pos.clamp(min=0) // B).clamp(max=table.shape[1] - 1)).long()
    slots = torch.where(live, page * B + pos.clamp(min=0) % B, -1)
    return {"block_table": table, "n_granted": granted.int(), "lens_after": (lens + granted).int(),
            "positions": pos.int(), "slots": slots,
            "free_count": (s["free_count"] - taken.sum()).int()}


def _norm_rope(x, gamma, cos, sin, rot, interleaved):
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * gamma
    r, rest = y[..., :rot], y[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, rest), -1).to(x.dtype)


def _split(s):
    c = s["case"]
    rows, hq, hkv, d = c["rows"], c["hq"], c["hkv"], c["d"]
    q, k, v = s["qkv"].split((hq * d, hkv * d, hkv * d), 1)
    return q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d)), v.unflatten(1, (hkv, d))


def _plain_rope(s):
    c = s["case"]
    q, k, v = _split(s)
    angle = (s["positions"].double()[:, None] * s["inv_freq"])[:, None]
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _norm_rope(q, s["q_gamma"], cos, sin, c["rot"], c["interleaved"])
    k = _norm_rope(k, s["k_gamma"], cos, sin, c["rot"], c["interleaved"])
    if c["pages"]:
        page, off = s["slots"] // c["block"], s["slots"] % c["block"]
        s["k_pool"][page, :, off] = k
        s["v_pool"][page, :, off] = v
        return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    live = (s["positions"] >= 0)[:, None, None]
    return {"q": torch.where(live, q, s["q_out"]), "k": torch.where(live, k, s["k_out"]),
            "v": torch.where(live, v, s["v_out"])}


def _plain_attn(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    b, T = s["q"].shape[:2]
    pages = s["table"].clamp(min=0).long()
    k = s["k_pool"][pages].transpose(2, 1).flatten(2, 3).float()        # [b][hkv][tokens][d]
    v = s["v_pool"][pages].transpose(2, 1).flatten(2, 3).float()
    q = s["q"].view(b, T, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).flatten(2, 3).float()
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).unflatten(2, (-1, T))
    t = torch.arange(T, device="cuda")
    pos = (s["lens"] - s["n_new"])[:, None] + t
    seen = torch.arange(k.shape[2], device="cuda") <= pos[:, :, None]   # [b][T][tokens]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(top).exp_()
    mass = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (-1, T)) / mass
    lse = (top + mass.log())[..., 0]
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3).to(s["q"].dtype)
    lse = lse.permute(0, 3, 1, 2).flatten(2, 3)
    live = t < s["n_new"][:, None]
    return {"out": torch.where(live[..., None, None], o, s["out"]),
            "lse": torch.where(live[..., None], lse, s["lse"])}


# ------------------------------------------------------------------------------- the framework's calls
def _own_plan(s):
    if "pool" not in s:                      # the allocator's handle, which a server keeps
        from block_sparse_linear_b200 import SplaBlockPool
        s["pool"] = SplaBlockPool(s["table"], s["free_list"], s["free_count"],
                                  s["case"]["block"])
    p = s["pool"].plan(s["lens"], s["n_new"], s["max_new"], commit=False)
    return {"block_table": s["table"], "n_granted": p.n_granted, "lens_after": p.lens_after,
            "positions": p.positions, "slots": p.slots, "free_count": p.free_count}


def _own_rope(s):
    c = s["case"]
    if "cfg" not in s:
        from block_sparse_linear_b200 import SplaConfig, SplaPagedKV, qk_norm_rope
        s["cfg"] = SplaConfig(num_q_heads=c["hq"], num_kv_heads=c["hkv"], head_dim=c["d"],
                              block_size=c["block"], top_k=1, dtype=c["dtype"])
        s["kv"] = (SplaPagedKV(s["cfg"], s["k_pool"], s["v_pool"]) if c["pages"] else None)
        s["call"] = qk_norm_rope
    q, k, v = _split(s)
    args = dict(positions=s["positions"], inv_freq=s["inv_freq"], q_gamma=s["q_gamma"],
                k_gamma=s["k_gamma"], eps=EPS, interleaved=c["interleaved"], q_out=s["q_out"])
    if c["pages"]:
        s["call"](s["cfg"], q, k, v, kv=s["kv"], slots=s["slots"], **args)
        return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    s["call"](s["cfg"], q, k, v, k_out=s["k_out"], v_out=s["v_out"], **args)
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _own_attn(s):
    c = s["case"]
    if "kv" not in s:                        # the cache's handle, which a server keeps
        from block_sparse_linear_b200 import SplaConfig, SplaPagedKV
        cfg = SplaConfig(num_q_heads=c["hq"], num_kv_heads=c["hkv"], head_dim=c["d"],
                         block_size=c["block"], top_k=1, dtype=c["dtype"])
        s["kv"] = SplaPagedKV(cfg, s["k_pool"], s["v_pool"], s["table"], s["lens"])
    s["kv"].chunk_attention(s["q"], s["n_new"], out=s["out"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _own_plan, "rope": _own_rope, "attn": _own_attn}[op](state)
    return {"plan": _plain_plan, "rope": _plain_rope, "attn": _plain_attn}[op](state)


# ------------------------------------------------------------------------------- floors
def work(case):
    c = case
    if c["op"] == "plan":
        past, new = _lengths(c)
        B, n = c["block"], c["batch"]
        fresh = sum(_blocks(p + k, B) - _blocks(p, B) for p, k in zip(past, new))
        fresh = int(fresh * min(1.0, c["spare"]))
        return {"bytes": 16 * n + 8 * fresh + 12 * n * max(1, max(new)) + 8, "flops": 0}
    e = 2 if c["dtype"] == "bf16" else 4
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    if c["op"] == "rope":
        live = c["rows"] - c["pad"]
        b = live * (hq + 2 * hkv) * d * e * 2 + c["rows"] * (12 if c["pages"] else 4)
        return {"bytes": b + c["rot"] * 4 + 8 * d,
                "flops": live * (hq + hkv) * (4 * d + 3 * c["rot"])}
    past, new = _lengths(c)
    held = sum(p + n for p, n in zip(past, new))
    pairs = sum(n * p + n * (n + 1) // 2 for p, n in zip(past, new))
    b = 2 * held * hkv * d * e + 2 * sum(new) * hq * d * e + 4 * sum(new) * hq
    b += 4 * sum(_blocks(p + n, c["block"]) for p, n in zip(past, new)) + 8 * c["batch"]
    return {"bytes": b, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------------------- in 64 bits
def _rotate64(x, gamma, positions, inv_freq, rot, interleaved):
    x = x.double()
    n = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * gamma.double()
    out = n.clone()
    i = torch.arange(rot // 2, device="cuda")
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       positions.double()[:, None] * inv_freq[None])[:, None]
    z = torch.complex(n[..., first], n[..., second]) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out


def exact(case, seed):
    if case["op"] == "plan":                 # whole numbers only
        return None
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        q, k, v = _split(s)
        a = (s["positions"], s["inv_freq"], c["rot"], c["interleaved"])
        q, k, v = _rotate64(q, s["q_gamma"], *a), _rotate64(k, s["k_gamma"], *a), v.double()
        if c["pages"]:
            kp, vp = s["k_pool"].double(), s["v_pool"].double()
            page, off = torch.div(s["slots"], c["block"], rounding_mode="floor"), s["slots"] % c["block"]
            kp.transpose(1, 2)[page, off] = k
            vp.transpose(1, 2)[page, off] = v
            return {"q": q, "k_pool": kp, "v_pool": vp}
        n = c["rows"] - c["pad"]
        for x in (q, k, v):
            x[n:] = 0
        return {"q": q, "k": k, "v": v}
    past, new = _lengths(c)
    hq, hkv, d, B = c["hq"], c["hkv"], c["d"], c["block"]
    g = hq // hkv
    out, lse = s["out"].double(), s["lse"].double()
    for b in range(c["batch"]):
        n, L = new[b], past[b] + new[b]
        pages = s["table"][b, :_blocks(L, B)].long()
        late = torch.arange(L, device="cuda")[None] > past[b] + torch.arange(n, device="cuda")[:, None]
        for h in range(hkv):
            K = s["k_pool"][pages, h].reshape(-1, d)[:L].double()
            V = s["v_pool"][pages, h].reshape(-1, d)[:L].double()
            for e in range(h * g, (h + 1) * g):
                x = s["q"][b, :n, e].double() @ K.T / math.sqrt(d)
                x[late] = -math.inf
                z = torch.logsumexp(x, 1)
                out[b, :n, e] = torch.exp(x - z[:, None]) @ V
                lse[b, :n, e] = z
    return {"out": out, "lse": lse}
