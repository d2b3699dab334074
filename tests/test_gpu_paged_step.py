"""The paged serving calls in a row, as a server makes them: blocks planned on the device,
q and k normed and rotated, a full-attention layer (pages written by slot, chunk attention)
and a sparse layer (append, decode) on the same block table; requests that end give their
blocks to others. Every step's outputs against the 64-bit forms of what was fed in."""
import math

import numpy as np
import pytest
import torch

from block_sparse_linear_b200 import (SplaBlockPool, SplaConfig, SplaDecodeCache, SplaPagedKV,
                                      qk_norm_rope)

from . import paged_ref as ref

pytestmark = pytest.mark.gpu

HQ, HKV, D, BLOCK, BATCH, MBP = 8, 2, 128, 64, 3, 12
PHYS = 26                                          # fewer than BATCH * MBP: requests can be refused


class Server:
    def __init__(self, seed):
        self.g = torch.Generator("cuda").manual_seed(seed)
        self.cfg = SplaConfig(num_q_heads=HQ, num_kv_heads=HKV, head_dim=D, block_size=BLOCK,
                              top_k=64)
        self.pool = SplaBlockPool.empty(BATCH, MBP, PHYS, BLOCK)
        self.lens = torch.zeros(BATCH, dtype=torch.int32, device="cuda")
        shape = (PHYS, HKV, BLOCK, D)
        pools = [torch.full(shape, math.nan, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
        self.full = SplaPagedKV(self.cfg, *pools, self.pool.block_table, self.lens)
        self.sparse = SplaDecodeCache(self.cfg, BATCH, self.pool.block_table, PHYS)
        assert self.sparse.block_table.data_ptr() == self.pool.block_table.data_ptr()
        self.inv = 1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
        self.qg, self.kg = (1 + 0.1 * torch.randn(D, device="cuda", generator=self.g) for _ in "qk")
        self.K = [np.zeros((0, HKV, D)) for _ in range(BATCH)]     # what each sequence was fed
        self.V = [np.zeros((0, HKV, D)) for _ in range(BATCH)]

    def step(self, n_new, max_new):
        n = torch.tensor(n_new, dtype=torch.int32, device="cuda")
        plan = self.pool.plan(self.lens, n, max_new)
        rows = BATCH * max_new
        qkv = torch.randn((rows, (HQ + 2 * HKV) * D), device="cuda", generator=self.g).bfloat16()
        q = qkv[:, :HQ * D].unflatten(1, (HQ, D))
        k = qkv[:, HQ * D:(HQ + HKV) * D].unflatten(1, (HKV, D))
        v = qkv[:, (HQ + HKV) * D:].unflatten(1, (HKV, D))
        norm = dict(positions=plan.positions, inv_freq=self.inv, q_gamma=self.qg, k_gamma=self.kg)
        # full-attention layer
        qr = qk_norm_rope(self.cfg, q, k, v, kv=self.full, slots=plan.slots, **norm)
        qr = qr.view(BATCH, max_new, HQ, D)
        out = self.full.chunk_attention(qr, plan.n_granted, lens=plan.lens_after)
        # sparse layer on the same tokens
        _, kr, vr = qk_norm_rope(self.cfg, q, k, v, **norm)
        kr, vr = (x.view(BATCH, max_new, HKV, D) for x in (kr, vr))
        self.sparse.append(kr, vr, plan.n_granted)
        self.lens.copy_(plan.lens_after)
        granted = plan.n_granted.tolist()
        last = (plan.n_granted.long() - 1).clamp(min=0)
        dec = self.sparse.decode(qr[torch.arange(BATCH, device="cuda"), last].contiguous())
        whole = self.sparse.chunk_attention(qr, plan.n_granted)
        for b, m in enumerate(granted):
            self.K[b] = np.concatenate([self.K[b], kr[b, :m].double().cpu().numpy()])
            self.V[b] = np.concatenate([self.V[b], vr[b, :m].double().cpu().numpy()])
        assert torch.equal(self.sparse.context_lens, self.lens)
        self.compare(qr, granted, out, whole, dec)
        return granted

    def compare(self, q, granted, out, whole, dec):
        assert torch.equal(out, whole)             # two layers, the same tokens
        for b, m in enumerate(granted):
            L = len(self.K[b])
            assert L == int(self.lens[b])
            if m == 0:
                continue
            for e in range(HQ):
                K, V = (torch.from_numpy(x[b][:, e // (HQ // HKV)]).cuda() for x in (self.K, self.V))
                o, _, to, _ = ref.chunk(q[b, :m, e].double(), K, V, L, 1 / math.sqrt(D),
                                        torch.bfloat16)
                assert ((out[b, :m, e].double() - o).abs() <= to).all()
                # every block is kept (top_k covers the table): the decode is exact attention too
                assert ((dec[b, e].double() - o[-1]).abs() <= to[-1]).all()

    def finish(self, b):
        keep = torch.full((BATCH,), 2 ** 30, dtype=torch.int32, device="cuda")
        keep[b] = 0
        self.pool.release(keep, self.lens)
        self.K[b], self.V[b] = self.K[b][:0], self.V[b][:0]
        # a sparse cache starts the sequence over: empty state, the shared length
        self.sparse.context_lens.copy_(self.lens)
        self.sparse.S[b], self.sparse.z[b] = 0, 0
        self.sparse.m[b] = -math.inf


def test_serving_steps():
    s = Server(1)
    assert s.step([300, 64, 1], 300) == [300, 64, 1]          # prompts, bulk append
    for _ in range(3):
        assert s.step([1, 1, 1], 1) == [1, 1, 1]              # decode
    assert s.step([5, 0, 5], 5) == [5, 0, 5]                  # drafts
    s.finish(0)
    assert s.step([100, 129, 3], 129) == [100, 129, 3]
    # 9 blocks are asked for by the first, the rest do not fit; nothing overtakes
    used = PHYS - int(s.pool.free_count)
    assert used == sum(-(-int(n) // BLOCK) for n in s.lens)
    got = s.step([600, 500, 500], 600)
    assert got[0] == 600 and 0 in got and s.pool.status() == 0x20
    s.pool.dev_status.zero_()
    for b in range(BATCH):
        s.finish(b)
    assert int(s.pool.free_count) == PHYS
    assert s.step([64, 1, 200], 200) == [64, 1, 200]
    assert s.pool.status() == 0 and s.full.status() == 0 and s.sparse.status() == 0


def test_decode_steps_in_one_graph():
    """Plan, norm, page write, chunk attention and the length update captured once and replayed:
    blocks are opened on the device, no host round trip."""
    s = Server(2)
    s.step([60, 63, 10], 63)
    one = torch.ones(BATCH, dtype=torch.int32, device="cuda")
    q = torch.zeros((BATCH, HQ, D), device="cuda", dtype=torch.bfloat16)
    k, v = (torch.zeros((BATCH, HKV, D), device="cuda", dtype=torch.bfloat16) for _ in "kv")
    res = {}

    def body():
        plan = s.pool.plan(s.lens, one, 1)
        qr = qk_norm_rope(s.cfg, q, k, v, plan.positions, s.inv, s.qg, s.kg, kv=s.full,
                          slots=plan.slots)
        res["q"] = qr
        res["out"] = s.full.chunk_attention(qr.view(BATCH, 1, HQ, D), plan.n_granted,
                                            lens=plan.lens_after)
        s.lens.copy_(plan.lens_after)

    before = s.lens.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        s.full.chunk_attention(q.view(BATCH, 1, HQ, D), torch.zeros_like(one))   # makes the workspace
        with torch.cuda.graph(graph, stream=side):
            body()
    torch.cuda.synchronize()
    assert torch.equal(s.lens, before)
    for i in range(7):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device="cuda", generator=s.g))
        pos = s.lens.clone()
        graph.replay()
        torch.cuda.synchronize()
        kr, _ = ref.norm_rope(k.double(), s.kg.double(), pos, s.inv, D, False, 1e-6)
        for b in range(BATCH):
            # the key the kernel rounded is within a step of the exact one: read it back
            p = int(pos[b])
            page = int(s.pool.block_table[b, p // BLOCK])
            got = s.full.k_pool[page, :, p % BLOCK].double()
            assert ((got - kr[b]).abs() <= 2 ** -8 * kr[b].abs() + 1e-5).all()
            s.K[b] = np.concatenate([s.K[b], got[None].cpu().numpy()])
            s.V[b] = np.concatenate([s.V[b], v[b][None].double().cpu().numpy()])
            for e in range(HQ):
                K, V = (torch.from_numpy(x[b][:, e // 4]).cuda() for x in (s.K, s.V))
                o, _, to, _ = ref.chunk(res["q"][b, e][None].double(), K, V, p + 1,
                                        1 / math.sqrt(D), torch.bfloat16)
                assert ((res["out"][b, 0, e].double() - o[0]).abs() <= to[0]).all()
    assert s.pool.status() == 0 and s.full.status() == 0
    assert s.lens.tolist() == (before + 7).tolist()
