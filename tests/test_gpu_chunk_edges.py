"""spla_chunk_attention where its parts meet: infinities and NaN in parts of little weight and
in units that follow one another, splits of long contexts and of large batches."""
import pytest
import torch

from .test_gpu_chunk_attention import INF, NAN, build, check, run

pytestmark = pytest.mark.gpu


def put(kv, pool, b, s, i, x):
    """Element i (a slice: all) of every KV head's token s of sequence b."""
    pool[kv.block_table[b, s // kv.cfg.block_size].long(), :, s % kv.cfg.block_size, i] = x


def one_query(q):
    """The same query in every row, so that one key can outweigh all others for all of them."""
    q.copy_(q[:1, :1, :1].expand_as(q).clone())
    return q[0, 0, 0]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,n", [(64, 1), (128, 5), (64, 150)])
def test_nan_values_far_from_the_weight_of_a_long_sequence(dtype, d, n):
    """NaN and infinities early in V, a logit hundreds of nats above all others thousands of
    tokens later: the early tokens lie in other thread blocks' partials, whose weights are zero
    in fp32. A NaN is seen all the same; an infinity gives itself or NaN."""
    L = 20000
    kv, q = build(40, [L], n, 4, 1, d, 64, dtype)
    big = 40 * one_query(q)
    put(kv, kv.k_pool, 0, L - 200, slice(None), big)
    put(kv, kv.v_pool, 0, 10, 3, NAN)
    put(kv, kv.v_pool, 0, 9000, 4, NAN)
    out, lse = run(kv, q, [n])
    check(kv, q, [n], [L], out, lse)
    assert torch.isnan(out[0, :, :, 3:5]).all()
    put(kv, kv.v_pool, 0, 700, 5, INF)
    out, _ = run(kv, q, [n])
    assert not torch.isfinite(out[0, :, :, 3:6]).any()
    assert torch.isfinite(out[0, :, :, :3]).all() and torch.isfinite(out[0, :, :, 6:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 40])
def test_nan_values_of_little_weight_within_a_unit(dtype, n):
    """The same in sequences of three steps, several whole ones a thread block: NaN in the step
    of one softmax stream (or warp) and the large logit in another's, either way round."""
    batch, L = 320, 330
    kv, q = build(41, [L] * batch, n, 4, 1, 64, 64, dtype)
    big = 40 * one_query(q)
    for b in range(batch):
        key, nan = ((20, 130), (130, 20), (20, 70), (200, 10))[b % 4]
        put(kv, kv.k_pool, b, key, slice(None), big)
        put(kv, kv.v_pool, b, nan, b % 64, NAN)
    out, lse = run(kv, q, [n] * batch)
    for b in range(0, batch, 7):
        check(kv, q, [n if x == b else 0 for x in range(batch)], [L] * batch,
              torch.where(torch.arange(batch, device="cuda")[:, None, None, None] == b, out, 5.0),
              torch.where(torch.arange(batch, device="cuda")[:, None, None] == b, lse, 5.0))
    want = torch.zeros((batch, 64), dtype=torch.bool, device="cuda")
    want[torch.arange(batch), torch.arange(batch) % 64] = True
    assert torch.equal(torch.isnan(out), want[:, None, None].expand_as(out))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,max_new", [(64, 1), (128, 1), (64, 20), (128, 60)])
def test_infinities_of_units_that_follow_one_another(dtype, d, max_new):
    """Hundreds of sequences of a step or two, several a thread block, each with an infinity or
    NaN of its own in V: no row misses its own or has its neighbours'."""
    batch, kinds = 700, (INF, -INF, NAN)
    lens = [1 + (53 * b) % (128 if b % 5 else 250) for b in range(batch)]
    n_new = [min(L, 1 + b % max_new) for b, L in enumerate(lens)]
    kv, q = build(42, lens, max_new, 4, 2, d, 64, dtype)
    want = torch.zeros((batch, d), device="cuda")
    for b, (L, n) in enumerate(zip(lens, n_new)):
        at, x = (L - n) * (b % 7) // 6, kinds[b % 3]      # a token that every query sees
        put(kv, kv.v_pool, b, at, (11 * b) % d, x)
        want[b, (11 * b) % d] = x
    live = torch.arange(max_new, device="cuda")[None] < torch.tensor(n_new, device="cuda")[:, None]
    for _ in range(5):
        out, _ = run(kv, q, n_new)
        got = torch.where(torch.isfinite(out), 0.0, out.float())
        expect = torch.where(live[..., None, None], want[:, None, None], 0.0).expand_as(got)
        assert torch.equal(got.nan_to_num(nan=7.0), expect.nan_to_num(nan=7.0))
    assert kv.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinities_that_only_later_queries_see(dtype):
    """Chunks of two query tiles that follow one another in a thread block, each with infinities
    in the tokens that only its second tile's last queries see: its earlier rows, and those of
    the next chunk, have none of them."""
    batch, G, d, n = 330, 4, 64, 64                       # 256 rows: two tiles of 32 tokens
    lens = [n + 64 * (b % 4) + 32 * (b % 2) for b in range(batch)]
    kv, q = build(43, lens, n, G, 1, d, 64, dtype)
    dims = torch.arange(batch, device="cuda") * 7 % d
    for b, L in enumerate(lens):
        put(kv, kv.v_pool, b, L - 1 - b % 16, int(dims[b]), INF)
    first = n - 1 - torch.arange(batch, device="cuda") % 16     # the first query that sees it
    seen = torch.arange(n, device="cuda")[None] >= first[:, None]
    want = torch.zeros((batch, n, G, d), device="cuda")
    want[torch.arange(batch), :, :, dims] = torch.where(seen, INF, 0.0)[..., None].expand(-1, -1, G)
    for _ in range(5):
        out, _ = run(kv, q, [n] * batch)
        assert torch.equal(torch.where(torch.isfinite(out), 0.0, out.float()), want)
    assert kv.status() == 0


# ---- every token once: queries of zeros weigh all tokens alike, values count them by place
def marked(kv):
    """Values that name the 64 tokens they belong to: of KV head 0 the place modulo d, of head
    1 the next digit. Slots past the lengths stay NaN."""
    d, half = kv.cfg.head_dim, kv.cfg.block_size // 64
    eye = torch.eye(d, dtype=kv.v_pool.dtype, device="cuda")
    for b in range(kv.c.batch):
        L = int(kv.context_lens[b])
        pages = kv.block_table[b, :-(-L // kv.cfg.block_size)].long()
        i = torch.arange(len(pages) * half, device="cuda")
        for h, digit in enumerate((i % d, i // d % d)):
            rows = eye[digit][:, None].expand(-1, 64, -1).reshape(len(pages), kv.cfg.block_size, d)
            old = kv.v_pool[pages, h]
            kv.v_pool[pages, h] = torch.where(torch.isnan(old), old, rows)


def expected_counts(T, d):
    """How many of the first T tokens bear each mark: float64 [...][2][d]."""
    I, r = (T // 64)[..., None], (T % 64)[..., None].double()
    j = torch.arange(d, device=T.device)
    low = I // d + (j < I % d)
    high = I // (d * d) * d + (I % (d * d) - j * d).clamp(0, d)
    part = torch.stack((j == I % d, j == I // d % d), -2) * r[..., None]
    return torch.stack((low, high), -2) * 64 + part


def check_marks(kv, n_new, lens, max_new, rounds=1):
    """q = 0: every probability is 1 and every sum a whole number below 2^24, so l and O are
    exact in fp32. The result is O (1 / l): two roundings of 2^-24, and the store's; lse is
    log2 l to a unit of its last place (2^-23) times ln 2, two more roundings."""
    d, G = kv.cfg.head_dim, kv.cfg.num_q_heads // 2
    q = torch.zeros((len(lens), max_new, 2 * G, d), dtype=kv.v_pool.dtype, device="cuda")
    marked(kv)
    n, L = (torch.tensor(x, device="cuda")[:, None] for x in (n_new, lens))
    t = torch.arange(max_new, device="cuda")[None]
    live = t < n
    seen = torch.where(live, L - n + t + 1, 1)
    counts = expected_counts(seen, d)
    assert torch.equal(counts.sum(-1), seen[..., None].expand(-1, -1, 2).double())
    want = (counts / seen[..., None, None])[:, :, :, None].expand(-1, -1, -1, G, -1).flatten(2, 3)
    tol = want * (torch.finfo(q.dtype).eps / 2 * (q.dtype != torch.float32) + 2.0 ** -22)
    want = torch.where(live[..., None, None], want, 5.0)
    wz = torch.where(live, seen.double().log(), 5.0)[..., None]
    for _ in range(rounds):
        out, lse = run(kv, q, n_new)
        bad = ((out.double() - want).abs() > torch.where(live[..., None, None], tol, 0.0)).nonzero()
        assert len(bad) == 0, bad[:4]
        bad = (lse.double() - wz).abs() > torch.where(live[..., None], 2.0 ** -22 * wz, 0.0)
        assert not bad.any(), bad.nonzero()[:4]
    assert kv.status() == 0


@pytest.mark.parametrize("dtype,d,block,lens,n_new", [
    ("bf16", 64, 64, [200003], [1]), ("bf16", 128, 128, [200003], [40]),
    ("f32", 64, 64, [60001], [1]), ("f32", 128, 64, [60001], [40]),
    ("bf16", 64, 64, [200003, 90, 130001], [1, 1, 1]), ("bf16", 128, 64, [200003, 90, 130001], [17, 3, 9]),
    ("f32", 64, 64, [100001, 90, 65003], [1, 1, 0]), ("f32", 64, 128, [100001, 90, 65003], [17, 17, 17]),
    ("bf16", 64, 128, [1048501], [1]), ("bf16", 64, 64, [70001], [1500]),
    ("bf16", 128, 64, [262144, 4096, 131072, 8191, 65537, 16385, 32767, 100000],
     [1, 33, 5, 2, 17, 1, 8, 64]),
    ("f32", 64, 64, [5000, 40000, 777, 20011], [500, 200, 777, 1]),
])
def test_every_token_counts_once(dtype, d, block, lens, n_new):
    """Long contexts over the whole GPU: a step that the split loses or takes twice changes lse
    and the counts by far more than their roundings."""
    kv, _ = build(44, lens, 1, 4, 2, d, block, dtype)
    check_marks(kv, n_new, lens, max(n_new))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch", [400, 1000, 2500])
@pytest.mark.parametrize("max_new", [1, 4, 70])
def test_every_token_of_hundreds_of_sequences(dtype, batch, max_new):
    """More sequences than a thread block has threads to scan them, some without new tokens, the
    chunks of one query tile and of two."""
    lens = [1 + (97 * i * i + 13 * i) % (90 if i % 17 else 1500) for i in range(batch)]
    n_new = [0 if i % 6 == 5 else min(L, 1 + (i * 31) % max_new) for i, L in enumerate(lens)]
    n_new[-1] = min(lens[-1], max_new)
    kv, _ = build(45, lens, 1, 4, 2, 64, 64, dtype)
    check_marks(kv, n_new, lens, max_new)
