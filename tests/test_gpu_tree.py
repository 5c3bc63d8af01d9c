"""GPU parity of a verify round over trees of drafted tokens against the fp64 oracle
(oracle/tree_oracle.py), through the binding.

Tree attention's tolerances are the paged attention's (test_gpu_paged.py: the same
sums in the same precision). Walks and moves are exact. Sampling is exact but where a
running sum comes within BORDER of a threshold that it is compared with, relative to
the sum of all weights: there a neighbour may be drawn, or one token more or less be
kept. A weight is within 2^-33 of its value (exponent 2^-36, polynomial 2^-35, the
last bits of the table's product 2^-36 and 2^-43, all of at least a half), plus a unit
of 2^-44 that each token adds to a sum: BORDER = 2^-32 + vocab 2^-44. prob: the weight and the sum
2^-33 each, the sum's units (it is 1 at least), vocab 2^-44, and the rounding to fp32, 2^-24:
2^-23 + vocab 2^-44 covers them."""

import math

import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from oracle import tree_oracle as T
from test_gpu_paged import Setup, host, mask_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from block_speculative_decoding_dflash_gb300 import build
    build.build()
    from block_speculative_decoding_dflash_gb300 import binding
    return binding


def random_tree(rng, n, deep=0.4):
    """Ends of a random tree of n rows in depth-first order."""
    open_rows, end = [], [n] * n
    for i in range(n):
        d = 0 if i == 0 else len(open_rows) if rng.random() < deep else int(rng.integers(1, len(open_rows) + 1))
        while len(open_rows) > d:
            end[open_rows.pop()] = i
        open_rows.append(i)
    return end


# ---- attention -------------------------------------------------------------------------


class Trees(Setup):
    """Setup whose new rows are trees: positions are the committed length plus the depth."""

    def __init__(self, B, lens, *a, shape="random", **kw):
        super().__init__(B, lens, *a, **kw)
        rng = np.random.default_rng(len(lens) + lens[0][0])
        lead = int(self.start[0])
        ends, ps = [0] * lead, self.k.shape[2]
        for s, (n, length) in enumerate(lens):
            end = [n] * n if shape == "chain" else [n] + list(range(2, n + 1)) if shape == "star" and n else random_tree(rng, n)
            ends += end
            depth = T.ancestors(end).sum(1) - 1
            first = int(self.q_pos[int(self.start[s])]) if n else 0
            for i in range(n):
                row = length - n + i
                self.pos[int(self.table[s, row // ps]), :, row % ps] = first + int(depth[i])
                self.q_pos[int(self.start[s]) + i] = first + int(depth[i])
        self.end = torch.tensor(ends + [0] * (self.rows - len(ends)), dtype=torch.int32)

    def call(self, cache, **mask):
        out = torch.full((self.rows, self.nq, self.hd), 77.0, dtype=self.dt, device="cuda")
        lse = torch.full((self.rows, self.nq), 77.0, device="cuda")
        dev = {n: x.cuda() if torch.is_tensor(x) else x for n, x in mask.items()}
        cache.tree_attention(self.q.cuda(), self.q_pos.cuda(), self.start.cuda(), self.end.cuda(), out, lse=lse, **dev)
        torch.cuda.synchronize()
        return out, lse

    def check(self, cache, **mask):
        out, lse = self.call(cache, **mask)
        opts = {n: x.numpy().astype(np.float64) if n == "slopes" and x is not None else x.numpy() if n == "prefix" and x is not None else x
                for n, x in mask.items() if n != "max_len"}
        want, want_lse, mag = T.attention(self.oracle(), host(self.q), self.q_pos.numpy(), self.start.numpy(), self.end.numpy(), self.scale, **opts)
        slopes = mask.get("slopes")
        self.compare(host(out), host(lse), want, want_lse, mag, mask.get("softcap", 0.0), None if slopes is None else slopes.numpy())
        return out, lse


SHAPES = [
    # lens (new, cached), nq, nkv, hd, page rows, dtype
    ([(1, 1)], 4, 2, 16, 8, "f32"),
    ([(1, 1)], 8, 8, 64, 16, "bf16"),
    ([(16, 300)], 32, 8, 128, 64, "bf16"),
    ([(16, 16)], 16, 8, 128, 32, "bf16"),
    ([(7, 133), (0, 40), (1, 128), (12, 12), (0, 0), (9, 260)], 8, 4, 64, 16, "bf16"),
    ([(64, 700), (30, 257)], 32, 8, 128, 16, "bf16"),
    ([(150, 300), (3, 640), (200, 200)], 14, 2, 128, 128, "bf16"),
    ([(33, 500)], 5, 1, 96, 256, "bf16"),
    ([(129, 129)], 6, 1, 80, 8, "bf16"),
    ([(40, 200), (2, 31)], 4, 4, 256, 16, "bf16"),
    ([(600, 900)], 4, 1, 64, 32, "bf16"),
    ([(2, 70)], 128, 1, 64, 16, "bf16"),
    ([(9, 200), (20, 65), (0, 12)], 16, 8, 128, 16, "f32"),
    ([(65, 130)], 12, 4, 80, 32, "f32"),
    ([(20, 150)], 2, 1, 200, 8, "f32"),
]
MASKS = [dict(), dict(window=20), dict(window=3, prefix=6), dict(softcap=5.0), dict(slopes=True), dict(causal=False, window=16, softcap=20.0, slopes=True)]


@pytest.mark.parametrize("mask", MASKS, ids=lambda m: "-".join(m) or "plain")
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{s[0][0][0]}of{s[0][0][1]}-{s[1]}_{s[2]}x{s[3]}-{s[4]}-{s[5]}")
def test_tree_attention(B, shape, mask):
    lens, nq, nkv, hd, ps, dtype = shape
    s = Trees(B, lens, nq, nkv, hd, ps, dtype, seed=len(lens) + hd, lead=2, tail=3)
    s.check(s.device(), **mask_of(mask, nq, len(lens)))
    assert int(s.status) == 0


@pytest.mark.parametrize("dtype,hd,nq", [("bf16", 128, 8), ("bf16", 64, 6), ("f32", 64, 4), ("bf16", 256, 2)])
@pytest.mark.parametrize("n", [1, 5, 40, 140])
@pytest.mark.parametrize("shape", ["star", "random"])
def test_trees_in_an_evicted_cache(B, dtype, hd, nq, n, shape):
    """The older rows in no order, other positions in every kv head; a star's leaves see the root and themselves."""
    s = Trees(B, [(n, 400), (n, 150)], nq, 2, hd, 32, dtype, seed=3, kept=True, shape=shape)
    cache = s.device()
    for m in (dict(), dict(window=350)):
        s.check(cache, **m)


@pytest.mark.parametrize("dtype,hd,nq", [("bf16", 128, 8), ("bf16", 64, 16), ("f32", 128, 4), ("bf16", 256, 2)])
@pytest.mark.parametrize("n,length", [(1, 300), (16, 700), (100, 100), (300, 1000)])
def test_a_chain_is_causal_attention_to_the_bit(B, dtype, hd, nq, n, length):
    s = Trees(B, [(n, length), (n, n)], nq, 2, hd, 16, dtype, seed=n, shape="chain")
    cache = s.device()
    for m in (dict(), dict(window=50), dict(softcap=10.0)):
        out, lse = s.call(cache, **m)
        want, want_lse = torch.full_like(out, 77.0), torch.full_like(lse, 77.0)
        cache.attention(s.q.cuda(), s.q_pos.cuda(), s.start.cuda(), want, lse=want_lse, **m)
        # (whether a tile counts as partly seen decides when a maximum is raised, not what is summed)
        assert torch.allclose(out.float(), want.float(), rtol=2.0 ** -7, atol=2.0 ** -9) and torch.allclose(lse, want_lse, rtol=1e-6, atol=1e-5)


@pytest.mark.parametrize("mask", [dict(), dict(softcap=20.0), dict(window=50)], ids=lambda m: "-".join(m) or "plain")
@pytest.mark.parametrize("dtype,hd,nq", [("bf16", 128, 8), ("bf16", 64, 6), ("f32", 128, 4), ("bf16", 200, 4)])
@pytest.mark.parametrize("n", [9, 70, 200])
def test_other_branches_have_no_say(B, dtype, hd, nq, n, mask):
    """Rows of other branches, infinite and NaN ones among them, do not reach a row's result (that branch's own queries see
    them, and share warps with these: when a maximum is raised may differ, so bits may)."""
    results = []
    for fill in (0.0, 1e4, math.inf, math.nan):
        s = Trees(B, [(n, n + 77)], nq, 2, hd, 16, dtype, seed=5)
        end = [n] + [n // 2] + [x if 2 <= i < n // 2 else n for i, x in enumerate([min(int(e), n // 2) for e in s.end])][2:]
        end[n // 2] = n                                    # two branches: 1 .. n / 2 - 1 and n / 2 .. n - 1
        s.end = torch.tensor(end, dtype=torch.int32)
        rows = 77 + torch.arange(n // 2, n)
        page, j = s.table[0, rows // 16].long(), rows % 16
        for x in (s.k, s.v):
            x[page, :, j] = fill
        out, lse = s.call(s.device(), **mask)
        results.append((out[: n // 2].clone(), lse[: n // 2].clone()))
        assert torch.isfinite(out[: n // 2]).all()
    for out, lse in results[1:]:
        assert torch.allclose(out.float(), results[0][0].float(), rtol=2.0 ** -7, atol=2.0 ** -9) and torch.allclose(lse, results[0][1], rtol=1e-6, atol=1e-5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("end", [[0] * 6, [-5, 2, 100, 3, 1 << 30, 6], [6, 1, 2, 3, 4, 5], [3, 6, 4, 5, 5, 6]])
def test_ends_that_no_tree_has(B, dtype, end):
    """Whatever the ends are, row i sees row j iff j <= i < end[j] (or j = i)."""
    s = Trees(B, [(6, 100)], 4, 2, 64, 16, dtype, seed=9)
    out = {}
    for name, e in (("given", end), ("cut", [min(max(x, j + 1), 6) for j, x in enumerate(end)])):
        s.end = torch.tensor(e, dtype=torch.int32)
        out[name] = s.call(s.device())
    assert torch.equal(out["given"][0], out["cut"][0]) and torch.equal(out["given"][1], out["cut"][1])
    want, want_lse, mag = T.attention(s.oracle(), host(s.q), s.q_pos.numpy(), s.start.numpy(), [6] * 6, s.scale)   # for the tolerance alone
    o = s.oracle()
    where = P.rows_of(o, 0)
    for i in range(6):
        seen = [r for r in range(100) if r < 94 or r - 94 == i or r - 94 < i < min(end[r - 94], 6)]
        page, j = np.array([where[r][0] for r in seen]), np.array([where[r][1] for r in seen])
        for head in range(4):
            h = head // 2
            ok = o["pos"][page, h, j] <= int(s.q_pos[i])
            t = host(s.q)[i, head] @ o["k"][page[ok], h, j[ok]].T * s.scale
            e = np.exp(t - t.max())
            want[i, head], mag[i, head] = e @ o["v"][page[ok], h, j[ok]] / e.sum(), e @ np.abs(o["v"][page[ok], h, j[ok]]) / e.sum()
            want_lse[i, head] = t.max() + np.log(e.sum())
    s.compare(host(out["cut"][0]), host(out["cut"][1]), want, want_lse, mag, 0.0, None)


@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("f32", 64), ("bf16", 256)])
def test_tree_attention_reports_what_cannot_be(B, dtype, hd):
    s = Trees(B, [(5, 60), (3, 40)], 4, 2, hd, 16, dtype, seed=2)
    s.table[0, 1] = 1 << 20                             # a page outside the pool
    cache = s.device()
    out, _ = s.call(cache)
    assert int(s.status) == B.PAGED_BAD_PAGE and torch.isfinite(out).all()
    s = Trees(B, [(5, 60), (3, 40)], 4, 2, hd, 16, dtype, seed=2)
    s.length[1] = 2                                     # fewer rows than new ones
    cache = s.device()
    out, _ = s.call(cache)
    assert int(s.status) == B.PAGED_BAD_ROWS and torch.isfinite(out).all()


@pytest.mark.parametrize("nq,nkv,hd,dtype,window", [(32, 8, 128, "bf16", 0), (8, 1, 64, "bf16", 0), (32, 8, 128, "bf16", 3000), (4, 2, 64, "f32", 0)])
@pytest.mark.parametrize("n", [1, 20, 64])
def test_trees_after_long_texts_many_times(B, nq, nkv, hd, dtype, window, n):
    """Rows split over many CTAs, with a workspace or a cluster; the same bits every time."""
    s = Trees(B, [(n, 6000), (n, 300)], nq, nkv, hd, 64, dtype, seed=n)
    cache = s.device()
    first = s.check(cache, window=window, max_len=6000)
    for max_len in (0, 6000):
        outs = [s.call(cache, window=window, max_len=max_len) for _ in range(5)]
        assert all(torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1]) for o in outs)
    assert torch.equal(outs[0][0], first[0]) and int(s.status) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,spare", [([(3, 1100 + 9 * i) for i in range(36)], 1), ([(1 + i % 3, 30 + i % 9) for i in range(270)], 70),
                                        ([(1 + 5 * (i % 3), 150 * i + 60) for i in range(24)], 0)])
def test_trees_of_many_sequences(B, lens, spare, dtype):
    """More sequences than are put in order, more than are cut into segments, and all lengths in one call."""
    s = Trees(B, lens, 2, 1, 64, 16, dtype, seed=1, spare=spare, lead=1, tail=2)
    s.check(s.device())
    assert int(s.status) == 0


def test_more_query_tiles_than_segments_are_made_for(B):
    s = Trees(B, [(1500, 1600)], 128, 8, 64, 16, seed=1, shape="chain")
    cache = s.device()
    out, lse = s.call(cache)
    want, want_lse = torch.full_like(out, 77.0), torch.full_like(lse, 77.0)
    cache.attention(s.q.cuda(), s.q_pos.cuda(), s.start.cuda(), want, lse=want_lse)
    assert torch.allclose(out.float(), want.float(), rtol=2.0 ** -7, atol=2.0 ** -9) and torch.allclose(lse, want_lse, rtol=1e-6, atol=1e-5)


@pytest.mark.parametrize("starts", [[0, 9, 4, 12], [12, 5, 9, 0], [-3, 40, 50, 60], [5, 5, 5, 5]])
def test_row_ranges_that_cannot_be(B, starts):
    """Descending and overlong ranges are cut; rows in none of them are not written."""
    s = Trees(B, [(4, 2000), (4, 300), (4, 1500)], 4, 2, 64, 16, seed=4)
    s.start = torch.tensor(starts, dtype=torch.int32)
    out, lse = s.call(s.device())
    held = {r for a, b in zip(starts, starts[1:]) for r in range(max(a, 0), min(b, 12))}
    free = [r for r in range(12) if r not in held]
    assert (out[free] == 77).all() and (lse[free] == 77).all()


# ---- sampling ----------------------------------------------------------------------------


def border(vocab):
    return 2.0 ** -32 + vocab * 2.0 ** -44


def draw(B, logits, u, **par):
    rows = logits.shape[0]
    token = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    prob = torch.full((rows,), -7.0, device="cuda")
    dev = {n: torch.as_tensor(x, dtype=torch.int32 if n == "top_k" else torch.float32).cuda() for n, x in par.items()}
    B.sample(logits, torch.as_tensor(u, dtype=torch.float32).cuda(), token, prob=prob, **dev)
    torch.cuda.synchronize()
    return token.cpu().numpy(), prob.double().cpu().numpy()


def check_draws(B, logits, u, near_allowed=0, **par):
    """Every row against the oracle; at most near_allowed rows may come so near a border that either side is right."""
    token, prob = draw(B, logits, u, **par)
    x, vocab = host(logits), logits.shape[1]
    u32 = np.asarray(u, dtype=np.float32)
    p32 = {n: np.asarray(v, dtype=np.int64 if n == "top_k" else np.float32) for n, v in par.items()}
    largest = float(torch.finfo(logits.dtype).max)
    near = 0
    for r in range(len(x)):
        want, p, margin = T.sample(x[r], float(u32[r]), **{n: (int(v[r]) if n == "top_k" else float(v[r])) for n, v in p32.items()}, largest=largest)
        if margin <= border(vocab) and want != token[r]:
            near += 1
            continue
        assert token[r] == want, f"row {r}: {token[r]} instead of {want} ({ {n: v[r] for n, v in p32.items()} }, u {u32[r]}, margin {margin:.3g})"
        assert abs(prob[r] - p) <= (2.0 ** -23 + vocab * 2.0 ** -44) * p, f"row {r}: prob {prob[r]} instead of {p}"
    assert near <= near_allowed


def logits_like(rows, vocab, dtype, seed, sigma=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, vocab, generator=g) * sigma).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()


FILTERS = [dict(), dict(temperature=0.7), dict(top_k=40), dict(top_p=0.9), dict(min_p=0.05), dict(temperature=1.3, top_k=500, top_p=0.8, min_p=0.01),
           dict(top_k=1), dict(top_p=0.0), dict(min_p=1.0), dict(temperature=0.0), dict(temperature=3.0, top_p=0.999), dict(top_k=100, top_p=0.5),
           dict(temperature=1e-3), dict(temperature=100.0, top_k=7), dict(top_p=0.95, min_p=0.3)]


@pytest.mark.parametrize("filters", FILTERS, ids=lambda f: "-".join(f"{n}{v}" for n, v in f.items()) or "plain")
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [1, 2, 9, 1000, 1024, 8193, 65537])
def test_sample(B, vocab, dtype, filters):
    rows = 24 if vocab < 10000 else 6
    u = np.random.default_rng(vocab).random(rows, dtype=np.float32)
    u[:3] = 0.0, 1 - 2.0 ** -24, 0.5
    check_draws(B, logits_like(rows, vocab, dtype, vocab), u, **{n: [v] * rows for n, v in filters.items()})


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [202048, 262144, 1 << 20])
def test_sample_large_vocabularies(B, dtype, vocab):
    """Rows that fill the shared memory of a cluster, and rows that do not fit it."""
    x = logits_like(6, vocab, dtype, 1)
    x[0] /= 10                                          # nearly flat
    x[1, 12345] = 40.0                                  # nearly certain
    x[2, ::2] = -math.inf
    u = [0.31, 0.9999, 0.77, 0.5, 0.123, 0.999]
    check_draws(B, x, u, near_allowed=1, temperature=[1.0, 1.0, 0.8, 1.0, 0.0, 2.0], top_p=[1.0, 1.0, 0.9, 0.95, 1.0, 0.6], top_k=[0, 0, 0, 50000, 0, 0])
    check_draws(B, x, u, near_allowed=1, top_k=[5, 1000, 3000, 64, 100000, vocab], min_p=[0.0, 0.0, 0.0, 0.1, 1e-4, 0.0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [5, 300, 20000])
def test_sample_ties_go_to_the_lowest_id(B, dtype, vocab):
    """Few different logits, so that every filter cuts within equal ones, whole rows of one value, and zeros of both signs."""
    rows = 40
    g = torch.Generator().manual_seed(vocab)
    x = torch.randint(0, 4, (rows, vocab), generator=g).float()
    x[0] = 2.0
    x[1] = torch.where(torch.rand(vocab, generator=g) < 0.5, 0.0, -0.0)
    x[2] = -1e4
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    r = np.random.default_rng(7)
    u = r.random(rows, dtype=np.float32)
    k = r.integers(1, vocab + 3, rows)
    p = r.random(rows, dtype=np.float32)
    check_draws(B, x, u, top_k=k)
    check_draws(B, x, u, top_p=p)
    check_draws(B, x, u, top_k=k, top_p=p, min_p=r.random(rows, dtype=np.float32))
    check_draws(B, x, u, top_k=np.full(rows, 3))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [300, 4100, 40000])
def test_sample_of_logits_near_zero(B, dtype, vocab):
    """Logits of both signs down to 2^-20, all of a row, beside larger ones, or with the largest at 2^-9."""
    rows = 24
    g = torch.Generator().manual_seed(vocab + 1)
    x = torch.exp2(torch.rand(rows, vocab, generator=g) * 12 - 20) * (torch.randint(0, 2, (rows, vocab), generator=g) * 2 - 1)
    x[8:16, ::3] = torch.randn(8, vocab, generator=g)[:, ::3] * 2
    x[16:] = x[16:].clamp(max=2.0 ** -9)
    x[16:, vocab // 2] = 2.0 ** -9
    x[::4, 1::5] = 0.0
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    r = np.random.default_rng(vocab)
    u, p = r.random(rows, dtype=np.float32), r.random(rows, dtype=np.float32)
    check_draws(B, x, u, near_allowed=1, top_p=p)
    check_draws(B, x, u, near_allowed=1, top_k=r.integers(257, vocab + 3, rows), temperature=0.05 + r.random(rows, dtype=np.float32))
    check_draws(B, x, u, near_allowed=1, top_p=p, top_k=r.integers(1, vocab + 3, rows), min_p=r.random(rows, dtype=np.float32) * np.float32(0.5))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [17, 4100])
def test_sample_rows_with_infinities_and_nan(B, dtype, vocab):
    big = float(torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).max)
    x = logits_like(12, vocab, dtype, 3)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, : vocab - 1] = -math.inf
    x[3, ::2] = math.nan
    x[4, 3] = x[4, 9] = math.inf
    x[5] = math.inf
    x[6] = -big
    x[7, 1:] = -big                                     # a mask of the type's lowest value
    x[8, 5] = big
    x[9, ::3] = -math.inf
    x[9, 1::3] = math.nan
    x[10] = 0.0
    x[10, 2] = 1e-38
    x[11, 4] = -math.nan
    u = np.linspace(0.02, 0.97, 12, dtype=np.float32)
    for par in (dict(), dict(top_k=[3] * 12), dict(top_p=[0.6] * 12), dict(min_p=[0.2] * 12), dict(temperature=[0.0] * 12), dict(temperature=[1e30] * 12),
                dict(temperature=[math.inf] * 12, top_p=[0.3] * 12)):
        if "temperature" in par and par["temperature"][0] > 1e20:
            rows = [i for i in range(12) if i not in (6, 7, 8)]   # (distances that fp32 does not reach)
            check_draws(B, x[rows].contiguous(), u[rows], **{n: v[: len(rows)] for n, v in par.items()})
        else:
            check_draws(B, x, u, **par)


def test_sample_parameters_out_of_range(B):
    """What the header says of each."""
    x = logits_like(16, 500, "bf16", 4)
    nan, inf = math.nan, math.inf
    t = [0.0, -1.0, nan, 1e-30, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, inf, 1.0]
    k = [0, 0, 0, 0, -3, 501, 500, 1 << 30, 0, 0, 0, 0, 0, 0, 0, 0]
    p = [1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, nan, 7.0, -1.0, 1.0, 1.0, 1.0, 1.0, 1.0]
    m = [0.0] * 11 + [nan, -1.0, 3.0, 0.0, 0.0]
    u = [0.3] * 16
    for shift in (u, [nan] * 16, [-0.5] * 16, [1.0] * 16, [inf] * 16):
        check_draws(B, x, shift, temperature=t, top_k=k, top_p=p, min_p=m)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset,stride", [(0, 1003), (1, 1003), (3, 1040), (7, 5001)])
def test_sample_rows_that_start_anywhere(B, dtype, offset, stride):
    """Bases and strides of any number of elements; what lies between the rows is infinite."""
    rows, vocab = 9, 1003
    wide = torch.full((offset + rows * stride,), math.inf, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    x = wide[offset:].as_strided((rows, vocab), (stride, 1), offset) if stride >= vocab else None
    x.copy_(logits_like(rows, vocab, dtype, 8))
    u = np.random.default_rng(offset).random(rows, dtype=np.float32)
    check_draws(B, x, u, top_p=[0.9] * rows)
    check_draws(B, x, u, top_k=[20] * rows)
    check_draws(B, x, u)


def test_sample_draws_the_distribution(B):
    """Uniforms on a grid fall on each token as often as its probability says, to one of them."""
    n, vocab = 4096, 64
    x = logits_like(1, vocab, "f32", 11, 2.0)
    token, _ = draw(B, x.expand(n, vocab).contiguous(), (np.arange(n) + 0.5) / n, top_p=[0.8] * n)
    want = torch.softmax(x[0].double(), 0)
    top = want.sort(descending=True)
    keep = top.indices[: int(((top.values.cumsum(0) - top.values) < np.float32(0.8)).sum())]
    p = torch.zeros_like(want)
    p[keep] = want[keep] / want[keep].sum()
    assert np.abs(np.bincount(token, minlength=vocab) / n - p.cpu().numpy()).max() <= 1.0 / n


def test_sample_many_rows(B):
    """More rows than CTAs fit, each with parameters of its own; and none."""
    rows, vocab = 700, 3001
    r = np.random.default_rng(12)
    x = logits_like(rows, vocab, "bf16", 12)
    par = dict(temperature=np.where(r.random(rows) < 0.2, 0.0, r.random(rows) + 0.4), top_k=np.where(r.random(rows) < 0.5, 0, r.integers(1, 300, rows)),
               top_p=np.where(r.random(rows) < 0.5, 1.0, r.random(rows)), min_p=np.where(r.random(rows) < 0.5, 0.0, r.random(rows) * 0.2))
    check_draws(B, x, r.random(rows, dtype=np.float32), near_allowed=1, **par)
    token = torch.zeros(0, dtype=torch.int32, device="cuda")
    B.sample(x[:0], torch.zeros(0, device="cuda"), token)


@pytest.mark.parametrize("rows, vocab, dtype", [(41, 30000, "f32"), (101, 150001, "bf16"), (120, 20000, "bf16"), (120, 65537, "f32"), (330, 9000, "bf16")])
def test_sample_by_fewer_ctas_to_a_row(B, rows, vocab, dtype):
    """So many rows that each has fewer CTAs, whose part of it is in shared memory or not; every third row has a large top_k."""
    r = np.random.default_rng(rows)
    x = logits_like(rows, vocab, dtype, rows)
    k = np.where(np.arange(rows) % 3 == 0, r.integers(300, vocab, rows), np.where(r.random(rows) < 0.5, 0, r.integers(1, 300, rows)))
    par = dict(temperature=np.where(r.random(rows) < 0.1, 0.0, r.random(rows) + 0.4), top_k=k, top_p=np.where(r.random(rows) < 0.3, 1.0, r.random(rows)),
               min_p=np.where(r.random(rows) < 0.5, 0.0, r.random(rows) * 0.2))
    check_draws(B, x, r.random(rows, dtype=np.float32), near_allowed=1, **par)


def test_sample_without_prob_and_rows_untouched(B):
    x = logits_like(4, 300, "f32", 13)
    token = torch.full((6,), -7, dtype=torch.int32, device="cuda")
    B.sample(x, torch.full((4,), 0.4, device="cuda"), token[1:5])
    assert token[[0, 5]].tolist() == [-7, -7] and token[1:5].tolist() == [T.sample(host(x)[i], float(np.float32(0.4)))[0] for i in range(4)]


# ---- the walk and the move ---------------------------------------------------------------


def walk(B, trees, width, rng, lead=0, tail=0, hit=0.8, alias=False):
    """tree_accept of the given trees, with samples that mostly are one of the children's tokens, and the oracle's answer."""
    starts = np.cumsum([lead] + [len(e) for e in trees])
    rows = int(starts[-1]) + tail
    end, draft, sampled = (np.zeros(rows, dtype=np.int32) for _ in range(3))
    draft[:], sampled[:] = rng.integers(0, 40, rows), rng.integers(0, 40, rows)
    want = []
    for s, e in enumerate(trees):
        a = int(starts[s])
        end[a:a + len(e)] = e
        up = T.parents(e)
        for i in range(len(e)):
            kids = [j for j in range(len(e)) if up[j] == i]
            if kids and rng.random() < hit:
                sampled[a + i] = draft[a + rng.choice(kids)]
        want.append(T.accept(e, draft[a:a + len(e)], sampled[a:a + len(e)], width))
    dev = lambda x: torch.from_numpy(x.astype(np.int32)).cuda()  # noqa: E731
    n = len(trees)
    length = torch.tensor([1000 + len(e) for e in trees], dtype=torch.int32, device="cuda")
    tokens, path, count, out = (torch.full(shape, 99, dtype=torch.int32, device="cuda") for shape in ((n, width), (n, width), (n,), (n,)))
    B.tree_accept(dev(end), dev(starts), dev(draft), dev(sampled), tokens, path, count, length=length, length_out=None if alias else out)
    torch.cuda.synchronize()
    out = length if alias else out
    for s, (p, t) in enumerate(want):
        assert path[s].tolist() == p + [-1] * (width - len(p)) and tokens[s].tolist() == t + [-1] * (width - len(t))
        assert int(count[s]) == len(p) and int(out[s]) == 1000 + len(p)
    return tokens, path, count


@pytest.mark.parametrize("width", [1, 3, 16, 50])
@pytest.mark.parametrize("sizes", [[1], [16], [0], [64, 0, 1, 30, 7], [200] * 3, [255, 256, 257, 700], [20] * 130])
def test_tree_accept(B, sizes, width):
    rng = np.random.default_rng(sum(sizes) + width)
    walk(B, [random_tree(rng, n) for n in sizes], width, rng, lead=3, tail=2)
    walk(B, [random_tree(rng, n, 0.9) for n in sizes], width, rng, hit=1.0, alias=True)


def test_tree_accept_of_chains_and_stars(B):
    rng = np.random.default_rng(0)
    walk(B, [[40] * 40, [300] * 300, [30] + list(range(2, 31)), [400] + list(range(2, 401))], 400, rng, hit=1.0)


def test_tree_accept_of_ends_that_no_tree_has(B):
    """The walk ends whatever the ends are, and goes only to later rows of the sequence."""
    rng = np.random.default_rng(1)
    n = 40
    for end in ([0] * n, [-9] * n, [1 << 30] * n, rng.integers(-5, 90, n).tolist(), list(range(n))):
        e = torch.tensor(end, dtype=torch.int32, device="cuda")
        same = torch.zeros(n, dtype=torch.int32, device="cuda")
        tokens, path, count = (torch.zeros(shape, dtype=torch.int32, device="cuda") for shape in ((1, 64), (1, 64), (1,)))
        B.tree_accept(e, torch.tensor([0, n], dtype=torch.int32, device="cuda"), same, same, tokens, path, count)
        p = path[0, : int(count[0])].tolist()
        assert p[0] == 0 and all(a < b for a, b in zip(p, p[1:])) and p[-1] < n and (path[0, int(count[0]):] == -1).all()


def test_tree_accept_cuts_row_ranges(B):
    e = torch.full((4,), 4, dtype=torch.int32, device="cuda")
    same = torch.zeros(4, dtype=torch.int32, device="cuda")
    for start, want in (([0, 100], 4), ([-3, 2], 2), ([3, 1], 0), ([50, 60], 0)):
        tokens, path, count = (torch.zeros(shape, dtype=torch.int32, device="cuda") for shape in ((1, 8), (1, 8), (1,)))
        B.tree_accept(e, torch.tensor(start, dtype=torch.int32, device="cuda"), same, same, tokens, path, count)
        assert int(count[0]) == want


def commit_setup(B, lens, counts, layers=1, nkv=2, hd=64, ps=16, dtype="bf16", width=24, weights=True, seed=0, n_rows=40):
    """Caches of random contents, and ascending paths of `counts` rows within n_rows new ones."""
    rng = np.random.default_rng(seed)
    caches, copies = [], []
    n_seq, max_pages = len(lens), -(-(max(lens) + n_rows) // ps)
    table = rng.permutation(n_seq * max_pages + 1)[: n_seq * max_pages].reshape(n_seq, max_pages).astype(np.int32)
    length = torch.tensor([l + c for l, c in zip(lens, counts)], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    for _ in range(layers):
        shape = (n_seq * max_pages + 1, nkv, ps)
        k, v = torch.randn(*shape, hd, generator=g).to(dt), torch.randn(*shape, hd, generator=g).to(dt)
        pos, w = torch.randint(0, 1 << 20, shape, generator=g, dtype=torch.int32), torch.rand(shape, generator=g)
        caches.append(B.PagedCache(k.cuda(), v.cuda(), pos.cuda(), torch.from_numpy(table).cuda(), length, weight=w.cuda() if weights else None, status=status))
        copies.append({"k": host(k), "v": host(v), "pos": pos.numpy().copy(), "weight": host(w), "table": table, "length": length.cpu().numpy()})
    path = np.full((n_seq, width), -1, dtype=np.int32)
    for s, c in enumerate(counts):
        path[s, :c] = np.sort(rng.choice(n_rows, c, replace=False))
        if s % 3 == 0 and c:
            path[s, : c // 2 + 1] = np.arange(c // 2 + 1)  # the first branch for a while
            path[s, :c] = np.sort(np.unique(np.concatenate([path[s, : c // 2 + 1], rng.choice(np.arange(c, n_rows), c, replace=False)]))[:c])
    return caches, copies, path, status


def check_caches(caches, copies, weights=True):
    for c, o in zip(caches, copies):
        assert (host(c.k) == o["k"]).all() and (host(c.v) == o["v"]).all() and (c.pos.cpu().numpy() == o["pos"]).all()
        if weights:
            assert (host(c.weight) == o["weight"]).all()


@pytest.mark.parametrize("layers,weights", [(1, True), (3, False), (50, True)])
@pytest.mark.parametrize("nkv,hd,ps,dtype", [(8, 128, 64, "bf16"), (1, 8, 8, "f32"), (3, 80, 16, "bf16"), (2, 256, 32, "f32")])
def test_tree_commit(B, nkv, hd, ps, dtype, layers, weights):
    lens, counts = [0, 5, 40, 17, 16, 3], [1, 3, 24, 0, 9, 12]
    caches, copies, path, status = commit_setup(B, lens, counts, layers, nkv, hd, ps, dtype, weights=weights, seed=hd)
    B.paged_tree_commit(caches, torch.from_numpy(path).cuda(), torch.tensor(counts, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    for o in copies:
        T.commit(o, path, counts)
    check_caches(caches, copies, weights)
    assert int(status) == 0


def test_tree_commit_of_long_paths(B):
    """Paths of more rows than are looked up at once, shifted by one to hundreds of places."""
    caches, copies, _, status = commit_setup(B, [100, 0], [300, 129], width=300, n_rows=900)
    path = np.full((2, 300), -1, dtype=np.int32)
    path[0], path[1, :129] = np.arange(300) * 3, np.concatenate([[0], np.arange(2, 130)])
    B.paged_tree_commit(caches, torch.from_numpy(path).cuda(), torch.tensor([300, 129], dtype=torch.int32, device="cuda"))
    T.commit(copies[0], path, [300, 129])
    check_caches(caches, copies)
    assert int(status) == 0


@pytest.mark.parametrize("what", ["descending", "negative", "before", "beyond", "count", "wide", "length", "page"])
def test_tree_commit_reports_what_cannot_be(B, what):
    """What is out of order stays, and the other sequence's rows move."""
    caches, copies, path, status = commit_setup(B, [30, 9], [4, 5], width=6)
    path[0, :4] = [0, 2, 5, 9]
    path[1, :5] = [0, 1, 2, 5, 6]
    counts, good = [4, 5], [4, 5]
    o = copies[0]
    bits = B.PAGED_BAD_ROWS
    if what == "descending":
        path[0, 2] = 1
        moved = [0, 2, 2, 9]
    elif what == "negative":
        path[0, 2] = -1
        moved = [0, 2, 2, 9]
    elif what == "before":
        path[0, :4] = [-2, 1, 2, 3]
        moved = [0, 1, 2, 3]
    elif what == "beyond":
        path[0, 3] = 1 << 30
        moved = [0, 2, 5, 3]
    elif what in ("count", "wide"):
        counts[0] = -1 if what == "count" else 7
        moved = []
    elif what == "length":
        caches[0].length[0] = 2                          # fewer rows than the path has
        moved = []
    else:
        bits = B.PAGED_BAD_PAGE
        t = caches[0].table
        t[0, 2] = 1 << 20                                # rows 32 .. 47: those of the path from the third on
        moved = [0, 1, 2, 3]
        path[0, :4] = [0, 1, 4, 5]
    # a row that cannot move counts as one that stays
    want = np.full((2, 6), -1)
    want[0, : len(moved)], want[1, :5] = moved, path[1, :5]
    good[0] = len(moved)
    if what == "length":
        o["length"][0] = 30
    T.commit({**o, "length": np.array([30 + good[0], 9 + 5])}, want, good)
    B.paged_tree_commit(caches, torch.from_numpy(path).cuda(), torch.tensor(counts, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    check_caches(caches, copies)
    assert int(status) == bits


# ---- together ----------------------------------------------------------------------------


class Rounds:
    """A model of `layers` caches whose rows are functions of tokens and depths, and whose logits are a projection of the
    last layer's attention: enough to run verify rounds as an engine does."""

    def __init__(self, B, n_seq, layers, dtype, seed=0, vocab=300, nodes=12, width=5, nq=4, nkv=2, hd=64, ps=16, max_pages=20, prompt=(37, 5, 64)):
        self.B, self.n_seq, self.width, self.vocab, self.nodes = B, n_seq, width, vocab, nodes
        self.nq, self.nkv, self.hd, self.ps = nq, nkv, hd, ps
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.wq, self.wk, self.wv = (torch.randn(layers, vocab, h, hd, generator=g, device="cuda").to(dt) for h in (nq, nkv, nkv))
        self.head = torch.randn(nq * hd, vocab, generator=g, device="cuda") * 0.3
        self.caches = [B.PagedCache.allocate(n_seq * max_pages, ps, nkv, hd, n_seq, max_pages, dtype) for _ in range(layers)]
        self.length = torch.zeros(n_seq, dtype=torch.int32, device="cuda")
        table = torch.randperm(n_seq * max_pages, generator=g, device="cuda").reshape(n_seq, max_pages).to(torch.int32)
        for c in self.caches:
            c.table.copy_(table)
        self.start = torch.arange(0, n_seq * nodes + 1, nodes, dtype=torch.int32, device="cuda")
        rows = n_seq * nodes
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.draft, self.end, self.depth, self.uniform = i32(rows), i32(rows), i32(rows), torch.zeros(rows, device="cuda")
        self.pos, self.sampled, self.tokens, self.path, self.count = i32(rows), i32(rows), i32(n_seq, width), i32(n_seq, width), i32(n_seq)
        self.logits = torch.zeros(rows, vocab, dtype=dt, device="cuda")
        self.q_out = torch.zeros(rows, nq, hd, dtype=dt, device="cuda")
        self.out = torch.zeros(rows, nq, hd, dtype=dt, device="cuda")
        self.temperature, self.top_p = torch.full((rows,), 0.7, device="cuda"), torch.full((rows,), 0.9, device="cuda")
        self.anchor = i32(n_seq)
        self.text = [torch.randint(0, vocab, (prompt[s % len(prompt)],), generator=g, device="cuda") for s in range(n_seq)]
        for c in self.caches:                             # the prompts
            for s in range(n_seq):
                n = len(self.text[s])
                at = torch.arange(n, device="cuda")
                page, r = table[s, at // ps].long(), at % ps
                l = self.caches.index(c)
                c.k[page, :, r], c.v[page, :, r], c.pos[page, :, r] = self.wk[l][self.text[s]], self.wv[l][self.text[s]], at.to(torch.int32)[:, None]
        self.length.copy_(torch.tensor([len(t) for t in self.text], dtype=torch.int32))
        self.anchor.copy_(torch.tensor([1] * n_seq, dtype=torch.int32))

    def propose(self, rng):
        """New trees: ends, drafted tokens (row 0 the anchor's) and uniforms."""
        end, depth = [], []
        for _ in range(self.n_seq):
            e = random_tree(rng, self.nodes)
            end += e
            depth += (T.ancestors(e).sum(1) - 1).tolist()
        self.end.copy_(torch.tensor(end, dtype=torch.int32))
        self.depth.copy_(torch.tensor(depth, dtype=torch.int32))
        self.draft.copy_(torch.from_numpy(rng.integers(0, self.vocab, len(end)).astype(np.int32)))
        self.uniform.copy_(torch.from_numpy(rng.random(len(end), dtype=np.float32)))

    def round(self):
        """One verify round, every step enqueued."""
        self.draft[self.start[:-1].long()] = self.anchor
        self.pos.copy_(self.length.repeat_interleave(self.nodes, output_size=len(self.pos)) + self.depth)
        for l, c in enumerate(self.caches):
            torch.add(self.length, self.nodes, out=c.length)
            x = self.draft.long()
            c.append(self.wq[l][x], self.wk[l][x], self.wv[l][x], self.pos, self.start, self.q_out)
            c.tree_attention(self.q_out, self.pos, self.start, self.end, self.out)
        self.logits.copy_(self.out.float().flatten(1) @ self.head)
        self.B.sample(self.logits, self.uniform, self.sampled, temperature=self.temperature, top_p=self.top_p)
        grown = self.length + self.nodes
        self.B.tree_accept(self.end, self.start, self.draft, self.sampled, self.tokens, self.path, self.count, length=grown, length_out=self.length)
        for c in self.caches:
            c.length.copy_(self.length)
        self.B.paged_tree_commit(self.caches, self.path, self.count)
        self.anchor.copy_(self.tokens.gather(1, (self.count.long() - 1)[:, None])[:, 0])

    def state(self):
        return [self.tokens, self.path, self.count, self.length, self.anchor] + [x for c in self.caches for x in (c.k, c.v, c.pos)]


class Right(Rounds):
    """The drafted tokens are changed to what will be sampled at their parents, in about two of three rows: the sampled
    tokens are functions of the drafted ones, so rounds are run until they agree."""

    def right(self, rng):
        for _ in range(self.nodes):
            held = [x.clone() for x in self.state()]
            self.round()
            sampled = self.sampled.cpu().numpy()
            for x, y in zip(self.state(), held):
                x.copy_(y)
            draft = self.draft.cpu().numpy()
            for s in range(self.n_seq):
                a = s * self.nodes
                up = T.parents(self.end[a:a + self.nodes].tolist())
                for i in range(1, self.nodes):
                    if self.lucky[a + i]:
                        draft[a + i] = sampled[a + up[i]]
            self.draft.copy_(torch.from_numpy(draft))

    def propose(self, rng):
        super().propose(rng)
        self.lucky = rng.random(len(self.draft)) < 0.7
        self.right(rng)


@pytest.mark.parametrize("dtype,n_seq", [("bf16", 3), ("f32", 2)])
def test_rounds_keep_the_caches_of_the_accepted_text(B, dtype, n_seq):
    """After each round every cache holds, bit for bit, the rows of the text so far in order; the walk and the samples follow
    the oracle's."""
    rng = np.random.default_rng(4)
    r = Right(B, n_seq, 2, dtype)
    text = [t.tolist() for t in r.text]
    accepted = 0
    for _ in range(4):
        r.propose(rng)
        anchors = r.anchor.tolist()
        r.round()
        torch.cuda.synchronize()
        x, u, sampled, end, draft = host(r.logits), r.uniform.cpu().numpy(), r.sampled.tolist(), r.end.tolist(), r.draft.tolist()
        for i in range(len(x)):
            want, _, margin = T.sample(x[i], float(u[i]), float(np.float32(0.7)), 0, float(np.float32(0.9)))
            assert want == sampled[i] or margin <= border(r.vocab)
        for s in range(n_seq):
            a = s * r.nodes
            p, t = T.accept(end[a:a + r.nodes], draft[a:a + r.nodes], sampled[a:a + r.nodes], r.width)
            assert r.path[s, : len(p)].tolist() == p and r.tokens[s, : len(p)].tolist() == t and int(r.count[s]) == len(p)
            text[s] += [anchors[s]] + t[:-1]
            accepted += len(p) - 1
            assert int(r.length[s]) == len(text[s]) and int(r.anchor[s]) == t[-1]
            at = torch.arange(len(text[s]), device="cuda")
            said = torch.tensor(text[s], device="cuda")
            for l, c in enumerate(r.caches):
                page, row = c.table[s, at // r.ps].long(), at % r.ps
                assert torch.equal(c.k[page, :, row], r.wk[l][said]) and torch.equal(c.v[page, :, row], r.wv[l][said])
                assert torch.equal(c.pos[page, :, row], at.to(torch.int32)[:, None].expand(-1, r.nkv))
    assert accepted >= 6                                 # (paths of several rows were among them)


def test_rounds_captured_in_a_graph_and_replayed(B):
    """A captured round replayed on new trees gives the bits of a round called step by step; two graphs and calls outside them
    share no memory that either keeps."""
    eager, graphed, other = (Rounds(B, 3, 2, "bf16", seed=1) for _ in range(3))
    rng = [np.random.default_rng(9) for _ in range(3)]
    for r, x in ((eager, rng[0]), (graphed, rng[1]), (other, rng[2])):
        r.propose(x)
        r.round()                                        # (also makes every kernel's first call outside the capture)
    torch.cuda.synchronize()
    graphs = []
    for r, x in ((graphed, rng[1]), (other, rng[2])):
        r.propose(x)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r.round()
        graphs.append(g)
    side = torch.cuda.Stream()
    eager.propose(rng[0])
    for _ in range(3):
        eager.round()
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        for x, y, z in zip(eager.state(), graphed.state(), other.state()):
            assert torch.equal(x, y) and torch.equal(x, z)
        for r, x in ((eager, rng[0]), (graphed, rng[1]), (other, rng[2])):
            r.propose(x)
        torch.cuda.synchronize()


def test_calls_on_two_streams_at_once(B):
    sets = [Trees(B, [(20, 3000), (7, 900)], 8, 2, 128, 32, seed=60 + i) for i in range(2)]
    caches = [s.device() for s in sets]
    logits = [logits_like(30, 50001, "bf16", 70 + i) for i in range(2)]
    u = torch.linspace(0.01, 0.99, 30, device="cuda")
    p = torch.full((30,), 0.9, device="cuda")
    streams = [torch.cuda.Stream() for _ in sets]
    args = [(s.q.cuda(), s.q_pos.cuda(), s.start.cuda(), s.end.cuda()) for s in sets]
    outs = [[torch.zeros(27, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(12)] for _ in sets]
    tokens = [[torch.zeros(30, dtype=torch.int32, device="cuda") for _ in range(12)] for _ in sets]
    torch.cuda.synchronize()
    for i in range(12):
        for c, st, a, o, l, t in zip(caches, streams, args, outs, logits, tokens):
            c.tree_attention(*a, o[i], stream=st)
            B.sample(l, u, t[i], top_p=p, stream=st)
    torch.cuda.synchronize()
    for s, c, o, l, t in zip(sets, caches, outs, logits, tokens):
        first, _ = s.check(c)
        assert all(torch.equal(x, first) for x in o)
        alone = torch.zeros_like(t[0])
        B.sample(l, u, alone, top_p=p)
        assert all(torch.equal(x, alone) for x in t)
