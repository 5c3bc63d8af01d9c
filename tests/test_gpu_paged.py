"""GPU parity of the paged-cache operators against the fp64 oracle
(oracle/paged_oracle.py), through the binding.

Tolerances count roundings. eps = 2^-24 is fp32's half step, u = 2^-8 (bf16) or
2^-24 (fp32) the storage type's.

* A score t is a dot product of hd terms in fp32, a scaling, a cap and a bias:
  dt = (hd + 8) eps sum |q k| scale + 8 eps (cap + |bias| + |t|), the largest over
  the call. The cap's slope is at most 1.
  fp32's products in two tf32 parts add 2^-21 of |q k| for what the parts drop and
  2^-22 for their smallest product, 12 eps at the worst, with both of one sign in
  every term; Cauchy-Schwarz's bound on sum |q k| leaves more than that.
* A weight p = exp(t - m) then is off by a factor of dt + 2^-20 (exp2's own error
  and the change to log2 units at |t| < 16), the sum l by as much.
* out: u |out| for its rounding, and 2 (dt + 2^-20) + n eps, for n summed keys,
  of sum p |v|, and in bf16 another 2^-8 of it, p's rounding for the product.
* lse: dt + 2^-20 + 4 eps |lse|.
* key weights: (dt + 2^-20 + 4 eps |lse|) of the sum, n eps for adding n terms, 4 eps of decay * weight.
* append: a rotated value from a norm of hd terms: (hd + 16) eps (|a| + |b|) for
  a pair (a, b), and the rounding.
Eviction and all integers are exact."""

import math

import numpy as np
import pytest
import torch

from oracle import paged_oracle as P

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from block_speculative_decoding_dflash_gb300 import build
    build.build()
    from block_speculative_decoding_dflash_gb300 import binding
    return binding


def unit(dtype):
    return 2.0 ** -8 if dtype == "bf16" else EPS


def host(t):
    return t.detach().double().cpu().numpy()


class Setup:
    """A cache of sequences with (new rows, cached rows) `lens` and its host copy. Pages and rows that no sequence holds
    are NaN, unused table entries are page ids outside the pool, weights are uniform in [0, 1)."""

    def __init__(self, B, lens, nq, nkv, hd, ps=16, dtype="bf16", seed=0, spare=1, lead=0, tail=0, kept=False, scale=1.5):
        g = torch.Generator().manual_seed(seed)
        self.B, self.dtype, self.hd, self.nq, self.nkv = B, dtype, hd, nq, nkv
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.dt = dt
        width = max(1, max(-(-l // ps) for _, l in lens)) + spare
        held = [-(-l // ps) for _, l in lens]
        n_pages = sum(held) + 2
        perm = torch.randperm(n_pages, generator=g).tolist()
        table = torch.full((len(lens), width), -7, dtype=torch.int32)
        table[:, -1] = n_pages
        shape = (n_pages, nkv, ps)
        k, v = torch.full((*shape, hd), math.nan), torch.full((*shape, hd), math.nan)
        pos, weight = torch.full(shape, 12345, dtype=torch.int32), torch.full(shape, math.nan)
        starts = [lead]
        self.pos_of = []
        q_pos = []
        for s, (n, length) in enumerate(lens):
            pages = [perm.pop() for _ in range(held[s])]
            table[s, :held[s]] = torch.tensor(pages, dtype=torch.int32)
            first = 0
            for h in range(nkv):
                p = torch.arange(length)
                if kept:
                    old = 2 * torch.arange(length - n) + torch.randint(0, 2, (length - n,), generator=g)
                    first = 2 * length
                    p = torch.cat([old[torch.randperm(length - n, generator=g)], first + torch.arange(n)])
                for r in range(length):
                    page, j = pages[r // ps], r % ps
                    pos[page, h, j] = p[r]
                    weight[page, h, j] = torch.rand((), generator=g)
                rows = torch.arange(length)
                pg, j = torch.tensor(pages, dtype=torch.long)[rows // ps], rows % ps
                k[pg, h, j] = torch.randn(length, hd, generator=g)
                v[pg, h, j] = torch.randn(length, hd, generator=g)
            q_pos += list(range((first if kept else length - n), (first + n if kept else length)))
            starts.append(starts[-1] + n)
        self.start = torch.tensor(starts, dtype=torch.int32)
        self.rows = starts[-1] + tail
        self.q_pos = torch.tensor([0] * lead + q_pos + [0] * tail, dtype=torch.int32)
        self.q = (torch.randn(self.rows, nq, hd, generator=g) * scale).to(dt)
        self.k, self.v, self.pos, self.weight, self.table = k.to(dt), v.to(dt), pos, weight, table
        self.length = torch.tensor([l for _, l in lens], dtype=torch.int32)
        self.scale = hd ** -0.5

    def device(self, **over):
        """The binding's cache over fresh device copies."""
        t = {n: over.get(n, getattr(self, n)).cuda() for n in ("k", "v", "pos", "table", "length", "weight")}
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        return self.B.PagedCache(t["k"], t["v"], t["pos"], t["table"], t["length"], weight=t["weight"], status=self.status)

    def oracle(self):
        return {"k": host(self.k), "v": host(self.v), "pos": self.pos.numpy(), "weight": host(self.weight),
                "table": self.table.numpy(), "length": self.length.numpy()}

    def score_error(self, softcap, slopes):
        # |q k| summed: at most |q| |k| by Cauchy-Schwarz
        qn = np.sqrt((host(self.q) ** 2).sum(-1)).max(initial=0.0)
        kn = np.sqrt((np.where(np.isfinite(host(self.k)), host(self.k), 0.0) ** 2).sum(-1)).max()
        t = qn * kn * self.scale
        far = float(max(int(self.q_pos.max()) if self.rows else 0, int(self.length.max()) if len(self.length) else 0)) * 2
        bias = 0.0 if slopes is None else float(slopes.max()) * far
        return (self.hd + 8) * EPS * t + 8 * EPS * (softcap + bias + t)

    def check_attention(self, cache, strided=False, **mask):
        slopes, prefix = mask.get("slopes"), mask.get("prefix")
        q = self.q.cuda()
        if strided:
            wide = torch.full((self.rows, self.nq * self.hd + 24), math.nan, dtype=self.dt, device="cuda")
            q = wide[:, 8:8 + self.nq * self.hd].unflatten(1, (self.nq, self.hd)).copy_(q)
        out = torch.full((self.rows, self.nq, self.hd), 77.0, dtype=self.dt, device="cuda")
        lse = torch.full((self.rows, self.nq), 77.0, device="cuda")
        dev = {n: None if x is None else x.cuda() for n, x in (("slopes", slopes), ("prefix", prefix))}
        cache.attention(q, self.q_pos.cuda(), self.start.cuda(), out, lse=lse, **{**mask, **dev})
        torch.cuda.synchronize()
        opts = {n: (x.numpy().astype(np.float64) if n == "slopes" and x is not None else None if x is None else x.numpy() if n == "prefix" else x)
                for n, x in mask.items() if n not in ("max_len", "scale")}
        want, want_lse, mag = P.attention(self.oracle(), host(self.q), self.q_pos.numpy(), self.start.numpy(), mask.get("scale") or self.scale, **opts)
        self.compare(host(out), host(lse), want, want_lse, mag, mask.get("softcap", 0.0), None if slopes is None else slopes.numpy())
        return out, lse

    def compare(self, out, lse, want, want_lse, mag, softcap, slopes):
        a, b = int(self.start[0]), int(self.start[-1])
        assert (out[:a] == 77).all() and (out[b:] == 77).all() and (lse[:a] == 77).all() and (lse[b:] == 77).all()
        out, lse, want, want_lse, mag = (x[a:b] for x in (out, lse, want, want_lse, mag))
        dt = self.score_error(softcap, slopes)
        n = float(self.length.max())
        tol = unit(self.dtype) * np.abs(want) + (2 * (dt + 2.0 ** -20) + n * EPS + (2.0 ** -8 if self.dtype == "bf16" else 0)) * mag + 1e-38
        none = np.isneginf(want_lse)
        assert (np.isneginf(lse) == none).all() and (out[none] == 0).all()
        fine = np.isfinite(want)
        assert np.isfinite(out[fine]).all(), f"{np.argwhere(~np.isfinite(out) & fine)[:5]}"
        assert not np.isfinite(out[~fine]).any()
        off = np.abs(out[fine] - want[fine]) / tol[fine]
        assert off.size == 0 or off.max() <= 1.0, f"out off by {off.max():.3g} of the tolerance"
        there = np.isfinite(want_lse)
        err = np.abs(lse[there] - want_lse[there]) / (dt + 2.0 ** -20 + 4 * EPS * np.abs(want_lse[there]))
        assert err.size == 0 or err.max() <= 1.0, f"lse off by {err.max():.3g} of the tolerance"

    def check_weight(self, cache, lse, decay=0.9, use_in=True, **mask):
        slopes, prefix = mask.get("slopes"), mask.get("prefix")
        dev = {n: None if x is None else x.cuda() for n, x in (("slopes", slopes), ("prefix", prefix))}
        w_out = torch.full(self.pos.shape, 77.0, device="cuda")
        cache.key_weight(self.q.cuda(), self.q_pos.cuda(), self.start.cuda(), lse, weight_out=w_out, decay=decay, **{**mask, **dev})
        torch.cuda.synchronize()
        opts = {n: (x.numpy().astype(np.float64) if n == "slopes" and x is not None else None if x is None else x.numpy() if n == "prefix" else x)
                for n, x in mask.items() if n not in ("max_len", "scale")}
        o = self.oracle()
        want, terms = P.key_weight(o, host(self.q), self.q_pos.numpy(), self.start.numpy(), host(lse), o["weight"], float(np.float32(decay)),
                                   np.full(self.pos.shape, 77.0), mask.get("scale") or self.scale, **opts)
        got = host(w_out)
        dt = self.score_error(mask.get("softcap", 0.0), None if slopes is None else slopes.numpy())
        big = np.abs(host(lse)[np.isfinite(host(lse))]).max(initial=0.0)
        old = np.nan_to_num(o["weight"]) * abs(decay)
        tol = (dt + 2.0 ** -20 + 4 * EPS * big + terms * EPS) * np.abs(want - np.where(want == 77, 77, old)) + 4 * EPS * old + terms * 1e-37 + 2 * EPS * np.abs(want)
        assert ((got == 77) == (want == 77)).all()
        off = np.abs(got - want) - tol
        assert (off <= 0).all(), f"key weight off by {np.abs(got - want).max():.3g}, {off.max():.3g} over the tolerance"
        return w_out


SHAPES = [
    # lens (new, cached), nq, nkv, hd, page rows, dtype
    ([(1, 1)], 4, 2, 16, 8, "f32"),
    ([(1, 1)], 8, 8, 64, 16, "bf16"),
    ([(1, 33), (1, 7), (1, 130)], 32, 8, 128, 16, "bf16"),
    ([(4, 300)], 32, 8, 128, 64, "bf16"),
    ([(16, 16)], 16, 8, 128, 32, "bf16"),
    ([(0, 40), (5, 5), (0, 0), (17, 129), (1, 128), (0, 3)], 8, 4, 64, 16, "bf16"),
    ([(70, 257), (3, 640)], 14, 2, 128, 128, "bf16"),
    ([(129, 129)], 6, 1, 80, 8, "bf16"),
    ([(33, 500)], 5, 1, 96, 256, "bf16"),
    ([(40, 200), (2, 31)], 4, 4, 256, 16, "bf16"),
    ([(3, 90)], 4, 2, 24, 16, "bf16"),
    ([(300, 700)], 16, 2, 64, 64, "bf16"),
    ([(9, 200), (1, 65), (0, 12)], 16, 8, 128, 16, "f32"),
    ([(65, 130)], 12, 4, 80, 32, "f32"),
    ([(20, 150)], 2, 1, 200, 8, "f32"),
    ([(2, 70)], 128, 1, 64, 16, "bf16"),
]
MASKS = [dict(), dict(window=20), dict(causal=False), dict(causal=False, window=9), dict(softcap=5.0), dict(slopes=True), dict(window=16, prefix=6, softcap=20.0, slopes=True)]


def mask_of(mask, nq, n_seq):
    m = dict(mask)
    if m.get("slopes"):
        m["slopes"] = torch.exp2(-8.0 * torch.arange(1, nq + 1) / nq)
    if "prefix" in m:
        m["prefix"] = torch.tensor([m["prefix"] * (s % 3) for s in range(n_seq)], dtype=torch.int32)
    return m


@pytest.mark.parametrize("mask", MASKS, ids=lambda m: "-".join(m) or "plain")
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{s[0][0][0]}of{s[0][0][1]}-{s[1]}_{s[2]}x{s[3]}-{s[4]}-{s[5]}")
def test_attention_and_key_weight(B, shape, mask):
    lens, nq, nkv, hd, ps, dtype = shape
    s = Setup(B, lens, nq, nkv, hd, ps, dtype, seed=len(lens) + hd, lead=2, tail=3)
    m = mask_of(mask, nq, len(lens))
    cache = s.device()
    _, lse = s.check_attention(cache, strided=True, **m)
    s.check_weight(cache, lse, **m)
    assert int(s.status) == 0


@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("bf16", 64), ("f32", 64), ("bf16", 256)])
@pytest.mark.parametrize("n", [1, 9, 140])
def test_an_evicted_cache(B, dtype, hd, n):
    """Rows in no order, other positions in every kv head."""
    s = Setup(B, [(n, 400), (1, 150)], 8, 4, hd, 32, dtype, seed=3, kept=True)
    cache = s.device()
    for m in (dict(), dict(window=350), dict(slopes=torch.full((8,), 0.01), softcap=30.0)):
        _, lse = s.check_attention(cache, **m)
        s.check_weight(cache, lse, **m)


@pytest.mark.parametrize("dtype,hd,nq", [("bf16", 128, 8), ("bf16", 64, 6), ("f32", 128, 8), ("bf16", 256, 2)])
@pytest.mark.parametrize("n", [1, 3, 40, 200])
def test_queries_that_see_nothing(B, dtype, hd, nq, n):
    s = Setup(B, [(n, 210), (n, 205)], nq, 2, hd, 16, dtype, seed=5)
    s.q_pos[::2] = -1                                   # before every row
    s.q_pos[1::2] += 100000                             # far behind the window
    if n > 1:
        s.q_pos[1] = 5
    cache = s.device()
    for m in (dict(window=8), dict(window=8, prefix=torch.tensor([0, 2], dtype=torch.int32))):
        _, lse = s.check_attention(cache, **m)
        s.check_weight(cache, lse, **m)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_positions_far_apart_and_far_out(B, dtype):
    """Distances of queries 2^30 positions apart in one tile, and of neighbours at 2^30."""
    s = Setup(B, [(4, 300), (3, 140)], 4, 2, 64, 16, dtype, seed=7)
    far = 1 << 30
    s.q_pos[:4] = torch.tensor([299, far, far + 5, 299 + (1 << 23)])
    s.q_pos[4:] += far
    for i in range(140):
        s.pos[int(s.table[1, i // 16]), :, i % 16] += far
    cache = s.device()
    _, lse = s.check_attention(cache, slopes=torch.tensor([2.0 ** -30, 2.0 ** -29, 0.01, 2.0 ** -8]), window=1 << 30)
    s.check_weight(cache, lse, slopes=torch.tensor([2.0 ** -30, 2.0 ** -29, 0.01, 2.0 ** -8]), window=1 << 30)


@pytest.mark.parametrize("softcap", [1e-18, 1e-6, 1e-3, 1e18])
@pytest.mark.parametrize("dtype,hd,nq", [("bf16", 128, 8), ("bf16", 64, 6), ("f32", 64, 4), ("bf16", 256, 2)])
@pytest.mark.parametrize("n", [1, 40, 200])
def test_caps_far_from_the_scores(B, dtype, hd, nq, n, softcap):
    """Zero scores under a cap stay zero, however small it is; a vast cap leaves scores as they are."""
    s = Setup(B, [(n, n + 150)], nq, 2, hd, 16, dtype, seed=n)
    s.q[: n - n // 2] = 0
    cache = s.device()
    # the scores' error in the formula counts 8 roundings of a cap that a vast one does not reach
    reach = min(softcap, 1e3)
    s_error = s.score_error
    s.score_error = lambda cap, slopes: s_error(reach, slopes)
    _, lse = s.check_attention(cache, softcap=softcap)
    s.check_weight(cache, lse, softcap=softcap)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype,hd,nq", [("bf16", 128, 8), ("bf16", 64, 32), ("f32", 128, 8), ("bf16", 136, 4)])
@pytest.mark.parametrize("n", [6, 80, 300])
def test_hidden_rows_may_hold_anything(B, dtype, hd, nq, n, bad):
    """The last new rows and a row outside the window of some queries are infinite or NaN in K and V: only queries that see
    them change."""
    length = 400
    s = Setup(B, [(n, length)], nq, 2, hd, 16, dtype, seed=6)
    for r in (length - 1, length - 3, length - n - 1, 40):
        page, j = int(s.table[0, r // 16]), r % 16
        s.v[page, :, j, ::3] = bad
        if r != 40:
            s.k[page, :, j, 5] = math.nan if bad != bad else s.k[page, :, j, 5]
    # NaN keys are only compared where they are hidden: what a query sees of them is NaN in the oracle too
    cache = s.device()
    s.check_attention(cache, window=150)
    s.check_attention(cache)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dtype,hd,nq", [("bf16", 128, 8), ("bf16", 64, 6), ("f32", 128, 8), ("bf16", 136, 4)])
@pytest.mark.parametrize("n", [6, 30, 200])
def test_infinite_values_of_rows_with_no_weight_left_are_seen(B, dtype, hd, nq, n, bad):
    """A row far away whose weight leaves fp32 (e^-150 and less) is seen all the same: what is infinite or NaN in its V
    makes the outputs so, in a tile that is seen wholly and in one with a hidden row."""
    s = Setup(B, [(n, 400)], nq, 2, hd, 16, dtype, seed=6)
    at = lambda r: (int(s.table[0, r // 16]), slice(None), r % 16)  # noqa: E731
    for hidden in (False, True):
        s.v[at(40)][:, ::3] = bad
        if hidden:
            s.pos[at(41)] = 1 << 20                         # later than every query
            s.v[at(41)] = math.nan
        cache = s.device()
        s.check_attention(cache, slopes=torch.full((nq,), 1.0))


@pytest.mark.parametrize("mask", [dict(), dict(softcap=20.0), dict(softcap=20.0, slopes=True), dict(window=50)], ids=lambda m: "-".join(m) or "plain")
@pytest.mark.parametrize("dtype,hd,nq", [("bf16", 128, 8), ("bf16", 64, 6), ("f32", 128, 4), ("bf16", 200, 4)])
@pytest.mark.parametrize("n", [3, 70, 200])
def test_hidden_rows_leave_every_bit(B, dtype, hd, nq, n, mask):
    """The same bits whatever stands in the rows behind the length and in those that no query sees."""
    results = []
    for fill in (0.0, 1e4, math.inf, math.nan):
        s = Setup(B, [(n, n + 77)], nq, 2, hd, 16, dtype, seed=5)
        length = n + 77
        hidden = list(range(10, 77, 7))
        page, j = s.table[0, torch.tensor(hidden) // 16].long(), torch.tensor(hidden) % 16
        for x in (s.k, s.v):
            x[torch.isnan(x)] = fill
            x[page, :, j] = fill
        s.pos[page, :, j] = 1 << 20                     # later than every query
        cache = s.device()
        out = torch.zeros(s.rows, nq, hd, dtype=s.dt, device="cuda")
        lse = torch.zeros(s.rows, nq, device="cuda")
        w = torch.zeros(s.pos.shape, device="cuda")
        m = {k: v.cuda() if torch.is_tensor(v) else v for k, v in mask_of(mask, nq, 1).items()}
        args = s.q.cuda(), s.q_pos.cuda(), s.start.cuda()
        cache.attention(*args, out, lse=lse, **m)
        cache.key_weight(*args, lse, weight_out=w, weight=torch.zeros_like(w), **m)
        assert torch.isfinite(out).all() and torch.isfinite(w).all() and length == int(s.length[0])
        results.append((out, lse, w))
    for r in results[1:]:
        assert [torch.equal(a, b) for a, b in zip(r, results[0])] == [True] * 3


@pytest.mark.parametrize("mask", [dict(), dict(softcap=20.0), dict(softcap=3.0, slopes=True), dict(window=600)], ids=lambda m: "-".join(m) or "plain")
@pytest.mark.parametrize("dtype,hd,nq", [("bf16", 128, 8), ("bf16", 64, 6), ("f32", 64, 4), ("bf16", 200, 4)])
@pytest.mark.parametrize("n", [1, 3, 70, 200])
def test_the_next_sequence_leaves_every_bit(B, dtype, hd, nq, n, mask):
    """out, lse and key weights of a sequence are the same bits whatever the queries of the next one are, and those of no
    sequence at all: a load brings them into its tile, and its warps vote on how scores are computed."""
    s = Setup(B, [(n, 1500), (5, 60)], nq, 2, hd, 16, dtype, seed=9, tail=4)
    m = {k: v.cuda() if torch.is_tensor(v) else v for k, v in mask_of(mask, nq, 2).items()}
    cache, q = s.device(), s.q.cuda()
    pages = s.table[0, :-(-1500 // 16)].long().cuda()
    results = []
    for fill in (None, 0.0, 1e4, math.inf, math.nan):
        if fill is not None:
            q[n:] = fill
        out, lse = torch.zeros_like(q), torch.zeros(s.rows, nq, device="cuda")
        w = torch.zeros(s.pos.shape, device="cuda")
        cache.attention(q, s.q_pos.cuda(), s.start.cuda(), out, lse=lse, **m)
        cache.key_weight(q, s.q_pos.cuda(), s.start.cuda(), lse, weight_out=w, weight=torch.zeros_like(w), **m)
        results.append((out[:n], lse[:n], w[pages]))
    assert torch.isfinite(results[0][0]).all()
    for r in results[1:]:
        assert [torch.equal(a, b) for a, b in zip(r, results[0])] == [True] * 3


@pytest.mark.parametrize("nq,hd", [(8, 128), (6, 64), (32, 128)])
@pytest.mark.parametrize("prompt", [0, 300])
def test_few_rows_beside_a_prompt_are_as_exact_as_alone(B, nq, hd, prompt):
    """A sequence of at most 64 packed rows has its weights in two bf16 parts, 2^-16 of each at most, whatever else is in the
    batch: values +1 and -1 nearly cancel, so that an output's own rounding is no cover for one part's 2^-8."""
    lens = [(1, 9), (1, 14), (2, 12), (3, 11)]
    s = Setup(B, ([(prompt, 320)] if prompt else []) + lens, nq, 2, hd, 16, seed=12, scale=0.3)
    s.v = torch.where(torch.isnan(s.v), s.v, torch.where(s.v > 0, 1.0, -1.0).to(s.dt))
    cache = s.device()
    out, lse = torch.zeros(s.rows, nq, hd, dtype=s.dt, device="cuda"), torch.zeros(s.rows, nq, device="cuda")
    cache.attention(s.q.cuda(), s.q_pos.cuda(), s.start.cuda(), out, lse=lse)
    few = slice(prompt, s.rows)
    want, want_lse, mag = (x[few] for x in P.attention(s.oracle(), host(s.q), s.q_pos.numpy(), s.start.numpy(), s.scale))
    dt = s.score_error(0.0, None)
    tol = unit("bf16") * np.abs(want) + (2 * (dt + 2.0 ** -20) + 14 * EPS + 2.0 ** -16) * mag
    off = np.abs(host(out)[few] - want) / tol
    assert off.max() <= 1.0, f"off by {off.max():.3g} of the tolerance"
    assert (np.abs(host(lse)[few] - want_lse) <= dt + 2.0 ** -20 + 4 * EPS * np.abs(want_lse)).all()


@pytest.mark.parametrize("mask", [dict(softcap=2.0), dict(softcap=30.0, slopes=True), dict(window=7, softcap=4.0), dict(slopes=True)], ids=lambda m: "-".join(m))
@pytest.mark.parametrize("nq,hd", [(8, 128), (6, 64)])
def test_few_rows_beside_a_prompt_under_caps_and_biases(B, nq, hd, mask):
    """The same with scores that are changed before they are weighed, in tiles that are seen wholly (a cap alone) and in part."""
    s = Setup(B, [(300, 320), (1, 129), (1, 300), (2, 260), (3, 11)], nq, 2, hd, 16, seed=13, scale=0.3)
    s.v = torch.where(torch.isnan(s.v), s.v, torch.where(s.v > 0, 1.0, -1.0).to(s.dt))
    m = mask_of(mask, nq, 5)
    cache = s.device()
    out, _ = s.check_attention(cache, **m)
    opts = {k: v.numpy().astype(np.float64) if torch.is_tensor(v) else v for k, v in m.items()}
    want, _, mag = (x[300:] for x in P.attention(s.oracle(), host(s.q), s.q_pos.numpy(), s.start.numpy(), s.scale, **opts))
    dt = s.score_error(m.get("softcap", 0.0), None if m.get("slopes") is None else m["slopes"].numpy())
    off = np.abs(host(out)[300:] - want) / (unit("bf16") * np.abs(want) + (2 * (dt + 2.0 ** -20) + 300 * EPS + 2.0 ** -16) * mag)
    assert off.max() <= 1.0, f"off by {off.max():.3g} of the tolerance"


@pytest.mark.parametrize("dtype,hd,nq", [("bf16", 128, 8), ("bf16", 64, 6), ("f32", 128, 4), ("bf16", 200, 4)])
@pytest.mark.parametrize("n", [200, 270])
def test_rows_behind_the_length_leave_every_bit_of_key_weights(B, dtype, hd, nq, n):
    """Every query sees every row there is, and the last tile of keys ends inside a page: what that page holds behind the length
    has no say in how the others' caps are computed."""
    results = []
    for fill in (0.0, 1e4, math.inf, math.nan):
        s = Setup(B, [(n, 277)], nq, 2, hd, 16, dtype, seed=5)
        s.k[torch.isnan(s.k)] = fill
        cache, args = s.device(), (s.q.cuda(), s.q_pos.cuda(), s.start.cuda())
        out, lse = torch.zeros(n, nq, hd, dtype=s.dt, device="cuda"), torch.zeros(n, nq, device="cuda")
        w = torch.zeros(s.pos.shape, device="cuda")
        cache.attention(*args, out, lse=lse, causal=False, softcap=20.0)
        cache.key_weight(*args, lse, weight_out=w, weight=torch.zeros_like(w), causal=False, softcap=20.0)
        assert torch.isfinite(w).all()
        results.append((lse, w))
    for r in results[1:]:
        assert [torch.equal(a, b) for a, b in zip(r, results[0])] == [True] * 2


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("mask", [dict(), dict(softcap=20.0), dict(slopes=True)], ids=lambda m: "-".join(m) or "plain")
@pytest.mark.parametrize("dtype,hd,nq", [("bf16", 128, 8), ("bf16", 64, 6), ("f32", 64, 4), ("bf16", 136, 4)])
@pytest.mark.parametrize("n", [5, 200])
def test_queries_without_an_lse_add_nothing_to_key_weights(B, dtype, hd, nq, n, mask, bad):
    """Rows of padding, lse = -inf, whatever their q holds, beside rows that see every key of a tile."""
    s = Setup(B, [(n, 500)], nq, 2, hd, 16, dtype, seed=14)
    m = mask_of(mask, nq, 1)
    cache = s.device()
    _, lse = s.check_attention(cache, **m)
    s.q[2:n:7] = bad
    lse[2::7] = -math.inf
    clean = s.q.clone()
    clean[2:n:7] = 0
    dev = {k: v.cuda() if torch.is_tensor(v) else v for k, v in m.items()}
    got = []
    for q in (s.q, clean):
        w = torch.zeros(s.pos.shape, device="cuda")
        cache.key_weight(q.cuda(), s.q_pos.cuda(), s.start.cuda(), lse, weight_out=w, weight=torch.zeros_like(w), **dev)
        got.append(w)
    assert torch.isfinite(got[0]).all() and torch.equal(got[0], got[1])
    s.q = clean
    s.check_weight(cache, lse, **m)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_pages_and_lengths_are_bounded(B, dtype):
    s = Setup(B, [(4, 100), (4, 60)], 8, 2, 64, 16, dtype, seed=8)
    s.table[0, 2] = 10 ** 6
    s.table[0, 3] = -1
    cache = s.device()
    _, lse = s.check_attention(cache)
    assert int(s.status) & B.PAGED_BAD_PAGE
    s.check_weight(cache, lse)
    # a length beyond the table is cut to it: every row of the (last, bad) pages is absent
    cache.length[1] = 10 ** 6
    s.length[1] = 60
    _, lse = s.check_attention(cache)
    cache.length[1] = -5
    s.length[1] = 0
    s.check_attention(cache)


@pytest.mark.parametrize("dtype,hd", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64), ("f32", 256)])
@pytest.mark.parametrize("n", [4, 150])
def test_every_call_reports_bad_pages(B, dtype, hd, n):
    s = Setup(B, [(n, 400), (4, 60)], 8, 2, hd, 16, dtype, seed=8)
    s.table[0, 2] = 10 ** 6
    cache, args = s.device(), (s.q.cuda(), s.q_pos.cuda(), s.start.cuda())
    out, lse = torch.zeros(s.rows, 8, hd, dtype=s.dt, device="cuda"), torch.zeros(s.rows, 8, device="cuda")
    w, p, length = torch.zeros(s.pos.shape, device="cuda"), torch.zeros_like(cache.pos), torch.zeros_like(cache.length)
    end = s.length.cuda()
    for call in (lambda: cache.attention(*args, out, lse=lse), lambda: cache.key_weight(*args, lse, weight_out=w),
                 lambda: cache.evict(50, 5, end, weight_out=w, pos_out=p, length_out=length),
                 lambda: cache.evict(1000, 5, end, weight_out=w, pos_out=p, length_out=length)):
        s.status.zero_()
        call()
        assert int(s.status) == B.PAGED_BAD_PAGE


def test_an_eviction_of_rows_that_no_cta_holds_reports_bad_pages(B):
    ps, pages = 1024, 1024
    shape = (pages, 1, ps)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].contiguous()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.arange(pages * ps, dtype=torch.int32, device="cuda").view(shape)
    k = torch.zeros(*shape, 8, device="cuda")
    c = B.PagedCache(k, k.clone(), pos, table, torch.tensor([pages * ps], dtype=torch.int32, device="cuda"), weight=torch.rand(shape, device="cuda"), status=status)
    c.evict(pages * ps - 3000, 0, torch.tensor([pages * ps], dtype=torch.int32, device="cuda"))
    assert int(status) == 0
    c.length.fill_(pages * ps)
    table[0, 700] = pages
    c.evict(pages * ps - 3000, 0, torch.tensor([pages * ps], dtype=torch.int32, device="cuda"))
    assert int(status) == B.PAGED_BAD_PAGE


@pytest.mark.parametrize("dtype,hd", [("bf16", 64), ("bf16", 256), ("f32", 64)])
@pytest.mark.parametrize("n", [4, 150])
@pytest.mark.parametrize("length", [10 ** 6, -5])
def test_every_call_reports_lengths_that_the_table_cannot_have(B, dtype, hd, n, length):
    s = Setup(B, [(n, 320), (4, 60)], 8, 2, hd, 16, dtype, seed=8, spare=0)
    cache, args = s.device(), (s.q.cuda(), s.q_pos.cuda(), s.start.cuda())
    out, lse = torch.zeros(s.rows, 8, hd, dtype=s.dt, device="cuda"), torch.zeros(s.rows, 8, device="cuda")
    w, p, left = torch.zeros(s.pos.shape, device="cuda"), torch.zeros_like(cache.pos), torch.zeros_like(cache.length)
    kv = torch.zeros(s.rows, 2, hd, dtype=s.dt, device="cuda")
    end = s.length.cuda()
    cache.attention(*args, out, lse=lse)
    assert int(s.status) == 0
    cache.length[0] = length
    for call in (lambda: cache.attention(*args, out, lse=lse), lambda: cache.key_weight(*args, lse, weight_out=w),
                 lambda: cache.evict(50, 5, end, weight_out=w, pos_out=p, length_out=left),
                 lambda: cache.append(s.q.cuda(), kv, kv, s.q_pos.cuda(), s.start.cuda(), out)):
        s.status.zero_()
        call()
        assert int(s.status) == B.PAGED_BAD_ROWS


def test_row_ranges_beyond_the_tensor_are_cut(B):
    s = Setup(B, [(4, 100), (4, 60)], 8, 2, 64, 16, seed=8)
    cache = s.device()
    start = torch.tensor([-3, 4, 10 ** 6], dtype=torch.int32, device="cuda")
    out = torch.zeros(8, 8, 64, dtype=torch.bfloat16, device="cuda")
    ref = torch.zeros_like(out)
    cache.attention(s.q.cuda(), s.q_pos.cuda(), s.start.cuda(), ref)
    cache.attention(s.q.cuda(), s.q_pos.cuda(), start, out)
    assert torch.equal(out, ref)


@pytest.mark.parametrize("dtype,nq,nkv,hd", [("bf16", 32, 8, 128), ("f32", 8, 4, 64), ("bf16", 28, 4, 64)])
@pytest.mark.parametrize("window", [0, 700])
def test_long_rows_split_over_many_ctas(B, dtype, nq, nkv, hd, window):
    """One row over thousands of keys, with and without a hint of the length; a hint that is too small changes nothing
    but the split."""
    s = Setup(B, [(2, 5003), (1, 1)], nq, nkv, hd, 64, dtype, seed=9)
    cache = s.device()
    for max_len in (0, 64, 5003):
        _, lse = s.check_attention(cache, window=window, max_len=max_len)
        s.check_weight(cache, lse, window=window, max_len=max_len)


def test_many_sequences(B):
    lens = [(i % 3, 1 + (i * 37) % 90 + i % 3) for i in range(150)]
    s = Setup(B, lens, 4, 2, 64, 8, seed=10)
    cache = s.device()
    _, lse = s.check_attention(cache, prefix=torch.arange(150, dtype=torch.int32))
    s.check_weight(cache, lse, prefix=torch.arange(150, dtype=torch.int32))


def test_no_rows(B):
    s = Setup(B, [(0, 10), (0, 3)], 4, 2, 64, 16, seed=11)
    cache = s.device()
    lse = torch.zeros(0, 4, device="cuda")
    cache.attention(s.q.cuda(), s.q_pos.cuda(), s.start.cuda(), torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda"), lse=lse)
    s.check_weight(cache, lse)
    empty = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    cache.append(s.q.cuda(), empty, empty, s.q_pos.cuda(), s.start.cuda(), s.q.cuda())


@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("f32", 64)])
def test_index_arrays_may_start_at_any_element(B, dtype, hd):
    """Slices of an engine's step buffers: everything that is read an element at a time."""
    s = Setup(B, [(9, 300), (3, 50), (1, 7)], 8, 2, hd, 16, dtype, seed=15)
    g = torch.Generator().manual_seed(1)
    new = [torch.randn(13, h, hd, generator=g).to(s.dt).cuda() for h in (8, 2, 2)]
    results = []
    for off in (0, 1, 2, 3):
        def put(t):
            flat = torch.zeros(t.numel() + off, dtype=t.dtype, device="cuda")
            flat[off:] = t.flatten().cuda()
            return flat[off:].view(t.shape)
        s.status = put(torch.zeros(1, dtype=torch.int32))
        c = B.PagedCache(s.k.cuda(), s.v.cuda(), s.pos.cuda(), put(s.table), put(s.length), weight=s.weight.cuda(), status=s.status)
        start, q_pos = put(s.start), put(s.q_pos)
        q, out, lse = torch.zeros_like(new[0]), torch.zeros_like(new[0]), put(torch.zeros(13, 8))
        c.append(*new, q_pos, start, q, rope_pos=put(torch.stack([s.q_pos, s.q_pos // 3])), pair_axis=bytes([0, 1] * (hd // 4)))
        mask = dict(slopes=put(torch.linspace(0, 0.1, 8)), prefix=put(torch.tensor([3, 0, 1], dtype=torch.int32)), window=100)
        c.attention(q, q_pos, start, out, lse=lse, **mask)
        c.key_weight(q, q_pos, start, lse, **mask)
        left = put(torch.zeros(3, dtype=torch.int32))
        c.evict(40, 5, put(s.length), length_out=left)
        assert int(s.status) == 0
        results.append([t.clone() for t in (c.k, c.v, c.pos, c.weight, q, out, lse, left)])
    for r in results[1:]:
        assert all(torch.equal(torch.nan_to_num(x.float(), 55.0), torch.nan_to_num(y.float(), 55.0)) for x, y in zip(r, results[0]))


@pytest.mark.parametrize("window", [0, 60])
def test_the_same_call_gives_the_same_bits(B, window):
    s = Setup(B, [(40, 900), (1, 500)], 8, 2, 128, 16, seed=12)
    cache = s.device()
    outs = []
    for _ in range(3):
        out, lse = torch.zeros(41, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(41, 8, device="cuda")
        w = torch.zeros(s.pos.shape, device="cuda")
        cache.attention(s.q.cuda(), s.q_pos.cuda(), s.start.cuda(), out, lse=lse, window=window)
        cache.key_weight(s.q.cuda(), s.q_pos.cuda(), s.start.cuda(), lse, weight_out=w, window=window)
        outs.append((out, lse, w))
    for o in outs[1:]:
        assert all(torch.equal(torch.nan_to_num(x), torch.nan_to_num(y)) for x, y in zip(o, outs[0]))


# ---- append ------------------------------------------------------------------------------

@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("lens,nq,nkv,hd,ps,dtype,axes,pairs", [
    ([(1, 1)], 4, 2, 16, 8, "f32", 1, 8),
    ([(5, 30), (0, 9), (3, 3)], 8, 4, 64, 16, "bf16", 3, 32),
    ([(16, 200)], 32, 8, 128, 64, "bf16", 1, 64),
    ([(2, 9), (7, 25)], 6, 2, 80, 16, "bf16", 2, 33),
    ([(3, 12)], 4, 1, 256, 8, "f32", 4, 128),
    ([(4, 12)], 4, 4, 8, 8, "bf16", 1, 0),
    ([(130, 300)], 3, 1, 96, 32, "f32", 1, 5),
    ([(1, 5)] * 70, 2, 1, 64, 8, "bf16", 1, 32),
])
def test_append(B, lens, nq, nkv, hd, ps, dtype, axes, pairs, norm, neox):
    s = Setup(B, lens, nq, nkv, hd, ps, dtype, seed=20 + hd, lead=1, tail=2)
    r = np.random.default_rng(hd + pairs)
    T = s.rows
    rope_pos = np.stack([r.integers(0, 10 ** (2 + 2 * i), T) for i in range(axes)]).astype(np.int32)
    axis = bytes(int(x) for x in r.integers(0, axes, pairs))
    qkv = torch.randn(T, nq + 2 * nkv, hd, generator=torch.Generator().manual_seed(hd)).to(s.dt)
    gains = [(1 + 0.2 * torch.randn(hd, generator=torch.Generator().manual_seed(i))).to(s.dt) if norm else None for i in (1, 2)]
    row_pos = torch.from_numpy(r.integers(0, 1 << 30, T).astype(np.int32))
    cache = s.device()
    dev = qkv.cuda()
    q_out = torch.full((T, nq, hd), 77.0, dtype=s.dt, device="cuda")
    cache.append(dev[:, :nq], dev[:, nq:nq + nkv], dev[:, nq + nkv:], row_pos.cuda(), s.start.cuda(), q_out, rope_pos=torch.from_numpy(rope_pos).cuda(), pair_axis=axis,
                 theta=1e6, neox=neox, q_norm=None if gains[0] is None else gains[0].cuda(), k_norm=None if gains[1] is None else gains[1].cuda())
    torch.cuda.synchronize()
    o = s.oracle()
    x = host(qkv)
    g = [None if y is None else host(y) for y in gains]
    want = P.append(o, x[:, :nq], x[:, nq:nq + nkv], x[:, nq + nkv:], row_pos.numpy(), s.start.numpy(), rope_pos, axis, 1e6, neox, g[0], g[1], 1e-6)
    a, b = int(s.start[0]), int(s.start[-1])
    got = host(q_out)
    assert (got[:a] == 77).all() and (got[b:] == 77).all()

    def close(got, want):
        # |a| + |b| of a pair is at most twice the row's largest magnitude
        near = np.abs(np.where(np.isfinite(want), want, 0)).max(-1, keepdims=True) * 2
        bad = ~((np.abs(got - want) <= unit(dtype) * np.abs(want) + (hd + 16) * EPS * near) | (np.isnan(got) & np.isnan(want)))
        assert not bad.any(), np.abs(got - want)[bad].max()

    close(got[a:b], want[a:b])
    close(host(cache.k), o["k"])
    assert np.array_equal(host(cache.v), o["v"], equal_nan=True)
    assert np.array_equal(cache.pos.cpu().numpy(), o["pos"]) and np.array_equal(host(cache.weight), o["weight"], equal_nan=True)
    assert int(s.status) == 0


@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("hd,pairs,dtype", [(64, 0, "bf16"), (128, 16, "bf16"), (128, 16, "f32"), (80, 8, "f32"), (96, 24, "bf16"), (64, 5, "bf16"), (128, 33, "f32")])
def test_append_leaves_what_is_not_rotated(B, hd, pairs, dtype, norm, neox):
    """Infinities, NaN and -0 in dimensions that are not rotated stay where they are, in both kernels."""
    s = Setup(B, [(6, 20)], 4, 2, hd, 16, dtype, seed=32)
    x = torch.randn(6, 8, hd, generator=torch.Generator().manual_seed(pairs))
    x[0, :, -3:] = -0.0
    x[1, :, -1] = math.inf
    x[2, :, -2] = -math.inf
    x[3, :, -2:] = math.inf
    x[4, :, -1] = math.nan
    x[5, :, 2 * pairs] = math.inf
    x = x.to(s.dt)
    gains = [(1 + 0.2 * torch.randn(hd, generator=torch.Generator().manual_seed(i))).to(s.dt) if norm else None for i in (1, 2)]
    rope_pos = torch.tensor([[3, 10, 200, 7, 5000, 1]], dtype=torch.int32)
    cache, dev = s.device(), x.cuda()
    q_out = torch.full((6, 4, hd), 77.0, dtype=s.dt, device="cuda")
    cache.append(dev[:, :4], dev[:, 4:6], dev[:, 6:], s.q_pos.cuda(), s.start.cuda(), q_out, rope_pos=rope_pos.cuda(), pair_axis=bytes(pairs), theta=1e4, neox=neox,
                 q_norm=None if gains[0] is None else gains[0].cuda(), k_norm=None if gains[1] is None else gains[1].cuda())
    o, y = s.oracle(), host(x)
    g = [None if t is None else host(t) for t in gains]
    with np.errstate(invalid="ignore"):
        want = P.append(o, y[:, :4], y[:, 4:6], y[:, 6:], s.q_pos.numpy(), s.start.numpy(), rope_pos.numpy(), bytes(pairs), 1e4, neox, g[0], g[1], 1e-6)
    rows = [(int(s.table[0, r // 16]), r % 16) for r in range(14, 20)]
    keys = np.stack([o["k"][p, :, j] for p, j in rows])
    got = [host(q_out), np.stack([host(cache.k[p, :, j]) for p, j in rows])]
    for a, b, given in ((got[0], want, y[:, :4]), (got[1], keys, y[:, 4:6])):
        assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(np.isinf(a), np.isinf(b))
        assert (a[np.isinf(b)] == b[np.isinf(b)]).all()
        near = np.abs(np.where(np.isfinite(b), b, 0)).max(-1, keepdims=True) * 2
        fine = np.isfinite(b)
        assert (np.abs(a[fine] - b[fine]) <= (unit(dtype) * np.abs(b) + (hd + 16) * EPS * near)[fine]).all()
        if not norm:
            still, was = a[..., 2 * pairs:], given[..., 2 * pairs:]
            assert np.array_equal(still, was, equal_nan=True) and np.array_equal(np.signbit(still)[~np.isnan(was)], np.signbit(was)[~np.isnan(was)])
    assert np.array_equal(host(cache.v), o["v"], equal_nan=True)


def test_append_in_place_and_far_positions(B):
    """q_out = q, and angles of positions up to 2^31 - 1: turns of pair 0 there are exact to 2^-24 of a turn."""
    s = Setup(B, [(3, 3)], 2, 1, 64, 8, "f32", seed=30)
    cache = s.device()
    pos = torch.tensor([[2 ** 31 - 1, 10 ** 9 + 7, 123456789]], dtype=torch.int32)
    q = s.q.cuda()
    kv = torch.randn(3, 1, 64, generator=torch.Generator().manual_seed(1))
    cache.append(q, kv.cuda(), kv.cuda(), s.q_pos.cuda(), s.start.cuda(), q, rope_pos=pos.cuda(), pair_axis=bytes(32), theta=1e4)
    want = P.append(s.oracle(), host(s.q), host(kv), host(kv), s.q_pos.numpy(), s.start.numpy(), pos.numpy(), bytes(32), 1e4, True, None, None, 1e-6)
    # the oracle's own angle in fp64 is off by 2^-53 of up to 2^31 radians: 2^-22
    np.testing.assert_allclose(host(q), want, atol=float(np.abs(host(s.q)).max()) * 2 * (2.0 ** -22 + 16 * EPS))


def test_append_beyond_what_is_there(B):
    """More new rows than the length says, a length beyond the table and a page outside the pool: nothing is written there."""
    s = Setup(B, [(4, 2 + 4), (4, 40)], 4, 2, 64, 16, seed=31)
    s.table[1, 2] = -1                                   # rows 32.. of sequence 1: its new rows
    s.length[0] = 2
    cache = s.device()
    k0, q = cache.k.clone(), s.q.cuda()
    kv = torch.ones(8, 2, 64, dtype=torch.bfloat16, device="cuda")
    q_out = torch.zeros_like(q)
    cache.append(q, kv, kv, s.q_pos.cuda(), s.start.cuda(), q_out)
    changed = (torch.nan_to_num(cache.k) != torch.nan_to_num(k0)).any(-1)
    page = int(s.table[0, 0])
    assert changed[page, :, :2].all() and int(changed.sum()) == 4
    assert torch.equal(q_out, q)
    assert int(s.status) == B.PAGED_BAD_PAGE | B.PAGED_BAD_ROWS
    cache.length[0] = 10 ** 6                            # cut to the table, whose last pages are outside the pool
    k0 = cache.k.clone()
    cache.append(q, kv, kv, s.q_pos.cuda(), s.start.cuda(), q_out)
    assert torch.equal(torch.nan_to_num(cache.k), torch.nan_to_num(k0))


# ---- eviction ------------------------------------------------------------------------------

@pytest.mark.parametrize("aliased", [False, True])
@pytest.mark.parametrize("lens,nkv,hd,ps,dtype,budget,recent,ties", [
    ([1, 2, 3], 2, 16, 8, "f32", 2, 0, False),
    ([300], 2, 64, 16, "bf16", 100, 10, False),
    ([300, 40, 0, 100, 101], 4, 128, 16, "bf16", 100, 30, True),
    ([2500], 1, 64, 64, "bf16", 2400, 64, False),
    ([2500, 1100], 2, 24, 32, "f32", 1, 0, True),
    ([700], 3, 256, 8, "bf16", 350, 350, False),
    ([700], 2, 64, 8, "bf16", 350, 500, True),
    ([90], 2, 64, 16, "bf16", 4000, 5, False),
    ([5000, 4100, 9], 2, 8, 128, "bf16", 4096, 1000, True),
    ([9000], 1, 64, 64, "bf16", 3000, 100, False),         # two to eight CTAs to a head
    ([20000, 6000], 2, 8, 16, "bf16", 9999, 0, True),
    ([40000], 1, 8, 256, "f32", 20000, 7, False),
])
def test_evict(B, lens, nkv, hd, ps, dtype, budget, recent, ties, aliased):
    s = Setup(B, [(0, n) for n in lens], nkv, nkv, hd, ps, dtype, seed=40 + hd, kept=True)
    g = torch.Generator().manual_seed(budget)
    if ties:
        s.weight = torch.where(torch.isnan(s.weight), s.weight, (s.weight * 4).round() / 2 - 0.5)
        s.weight[s.weight == 0] = -0.0
        odd = torch.rand(s.weight.shape, generator=g)
        s.weight[odd < 0.02] = math.nan
        s.weight[(odd > 0.02) & (odd < 0.04)] = math.inf
        s.weight[(odd > 0.04) & (odd < 0.06)] = -math.inf
        s.weight[(odd > 0.06) & (odd < 0.1)] = 0.0
    next_pos = 2 * s.length
    cache = s.device()
    o = s.oracle()
    if aliased:
        w_out, p_out, l_out = cache.weight, cache.pos, cache.length
        want_w, want_p = o["weight"].copy(), o["pos"].copy()
        cache.evict(budget, recent, next_pos.cuda())
    else:
        w_out, p_out, l_out = torch.full_like(cache.weight, 77.0), torch.full_like(cache.pos, 77), torch.full_like(cache.length, 77)
        want_w, want_p = np.full(o["weight"].shape, 77.0), np.full(o["pos"].shape, 77, dtype=np.int32)
        cache.evict(budget, recent, next_pos.cuda(), weight_out=w_out, pos_out=p_out, length_out=l_out)
    want_l = P.evict(o, budget, recent, next_pos.numpy(), want_w, want_p)
    assert np.array_equal(l_out.cpu().numpy(), want_l)
    assert np.array_equal(p_out.cpu().numpy(), want_p)
    assert np.array_equal(host(w_out), want_w, equal_nan=True)
    assert np.array_equal(host(cache.k), o["k"], equal_nan=True) and np.array_equal(host(cache.v), o["v"], equal_nan=True)
    assert int(s.status) == 0


def test_evict_rows_that_no_cta_holds(B):
    """A table of 2^20 rows, more than eight CTAs hold in shared memory, against torch's stable sort."""
    n, ps, budget = (1 << 20) - 5, 1024, 400001
    pages = (1 << 20) // ps
    g = torch.Generator(device="cuda").manual_seed(3)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None]
    shape = (pages, 1, ps)
    w = (torch.rand(shape, generator=g, device="cuda") * 1000).round()          # many equal ones
    pos = torch.zeros(shape, dtype=torch.int32, device="cuda")
    pos[table[0].long(), 0] = torch.arange(pages * ps, dtype=torch.int32, device="cuda").view(pages, ps)
    k = pos[..., None].expand(-1, -1, -1, 8).to(torch.float32).contiguous()
    c = B.PagedCache(k, -k, pos, table, torch.tensor([n], dtype=torch.int32, device="cuda"), weight=w)
    flat = w[table[0].long(), 0].flatten()[:n]
    keep = flat.sort(stable=True, descending=True).indices[:budget].sort().values
    late = keep[keep >= budget]
    holes = torch.ones(budget, dtype=torch.bool, device="cuda").index_fill(0, keep[keep < budget], False).nonzero().flatten()
    want = torch.arange(budget, device="cuda").index_copy(0, holes, late)
    c.evict(budget, 0, torch.tensor([n], dtype=torch.int32, device="cuda"))
    got = pos[table[0].long(), 0].flatten()[:budget]
    assert torch.equal(got.long(), want) and int(c.length[0]) == budget
    assert torch.equal(w[table[0].long(), 0].flatten()[:budget], flat[want])
    assert torch.equal(k[table[0].long(), 0].reshape(-1, 8)[:budget, 3].long(), want) and torch.equal(c.v, -k)


# ---- together ------------------------------------------------------------------------------

class Round:
    """A serving loop's tensors: two sequences that verify blocks, trim, and evict."""

    def __init__(self, B, dtype, hd, seed=50):
        s = Setup(B, [(0, 90), (0, 47)], 8, 2, hd, 16, dtype, seed=seed, spare=1)
        # every table entry a page of its own, so that the sequences can grow
        width = 12
        s.table = torch.randperm(2 * width, generator=torch.Generator().manual_seed(seed))[: 2 * width].reshape(2, width).to(torch.int32)
        g = torch.Generator().manual_seed(seed + 1)
        shape = (2 * width, 2, 16)
        s.k, s.v = torch.randn(*shape, hd, generator=g).to(s.dt), torch.randn(*shape, hd, generator=g).to(s.dt)
        s.pos, s.weight = torch.zeros(shape, dtype=torch.int32), torch.rand(shape, generator=g)
        for q in range(2):
            for i in range(int(s.length[q])):
                s.pos[int(s.table[q, i // 16]), :, i % 16] = i
        self.s, self.block = s, 8
        self.cache = s.device()
        self.next = s.length.cuda().clone()
        self.start = torch.tensor([0, 8, 16], dtype=torch.int32, device="cuda")
        z = lambda *shape, **kw: torch.zeros(*shape, device="cuda", **kw)  # noqa: E731
        self.q, self.k, self.v = z(16, 8, hd, dtype=s.dt), z(16, 2, hd, dtype=s.dt), z(16, 2, hd, dtype=s.dt)
        self.rope = z(1, 16, dtype=torch.int32)
        self.q_out, self.out, self.lse = z(16, 8, hd, dtype=s.dt), z(16, 8, hd, dtype=s.dt), z(16, 8)
        self.drop = z(2, dtype=torch.int32)
        self.axis = bytes(hd // 2)
        self.steps = torch.arange(8, dtype=torch.int32, device="cuda")

    def fill(self, seed):
        g = torch.Generator().manual_seed(seed)
        for t in (self.q, self.k, self.v):
            t.copy_(torch.randn(t.shape, generator=g).to(t.dtype))
        self.drop.copy_(torch.randint(0, 8, (2,), generator=g).to(torch.int32))

    def work(self):
        c = self.cache
        c.length += 8
        self.rope.copy_((self.next[:, None] + self.steps).view(1, 16))
        c.append(self.q, self.k, self.v, self.rope[0], self.start, self.q_out, rope_pos=self.rope, pair_axis=self.axis)
        c.attention(self.q_out, self.rope[0], self.start, self.out, lse=self.lse, window=120)
        c.key_weight(self.q_out, self.rope[0], self.start, self.lse, decay=0.95, window=120)
        c.length -= self.drop                             # the rejected rows
        self.next += 8 - self.drop
        c.evict(100, 40, self.next)

    def state(self):
        c = self.cache
        return [t.clone() for t in (c.k, c.v, c.pos, c.weight, c.length, self.next, self.q_out, self.out, self.lse)]


@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("f32", 64)])
def test_rounds_together_follow_the_oracle(B, dtype, hd):
    r = Round(B, dtype, hd)
    c, s = r.cache, r.s
    for step in range(6):
        r.fill(step)
        # the oracle starts every round from the GPU's cache, so that roundings do not add up
        o = {"k": host(c.k), "v": host(c.v), "pos": c.pos.cpu().numpy(), "weight": host(c.weight), "table": s.table.numpy(),
             "length": c.length.cpu().numpy() + 8}
        nxt, drop = r.next.cpu().numpy().copy(), r.drop.cpu().numpy()
        r.work()
        torch.cuda.synchronize()
        row_pos = (nxt[:, None] + np.arange(8)).reshape(-1).astype(np.int32)
        start = np.array([0, 8, 16])
        P.append(o, host(r.q), host(r.k), host(r.v), row_pos, start, row_pos[None], r.axis, 1e6, True, None, None, 1e-6)
        q, lse = host(r.q_out), host(r.lse)
        o["k"] = np.float64(torch.from_numpy(o["k"]).to(s.dt).double().numpy())
        want, want_lse, mag = P.attention(o, q, row_pos, start, s.scale, window=120)
        s.start, s.q_pos, s.rows, s.length, s.q, s.k = torch.tensor([0, 8, 16]), torch.from_numpy(row_pos), 16, torch.from_numpy(o["length"]), r.q_out.cpu(), c.k.cpu()
        # K in the pages may differ by a rounding from the oracle's where a value sat between two: another half step of each score
        dt = s.score_error(0.0, None) + (2 * unit(dtype)) * 0.02 * np.sqrt(hd)
        off = np.abs(host(r.out) - want) - (unit(dtype) * np.abs(want) + (2 * dt + 2.0 ** -8) * mag)
        assert (off <= 0).all()
        w, _ = P.key_weight(o, q, row_pos, start, lse, o["weight"], float(np.float32(0.95)), o["weight"].copy(), s.scale, window=120)
        o["weight"] = w
        o["length"] = o["length"] - drop
        # eviction against the GPU's own weights would need them before it; the lengths, the number of rows each head
        # keeps and the protected positions are the oracle's
        assert c.length.cpu().numpy().tolist() == np.minimum(o["length"], 100).tolist()
        for q_ in range(2):
            n = int(c.length[q_])
            rows = P.rows_of({"k": c.k, "table": s.table, "length": c.length}, q_, n)
            for h in range(2):
                got = sorted(int(c.pos[p, h, j]) for p, j in rows)
                end = int(r.next[q_])
                assert len(set(got)) == n and got[-1] == end - 1 and got[-min(40, n):] == list(range(end - min(40, n), end))


def test_rounds_captured_in_graphs_and_replayed(B):
    """Two rounds of one loop captured in two graphs, replayed in turn on another stream, against the same calls made one by one."""
    a, b = Round(B, "bf16", 128), Round(B, "bf16", 128)
    warm = Round(B, "bf16", 128)
    warm.fill(0)
    warm.work()
    graphs = []
    side = torch.cuda.Stream()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.work()
        graphs.append(g)
    for step in range(6):
        a.fill(step)
        a.work()
        b.fill(step)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[step % 2].replay()
        torch.cuda.synchronize()
        for x, y in zip(a.state(), b.state()):
            assert torch.equal(x, y)


def test_calls_on_two_streams_at_once(B):
    """Calls of two caches on two streams, many in flight, each with a workspace of its own."""
    sets = [Setup(B, [(1, 2000), (2, 900)], 8, 2, 128, 32, seed=60 + i) for i in range(2)]
    caches = [s.device() for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    args = [(s.q.cuda(), s.q_pos.cuda(), s.start.cuda()) for s in sets]
    outs = [[torch.zeros(3, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(20)] for _ in sets]
    torch.cuda.synchronize()
    for i in range(20):
        for c, st, x, o in zip(caches, streams, args, outs):
            c.attention(*x, o[i], stream=st)
    torch.cuda.synchronize()
    for s, c, o in zip(sets, caches, outs):
        first, _ = s.check_attention(c)
        assert all(torch.equal(x, first) for x in o)


def dense64(s, cache):
    """out, sum p |v| and lse of causal attention in torch fp64 on the GPU, one sequence and kv head after the other."""
    q, out = cache.q64, torch.zeros(s.rows, s.nq, s.hd, dtype=torch.float64, device="cuda")
    mag, lse, G = torch.zeros_like(out), torch.zeros(s.rows, s.nq, dtype=torch.float64, device="cuda"), s.nq // s.nkv
    ps = cache.k.shape[2]
    for i in range(len(s.length)):
        a, b, n = int(s.start[i]), int(s.start[i + 1]), int(s.length[i])
        pages = cache.table[i, :-(-n // ps)].long()
        for h in range(s.nkv):
            k, v, pos = (t[pages, h].flatten(0, 1)[:n] for t in (cache.k, cache.v, cache.pos))
            t = torch.einsum("ngd,ld->ngl", q[a:b, h * G:(h + 1) * G], k.double()) * s.scale
            t = t.masked_fill((pos[None] > s.q_pos[a:b].cuda()[:, None])[:, None], -math.inf)
            lse[a:b, h * G:(h + 1) * G] = t.logsumexp(-1)
            p = t.softmax(-1)
            out[a:b, h * G:(h + 1) * G], mag[a:b, h * G:(h + 1) * G] = p @ v.double(), p @ v.double().abs()
    return host(out), host(lse), host(mag)


@pytest.mark.parametrize("n,lens,nq,nkv,hd,dtype", [
    (1, [9000 - 150 * i for i in range(44)], 32, 8, 128, "bf16"),        # more tiles to a CTA, and CTAs to the GPU, than stages
    (30, [5000 - 300 * i for i in range(12)], 16, 8, 64, "bf16"),
    (500, [6000, 500, 4321], 32, 8, 128, "bf16"),
    (300, [6000, 2500, 300], 8, 1, 64, "bf16"),
    (7, [6000 - 500 * i for i in range(10)], 16, 8, 128, "f32"),
])
def test_a_loaded_gpu(B, n, lens, nq, nkv, hd, dtype):
    """Long sequences on every SM at once, the same call many times in a row."""
    g = torch.Generator(device="cuda").manual_seed(len(lens))
    s = Setup.__new__(Setup)
    s.B, s.dtype, s.hd, s.nq, s.nkv, s.scale = B, dtype, hd, nq, nkv, hd ** -0.5
    s.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    ps, width, S = 64, -(-max(lens) // 64), len(lens)
    s.rows, s.length, s.start = n * S, torch.tensor(lens, dtype=torch.int32), torch.arange(0, n * S + 1, n, dtype=torch.int32)
    s.q_pos = torch.cat([torch.arange(l - n, l) for l in lens]).to(torch.int32)
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(s.dt)  # noqa: E731
    s.k, s.v = normal(S * width, nkv, ps, hd), normal(S * width, nkv, ps, hd)
    s.table = torch.randperm(S * width, generator=torch.Generator().manual_seed(1)).reshape(S, width).to(torch.int32)
    s.pos = torch.zeros(S * width, nkv, ps, dtype=torch.int32)
    s.pos[s.table.long()] = torch.arange(width * ps, dtype=torch.int32).reshape(1, width, 1, ps).expand(S, width, nkv, ps)
    s.weight = torch.zeros(S * width, nkv, ps)
    s.q = normal(s.rows, nq, hd)
    cache = s.device()
    cache.q64 = s.q.double()
    want, want_lse, mag = dense64(s, cache)
    outs = []
    for _ in range(20):
        out, lse = torch.full((s.rows, nq, hd), 77.0, dtype=s.dt, device="cuda"), torch.full((s.rows, nq), 77.0, device="cuda")
        cache.attention(s.q, s.q_pos.cuda(), s.start.cuda(), out, lse=lse)
        outs.append((out, lse))
    torch.cuda.synchronize()
    assert int(s.status) == 0
    s.compare(host(outs[0][0]), host(outs[0][1]), want, want_lse, mag, 0.0, None)
    assert all(torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1]) for o in outs)
    w = torch.zeros(s.pos.shape, device="cuda")
    cache.key_weight(s.q, s.q_pos.cuda(), s.start.cuda(), outs[0][1], weight=w, weight_out=w)
    # each query gives every kv head's rows as much as it has heads there, in all
    per = w[cache.table.long()].sum((1, 3)).double()
    assert (per - n * (nq // nkv)).abs().max() <= n * (nq // nkv) * 2 * (s.score_error(0.0, None) + 2.0 ** -18)


def capped64(s, cache, softcap=0.0):
    """dense64 with scores under a cap: its cache's k scaled into t, capped, one sequence and kv head after the other."""
    if not softcap:
        return dense64(s, cache)
    out, G, ps = torch.zeros(s.rows, s.nq, s.hd, dtype=torch.float64, device="cuda"), s.nq // s.nkv, cache.k.shape[2]
    mag, lse = torch.zeros_like(out), torch.zeros(s.rows, s.nq, dtype=torch.float64, device="cuda")
    for i in range(len(s.length)):
        a, b, n = int(s.start[i]), int(s.start[i + 1]), int(s.length[i])
        pages = cache.table[i, :-(-n // ps)].long()
        for h in range(s.nkv if b > a else 0):
            k, v, pos = (t[pages, h].flatten(0, 1)[:n] for t in (cache.k, cache.v, cache.pos))
            heads = slice(h * G, (h + 1) * G)
            t = softcap * torch.tanh(torch.einsum("ngd,ld->ngl", cache.q64[a:b, heads], k.double()) * s.scale / softcap)
            t = t.masked_fill((pos[None] > s.q_pos[a:b].cuda()[:, None])[:, None], -math.inf)
            p = t.softmax(-1)
            lse[a:b, heads], out[a:b, heads], mag[a:b, heads] = t.logsumexp(-1), p @ v.double(), p @ v.double().abs()
    return host(out), host(lse), host(mag)


@pytest.mark.parametrize("mask", [dict(), dict(softcap=30.0)], ids=lambda m: "-".join(m) or "plain")
@pytest.mark.parametrize("spare,max_len", [(0, 0), (400, 0), (400, 9000)])
def test_prompt_chunks_with_decode_rows_in_long_tables(B, spare, max_len, mask):
    """Chunks, verify blocks and single tokens of long sequences in one call, many times in a row, in tables that are far longer
    than any of them."""
    lens = [(700, 6000), (1, 9000), (16, 5000), (130, 130), (1, 1), (0, 700)] + [(1, 8500 - 200 * i) for i in range(30)]
    nq, nkv, hd, ps = 16, 4, 128, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    s = Setup.__new__(Setup)
    s.B, s.dtype, s.hd, s.nq, s.nkv, s.scale, s.dt = B, "bf16", hd, nq, nkv, hd ** -0.5, torch.bfloat16
    S, held = len(lens), -(-max(n for _, n in lens) // ps)
    s.length = torch.tensor([n for _, n in lens], dtype=torch.int32)
    s.start = torch.tensor([0] + [n for n, _ in lens], dtype=torch.int32).cumsum(0).to(torch.int32)
    s.rows = int(s.start[-1])
    s.q_pos = torch.cat([torch.arange(n - k, n) for k, n in lens]).to(torch.int32)
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(s.dt)  # noqa: E731
    s.k, s.v, s.q = normal(S * held, nkv, ps, hd), normal(S * held, nkv, ps, hd), normal(s.rows, nq, hd)
    pages = torch.randperm(S * held, generator=torch.Generator().manual_seed(1)).reshape(S, held).to(torch.int32)
    s.table = torch.cat([pages, torch.full((S, spare), -1, dtype=torch.int32)], 1).contiguous()
    s.pos = torch.zeros(S * held, nkv, ps, dtype=torch.int32)
    s.pos[pages.long()] = torch.arange(held * ps, dtype=torch.int32).reshape(1, held, 1, ps).expand(S, held, nkv, ps)
    s.weight = torch.zeros(S * held, nkv, ps)
    cache = s.device()
    cache.q64 = s.q.double()
    outs = []
    for _ in range(10):
        out, lse = torch.full((s.rows, nq, hd), 77.0, dtype=s.dt, device="cuda"), torch.full((s.rows, nq), 77.0, device="cuda")
        cache.attention(s.q, s.q_pos.cuda(), s.start.cuda(), out, lse=lse, max_len=max_len, **mask)
        outs.append((out, lse))
    torch.cuda.synchronize()
    assert int(s.status) == 0 and all(torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1]) for o in outs)
    want, want_lse, mag = capped64(s, cache, **mask)
    s.compare(host(outs[0][0]), host(outs[0][1]), want, want_lse, mag, mask.get("softcap", 0.0), None)


def test_offsets_beyond_32_bits(B):
    """A pool of more than 2^31 elements (5 GB): rows in its last pages."""
    pages, nkv, ps, hd = 1100, 8, 1024, 256
    shape = (pages, nkv, ps)
    k, v = torch.zeros(*shape, hd, dtype=torch.bfloat16, device="cuda"), torch.zeros(*shape, hd, dtype=torch.bfloat16, device="cuda")
    pos, weight = torch.zeros(shape, dtype=torch.int32, device="cuda"), torch.zeros(shape, device="cuda")
    table = torch.tensor([[pages - 1, 0]], dtype=torch.int32, device="cuda")
    length = torch.tensor([40], dtype=torch.int32, device="cuda")
    c = B.PagedCache(k, v, pos, table, length, weight=weight)
    g = torch.Generator().manual_seed(1)
    new = [torch.randn(40, h, hd, generator=g).to(torch.bfloat16).cuda() for h in (16, 8, 8)]
    at = torch.arange(40, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    q = torch.zeros_like(new[0])
    c.append(*new, at, start, q)
    assert torch.equal(k[pages - 1, :, :40].transpose(0, 1), new[1])
    out, lse = torch.zeros_like(q), torch.zeros(40, 16, device="cuda")
    c.attention(q, at, start, out, lse=lse)
    kk, vv = (x.float().transpose(0, 1).repeat_interleave(2, 0) for x in new[1:])
    t = (q.float().transpose(0, 1) @ kk.transpose(1, 2) / 16).masked_fill(at[:, None] < at[None], -math.inf)
    want = (t.softmax(-1) @ vv).transpose(0, 1)
    assert (out.float() - want).abs().max() < 0.05
    c.key_weight(q, at, start, lse)
    # nothing elsewhere: counted, as the two sums of the same 320 values may differ by their order's roundings (one
    # step of 640 is 2^-14)
    assert abs(float(weight[pages - 1, :, :40].sum()) - 40 * 16) < 0.1
    assert int(weight.count_nonzero()) == int(weight[pages - 1, :, :40].count_nonzero())
    c.evict(20, 5, torch.tensor([40], dtype=torch.int32, device="cuda"))
    assert int(length[0]) == 20 and (pos[pages - 1, :, :20].sort(-1).values[:, -5:] == at[35:]).all()
