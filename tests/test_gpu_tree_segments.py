"""GPU parity of tree attention where a batch is cut into segments of keys, which join in
a workspace, against the fp64 oracle (oracle/tree_oracle.py). Every test makes sure that its calls are cut:
few query tiles over short tables are clusters, which need no workspace. The tolerances
are those of test_gpu_paged.py."""

import math

import numpy as np
import pytest
import torch

from oracle import tree_oracle as T
from test_gpu_paged import host, mask_of
from test_gpu_tree import Trees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from block_speculative_decoding_dflash_gb300 import build
    build.build()
    from block_speculative_decoding_dflash_gb300 import binding
    return binding


def in_segments(s, cache, rows_of):
    """The last call's workspace is that of segments with partials of `rows_of` rows (128 and 256: one and two
    query tiles to a CTA, 16: the kernel of fp32 and large heads): two to five rounds of what runs at once."""
    at_once = 304 if rows_of == 16 and (s.hd <= 128 or s.dtype == "bf16") else 152
    left, unit = cache._tree_bytes[1] - 16 * s.rows, max(1, at_once // s.nkv) * s.nkv * rows_of * (s.hd + 2) * 4
    return left % unit == 0 and 2 <= left // unit <= 5


def batch(sizes, lengths, n):
    """n sequences of (new rows, cached rows), sizes and lengths in turn."""
    return [(sizes[i % len(sizes)], lengths[i % len(lengths)]) for i in range(n)]


# groups of query heads that do not divide 32, one query tile to a CTA: trees that are there once, twice and four
# times in their tile, in one batch, and a tree whose rows are there once alone
ODD_GROUPS = [
    (batch([40, 21, 30, 9, 15, 42], [2300, 650, 1400, 1024, 300], 24), 12, 4, 128),
    (batch([25, 13, 20, 6, 11], [700, 2100, 1290, 128], 22), 20, 4, 64),
    (batch([21, 11, 5, 9, 1, 0], [1500, 1800, 260], 23), 24, 4, 96),
    (batch([16, 18, 9, 4, 8], [2048, 900, 1700], 20), 28, 4, 128),
    ([(30, 9000)], 6, 2, 128),
]


@pytest.mark.parametrize("lens,nq,nkv,hd", ODD_GROUPS, ids=lambda x: f"{len(x)}x{x[0][0]}" if isinstance(x, list) else str(x))
def test_groups_that_do_not_divide_a_tile(B, lens, nq, nkv, hd):
    s = Trees(B, lens, nq, nkv, hd, 64, seed=nq, lead=1, tail=2)
    cache = s.device()
    first = s.check(cache)
    assert in_segments(s, cache, 128) and int(s.status) == 0
    for _ in range(20):
        out, lse = s.call(cache)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


EMPTY = [(9, 23, 3600, "bf16", 32, 8, 128), (3, 29, 3600, "bf16", 24, 8, 64), (9, 23, 1500, "f32", 16, 16, 64), (12, 60, 1500, "bf16", 16, 8, 128)]


@pytest.mark.parametrize("long,empty,length,dtype,nq,nkv,hd", EMPTY)
def test_new_rows_of_empty_sequences(B, long, empty, length, dtype, nq, nkv, hd):
    """Rows of sequences whose length is 0 see nothing and are reported, however many there are beside long texts."""
    lens = [(1, length if i < long else 1) for i in range(long + empty)]
    lens = lens[long:long + empty // 2] + lens[:long] + lens[long + empty // 2:]
    s = Trees(B, lens, nq, nkv, hd, 64, dtype, seed=long)
    s.length[[i for i, (_, n) in enumerate(lens) if n == 1]] = 0
    cache = s.device()
    s.check(cache)
    assert in_segments(s, cache, 128 if dtype == "bf16" else 16) and int(s.status) == B.PAGED_BAD_ROWS


# lens, nq, nkv, hd, page rows, dtype, rows of a segment's partials
SHAPES = [
    (batch([32, 9, 17, 1, 0, 20], [2300, 260, 1400, 1024, 700], 24), 16, 4, 128, 64, "bf16", 128),
    (batch([64, 40, 64, 3, 33], [1900, 300, 1200, 129], 16), 16, 4, 128, 32, "bf16", 256),       # two query tiles to a CTA
    (batch([36, 20, 30, 19], [1500, 2600, 640], 20), 28, 4, 64, 128, "bf16", 256),
    (batch([10, 1, 128, 70], [1100, 400, 2000], 12), 8, 8, 80, 16, "bf16", 128),
    (batch([3, 1, 2], [1300, 200, 1029], 30), 80, 2, 64, 16, "bf16", 128),                      # a token's heads alone are more than a quarter
    (batch([64, 1, 33, 150], [1500, 257, 900, 400], 24), 4, 4, 64, 64, "bf16", 128),
    ([(64, 9000)], 8, 2, 128, 64, "bf16", 256),
    ([(40, 9000)], 5, 1, 96, 256, "bf16", 256),
    (batch([1, 2, 5], [300, 1200], 40), 4, 2, 128, 32, "bf16", 128),                            # more sequences than are put in order
    ([(20, 2500), (3, 300), (33, 1100)], 6, 2, 256, 32, "bf16", 16),
    ([(17, 2000), (2, 1300), (40, 500), (0, 9)], 5, 1, 64, 16, "f32", 16),
    ([(9, 1200), (30, 1700)], 14, 2, 128, 64, "f32", 16),
    ([(20, 1500), (1, 700)], 6, 2, 200, 8, "f32", 16),
]
MASKS = [dict(), dict(window=20), dict(window=900), dict(window=30, prefix=200), dict(prefix=1000, window=5, softcap=5.0), dict(slopes=True),
         dict(softcap=5.0, slopes=True), dict(causal=False, window=16, softcap=20.0, slopes=True), dict(causal=False)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{s[0][0][0]}of{s[0][0][1]}-{s[1]}_{s[2]}x{s[3]}-{s[4]}-{s[5]}")
def test_segments_under_every_mask(B, shape):
    lens, nq, nkv, hd, ps, dtype, rows_of = shape
    s = Trees(B, lens, nq, nkv, hd, ps, dtype, seed=len(lens) + hd, lead=2, tail=3)
    cache = s.device()
    for mask in MASKS:
        s.check(cache, **mask_of(mask, nq, len(lens)))
        assert in_segments(s, cache, rows_of)
    assert int(s.status) == 0


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[1], SHAPES[6], SHAPES[9], SHAPES[11]], ids=lambda s: f"{len(s[0])}x{s[0][0][0]}-{s[3]}-{s[5]}")
@pytest.mark.parametrize("tree", ["star", "chain"])
def test_segments_of_evicted_caches(B, shape, tree):
    """The older rows in no order, other positions in every kv head."""
    lens, nq, nkv, hd, ps, dtype, rows_of = shape
    lens = [(n, max(n, length)) for n, length in lens]
    s = Trees(B, lens, nq, nkv, hd, ps, dtype, seed=3, kept=True, shape=tree)
    cache = s.device()
    for m in (dict(), dict(window=700), dict(softcap=10.0, prefix=60)):
        s.check(cache, **mask_of(m, nq, len(lens)))
        assert in_segments(s, cache, rows_of)
    assert int(s.status) == 0


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[1], SHAPES[2], SHAPES[6], SHAPES[9], SHAPES[11]], ids=lambda s: f"{len(s[0])}x{s[0][0][0]}-{s[3]}-{s[5]}")
@pytest.mark.parametrize("fill", [math.inf, math.nan, 1e30])
def test_segments_with_rows_that_are_not_finite(B, shape, fill):
    """V, or K and V, of rows that no query sees, of rows that all see, and of a branch that some do: those that do not see them
    are as the oracle has them, the others are not finite, as its are."""
    lens, nq, nkv, hd, ps, dtype, rows_of = shape
    for what in ("v", "kv"):
        s = Trees(B, lens, nq, nkv, hd, ps, dtype, seed=7)
        for i, (n, length) in enumerate(lens):
            if n == 0 or length - n < 200:
                continue
            rows = [3, 70, length - n - 150]             # behind a window of 100
            if i % 3 == 1:
                rows.append(length - 1)                  # the tree's last row: seen by itself alone
            elif i % 3 == 2:
                rows.append(length - n - 2)              # seen by all
            for r in rows:
                page, j = int(s.table[i, r // ps]), r % ps
                s.v[page, :, j] = fill
                if what == "kv":
                    s.k[page, :, j] = math.nan
        cache = s.device()
        with np.errstate(all="ignore"):
            s.check(cache, window=100)
        assert in_segments(s, cache, rows_of) and int(s.status) == 0


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[1], SHAPES[6], SHAPES[9], SHAPES[11]], ids=lambda s: f"{len(s[0])}x{s[0][0][0]}-{s[3]}-{s[5]}")
def test_segments_report_bad_pages_and_lengths(B, shape):
    """Rows of pages outside the pool are not there; lengths that the table cannot have are cut."""
    lens, nq, nkv, hd, ps, dtype, rows_of = shape
    s = Trees(B, lens, nq, nkv, hd, ps, dtype, seed=8)
    for i, (n, length) in enumerate(lens):
        if i % 2 == 0 and length > 600:
            s.table[i, [0, 512 // ps]] = torch.tensor([1 << 20, -3], dtype=torch.int32)
    cache = s.device()
    s.check(cache)
    assert in_segments(s, cache, rows_of) and int(s.status) == B.PAGED_BAD_PAGE
    s = Trees(B, lens, nq, nkv, hd, ps, dtype, seed=8)
    s.length[0] = -5
    if len(lens) > 1:
        s.length[1] = max(0, lens[1][0] - 1)             # fewer rows than new ones
    cache = s.device()
    out, lse = s.call(cache)
    assert int(s.status) == B.PAGED_BAD_ROWS
    a, b = int(s.start[0]), int(s.start[1])
    assert (out[a:b] == 0).all() and torch.isneginf(lse[a:b]).all()


def test_two_rounds_of_segments(B):
    """More query tiles than CTAs of a head at once."""
    lens = batch([150, 64, 90, 1, 130], [1500, 900, 2000, 300], 24)
    s = Trees(B, lens, 16, 4, 64, 64, seed=2, lead=1)
    cache = s.device()
    for m in (dict(), dict(window=400)):
        first = s.check(cache, **m)
        assert in_segments(s, cache, 256)
        again = s.call(cache, **m)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert int(s.status) == 0


@pytest.mark.parametrize("starts", [[0, 9, 4, 12], [-3, 40, 50, 60], [5, 5, 5, 5], [2, 3, 3, 9]])
@pytest.mark.parametrize("dtype,hd", [("bf16", 256), ("f32", 64)])
def test_segments_of_row_ranges_that_cannot_be(B, starts, dtype, hd):
    """Ranges are cut to the rows; rows in one range alone are that sequence's, rows in none are not written."""
    s = Trees(B, [(4, 2000), (4, 300), (4, 1500)], 4, 2, hd, 16, dtype, seed=4)
    s.start = torch.tensor(starts, dtype=torch.int32)
    cache = s.device()
    out, lse = s.call(cache)
    assert in_segments(s, cache, 16)
    of = [[i for i, (a, b) in enumerate(zip(starts, starts[1:])) if max(a, 0) <= r < min(b, 12)] for r in range(12)]
    free = [r for r in range(12) if not of[r]]
    assert (out[free] == 77).all() and (lse[free] == 77).all()
    for i, (a, b) in enumerate(zip(starts, starts[1:])):
        a, b = max(a, 0), min(b, 12)
        if b <= a or any(len(of[r]) > 1 for r in range(a, b)):
            continue
        o = s.oracle()
        one = {**o, "table": o["table"][i:i + 1], "length": o["length"][i:i + 1]}
        want, want_lse, mag = T.attention(one, host(s.q), s.q_pos.numpy(), np.array([a, b]), s.end.numpy(), s.scale)
        held, s.start = s.start, torch.tensor([a, b], dtype=torch.int32)
        full, full_lse = torch.full_like(out, 77.0), torch.full_like(lse, 77.0)
        full[a:b], full_lse[a:b] = out[a:b], lse[a:b]
        s.compare(host(full), host(full_lse), want, want_lse, mag, 0.0, None)
        s.start = held


@pytest.mark.parametrize("shape", [SHAPES[1], SHAPES[6], SHAPES[11]], ids=lambda s: f"{len(s[0])}x{s[0][0][0]}-{s[3]}-{s[5]}")
def test_segments_of_a_captured_call_follow_the_lengths(B, shape):
    """A graph replayed after lengths, rows and ends have changed: each CTA finds its segment from them."""
    lens, nq, nkv, hd, ps, dtype, rows_of = shape
    s = Trees(B, lens, nq, nkv, hd, ps, dtype, seed=5)
    other = Trees(B, [(n, max(n, length // 3)) for n, length in lens], nq, nkv, hd, ps, dtype, seed=6, spare=s.table.shape[1] - max(1, max(-(-max(n, x // 3) // ps) for n, x in lens)))
    cache = s.device()
    out, lse = (torch.full((s.rows, nq, *x), 77.0, dtype=t, device="cuda") for x, t in (((hd,), s.dt), ((), torch.float32)))
    args = [x.cuda() for x in (s.q, s.q_pos, s.start, s.end)]
    cache.tree_attention(*args, out, lse=lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.tree_attention(*args, out, lse=lse)
    for now in (s, other, s):
        pages = min(len(now.k), len(s.k))
        for held, x in zip((cache.k, cache.v, cache.pos), (now.k, now.v, now.pos)):
            held[:pages].copy_(x[:pages])
        table = now.table.clone()
        table[table >= pages] = pages                    # (unused entries)
        cache.table.copy_(table)
        cache.length.copy_(now.length)
        for held, x in zip(args, (now.q, now.q_pos, now.start, now.end)):
            held.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        opts = T.attention(now.oracle(), host(now.q), now.q_pos.numpy(), now.start.numpy(), now.end.numpy(), now.scale)
        now.compare(host(out), host(lse), *opts, 0.0, None)
    assert in_segments(s, cache, rows_of)


def test_segments_on_two_streams_at_once(B):
    """Calls of their own workspaces, and one held by the caller."""
    sets = [Trees(B, batch([64, 40, 20], [1900, 1200, 700], 18), 16, 4, 128, 32, seed=60 + i) for i in range(2)]
    caches = [s.device() for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    args = [[x.cuda() for x in (s.q, s.q_pos, s.start, s.end)] for s in sets]
    outs = [[torch.zeros(s.rows, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(12)] for s in sets]
    first = [s.check(c)[0] for s, c in zip(sets, caches)]
    assert all(in_segments(s, c, 256) for s, c in zip(sets, caches))
    mine = [torch.full((c._tree_bytes[1],), 255, dtype=torch.uint8, device="cuda") for c in caches]      # NaN in all of it
    torch.cuda.synchronize()
    for i in range(12):
        for c, st, a, o, w in zip(caches, streams, args, outs, mine):
            c.tree_attention(*a, o[i], workspace=w if i % 2 else None, stream=st)
    torch.cuda.synchronize()
    for o, x in zip(outs, first):
        assert all(torch.equal(y, x) for y in o)
