"""GPU parity of tree attention where a batch is cut into segments of keys, which join in
a workspace, against the fp64 oracle (oracle/tree_oracle.py). Every test makes sure that its calls are cut:
few query tiles over short tables are clusters, which need no workspace. The tolerances
are those of test_gpu_paged.py."""

import pytest
import torch

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
