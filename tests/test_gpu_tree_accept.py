"""GPU parity of the walk through trees where rows had nothing to draw, against the oracle (oracle/tree_oracle.py): exact."""

import math

import numpy as np
import pytest
import torch

from oracle import tree_oracle as T
from test_gpu_tree import random_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from block_speculative_decoding_dflash_gb300 import build
    build.build()
    from block_speculative_decoding_dflash_gb300 import binding
    return binding


def accept(B, trees, draft, sampled, width):
    """tree_accept against the oracle's walks; length_out against the rows that stay."""
    starts = np.cumsum([0] + [len(e) for e in trees])
    dev = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()  # noqa: E731
    n = len(trees)
    tokens, path, count, out = (torch.full(shape, 99, dtype=torch.int32, device="cuda") for shape in ((n, width), (n, width), (n,), (n,)))
    B.tree_accept(dev(np.concatenate([np.asarray(e, dtype=np.int32) for e in trees])), dev(starts), dev(draft), dev(sampled), tokens, path, count,
                  length=dev([1000 + len(e) for e in trees]), length_out=out)
    torch.cuda.synchronize()
    for s, e in enumerate(trees):
        a, b = starts[s], starts[s + 1]
        p, t = T.accept(e, draft[a:b], sampled[a:b], width)
        assert path[s].tolist() == p + [-1] * (width - len(p)) and tokens[s].tolist() == t + [-1] * (width - len(t))
        assert int(count[s]) == len(p) and int(out[s]) == 1000 + len(p)
    return count


@pytest.mark.parametrize("width", [1, 4, 40])
@pytest.mark.parametrize("none", [-1, -(1 << 31)])
def test_rows_with_nothing_to_draw_end_the_walk(B, width, none):
    """In every row, in some, in row 0 alone; drafted tokens that are negative too."""
    rng = np.random.default_rng(width)
    trees = [random_tree(rng, n, 0.7) for n in (1, 16, 64, 30, 300, 7)]
    rows = sum(len(e) for e in trees)
    for share in (1.0, 0.3, 0.05):
        draft = rng.integers(0, 5, rows).astype(np.int32)
        sampled = rng.integers(0, 5, rows).astype(np.int32)
        sampled[rng.random(rows) < share] = none
        draft[rng.random(rows) < 0.3] = none
        accept(B, trees, draft, sampled, width)
    draft, sampled = np.zeros(rows, dtype=np.int32), np.zeros(rows, dtype=np.int32)
    sampled[np.cumsum([0] + [len(e) for e in trees])[:-1]] = none
    assert (accept(B, trees, draft, sampled, width) == 0).all()


def test_sampled_rows_without_logits(B):
    """From logits to the path: a row whose logits are all masked is not on it."""
    end = [5] * 5                                        # a chain
    logits = torch.full((5, 40), -2.0, device="cuda")
    draft = [0, 7, 8, 9, 10]
    for i, t in enumerate([7, 8, 9, 10, 11]):
        logits[i, t] = 30.0
    logits[3] = -math.inf
    sampled = torch.zeros(5, dtype=torch.int32, device="cuda")
    B.sample(logits, torch.full((5,), 0.5, device="cuda"), sampled)
    assert sampled.tolist() == [7, 8, 9, -1, 11]
    count = accept(B, [end], np.array(draft, dtype=np.int32), sampled.cpu().numpy(), 8)
    assert count.tolist() == [3]
