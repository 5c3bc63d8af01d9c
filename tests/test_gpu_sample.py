"""GPU parity of sampling where the kernel's own arithmetic could part ways with itself, against the fp64 oracle
(oracle/tree_oracle.py); the tolerances are those of test_gpu_tree.py."""

import numpy as np
import pytest
import torch

from test_gpu_tree import check_draws

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from block_speculative_decoding_dflash_gb300 import build
    build.build()
    from block_speculative_decoding_dflash_gb300 import binding
    return binding


def border_distances(temperature):
    """fp32 distances from the largest logit whose bin (of a factor of 2^(1/8), found by rounding the distance in steps of
    2^-10 to a factor of 2) depends on whether the product is rounded before the sum."""
    chi = np.float32(1.44269504088896340736 / float(np.float32(temperature)))
    out = []
    for b in range(4, 320):
        d = np.float32((128 * b - 0.5) / 1024 / float(chi))
        for _ in range(4):
            d = np.nextafter(d, np.float32(0))
        for _ in range(9):
            exact = np.longdouble(d) * np.longdouble(chi)
            apart = np.float32(np.float32(exact) + np.float32(12288))
            if apart != np.float32(exact + np.longdouble(12288)):
                out.append(float(d))
            d = np.nextafter(d, np.float32(1e9))
    return out


@pytest.mark.parametrize("vocab", [700, 4100, 65537, 400001])
@pytest.mark.parametrize("share", [0.0, 0.5])
def test_logits_on_the_borders_of_bins(B, vocab, share):
    """fp32 rows whose logits lie where two roundings of a distance give two bins, all of them or half: a cut by weight
    falls within such bins."""
    r = np.random.default_rng(vocab)
    temperature = np.array([0.6, 0.7341, 0.8, 0.93, 1.0, 1.1, 1.37, 2.5] * 2, dtype=np.float32)
    rows = len(temperature)
    x = np.zeros((rows, vocab), dtype=np.float32)
    for i, t in enumerate(temperature):
        d = np.array(border_distances(t), dtype=np.float32)
        assert len(d) >= 20
        # as many of each as make its bin's weight a part of the row's that cuts fall into
        w = np.exp(-d.astype(np.float64) / float(t))
        chosen = d[r.choice(len(d), vocab, p=w ** -0.5 / (w ** -0.5).sum() if i % 2 else None)]
        plain = r.random(vocab) < share
        x[i] = np.where(plain, r.standard_normal(vocab).astype(np.float32) * 3 - 10, -chosen)
        x[i, vocab // 3] = 0.0
        x[i] = np.minimum(x[i], 0.0)
    logits = torch.from_numpy(x).cuda()
    u = r.random(rows, dtype=np.float32)
    for p in (r.random(rows, dtype=np.float32), np.linspace(0.1, 0.999, rows, dtype=np.float32)):
        check_draws(B, logits, u, near_allowed=1, temperature=temperature, top_p=p)
        check_draws(B, logits, u, near_allowed=1, temperature=temperature, top_p=p, top_k=r.integers(257, vocab + 9, rows))
        check_draws(B, logits, u, near_allowed=1, temperature=temperature, top_p=p, min_p=r.random(rows, dtype=np.float32) * np.float32(0.01))
    check_draws(B, logits, u, near_allowed=1, temperature=temperature)
    check_draws(B, logits, u, near_allowed=1, temperature=temperature, top_k=r.integers(1, 257, rows))
