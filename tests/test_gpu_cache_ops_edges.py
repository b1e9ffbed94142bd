"""Cache operators at the edges of their range: precision, odd states of the layer, bad pages, sizes
that take the rarer branches of the kernels. Float64 references as in test_gpu_cache_ops.py.

Tolerances, fixed before the first run. With A = sum_t p_t |v_t| from the oracle and T visible
positions: weights as two bf16 parts are off by at most 2^-14 of themselves, fp32 scores by
X / 2 = d 2^-23 scale max_t sum_i |q_i k_ti| + 2^-20 as a factor on each weight and on their sum, the
sums over T positions (two products each, and the sum of weights) by 3 T 2^-23 A, the bf16 output by
half a step (2^-8 of its value).
"""

import math

import numpy as np
import pytest
import torch

from oracle import cache_ops as C
from test_gpu_cache_ops import (NAN, Paged, _built, _clean_flags, cuda, f64, jssa,  # noqa: F401
                                random_tree)

pytestmark = pytest.mark.gpu


def weight_slack(q, k, scale, positions):
    """Factor on A from scores, split weights and sums; ``q`` [..., d], ``k`` [..., d], NaN left out."""
    d = q.shape[-1]
    k = np.abs(np.where(np.isfinite(k), k, 0)).reshape(-1, d)
    top = float((np.abs(q).reshape(-1, d) @ k.T).max())
    return 2.0 ** -14 + 2 * (d * 2.0 ** -23 * abs(scale) * top + 2.0 ** -20) + 3 * positions * 2.0 ** -23


def check_close(got, ref, mag, slack):
    assert np.isfinite(got).all()
    tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * slack * mag
    assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) - tol))


# ------------------------------------------------------------------------------------------------
# tree attention
# ------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("n,g,d", [(7, 4, 128), (40, 4, 128), (9, 4, 256), (64, 2, 256)])
def test_tree_attend_weights_are_not_rounded_once(n, g, d):
    # the weights keep more than a bf16's digits, as in the decode kernels: outputs near zero show it
    J = jssa()
    c = Paged([230, 64], n, 1, d, seed=50 + n)
    q, kn, vn = c.normal(2, n, g, d), c.normal(2, n, 1, d), c.normal(2, n, 1, d)
    parents = [random_tree(c.rng, n, b) for b in range(2)]
    scale = 1 / math.sqrt(d)
    out = J.tree_attend(q.cuda(), c.k, c.v, c.bt, c.seq_lens, cuda(parents), kn.cuda(), vn.cuda())
    ref, mag = C.tree_attend(f64(q), f64(c.k), f64(c.v), c.table, c.lens, parents, scale)
    check_close(f64(out), ref, mag, weight_slack(f64(q), f64(c.k), scale, 230 + n))
    assert J.device_error() == 0


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n", [6, 64])
def test_tree_attend_visible_infinities(n, d):
    # an infinite value that every row sees reaches that element of every row, and no other
    J = jssa()
    c = Paged([200], n, 1, d, seed=60 + n)
    q, kn, vn = c.normal(1, n, 4, d), c.normal(1, n, 1, d), c.normal(1, n, 1, d)
    parents = cuda([random_tree(c.rng, n)])
    for t, e, x in ((3, 5, math.inf), (90, 7, -math.inf)):
        c.v[c.table[0, t // 16], t % 16, 0, e] = x
    out = J.tree_attend(q.cuda(), c.k, c.v, c.bt, c.seq_lens, parents, kn.cuda(), vn.cuda())[0].float()
    assert bool((out[..., 5] == math.inf).all()) and bool((out[..., 7] == -math.inf).all())
    out[..., 5] = out[..., 7] = 0.0
    assert bool(torch.isfinite(out).all())
