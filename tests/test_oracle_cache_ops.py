"""Pins of the cache-maintenance oracle: trees against causal attention, masses against their
defining sums, kept sets against a full sort."""

import math

import numpy as np
import pytest
import torch

from oracle import cache_ops as C


def _paged(rng, length, ps, h, d):
    pages = -(-length // ps)
    table = rng.permutation(pages + 2)[:pages]
    return (rng.standard_normal((pages + 2, ps, h, d)), rng.standard_normal((pages + 2, ps, h, d)),
            table)


def _flat(cache, table, length, h):
    return np.concatenate([cache[p, :, h] for p in table])[:length]


@pytest.mark.parametrize("window", [-1, 3, 7])
def test_a_chain_is_causal_attention(window):
    rng = np.random.default_rng(3)
    L, n, d = 11, 6, 8
    k, v, table = _paged(rng, L + n, 4, 1, d)
    q = rng.standard_normal((1, n, 2, d))
    out, _ = C.tree_attend(q, k, v, [table], [L], [list(range(-1, n - 1))], 0.3, window)
    kk, vv = (torch.from_numpy(_flat(c, table, L + n, 0)) for c in (k, v))
    i, j = torch.arange(n)[:, None] + L, torch.arange(L + n)[None]
    see = (j <= i) & ((j > i - window) if window > 0 else (j >= 0))
    for hq in range(2):
        ref = torch.nn.functional.scaled_dot_product_attention(
            torch.from_numpy(q[0, :, hq])[None], kk[None], vv[None], attn_mask=see, scale=0.3)[0]
        assert np.allclose(out[0, :, hq], ref.numpy(), atol=1e-12)


def test_siblings_do_not_see_each_other_and_padding_is_zero():
    assert C.ancestors([-1, 0, 0, 1, -2, 4, 9, -1]) == [[0], [0, 1], [0, 2], [0, 1, 3], [], [], [], [7]]
    assert C.tree_positions([-1, 0, 0], 2, 5) == [0, 1, 2, 3, 4, 5, 7]
    assert C.tree_positions([-1, 0, 0], 2, 5, window=2) == [5, 7]
    assert C.tree_positions([-1, 0, 0], 2, 5, idx=[1, 4]) == [1, 4, 5, 7]
    assert C.tree_positions([-2], 0, 5) == []


def test_mass_of_a_step_sums_to_the_group_size():
    rng = np.random.default_rng(5)
    k, v, table = _paged(rng, 13, 4, 2, 8)
    q = rng.standard_normal((1, 6, 8))
    out, m = C.mass_step(q, k, v, [table], [13], 0.4, np.zeros((1, 2, 16)))
    assert np.allclose(m.sum(2), 3.0) and np.all(m[:, :, 13:] == 0)
    _, m2 = C.mass_step(q, k, v, [table], [13], 0.4, m, window=5)
    assert np.allclose((m2 - m).sum(2), 3.0) and np.all((m2 - m)[:, :, :8] == 0)
    _, m3 = C.mass_step(q, k, v, [table], [13], 0.4, np.zeros((1, 2, 16)),
                        idx=np.tile(np.arange(13), (1, 2, 1)), count=np.full((1, 2), 13))
    assert np.allclose(m3, m)
    # an unusable page holds no weight
    bad = table.copy()
    bad[1] = 99
    _, m4 = C.mass_step(q, k, v, [bad], [13], 0.4, np.zeros((1, 2, 16)))
    assert np.all(m4[:, :, 4:8] == 0) and np.allclose(m4.sum(2), 3.0)


def test_kept_positions():
    m = [5.0, 1.0, 3.0, 3.0, 0.0, math.nan, 3.0, 9.0]
    assert C.kept_positions(m, 8, 4, 1).tolist() == [0, 2, 5, 7]
    assert C.kept_positions(m, 8, 5, 1).tolist() == [0, 2, 3, 5, 7]
    assert C.kept_positions(m, 8, 3, 3).tolist() == [5, 6, 7]
    assert C.kept_positions(m, 8, 2, 0).tolist() == [5, 7]
    assert C.kept_positions(m, 3, 4, 1).tolist() == [0, 1, 2]
    assert C.kept_positions(m, 0, 4, 1).tolist() == []
