"""Pins of the fp64 reference of the decay rule, the draft trees and the 8-bit rows."""
import numpy as np
import pytest
import torch

import oracle
from oracle import decay as ref


def rand(rng, *shape):
    return rng.standard_normal(shape)


def test_gradients_match_finite_differences():
    rng = np.random.default_rng(1)
    B, T, Hqk, Hv, d = 2, 5, 2, 4, 3
    x = {"q": rand(rng, B, T, Hqk, d), "k": rand(rng, B, T, Hqk, d), "v": rand(rng, B, T, Hv, d),
         "S0": rand(rng, B, Hv, d, d)}
    lam = np.array([0.3, 0.9, 1.0, 0.6])
    dO, dS = rand(rng, B, T, Hv, d), rand(rng, B, Hv, d, d)

    def loss():
        o, S = ref.decay_forward(x["q"], x["k"], x["v"], lam, x["S0"])
        return (o * dO).sum() + (S * dS).sum()

    grads = dict(zip(("q", "k", "v", "S0"), ref.decay_backward(x["q"], x["k"], x["v"], lam, x["S0"], dO, dS)))
    for name, g in grads.items():
        a = x[name]
        for i in range(0, a.size, 3):
            at = np.unravel_index(i, a.shape)
            keep = a[at]
            a[at] = keep + 1e-6
            up = loss()
            a[at] = keep - 1e-6
            down = loss()
            a[at] = keep
            assert abs((up - down) / 2e-6 - g[at]) < 1e-7, (name, at)


def test_no_decay_is_a_sum_of_outer_products():
    rng = np.random.default_rng(2)
    q, k, v = rand(rng, 1, 6, 1, 4), rand(rng, 1, 6, 1, 4), rand(rng, 1, 6, 1, 4)
    o, S = ref.decay_forward(q, k, v, np.array([1.0]))
    assert np.allclose(S[0, 0], k[0, :, 0].T @ v[0, :, 0], atol=1e-13)
    causal = np.tril(q[0, :, 0] @ k[0, :, 0].T)
    assert np.allclose(o[0, :, 0], causal @ v[0, :, 0], atol=1e-13)


def test_a_chain_of_drafts_is_the_recurrence():
    rng = np.random.default_rng(3)
    B, n, Hqk, Hv, d = 2, 6, 1, 3, 128
    q, k, v = rand(rng, B, n, Hqk, d) * 0.1, rand(rng, B, n, Hqk, d) * 0.1, rand(rng, B, n, Hv, d)
    alpha, beta = rng.uniform(0.5, 1, (B, n, Hv)), rng.uniform(0, 1, (B, n, Hv))
    S = rand(rng, B, Hv, d, d)
    parents = np.tile(np.arange(-1, n - 1), (B, 1))
    o, states, alive = ref.tree(q, k, v, parents, S, alpha=alpha, beta=beta)
    ro, rS = oracle.forward(*(torch.from_numpy(x) for x in (q, k, v, alpha, beta, S)))
    assert alive.all()
    assert np.allclose(o, ro, atol=1e-6) and np.allclose(states[:, -1], rS, atol=1e-6)   # the C oracle's inputs are fp32
    lam = np.array([0.2, 0.9, 1.0])
    o, states, _ = ref.tree(q, k, v, parents, S, decay=lam)
    ro, rS = ref.decay_forward(q, k, v, lam, S)
    assert np.allclose(o, ro, atol=1e-12) and np.allclose(states[:, -1], rS, atol=1e-12)


def test_branches_do_not_see_each_other():
    rng = np.random.default_rng(4)
    q, k, v = rand(rng, 1, 4, 1, 5), rand(rng, 1, 4, 1, 5), rand(rng, 1, 4, 1, 5)
    S = rand(rng, 1, 1, 5, 5)
    lam = np.array([0.7])
    o, _, _ = ref.tree(q, k, v, np.array([[-1, 0, 0, 1]]), S, decay=lam)
    for path in ([0], [0, 1], [0, 2], [0, 1, 3]):
        ro, _ = ref.decay_forward(q[:, path], k[:, path], v[:, path], lam, S)
        assert np.allclose(o[0, path[-1]], ro[0, -1], atol=1e-12)


def test_padding_reaches_down_the_tree():
    assert ref.tree_alive([[-1, 0, -2, 2, 3, 1, 7, 0, 9]]).tolist() == [
        [True, True, False, False, False, True, False, True, False]]


def test_majorants_bound_the_values():
    rng = np.random.default_rng(5)
    q, k, v = rand(rng, 1, 9, 1, 4), rand(rng, 1, 9, 1, 4), rand(rng, 1, 9, 2, 4)
    lam, S = np.array([0.5, 0.99]), rand(rng, 1, 2, 4, 4)
    for a, b in zip(ref.decay_forward(q, k, v, lam, S), ref.decay_forward_majorant(q, k, v, lam, S)):
        assert (np.abs(a) <= b + 1e-12).all()
    p = np.array([[-1, 0, 1, 0, 3, 2, 5, 4, 4]])
    alpha, beta = rng.uniform(0.5, 1, (1, 9, 2)), rng.uniform(0, 1, (1, 9, 2))
    for a, b in zip(ref.tree(q, k, v, p, S, alpha=alpha, beta=beta)[:2],
                    ref.tree(q, k, v, p, S, alpha=alpha, beta=beta, majorant=True)[:2]):
        assert (np.abs(a) <= b + 1e-12).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_rows_of_the_state_cache(fmt):
    rng = np.random.default_rng(6)
    x = (rng.standard_normal((40, 128)) * np.exp(rng.standard_normal((40, 1)) * 5)).astype(np.float32)
    x[3] = 0
    x[4, 7] = np.inf
    x[5, 0] = np.nan
    x[6] *= np.float32(1e-33)
    c, s = ref.quantise_rows(x, fmt)
    back = c * s[:, None]
    good = np.ones(40, bool)
    good[[3, 4, 5, 6]] = False
    step = s[good, None] * (0.5 if fmt == "int8" else np.maximum(np.abs(c[good]) * 2.0 ** -4, 2.0 ** -10))
    assert (np.abs(back[good] - x[good]) <= step * (1 + 1e-5)).all()
    assert s[3] == 0 and s[6] == 0 and (c[[3, 4, 5, 6]] == 0).all() and np.isnan(s[[4, 5]]).all()


def test_e4m3_rounding_is_torchs():
    y = np.concatenate([np.linspace(-448, 448, 9973), np.linspace(-0.02, 0.02, 4001)]).astype(np.float32)
    t = torch.from_numpy(y).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(ref.round_e4m3(y.astype(np.float64)), t.astype(np.float64))
