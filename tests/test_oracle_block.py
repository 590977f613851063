"""Pins of the oracle of norms, product and balance: against formulas written
another way, values known by hand, and differences for the gradient."""

import math

import numpy as np
import pytest
import torch

from oracle import block as B


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def test_norms_against_torch():
    g = rng(1)
    x, w, b = g.normal(size=(5, 40)), g.normal(size=40), g.normal(size=40)
    t = [torch.from_numpy(v) for v in (x, w, b)]
    assert np.allclose(B.norm(x, w, b, "layer", 1e-5), torch.nn.functional.layer_norm(t[0], (40,), t[1], t[2], 1e-5))
    assert np.allclose(B.norm(x, w - 1, None, "rms", 1e-5, 1.0),
                       torch.nn.functional.rms_norm(t[0], (40,), t[1], 1e-5))


def test_block_norm_is_made_of_its_stages():
    g = rng(2)
    x, r, w = g.normal(size=(4, 24)), g.normal(size=(4, 24)), g.normal(size=24)
    gate = g.normal(size=(4, 1))
    part = (w, None, "rms", 1e-6)
    s, _, y, _ = B.block_norm(x, part, gate, True, r, 0.5, part)
    u = x / np.sqrt((x ** 2).mean(1, keepdims=True) + 1e-6) * w
    want = r + 0.5 / (1 + np.exp(-gate)) * u
    assert np.allclose(s, want)
    assert np.allclose(y, want / np.sqrt((want ** 2).mean(1, keepdims=True) + 1e-6) * w)


def test_activations_by_hand():
    z = np.array([-30.0, -1.0, 0.0, 1.0, 30.0])
    phi = [0.5 * (1 + math.erf(v / math.sqrt(2))) for v in z]
    assert np.allclose(B.activation(z, "gelu"), z * phi)
    assert np.allclose(B.activation(z, "silu"), z / (1 + np.exp(-z)))
    assert np.allclose(B.activation(z, "relu"), [0, 0, 0, 1, 30])
    t = torch.from_numpy(z)
    assert np.allclose(B.activation(z, "gelu_tanh"), torch.nn.functional.gelu(t, approximate="tanh"))


def test_linear_gated_rows():
    g = rng(3)
    x, w, b, r = g.normal(size=(3, 8)), g.normal(size=(10, 8)), g.normal(size=10), g.normal(size=(3, 5))
    out, _ = B.linear(x, w, b, "silu", True, 2.0, r)
    gate, up = x @ w[:5].T + b[:5], x @ w[5:].T + b[5:]
    assert np.allclose(out, r + 2.0 * gate / (1 + np.exp(-gate)) * up)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_balance_gradient_against_differences(sigmoid):
    """f is a constant to the gradient: sum over sequences of g * sum f P, by the
    logits."""
    g = rng(4 + sigmoid)
    T, E, k, S = 6, 5, 2, 2
    z = g.normal(size=(T, E))
    z[1, 3] = -np.inf
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)])
    ids[4] = -1                      # padding
    ids[0] = [2, 2]                  # the same expert twice
    up = np.array([0.7, 1.9])
    r = B.balance(z, ids, sigmoid, S, grad_loss=up)
    f = np.stack([E * r["counts"][s] / (k * max(1, r["tokens"][s])) for s in range(S)])

    def value(z):
        probs = B.balance(z, ids, sigmoid, S)["probs"]
        return (up[:, None] * f * probs).sum()

    h = 1e-6
    for t in range(T):
        for e in range(E):
            if z[t, e] == -np.inf:
                assert r["grad"][t, e] == 0
                continue
            a, b = z.copy(), z.copy()
            a[t, e] += h
            b[t, e] -= h
            assert abs((value(a) - value(b)) / (2 * h) - r["grad"][t, e]) < 1e-8


def test_balance_by_hand():
    """Even tokens and scores: every loss is 1, and no gradient."""
    z, ids = np.zeros((8, 4)), np.arange(8).reshape(8, 1) % 4
    for sigmoid in (False, True):
        r = B.balance(z, ids, sigmoid, 2)
        assert np.allclose(r["loss"], 1) and np.allclose(r["grad"], 0) and np.all(r["counts"] == 1)
    # All tokens to one expert whose scores are 1: E times that.
    z[:, 0] = 1000.0
    r = B.balance(z, np.zeros((8, 1), int), False, 1)
    assert np.allclose(r["loss"], 4) and r["counts"].tolist() == [[8, 0, 0, 0]]
    r = B.balance(z, np.full((8, 1), 7), False, 1)   # nothing but padding
    assert r["loss"][0] == 0 and r["tokens"][0] == 0 and not r["grad"].any() and not r["probs"].any()
