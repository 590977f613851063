"""CPU oracle of the operators around a layer: norms between blocks, the dense
16-bit product with its epilogue, and the router's balance.

TEST INFRASTRUCTURE ONLY, as ``oracle.moe``.  Everything is fp64 NumPy written
from the definitions; it shares no code with the HIP path.

The ``*_bound`` results say how far a kernel that rounds to fp32 after every
operation may be from the fp64 value:

  * a sum of n terms in fp32 is off by at most n 2^-23 (sum of magnitudes);
    one whose terms are added in a tree of depth d by d 2^-23 of it;
  * exp, erfc, division and square root in fp32 are within 4 units of 2^-24,
    beside what an argument that is off does to them (e^u turns an absolute
    error of u into a relative one);
  * a rounding to the output's type by half a step of it at most.
"""

from __future__ import annotations

import math

import numpy as np

U32 = 2.0 ** -24
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
# Half a step below the smallest normal number.
TINY_STEP = {"float32": 2.0 ** -150, "bfloat16": 2.0 ** -134, "float16": 2.0 ** -25}

_erfc = np.frompyfunc(math.erfc, 1, 1)


def rounding(v, dtype):
    return HALF[dtype] * np.abs(v) + TINY_STEP[dtype]


# -- norms ---------------------------------------------------------------------

# Depth of the sums over a row: up to 32 values a thread, 6 steps inside a wave, 16
# waves, and the roundings of a mean, a difference, a square and a root beside them.
ROW_DEPTH = 32 + 6 + 16 + 10


def norm(v, weight, bias, kind, eps, offset=0.0):
    d = v - v.mean(axis=1, keepdims=True) if kind == "layer" else v
    y = d / np.sqrt((d * d).mean(axis=1, keepdims=True) + eps) * (weight + offset)
    return y if bias is None else y + bias


def norm_bound(v, err, weight, bias, kind, eps, offset=0.0):
    """Of norm(v) where v is off by up to err."""
    mean = v.mean(axis=1, keepdims=True) if kind == "layer" else 0.0
    d = v - mean
    depth = ROW_DEPTH * 2.0 ** -23
    if kind == "layer":
        err = err + err.mean(axis=1, keepdims=True) + depth * np.abs(v).mean(axis=1, keepdims=True) \
            + U32 * np.abs(v)
    q = (d * d).mean(axis=1, keepdims=True) + eps
    # Relative error of 1 / sqrt(q): half that of q.
    rel = (np.abs(d) * err + err * err).mean(axis=1, keepdims=True) / q + depth
    w = np.abs(weight + offset)
    y = np.abs(d) / np.sqrt(q) * w
    bound = err / np.sqrt(q) * w * (1 + rel) + y * (rel + 8 * U32)
    return bound if bias is None else bound + U32 * (y + np.abs(bias) + bound) * 2


def block_norm(x, post=None, gate=None, gate_sigmoid=False, residual=None, scale=1.0, pre=None):
    """(sum, y) and how far each may be off before its own rounding.  post, pre: the
    arguments of norm behind v, as a tuple."""
    s, err = x, np.zeros_like(x)
    if post is not None:
        s, err = norm(x, *post), norm_bound(x, err, *post)
    if gate is not None:
        g = 1.0 / (1.0 + np.exp(-gate)) if gate_sigmoid else gate
        # e^-g: its argument is exact, so 4 units, and one each of sum and quotient.
        err = (err + 8 * U32 * np.abs(s)) * np.abs(g)
        s = s * g
    err = np.abs(scale) * (err + 2 * U32 * np.abs(s))
    s = s * scale
    if residual is not None:
        s = residual + s
    err = err + 2 * U32 * np.abs(s)
    if pre is None:
        return s, err, None, None
    return s, err, norm(s, *pre), norm_bound(s, err, *pre)


# -- product -------------------------------------------------------------------

def activation(z, act):
    if act == "relu":
        return np.maximum(z, 0.0)
    if act == "silu":
        return z / (1.0 + np.exp(-z))
    if act == "gelu":
        return 0.5 * z * _erfc(-z / math.sqrt(2.0)).astype(np.float64)
    if act == "gelu_tanh":
        # (1 + tanh a) / 2 = 1 / (1 + e^-2a), where nothing cancels.
        with np.errstate(over="ignore"):
            return z / (1.0 + np.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def activation_bound(z, err, act):
    """Slopes are below 1.13; an exponent of magnitude u is off by a few units of u."""
    if act in ("none", "relu"):
        return err
    u = {"silu": np.abs(z), "gelu": z * z / 2, "gelu_tanh": np.abs(1.6 * (z + 0.045 * z ** 3))}[act]
    with np.errstate(invalid="ignore"):
        h = np.abs(activation(z, act))
        return 1.13 * err + (8 + 4 * u) * U32 * np.where(h > 0, h, 0) + 2.0 ** -126


def linear(x, w, bias=None, act="none", gated=False, scale=1.0, residual=None):
    """(out, how far it may be off before its rounding)."""
    with np.errstate(over="ignore"):
        z, size = x @ w.T, np.abs(x) @ np.abs(w).T
        err = x.shape[1] * 2.0 ** -23 * size
        if bias is not None:
            z = z + bias
            err = err + U32 * (np.abs(z) + err)
        N = w.shape[0] // 2 if gated else w.shape[0]
        h, bound = activation(z[:, :N], act), activation_bound(z[:, :N], err[:, :N], act)
        if gated:
            up, eu = z[:, N:], err[:, N:]
            bound = bound * (np.abs(up) + eu) + np.abs(h) * eu + U32 * np.abs(h * up)
            h = h * up
        h, bound = scale * h, np.abs(scale) * (bound + 2 * U32 * np.abs(h))
        if residual is not None:
            h = residual + h
            bound = bound + U32 * (np.abs(h) + bound)
    return h, bound


# -- balance -------------------------------------------------------------------

def balance(logits, ids, sigmoid, n_seq=1, bias=None, grad_loss=None):
    """counts, tokens, probs, loss, grad, and how far the last three may be off."""
    T, E = logits.shape
    k = ids.shape[1]
    L = T // n_seq
    with np.errstate(invalid="ignore"):
        there = logits > -np.inf
        if bias is not None:
            there = there & (bias > -np.inf)
    z = np.minimum(np.where(there, logits, 0.0), np.finfo(np.float32).max)
    if sigmoid:
        with np.errstate(over="ignore"):
            e, slope = 1.0 / (1.0 + np.exp(-z)), 1.0 / (1.0 + np.exp(z))
        u = np.zeros_like(z)     # (the argument of the exponential is exact)
    else:
        top = np.where(there, z, -np.inf).max(axis=1, keepdims=True)
        u = np.where(there, z - np.where(there.any(axis=1, keepdims=True), top, 0.0), 0.0)
        e, slope = np.exp(u), np.ones_like(z)
    e = np.where(there, e, 0.0)
    p = e / (e.sum(axis=1, keepdims=True) + 1e-20)
    # The exponential and its argument, a sum of up to 16 values a lane and 6 steps
    # between lanes, the quotient.
    rel = (np.abs(u) + 8) * U32
    rel = rel + (rel * p).sum(axis=1, keepdims=True) + 24 * 2.0 ** -23
    found = (ids >= 0) & (ids < E)
    real = found.any(axis=1)
    counts, tokens = np.zeros((n_seq, E), np.int64), np.zeros(n_seq, np.int64)
    probs, loss, grad = np.zeros((n_seq, E)), np.zeros(n_seq), np.zeros((T, E))
    e_probs, e_loss, e_grad = np.zeros((n_seq, E)), np.zeros(n_seq), np.zeros((T, E))
    for s in range(n_seq):
        rows = np.arange(s * L, (s + 1) * L)[real[s * L:(s + 1) * L]]
        n = tokens[s] = len(rows)
        if n == 0:
            continue
        chosen = ids[rows][found[rows]]
        counts[s] = np.bincount(chosen, minlength=E)
        f = E * counts[s] / (k * n)
        probs[s] = p[rows].sum(axis=0) / n
        loss[s] = (f * probs[s]).sum()
        # fp32 sums of a wave's rows (at most a 1024th of the call's, an eighth of
        # its workgroup's 32), and of 8 waves.
        depth = (max(32, -(-T // 1024)) + 8) * 2.0 ** -23
        e_probs[s] = (rel[rows] * p[rows]).sum(axis=0) / n + depth * probs[s]
        e_loss[s] = (f * e_probs[s]).sum() + U32 * loss[s]
        g = (1.0 if grad_loss is None else grad_loss[s]) / n
        mean = p[rows] @ f
        less = f - mean[:, None]
        # of f - 1 and its mean: a rounding of each, and the sum's
        big = np.abs(f - 1) + 2 * U32 * f
        e_less = 3 * U32 * f + 2 * U32 * np.abs(f - 1) + (
            (p[rows] * (big * rel[rows] + 3 * U32 * f)).sum(axis=1) + 24 * 2.0 ** -23 * (p[rows] @ big))[:, None]
        if sigmoid:
            # f - sum f p is (f - 1) - (sum (f - 1) p) + (1 - sum p), and the last is 1e-20 over
            # the scores' sum: a constant, a quotient, a product and an addition to the mean.
            short = 1e-20 / (e[rows].sum(axis=1, keepdims=True) + 1e-20)
            e_less = e_less + short * (rel[rows].max(axis=1, keepdims=True) + 4 * U32)
        t = g * p[rows] * slope[rows]
        grad[rows] = t * less
        # Scores, slopes and products below 2^-126 are off by up to 2^-150 each instead;
        # four of those, times f < 2^10 and a g below 2^4, stay below 2^-126.
        e_grad[rows] = np.abs(t) * (e_less + (rel[rows] + 16 * U32) * np.abs(less)) + 2.0 ** -126
    return dict(counts=counts, tokens=tokens, probs=probs, loss=loss, grad=grad, e_probs=e_probs, e_loss=e_loss,
                e_grad=e_grad)
