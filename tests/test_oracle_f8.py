"""Pins of the 8-bit oracle and of the router's oracle: the code table against
torch's float8 type, rounding by brute force over all neighbours, the router
against torch.topk where that is defined."""

import numpy as np
import pytest
import torch

from oracle import f8


def test_decode_agrees_with_torch_for_all_codes():
    codes = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    got = f8.decode(codes)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[~np.isnan(got)], ref[~np.isnan(ref)])
    assert np.nanmax(got) == f8.F8_MAX


def test_rounding_is_nearest_even_by_brute_force():
    rng = np.random.default_rng(0)
    table = np.unique(f8.decode(np.arange(256, dtype=np.uint8))[~np.isnan(f8.decode(np.arange(256, dtype=np.uint8)))])
    mids = (table[1:] + table[:-1]) / 2
    v = np.concatenate([rng.uniform(-448, 448, 4000), rng.uniform(-0.05, 0.05, 4000), table, mids,
                        np.nextafter(mids, 1e9), np.nextafter(mids, -1e9)])
    d = np.abs(v[:, None] - table[None, :])
    near = d == d.min(axis=1, keepdims=True)
    got = f8.round_e4m3(v)
    for i in range(v.size):
        best = table[near[i]]
        if best.size == 1:
            assert got[i] == best[0], v[i]
        else:  # a tie: the even fraction
            even = [b for b in best if f8.encode(np.array(b)) % 2 == 0]
            assert got[i] == even[0], v[i]


def test_encode_inverts_decode():
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F and c != 0x80], np.uint8)
    assert np.array_equal(f8.encode(f8.decode(codes)), codes)


def test_quantize_edges():
    x = np.zeros((4, 300))
    x[0, 0], x[0, 130], x[1, 299] = 448.0, 2.0 ** -101, 1.0
    x[2, 5], x[3, 5] = np.inf, np.nan
    v, s, _ = f8.quantize(x)
    assert v.shape == (4, 384) and s.shape == (4, 3)
    assert s[0, 0] == 1.0 and v[0, 0] == 448.0 and s[0, 1] == 0.0 and v[0, 130] == 0.0
    assert v[1, 299] == 448.0 and s[1, 2] == 1 / 448.0
    assert np.isnan(s[2, 0]) and np.isnan(s[3, 0]) and not np.isnan(v).any()


@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_agrees_with_topk_without_groups(sigmoid):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((50, 40))
    ids, w = f8.route(x, None, 6, sigmoid, 1, 1, False, 1.0)
    s = torch.from_numpy(x).sigmoid() if sigmoid else torch.from_numpy(x).softmax(1)
    rw, rid = s.topk(6, dim=1)
    assert np.array_equal(ids, rid.numpy())
    assert np.allclose(w, rw.numpy(), rtol=1e-12, atol=0)


def test_route_groups_bias_and_ties():
    x = np.zeros((1, 8))
    ids, w = f8.route(x, None, 3, True, 1, 1, True, 3.0)
    assert ids.tolist() == [[0, 1, 2]] and np.allclose(w, 1.0)
    bias = np.array([0.0, 9.0, 0, 0, 5.0, 5.0, 0, 0])   # group sums 9.x, 0.x, 10.x, 0.x
    ids, _ = f8.route(x, bias, 2, True, 4, 1, True, 1.0)
    assert ids.tolist() == [[4, 5]]
    ids, _ = f8.route(x, bias, 4, True, 4, 2, True, 1.0)
    assert ids.tolist() == [[1, 4, 5, 0]]
    x[0, 4:] = -np.inf
    ids, w = f8.route(x, bias, 4, True, 4, 2, True, 1.0)
    assert ids.tolist() == [[1, 0, 2, 3]]
    ids, w = f8.route(np.full((1, 4), np.nan), None, 2, False, 1, 1, True, 1.0)
    assert ids.tolist() == [[-1, -1]] and not w.any()


def test_moe_bounds_cover_an_fp32_computation():
    """The same layer in fp32 numpy stays within both bounds, and one that is 1 %
    off does not."""
    rng = np.random.default_rng(5)
    T, H, I, E, k = 6, 256, 128, 3, 2
    x = rng.standard_normal((T, H)).astype(np.float32).astype(np.float64)
    w13 = f8.round_e4m3(rng.uniform(-400, 400, (E, 2 * I, H))) / 400 / 16
    w2 = f8.round_e4m3(rng.uniform(-400, 400, (E, H, I))) / 400 / 11
    ids = np.stack([rng.choice(E, k, replace=False) for _ in range(T)])
    wt = rng.uniform(0.1, 1, (T, k)).astype(np.float32)
    out, bound, norm = f8.moe(x, ids, wt, w13, w2, 0)
    xd = f8.dequantize(*f8.quantize(x)[:2]).astype(np.float32)
    got = np.zeros((T, H), np.float32)
    for t in range(T):
        for j in range(k):
            gu = w13[ids[t, j]].astype(np.float32) @ xd[t]
            h = gu[:I] / (1 + np.exp(-gu[:I])) * gu[I:]
            hd = f8.dequantize(*f8.quantize(h[None].astype(np.float64))[:2])[0].astype(np.float32)
            got[t] += wt[t, j] * (w2[ids[t, j]].astype(np.float32) @ hd)
    assert np.all(np.abs(got - out) <= bound)
    assert np.linalg.norm(got - out) <= norm
    assert np.linalg.norm(1.01 * got - out) > norm
