"""The check of single tokens of the W8A8 layer, on the CPU: the layer in fp32
passes it, one token that is 5 % (or 1 %) off does not."""

import numpy as np

from oracle import f8
from tests import f8_inputs


def layer_fp32(x, ids, wt, w13, w2):
    """The layer in fp32 NumPy, rounded to bf16 at the end."""
    import torch
    I = w2.shape[2]
    xd = f8.dequantize(*f8.quantize(x)[:2]).astype(np.float32)
    got = np.zeros(x.shape, np.float32)
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            gu = w13[ids[t, j]].astype(np.float32) @ xd[t]
            h = gu[:I] / (1 + np.exp(-gu[:I])) * gu[I:]
            hd = f8.dequantize(*f8.quantize(h[None].astype(np.float64))[:2])[0].astype(np.float32)
            got[t] += wt[t, j] * (w2[ids[t, j]].astype(np.float32) @ hd)
    return torch.from_numpy(got).bfloat16().double().numpy()


def test_a_token_that_is_off_is_seen():
    T, H, I, E, k = 40, 384, 256, 3, 2
    rng = np.random.default_rng(1)
    _, _, w13 = f8_inputs.gate_up(E, H, I, 2)
    w2 = f8.round_e4m3(rng.uniform(-400, 400, (E, H, I))) / 400 / I ** 0.5
    ids = np.stack([rng.choice(E, k, replace=False) for _ in range(T)])
    wt = rng.uniform(0.1, 1, (T, k)).astype(np.float32)
    x = f8_inputs.tokens(T, H, 3).double().numpy()
    ref, _, _ = f8.moe(x, ids, wt, w13, w2, 0)
    got = layer_fp32(x, ids, wt, w13, w2)
    assert np.all(f8.rows_off(got, ref) <= f8.HALF_BF16)
    for factor in (1.01, 1.05, 0.95):
        bad = got.copy()
        bad[17] *= factor
        assert list(np.nonzero(f8.rows_off(bad, ref) > f8.HALF_BF16)[0]) == [17]
    bad = got.copy()
    bad[17] *= 1.05
    assert f8.rows_off(bad, ref)[17] > 0.04   # also with the wider limit of large tiles
    bad[17] = got[16]
    assert f8.rows_off(bad, ref)[17] > 0.04


def test_products_of_the_inputs_are_exact_on_the_grid():
    """Within a block of 128 every product is a whole multiple of the smallest
    possible one, and the largest is 2^5 of those."""
    codes, _, _ = f8_inputs.gate_up(1, 256, 128, 5)
    v, _, _ = f8.quantize(f8_inputs.tokens(9, 256, 6).double().numpy())
    assert set(np.unique(np.abs(v))) == {448.0, 224.0, 112.0, 56.0}
    assert set(np.unique(np.abs(codes.float().numpy()))) == {1.0, 2.0, 4.0}


def test_rows_off_of_empty_rows():
    z = np.zeros((2, 4))
    assert list(f8.rows_off(z, z)) == [0.0, 0.0]
    assert np.isinf(f8.rows_off(z + 1, z)).all()
