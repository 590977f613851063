"""Further GPU tests of the W8A8 layer and the dense 8-bit product against the
fp64 oracle: every form on its own, named by its plan."""

import numpy as np
import pytest
import torch

from oracle import f8
from tests.gpu_util import banner
from tests.test_gpu_f8 import C, activations, f64, routing, weights  # noqa: F401  (C: a fixture)

pytestmark = pytest.mark.gpu


LAYER_FORMS = [
    # T, H, I, E, k, plan
    (3, 256, 128, 4, 2, "a handful of tokens, two launches"),
    (40, 512, 384, 8, 2, "blocks of 16 rows, streaming gate_up"),   # tiled down
    (40, 512, 256, 8, 2, "blocks of 16 rows, streaming gate_up"),   # down of short K
    (120, 640, 384, 90, 4, "blocks of 16 rows"),
    (90, 896, 256, 100, 4, "blocks of 16 rows"),
    (450, 640, 128, 70, 3, "blocks of 32 rows"),
    (300, 384, 256, 50, 2, "blocks of 32 rows"),
    (420, 640, 768, 16, 2, "blocks of 32 rows"),
    (800, 384, 768, 16, 2, "tiles of up to 224 rows"),
]


@pytest.mark.parametrize("T,H,I,E,k,plan", LAYER_FORMS)
def test_moe_one_output_that_is_not_finite(C, T, H, I, E, k, plan):  # noqa: F811
    """A NaN code in one row of w2 makes that output of its expert's tokens NaN, and
    a row whose sums leave fp32 makes it infinite; neither touches another output."""
    from quantized_moe_amd.moe import W8A8MoE
    banner(f"f8 moe not finite T={T} H={H} I={I} E={E} k={k}")
    c13, s13, d13 = weights(E, 2 * I, H, 3)
    c2, s2, d2 = weights(E, H, I, 4)
    ids, w = routing(T, E, k, 5)
    x = activations(T, H, 6)
    nan_row, inf_row, e = 37, H - 1, int(ids[1, 0])
    bits = c2.view(torch.uint8)
    # Expert e's last 128 outputs, scaled by 1e37: codes of 2^-9 keep them finite
    # (below I^0.5 2^-9 1e37 |h|), the last output has codes of 448, in its first
    # chunk alone, so that no two infinities of different sign meet.
    bits[e, H - 128:, :] = bits[e, H - 128:, :] & 0x80 | 1
    bits[e, inf_row, :128] = bits[e, inf_row, :128] & 0x80 | 0x7E
    bits[e, inf_row, 128:] = 0
    s2[e, -1, :] = 1e37
    d2[e] = f8.dequantize_weight(f64(c2[e].float()), f64(s2[e]))
    ref, bound, _ = f8.moe(f64(x), ids, w, d13, d2, 0)
    bits[e, nan_row, I // 2] = 0x7F
    layer = W8A8MoE(c13.cuda(), s13.cuda(), c2.cuda(), s2.cuda())
    got = f64(layer.indexed(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), 0, E))
    assert C.last_plan() == "f8 moe: " + plan
    uses = (ids == e).any(axis=1)
    assert np.isnan(got[uses, nan_row]).all() and uses.any()
    big = float(torch.finfo(torch.float32).max)
    over = uses & (np.abs(ref[:, inf_row]) > 8 * big)   # (surely: the sum over slots included)
    assert over.any() and np.isinf(got[over, inf_row]).all()
    keep = np.ones(got.shape, bool)
    keep[uses, nan_row] = keep[uses, inf_row] = False
    assert np.abs(ref[keep]).max() < big / 8            # what is compared is finite
    err = np.abs(got - ref)
    assert np.all(err[keep] <= bound[keep]), np.argwhere(keep & ~(err <= bound))[:5]
