"""Further GPU tests of the W8A8 layer and the dense 8-bit product against the
fp64 oracle: every form on its own, named by its plan."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import f8
from tests import f8_inputs
from tests.gpu_util import banner, host
from tests.test_gpu_f8 import C, activations, cold_calls, f64, make_layer, routing, weights  # noqa: F401  (C: a fixture)

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


GEMM_FORMS = [
    # M, N, K, plan: the last tile has 1, 33, .. rows, so every count of token
    # groups up to the tallest; 0 to 3 chunks behind the loop of four; ragged N
    (12, 300, 900, "streaming"),
    (100, 1024, 1024, "streaming"),
    (200, 520, 4000, "tiles of 64 rows, K in 8"),
    (161, 1300, 640, "tiles of 64 rows, K in 1"),
    (225, 1300, 768, "tiles of 64 rows, K in 1"),
    (255, 1300, 896, "tiles of 64 rows, K in 1"),
    (5473, 553, 1024, "tiles of 96 rows, K in 1"),
    (5601, 516, 640, "tiles of 96 rows, K in 1"),
    (5663, 515, 768, "tiles of 96 rows, K in 1"),
    (5728, 542, 832, "tiles of 96 rows, K in 1"),
    (5249, 1043, 576, "tiles of 128 rows, K in 1"),
    (6177, 833, 728, "tiles of 128 rows, K in 1"),
    (6271, 781, 832, "tiles of 128 rows, K in 1"),
    (6400, 779, 984, "tiles of 128 rows, K in 1"),
    (10977, 523, 600, "tiles of 192 rows, K in 1"),
    (11094, 516, 767, "tiles of 192 rows, K in 1"),
    (11711, 514, 856, "tiles of 192 rows, K in 1"),
    (10945, 564, 1024, "tiles of 192 rows, K in 1"),
    (12289, 819, 960, "tiles of 256 rows, K in 1"),
    (13345, 802, 576, "tiles of 256 rows, K in 1"),
    (12438, 856, 704, "tiles of 256 rows, K in 1"),
    (12488, 771, 896, "tiles of 256 rows, K in 1"),
    (12799, 828, 576, "tiles of 256 rows, K in 1"),
    (12800, 772, 704, "tiles of 256 rows, K in 1"),
    (8160, 1365, 576, "tiles of 256 rows, K in 1"),
    (8191, 4096, 7168, "tiles of 256 rows, K in 1"),
    # K in parts that a second launch adds
    (5471, 66, 2176, "tiles of 96 rows, K in 3"),
    (2721, 40, 1368, "tiles of 96 rows, K in 6"),
    (1633, 50, 4607, "tiles of 96 rows, K in 12"),
    (4129, 260, 3712, "tiles of 128 rows, K in 3"),
    (4223, 42, 2176, "tiles of 128 rows, K in 6"),
    (2305, 40, 4480, "tiles of 128 rows, K in 12"),
]


@pytest.mark.parametrize("M,N,K,plan", GEMM_FORMS)
def test_gemm_forms(C, M, N, K, plan):  # noqa: F811
    """The streaming kernel and every height of tile, inputs cold, equal bits from
    equal calls.  Value by value on a sample of rows (the first and last tiles and
    200 of the rest) against the oracle's bound.  Row by row on all: half a step of
    bf16 at every value, so of the row's norm; the sums' own errors are random and
    far smaller (a row that is 1 % off, or another row, is not)."""
    banner(f"gemm M={M} N={N} K={K} {plan}")
    codes, scales, deq = weights(1, N, K, M)
    w = C.chord_f8_pack(C.ROLE_PLAIN, codes.cuda(), scales.cuda())
    q, s = C.chord_f8_quantize(activations(M, K, M + 1).cuda())
    outs = cold_calls(lambda: C.chord_f8_gemm(q, s, w), 3)
    assert C.last_plan() == "f8 gemm: " + plan
    assert all(torch.equal(o, outs[0]) for o in outs)
    a = f8.dequantize(f8.decode(host(q.view(torch.uint8))), f64(s))[:, :K]
    rng = np.random.default_rng(M)
    ends = min(256, M)
    rows = np.unique(np.concatenate([np.arange(ends), np.arange(M - ends, M), rng.integers(0, M, 200)]))
    if K * N > 1 << 23:
        rows = rows[::4]
    got = f64(outs[0])
    ref, bound = f8.gemm(a[rows], deq[0])
    bound = bound + f8.HALF_BF16 * (np.abs(ref) + bound)
    err = np.abs(got[rows] - ref)
    assert np.all(err <= bound), (float((err / np.maximum(bound, 1e-300)).max()), rows[np.argwhere(err > bound)[:5, 0]])
    whole = (torch.from_numpy(a).cuda() @ torch.from_numpy(deq[0].T.copy()).cuda()).cpu().numpy()
    assert np.allclose(whole[rows], ref, rtol=0, atol=1e-9 * np.abs(ref).max())
    off = np.linalg.norm(got - whole, axis=1) / np.linalg.norm(whole, axis=1)
    assert np.all(off <= f8.HALF_BF16), (off.max(), np.argwhere(off > f8.HALF_BF16)[:5, 0])
    banner(f"  worst row {off.max():.5f}")


MANY_ROWS = [
    # T, H, I, E, k, hot, plan
    (300, 384, 256, 50, 2, 0, "blocks of 32 rows"),
    (450, 640, 128, 70, 3, 0, "blocks of 32 rows"),
    (230, 768, 640, 24, 2, 0, "blocks of 32 rows"),
    (420, 640, 768, 16, 2, 0, "blocks of 32 rows"),
    (900, 384, 1152, 20, 1, 0, "tiles of up to 224 rows"),   # 45 rows an expert: fp32 sums
    (1500, 640, 768, 40, 1, 1, "tiles of up to 224 rows"),
    (1100, 896, 896, 30, 1, 2, "tiles of up to 224 rows"),
    (800, 384, 768, 16, 2, 0, "tiles of up to 224 rows"),    # 100 rows: 8-bit sums
    (1000, 640, 640, 18, 2, 2, "tiles of up to 224 rows"),
    (1400, 896, 896, 12, 1, 1, "tiles of up to 224 rows"),
    (1900, 512, 640, 10, 2, 0, "tiles of up to 224 rows"),
]


@pytest.mark.parametrize("T,H,I,E,k,hot,plan", [(*c[:5], 0, c[5]) for c in LAYER_FORMS] + MANY_ROWS[1:4] + MANY_ROWS[4:7] + MANY_ROWS[8:])
def test_moe_every_row_with_exact_sums(C, T, H, I, E, k, hot, plan):  # noqa: F811
    """Inputs whose gate_up products are exact (tests/f8_inputs.py): every token is
    within half a step of bf16 of its norm.  At the norms of an fp32 error of
    2e-6 a value of h takes another code at 6e-5 of the values (as in
    test_moe_rows_of_few_are_as_exact_as_bf16), and shows where it is one of the
    few that are more than 0.06 of the token: below 1 % of the tokens."""
    from quantized_moe_amd.moe import W8A8MoE
    banner(f"f8 moe rows T={T} H={H} I={I} E={E} k={k} hot={hot}")
    c13, s13, d13 = f8_inputs.gate_up(E, H, I, T)
    c2, s2, d2 = weights(E, H, I, T + 1)
    layer = W8A8MoE(c13.cuda(), s13.cuda(), c2.cuda(), s2.cuda())
    ids, w = routing(T, E, k, T + 2, hot)
    x = f8_inputs.tokens(T, H, T + 3)
    ref, _, _ = f8.moe(f64(x), ids, w, d13, d2, 0)
    got = layer.indexed(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), 0, E)
    assert C.last_plan() == "f8 moe: " + plan
    off = f8.rows_off(f64(got), ref)
    banner(f"  worst token {off.max():.5f}")
    assert (off > f8.HALF_BF16).sum() <= max(1, T // 100), np.sort(off)[-T // 100 - 3:]
    assert off.max() <= 0.04


@pytest.mark.parametrize("T,H,I,E,k,hot,plan", MANY_ROWS)
def test_moe_every_row_of_many(C, T, H, I, E, k, hot, plan):  # noqa: F811
    """Ordinary inputs.  gate_up below 64 rows an expert is summed in fp32, so the
    tokens are as exact as bf16 but for 1 % (see above).  Above, eights of products are
    summed on a grid of 2^-13: h is off by about 1e-4 of itself and every
    few hundredth value takes the neighbouring code, an eighth of it away at most.
    No token may be off by more than 0.04: that would take a flip of a value that
    makes up a third of the token's norm (the largest of each 128, whose code is 448
    by construction, cannot flip)."""
    banner(f"f8 moe many rows T={T} H={H} I={I} E={E} k={k} hot={hot}")
    layer, d13, d2 = make_layer(E, H, I, T + E)
    ids, w = routing(T, E, k, I + T, hot)
    x = activations(T, H, 3)
    ref, _, _ = f8.moe(f64(x), ids, w, d13, d2, 0)
    got = layer.indexed(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), 0, E)
    assert C.last_plan() == "f8 moe: " + plan
    off = f8.rows_off(f64(got), ref)
    banner(f"  worst token {off.max():.5f}, over half a step of bf16 {(off > f8.HALF_BF16).mean():.3f}")
    assert off.max() <= 0.04
    if plan == "blocks of 32 rows" or T * k < 64 * E:
        assert (off > f8.HALF_BF16).sum() <= max(1, T // 100), np.sort(off)[-T // 100 - 3:]


def test_gemm_sums_inside_a_block_as_documented(C):  # noqa: F811
    """A small term beside two that cancel: kept exactly where it stands in another
    eight of the block, off by the grid of its own eight at most (7 products on
    2^-13 of the largest's power of two) where it stands beside them."""
    for where, exact in ((8, True), (120, True), (2, False), (7, False)):
        x = torch.zeros((1, 128), dtype=torch.bfloat16)
        codes = torch.zeros((1, 1, 128))
        x[0, :2] = 1.0                      # code 448, scale 1 / 448
        codes[0, 0, 0], codes[0, 0, 1] = 448.0, -448.0
        x[0, where] = 2.0 ** -9             # code 0.875
        codes[0, 0, where] = 1.0
        w = C.chord_f8_pack(C.ROLE_PLAIN, codes.to(torch.float8_e4m3fn).cuda(), torch.ones((1, 1, 1), device="cuda"))
        got = float(C.chord_f8_gemm(*C.chord_f8_quantize(x.cuda()), w))
        want = 0.875 / 448
        if exact:
            assert abs(got - want) <= (f8.HALF_BF16 + 4 * f8.U32) * want
        else:
            assert abs(got - want) <= 7 * 2.0 ** -13 * 2.0 ** 17 / 448 * (1 + f8.HALF_BF16)


def test_moe_slots_past_32_bits(C):  # noqa: F811
    """40000 tokens of 8 slots and 7168 outputs: y of the last slots lies past 4 GiB.
    Tokens without a local expert are zeros, a sample of the others (first, last,
    and between) is compared with the oracle."""
    T, H, I, E, E_g, k = 40000, 7168, 128, 2, 64, 8
    banner(f"f8 moe T={T} H={H} I={I} E={E} k={k}")
    layer, d13, d2 = make_layer(E, H, I, 21)
    rng = np.random.default_rng(22)
    ids = np.argsort(rng.random((T, E_g)), axis=1)[:, :k].astype(np.int32)
    w = rng.uniform(0.1, 1.0, (T, k)).astype(np.float32)
    ids[-3:, -1] = [0, 1, 0]   # (the very last slot is local; an expert may stand twice)
    g = torch.Generator(device="cuda").manual_seed(23)
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    got = layer.indexed(x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), 0, E_g)
    local = (ids < E).any(axis=1)
    rows = np.nonzero(local)[0]
    rows = np.concatenate([rows[:20], rng.choice(rows, 60, replace=False), rows[-40:]])
    assert not got[torch.from_numpy(~local).cuda()].any()
    at = torch.from_numpy(rows).cuda()
    ref, bound, _ = f8.moe(f64(x[at]), ids[rows], w[rows], d13, d2, 0)
    part = f64(got[at])
    assert np.all(np.abs(part - ref) <= bound)
    assert f8.rows_off(part, ref).max() <= 0.04


CHILD = """
import torch
from quantized_moe_amd import chord as C
from quantized_moe_amd.moe import W8A8MoE
s = torch.load(r"{path}", weights_only=True)
w = [t.view(torch.float8_e4m3fn).cuda() if t.dtype is torch.uint8 else t.cuda() for t in s["weights"]]
layer, a = W8A8MoE(*w), (s["x"].cuda(), s["ids"].cuda(), s["w"].cuda(), 0, {E})
junk = torch.empty(1 << 27, device="cuda")
outs = []
for i in range(4):
    junk.fill_(i)   # pushes the inputs out of the caches
    outs.append(layer.indexed(*a))
torch.cuda.synchronize()
same = all(torch.equal(o, outs[0]) for o in outs)
torch.save({{"out": outs[0].cpu(), "plan": C.last_plan(), "same": same}}, r"{path}")
"""


def test_moe_fp32_sums_at_every_size(C, tmp_path):  # noqa: F811
    """CHORD_F8_FP32_SUMS=1, in a process of its own: large tiles, in every number of
    token groups and of chunks behind the loop, give every token as exact as bf16
    (but for 1 %, as above), and equal bits on every call."""
    for T, H, I, E, k, hot in ((800, 384, 768, 16, 2, 0), (1000, 640, 640, 18, 2, 2), (1500, 768, 384, 30, 2, 0),
                               (1400, 896, 896, 12, 1, 1), (1900, 512, 640, 10, 2, 0)):
        check_fp32_sums(T, H, I, E, k, hot, str(tmp_path / f"layer{T}.pt"))


def check_fp32_sums(T, H, I, E, k, hot, path):
    banner(f"f8 moe fp32 sums T={T} H={H} I={I} E={E} k={k} hot={hot}")
    c13, s13, d13 = weights(E, 2 * I, H, 31)
    c2, s2, d2 = weights(E, H, I, 32)
    ids, w = routing(T, E, k, 33, hot)
    x = activations(T, H, 34)
    torch.save({"weights": [c13.view(torch.uint8), s13, c2.view(torch.uint8), s2], "x": x,
                "ids": torch.from_numpy(ids), "w": torch.from_numpy(w)}, path)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CHILD.format(path=path, E=E)], cwd=root, timeout=100,
                       env=dict(os.environ, CHORD_F8_FP32_SUMS="1"), capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    got = torch.load(path, weights_only=True)
    assert got["plan"] == "f8 moe: tiles of up to 224 rows" and got["same"]
    ref, _, _ = f8.moe(f64(x), ids, w, d13, d2, 0)
    off = f8.rows_off(f64(got["out"]), ref)
    assert (off > f8.HALF_BF16).sum() <= T // 100 and off.max() <= 0.04, np.sort(off)[-10:]
