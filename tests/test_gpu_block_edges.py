"""Balance, norms and the 16-bit product where their arithmetic or their schedule is at an
edge: scores that are all small beside the 1e-20 of their sum, rows of one huge value,
factors that leave fp32 before they meet, products whose workgroups go through several
items.  Bounds are those of the operators' own tests."""

import numpy as np
import pytest
import torch

from oracle import block as B
from tests import test_gpu_balance, test_gpu_block_sizes, test_gpu_linear, test_gpu_norm
from tests.gpu_util import banner

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def C():
    from quantized_moe_amd import chord
    return chord


# ---- balance: sigmoids whose sum is near 1e-20 -----------------------------------
@pytest.mark.parametrize("level", [-20, -30, -36, -40, -44, -46, -48, -50, -60, -80])
@pytest.mark.parametrize("E,left", [(4, 4), (8, 8), (256, 256), (384, 5)])
def test_small_sigmoids(C, level, E, left):
    """All scores of a row are small, so they do not add up to 1.  (`left` experts are
    in service.)"""
    T, k = 24, 2
    banner(f"balance of logits near {level}, {left} of {E} experts")
    for dtype in (F32, BF16):
        logits, ids = test_gpu_balance.draw(T, E, k, E - level, dtype)
        logits = (0.3 * logits.float() + level).to(dtype)
        logits[7] = logits[7].abs()  # a row among them whose scores do
        logits[:, left:] = -np.inf
        ids %= left
        ids[3] = -1
        for n_seq in (1, 4):
            up = torch.linspace(0.5, 2, n_seq).cuda()
            test_gpu_balance.check(C, logits.cuda(), ids.cuda(), True, n_seq, grad_loss=up)
            test_gpu_balance.check(C, logits.cuda(), ids.cuda(), False, n_seq, grad_loss=up)


def test_gradient_of_small_sigmoids_against_differences(C):
    """As test_gradient_against_differences has it, at scores of some 1e-20."""
    logits, ids = test_gpu_balance.draw(48, 32, 2, 9)
    logits = 0.3 * logits - 49
    r = C.chord_moe_balance(logits.cuda(), ids.cuda(), C.SCORE_SIGMOID, want_grad=True)
    g = r.grad.double()
    size = g.norm().item()
    step = 0.5 * g / size
    two = [C.chord_moe_balance((logits.cuda().double() + s * step).float(), ids.cuda(), C.SCORE_SIGMOID).loss.item()
           for s in (1, -1)]
    # (Logits of 49 are rounded to 2^-19, the steps with them: 2^-19 sqrt(48 * 32) |g| at most.)
    assert size > 0.01
    assert abs((two[0] - two[1]) - size) < 0.05 * size + 2.0 ** -22 + 2.0 ** -18 * 40 * size


# ---- norms: rows of one huge value -------------------------------------------------
@pytest.mark.parametrize("H", [1, 384, 512, 5000, 7113, 20001])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_constant_rows(C, H, dtype):
    """Rows of one value, up to those whose sums or squares leave fp32.  Their layer norm
    is the bias: powers of two add up exactly, so it is that to the bit, also as the
    norm behind a block."""
    values = [2.5, 2.0 ** 60, 2.0 ** 100, -2.0 ** 116, 2.0 ** 120, 2.0 ** 125, -2.0 ** 127, 3e38, -3.38e38]
    T = len(values)
    banner(f"constant rows H={H} {dtype}")
    x = torch.tensor(values).to(dtype)[:, None].repeat(1, H).cuda()
    exact = [t for t in range(T) if np.log2(abs(values[t])) % 1 == 0]
    for kind in ("rms", "layer"):
        p = test_gpu_norm.Part(C, H, kind, F32, bias=kind == "layer")
        r = test_gpu_norm.check(C, x, p, codes=True)
        assert torch.isfinite(r.out).all()
        res = test_gpu_norm.rows(T, H, F32, 3).cuda()
        behind = C.chord_norm(x, post=p.gpu, residual=res).sum
        torch.cuda.synchronize()
        assert torch.isfinite(behind).all()
        if kind == "layer":
            assert torch.equal(r.out[exact], p.gpu.bias.to(dtype).expand(T, H)[exact])
            assert torch.equal(behind[exact], (res + p.gpu.bias)[exact])


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_eps_beside_squares_that_overflow(C, kind):
    """An eps of the size of the squares' mean counts, though their sum leaves fp32."""
    banner(f"large eps {kind}")
    for H in (384, 5000):
        p = test_gpu_norm.Part(C, H, kind, F32, eps=1e37)
        x = torch.cat([test_gpu_norm.rows(4, H, F32, 1, 2.0 ** e) for e in (50, 60, 62, 70)]).cuda()
        test_gpu_norm.check(C, x, p)


# ---- norms: weights that have moved --------------------------------------------------
def test_weights_that_have_moved(C):
    """A norm reads its tensors where they are at the call."""
    banner("weights that have moved")
    H = 200
    x = test_gpu_norm.rows(3, H, BF16, 1).cuda()
    for bias in (False, True):
        p, q = (test_gpu_norm.Part(C, H, "layer", BF16, bias, seed=s) for s in (1, 2))
        n = p.gpu
        before = [n.weight.data, n.bias.data if bias else None]   # (kept, so that nothing is freed)
        n.weight.data = q.gpu.weight.clone()
        if bias:
            n.bias.data = q.gpu.bias.clone()
        assert torch.equal(C.chord_norm(x, n).out, C.chord_norm(x, q.gpu).out)
        n.weight = before[0].float()
        n.bias = before[1].float() if bias else None
        want = C.chord_norm(x, C.Norm(n.weight, n.bias, 1e-6, C.NORM_LAYER)).out
        assert torch.equal(C.chord_norm(x, n).out, want)
        n.weight = before[0][::2]
        with pytest.raises(C.ChordError):
            C.chord_norm(x, n)


# ---- norms: factors that leave fp32 before they meet --------------------------------
@pytest.mark.parametrize("shape", ["token", "column", "full"])
@pytest.mark.parametrize("H", [200, 7168])
def test_scale_and_gate_meet_the_value_one_by_one(C, shape, H):
    """scale * gate is beyond fp32 both ways, scale * (gate * u) is not."""
    T = 5
    banner(f"far gates by {shape} H={H}")
    gate = {"token": (T, 1), "column": (H,), "full": (T, H)}[shape]
    for e in (-75, 70):
        x = (test_gpu_norm.rows(T, H, F32, 1) * 2.0 ** -e).cuda()
        g = torch.full(gate, 2.0 ** e, dtype=F32).cuda()
        r = test_gpu_norm.check(C, x, gate=g, scale=1.5 * 2.0 ** e)
        assert torch.isfinite(r.sum).all() and r.sum.abs().max() > 2.0 ** (e - 1)


@pytest.mark.parametrize("shape", ["token", "column", "full"])
def test_sigmoid_gates_far_from_zero(C, shape):
    """Gates of -120 to 120: e^120 is beyond fp32, the sigmoid beside it only small (from
    2^-126 down to nothing in steps of 2^-149)."""
    T, H = 61, 264
    banner(f"far sigmoid gates by {shape}")
    x = test_gpu_norm.rows(T, H, F32, 1)
    g = torch.linspace(-120, 120, T)[:, None].expand(T, H)
    if shape == "column":
        g = torch.linspace(-120, 120, H)[None, :].expand(T, H)
    gpu = {"token": g[:, :1], "column": g[0], "full": g}[shape].contiguous().cuda()
    r = C.chord_norm(x.cuda(), gate=gpu, gate_sigmoid=True)
    torch.cuda.synchronize()
    g = g.double().numpy()
    s, err, _, _ = B.block_norm(x.double().numpy(), gate=g, gate_sigmoid=True)
    # A sigmoid below 2^-126 is off by a step of 2^-149 instead, for its value's size.
    err = err + 2.0 ** -149 * np.abs(x.double().numpy()) * (g < -80)
    test_gpu_norm.close(r.sum, s, err, F32, "sum")


# ---- products: several items a workgroup --------------------------------------------
CUS, TILE = 256, 256
ROUNDS = [
    # M, rows of W, K, whole rounds of tiles of 256 x 256, items behind them
    (2000, 4104, 584, 0, 136),   # one round of whole tiles, nine chunks and an eighth
    (4300, 4104, 264, 1, 33),    # ... and a last one in halves; five chunks
    (4200, 4104, 328, 1, 33),    # ... of which the last token tile's second has no rows
    (5300, 5128, 264, 1, 185),   # ... of whole tiles
    (5700, 5640, 264, 2, 17),
]


@pytest.mark.parametrize("M,R,K,rounds,rest", ROUNDS)
def test_rounds_of_large_tiles(C, M, R, K, rounds, rest):
    """Outputs that go straight to memory and through LDS, plain and gated."""
    assert torch.cuda.get_device_properties(0).multi_processor_count == CUS
    tiles = -(-M // TILE)
    for dtype, rows, kw in ((BF16, R, dict(residual=True)),
                            (F16, R - 2, dict(out=F32, bias=F16, act="relu")),
                            (BF16, R - 6, dict(act="gelu_tanh", residual=True, scale=0.5)),
                            (BF16, R, dict(gated=True, act="silu", bias=F32, residual=True, scale=0.7)),
                            (F16, R - 4, dict(gated=True, act="silu", residual=True))):
        items = tiles * -(-rows // TILE)
        assert items == rounds * CUS + rest
        test_gpu_linear.check(C, M, rows // (1 + kw.get("gated", False)), K, dtype, **kw)
        assert C.last_plan() == "linear: tiles of 256 x 256, K in 1"


def test_rounds_of_large_tiles_through_the_long_activation(C):
    for M, R, K in ((2000, 4104, 328), (4300, 4104, 264)):
        test_gpu_linear.check(C, M, R, K, act="gelu", residual=True)
        assert C.last_plan() == "linear: tiles of 256 x 256, K in 1"


@pytest.mark.parametrize("M,R,K,form", [
    (3723, 264, 5704, "tiles of 256 x 256, K in 4"),     # 120 items: halves of parts
    (6773, 522, 19448, "tiles of 256 x 256, K in 4"),    # 324: and a round of whole ones in front
    (4948, 3080, 328, "tiles of 128 x 256, K in 1"),     # 507
    (4098, 5658, 264, "tiles of 128 x 256, K in 1"),     # 759
    (5481, 1292, 520, "tiles of 128 x 128, K in 1"),     # 473
    (5897, 2570, 1032, "tiles of 128 x 128, K in 1"),    # 987
])
def test_rounds_of_other_tiles(C, M, R, K, form):
    for dtype, gated, kw in ((BF16, False, dict(residual=True)), (F16, True, dict(act="silu", bias=F32))):
        test_gpu_linear.check(C, M, R // (1 + gated), K, dtype, gated=gated, **kw)
        assert C.last_plan() == "linear: " + form


def test_equal_calls_of_several_rounds(C):
    """Equal bits, also beside a second stream's call and from a graph."""
    x, w = test_gpu_linear.rows(4300, 264, BF16, 1).cuda(), test_gpu_linear.rows(4104, 264, BF16, 2, 0.06).cuda()
    res = test_gpu_linear.rows(4300, 4104, BF16, 3).cuda()
    want = C.chord_linear(x, w, residual=res, act=C.ACT_SILU)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = [C.chord_linear(x, w, residual=res, act=C.ACT_SILU, stream=s) for _ in range(4) for s in sides]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = C.chord_linear(x, w, residual=res, act=C.ACT_SILU)
    for seed in range(3):
        x.copy_(test_gpu_linear.rows(4300, 264, BF16, 10 + seed))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, C.chord_linear(x, w, residual=res, act=C.ACT_SILU))


# ---- balance: drawn from the seed alone ---------------------------------------------
@pytest.mark.parametrize("seed", range(30))
def test_drawn_balances_of_a_seed(C, seed):
    """Everything that is drawn, experts out of service and upstream gradients among it,
    comes from the seed."""
    rng = np.random.Generator(np.random.PCG64(500 + seed))
    n_seq, E = test_gpu_block_sizes.drawn(rng, 1, 40), test_gpu_block_sizes.drawn(rng, 1, 1024)
    T, k = n_seq * test_gpu_block_sizes.drawn(rng, 1, 300), test_gpu_block_sizes.drawn(rng, 1, min(E, 64))
    banner(f"balance seed={seed} T={T} E={E} k={k} n_seq={n_seq}")
    logits, ids = test_gpu_balance.draw(T, E, k, seed, (F32, BF16, F16)[rng.integers(3)], 0.2 * rng.integers(2))
    bias = torch.from_numpy(np.where(rng.random(E) < 0.1, -np.inf, 0.0).astype(np.float32)).cuda()
    up = torch.from_numpy((rng.random(n_seq) + 0.5).astype(np.float32)).cuda()
    test_gpu_balance.check(C, logits.cuda(), ids.cuda(), bool(rng.integers(2)), n_seq, bias if rng.integers(2) else None,
                           up if rng.integers(2) else None)


# ---- products: activations far below 0 ----------------------------------------------
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu"])
@pytest.mark.parametrize("M,K,gated", [(3, 8, False), (40, 16, True), (300, 8, False), (700, 72, True)])
def test_activations_that_nearly_vanish(C, act, M, K, gated):
    """z of -120 to 0 (exact: one product of a power of two each), where e^-z leaves fp32 and
    the result does not: it is off by 8 units and some for each of the exponent's, or by a
    step or two of 2^-149.  The exponential rounds its argument times log2 e, itself
    rounded: 2 units for each of the argument's, and erfc takes no more than twice that.
    GELU_TANH's argument c (z + d z z z) has its own roundings, of d, of three products, of
    the sum, of c and of the last product: 7 more."""
    N = 512
    banner(f"{act} far below 0, M={M} K={K} gated={gated}")
    z = torch.linspace(-120 if act == "silu" else -15, 0, N).to(BF16)
    x = torch.zeros((M, K), dtype=BF16)
    x[:, 0], x[:, 1] = 1, 2
    w = torch.zeros((N * (1 + gated), K), dtype=BF16)
    w[:N, 0] = z
    w[N:, 1] = 0.5
    got = C.chord_linear(x.cuda(), w.cuda(), act=getattr(C, "ACT_" + act.upper()), gated=gated, out_dtype=F32)
    torch.cuda.synchronize()
    z = z.double().numpy()
    ref = B.activation(z, act)
    u = {"silu": np.abs(z), "gelu": z * z / 2, "gelu_tanh": np.abs(1.6 * (z + 0.045 * z ** 3))}[act]
    # Half a step each of z h, z h h and the last product; of GELU's erfc a step for each unit of z.
    each = 9 if act == "gelu_tanh" else 4
    bound = (8 + each * u) * B.U32 * np.abs(ref) + 2.0 ** -149 * (2 + np.abs(z))
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= bound), (np.argwhere(err > bound)[:4], z[(err > bound).any(axis=0)][:4])


@pytest.mark.parametrize("E,rows", [(384, 64), (385, 54), (512, 48), (1000, 24), (1024, 24)])
def test_both_sides_of_one_launch(C, E, rows):
    """Rows that one launch takes, and one more."""
    for L in (rows, rows + 1):
        for n_seq in (1, 3):
            banner(f"balance n_seq={n_seq} rows={L} E={E}")
            logits, ids = test_gpu_balance.draw(n_seq * L, E, 7, E + L, BF16, 0.1)
            for sigmoid in (False, True):
                a = test_gpu_balance.check(C, logits.cuda(), ids.cuda(), sigmoid, n_seq)
                b = C.chord_moe_balance(logits.cuda(), ids.cuda(), int(sigmoid), n_seq=n_seq, want_grad=True)
                torch.cuda.synchronize()
                assert all(torch.equal(p, q) for p, q in zip(a, b))
