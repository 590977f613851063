"""Norms, 16-bit product and balance over drawn sizes and options, in every form that
the product's plan chooses between, on tensors whose rows lie behind 4 GB, and on two
streams at once.  Bounds are those of the operators' own tests."""

import math

import numpy as np
import pytest
import torch

from tests import test_gpu_balance, test_gpu_linear, test_gpu_norm
from tests.gpu_util import banner

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
FAR = 1 << 21  # elements between rows: 4 MB in 16 bits


@pytest.fixture(scope="module")
def C():
    from quantized_moe_amd import chord
    return chord


# ---- the forms of the product --------------------------------------------------
FORMS = [
    (8, 40, 72, "streaming, 16 tokens"),
    (24, 2056, 72, "streaming, 32 tokens"),
    (40, 2056, 72, "streaming, 64 tokens"),
    (700, 4104, 72, "tiles of 256 x 256, K in 1"),
    (900, 4104, 1032, "tiles of 128 x 256, K in 1"),
    (1500, 1300, 72, "tiles of 128 x 128, K in 1"),
    (2050, 130, 4104, "tiles of 128 x 128, K in 4"),
    (8, 4104, 72, "tiles of 64 x 128, K in 1"),
    (24, 4104, 2056, "tiles of 64 x 128, K in 4"),
]


@pytest.mark.parametrize("M,R,K,form", FORMS)
def test_forms_of_the_product(C, M, R, K, form):
    """R rows of W: as outputs, and as gate and up rows with everything behind them."""
    for dtype, N, kw in ((BF16, R, {}), (F16, R, dict(out=F32, bias=F16, act="gelu")),
                         (BF16, R // 2, dict(gated=True, act="silu", bias=F32, residual=True, scale=0.7)),
                         (F16, R // 2, dict(gated=True, act="gelu_tanh", out=F32))):
        test_gpu_linear.check(C, M, N, K, dtype, **kw)
        if not kw.get("gated"):  # (8 outputs to a streaming workgroup, so another form may be cheaper)
            assert C.last_plan() == "linear: " + form


def drawn(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


@pytest.mark.parametrize("seed", range(40))
def test_drawn_products(C, seed):
    rng = np.random.Generator(np.random.PCG64(seed))
    M, N, K = drawn(rng, 1, 900), drawn(rng, 1, 900), drawn(rng, 1, 3000)
    dtype = (BF16, F16)[rng.integers(2)]
    out = F32 if K >= 64 and rng.integers(2) else dtype
    gated = bool(rng.integers(2))
    bias = (None, F32, dtype)[rng.integers(3)]
    act = test_gpu_linear.ACTS[rng.integers(5)]
    pad, off = int(rng.integers(0, 12)), int(rng.integers(0, 9))
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K + pad + off), generator=g).to(dtype).cuda()[:, off:off + K]
    w = (K ** -0.5 * torch.randn((N * (1 + gated), K + pad), generator=g)).to(dtype).cuda()[:, :K]
    test_gpu_linear.check(C, M, N, K, dtype, out, act, gated, bias, bool(rng.integers(2)),
                          float(rng.choice([1.0, -0.3, 4.0])), x, w)


# ---- norms -------------------------------------------------------------------
@pytest.mark.parametrize("seed", range(40))
def test_drawn_norms(C, seed):
    rng = np.random.Generator(np.random.PCG64(100 + seed))
    T, H = drawn(rng, 1, 600), drawn(rng, 1, 12000)
    dtype = (BF16, F16, F32)[rng.integers(3)]
    banner(f"norm T={T} H={H} {dtype}")

    def part(n):
        return test_gpu_norm.Part(C, H, ("rms", "layer")[rng.integers(2)], (dtype, F32)[rng.integers(2)],
                                  bool(rng.integers(2)), 1e-5, float(rng.integers(2)), n)
    pre = part(1) if rng.integers(4) else None
    post = part(2) if rng.integers(2) else None
    g = (None, "token", "column", "full")[rng.integers(4)]
    gate = None
    if g:
        gate = test_gpu_norm.rows(T, H, (dtype, F32)[rng.integers(2)], seed)
        gate = (gate[:, :1] if g == "token" else gate[0] if g == "column" else gate).contiguous().cuda()
    stream = (dtype, F32)[rng.integers(2)]
    pad, off = int(rng.integers(0, 9)), int(rng.integers(0, 5))
    x = test_gpu_norm.rows(T, H + pad + off, dtype, seed + 1).cuda()[:, off:off + H]
    res = test_gpu_norm.rows(T, H + pad, stream, seed + 2).cuda()[:, :H] if rng.integers(2) else None
    test_gpu_norm.check(C, x, pre, post, gate, bool(rng.integers(2)), res, float(rng.choice([1.0, 0.22])), stream,
                        codes=pre is not None and bool(rng.integers(2)))


@pytest.mark.parametrize("T,H", [(3, 7168), (700, 7168), (3, 16384), (600, 16384), (2, 20001), (5, 32768)])
def test_more_columns_than_lds_holds(C, T, H):
    """Two layer norms with biases and a gate by column, all fp32: five vectors."""
    pre, post = (test_gpu_norm.Part(C, H, "layer", F32, True, seed=s) for s in (1, 2))
    for dtype in (BF16, F32):
        banner(f"norm T={T} H={H} {dtype}")
        test_gpu_norm.check(C, test_gpu_norm.rows(T, H, dtype, 1).cuda(), pre, post,
                            test_gpu_norm.rows(1, H, F32, 2)[0].cuda(), True,
                            test_gpu_norm.rows(T, H, F32, 3).cuda(), 0.5, codes=True)


# ---- balance -----------------------------------------------------------------
@pytest.mark.parametrize("seed", range(30))
def test_drawn_balances(C, seed):
    rng = np.random.Generator(np.random.PCG64(200 + seed))
    n_seq, E = drawn(rng, 1, 40), drawn(rng, 1, 1024)
    T, k = n_seq * drawn(rng, 1, 300), drawn(rng, 1, min(E, 64))
    banner(f"balance T={T} E={E} k={k} n_seq={n_seq}")
    logits, ids = test_gpu_balance.draw(T, E, k, seed, (F32, BF16, F16)[rng.integers(3)], 0.2 * rng.integers(2))
    logits = logits.cuda()
    if rng.integers(2):
        wide = torch.full((T, E + 3), float("nan"), dtype=logits.dtype, device="cuda")
        wide[:, 1:E + 1] = logits
        logits = wide[:, 1:E + 1]
    bias = torch.where(torch.rand(E) < 0.1, -np.inf, 0.0).cuda() if rng.integers(2) else None
    up = (torch.rand(n_seq) + 0.5).cuda() if rng.integers(2) else None
    test_gpu_balance.check(C, logits, ids.cuda(), bool(rng.integers(2)), n_seq, bias, up)


# ---- rows behind 4 GB -----------------------------------------------------------
def far_rows(values):
    """The same rows, 4 MB (fp32: 8 MB) apart, NaN between them."""
    M, K = values.shape
    big = torch.full((M - 1, FAR), float("nan"), dtype=values.dtype, device="cuda")
    big = torch.cat([big.view(-1), torch.full((K,), float("nan"), dtype=values.dtype, device="cuda")])
    view = big.as_strided((M, K), (FAR, 1))
    view.copy_(values)
    return view


@pytest.mark.parametrize("M,N", [(1040, 40), (1040, 1040), (5, 1040)])
def test_products_of_far_rows(C, M, N):
    """Rows and outputs that end behind 4 GB, in place (K = 72) and copied (K = 70)."""
    for K in (72, 70):
        banner(f"linear of far rows M={M} N={N} K={K}")
        x, w = test_gpu_linear.rows(M, K, BF16, 1).cuda(), test_gpu_linear.rows(N, K, BF16, 2, 0.1).cuda()
        res = test_gpu_linear.rows(M, N, BF16, 3).cuda()
        want = C.chord_linear(x, w, residual=res)
        out = far_rows(res)
        C.chord_linear(far_rows(x), far_rows(w), residual=out, out=out)
        torch.cuda.synchronize()
        # (sums in the same order, in whatever form: the plan depends on K and the counts alone)
        assert torch.equal(out, want)
        between = out.as_strided((M - 1, 8), (FAR, 1), N)
        assert torch.isnan(between).all()


def test_norms_and_balance_of_far_rows(C):
    T, H = 1040, 200
    banner("norm and balance of far rows")
    n = test_gpu_norm.Part(C, H)
    x, res = test_gpu_norm.rows(T, H, BF16, 1).cuda(), test_gpu_norm.rows(T, H, BF16, 2).cuda()
    gate = test_gpu_norm.rows(T, H, BF16, 3).cuda()
    want = C.chord_norm(x, n.gpu, n.gpu, gate, True, res)
    stream, out = far_rows(res), far_rows(x)
    got = C.chord_norm(out, n.gpu, n.gpu, far_rows(gate), True, stream, sum_out=stream, out=out)
    torch.cuda.synchronize()
    assert torch.equal(got.sum, want.sum) and torch.equal(got.out, want.out)
    assert torch.isnan(stream.as_strided((T - 1, 8), (FAR, 1), H)).all()
    logits, ids = test_gpu_balance.draw(T, 96, 4, 1, BF16)
    logits, ids = logits.cuda(), ids.cuda()
    a = C.chord_moe_balance(logits, ids, n_seq=2, want_grad=True)
    b = C.chord_moe_balance(far_rows(logits), ids, n_seq=2, want_grad=True)
    torch.cuda.synchronize()
    assert torch.equal(a.loss, b.loss) and torch.equal(a.grad, b.grad)


# ---- two streams -------------------------------------------------------------
def test_calls_on_two_streams_at_once(C):
    """Calls with workspaces of their own (K in parts, copies, counts) side by side."""
    banner("two streams")
    x, w = test_gpu_linear.rows(100, 7168, BF16, 1).cuda(), test_gpu_linear.rows(2112, 7168, BF16, 2, 0.01).cuda()
    odd = test_gpu_linear.rows(300, 701, F16, 3).cuda()
    wodd = test_gpu_linear.rows(500, 701, F16, 4, 0.04).cuda()
    logits, ids = test_gpu_balance.draw(3000, 160, 8, 5)
    logits, ids = logits.cuda(), ids.cuda()

    def calls():
        b = C.chord_moe_balance(logits, ids, want_grad=True)
        return [C.chord_linear(x, w), C.chord_linear(odd, wodd, act=C.ACT_RELU), b.loss, b.grad, b.counts,
                C.chord_linear(x, w, gated=True, act=C.ACT_SILU)]
    want = calls()
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for s in sides:
            with torch.cuda.stream(s):
                got.append(calls())
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(p, q) for p, q in zip(g, want))


def test_two_graphs_of_one_pool(C):
    """Two captured graphs whose scratch memory shares a pool, replayed in turn on
    new inputs."""
    banner("two graphs")
    x, w = test_gpu_linear.rows(100, 7168, BF16, 1).cuda(), test_gpu_linear.rows(2112, 7168, BF16, 2, 0.01).cuda()
    logits, ids = test_gpu_balance.draw(3000, 160, 8, 5)
    logits, ids = logits.cuda(), ids.cuda()
    C.chord_linear(x, w)
    C.chord_moe_balance(logits, ids, want_grad=True)
    torch.cuda.synchronize()
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        y = C.chord_linear(x, w)
    with torch.cuda.graph(two, pool=one.pool()):
        b = C.chord_moe_balance(logits, ids, want_grad=True)
        z = C.chord_linear(x, w, act=C.ACT_RELU)
    for seed in range(3):
        x.copy_(test_gpu_linear.rows(100, 7168, BF16, 10 + seed))
        logits.copy_(test_gpu_balance.draw(3000, 160, 8, 20 + seed)[0])
        one.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, C.chord_linear(x, w))
        two.replay()
        torch.cuda.synchronize()
        want = C.chord_moe_balance(logits, ids, want_grad=True)
        assert torch.equal(b.loss, want.loss) and torch.equal(b.grad, want.grad)
        assert torch.equal(z, C.chord_linear(x, w, act=C.ACT_RELU))


@pytest.mark.parametrize("E", [1, 64, 65, 128, 200, 256, 257, 512])
def test_one_workgroup_balances(C, E):
    """Sequences that one workgroup finishes, several threads to an expert: the sums of
    P come from other threads than those that use them."""
    for T in (1, 7, 8, 9, 64):
        logits, ids = test_gpu_balance.draw(T, E, min(E, 3), T + E)
        for sigmoid in (False, True):
            first = test_gpu_balance.check(C, logits.cuda(), ids.cuda(), sigmoid)
            many = [C.chord_moe_balance(logits.cuda(), ids.cuda(), int(sigmoid)) for _ in range(8)]
            torch.cuda.synchronize()
            assert all(torch.equal(m.loss, first.loss) and torch.equal(m.probs, first.probs) for m in many)
