"""GPU 16-bit product against the fp64 oracle (oracle/block.py, whose header says
how the bounds are made).  Beside the bound at every value the error over all
outputs is held to that of its roundings: half a step of the output's type each, and
sqrt(K) roundings of fp32 sums that are no larger than the outputs by much."""

import numpy as np
import pytest
import torch

from oracle import block as B
from tests.gpu_util import banner

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module")
def C():
    from quantized_moe_amd import chord
    return chord


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def rows(M, K, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn((M, K), generator=g)).to(dtype)


def check(C, M, N, K, dtype=BF16, out=None, act="none", gated=False, bias=None, residual=False, scale=1.0, x=None,
          w=None, **kw):
    banner(f"linear M={M} N={N} K={K} {dtype} out={out} {act} gated={gated} bias={bias} residual={residual}")
    out = out or dtype
    R = 2 * N if gated else N
    x = rows(M, K, dtype, M + K).cuda() if x is None else x
    w = rows(R, K, dtype, N, K ** -0.5).cuda() if w is None else w
    b = rows(1, R, bias, 5, 0.5)[0].cuda() if bias else None
    r = rows(M, N, out, 6).cuda() if residual else None
    got = C.chord_linear(x, w, b, getattr(C, "ACT_" + act.upper()), gated, scale, r, out_dtype=out, **kw)
    torch.cuda.synchronize()
    assert got.shape == (M, N) and got.dtype is out
    ref, bound = B.linear(f64(x), f64(w), f64(b), act, gated, float(np.float32(scale)), f64(r))
    name = str(out).replace("torch.", "")
    bound = bound + B.rounding(np.abs(ref) + bound, name)
    err = np.abs(f64(got) - ref)
    assert np.all(err <= bound), (float((err / bound).max()), np.argwhere(err > bound)[:5])
    if M * N >= 1000:
        size = np.linalg.norm(ref)
        assert np.linalg.norm(err) <= (B.HALF[name] + 4 * K ** 0.5 * B.U32) * size, np.linalg.norm(err) / size
    return got


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 31, 33, 64, 65, 100, 128, 129, 200, 256, 257, 400])
@pytest.mark.parametrize("N,K,gated", [(256, 512, False), (300, 200, False), (136, 448, True)])
def test_rows(C, M, N, K, gated):
    check(C, M, N, K, gated=gated, act="silu" if gated else "none", residual=M % 2 == 1, bias=BF16 if M % 3 else None)


@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (3, 7, 128), (20, 17, 129), (1, 16, 1), (40, 128, 4096), (9, 2112, 1536), (130, 130, 130),
    (70, 513, 1290), (300, 1000, 384), (515, 776, 640), (1, 4096, 7168), (2000, 96, 256), (64, 384, 7168),
    (200, 520, 4000), (333, 1025, 2500), (120, 2100, 2900), (70, 300, 7168), (700, 2000, 1800), (1000, 8, 8),
    (5, 4000, 24), (257, 257, 72), (513, 640, 8), (1, 50, 7000), (17, 40, 6152), (900, 1100, 104),
])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_odd_sizes(C, M, N, K, dtype):
    check(C, M, N, K, dtype)
    check(C, M, N, K, dtype, out=F32, bias=F32, residual=True, scale=0.75)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N,K", [(5, 200, 512), (300, 392, 512), (70, 37, 100)])
def test_epilogues(C, act, gated, M, N, K):
    for dtype, out, bias, residual in ((BF16, BF16, F32, True), (F16, F32, F16, False), (BF16, F32, BF16, True)):
        check(C, M, N, K, dtype, out, act, gated, bias, residual, -1.5)


def test_steep_activations(C):
    """Values far out on both sides: results that vanish keep their relative error,
    large ones pass."""
    K = 64
    x = torch.zeros((40, K), dtype=BF16)
    x[:, 0] = torch.linspace(-40, 40, 40).to(BF16)
    w = torch.zeros((48, K), dtype=BF16)
    w[:, 0] = torch.linspace(0.05, 4, 48).to(BF16)
    for act in ACTS:
        check(C, 40, 48, K, act=act, out=F32, x=x.cuda(), w=w.cuda())


@pytest.mark.parametrize("M", [3, 40, 300])
def test_infinities_and_nan_stay_in_their_rows(C, M):
    N, K = 200, 200
    x, w = rows(M, K, BF16, 1), rows(N, K, BF16, 2, 0.07)
    clean = C.chord_linear(x.cuda(), w.cuda())
    x2, w2 = x.clone(), w.clone()
    x2[1, K - 1], x2[2, 0] = np.inf, np.nan
    w2[7, K - 1], w2[9, 3] = np.nan, -np.inf
    got = C.chord_linear(x2.cuda(), w2.cuda())
    m, n = np.ones(M, bool), np.ones(N, bool)
    m[1:3] = False
    n[[7, 9]] = False
    g, c = f64(got), f64(clean)
    assert np.array_equal(g[np.ix_(m, n)], c[np.ix_(m, n)])
    assert not np.isfinite(g[1]).any() and np.isnan(g[2]).all() and np.isnan(g[:, 7]).all()
    assert not np.isfinite(g[:, 9]).any()


@pytest.mark.parametrize("M,K", [(5, 384), (300, 384), (64, 4096), (40, 100)])
def test_strides_alignment_and_untouched_columns(C, M, K):
    for off, ld, N in ((0, 1024, 600), (3, 633, 600), (4, 1024, 512)):
        buf = torch.full((M + 2, ld), 7.0, dtype=BF16, device="cuda")
        big, wig = rows(M, K + 40, BF16, 3).cuda(), rows(N, K + 24, BF16, 4, K ** -0.5).cuda()
        for xo, wo in ((0, 0), (8, 16), (5, 0), (0, 3)):
            check(C, M, N, K, x=big[:, xo:xo + K], w=wig[:, wo:wo + K], act="silu", bias=BF16, residual=True) \
                if off == 0 else None
        x, w = big[:, :K], wig[:, :K]
        view = buf[1:M + 1, off:off + N]
        C.chord_linear(x, w, out=view)
        torch.cuda.synchronize()
        assert torch.equal(view, C.chord_linear(x.contiguous(), w.contiguous()))
        b = f64(buf)
        assert np.all(b[0] == 7) and np.all(b[M + 1] == 7) and np.all(b[:, :off] == 7) and np.all(b[:, off + N:] == 7)
        # the residual in the output's place
        want = C.chord_linear(x, w, residual=view, scale=0.5)
        C.chord_linear(x, w, residual=view, scale=0.5, out=view)
        torch.cuda.synchronize()
        assert torch.equal(view, want)


@pytest.mark.parametrize("M,N,K", [(1, 384, 7168), (64, 384, 7168), (100, 2110, 4000), (300, 520, 2048), (600, 900, 520)])
def test_equal_calls_equal_bits_streams_and_graphs(C, M, N, K):
    x, w = rows(M, K, BF16, 7).cuda(), rows(N, K, BF16, 8, K ** -0.5).cuda()
    res = rows(M, N, BF16, 9).cuda()
    want = C.chord_linear(x, w, act=C.ACT_SILU, residual=res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [C.chord_linear(x, w, act=C.ACT_SILU, residual=res, stream=side) for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(C.chord_linear(x, w, act=C.ACT_SILU, residual=res))
    for seed in range(3):
        x.copy_(rows(M, K, BF16, 40 + seed))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = C.chord_linear(x, w, act=C.ACT_SILU, residual=res)
        assert all(torch.equal(o, want) for o in outs)


def test_given_workspace_and_nothing(C):
    x, w = rows(40, 100, BF16, 1).cuda(), rows(64, 100, BF16, 2).cuda()
    need = C.chord_linear_workspace_bytes(x, w)
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    assert torch.equal(C.chord_linear(x, w, workspace=ws[:max(need, 1)]), C.chord_linear(x, w))
    if need:
        with pytest.raises(C.ChordError):
            C.chord_linear(x, w, workspace=ws[:need - 1])
        with pytest.raises(C.ChordError):
            C.chord_linear(x, w, workspace=ws[8:8 + need])
    assert C.chord_linear(x[:0], w).shape == (0, 64)


def test_refusals(C):
    x, w = rows(4, 64, BF16, 1).cuda(), rows(6, 64, BF16, 2).cuda()
    for kw in (dict(w=w.half()), dict(w=w[:, :32]), dict(w=w[:5], gated=True), dict(bias=x[0]), dict(bias=w[:, 0].half()),
               dict(residual=x[:, :6].float()), dict(residual=x[:, :5]), dict(out_dtype=F16), dict(act=7),
               dict(out=torch.empty((4, 5), dtype=BF16, device="cuda")), dict(w=w.cpu()), dict(scale=float("inf"))):
        with pytest.raises(C.ChordError):
            C.chord_linear(x, **{"w": w, **kw})
    for bad in (x.float(), x.t()):
        with pytest.raises(C.ChordError):
            C.chord_linear(bad, w)
