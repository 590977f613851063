"""GPU 8-bit operators against the fp64 oracle (oracle/f8.py, whose header says
how the bounds are made).  Quantisation has to match code for code."""

import numpy as np
import pytest
import torch

from oracle import f8
from tests.gpu_util import banner, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def C():
    from quantized_moe_amd import chord
    return chord


def f64(t):
    return t.detach().double().cpu().numpy()


def activations(T, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, K), generator=g)
    return (x * torch.where(torch.rand(K, generator=g) < 0.02, 10.0, 1.0)).bfloat16()


def weights(E, N, K, seed):
    """Codes [E, N, K] on the host, scales, and the fp64 values."""
    g = torch.Generator().manual_seed(seed)
    codes = (80 * torch.randn((E, N, K), generator=g)).clamp(-448, 448).to(torch.float8_e4m3fn)
    scales = (0.5 + torch.rand((E, -(-N // 128), -(-K // 128)), generator=g)) / (80 * K ** 0.5)
    deq = np.stack([f8.dequantize_weight(f64(codes[e].float()), f64(scales[e])) for e in range(E)])
    return codes, scales, deq


# -- quantise ----------------------------------------------------------------

def check_quantize(C, x, **kw):
    q, s = C.chord_f8_quantize(x, **kw)
    torch.cuda.synchronize()
    v, rs, _ = f8.quantize(f64(x))
    gs = host(s)
    want = rs.astype(np.float32)
    assert np.array_equal(np.isnan(gs), np.isnan(want))
    assert np.array_equal(gs[~np.isnan(gs)], want[~np.isnan(want)])
    assert np.array_equal(f8.decode(host(q.view(torch.uint8))), v)
    return q, s


@pytest.mark.parametrize("T,K", [(1, 1), (1, 128), (3, 127), (5, 136), (17, 129), (64, 7168), (300, 1000),
                                 (2, 20000), (4097, 264)])
def test_quantize_is_exact(C, T, K):
    banner(f"quantize T={T} K={K}")
    check_quantize(C, activations(T, K, T + K).cuda())


def test_quantize_all_ties_and_ranges(C):
    """Every pair of a bf16 maximum and a smaller bf16 fraction, so every quotient
    that lies on a border of two codes; magnitudes up to the largest bf16."""
    fr = torch.arange(128, dtype=torch.float32) / 128 + 1
    for e in (0, -60, 126, -99):
        rows = []
        for top in fr.tolist():
            for lo in range(0, 3):
                row = fr * 2.0 ** (-lo * 4)
                rows.append(torch.cat([torch.tensor([2 * top]), row[1:]]) * 2.0 ** e)
        check_quantize(C, torch.stack(rows).bfloat16().cuda())


def test_quantize_special_values(C):
    x = activations(8, 384, 5).float()
    x[0] = 0
    x[1, :128] = 2.0 ** -101
    x[2, 5], x[3, 200], x[4, 300] = np.inf, -np.inf, np.nan
    x[5, :] = 2.0 ** -100
    x[6, :] *= 1e-44
    x[7, 7] = 3.3e38
    check_quantize(C, x.bfloat16().cuda())


def test_quantize_strided_unaligned_and_out(C):
    x = activations(40, 600, 6).cuda()
    check_quantize(C, x[:, 8:264])            # aligned view
    check_quantize(C, x[:, 3:259])            # rows off by 6 bytes
    check_quantize(C, x[::2, :130])
    q = torch.zeros((42, 640), dtype=torch.uint8, device="cuda").fill_(0x55).view(torch.float8_e4m3fn)
    s = torch.full((42, 5), 7.0, device="cuda")
    check_quantize(C, x, out=(q[1:41], s[1:41]))
    b = host(q.view(torch.uint8))
    assert np.all(b[0] == 0x55) and np.all(b[41] == 0x55) and host(s)[0, 0] == 7.0 and host(s)[41, 4] == 7.0
    q, s = C.chord_f8_quantize(x[:0])
    assert q.shape == (0, 640) and s.shape == (0, 5)


# -- product -----------------------------------------------------------------

def check_gemm(C, M, N, K, seed=1, out=None, x=None):
    codes, scales, deq = weights(1, N, K, seed)
    w = C.chord_f8_pack(C.ROLE_PLAIN, codes.cuda(), scales.cuda())
    x = activations(M, K, seed + 1).cuda() if x is None else x
    q, s = C.chord_f8_quantize(x)
    got = C.chord_f8_gemm(q, s, w, out=out)
    torch.cuda.synchronize()
    a = f8.dequantize(f8.decode(host(q.view(torch.uint8))), f64(s))[:, :K]
    ref, bound = f8.gemm(a, deq[0])
    bound = bound + f8.HALF_BF16 * (np.abs(ref) + bound)
    err = np.abs(f64(got) - ref)
    assert np.all(err <= bound), (float((err / np.maximum(bound, 1e-300)).max()), np.argwhere(err > bound)[:5])
    # over all outputs: half a step of bf16 each (on average 0.6 of that)
    assert np.linalg.norm(err) <= f8.HALF_BF16 * np.linalg.norm(ref)
    return got


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 127, 129, 200, 256, 257, 400])
@pytest.mark.parametrize("N,K", [(256, 512), (300, 200)])
def test_gemm_rows(C, M, N, K):
    banner(f"gemm M={M} N={N} K={K}")
    check_gemm(C, M, N, K)


@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (3, 7, 128), (20, 17, 129), (1, 16, 1), (40, 128, 4096), (9, 2112, 1536), (130, 130, 130),
    (70, 513, 1290), (300, 1000, 384), (515, 776, 640), (1, 4096, 7168), (2000, 96, 256),
    # K in 8, 4 and 6 parts, uneven ones, a ragged last chunk; long rows without
    (200, 520, 4000), (333, 1025, 2500), (120, 2100, 3000), (70, 300, 7168), (700, 2000, 1800),
])
def test_gemm_odd_sizes(C, M, N, K):
    banner(f"gemm M={M} N={N} K={K}")
    check_gemm(C, M, N, K, seed=M + N)


@pytest.mark.parametrize("M,K", [(5, 384), (300, 384), (300, 4096)])
def test_gemm_strided_output_leaves_the_rest(C, M, K):
    for off, ld, N in ((0, 1024, 600), (3, 633, 600), (4, 1024, 512)):
        buf = torch.full((M + 2, ld), 7.0, dtype=torch.bfloat16, device="cuda")
        check_gemm(C, M, N, K, out=buf[1:M + 1, off:off + N])
        b = f64(buf)
        assert np.all(b[0] == 7) and np.all(b[M + 1] == 7)
        assert np.all(b[:, :off] == 7) and np.all(b[:, off + N:] == 7)


def test_gemm_nan_rows_stay_rows(C):
    """A row with a NaN or infinity is NaN throughout and touches no other row."""
    for M in (20, 300):
        x = activations(M, 512, 9)
        x[3, 17], x[M - 1, 500] = float("nan"), float("inf")
        codes, scales, deq = weights(1, 256, 512, 2)
        w = C.chord_f8_pack(C.ROLE_PLAIN, codes.cuda(), scales.cuda())
        got = f64(C.chord_f8_gemm(*C.chord_f8_quantize(x.cuda()), w))
        bad = np.isnan(got)
        assert bad[3].all() and bad[M - 1].all()
        assert not np.delete(bad, [3, M - 1], axis=0).any()


def test_gemm_random_sizes(C):
    rng = np.random.default_rng(11)
    for _ in range(25):
        M, N, K = (int(np.exp(rng.uniform(np.log(lo), np.log(hi)))) for lo, hi in ((1, 1500), (1, 1500), (1, 3000)))
        banner(f"gemm random M={M} N={N} K={K}")
        check_gemm(C, M, N, K, seed=M)


def test_gemm_workspace_and_graphs(C):
    """A product with K in parts: its workspace is checked, two streams at once and
    graphs that replay in turn equal the eager call."""
    M, N, K = 200, 520, 4000
    codes, scales, _ = weights(1, N, K, 6)
    w = C.chord_f8_pack(C.ROLE_PLAIN, codes.cuda(), scales.cuda())
    sets = [C.chord_f8_quantize(activations(M, K, s).cuda()) for s in (1, 2)]
    need = C.chord_f8_gemm_workspace_bytes(M, N, K)
    assert need > 0
    with pytest.raises(C.ChordError):
        C.chord_f8_gemm(*sets[0], w, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    want = [C.chord_f8_gemm(*a, w, workspace=torch.empty(need, dtype=torch.uint8, device="cuda")) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = [C.chord_f8_gemm(*a, w, stream=s) for a, s in zip(sets, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for a in sets:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(C.chord_f8_gemm(*a, w))
        graphs.append(gr)
    for rep in range(3):
        for i in (0, 1):
            for dst, src in zip(sets[i], C.chord_f8_quantize(activations(M, K, 30 + 2 * rep + i).cuda())):
                dst.copy_(src)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        again = [C.chord_f8_gemm(*a, w) for a in sets]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, again))


def test_linear_module_and_empty(C):
    from quantized_moe_amd.moe import F8Linear
    codes, scales, deq = weights(1, 192, 320, 3)
    lin = F8Linear(codes[0].cuda(), scales[0].cuda())
    x = activations(11, 320, 4).cuda()
    q, s = C.chord_f8_quantize(x)
    assert torch.equal(lin(x), C.chord_f8_gemm(q, s, lin.w))
    assert lin(x[:0]).shape == (0, 192)
    with pytest.raises(C.ChordError):
        lin(x[:, :319])


# -- layer ---------------------------------------------------------------------

def make_layer(E, H, I, seed):
    from quantized_moe_amd.moe import W8A8MoE
    c13, s13, d13 = weights(E, 2 * I, H, seed)
    c2, s2, d2 = weights(E, H, I, seed + 50)
    return W8A8MoE(c13.cuda(), s13.cuda(), c2.cuda(), s2.cuda()), d13, d2


def routing(T, E_g, k, seed, hot=0):
    rng = np.random.default_rng(seed)
    p = np.ones(E_g)
    p[:hot] = 60.0
    ids = np.stack([rng.choice(E_g, k, replace=False, p=p / p.sum()) for _ in range(T)]).astype(np.int32)
    w = rng.uniform(0.1, 1.0, (T, k)).astype(np.float32)
    return ids, w / w.sum(axis=1, keepdims=True)


def check_moe(layer, d13, d2, x, ids, w, first, E_g, **kw):
    got = layer.indexed(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), first, E_g, **kw)
    torch.cuda.synchronize()
    ref, bound, norm = f8.moe(f64(x), ids, w, d13, d2, first)
    err = np.abs(f64(got) - ref)
    assert np.all(err <= bound), (float((err / np.maximum(bound, 1e-300)).max()), np.argwhere(err > bound)[:5])
    assert np.linalg.norm(err) <= norm
    none = ~((ids >= first) & (ids < first + layer.E_l)).any(axis=1)
    assert np.all(f64(got)[none] == 0)
    return got


MOE_CASES = [
    # T, H, I, E_g, E_l, k, first, hot
    (1, 256, 128, 8, 8, 2, 0, 0),
    (1, 1024, 256, 64, 64, 8, 0, 0),
    (7, 384, 128, 8, 4, 1, 4, 0),
    (33, 512, 384, 16, 16, 4, 0, 1),
    (64, 1024, 256, 32, 4, 8, 8, 0),
    (100, 256, 512, 4, 2, 2, 1, 0),        # ~50 rows an expert
    (400, 640, 256, 6, 3, 2, 0, 1),        # a hot expert of several tiles
    (700, 256, 256, 8, 8, 3, 0, 0),
    (50, 256, 128, 300, 300, 5, 0, 0),     # mostly one row an expert
    (40, 256, 128, 16, 4, 2, 100, 0),      # no local expert
    (3, 256, 128, 16, 4, 2, 100, 0),       # no local expert, two-launch form
    (16, 256, 128, 2, 2, 2, 0, 0),         # two-launch form, a full tile and a second one
    (4, 2048, 640, 40, 20, 8, 10, 0),      # two-launch form, 32 slots
    (40, 256, 256, 100, 100, 2, 0, 0),     # blocks of 16 rows, K = 256 down
    (70, 256, 128, 8, 8, 2, 0, 0),         # blocks of 32 rows, K = 128 down
    (60, 384, 1152, 5, 5, 1, 0, 0),        # blocks of 32 rows, partial slices
    (200, 128, 2048, 130, 130, 4, 0, 0),   # many blocks of 16 rows
]


@pytest.mark.parametrize("T,H,I,E_g,E_l,k,first,hot", MOE_CASES)
def test_moe_matches_oracle(C, T, H, I, E_g, E_l, k, first, hot):
    banner(f"f8 moe T={T} H={H} I={I} E={E_l}/{E_g} k={k} first={first}")
    layer, d13, d2 = make_layer(E_l, H, I, T)
    ids, w = routing(T, E_g, k, T + 1, hot)
    check_moe(layer, d13, d2, activations(T, H, T + 2), ids, w, first, E_g)
    banner(f"  plan {C.last_plan()}")


def test_moe_repeated_and_foreign_ids(C):
    """The same expert twice in a token, ids of -1 and past the last expert."""
    layer, d13, d2 = make_layer(4, 256, 128, 3)
    ids, w = routing(30, 4, 3, 4)
    ids[0] = [2, 2, 2]
    ids[1] = [-1, 1, 1000]
    ids[2] = -1
    ids[3] = [2**31 - 1, -2**31, 0]
    got = check_moe(layer, d13, d2, activations(30, 256, 5), ids, w, 0, 4)
    assert not f64(got)[2].any()
    T0 = layer.indexed(torch.zeros((0, 256), dtype=torch.bfloat16, device="cuda"),
                       torch.zeros((0, 3), dtype=torch.int32, device="cuda"),
                       torch.zeros((0, 3), device="cuda"), 0, 4)
    assert T0.shape == (0, 256)


@pytest.mark.parametrize("T", [3, 90])
def test_route_and_layers_together(C, T):
    """Router -> W8A8 layer, and the same routing into the W4A16 alignment: as a
    serving step runs them, with experts out of service."""
    layer, d13, d2 = make_layer(16, 512, 256, 8)
    g = torch.Generator().manual_seed(T)
    logits = torch.randn((T, 32), generator=g)
    logits[:, 20:24] = -np.inf
    bias = 0.1 * torch.randn(32, generator=g)
    x = activations(T, 512, 9)
    kw = dict(scoring=C.SCORE_SIGMOID, bias=bias.cuda(), n_group=4, topk_group=3, scaling=2.5)
    got = layer.routed(x.cuda(), logits.cuda(), 4, expert_begin=16, **kw)
    torch.cuda.synchronize()
    ids, w = f8.route(logits.double().numpy(), bias.double().numpy(), 4, True, 4, 3, True, 2.5)
    ref, bound, norm = f8.moe(f64(x), ids, w.astype(np.float32), d13, d2, 16)
    bound = bound + 48 * 2.0 ** -24 * (np.abs(ref) + bound)   # of the router's weights
    assert np.all(np.abs(f64(got) - ref) <= bound)
    assert np.linalg.norm(f64(got) - ref) <= norm
    gi, gw = C.chord_moe_route(logits.cuda(), 4, **kw)
    s, e, n = C.chord_moe_align(gi, 16, 16, 16)
    torch.cuda.synchronize()
    local = np.sort(np.nonzero((ids.reshape(-1) >= 16))[0])
    s = host(s)
    assert np.array_equal(np.sort(s[s < T * 4]), local)


@pytest.mark.parametrize("T", [5, 40, 120])
def test_moe_streams_and_graphs(C, T):
    """One layer on two streams at once, and captured in two graphs that replay
    in turn with eager calls between: all equal to the eager call."""
    layer, d13, d2 = make_layer(8, 512, 256, 11)
    def inputs(seed):
        ids, w = routing(T, 8, 2, seed)
        return activations(T, 512, seed).cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    sets = [inputs(s) for s in (1, 2)]
    want = [layer.indexed(*a, 0, 8) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = [layer.indexed(*a, 0, 8, stream=s) for a, s in zip(sets, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for a in sets:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(layer.indexed(*a, 0, 8))
        graphs.append(gr)
    for rep in range(3):
        for i in (0, 1):
            new = inputs(20 + 2 * rep + i)
            for dst, src in zip(sets[i], new):
                dst.copy_(src)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        again = [layer.indexed(*a, 0, 8) for a in sets]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, again))


@pytest.mark.parametrize("T,E", [(3, 4), (30, 40), (60, 8), (200, 4)])
def test_moe_nan_tokens_stay_tokens(C, T, E):
    layer, _, _ = make_layer(E, 512, 384, 13)
    x = activations(T, 512, 2)
    ids, w = routing(T, E, 2, 3)
    args = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), 0, E
    want = f64(layer.indexed(x.cuda(), *args))
    x[1, 100], x[T - 1, 511] = float("nan"), float("-inf")
    got = f64(layer.indexed(x.cuda(), *args))
    assert np.isnan(got[1]).all() and np.isnan(got[T - 1]).all()
    keep = np.delete(np.arange(T), [1, T - 1])
    assert np.array_equal(got[keep], want[keep])


def test_moe_extreme_values(C):
    """Tokens of zeros, and weights so small or large that h and y leave bf16's and
    fp16's comfortable range: zero stays zero, magnitudes are kept."""
    from quantized_moe_amd.moe import W8A8MoE
    for T, E in ((4, 4), (100, 2)):
        for size in (1e-8, 1e8):
            c13, s13, _ = weights(E, 256, 256, 4)
            c2, s2, _ = weights(E, 256, 128, 5)
            layer = W8A8MoE(c13.cuda(), s13.cuda(), c2.cuda(), (s2 * size).cuda())
            d13 = np.stack([f8.dequantize_weight(f64(c13[e].float()), f64(s13[e])) for e in range(E)])
            d2 = np.stack([f8.dequantize_weight(f64(c2[e].float()), f64((s2 * size)[e])) for e in range(E)])
            ids, w = routing(T, E, 2, 6)
            x = activations(T, 256, 7)
            x[2] = 0
            got = check_moe(layer, d13, d2, x, ids, w, 0, E)
            assert not f64(got)[2].any()


def test_moe_refused_tensors(C):
    layer, _, _ = make_layer(2, 256, 128, 12)
    x = activations(4, 256, 1).cuda()
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    w = torch.ones((4, 2), device="cuda")
    for bad in (dict(x=x.float()), dict(x=x[:, :128]), dict(x=x.t()), dict(ids=ids.long()), dict(ids=ids[:3]),
                dict(w=w.double()), dict(w=w.cpu()), dict(out=x[:3]),
                dict(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))):
        a = dict(x=x, ids=ids, w=w)
        a.update(bad)
        with pytest.raises(C.ChordError):
            layer.indexed(a.pop("x"), a.pop("ids"), a.pop("w"), **a)


# -- chunks behind the tile kernel's loop of four --------------------------------

def cold_calls(run, n=6):
    """Results of n calls, each after its inputs were pushed out of the caches by
    0.5 GB of other work that is still running when the call is queued."""
    junk = torch.empty(1 << 27, device="cuda")
    outs = []
    for i in range(n):
        junk.fill_(i)
        outs.append(run())
    torch.cuda.synchronize()
    return outs


@pytest.mark.parametrize("M", [40, 64, 100, 160, 200, 256])
@pytest.mark.parametrize("K", [7168, 6656, 1664, 1152, 384, 640])
def test_gemm_chunks_behind_the_loop(C, M, K):
    """1, 2 and 3 chunks behind the loop, of every part of K and tile height: the
    tokens' copies into shared memory are waited for there too."""
    N = 1056
    codes, scales, deq = weights(1, N, K, M + K)
    w = C.chord_f8_pack(C.ROLE_PLAIN, codes.cuda(), scales.cuda())
    q, s = C.chord_f8_quantize(activations(M, K, M).cuda())
    a = f8.dequantize(f8.decode(host(q.view(torch.uint8))), f64(s))[:, :K]
    ref, bound = f8.gemm(a, deq[0])
    bound = bound + f8.HALF_BF16 * (np.abs(ref) + bound)
    for got in cold_calls(lambda: C.chord_f8_gemm(q, s, w)):
        assert np.all(np.abs(f64(got) - ref) <= bound)


@pytest.mark.parametrize("T,E,k,H,I", [
    (70, 16, 2, 640, 384), (70, 16, 2, 768, 640), (60, 40, 4, 896, 768), (300, 4, 2, 640, 896),
    (300, 4, 2, 1792, 640), (400, 4, 1, 768, 768), (150, 2, 2, 384, 1152),
])
def test_moe_chunks_behind_the_loop(C, T, E, k, H, I):
    layer, d13, d2 = make_layer(E, H, I, T + H)
    ids, w = routing(T, E, k, I)
    x = activations(T, H, 3)
    ref, bound, norm = f8.moe(f64(x), ids, w, d13, d2, 0)
    xg, ig, wg = x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    for got in cold_calls(lambda: layer.indexed(xg, ig, wg, 0, E)):
        err = np.abs(f64(got) - ref)
        assert np.all(err <= bound) and np.linalg.norm(err) <= norm


TILED_CASES = [
    # T, H, I, E, k, hot, plan; chunks 1 .. 7 of both products, partial slices,
    # experts from one row to several tiles
    (120, 640, 384, 90, 4, 0, "blocks of 16 rows"),
    (150, 768, 896, 60, 3, 0, "blocks of 16 rows"),
    (90, 896, 256, 100, 4, 0, "blocks of 16 rows"),
    (300, 384, 256, 50, 2, 0, "blocks of 32 rows"),
    (330, 640, 128, 50, 3, 0, "blocks of 16 rows, streaming gate_up"),
    (450, 640, 128, 70, 3, 0, "blocks of 32 rows"),
    (120, 896, 1152, 10, 1, 0, "blocks of 32 rows"),
    (230, 768, 640, 24, 2, 0, "blocks of 32 rows"),
    (420, 640, 768, 16, 2, 0, "blocks of 32 rows"),
    (800, 384, 768, 16, 2, 0, "tiles of up to 224 rows"),
    (1000, 640, 640, 18, 2, 2, "tiles of up to 224 rows"),
    (1500, 768, 384, 30, 2, 0, "tiles of up to 224 rows"),
    (1400, 896, 896, 12, 1, 1, "tiles of up to 224 rows"),
    (1900, 512, 640, 10, 2, 0, "tiles of up to 224 rows"),
    (900, 128, 1152, 20, 1, 1, "tiles of up to 224 rows"),
]


@pytest.mark.parametrize("T,H,I,E,k,hot,plan", TILED_CASES)
def test_moe_tiled_forms(C, T, H, I, E, k, hot, plan):
    """The forms of larger layers, inputs cold, results repeatable bit for bit."""
    banner(f"f8 moe T={T} H={H} I={I} E={E} k={k} hot={hot}")
    layer, d13, d2 = make_layer(E, H, I, T + E)
    ids, w = routing(T, E, k, I + T, hot)
    x = activations(T, H, 3)
    ref, bound, norm = f8.moe(f64(x), ids, w, d13, d2, 0)
    xg, ig, wg = x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    outs = cold_calls(lambda: layer.indexed(xg, ig, wg, 0, E), 4)
    assert C.last_plan() == "f8 moe: " + plan
    err = np.abs(f64(outs[0]) - ref)
    assert np.all(err <= bound) and np.linalg.norm(err) <= norm
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_moe_tiled_forms_with_nan_and_foreign_rows(C):
    """Tokens of NaN, of foreign experts only and with an expert twice, in layers
    whose tiles hold them beside ordinary ones."""
    for T, E, k, I in ((150, 60, 3, 896), (420, 16, 2, 768), (800, 16, 2, 768)):
        layer, d13, d2 = make_layer(E, 384, I, T)
        ids, w = routing(T, E, k, T)
        ids[5], ids[6] = E + 3, ids[6][0]
        x = activations(T, 384, 3)
        ref, bound, _ = f8.moe(f64(x), ids, w, d13, d2, 0)
        x[7, 11] = np.nan
        got = f64(layer.indexed(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), 0, E))
        assert np.isnan(got[7]).all() and not got[5].any()
        rest = np.arange(T) != 7
        assert np.all(np.abs(got - ref)[rest] <= bound[rest])


@pytest.mark.parametrize("T,H,I,E,k", [(1, 2048, 512, 64, 8), (7, 1024, 1024, 8, 4), (12, 2048, 512, 8, 4),
                                       (40, 2048, 256, 16, 2), (120, 1024, 384, 90, 4)])
def test_moe_rows_of_few_are_as_exact_as_bf16(C, T, H, I, E, k):
    """Layers of few rows sum gate_up in fp32, so a code of h differs from the
    oracle's only on a border, and without one a row's error is that of its rounding
    to bf16: half a step at every value at worst, so half a step of the row's norm.

    Borders: h is off by about 2e-6 of itself (2^-24 for sqrt(K) sums, a few of
    them cancelled), codes lie 1/16 to 1/8 apart, so 2 * 2e-6 * 16 = 6e-5 of the
    values may take the other code; one of them shows in its row only if it is
    more than 16 * 0.0035 = 0.06 of the row's norm, a tenth of the values at I =
    256.  With k * I <= 1536 values a row that is below 1 % of the rows (with sums
    on a grid of 2^-13, a hundred times as far off, it would be every few rows)."""
    layer, d13, d2 = make_layer(E, H, I, 7 * T)
    over = 0
    for seed in range(3):
        ids, w = routing(T, E, k, T + seed)
        x = activations(T, H, seed)
        ref, _, _ = f8.moe(f64(x), ids, w, d13, d2, 0)
        got = layer.indexed(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), 0, E)
        err = np.linalg.norm(f64(got) - ref, axis=1)
        over += int((err > f8.HALF_BF16 * np.linalg.norm(ref, axis=1)).sum())
    assert over <= max(1, 3 * T // 100), (over, C.last_plan())
