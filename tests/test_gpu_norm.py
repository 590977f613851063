"""GPU norms against the fp64 oracle (oracle/block.py, whose header says how the
bounds are made).  Codes are compared as the values they stand for: within half a
step of e4m3 of them and of their scale, beside what y itself may be off."""

import numpy as np
import pytest
import torch

from oracle import block as B
from oracle import f8
from tests.gpu_util import banner, host

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def C():
    from quantized_moe_amd import chord
    return chord


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def name(dtype):
    return str(dtype).replace("torch.", "")


class Part:
    """A norm's weights, on the GPU and for the oracle."""

    def __init__(self, C, H, kind="rms", dtype=BF16, bias=False, eps=1e-6, offset=0.0, seed=0):
        g = torch.Generator().manual_seed(1000 + seed)
        w = (1 - offset + 0.2 * torch.randn(H, generator=g)).to(dtype)
        b = (0.3 * torch.randn(H, generator=g)).to(dtype) if bias else None
        self.gpu = C.Norm(w.cuda(), None if b is None else b.cuda(), eps,
                          C.NORM_RMS if kind == "rms" else C.NORM_LAYER, offset)
        eps32, offset32 = float(np.float32(eps)), float(np.float32(offset))
        self.args = (f64(w), f64(b), kind, eps32, offset32)


def rows(T, H, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H), generator=g) * torch.where(torch.rand(H, generator=g) < 0.02, 10.0, 1.0)
    return (scale * x + 0.3).to(dtype)


def close(got, ref, bound, dtype, what):
    got = f64(got)
    bad = ~(np.abs(got - ref) <= bound + B.rounding(np.abs(ref) + bound, name(dtype)))
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])


def check(C, x, pre=None, post=None, gate=None, sigmoid=False, residual=None, scale=1.0, stream=None, codes=False,
          out=True, **kw):
    r = C.chord_norm(x, pre=pre and pre.gpu, post=post and post.gpu, gate=gate, gate_sigmoid=sigmoid,
                     residual=residual, scale=scale, sum_dtype=stream, want_out=out, want_codes=codes, **kw)
    torch.cuda.synchronize()
    g = f64(gate)
    if g is not None and g.ndim == 1:
        g = g[None, :]
    s, es, y, ey = B.block_norm(f64(x), post and post.args, g, sigmoid, f64(residual), float(np.float32(scale)),
                                pre and pre.args)
    stream = residual.dtype if residual is not None else stream or x.dtype
    if r.sum is not None:
        assert r.sum.dtype is stream
        close(r.sum, s, es, stream, "sum")
    if r.out is not None:
        assert r.out.dtype is x.dtype
        close(r.out, y, ey, x.dtype, "out")
    if codes:
        check_codes(r.codes, r.scales, y, ey)
    return r


def check_codes(codes, scales, y, ey):
    T, H = y.shape
    groups = -(-H // 128)
    pad = ((0, 0), (0, groups * 128 - H))
    y3, e3 = np.pad(y, pad).reshape(T, groups, 128), np.pad(ey, pad).reshape(T, groups, 128)
    top, s = np.abs(y3).max(axis=2), f64(scales)
    # the largest magnitude is off by at most the largest error; the quotient is rounded
    assert np.all(np.abs(s - top / 448) <= e3.max(axis=2) / 448 + 2.0 ** -23 * top / 448)
    v = f8.decode(host(codes.view(torch.uint8))).reshape(T, groups, 128) * s[:, :, None]
    # half a step: 2^-4 of a value, 2^-10 of the scale below the normal codes
    assert np.all(np.abs(v - y3) <= (np.abs(y3) + e3) * 2.0 ** -4 * (1 + 2.0 ** -20) + s[:, :, None] * 2.0 ** -10 + e3)
    assert not v.reshape(T, -1)[:, H:].any()


@pytest.mark.parametrize("T,H", [(1, 1), (1, 7168), (3, 7), (2, 8), (5, 64), (4, 127), (7, 513), (6, 520), (5, 1000),
                                 (9, 2048), (3, 2056), (2, 4104), (3, 8192), (2, 8200), (2, 20001), (1, 32768),
                                 (300, 7168), (4097, 264)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_in_front(C, T, H, dtype):
    banner(f"norm T={T} H={H} {dtype}")
    p = Part(C, H, dtype=dtype if T % 2 else F32)
    check(C, rows(T, H, dtype, T + H).cuda(), p, residual=rows(T, H, dtype, T, 3.0).cuda(), codes=True)
    r = check(C, rows(T, H, dtype, T + H).cuda(), p)
    assert r.sum is None and r.codes is None


CASES = [
    # kind, bias, post, gate, sigmoid, residual, stream, offset
    ("rms", False, True, "token", True, True, None, 0.0),
    ("layer", True, True, "column", False, True, F32, 0.0),
    ("layer", False, False, "full", True, True, None, 1.0),
    ("rms", True, True, "full", False, False, F32, 1.0),
    ("rms", False, False, "token", False, False, None, 0.0),
    ("layer", True, True, None, False, False, None, 0.0),
]


@pytest.mark.parametrize("kind,bias,post,gate,sigmoid,residual,stream,offset", CASES)
@pytest.mark.parametrize("T,H,dtype", [(33, 7168, BF16), (5, 515, F16), (130, 384, BF16), (3, 9000, F32)])
def test_between_blocks(C, T, H, dtype, kind, bias, post, gate, sigmoid, residual, stream, offset):
    pre = Part(C, H, kind, F32 if bias else dtype, bias, 1e-5, offset, 1)
    behind = Part(C, H, kind, dtype, bias, 1e-6, offset, 2) if post else None
    g = None
    if gate:
        g = rows(T, H, dtype, 5)[:, :1] if gate == "token" else rows(T, H, dtype, 5)
        g = (g[0] if gate == "column" else g).contiguous().cuda()
    res = rows(T, H, stream or dtype, 6, 2.0).cuda() if residual else None
    r = check(C, rows(T, H, dtype, 7).cuda(), pre, behind, g, sigmoid, res, 0.37, stream, codes=True)
    assert r.sum is not None
    # The sum alone, and the codes alone, are the same values.
    alone = C.chord_norm(rows(T, H, dtype, 7).cuda(), post=behind and behind.gpu, gate=g, gate_sigmoid=sigmoid,
                         residual=res, scale=0.37, sum_dtype=stream)
    assert torch.equal(alone.sum, r.sum) and alone.out is None
    only = C.chord_norm(rows(T, H, dtype, 7).cuda(), pre.gpu, behind and behind.gpu, g, sigmoid, res, 0.37, stream,
                        want_sum=False, want_out=False, want_codes=True)
    assert torch.equal(only.codes.view(torch.uint8), r.codes.view(torch.uint8)) and torch.equal(only.scales, r.scales)
    assert only.sum is None and only.out is None


def test_gate_and_residual_without_a_norm(C):
    x, res = rows(9, 640, BF16, 1).cuda(), rows(9, 640, F32, 2).cuda()
    r = check(C, x, gate=rows(9, 640, F32, 3)[:, 5:6].cuda(), sigmoid=True, residual=res, scale=2.0)
    assert r.out is None


def test_strided_unaligned_and_in_place(C):
    T, H = 21, 600
    p = Part(C, H)
    big = rows(T, 1400, BF16, 11).cuda()
    for off, ld in ((0, 1400), (8, 1400), (3, 1400)):
        x = big[:, off:off + H]
        res = rows(T, 1333, BF16, 12).cuda()[:, 7:7 + H]
        buf = torch.full((T + 2, 1216), 7.0, dtype=BF16, device="cuda")
        sums = torch.full((T + 2, 1216), 9.0, dtype=BF16, device="cuda")
        check(C, x, p, residual=res, out=buf[1:T + 1, off:off + H], sum_out=sums[1:T + 1, off:off + H])
        for t, fill in ((buf, 7.0), (sums, 9.0)):
            b = f64(t)
            assert np.all(b[0] == fill) and np.all(b[T + 1] == fill)
            assert np.all(b[:, :off] == fill) and np.all(b[:, off + H:] == fill)
    # in place: the sum onto the residual, the normed rows onto x
    x, res = rows(T, H, BF16, 13).cuda(), rows(T, H, BF16, 14).cuda()
    want = C.chord_norm(x, p.gpu, residual=res)
    got = C.chord_norm(x, p.gpu, residual=res, sum_out=res, out=x)
    torch.cuda.synchronize()
    assert torch.equal(got.sum, want.sum) and torch.equal(got.out, want.out)
    assert got.sum.data_ptr() == res.data_ptr() and got.out.data_ptr() == x.data_ptr()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("H", [384, 5000])
def test_extreme_rows(C, kind, H):
    """Rows of zeros, of magnitudes whose squares leave fp32 either way, of one value;
    rows with an infinity or NaN, which leave the others alone."""
    x = rows(10, H, F32, 15)
    x[0] = 0
    x[1] *= 1e30
    x[2] *= 1e-30
    x[3] = 2.5
    x[4, 3], x[5, 7], x[6, 9] = np.inf, -np.inf, np.nan
    x[7] = 3e38 * torch.sign(x[7])
    x[8] = 0
    x[8, 1] = 3e38
    x = x.to(BF16)
    p = Part(C, H, kind, bias=kind == "layer")
    r = C.chord_norm(x.cuda(), p.gpu, want_codes=True)
    got = f64(r.out)
    good = [0, 1, 2, 3, 7, 8, 9]
    y, ey = B.norm(f64(x)[good], *p.args), B.norm_bound(f64(x)[good], np.zeros((7, H)), *p.args)
    close(r.out[good], y, ey, BF16, "rows")
    check_codes(r.codes[good], r.scales[good], y, ey)
    for t in (4, 5, 6):  # inf / inf in the place of the infinity, what the formula gives elsewhere
        assert np.isnan(got[t, {4: 3, 5: 7, 6: 9}[t]])
        assert np.isnan(f64(r.scales)[t]).any()
    if kind == "rms":
        assert np.all(got[4, 4:] == 0) and np.isnan(got[6]).all()
    assert np.isfinite(got[good]).all()


def test_codes_feed_the_product(C):
    """The quantised product takes the codes in the place of chord_f8_quantize's."""
    g = torch.Generator().manual_seed(3)
    H, N, T = 1000, 96, 40
    p = Part(C, H)
    codes = (80 * torch.randn((1, N, H), generator=g)).clamp(-448, 448).to(torch.float8_e4m3fn)
    w = C.chord_f8_pack(C.ROLE_PLAIN, codes.cuda(), torch.ones((1, 1, 8), device="cuda"))
    r = C.chord_norm(rows(T, H, BF16, 4).cuda(), p.gpu, want_codes=True, want_out=False)
    got = f64(C.chord_f8_gemm(r.codes, r.scales, w))
    a = f8.dequantize(f8.decode(host(r.codes.view(torch.uint8))), f64(r.scales))[:, :H]
    ref, bound = f8.gemm(a, f64(codes[0].float()))
    assert np.all(np.abs(got - ref) <= bound + f8.HALF_BF16 * (np.abs(ref) + bound))


def test_streams_graphs_and_nothing(C):
    T, H = 64, 1024
    p, q = Part(C, H), Part(C, H, seed=3)
    x, res = rows(T, H, BF16, 21).cuda(), rows(T, H, BF16, 22).cuda()
    want = C.chord_norm(x, p.gpu, q.gpu, residual=res, want_codes=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = C.chord_norm(x, p.gpu, q.gpu, residual=res, want_codes=True, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got.out, want.out) and torch.equal(got.sum, want.sum)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = C.chord_norm(x, p.gpu, q.gpu, residual=res, want_codes=True)
    for seed in range(3):
        x.copy_(rows(T, H, BF16, 30 + seed))
        graph.replay()
        torch.cuda.synchronize()
        e = C.chord_norm(x, p.gpu, q.gpu, residual=res, want_codes=True)
        assert torch.equal(r.out, e.out) and torch.equal(r.sum, e.sum) and torch.equal(r.scales, e.scales)
        assert torch.equal(r.codes.view(torch.uint8), e.codes.view(torch.uint8))
    r = C.chord_norm(x[:0], p.gpu, residual=res[:0], want_codes=True)
    assert r.out.shape == (0, H) and r.codes.shape == (0, H) and r.scales.shape == (0, 8)


def test_refusals(C):
    p = Part(C, 64)
    x = rows(4, 64, BF16, 1).cuda()
    bad = [dict(pre=Part(C, 72).gpu), dict(pre=p.gpu, residual=x.half()), dict(pre=p.gpu, residual=x[:3]),
           dict(pre=p.gpu, gate=x[:, :3]), dict(pre=p.gpu, gate=x.int()), dict(pre=p.gpu, sum_dtype=F16),
           dict(pre=p.gpu, residual=x, sum_dtype=F32), dict(pre=p.weight if hasattr(p, "weight") else x),
           dict(out=x.clone()), dict(pre=p.gpu, out=x.float()), dict(pre=p.gpu, gate=x.cpu()), dict(want_sum=False),
           dict(pre=p.gpu, gate=x.t()[:, :4].t()[:, :1].expand(4, 64)), dict(pre=p.gpu, want_out=False)]
    for kw in bad:
        with pytest.raises(C.ChordError):
            C.chord_norm(x, **kw)
    with pytest.raises(C.ChordError):
        C.chord_norm(x.t(), p.gpu)
    with pytest.raises(C.ChordError):
        C.chord_norm(x.int(), p.gpu)
