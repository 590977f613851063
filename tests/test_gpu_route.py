"""GPU router against the fp64 oracle: the experts have to be the oracle's, the
weights within fp32 roundings.

Tolerance of a weight: a score is at most two roundings off, a softmax sum of
E terms adds 4 ulp of the exponentials and at most 22 additions in a row, the
renormalising sum 6 additions, and the divisions and the factor 4 more: below
48 x 2^-24 in all.  Underflowed scores are compared absolutely (2^-126).
"""

import numpy as np
import pytest
import torch

from oracle import f8
from tests.gpu_util import banner, host

pytestmark = pytest.mark.gpu

RTOL, ATOL = 48 * 2.0 ** -24, 2.0 ** -126


@pytest.fixture(scope="module")
def C():
    from quantized_moe_amd import chord
    return chord


def check(C, logits, k, bias=None, sigmoid=False, n_group=1, topk_group=1, renorm=True, scaling=1.0, **kw):
    ids, w = C.chord_moe_route(logits, k, scoring=C.SCORE_SIGMOID if sigmoid else C.SCORE_SOFTMAX,
                               bias=bias, n_group=n_group, topk_group=topk_group, renormalize=renorm,
                               scaling=scaling, **kw)
    torch.cuda.synchronize()
    ri, rw = f8.route(logits.double().cpu().numpy(), None if bias is None else bias.double().cpu().numpy(),
                      k, sigmoid, n_group, topk_group, renorm, scaling)
    gi, gw = host(ids), host(w).astype(np.float64)
    assert np.array_equal(gi, ri), f"rows {np.nonzero((gi != ri).any(1))[0][:5]}"
    assert np.all(np.abs(gw - rw) <= RTOL * np.abs(rw) + ATOL), np.abs(gw - rw).max()
    return gi, gw


CASES = [
    # T, E, k, sigmoid, bias, n_group, topk_group, dtype
    (1, 384, 8, False, False, 1, 1, torch.float32),
    (1, 1, 1, False, True, 1, 1, torch.float32),
    (5, 7, 7, True, True, 1, 1, torch.float32),          # k == E
    (65, 64, 6, False, True, 1, 1, torch.bfloat16),
    (33, 65, 8, True, False, 1, 1, torch.float16),       # one expert in a lane's second place
    (200, 256, 8, True, True, 8, 4, torch.float32),
    (200, 256, 8, True, True, 8, 4, torch.bfloat16),
    (100, 384, 8, True, True, 1, 1, torch.float32),
    (100, 160, 6, False, False, 8, 3, torch.float32),    # groups of 20, softmax, best expert of a group
    (60, 130, 4, False, True, 13, 5, torch.float32),     # groups that straddle the waves' strides
    (40, 64, 3, True, True, 64, 9, torch.float32),       # groups of one expert
    (30, 1024, 32, True, True, 4, 2, torch.float32),
    (30, 1024, 32, False, False, 1, 1, torch.float32),
    (17, 513, 31, False, True, 1, 1, torch.bfloat16),
]


@pytest.mark.parametrize("T,E,k,sigmoid,bias,n_group,topk_group,dtype", CASES)
@pytest.mark.parametrize("renorm", [True, False])
def test_route_matches_oracle(C, T, E, k, sigmoid, bias, n_group, topk_group, dtype, renorm):
    banner(f"route T={T} E={E} k={k} sigmoid={sigmoid} bias={bias} groups={n_group}/{topk_group} {dtype}")
    g = torch.Generator().manual_seed(T * 7 + E)
    logits = (2 * torch.randn((T, E), generator=g)).to(dtype).cuda()
    b = (0.2 * torch.randn(E, generator=g)).cuda() if bias else None
    check(C, logits, k, b, sigmoid, n_group, topk_group, renorm, 2.5)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("n_group,topk_group", [(1, 1), (4, 2)])
def test_equal_logits_go_to_the_lowest_experts(C, bias, n_group, topk_group):
    """More than 64 candidates tie: with a bias this is the 64-bit path."""
    logits = torch.zeros((3, 256), device="cuda")
    b = torch.full((256,), 0.25, device="cuda") if bias else None
    ids, w = check(C, logits, 8, b, True, n_group, topk_group)
    assert ids.tolist() == [list(range(8))] * 3


def test_neighbours_closer_than_32_bits(C):
    """Choices that differ by 2^-26 and less at 0.5: equal in fp32, ordered in 64
    bits; also in the sums that rank groups."""
    E = 64
    logits = torch.zeros((2, E), device="cuda")
    bias = torch.tensor([2.0 ** -27 * ((e * 37) % E) for e in range(E)], device="cuda")
    ids, _ = check(C, logits, 8, bias, True)
    assert ids[0].tolist() != list(range(8))
    check(C, logits, 8, bias, True, 16, 3)
    check(C, logits, 8, bias, False, 16, 3)


def test_unavailable_experts(C):
    g = torch.Generator().manual_seed(1)
    logits = torch.randn((6, 96), generator=g)
    logits[0] = -np.inf                       # nobody
    logits[1, 3:] = -np.inf                   # fewer than k
    logits[2, ::2] = np.nan
    logits[3, :40] = -np.inf                  # whole groups gone
    logits[4, 5] = np.inf
    bias = torch.zeros(96)
    bias[7], bias[50] = -np.inf, np.nan
    logits, bias = logits.cuda(), bias.cuda()
    for sigmoid in (False, True):
        for b in (None, bias):
            for grp in ((1, 1), (8, 2), (8, 7)):
                banner(f"unavailable sigmoid={sigmoid} bias={b is not None} groups={grp}")
                ids, w = check(C, logits, 6, b, sigmoid, *grp)
                assert np.all(ids[0] == -1) and np.all(w[0] == 0)
                assert np.all(ids[1][3:] == -1)
                if b is not None:
                    assert not np.isin(ids, [7, 50]).any()


def test_large_values(C):
    """Biases that drown the scores, saturated sigmoids, extreme logits."""
    g = torch.Generator().manual_seed(2)
    logits = torch.randn((4, 100), generator=g)
    logits[1] *= 1e4
    logits[2] = 30 + torch.arange(100) * 0.01
    logits = logits.cuda()
    for size in (1e3, 1e9, 3e38, float("inf")):
        bias = torch.randn(100, generator=g)
        bias[::3] = size
        bias[1::3] = -min(size, 3e38)
        for sigmoid in (False, True):
            check(C, logits, 7, bias.cuda(), sigmoid)
            check(C, logits, 7, bias.cuda(), sigmoid, 10, 4)
    check(C, logits, 7, None, True)
    check(C, logits, 7, None, False)


def test_strided_rows_outputs_and_untouched_neighbours(C):
    g = torch.Generator().manual_seed(3)
    wide = torch.randn((20, 100), generator=g).cuda()
    view = wide[:, 3:75]                       # rows 400 bytes apart, not 16-byte aligned
    ids = torch.full((22, 4), 77, dtype=torch.int32, device="cuda")
    w = torch.full((22, 4), 77.0, device="cuda")
    check(C, view, 4, out=(ids[1:21], w[1:21]))
    assert ids[0].tolist() == [77] * 4 and ids[21].tolist() == [77] * 4
    assert w[0].tolist() == [77.0] * 4 and w[21].tolist() == [77.0] * 4


def test_refused_tensors(C):
    x = torch.zeros((4, 64), device="cuda")
    for bad in (dict(logits=x.double()), dict(logits=x.t()), dict(logits=x[0]), dict(bias=x[0].cpu()),
                dict(bias=x[0, :63]), dict(bias=x[0].double()), dict(k=65), dict(k=0),
                dict(logits=x[:1].expand(4, 64)),
                dict(out=(torch.zeros((4, 2), device="cuda"), torch.zeros((4, 2), device="cuda")))):
        a = dict(logits=x, k=2)
        a.update(bad)
        with pytest.raises(C.ChordError):
            C.chord_moe_route(a.pop("logits"), a.pop("k"), **a)
    ids, w = C.chord_moe_route(x[:0], 3)
    assert ids.shape == (0, 3) and w.shape == (0, 3)


def test_route_on_another_stream_and_in_a_graph(C):
    g = torch.Generator().manual_seed(4)
    logits = torch.randn((64, 384), generator=g).cuda()
    bias = (0.1 * torch.randn(384, generator=g)).cuda()
    kw = dict(scoring=C.SCORE_SIGMOID, bias=bias, n_group=8, topk_group=4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = C.chord_moe_route(logits, 8, stream=s, **kw)
    torch.cuda.synchronize()
    b = C.chord_moe_route(logits, 8, **kw)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = C.chord_moe_route(logits, 8, **kw)
    for seed in range(3):
        logits.copy_(torch.randn((64, 384), generator=torch.Generator().manual_seed(10 + seed)))
        graph.replay()
        torch.cuda.synchronize()
        want = C.chord_moe_route(logits, 8, **kw)
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
