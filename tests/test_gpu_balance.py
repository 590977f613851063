"""GPU balance against the fp64 oracle (oracle/block.py, whose header says how the
bounds are made): counts exactly, scores, losses and gradients within fp32."""

import numpy as np
import pytest
import torch

from oracle import block as B
from tests.gpu_util import banner, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def C():
    from quantized_moe_amd import chord
    return chord


def draw(T, E, k, seed, dtype=torch.float32, padded=0.0):
    g = torch.Generator().manual_seed(seed)
    logits = (1.5 * torch.randn((T, E), generator=g) + 0.5 * torch.randn(E, generator=g)).to(dtype)
    ids = torch.rand((T, E), generator=g).argsort(dim=1)[:, :k].to(torch.int32)
    if padded:
        ids[torch.rand(T, generator=g) < padded] = -1
    return logits, ids


def check(C, logits, ids, sigmoid=False, n_seq=1, bias=None, grad_loss=None, **kw):
    r = C.chord_moe_balance(logits, ids, C.SCORE_SIGMOID if sigmoid else C.SCORE_SOFTMAX, bias, n_seq, grad_loss,
                            want_grad=True, **kw)
    torch.cuda.synchronize()
    as64 = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    o = B.balance(as64(logits), host(ids), sigmoid, n_seq, as64(bias), as64(grad_loss))
    assert np.array_equal(host(r.counts), o["counts"]) and np.array_equal(host(r.tokens), o["tokens"])
    for name in ("probs", "loss", "grad"):
        got, ref = as64(getattr(r, name)), o[name]
        bad = ~(np.abs(got - ref) <= o["e_" + name] + B.rounding(ref, "float32"))
        assert not bad.any(), (name, np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])
    return r


CASES = [
    # T, E, k, n_seq, sigmoid, dtype, padded
    (1, 1, 1, 1, False, torch.float32, 0),
    (1, 384, 8, 1, False, torch.float32, 0),
    (1, 8, 8, 1, True, torch.bfloat16, 0),
    (7, 65, 3, 7, True, torch.float32, 0),
    (64, 256, 8, 1, True, torch.bfloat16, 0.2),
    (65, 64, 1, 5, False, torch.float16, 0.3),
    (33, 1000, 32, 3, False, torch.float32, 0.1),
    (100, 513, 70, 1, True, torch.float32, 0.1),
    (333, 100, 4, 3, True, torch.float32, 0.5),
    (1024, 384, 8, 8, False, torch.float32, 0.2),
    (2500, 160, 16, 1, False, torch.bfloat16, 0.1),     # slots counted by several workgroups
    (4096, 1024, 8, 1, True, torch.float32, 0.1),
    (16384, 64, 6, 2, False, torch.float32, 0.1),
]


@pytest.mark.parametrize("T,E,k,n_seq,sigmoid,dtype,padded", CASES)
def test_balance(C, T, E, k, n_seq, sigmoid, dtype, padded):
    banner(f"balance T={T} E={E} k={k} n_seq={n_seq} sigmoid={sigmoid}")
    logits, ids = draw(T, E, k, T + E, dtype, padded)
    up = 0.5 + torch.arange(n_seq, dtype=torch.float32)
    a = check(C, logits.cuda(), ids.cuda(), sigmoid, n_seq, grad_loss=up.cuda())
    b = check(C, logits.cuda(), ids.cuda(), sigmoid, n_seq)
    assert torch.equal(a.loss, b.loss) and torch.equal(a.probs, b.probs)
    c = C.chord_moe_balance(logits.cuda(), ids.cuda(), int(sigmoid), n_seq=n_seq)
    assert c.grad is None and torch.equal(c.loss, b.loss) and torch.equal(c.counts, b.counts)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_masks_and_extremes(C, sigmoid):
    """Experts out of service by their logits or the bias, rows without any, rows of
    padding, ids that are no expert, an expert in every slot, infinities."""
    T, E, k = 40, 130, 4
    logits, ids = draw(T, E, k, 5)
    logits[:, 7] = -np.inf
    logits[3, 20:60] = np.nan
    logits[4] = -np.inf            # no expert left, though the ids name some
    logits[5] = -3.4028234663852886e38
    logits[6, 9] = np.inf
    logits[8, 11:13] = np.inf
    logits[9] *= 300
    ids[10] = torch.tensor([-1, E, 2 ** 31 - 1, -2 ** 31])   # padding
    ids[11] = torch.tensor([5, -1, 5, 5])
    ids[12] = 9
    bias = torch.zeros(E)
    bias[30], bias[31], bias[32] = -np.inf, np.nan, 5.0
    for b in (None, bias.cuda()):
        for n_seq in (1, 4, 40):
            check(C, logits.cuda(), ids.cuda(), sigmoid, n_seq, b)
    r = check(C, logits.cuda(), torch.full_like(ids, -1).cuda(), sigmoid, 2)
    assert not r.loss.any() and not r.grad.any() and not r.probs.any() and not r.tokens.any()


def test_near_balance(C):
    """Tokens as even as they can be: the loss is 1 but for rounding, and the gradient
    a small difference."""
    T, E, k = 768, 96, 4
    ids = (torch.arange(T * k).reshape(T, k) % E).to(torch.int32)
    logits, _ = draw(T, E, k, 8)
    r = check(C, logits.cuda(), ids.cuda())
    assert torch.equal(r.counts, torch.full_like(r.counts, T * k // E)) and abs(r.loss.item() - 1) < 1e-6
    assert r.grad.abs().max().item() < 1e-9
    ids[0] = ids[1]
    check(C, logits.cuda(), ids.cuda())


def test_gradient_against_differences(C):
    """In the direction of the gradient, from the kernel's own losses: the second order
    is below h |g| of the first, the loss's rounding 2^-24 over 2 h |g|."""
    T, E, k = 48, 32, 2
    logits, ids = draw(T, E, k, 9)
    for sigmoid in (False, True):
        # f is constant here as ids do not move.
        r = C.chord_moe_balance(logits.cuda(), ids.cuda(), int(sigmoid), want_grad=True)
        g = r.grad.double()
        size = g.norm().item()
        step = 0.5 * g / size
        two = [C.chord_moe_balance((logits.cuda().double() + s * step).float(), ids.cuda(), int(sigmoid)).loss.item()
               for s in (1, -1)]
        assert abs((two[0] - two[1]) - size) < 0.05 * size + 2.0 ** -22


def test_strides_out_and_nothing(C):
    logits, ids = draw(50, 100, 3, 10, torch.bfloat16, 0.2)
    wide = torch.full((50, 133), 9.0, dtype=torch.bfloat16)
    wide[:, 5:105] = logits
    a = check(C, wide.cuda()[:, 5:105], ids.cuda(), n_seq=2)
    b = C.Balance(*[torch.zeros_like(t) for t in a])
    r = C.chord_moe_balance(logits.cuda(), ids.cuda(), n_seq=2, out=b)
    assert r is b and all(torch.equal(x, y) for x, y in zip(a, b))
    r = C.chord_moe_balance(logits.cuda()[:0], ids.cuda()[:0], n_seq=3, want_grad=True)
    assert r.counts.shape == (3, 100) and not r.counts.any() and not r.loss.any() and not r.probs.any()
    assert not r.tokens.any() and r.grad.shape == (0, 100)


@pytest.mark.parametrize("T,n_seq", [(64, 1), (2048, 2), (6000, 1)])
def test_streams_and_graphs(C, T, n_seq):
    E, k = 96, 4
    logits, ids = (t.cuda() for t in draw(T, E, k, 11, padded=0.1))
    want = C.chord_moe_balance(logits, ids, n_seq=n_seq, want_grad=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = C.chord_moe_balance(logits, ids, n_seq=n_seq, want_grad=True, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(C.chord_moe_balance(logits, ids, n_seq=n_seq, want_grad=True))
    for seed in range(3):
        a, b = draw(T, E, k, 20 + seed, padded=0.3)
        logits.copy_(a)
        ids.copy_(b)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = C.chord_moe_balance(logits, ids, n_seq=n_seq, want_grad=True)
        for got in outs:
            assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_refusals(C):
    logits, ids = (t.cuda() for t in draw(8, 16, 2, 1))
    for kw in (dict(n_seq=3), dict(n_seq=0), dict(scoring=4), dict(bias=logits[0].half()), dict(grad_loss=logits[0, :2]),
               dict(topk_ids=ids.long()), dict(topk_ids=ids[:5]), dict(topk_ids=ids.cpu())):
        with pytest.raises(C.ChordError):
            C.chord_moe_balance(logits, **{"topk_ids": ids, **kw})
