"""The operators together, as a model's block calls them: norm with the residual,
the gate's logits, the router and its balance, the experts, the shared expert onto
their output, and the norm that adds the block's output to the residual stream and
prepares the next block's input.  Each step is checked against the oracle on the
inputs that it had."""

import numpy as np
import pytest
import torch

from moe_inputs import gen as G
from oracle import block as B
from oracle import f8
import oracle
from tests.gpu_util import banner, dev, dev_bf16, host, host_bf16
from tests.tolerance import check_close

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().double().cpu().numpy()


def near(got, ref, bound):
    name = str(got.dtype).replace("torch.", "")
    return np.all(np.abs(f64(got) - ref) <= bound + B.rounding(np.abs(ref) + bound, name))


@pytest.mark.parametrize("T", [1, 5, 70, 300])
def test_block(T):
    from quantized_moe_amd import chord as C
    from quantized_moe_amd.moe import Linear, SharedExpert, W4A16MoE
    banner(f"block T={T}")
    H, I, Is, E, k = 512, 256, 384, 16, 4
    rng = np.random.Generator(np.random.PCG64(T))
    q13, s13 = G.draw_weights(rng, E, 2 * I, H, scale_mult=(256.0 / H) ** 0.5)
    q2, s2 = G.draw_weights(rng, E, H, I, scale_mult=(256.0 / I) ** 0.5)
    layer = W4A16MoE(dev(q13), dev_bf16(s13), dev(q2), dev_bf16(s2))
    g = torch.Generator().manual_seed(T)
    draw = lambda *s, scale=1.0, dtype=BF16: (scale * torch.randn(s, generator=g)).to(dtype).cuda()  # noqa: E731
    before, behind, following = (C.Norm(draw(H, scale=0.1) + 1) for _ in range(3))
    gate_w, w13, w2 = draw(E, H, scale=H ** -0.5), draw(2 * Is, H, scale=H ** -0.5), draw(H, Is, scale=Is ** -0.5)
    attn, stream = draw(T, H), draw(T, H, dtype=F32)
    part = lambda n: (f64(n.weight), None, "rms", float(np.float32(1e-6)))  # noqa: E731

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        n1 = C.chord_norm(attn, before, residual=stream)
        logits = Linear(gate_w)(n1.out, out_dtype=F32)
        ids, w = C.chord_moe_route(logits, k)
        balance = C.chord_moe_balance(logits, ids, want_grad=True)
        routed = layer.indexed(n1.out, ids, w, 0, E)
        both = SharedExpert(w13, w2)(n1.out, routed)
        n2 = C.chord_norm(both, following, behind, residual=n1.sum, scale=0.5, want_codes=True)
    torch.cuda.synchronize()

    s, es, y, ey = B.block_norm(f64(attn), residual=f64(stream), pre=part(before))
    assert near(n1.sum, s, es) and near(n1.out, y, ey)
    ref, bound = B.linear(f64(n1.out), f64(gate_w))
    assert near(logits, ref, bound)
    ri, rw = f8.route(f64(logits), None, k, False, 1, 1, True, 1.0)
    assert np.array_equal(host(ids), ri)
    o = B.balance(f64(logits), host(ids), False)
    assert np.array_equal(host(balance.counts), o["counts"]) and int(balance.counts.sum()) == T * k
    assert near(balance.loss, o["loss"], o["e_loss"]) and near(balance.grad, o["grad"], o["e_grad"])
    check_close(host_bf16(routed), oracle.moe_layer(host_bf16(n1.out), host(ids), host(w), q13, s13, q2, s2, 0))
    h = Linear(w13, act=C.ACT_SILU, gated=True)(n1.out)
    ref, bound = B.linear(f64(n1.out), f64(w13), act="silu", gated=True)
    assert near(h, ref, bound)
    ref, bound = B.linear(f64(h), f64(w2), residual=f64(routed))
    assert near(both, ref, bound)
    s, es, y, ey = B.block_norm(f64(both), part(behind), residual=f64(n1.sum), scale=0.5, pre=part(following))
    assert near(n2.sum, s, es) and near(n2.out, y, ey)
    assert n2.codes.shape == (T, H) and n2.sum.dtype is F32


def test_shared_expert_in_place():
    from quantized_moe_amd.moe import SharedExpert
    g = torch.Generator().manual_seed(1)
    x, w13, w2 = (torch.randn(s, generator=g).to(BF16).cuda() for s in ((33, 128), (192, 128), (128, 96)))
    shared = SharedExpert(w13, w2)
    routed = x.clone()
    want = shared(x, routed)
    got = shared(x, routed, out=routed)
    torch.cuda.synchronize()
    assert got.data_ptr() == routed.data_ptr() and torch.equal(got, want)
    assert torch.equal(shared(x), shared(x, torch.zeros_like(x)))
