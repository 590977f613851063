"""Refusals of the norms, the 16-bit product and the balance: every call here fails
the host's checks before any HIP call, so no GPU is needed."""

import ctypes

import pytest
import torch

from quantized_moe_amd import chord as C

FAKE = ctypes.c_void_p(0x1000)   # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x1001)
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4
F32, BF16, F16 = 0, 1, 2


def part(kind=0, dtype=BF16, eps=1e-6, offset=0.0, weight=0x1000, bias=None):
    return ctypes.byref(C.NormWeight(kind, dtype, eps, offset, weight, bias))


def norm(**kw):
    a = dict(x=FAKE, ldx=64, dtype=BF16, T=4, H=64, post=None, gate=None, gate_dtype=BF16, gate_row=0, gate_col=0,
             sigmoid=0, scale=1.0, residual=None, ldr=64, sum=None, lds=64, stream_dtype=BF16, pre=part(), out=FAKE,
             ldo=64, codes=None, scales=None)
    a.update(kw)
    return C.lib.chord_norm(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(stream_dtype=F16), dict(dtype=F32, stream_dtype=BF16), dict(T=-1), dict(H=0), dict(ldx=63),
    dict(residual=FAKE, ldr=63), dict(sum=FAKE, lds=63), dict(ldo=63), dict(scale=float("nan")),
    dict(out=None), dict(pre=None), dict(pre=None, out=None), dict(out=None, sum=FAKE), dict(x=None),
    dict(codes=FAKE), dict(scales=FAKE), dict(codes=ODD, scales=FAKE), dict(pre=None, out=None, codes=FAKE, scales=FAKE),
    dict(gate=FAKE, gate_dtype=3), dict(gate=FAKE, gate_col=2), dict(gate=FAKE, gate_row=-1),
    dict(pre=part(kind=2)), dict(pre=part(dtype=3)), dict(pre=part(eps=0.0)), dict(pre=part(eps=-1.0)),
    dict(pre=part(eps=float("inf"))), dict(pre=part(eps=1e-42)), dict(pre=part(offset=float("inf"))),
    dict(pre=part(weight=None)), dict(post=part(weight=None)),
])
def test_norm_refusals(kw):
    assert norm(**kw) == INVALID
    assert C.lib.chord_last_error()


def test_norm_limits():
    assert norm(H=32769, ldx=40000, ldo=40000) == UNSUPPORTED
    assert norm(T=1 << 31) == UNSUPPORTED
    assert norm(T=0, x=None) == 0


def linear(**kw):
    a = dict(x=FAKE, ldx=64, w=FAKE, ldw=64, dtype=BF16, M=4, N=32, K=64, bias=None, bias_dtype=BF16, act=0, gated=0,
             scale=1.0, residual=None, ldr=32, out=FAKE, ldo=32, out_dtype=BF16, ws=FAKE, n=1 << 30)
    a.update(kw)
    return C.lib.chord_linear(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(dtype=5), dict(out_dtype=F16), dict(bias=FAKE, bias_dtype=F16), dict(act=5), dict(act=-1),
    dict(scale=float("inf")), dict(M=-1), dict(N=0), dict(K=0), dict(ldx=63), dict(ldw=63), dict(ldo=31),
    dict(residual=FAKE, ldr=31), dict(x=None), dict(w=None), dict(out=None),
])
def test_linear_refusals(kw):
    assert linear(**kw) == INVALID
    assert C.lib.chord_last_error()


def test_linear_limits():
    assert linear(dtype=F32, out_dtype=F32) == UNSUPPORTED
    assert linear(M=1 << 29) == UNSUPPORTED
    assert linear(N=1 << 28, gated=1, ldo=1 << 28) == UNSUPPORTED
    assert linear(K=(1 << 20) + 1, ldx=1 << 21, ldw=1 << 21) == UNSUPPORTED
    assert linear(M=0, x=None, w=None, out=None) == 0
    f = C.lib.chord_linear_workspace_bytes
    for bad in ((63, 64, 4, 32, 64, 0), (64, 63, 4, 32, 64, 0), (64, 64, -1, 32, 64, 0), (64, 64, 4, 0, 64, 0)):
        assert f(FAKE, bad[0], FAKE, *bad[1:]) == 0 and C.lib.chord_last_error()


def balance(**kw):
    a = dict(logits=FAKE, dtype=F32, ld=64, T=8, E=64, bias=None, ids=FAKE, k=8, scoring=0, n_seq=2, counts=FAKE,
             tokens=FAKE, probs=FAKE, loss=FAKE, grad_loss=None, grad=None, ws=FAKE, n=1 << 30)
    a.update(kw)
    return C.lib.chord_moe_balance(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(scoring=2), dict(T=-2), dict(E=0), dict(E=1025, ld=1025), dict(ld=63), dict(k=0),
    dict(k=1025), dict(n_seq=0), dict(n_seq=3), dict(logits=None), dict(ids=None), dict(counts=None),
    dict(tokens=None), dict(probs=None), dict(loss=None),
])
def test_balance_refusals(kw):
    assert balance(**kw) == INVALID
    assert C.lib.chord_last_error()


def test_balance_limits():
    assert balance(T=(1 << 25) + 2) == UNSUPPORTED
    assert balance(T=1 << 25, k=64) == UNSUPPORTED
    assert balance(T=0, n_seq=65536) == UNSUPPORTED
    need = C.chord_moe_balance_workspace_bytes(8192, 384, 8, 1)
    assert need > 0
    for kw in (dict(ws=None), dict(n=need - 1), dict(ws=ODD)):
        assert balance(T=8192, E=384, ld=384, n_seq=1, **kw) == WORKSPACE
    assert C.chord_moe_balance_workspace_bytes(8, 64, 8, 3) == 0


def test_python_wrappers_refuse_host_tensors():
    b = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(C.ChordError):
        C.Norm(torch.ones(8))
    with pytest.raises(C.ChordError):
        C.chord_norm(b)
    with pytest.raises(C.ChordError):
        C.chord_linear(b, b)
    with pytest.raises(C.ChordError):
        C.chord_moe_balance(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32))
