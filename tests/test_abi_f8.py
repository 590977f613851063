"""Refusals of the router and the 8-bit entry points: every call here fails the
host's checks before any HIP call, so no GPU is needed."""

import ctypes

import pytest
import torch

from quantized_moe_amd import chord as C

FAKE = ctypes.c_void_p(0x1000)   # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x1001)
INVALID, UNSUPPORTED, MISMATCH, WORKSPACE = 1, 2, 3, 4


def _route(**kw):
    a = dict(logits=FAKE, dtype=0, ld=64, T=4, E=64, bias=None, k=8, scoring=0, n_group=1,
             topk_group=1, renorm=1, scaling=1.0, ids=FAKE, weights=FAKE)
    a.update(kw)
    return C.lib.chord_moe_route(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(dtype=-1), dict(scoring=2), dict(T=-1), dict(E=0), dict(E=1025, ld=1025),
    dict(ld=63), dict(k=0), dict(k=33), dict(E=4, k=5), dict(n_group=3), dict(n_group=0),
    dict(n_group=8, topk_group=9), dict(n_group=8, topk_group=0), dict(n_group=8, topk_group=1, k=9),
    dict(E=130, ld=130, n_group=65), dict(scaling=float("nan")), dict(scaling=float("inf")),
    dict(logits=None), dict(ids=None), dict(weights=None),
])
def test_route_refusals(kw):
    assert _route(**kw) == INVALID
    assert C.lib.chord_last_error()


def test_route_without_tokens_is_a_no_op():
    assert _route(T=0, logits=None, ids=None, weights=None) == 0


def test_f8_packed_bytes():
    assert C.chord_f8_packed_bytes(C.ROLE_GATE_UP, 48, 4096, 7168) == 48 * 4096 * 7168 + 48 * 32 * 56 * 4
    assert C.chord_f8_packed_bytes(C.ROLE_PLAIN, 1, 1, 1) == 16 * 128 + 4
    assert C.chord_f8_packed_bytes(C.ROLE_PLAIN, 1, 130, 129) == 144 * 256 + 2 * 2 * 4
    for role, E, N, K in ((C.ROLE_PLAIN, 2, 128, 128), (C.ROLE_DOWN, 1, 120, 128), (C.ROLE_DOWN, 1, 128, 64),
                          (C.ROLE_GATE_UP, 1, 128, 128), (C.ROLE_DOWN, 1025, 128, 128), (7, 1, 128, 128),
                          (C.ROLE_PLAIN, 1, 0, 128), (C.ROLE_PLAIN, 1, 1 << 16, 1 << 16)):
        assert C.chord_f8_packed_bytes(role, E, N, K) == 0, (role, E, N, K)


def _pack(role=2, q=FAKE, s=FAKE, E=1, N=256, K=256, block=128, dst=FAKE, n=1 << 30, h=True):
    w = C.F8Weight()
    return C.lib.chord_f8_pack(role, q, s, E, N, K, block, dst, n, ctypes.byref(w) if h else None, None)


def test_f8_pack_refusals():
    assert _pack(block=64) == UNSUPPORTED
    assert _pack(role=9) == INVALID
    assert _pack(q=None) == INVALID and _pack(s=None) == INVALID and _pack(dst=None) == INVALID
    assert _pack(h=False) == INVALID
    assert _pack(dst=ctypes.c_void_p(0x1008)) == INVALID
    assert _pack(n=256 * 256) == INVALID          # no room for the scales
    assert _pack(role=0, N=128) == UNSUPPORTED    # I = 64


def test_quantize_refusals():
    f = C.lib.chord_f8_quantize
    assert f(FAKE, 4, 128, 127, FAKE, FAKE, None) == INVALID
    assert f(FAKE, -1, 128, 128, FAKE, FAKE, None) == INVALID
    assert f(FAKE, 4, 0, 128, FAKE, FAKE, None) == INVALID
    assert f(None, 4, 128, 128, FAKE, FAKE, None) == INVALID
    assert f(FAKE, 4, 128, 128, ODD, FAKE, None) == INVALID
    assert f(FAKE, 4, 128, 128, FAKE, None, None) == INVALID
    assert f(None, 0, 128, 128, None, None, None) == 0


def _handle(role, E=1, N=256, K=256):
    h = C.F8Weight()
    h.magic, h.version, h.role, h.num_experts = 0x57384538, 1, role, E
    h.n, h.k, h.block, h.data, h.bytes = N, K, 128, 0x2000, 1 << 30
    return h


def _gemm(h, codes=FAKE, s=FAKE, M=4, out=FAKE, ld=256, ws=FAKE, n=1 << 30):
    return C.lib.chord_f8_gemm(codes, s, M, None if h is None else ctypes.byref(h), out, ld, ws, n, None)


def test_gemm_refusals():
    good = _handle(2)
    assert _gemm(None) == INVALID
    assert _gemm(_handle(1)) == MISMATCH
    assert _gemm(good, ld=255) == INVALID
    assert _gemm(good, M=-1) == INVALID
    assert _gemm(good, M=1 << 31) == UNSUPPORTED
    assert _gemm(good, codes=None) == INVALID and _gemm(good, out=None) == INVALID
    assert _gemm(good, codes=ODD) == INVALID
    assert _gemm(good, M=0, codes=None, out=None) == 0
    bad = _handle(2)
    bad.magic = 0x43573441                         # a 4-bit handle's
    assert _gemm(bad) == INVALID
    bad = _handle(2)
    bad.bytes = 100
    assert _gemm(bad) == INVALID
    bad = _handle(2)
    bad.block = 64
    assert _gemm(bad) == UNSUPPORTED


def test_gemm_workspace():
    """Only products with K in parts need one; it has to be there, whole and aligned."""
    assert C.chord_f8_gemm_workspace_bytes(1, 4096, 7168) == 0
    assert C.chord_f8_gemm_workspace_bytes(8192, 4096, 7168) == 0
    need = C.chord_f8_gemm_workspace_bytes(200, 520, 4000)
    assert need > 0 and need % (200 * 528 * 4) == 0
    h = _handle(2, N=520, K=4000)
    assert _gemm(h, M=200, ld=520, ws=None) == WORKSPACE
    assert _gemm(h, M=200, ld=520, n=need - 1) == WORKSPACE
    assert _gemm(h, M=200, ld=520, ws=ODD) == WORKSPACE
    for bad in ((-1, 300, 4096), (150, 0, 4096), (150, 300, 0), (150, 1 << 16, 1 << 16), (1, 16, 1 << 23)):
        assert C.chord_f8_gemm_workspace_bytes(*bad) == 0


def _moe(w13=None, w2=None, x=FAKE, T=4, H=256, I=128, k=2, ids=FAKE, out=FAKE, ws=FAKE, n=1 << 30):
    w13 = w13 or _handle(0, E=2, N=256, K=256)
    w2 = w2 or _handle(1, E=2, N=256, K=128)
    return C.lib.chord_f8_moe(x, T, H, I, ctypes.byref(w13), ctypes.byref(w2), ids, FAKE, k, 0, 0, out,
                              ws, n, None)


def test_moe_refusals():
    assert _moe(w13=_handle(1, E=2, N=256, K=256)) == MISMATCH
    assert _moe(w2=_handle(1, E=3, N=256, K=128)) == INVALID
    assert _moe(w2=_handle(1, E=2, N=256, K=256)) == INVALID
    assert _moe(I=64) == UNSUPPORTED
    assert _moe(k=0) == INVALID and _moe(T=-1) == INVALID
    assert _moe(x=None) == INVALID and _moe(ids=None) == INVALID and _moe(out=None) == INVALID
    assert _moe(x=ctypes.c_void_p(0x1008)) == INVALID
    assert _moe(ws=None) == WORKSPACE and _moe(n=100) == WORKSPACE
    assert _moe(ws=ctypes.c_void_p(0x1010)) == WORKSPACE
    assert _moe(T=1 << 22, k=8) == UNSUPPORTED     # rows past 2 GiB
    assert _moe(T=0, x=None, ids=None, out=None, ws=None, n=0) == 0
    assert C.chord_f8_moe_workspace_bytes(4, 2, 2, 256, 100) == 0
    assert C.chord_f8_moe_workspace_bytes(4, 2, 2, 256, 128) > 0


def test_python_wrappers_refuse_host_tensors():
    with pytest.raises(C.ChordError):
        C.chord_moe_route(torch.zeros(4, 8), 2)
    with pytest.raises(C.ChordError):
        C.chord_f8_quantize(torch.zeros(4, 128, dtype=torch.bfloat16))
    with pytest.raises(C.ChordError):
        C.chord_f8_pack(C.ROLE_PLAIN, torch.zeros(1, 128, 128).to(torch.float8_e4m3fn), torch.ones(1, 1, 1))
