"""Size limits of the router and the 8-bit layer, by the host's checks alone."""

import ctypes

from quantized_moe_amd import chord as C


def test_moe_sizes():
    """The codes of x and h stay below 2 GiB; y, stored with 64-bit offsets, does
    not have to."""
    f = C.chord_f8_moe_workspace_bytes
    T, k, H, I = 40000, 8, 7168, 128
    need = f(T, k, 2, H, I)
    assert need > T * k * H * 2 > 1 << 32
    assert f(1 << 18, 1, 1, 8064, 128) > 0 and f(1 << 18, 1, 1, 8192, 128) == 0   # x
    assert f(1 << 17, 8, 1, 128, 1920) > 0 and f(1 << 17, 8, 1, 128, 2048) == 0   # h
    assert f(1 << 27, 8, 1, 128, 128) == 0


def test_route_tokens():
    """More tokens than a launch has waves for are refused by the host."""
    fake = ctypes.c_void_p(0x1000)
    for T in ((1 << 25) + 1, 2**31 - 1):
        st = C.lib.chord_moe_route(fake, 0, 8, T, 8, None, 2, 0, 1, 1, 1, 1.0, fake, fake, None)
        assert st == 2 and b"above" in C.lib.chord_last_error()
