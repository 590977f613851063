"""Inputs of the W8A8 layer whose gate and up products come out exact in every
kind of sum: tokens of +-1, 1/2, 1/4, 1/8 (codes 448 and its halves) and weights of
codes +-1, 2, 4, so the products of a block of 128 are whole multiples of the
smallest of them and the largest is 2^5 times that, far from the 2^13 that the
8-bit matrix instruction keeps.  h is then off by a few roundings of fp32, takes
another code than the oracle's about never, and a row of outputs is as exact as
its rounding to bf16, whatever form the layer ran in."""

import numpy as np
import torch

from oracle import f8


def tokens(T, H, seed):
    """bf16 [T, H]."""
    g = torch.Generator().manual_seed(seed)
    x = 2.0 ** -torch.randint(0, 4, (T, H), generator=g).float()
    x = x * torch.where(torch.rand((T, H), generator=g) < 0.5, -1.0, 1.0)
    x[:, ::f8.BLOCK] = 1.0   # every group's largest
    return (x * 2.0 ** torch.randint(-1, 2, (T, 1), generator=g)).bfloat16()


def gate_up(E, H, I, seed):
    """Codes [E, 2I, H] on the host, scales, fp64 values; gates of the order of one."""
    g = torch.Generator().manual_seed(seed)
    v = 2.0 ** torch.randint(0, 3, (E, 2 * I, H), generator=g).float()
    v = v * torch.where(torch.rand((E, 2 * I, H), generator=g) < 0.5, -1.0, 1.0)
    scales = (0.5 + torch.rand((E, 2 * I // f8.BLOCK, H // f8.BLOCK), generator=g)) / (1.5 * H ** 0.5)
    deq = np.stack([f8.dequantize_weight(v[e].double().numpy(), scales[e].double().numpy()) for e in range(E)])
    return v.to(torch.float8_e4m3fn), scales, deq
