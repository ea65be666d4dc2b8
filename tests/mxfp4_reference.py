"""The 4-bit cache format on the CPU in 64 bits, for the tests of the calls that
write, read and attend to it."""
import math

import torch

LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
BLOCK = 32


def encode(x):
    """float64 [..., dim] -> (code bytes [..., dim / 2], exponent bytes [..., dim / 32]).

    The scale is the smallest power of two, between 2^-125 and 2^125, by which
    the block's largest magnitude is at most 7; an element takes the nearest
    level, the even code of two as near."""
    shape = x.shape[:-1] + (x.shape[-1] // BLOCK, BLOCK)
    b = x.reshape(shape)
    nan = torch.isnan(b).any(-1)
    most = torch.where(nan, torch.zeros(()).double(), b.abs().amax(-1))
    e = torch.full(most.shape, -125, dtype=torch.int64)
    for p in range(-124, 126):
        e = torch.where(most > 7.0 * 2.0 ** (p - 1), torch.full_like(e, p), e)
    y = (b / torch.pow(torch.tensor(2.0, dtype=torch.float64), e[..., None])).abs()
    code = torch.zeros(y.shape, dtype=torch.int64)
    for i in range(7):
        border = (LEVELS[i] + LEVELS[i + 1]) / 2
        # half-way goes to the even of codes i and i + 1
        code += (y > border) if i % 2 == 0 else (y >= border)
    code += 8 * torch.signbit(b)
    code = torch.where(nan[..., None], torch.zeros_like(code), code).reshape(x.shape)
    e = torch.where(nan, torch.full_like(e, 128), e)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), (e + 127).to(torch.uint8)


def decode(codes, exponents):
    """What they stand for, float64; blocks of exponent bytes above 252 are NaN."""
    levels = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=torch.float64)
    both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    scale = torch.pow(torch.tensor(2.0, dtype=torch.float64), exponents.double() - 127.0)
    scale = torch.where(exponents > 252, torch.full_like(scale, math.nan), scale)
    return levels[both] * scale.repeat_interleave(BLOCK, -1)
