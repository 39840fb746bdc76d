"""The 8-bit matrices' definitions (``include/tn_block8.h``) in 64 bits, on the CPU."""
import torch


def scale(top):
    """Smallest power of two s from 2^-126 on with top <= 448 s; 1 for 0, NaN for no number."""
    if not (top < float("inf")):
        return float("nan")
    if top == 0.0:
        return 1.0
    s = 2.0 ** -126
    while top > 448.0 * s:
        s *= 2.0
    return s


def e4m3(v):
    """Rounded to e4m3's values, ties to even."""
    v = v.double()
    step = torch.ldexp(torch.ones_like(v), torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent - 4)
    return torch.round(v / step) * step


def quantize(x, square):
    """(values of the codes, scales) of a matrix."""
    x = x.double()
    R, C = x.shape
    tall = 128 if square else 1
    codes = torch.zeros_like(x)
    scales = torch.zeros(-(-R // tall), -(-C // 128), dtype=torch.float64)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = slice(i * tall, (i + 1) * tall), slice(j * 128, (j + 1) * 128)
            top = x[at].abs().max().item() if not x[at].isnan().any() else float("nan")
            s = scales[i, j] = scale(top)
            if s == s:
                codes[at] = e4m3(x[at] / s)
    return codes, scales


def values(codes, scales):
    if scales.shape[0] != codes.shape[0]:
        scales = scales.repeat_interleave(128, 0)[:codes.shape[0]]
    return codes.double() * scales.double().repeat_interleave(128, 1)[:, :codes.shape[1]]


def product_bound(a, b, dtype):
    """(a b^T, how far the kernels' result may be from it) of two matrices of values.

    Within a block of 128, four instructions add 32 products each to the sum.  An
    addend that is aligned to the largest loses less than 2^-23 of it (24 bits
    kept): 33 addends, 33 2^-23 of the largest at most, which is no more than the sum
    of magnitudes; over four instructions it is no more than that of the
    block's (each instruction's largest addend is one of its own products or
    the sum before): 4 x 33 2^-23.  Scaling and adding a block are two roundings
    (three with separate scales), each 2^-24, the sum before being rounded once a block.
    Last, the output's rounding."""
    c = a @ b.t()
    size = a.abs() @ b.abs().t()
    blocks = -(-a.shape[1] // 128)
    far = size * (4 * 33 * 2.0 ** -23 + (blocks + 3) * 2.0 ** -24)
    return c, far + (c.abs() + far) * (torch.finfo(dtype).eps / 2) + torch.finfo(dtype).tiny
