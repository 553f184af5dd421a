"""8-bit codes and their scales in 64 bits, from the definition (no code of the package)."""

import torch

KINDS = {"e4m3": 3, "i8": 4}  # DEC_T_*
TOP = {"e4m3": 448.0, "i8": 127.0}
E_MIN, E_MAX = -40, 40


def two(e):
    """2^e of whole e of -126 .. 127 (torch.exp2 rounds on some devices)."""
    return ((e.int() + 127) << 23).view(torch.float32).double()


def log2(scale):
    """e of the fp32 scales 2^e."""
    return (torch.frexp(scale)[1] - 1).double()


def need(amax, kind):
    """The smallest e of -40 .. 40 with amax <= top 2^e, for every element."""
    e = torch.full_like(amax, float(E_MIN))
    for _ in range(E_MAX - E_MIN):
        e = torch.where(amax > TOP[kind] * two(e), (e + 1).clamp(max=E_MAX), e)
    return e


def rounded(y, kind):
    """The nearest number that a code stands for, ties to even."""
    if kind == "i8":
        return torch.round(y).clamp(-127, 127)
    y = y.clamp(-448, 448)
    step = two(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)  # three bits behind the leading one, 2^-9 at least
    return torch.round(y / step) * step


def codes_of(x, e, kind):
    """The bytes of x / 2^e."""
    y = rounded(x / two(e), kind)
    if kind == "i8":
        return y.to(torch.int8).view(torch.uint8)
    return y.float().to(torch.float8_e4m3fn).view(torch.uint8)  # exact


def numbers(codes, kind):
    """What the bytes stand for, without their scale."""
    return codes.view(torch.int8).double() if kind == "i8" else codes.view(torch.float8_e4m3fn).float().double()
