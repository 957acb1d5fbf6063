"""Plain 64-bit forms of what the cache's 8-bit rows hold, for the GPU tests: a row is [Hkv][D] e4m3, then a byte
127 + e for each head, then zeros up to a multiple of 16 bytes; a value is e4m3 * 2^e."""
import math

import torch

LARGEST, HI = 448.0, 7
LO = {torch.bfloat16: -126, torch.float16: -15}


def row_bytes(Hkv, D):
    return -(-Hkv * (D + 1) // 16) * 16


def grid():
    """What e4m3's bits stand for, 0 .. 127 (the last is NaN)."""
    got = [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)]
    return torch.tensor(got[:127] + [math.nan], dtype=torch.float64)


def two_to(e):
    """2^e in 64 bits, by its bits (a library's power need not be exact)."""
    return (e.long() + 1023 << 52).view(torch.float64)


def exponents(x, dtype):
    """x [..., D] in 64 bits: each head's e."""
    m, e = torch.frexp(torch.nan_to_num(x, nan=0.0, posinf=1e300, neginf=1e300).abs().amax(-1) / LARGEST)
    e = e - (m == 0.5).int()
    return torch.where(m == 0, LO[dtype], e).clamp(LO[dtype], HI)


def encode(x, dtype):
    """x [..., Hkv, D] (values of dtype, exactly) to rows of bytes [..., row_bytes]."""
    x = x.double()
    Hkv, D = x.shape[-2:]
    e = exponents(x, dtype)
    g = grid()[:127].to(x.device)
    mid = (g[1:] + g[:-1]) / 2
    y = torch.nan_to_num((x.abs() / two_to(e)[..., None]), posinf=LARGEST).clamp(max=LARGEST)
    lower, upper = torch.bucketize(y, mid), torch.bucketize(y, mid, right=True)
    bits = torch.where(lower % 2 == 0, lower, upper)  # they differ at a tie: the even one
    bits = torch.where(torch.isnan(x), 127, bits + 128 * torch.signbit(x))
    rows = torch.zeros((*x.shape[:-2], row_bytes(Hkv, D)), dtype=torch.uint8, device=x.device)
    rows[..., : Hkv * D] = bits.to(torch.uint8).flatten(-2)
    rows[..., Hkv * D: Hkv * (D + 1)] = (e + 127).to(torch.uint8)
    return rows


def decode(rows, Hkv, D):
    """Rows of bytes to their values [..., Hkv, D] in 64 bits."""
    bits = rows[..., : Hkv * D].long()
    x = grid().to(rows.device)[bits & 127] * (1.0 - 2.0 * (bits >> 7))
    return x.unflatten(-1, (Hkv, D)) * two_to(rows[..., Hkv * D: Hkv * (D + 1)].int() - 127)[..., None]
