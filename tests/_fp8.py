"""Plain 64-bit forms of the 8-bit floating point layer (scales for blocks of 128), on the CPU, written
from the definitions in include/rtq.h and sharing nothing with the library."""
import math

import torch

E4M3, E5M2, E8M0 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu
TOP = {E4M3: 448.0, E5M2: 57344.0}
MANTISSA = {E4M3: 3, E5M2: 2}
LOW = {E4M3: -6, E5M2: -14}     # exponent of the smallest normal code


def groups(d):
    return -(-d // 128)


def round_to(v, fmt):
    """v (float64, |v| <= top) to the nearest code's value, ties to even."""
    lead = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** LOW[fmt])))
    step = torch.exp2(lead - MANTISSA[fmt])
    return torch.round(v / step) * step


def scale_of(m, fmt):
    """The block scale for a largest finite magnitude m (a float): smallest 2^e >= 2^-120 with m <= top 2^e."""
    if m == 0.0:
        return 1.0
    e = -120
    while math.ldexp(TOP[fmt], e) < m:
        e += 1
    return math.ldexp(1.0, e)


def quantise(x, fmt, blocks=False):
    """(codes' values, scales): scales [groups][rows], or with blocks [row blocks][column blocks]."""
    x = x.double()
    rows, d = x.shape
    q = torch.empty_like(x)
    rb = 128 if blocks else 1
    s = torch.empty(groups(d), rows, dtype=torch.float64) if not blocks else \
        torch.empty(groups(rows), groups(d), dtype=torch.float64)
    for i in range(0, rows, rb):
        for j in range(groups(d)):
            part = x[i:i + rb, 128 * j:128 * j + 128]
            finite = part[torch.isfinite(part)]
            sc = scale_of(float(finite.abs().max()) if finite.numel() else 0.0, fmt)
            v = round_to(torch.where(torch.isfinite(part), part / sc, torch.zeros_like(part)), fmt)
            bad = torch.full_like(part, math.nan) if fmt == E4M3 else part
            q[i:i + rb, 128 * j:128 * j + 128] = torch.where(torch.isfinite(part), v, bad)
            if blocks:
                s[i // 128, j] = sc
            else:
                s[j, i] = sc
    return q, s


def row_values(codes, scale):
    """The values that row-group codes stand for (float64)."""
    v = codes.cpu().double()
    return v * scale.cpu().double().t().repeat_interleave(128, 1)[:, :v.shape[1]]


def block_values(codes, scale):
    v = codes.cpu().double()
    s = scale.cpu().double().repeat_interleave(128, 0)[:v.shape[0]]
    return v * s.repeat_interleave(128, 1)[:, :v.shape[1]]


def act(h, name):
    if name == "silu":
        return h * torch.sigmoid(h)
    if name == "gelu":
        return 0.5 * h * torch.erfc(-h / math.sqrt(2.0))
    return h * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (h + 0.044715 * h ** 3))


def slope(h, name):
    h = h.clone().requires_grad_(True)
    (g,) = torch.autograd.grad(act(h, name).sum(), h)
    return g


def rel(a, b):
    a, b = a.cpu().double(), b.cpu().double()
    return float((a - b).norm() / b.norm().clamp(min=1e-300))
