"""Plain 64-bit forms of the calls around the 8-bit layers of an MLP block (norm, gated feed-forward, clipping), on the
tensors' own device, written from the definitions in include/rtq.h and sharing nothing with the library."""
import torch

from _fp8 import E4M3, TOP, act, groups, round_to, slope

EPS = 1e-6


def rms(h):
    return 1.0 / torch.sqrt(h.double().square().mean(1, keepdim=True) + EPS)


def norm(h, gamma):
    return h.double() * rms(h) * gamma.double()


def norm_gradients(dn, h, gamma, dresidual=None):
    """(dh, dgamma, the sums of the magnitudes that either is made of)."""
    dn, h, gamma = dn.double(), h.double(), gamma.double()
    rho, a = rms(h), dn * gamma
    back = rho ** 3 * (a * h).mean(1, keepdim=True)
    dr = torch.zeros_like(h) if dresidual is None else dresidual.double()
    size = dr.abs() + rho * a.abs() + h.abs() * rho ** 3 * (a * h).abs().mean(1, keepdim=True)
    terms = dn * h * rho
    return dr + rho * a - h * back, terms.sum(0), size, terms.abs().sum(0)


def glu(h, name):
    N = h.shape[1] // 2
    return act(h[:, :N], name) * h[:, N:]


def glu_gradient(dy, h, name):
    N, dy = h.shape[1] // 2, dy.double()
    return torch.cat([dy * h[:, N:] * slope(h[:, :N], name), dy * act(h[:, :N], name)], 1)


def scales_of(m, fmt):
    """The group scales for largest magnitudes m (float64 tensor): smallest 2^e >= 2^-120 with m <= top 2^e."""
    e = torch.ceil(torch.log2(m.clamp(min=1e-300) / TOP[fmt])).clamp(min=-120)
    e = torch.where(m > TOP[fmt] * torch.exp2(e), e + 1, torch.where((m <= TOP[fmt] * torch.exp2(e - 1)) & (e > -120), e - 1, e))
    return torch.where(m > 0, torch.exp2(e), torch.ones_like(m))


def check_codes(codes, scale, exact, off, fmt=E4M3):
    """Codes and scales are those of numbers within `off` (absolute, a tensor like exact) of the exact ones: each scale is
    the rule's for a largest magnitude in that range, and each code the rounding of a number in its range."""
    T, d = exact.shape
    g = groups(d)
    pad = torch.nn.functional.pad
    mag, o = pad(exact.abs(), (0, g * 128 - d)).view(T, g, 128), pad(off, (0, g * 128 - d)).view(T, g, 128)
    lo, hi = scales_of((mag - o).clamp(min=0).amax(2), fmt).t(), scales_of((mag + o).amax(2), fmt).t()
    s = scale.double()
    assert s.shape == lo.shape
    assert ((s == lo) | (s == hi)).all(), "scales"
    per = s.t().repeat_interleave(128, 1)[:, :d]
    c = codes.double()
    top = TOP[fmt]
    below = round_to(((exact - off) / per).clamp(-top, top), fmt)
    above = round_to(((exact + off) / per).clamp(-top, top), fmt)
    assert ((c >= below) & (c <= above)).all(), "codes"
