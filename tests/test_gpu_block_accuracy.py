"""GPU tests of what the calls around the 8-bit layers of an MLP block keep of their operands' range and bits, against 64-bit
forms (u = 2^-24, half a step of fp32; a rounding to bf16 adds 2^-8 of the value)."""
import pytest
import torch

import rotation_then_quantize_amd as rtq
from _fp8 import E4M3, groups

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U, HALF_BF16 = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    rtq.load_library()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def step(name, *what):
    print(name, *what, flush=True)


def near(got, want, bound):
    bound = bound + (HALF_BF16 * want.abs() if got.dtype == BF16 else 0.0)
    off = (got.double() - want).abs()
    assert (off <= bound).all(), float((off / bound.clamp(min=1e-300)).max())


def same(a, b):
    t = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.view(t), b.view(t))


# ------------------------------------------------------------------ norm

@pytest.mark.parametrize("T,d", [(6, 272), (9, 4112), (5, 8208), (3, 16400)])
@pytest.mark.parametrize("ht", [F32, BF16])
@pytest.mark.parametrize("at,eps", [(60, 1e-6), (100, 1e-6), (122, 1e-6), (-100, 1e-6), (-20, 1e-12), (-72, 2.0 ** -149)])
def test_norm_backward_far_from_one(T, d, ht, at, eps):
    """Rows of size 2^at, gradients of size 1.  dh = dr + rho (a - h k), a = gamma dn, k = rho^2 mean(a h): with rho and a
    rounded once each, k once from products that are, and two multiply-adds, each term is within 6 u of the terms'
    magnitudes; k and dh of less than 2^-126 are within 2^-150 of themselves.  dgamma: h rho has two roundings, a sum of T
    products is within (T + 4) u of the summed magnitudes."""
    step("norm backward far", T, d, ht, at, eps)
    h, dn = (randn(gen(T), T, d) * 2.0 ** at).to(ht), randn(gen(1), T, d)
    gamma = 1 + 0.3 * randn(gen(d), d)
    eps = float(torch.tensor(eps, dtype=F32))
    a, h64 = dn.double() * gamma.double(), h.double()
    rho = 1.0 / torch.sqrt(h64.square().mean(1, keepdim=True) + eps)
    want = rho * a - h64 * rho ** 3 * (a * h64).mean(1, keepdim=True)
    size = rho * a.abs() + h64.abs() * rho ** 3 * (a * h64).abs().mean(1, keepdim=True)
    terms = dn.double() * h64 * rho
    dh, dgamma = torch.empty(T, d, dtype=ht, device="cuda"), torch.empty(d, device="cuda")
    rtq.rmsnorm_backward(dn, h, gamma, eps, dh, dgamma=dgamma)
    near(dgamma, terms.sum(0), (T + 4) * U * terms.abs().sum(0))
    near(dh, want, 6 * U * size + 2.0 ** -149 * (1 + h64.abs() * rho) + (2.0 ** -134 if ht == BF16 else 0.0))


# ------------------------------------------------------------------ gated feed-forward

def quantised(x, w, st, general):
    """Codes and scales of x [T][K] and w [rows][K]; general: the scales (fp32) are no powers of two."""
    (T, K), rows = x.shape, w.shape[0]
    xc, xs = torch.empty(T, K, dtype=E4M3, device="cuda"), torch.empty(groups(K), T, dtype=st, device="cuda")
    wc, ws = torch.empty(rows, K, dtype=E4M3, device="cuda"), torch.empty(groups(rows), groups(K), dtype=st, device="cuda")
    rtq.fp8_quantize(x, xc, xs)
    rtq.fp8_quantize(w, wc, ws, blocks=True)
    if general:
        xs *= 0.75 + 0.5 * torch.rand(xs.shape, generator=gen(1), device="cuda")
        ws *= 0.75 + 0.5 * torch.rand(ws.shape, generator=gen(2), device="cuda")
    return xc, xs, wc, ws


@pytest.mark.parametrize("T,N,K", [(2100, 4096, 272), (4610, 2176, 2064)])
def test_scales_of_other_tokens_and_channels_change_nothing(T, N, K):
    """fp32 scales: the bits of a token's outputs of a channel go by its own operands alone, whether the scales beside are powers
    of two or not."""
    step("glu neighbours", T, N, K)
    xc, xs, wc, ws = quantised(randn(gen(T), T, K), randn(gen(N), 2 * N, K) / K ** 0.5, F32, False)
    y, z = torch.empty(T, N, device="cuda"), torch.empty(T, N, device="cuda")
    rtq.fp8_glu(xc, xs, wc, ws, rtq.RTQ_ACT_SILU, y=y)
    for token in (0, 700, T - 1):
        odd = xs.clone()
        odd[:, token] *= 1.25
        rtq.fp8_glu(xc, odd, wc, ws, rtq.RTQ_ACT_SILU, y=z)
        rest = torch.arange(T, device="cuda") != token
        assert same(z[rest], y[rest]), token
    for block in (1, N // 128 + 3):
        odd = ws.clone()
        odd[block, -1] *= 1.25
        rtq.fp8_glu(xc, xs, wc, odd, rtq.RTQ_ACT_SILU, y=z)
        rest = torch.arange(N, device="cuda") // 128 != block % (N // 128)
        assert same(z[:, rest], y[:, rest]), block
