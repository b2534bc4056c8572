"""GPU tests of what the calls around the 8-bit layers of an MLP block keep of their operands' range and bits, against 64-bit
forms (u = 2^-24, half a step of fp32; a rounding to bf16 adds 2^-8 of the value)."""
import pytest
import torch

import rotation_then_quantize_amd as rtq

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
