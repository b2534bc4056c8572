"""GPU tests of the longest rows, reductions and widths that the calls around the 8-bit layers of an MLP block take, against
64-bit forms of some of the tokens (u = 2^-24, half a step of fp32)."""
import pytest
import torch

import rotation_then_quantize_amd as rtq
from _block import EPS, check_codes, glu, norm, norm_gradients
from _fp8 import E4M3, groups

pytestmark = pytest.mark.gpu
F32, U = torch.float32, 2.0 ** -24


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def near(got, want, bound):
    off = (got.double() - want).abs()
    assert (off <= bound).all(), float((off - bound).max())


def test_longest_rows_of_the_norm():
    T, d = 3, 1 << 20
    print("norm", T, d, flush=True)
    x, r = torch.randn(T, d, generator=gen(1), device="cuda"), torch.randn(T, d, generator=gen(2), device="cuda")
    gamma = 1 + 0.3 * torch.randn(d, generator=gen(3), device="cuda")
    h, y = torch.empty_like(x), torch.empty_like(x)
    codes, scale = torch.empty(T, d, dtype=E4M3, device="cuda"), torch.empty(groups(d), T, device="cuda")
    rtq.rmsnorm_forward(x, gamma, EPS, residual=r, h=h, codes=codes, scale=scale, y=y)
    assert torch.equal(h, x + r)
    n = norm(h, gamma)
    near(y, n, 4 * U * n.abs())
    check_codes(codes.float(), scale, n, 4 * U * n.abs())
    dn = torch.randn(T, d, generator=gen(4), device="cuda")
    dh, dgamma = torch.empty_like(x), torch.empty(d, device="cuda")
    rtq.rmsnorm_backward(dn, h, gamma, EPS, dh, dgamma=dgamma, dresidual=r)
    want, want_g, size, size_g = norm_gradients(dn, h, gamma, r)
    near(dh, want, 6 * U * size)
    near(dgamma, want_g, (T + 4) * U * size_g)


# widest layer; longest reductions of few tokens, of sums, of tiles of 128 tokens and of large ones
@pytest.mark.parametrize("T,N,K", [(1, 1 << 19, 144), (18, 1 << 19, 80), (3, 128, 1 << 20), (16, 4096, 1 << 17), (40, 128, 1 << 20),
                                   (450, 2304, 1 << 17), (2100, 2048, 1 << 17)])
def test_longest_reductions_and_widest_layers(T, N, K):
    """Whole-number codes to 4 and power-of-two scales of 2^-11 to 2^-5 together: products are multiples of 2^-11, and sums of
    2^20 random ones stay below 2^13, so that fp32 has them exactly."""
    print("glu", T, N, K, flush=True)
    g = gen(T + N + K)
    whole = lambda rows: torch.randint(-4, 5, (rows, K), generator=g, device="cuda", dtype=torch.int8).half().to(E4M3)
    x, w = whole(T), whole(2 * N)
    sx = torch.exp2(torch.randint(-6, -3, (groups(K), T), generator=g, device="cuda").float())
    sw = torch.exp2(torch.randint(-5, -2, (groups(2 * N), groups(K)), generator=g, device="cuda").float())
    y = torch.empty(T, N, device="cuda")
    rtq.fp8_glu(x, sx, w, sw, rtq.RTQ_ACT_SILU, y=y)
    rows = torch.tensor(sorted({0, T // 2, T - 1}), device="cuda")
    xv = x[rows].double() * sx[:, rows].double().t().repeat_interleave(128, 1)[:, :K]
    h = torch.empty(len(rows), 2 * N, dtype=torch.float64, device="cuda")
    for a in range(0, 2 * N, 1024):
        b = min(a + 1024, 2 * N)
        wv = w[a:b].double() * sw[a // 128:-(-b // 128)].double().repeat_interleave(128, 0)[:b - a].repeat_interleave(128, 1)[:, :K]
        h[:, a:b] = xv @ wv.t().contiguous()
    want = glu(h, "silu")
    # f within (3 |g| + 4) 2^-23, the product one more
    near(y[rows], want, (3 * h[:, :N].abs() + 6) * 2.0 ** -23 * want.abs() + 2.0 ** -119 * (1 + h[:, N:].abs()))
