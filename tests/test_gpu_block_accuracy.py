"""GPU tests of what the calls around the 8-bit layers of an MLP block keep of their operands' range and bits, against 64-bit
forms (u = 2^-24, half a step of fp32; a rounding to bf16 adds 2^-8 of the value)."""
import pytest
import torch

import rotation_then_quantize_amd as rtq
from _block import check_codes, glu
from _fp8 import E4M3, E8M0, groups, rel

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


@pytest.mark.parametrize("T,d", [(6, 272), (3, 16400)])
def test_norm_of_the_largest_rows(T, d):
    """Past a root mean square of 2^126, rho has down to 22 bits: within 2^-22, with the products by h and gamma 6 u."""
    step("norm largest", T, d)
    x = (1 + torch.rand(T, d, generator=gen(T), device="cuda")) * 2.0 ** 126.99
    x[0] = -3.3e38
    gamma, y = 1 + 0.3 * randn(gen(d), d), torch.empty(T, d, device="cuda")
    rtq.rmsnorm_forward(x, gamma, 1e-6, y=y)
    want = x.double() / torch.sqrt(x.double().square().mean(1, keepdim=True)) * gamma.double()
    near(y, want, 8 * U * want.abs())


# ------------------------------------------------------------------ gated feed-forward

# few tokens as weights stream, sums of split parts, tiles of 32, 64 and 128 tokens, and large ones of short and long reductions
SIZES = [(13, 2560, 4096), (2, 128, 16384), (64, 1024, 1040), (300, 512, 4112), (230, 2048, 2064), (450, 2304, 2064),
         (2100, 2048, 1040), (2100, 2048, 16384)]


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


def values(xc, xs, wc, ws):
    rows, K = wc.shape
    return (xc.double() * xs.double().t().repeat_interleave(128, 1)[:, :K],
            wc.double() * ws.double().repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :K])


def largest(v):
    """The largest magnitude of each row's blocks of 128."""
    return torch.nn.functional.pad(v.abs(), (0, groups(v.shape[1]) * 128 - v.shape[1])).view(v.shape[0], -1, 128).amax(2)


def off_of(xv, wv, inside):
    """What the products' sums may be off by, elementwise: in each block of 128 the matrix instruction cuts a product off below
    2^-14 of the largest one, which is at most the product of the rows' largest; a block's sum is scaled (a rounding for the
    scales' product, one for the multiply-add) and added in fp32; inside the instruction (large outputs with E8M0 scales) each
    block cuts up to 2^-20 of the running sum off."""
    blocks = groups(xv.shape[1])
    per = (blocks + 3) * U + (blocks * 2.0 ** -20 if inside else 0.0)
    return 128 * 2.0 ** -14 * (largest(xv) @ largest(wv).t().contiguous()) + per * (xv.abs() @ wv.abs().t().contiguous())


def norm_bound(K, inside):
    """The sums' error in the 2-norm as the header states it."""
    return 4e-5 + (groups(K) * 2.0 ** -20 if inside else 0.0)


def kinds(f):
    return pytest.mark.parametrize("st,general", [(F32, True), (F32, False), (E8M0, False)])(f)


@kinds
@pytest.mark.parametrize("one_sign", [False, True])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_sums_of_the_gated_product(T, N, K, st, general, one_sign):
    """The gate is a number of 32 or more that is exact in every form (one product), where SiLU is the identity, so that y / g is
    the other projection's sum."""
    step("glu sums", T, N, K, st, general, one_sign)
    x, w = randn(gen(T), T, K), torch.zeros(2 * N, K, device="cuda")
    w[N:] = randn(gen(N), N, K) / K ** 0.5
    if one_sign:
        x, w = x.abs(), w.abs()
    x[:, 0], w[:N, 0] = 2.0, 2.0 ** 12
    ops = quantised(x, w, st, general)
    xv, wv = values(*ops)
    g = xv[:, :1] * wv[:N, :1].t()
    u = xv @ wv[N:].t().contiguous()
    assert float(g.min()) >= 32
    y = torch.empty(T, N, device="cuda")
    rtq.fp8_glu(*ops, rtq.RTQ_ACT_SILU, y=y)
    got, inside = y.double() / g, T == 2100 and st == E8M0
    near(got, u, off_of(xv, wv[N:], inside) + 6 * U * u.abs())      # g's two roundings, the sigmoid's and the product's
    assert rel(got, u) <= norm_bound(K, inside) + 6 * U


@kinds
@pytest.mark.parametrize("T,N,K", SIZES)
def test_gated_product_of_codes_of_the_whole_range(T, N, K, st, general):
    """y, its codes and the checkpoint's against 64 bits, each within what the sums may be off by.  |f'| of SiLU is at most
    1.1, |f(z)| at most |z|."""
    step("glu range", T, N, K, st, general)
    x = randn(gen(T), T, K) * torch.exp(0.5 * randn(gen(5), T, K))
    ops = quantised(x, randn(gen(N), 2 * N, K) / K ** 0.5, st, general)
    xv, wv = values(*ops)
    h = xv @ wv.t().contiguous()
    inside = T == 2100 and st == E8M0
    off = off_of(xv, wv, inside)
    del xv, wv
    g, u, want = h[:, :N], h[:, N:], glu(h, "silu")
    off_y = (3 * g.abs() + 6) * 2.0 ** -23 * want.abs() + 1.1 * off[:, :N] * (u.abs() + off[:, N:]) + g.abs() * off[:, N:]
    y = torch.empty(T, N, device="cuda")
    rtq.fp8_glu(*ops, rtq.RTQ_ACT_SILU, y=y)
    near(y, want, off_y)
    # |dy| <= 1.1 |u| |dg| + |f| |du|: with |u| and |g| independent of the errors, three times the sums'
    assert rel(y, want) <= 3 * norm_bound(K, inside)
    yc, ys = torch.empty(T, N, dtype=E4M3, device="cuda"), torch.empty(groups(N), T, dtype=st, device="cuda")
    hc, hs = torch.empty(T, 2 * N, dtype=E4M3, device="cuda"), torch.empty(groups(2 * N), T, dtype=st, device="cuda")
    rtq.fp8_glu(*ops, rtq.RTQ_ACT_SILU, y_codes=yc, y_scale=ys, h_codes=hc, h_scale=hs)
    check_codes(hc.float(), hs.float(), h, off)
    check_codes(yc.float(), ys.float(), want, off_y)


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


@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("T,N", [(2, 384), (64, 1024), (450, 2304), (2100, 4096)])
def test_small_blocks_beside_a_large_one(T, N, st):
    """Blocks whose products of 16 are three quarters of the running sum's last place: with fp32 scales their sums are added
    whole, all numbers here being exact in fp32 (the gate is 32, where SiLU is the identity); with E8M0 scales a large output may
    lose 2^-20 of the running sum for each block."""
    step("glu small blocks", T, N, st)
    K, blocks = 1024, 8
    x, w = torch.zeros(T, K, device="cuda"), torch.zeros(2 * N, K, device="cuda")
    x[:, 0], w[:N, 0], w[N:, 0] = 1.0, 2.0 ** -5, 1.0
    x[:, 128:], w[N:, 128:] = 1.0, 1.5
    xs, ws = torch.ones(blocks, T, device="cuda"), torch.ones(groups(2 * N), blocks, device="cuda")
    xs[0], ws[:N // 128, 0], xs[1:] = 2.0 ** 10, 1.0, 2.0 ** -7
    ws[N // 128:, 0] = 2.0 ** 11
    y = torch.empty(T, N, device="cuda")
    rtq.fp8_glu(x.to(E4M3), xs.to(st), w.to(E4M3), ws.to(st), rtq.RTQ_ACT_SILU, y=y)
    want = 32.0 * (2.0 ** 21 + 7 * 1.5)
    if T == 2100 and st == E8M0:
        assert ((y <= want) & (y >= want * (1 - 7 * 2.0 ** -20))).all()
    else:
        assert (y == want).all(), float((y.double() - want).abs().max())
