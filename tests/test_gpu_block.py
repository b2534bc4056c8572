"""GPU tests of the calls around the 8-bit layers of an MLP block against plain 64-bit forms.

Tolerances, counted in roundings (u = 2^-24, half a step of fp32; a rounding to bf16 adds 2^-8 of the value):
  norm       rho, h rho and the product with gamma are rounded once each and rho is within u of its own: n is within 4 u.
  dh         gamma dn, rho, k = rho^3 mean(a h) and the two multiply-adds: each term is within 6 u of the terms' magnitudes.
  dgamma     a sum of T products of two roundings: within (T + 4) u of the summed magnitudes.
  f(g) u     f within (3 |z| + 4) 2^-23 as the header says (z: the exponential's argument), the product one more; the
             slope has a few more terms of that size: (3 |z| + 12) 2^-23 of the terms' magnitudes.
  products   whole-number operands are exact in fp32; general ones are within 2^-9 in the 2-norm (the matrix unit's alignment),
             and f(g) u moves by at most |f'| |u| |dg| + |f| |du|, which is three times that for g of a normal distribution.
  clip       the norm is rounded once; norm + 1e-6, the quotient and the product: 4 u, then the type's rounding.
Codes and scales have to be those of some number in that range (_block.check_codes)."""
import pytest
import torch

import rotation_then_quantize_amd as rtq
from _block import EPS, check_codes, glu, glu_gradient, norm, norm_gradients
from _fp8 import E4M3, E5M2, E8M0, act, groups, rel

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ACTS = {"gelu_tanh": rtq.RTQ_ACT_GELU_TANH, "gelu": rtq.RTQ_ACT_GELU, "silu": rtq.RTQ_ACT_SILU}
U, HALF_BF16, GENERAL = 2.0 ** -24, 2.0 ** -8, 2.0 ** -9
TINY = 2.0 ** -119      # what may come out as 0


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    rtq.load_library()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def rows_like(seed, T, d, dtype=BF16):
    """Heavy-tailed rows with a zero group and an outlier."""
    g = gen(seed)
    x = randn(g, T, d) * torch.exp(randn(g, T, d))
    if T > 2:
        x[1, :128] = 0.0
        x[2, d // 2] = 300.0
    return x.to(dtype)


def step(name, *what):
    print(name, *what, flush=True)


def near(got, want, bound):
    """|got - want| <= bound, elementwise; bound for got's type is the caller's but for its rounding."""
    bound = bound + (HALF_BF16 * want.abs() if got.dtype == BF16 else 0.0)
    off = (got.double() - want).abs()
    assert (off <= bound).all(), float((off - bound).max())


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def same(a, b):
    return torch.equal(bits(a), bits(b))


def empty_rows(T, d, fmt=E4M3, st=F32):
    return torch.empty(T, d, dtype=fmt, device="cuda"), torch.empty(groups(d), T, dtype=st, device="cuda")


# ------------------------------------------------------------------ norm

LENGTHS = [(1, 16), (1, 4096), (3, 528), (130, 128), (5, 1024), (9, 1040), (70, 2064), (33, 4112), (7, 8192), (5, 8208), (4, 16384),
           (3, 16400), (2, 40000)]


@pytest.mark.parametrize("T,d", LENGTHS)
@pytest.mark.parametrize("xt,rt", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16), (BF16, None), (F32, None)])
def test_norm(T, d, xt, rt):
    step("norm", T, d, xt, rt)
    x = rows_like(T + d, T, d, xt)
    for gt, st in ((BF16, E8M0), (F32, F32)):
        gamma = (1 + 0.3 * randn(gen(d), d)).to(gt)
        if rt is None:
            r, h, want_h = None, None, x
        else:
            r = (3 * rows_like(T * d, T, d, F32)).to(rt)
            want_h = (x.float() + r.float()).to(rt)
            h = torch.full((T + 1, d), 7.0, dtype=rt, device="cuda")
        codes = torch.zeros(T + 1, d, dtype=torch.uint8, device="cuda").view(E4M3)
        scale = torch.empty(groups(d), T, dtype=st, device="cuda")
        y = torch.full((T + 1, d), 7.0, dtype=xt, device="cuda")
        rtq.rmsnorm_forward(x, gamma, EPS, residual=r, h=None if h is None else h[:T], codes=codes[:T], scale=scale, y=y[:T])
        if h is not None:
            assert same(h[:T], want_h) and (h[T] == 7.0).all()      # the row behind the last stays as it was
        n = norm(want_h, gamma)
        near(y[:T], n, 4 * U * n.abs())
        check_codes(codes[:T].float(), scale.float(), n, 4 * U * n.abs())
        assert not codes[T].view(torch.uint8).any() and (y[T] == 7.0).all()
        # either output alone, and the residual stream in place, give the same
        c2, s2 = empty_rows(T, d, st=st)
        own = None if r is None else r.clone()
        rtq.rmsnorm_forward(x, gamma, EPS, residual=own, h=own, codes=c2, scale=s2)
        assert same(c2, codes[:T].contiguous()) and same(s2, scale) and (own is None or same(own, want_h))
        y2 = torch.empty(T, d, dtype=xt, device="cuda")
        if r is not None and rt == xt:
            own = x.clone()
            rtq.rmsnorm_forward(own, gamma, EPS, residual=r, h=own, y=y2)     # over the branch's output
            assert same(own, want_h)
        else:
            rtq.rmsnorm_forward(x, gamma, EPS, residual=r, h=None if r is None else h[:T], y=y2)
        assert same(y2, y[:T].contiguous())
        own = x.clone()
        rtq.rmsnorm_forward(own, gamma, EPS, residual=r, h=None if r is None else h[:T], y=own)
        assert same(own, y2)


@pytest.mark.parametrize("T,d", [(4608, 4096), (2050, 208), (8190, 16)])
def test_norm_many_rows(T, d):
    step("norm many", T, d)
    x, r, gamma = rows_like(1, T, d), rows_like(2, T, d, F32), (1 + 0.3 * randn(gen(d), d)).to(BF16)
    h, (codes, scale) = torch.empty(T, d, device="cuda"), empty_rows(T, d, st=E8M0)
    rtq.rmsnorm_forward(x, gamma, EPS, residual=r, h=h, codes=codes, scale=scale)
    assert same(h, x.float() + r)
    n = norm(h, gamma)
    check_codes(codes.float(), scale.float(), n, 4 * U * n.abs())


def test_norm_extreme_rows():
    """Rows of zeros, of the largest and the smallest numbers, a large eps; NaN and infinity stay in their row."""
    step("norm extreme")
    d = 272
    for dtype in (F32, BF16):
        base = randn(gen(5), 9, d).clamp(-2, 2)
        base[1] = 0.0
        base[2] *= 2.0 ** 126
        base[3] *= 2.0 ** -100
        base[4] = 0.0
        base[4, 100] = 2.0 ** 127
        x = base.to(dtype)
        x[6, 5] = float("nan")
        x[7, 9] = float("inf")
        gamma = (1 + 0.3 * randn(gen(d), d))
        y = torch.empty(9, d, dtype=dtype, device="cuda")
        codes, scale = empty_rows(9, d)
        rtq.rmsnorm_forward(x, gamma, EPS, y=y, codes=codes, scale=scale)
        rows = [0, 1, 2, 3, 4, 5, 8]
        n = norm(x[rows], gamma)
        # (what is smaller than the smallest normal number has fewer bits)
        near(y[rows], n, 4 * U * n.abs() + 2.0 ** -126)
        check_codes(codes[rows].float(), scale[:, rows], n, 4 * U * n.abs() + 2.0 ** -126)
        assert torch.isnan(y[6]).all() and torch.isnan(y[7, 9]) and (torch.isnan(y[7]) | (y[7] == 0)).all()
        assert torch.isnan(codes[6].float()).all()
    z = torch.empty(9, d, device="cuda")
    rtq.rmsnorm_forward(base, gamma, 3.0, y=z)
    want = base.double() / torch.sqrt(base.double().square().mean(1, keepdim=True) + 3.0) * gamma.double()
    near(z, want, 4 * U * want.abs() + 2.0 ** -126)


@pytest.mark.parametrize("T,d", LENGTHS + [(600, 1936), (4608, 512)])
@pytest.mark.parametrize("nt,ht", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
def test_norm_backward(T, d, nt, ht):
    step("norm backward", T, d, nt, ht)
    h, dn = (3 * rows_like(T + d, T, d, F32)).to(ht), (1e-3 * randn(gen(1), T, d)).to(nt)
    for gt, dgt, with_dr in ((BF16, F32, True), (F32, BF16, False)):
        gamma = (1 + 0.3 * randn(gen(d), d)).to(gt)
        dr = (1e-3 * randn(gen(2), T, d)).to(ht) if with_dr else None
        want, want_g, size, size_g = norm_gradients(dn, h, gamma, dr)
        dh = torch.full((T + 1, d), 7.0, dtype=ht, device="cuda")
        dgamma = torch.full((d,), 7.0, dtype=dgt, device="cuda")
        rtq.rmsnorm_backward(dn, h, gamma, EPS, dh[:T], dgamma=dgamma, dresidual=dr)
        near(dh[:T], want, 6 * U * size)
        assert (dh[T] == 7.0).all()
        near(dgamma, want_g, (T + 4) * U * size_g)
        start = randn(gen(4), d).to(dgt)
        added = start.clone()
        need = rtq.rmsnorm_backward_workspace(T, d)
        ws = torch.zeros(need + 64, dtype=torch.uint8, device="cuda")
        again = torch.empty(T, d, dtype=ht, device="cuda")
        rtq.rmsnorm_backward(dn, h, gamma, EPS, again, dgamma=added, dresidual=dr, accumulate=True, workspace=ws[:need])
        near(added, want_g + start.double(), (T + 5) * U * (size_g + start.double().abs()))
        assert same(again, dh[:T].contiguous()) and not ws[need:].any()      # nothing past the size asked for
        if dr is not None:
            rtq.rmsnorm_backward(dn, h, gamma, EPS, dr, dresidual=dr)         # in place, without dgamma
            assert same(dr, again)
        elif nt == ht:
            own = dn.clone()
            rtq.rmsnorm_backward(own, h, gamma, EPS, own)
            assert same(own, again)


def test_norm_backward_without_rows():
    step("norm backward T=0")
    e, gamma = torch.empty(0, 48, device="cuda"), torch.ones(48, device="cuda")
    dgamma = torch.full((48,), 7.0, device="cuda")
    rtq.rmsnorm_backward(e, e, gamma, EPS, torch.empty(0, 48, device="cuda"), dgamma=dgamma, accumulate=True)
    assert (dgamma == 7.0).all()
    rtq.rmsnorm_backward(e, e, gamma, EPS, torch.empty(0, 48, device="cuda"), dgamma=dgamma)
    assert (dgamma == 0.0).all()


# ------------------------------------------------------------------ gated feed-forward

def glu_operands(T, N, K, st, by=1.0):
    """Whole-number codes to 4 and power-of-two scales, the weights' times `by`: sums are exact in fp32, of some hundredths to
    tens."""
    g = gen(T + N + K)
    x = torch.randint(-4, 5, (T, K), generator=g, device="cuda").float().to(E4M3)
    w = torch.randint(-4, 5, (2 * N, K), generator=g, device="cuda").float().to(E4M3)
    sx = torch.exp2(torch.randint(-6, -3, (groups(K), T), generator=g, device="cuda").float())
    sw = by * torch.exp2(torch.randint(-5, -2, (groups(2 * N), groups(K)), generator=g, device="cuda").float())
    xv = x.double() * sx.double().t().repeat_interleave(128, 1)[:, :K]
    wv = w.double() * sw.double().repeat_interleave(128, 0).repeat_interleave(128, 1)[:, :K]
    return (x, sx.to(st), w, sw.to(st)), xv @ wv.t().contiguous()


def act_bound(h, name, terms=12):
    """(3 |z| + terms) 2^-23 for each of the gate's channels."""
    N = h.shape[1] // 2
    g = h[:, :N].abs()
    z = {"silu": g, "gelu": g * g, "gelu_tanh": 1.6 * g * (1 + 0.0448 * g * g)}[name]
    return (3 * z + terms) * 2.0 ** -23


GLU_SIZES = [(1, 128, 16), (1, 16384, 256), (2, 128, 272), (5, 1152, 1936), (13, 2560, 4096), (16, 256, 144), (17, 128, 400), (64, 384, 128),
             (65, 1152, 528), (130, 256, 4112), (257, 512, 640), (391, 1152, 1936), (600, 4096, 272), (1030, 1920, 400)]


@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("T,N,K", GLU_SIZES)
def test_glu(T, N, K, st):
    name = ("silu", "gelu", "gelu_tanh")[(T + K // 16) % 3]
    check_glu(T, N, K, st, name)


@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("T,N,K", [(16, 14336, 528), (2, 32896, 272), (17, 4096, 1296), (32, 4096, 2064), (31, 8192, 1040), (20, 10880, 1168),
                                   (27, 16384, 2064), (32, 33280, 2320)])
def test_glu_few_tokens(T, N, K, st):
    """One or two tiles of tokens, one to four of channels a workgroup, the last one's in part."""
    check_glu(T, N, K, st, "gelu_tanh")


@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("T,N,K", [(33, 128, 16), (63, 1152, 1680), (391, 1152, 2048), (230, 4096, 1024), (64, 10880, 2192), (520, 2048, 144),
                                   (450, 2304, 528), (1000, 2048, 400)])
def test_glu_few_tiles(T, N, K, st):
    """Tiles of 32, 64 and 128 tokens, the last one's in part."""
    check_glu(T, N, K, st, "silu")


@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T,N,K", [(9, 384, 528), (300, 2048, 400), (2100, 4096, 272)])
def test_glu_activations(T, N, K, st, name):
    check_glu(T, N, K, st, name)


@pytest.mark.parametrize("st,by", [(F32, 1.0), (F32, 1.5), (E8M0, 1.0)])
@pytest.mark.parametrize("T,N,K", [(4608, 2176, 640), (4099, 4096, 144), (2500, 2816, 2064), (8300, 1152, 272), (1500, 16384, 384),
                                   (4608, 1024, 112)])
def test_glu_large(T, N, K, st, by):
    """Whole rounds of tiles and parts of one, few blocks of the reduction and many, ragged last rows; scales inside the
    instruction and outside."""
    check_glu(T, N, K, st, "silu", by)


def check_glu(T, N, K, st, name, by=1.0):
    step("glu", T, N, K, st, name, by)
    dev, h = glu_operands(T, N, K, st, by)
    want = glu(h, name)
    off = act_bound(h, name) * want.abs() + TINY * (1 + h[:, N:].abs())
    need = rtq.fp8_glu_workspace(T, N, K)
    ws = torch.zeros(need + 64, dtype=torch.uint8, device="cuda")
    for dtype, keep in ((F32, False), (BF16, True), (None, False), (None, True)):
        y = y_codes = y_scale = h_codes = h_scale = None
        if keep:
            h_codes = torch.zeros(T + 1, 2 * N, dtype=torch.uint8, device="cuda").view(E4M3)
            h_scale = torch.empty(groups(2 * N), T, dtype=st, device="cuda")
        if dtype is None:
            y_codes = torch.zeros(T + 1, N, dtype=torch.uint8, device="cuda").view(E4M3)
            y_scale = torch.empty(groups(N), T, dtype=st, device="cuda")
        else:
            y = torch.full((T + 1, N), 7.0, dtype=dtype, device="cuda")
        rtq.fp8_glu(*dev, ACTS[name], y=None if y is None else y[:T], y_codes=None if y_codes is None else y_codes[:T], y_scale=y_scale,
                    h_codes=None if h_codes is None else h_codes[:T], h_scale=h_scale, workspace=ws[:need])
        if y is not None:
            near(y[:T], want, off)
            assert (y[T] == 7.0).all()                   # the row behind the last stays as it was
        else:
            check_codes(y_codes[:T].float(), y_scale.float(), want, off)
            assert not y_codes[T].view(torch.uint8).any()
        if keep:
            check_codes(h_codes[:T].float(), h_scale.float(), h, torch.zeros_like(h))
            assert not h_codes[T].view(torch.uint8).any()
    assert not ws[need:].any()                            # nothing past the size asked for


@pytest.mark.parametrize("odd", [3.0, 0.0, -1.0, 2.0 ** -140, 2.0 ** -126])
@pytest.mark.parametrize("T,N,K", [(2100, 4096, 272), (4610, 2176, 2064)])
def test_glu_large_with_an_odd_scale(T, N, K, odd):
    """One scale among powers of two that is none, or at the ends of their range, of a token or of a block of weights."""
    step("glu odd scale", T, N, K, odd)
    for rows, at in ((1, (-1, T - 1)), (1, (0, 700)), (3, (N // 128 + 5, 1)), (3, (2, -1))):
        dev, _ = glu_operands(T, N, K, F32)
        dev[rows][at] = odd
        x, sx, w, sw = (t.double() for t in dev)
        xv, wv = x * sx.t().repeat_interleave(128, 1)[:, :K], w * sw.repeat_interleave(128, 0).repeat_interleave(128, 1)[:, :K]
        h = xv @ wv.t().contiguous()
        y = torch.empty(T, N, device="cuda")
        rtq.fp8_glu(*dev, ACTS["silu"], y=y)
        want = glu(h, "silu")
        lost = 0.0
        if 0.0 < odd < 2.0 ** -100:    # each of a block's eight additions may cut the running sum off by a unit of its last place
            most = 8 * 2.0 ** -23 * (xv.abs() @ wv.abs().t().contiguous())
            lost = 1.1 * h[:, N:].abs() * most[:, :N] + h[:, :N].abs() * most[:, N:] + 1.1 * most[:, :N] * most[:, N:]
        near(y, want, act_bound(h, "silu") * want.abs() + TINY * (1 + h[:, N:].abs()) + lost)


@pytest.mark.parametrize("T,N,K", [(1, 512, 2048), (16, 256, 4096), (30, 4096, 2064), (100, 384, 1040), (300, 512, 2064), (1100, 4096, 1040)])
def test_glu_general(T, N, K):
    """General fp32 scales and codes over the whole range; equal calls give equal bits."""
    step("glu general", T, N, K)
    x, sx = empty_rows(T, K)
    rtq.fp8_quantize(rows_like(T, T, K), x, sx)
    w, sw = torch.empty(2 * N, K, dtype=E4M3, device="cuda"), torch.empty(groups(2 * N), groups(K), device="cuda")
    rtq.fp8_quantize(randn(gen(N), 2 * N, K) * 0.5 / K ** 0.5, w, sw, blocks=True)
    sx *= 0.75 + 0.5 * torch.rand(sx.shape, generator=gen(1), device="cuda")
    sw *= 0.75 + 0.5 * torch.rand(sw.shape, generator=gen(2), device="cuda")
    xv = x.double() * sx.double().t().repeat_interleave(128, 1)[:, :K]
    wv = w.double() * sw.double().repeat_interleave(128, 0).repeat_interleave(128, 1)[:, :K]
    h = xv @ wv.t().contiguous()
    y = torch.empty(T, N, device="cuda")
    rtq.fp8_glu(x, sx, w, sw, ACTS["silu"], y=y)
    assert rel(y, glu(h, "silu")) <= 3 * GENERAL
    again, hc, hs = torch.empty(T, N, device="cuda"), *empty_rows(T, 2 * N)
    rtq.fp8_glu(x, sx, w, sw, ACTS["silu"], y=again, h_codes=hc, h_scale=hs)
    assert same(again, y)
    hq = hc.double() * hs.double().t().repeat_interleave(128, 1)
    assert rel(hq, h) <= GENERAL + 2.0 ** -4


@pytest.mark.parametrize("T,N,K", [(5, 256, 528), (22, 4096, 1168), (70, 256, 528), (2100, 4096, 272)])
def test_glu_non_finite(T, N, K):
    """NaN and infinite operands spread along their row or channel only."""
    step("glu non-finite", T, N, K)
    (x, sx, w, sw), _ = glu_operands(T, N, K, F32)
    clean = torch.empty(T, N, device="cuda")
    rtq.fp8_glu(x, sx, w, sw, ACTS["silu"], y=clean)
    x.view(torch.uint8)[3, 200] = 0x7f                   # a token
    w.view(torch.uint8)[150, 100] = 0xff                 # a gate channel
    w.view(torch.uint8)[N + 31, 5] = 0x7f                # another's second projection
    y, (c, s) = torch.empty(T, N, device="cuda"), empty_rows(T, N)
    rtq.fp8_glu(x, sx, w, sw, ACTS["silu"], y=y)
    assert torch.isnan(y[3]).all() and torch.isnan(y[:, 150]).all() and torch.isnan(y[:, 31]).all()
    rows, cols = [t for t in range(T) if t != 3], [n for n in range(N) if n not in (31, 150)]
    assert same(y[rows][:, cols], clean[rows][:, cols])
    rtq.fp8_glu(x, sx, w, sw, ACTS["silu"], y_codes=c, y_scale=s)
    cf = c.float()
    assert torch.isnan(cf[3]).all() and torch.isnan(cf[:, 150]).all() and torch.isfinite(cf[rows][:, cols]).all()
    # the other channels' codes go by the largest finite magnitude of their group
    finite = torch.isfinite(y[rows])
    want = torch.where(finite, y[rows], torch.zeros_like(y[rows])).double()
    check_codes(torch.where(finite, cf[rows], torch.zeros_like(cf[rows])), s[:, rows], want, torch.zeros_like(want))


@pytest.mark.parametrize("T,N,K", [(5, 256, 144), (16, 128, 1040), (21, 4096, 1168), (40, 256, 2064), (100, 128, 144), (300, 256, 4112), (2100, 4096, 272)])
def test_glu_infinite_scale_of_the_last_block(T, N, K):
    """Nothing that fills a block, a stage or a turn meets the infinite scales: the last token's sums stay infinite, the first
    gate block's too."""
    step("glu infinite scale", T, N, K)
    x, w = torch.ones(T, K, device="cuda").to(E4M3), torch.ones(2 * N, K, device="cuda").to(E4M3)
    sx, sw = torch.ones(groups(K), T, device="cuda"), torch.ones(groups(2 * N), groups(K), device="cuda") / K
    sx[-1, T - 1] = float("inf")
    y = torch.empty(T, N, device="cuda")
    rtq.fp8_glu(x, sx, w, sw, ACTS["silu"], y=y)
    assert (y[T - 1] == float("inf")).all() and torch.isfinite(y[:T - 1]).all()
    (c, s), (hc, hs) = empty_rows(T, N), empty_rows(T, 2 * N)
    rtq.fp8_glu(x, sx, w, sw, ACTS["silu"], y_codes=c, y_scale=s, h_codes=hc, h_scale=hs)
    assert torch.isnan(c[T - 1].float()).all() and torch.isnan(hc[T - 1].float()).all()      # e4m3 has no infinity
    assert (s[:, T - 1] == 1.0).all() and (hs[:, T - 1] == 1.0).all() and torch.isfinite(c[:T - 1].float()).all()
    sx[-1, T - 1] = 1.0
    sw[0, -1] = float("inf")
    rtq.fp8_glu(x, sx, w, sw, ACTS["silu"], y=y)
    assert (y[:, :128] == float("inf")).all() and torch.isfinite(y[:, 128:]).all()


@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T,N,dtype", [(1, 128, BF16), (3, 640, F32), (130, 384, BF16), (517, 1152, F32), (2100, 1024, BF16)])
def test_glu_backward(T, N, dtype, name, fmt, st):
    step("glu backward", T, N, dtype, name, fmt, st)
    hc, hs = empty_rows(T, 2 * N, st=st)
    rtq.fp8_quantize(2 * randn(gen(T), T, 2 * N), hc, hs)
    h = hc.double() * hs.double().t().repeat_interleave(128, 1)
    dy = (1e-3 * randn(gen(2), T, N)).to(dtype)
    want = glu_gradient(dy, h, name)
    g, u, d = h[:, :N], h[:, N:], dy.double().abs()
    size = torch.cat([d * u.abs() * (1 + g.abs()), d * (act(g, name).abs())], 1)
    off = act_bound(h, name).repeat(1, 2) * size + TINY
    dh = torch.full((T + 1, 2 * N), 7.0, dtype=dtype, device="cuda")
    codes = torch.zeros(T + 1, 2 * N, dtype=torch.uint8, device="cuda").view(fmt)
    scale = torch.empty(groups(2 * N), T, dtype=st, device="cuda")
    rtq.glu_fp8_backward(dy, hc, hs, ACTS[name], dh=dh[:T], dh_codes=codes[:T], dh_scale=scale)
    near(dh[:T], want, off)
    check_codes(codes[:T].float(), scale.float(), want, off, fmt)
    assert (dh[T] == 7.0).all() and not codes[T].view(torch.uint8).any()
    d2, (c2, s2) = torch.empty(T, 2 * N, dtype=dtype, device="cuda"), empty_rows(T, 2 * N, fmt, st)
    rtq.glu_fp8_backward(dy, hc, hs, ACTS[name], dh=d2)
    rtq.glu_fp8_backward(dy, hc, hs, ACTS[name], dh_codes=c2, dh_scale=s2)
    assert same(d2, dh[:T].contiguous()) and same(c2, codes[:T].contiguous()) and same(s2, scale)


# ------------------------------------------------------------------ gradient norm and clipping

def grads_like(sizes, dtype, g=7, size=1e-2):
    return [(size * randn(gen(g + i), n)).to(dtype) for i, n in enumerate(sizes)]


@pytest.mark.parametrize("dtype", [F32, BF16, None])
@pytest.mark.parametrize("sizes", [[1], [7], [8], [9, 1, 255], [16384], [16385, 3, 0, 70001], [5] * 96, [130] * 97, [2049] * 300, [3_000_003]])
def test_grad_norm_and_clip(sizes, dtype):
    step("clip", len(sizes), sizes[:4], dtype)
    t = grads_like(sizes, dtype or F32)
    if dtype is None:                                     # both types in one list
        t = [x.bfloat16() if i % 2 else x for i, x in enumerate(t)]
    want = float(torch.sqrt(sum(x.double().square().sum() for x in t)))
    backs = [torch.full((x.numel() + 8,), 7.0, dtype=x.dtype, device="cuda") for x in t]
    outs = [b[:x.numel()] for b, x in zip(backs, t)]
    lst, norm_ = rtq.TensorList(t, outs), torch.empty(1, device="cuda")
    need = rtq.grad_norm_workspace(lst)
    ws = torch.zeros(need + 64, dtype=torch.uint8, device="cuda")
    rtq.grad_norm(lst, norm_, workspace=ws[:need])
    assert abs(float(norm_) - want) <= 1.01 * U * want and not ws[need:].any()
    for most in (0.3 * want, 2 * want, 0.0):
        rtq.grad_clip(lst, norm_, most)
        c = min(1.0, most / (want + 1e-6))
        for x, o, b in zip(t, outs, backs):
            ref = x.double() * c
            near(o, ref, 4 * U * ref.abs() + 2.0 ** -149)
            assert (b[x.numel():] == 7.0).all()            # what lies behind stays as it was
    rtq.grad_clip(lst, norm_, 0.3 * want)
    own = [x.clone() for x in t]
    rtq.grad_clip(rtq.TensorList(own), norm_, 0.3 * want)  # in place
    assert all(same(a, b) for a, b in zip(own, outs))
    rtq.grad_clip(rtq.TensorList(own), norm_, 2 * want)    # nothing to clip: as they are
    assert all(same(a, b) for a, b in zip(own, outs))


def test_grad_norm_extremes():
    """Squares past fp32's range, zeros, infinities and NaN; the norm of no elements."""
    step("clip extremes")
    n = torch.empty((), device="cuda")
    big = torch.full((1000,), 2.0 ** 100, device="cuda")
    assert float(rtq.grad_norm(rtq.TensorList([big]), n)) == pytest.approx(2.0 ** 100 * 1000 ** 0.5, rel=1e-6)
    small = torch.full((1000,), 2.0 ** -120, device="cuda")
    assert float(rtq.grad_norm(rtq.TensorList([small]), n)) == pytest.approx(2.0 ** -120 * 1000 ** 0.5, rel=1e-6)
    zero = torch.zeros(77, device="cuda", dtype=BF16)
    assert float(rtq.grad_norm(rtq.TensorList([zero]), n)) == 0.0
    rtq.grad_clip(rtq.TensorList([zero]), n, 1.0)
    assert not zero.any()
    assert float(rtq.grad_norm(rtq.TensorList([torch.empty(0, device="cuda")]), n)) == 0.0
    for bad in (float("nan"), float("inf")):
        x = torch.ones(300, device="cuda")
        x[17] = bad
        y = torch.ones(5, device="cuda", dtype=BF16)
        lst = rtq.TensorList([x, y])
        v = float(rtq.grad_norm(lst, n))
        assert v != v if bad != bad else v == float("inf")
        rtq.grad_clip(lst, n, 1.0)
        if bad != bad:
            assert torch.isnan(x).all() and torch.isnan(y).all()
        else:                                             # a factor of 0
            assert torch.isnan(x[17]) and not x[:17].any() and not y.any()


# ------------------------------------------------------------------ as they are used

def block_step(x, r, p, buf):
    """A training step of the pre-norm gated block y = h + down(glu(norm(h))), h = x + r, by the library: gradients of a
    given dy, all clipped together."""
    rtq.rmsnorm_forward(x, p["gamma"], EPS, residual=r, h=buf["h"], codes=buf["n"], scale=buf["ns"])
    rtq.fp8_glu(buf["n"], buf["ns"], p["w"], p["ws"], ACTS["silu"], y_codes=buf["a"], y_scale=buf["as"], h_codes=buf["hc"], h_scale=buf["hs"])
    rtq.fp8_qgemm(buf["a"], buf["as"], p["v"], p["vs"], buf["y"])
    rtq.fp8_linear_dgrad(buf["dy"], p["v"], p["vs"], buf["da"], grad_dtype=E5M2)
    rtq.fp8_wgrad(buf["dy"], buf["a"], buf["as"], buf["dv"])
    rtq.glu_fp8_backward(buf["da"], buf["hc"], buf["hs"], ACTS["silu"], dh=buf["dg"], dh_codes=buf["dgc"], dh_scale=buf["dgs"])
    rtq.fp8_dgrad(buf["dgc"], buf["dgs"], p["w"], p["ws"], buf["dn"])
    rtq.fp8_wgrad(buf["dg"], buf["n"], buf["ns"], buf["dw"])
    rtq.rmsnorm_backward(buf["dn"], buf["h"], p["gamma"], EPS, buf["dx"], dgamma=buf["dgamma"], dresidual=buf["dy"])
    rtq.grad_norm(buf["list"], buf["norm"])
    rtq.grad_clip(buf["list"], buf["norm"], 0.5)


def block_case(T, d, N, st=E8M0):
    g = gen(T + d + N)
    e = lambda *s, dt=BF16: torch.empty(*s, dtype=dt, device="cuda")
    p = {"gamma": 1 + 0.2 * randn(g, d), "w": e(2 * N, d, dt=E4M3), "ws": e(groups(2 * N), groups(d), dt=st), "v": e(d, N, dt=E4M3),
         "vs": e(groups(d), groups(N), dt=st)}
    rtq.fp8_quantize(randn(g, 2 * N, d) / d ** 0.5, p["w"], p["ws"], blocks=True)
    rtq.fp8_quantize(randn(g, d, N) / N ** 0.5, p["v"], p["vs"], blocks=True)
    buf = {"h": e(T, d), "n": e(T, d, dt=E4M3), "ns": e(groups(d), T, dt=st), "a": e(T, N, dt=E4M3), "as": e(groups(N), T, dt=st),
           "hc": e(T, 2 * N, dt=E4M3), "hs": e(groups(2 * N), T, dt=st), "y": e(T, d), "dy": randn(g, T, d).bfloat16(), "da": e(T, N),
           "dg": e(T, 2 * N), "dgc": e(T, 2 * N, dt=E5M2), "dgs": e(groups(2 * N), T, dt=st), "dn": e(T, d), "dx": e(T, d),
           "dw": e(2 * N, d, dt=F32), "dv": e(d, N, dt=F32), "dgamma": e(d, dt=F32), "norm": e(1, dt=F32)}
    buf["list"] = rtq.TensorList([buf["dw"], buf["dv"], buf["dgamma"]])
    return randn(g, T, d).bfloat16(), randn(g, T, d).bfloat16(), p, buf


@pytest.mark.parametrize("T,d,N", [(70, 272, 384), (600, 1040, 1152)])
def test_block_training_step(T, d, N):
    """Against the unquantised block's 64-bit gradients.  Each quantised tensor is off by at most 2^-4 of an element (e4m3;
    e5m2 2^-3), in the 2-norm by 1/sqrt(3) of a uniform error's end at most, and the errors of one element are independent of
    another's: with the norm's output, the pre-activations and the activations in e4m3 (0.036 each) and two gradients in e5m2
    (0.072 each), each counted as if it passed whole into the result, and the activation's curvature doubling that of the
    pre-activations, dx and the weights' gradients are within 3 * 0.036 + 0.036 + 2 * 0.072 = 0.29."""
    step("block", T, d, N)
    x, r, p, buf = block_case(T, d, N)
    block_step(x, r, p, buf)
    wv = p["w"].double() * p["ws"].double().repeat_interleave(128, 0).repeat_interleave(128, 1)[:, :d]
    vv = p["v"].double() * p["vs"].double().repeat_interleave(128, 0)[:d].repeat_interleave(128, 1)[:, :N]
    h = (x.float() + r.float()).bfloat16().double().requires_grad_(True)
    wv, vv, gamma = wv.requires_grad_(True), vv.requires_grad_(True), p["gamma"].double().requires_grad_(True)
    n = norm(h, gamma)
    z = n @ wv.t().contiguous()
    y = h + glu(z, "silu") @ vv.t().contiguous()
    dh, dw, dv, dgamma = torch.autograd.grad(y, (h, wv, vv, gamma), buf["dy"].double())
    total = float(torch.sqrt(dw.square().sum() + dv.square().sum() + dgamma.square().sum()))
    got = float(buf["norm"])
    assert abs(got - total) <= 0.29 * total
    c = 0.5 / (got + 1e-6)
    assert rel(buf["dx"], dh) <= 0.29
    for name, want in (("dw", dw), ("dv", dv), ("dgamma", dgamma)):
        assert rel(buf[name] / c, want) <= 0.29, name
    assert float(torch.sqrt(sum(buf[k].double().square().sum() for k in ("dw", "dv", "dgamma")))) == pytest.approx(0.5, rel=1e-4)


@pytest.mark.parametrize("T,d,N", [(1, 256, 384), (200, 272, 1152), (2304, 512, 4096)])
def test_block_captured_and_on_other_streams(T, d, N):
    """A captured step, replayed over changed inputs with eager work in between, equals the eager one's bits; so does one on
    another stream, and two at once."""
    step("block captured", T, d, N)
    x, r, p, buf = block_case(T, d, N)
    names = ("h", "n", "ns", "a", "as", "hc", "hs", "y", "dx", "dw", "dv", "dgamma", "norm")
    block_step(x, r, p, buf)
    torch.cuda.synchronize()
    want = {k: buf[k].clone() for k in names}
    first = x.clone()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        block_step(x, r, p, buf)
    side.synchronize()
    assert all(same(buf[k], want[k]) for k in names)
    with torch.cuda.graph(graph):
        block_step(x, r, p, buf)
    for turn in range(3):
        x.copy_(first if turn != 1 else first * 2)
        for k in names:
            buf[k].view(torch.uint8).zero_()
        graph.replay()
        torch.cuda.synchronize()
        if turn != 1:
            assert all(same(buf[k], want[k]) for k in names), turn
        else:
            got = {k: buf[k].clone() for k in names}
            block_step(x, r, p, buf)
            torch.cuda.synchronize()
            assert all(same(buf[k], got[k]) for k in names)
    x2, r2, p2, buf2 = block_case(T, d, N)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        block_step(x2, r2, p2, buf2)
    block_step(x, r, p, buf)
    torch.cuda.synchronize()
    assert all(same(buf[k], want[k]) and same(buf2[k], want[k]) for k in names)


def test_past_32_bits():
    """More than 2^31 elements: the last rows equal the same rows alone."""
    step("past 2^31: norm")
    T, d = 530000, 4112
    x = torch.empty(T, d, dtype=BF16, device="cuda")
    x[:] = rows_like(3, 1000, d).repeat(530, 1)
    gamma = (1 + 0.3 * randn(gen(d), d)).to(BF16)
    codes, scale = empty_rows(T, d, st=E8M0)
    rtq.rmsnorm_forward(x, gamma, EPS, residual=x, h=x, codes=codes, scale=scale)
    tail = rows_like(3, 1000, d)
    c2, s2 = empty_rows(1000, d, st=E8M0)
    rtq.rmsnorm_forward(tail, gamma, EPS, residual=tail, h=tail, codes=c2, scale=s2)
    for i in (0, 500, 529):
        part = slice(1000 * i, 1000 * i + 1000)
        assert same(x[part], tail) and same(codes[part], c2) and same(scale[:, part].contiguous(), s2)
    step("past 2^31: norm backward")
    dgamma, dg1 = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    del codes, scale
    dh = torch.empty_like(x)
    rtq.rmsnorm_backward(x, x, gamma, EPS, dh, dgamma=dgamma)
    d2 = torch.empty_like(tail)
    rtq.rmsnorm_backward(tail, tail, gamma, EPS, d2, dgamma=dg1)
    assert same(dh[-1000:], d2) and rel(dgamma, 530 * dg1) <= 1e-5
    step("past 2^31: clip")
    n = torch.empty(1, device="cuda")
    rtq.grad_norm(rtq.TensorList([x]), n)
    one = torch.empty(1, device="cuda")
    rtq.grad_norm(rtq.TensorList([tail]), one)
    assert float(n) == pytest.approx(float(one) * 530 ** 0.5, rel=1e-6)
    rtq.grad_clip(rtq.TensorList([x], [dh]), n, float(n) / 2)
    assert rel(dh[-1000:], tail.double() / 2) <= 2.0 ** -8
    del dh, x
    step("past 2^31: glu backward")
    T, N = 530000, 2048
    hc, hs = torch.empty(T, 2 * N, dtype=torch.uint8, device="cuda"), torch.empty(groups(2 * N), T, device="cuda")
    c1, s1 = empty_rows(1000, 2 * N)
    rtq.fp8_quantize(2 * randn(gen(1), 1000, 2 * N), c1, s1)
    hc[:], hs[:] = c1.view(torch.uint8).repeat(530, 1), s1.repeat(1, 530)
    dy1 = randn(gen(2), 1000, N).bfloat16()
    dh, d1 = torch.empty(T, 2 * N, dtype=BF16, device="cuda"), torch.empty(1000, 2 * N, dtype=BF16, device="cuda")
    rtq.glu_fp8_backward(dy1.repeat(530, 1), hc.view(E4M3), hs, ACTS["silu"], dh=dh)
    rtq.glu_fp8_backward(dy1, c1, s1, ACTS["silu"], dh=d1)
    assert same(dh[-1000:], d1) and same(dh[:1000], d1)
    del dh, hc, hs
    step("past 2^31: glu")
    T, N, K = 140000, 8192, 272
    (x, sx, w, sw), _ = glu_operands(1000, N, K, E8M0)
    (c1, s1), (hc1, hs1) = empty_rows(1000, N, st=E8M0), empty_rows(1000, 2 * N, st=E8M0)
    rtq.fp8_glu(x, sx, w, sw, ACTS["silu"], y_codes=c1, y_scale=s1, h_codes=hc1, h_scale=hs1)
    many = lambda t, n: t.view(torch.uint8).repeat(*n).view(t.dtype)
    (c, s), (hc, hs) = empty_rows(T, N, st=E8M0), empty_rows(T, 2 * N, st=E8M0)
    rtq.fp8_glu(many(x, (140, 1)), many(sx, (1, 140)), w, sw, ACTS["silu"], y_codes=c, y_scale=s, h_codes=hc, h_scale=hs)
    for i in (0, 70, 139):
        part = slice(1000 * i, 1000 * i + 1000)
        assert same(c[part], c1) and same(hc[part], hc1)
        assert same(s[:, part].contiguous(), s1) and same(hs[:, part].contiguous(), hs1)


def test_binding_refusals():
    step("refusals")
    bf, e = BF16, lambda *s, dt=BF16: torch.empty(*s, dtype=dt, device="cuda")
    x, gamma, (codes, scale) = e(4, 256), e(256), empty_rows(4, 256)
    good = dict(codes=codes, scale=scale)
    for change, error, match in (
            (dict(codes=codes, scale=None), ValueError, "codes and scale"), (dict(), ValueError, "give y"),
            (dict(good, residual=x), ValueError, "together"), (dict(good, residual=x, h=e(4, 256, dt=F32)), TypeError, "h: unsupported dtype"),
            (dict(y=e(4, 256, dt=F32)), TypeError, "y: unsupported"), (dict(y=e(4, 128)), ValueError, "y: shape"),
            (dict(y=e(256, 4).t()), ValueError, "contiguous"), (dict(codes=codes.view(torch.uint8), scale=scale), TypeError, "codes"),
            (dict(codes=codes, scale=e(4, 2, dt=F32)), ValueError, "scale: shape"), (dict(good, stream=7), AttributeError, "device_index"),
            (dict(y=torch.empty(4, 256, dtype=bf)), ValueError, "GPU tensor"), (dict(y="no"), TypeError, "tensor")):
        with pytest.raises(error, match=match):
            rtq.rmsnorm_forward(x, gamma, EPS, **change)
    with pytest.raises(ValueError, match="gamma: shape"):
        rtq.rmsnorm_forward(x, e(128), EPS, **good)
    with pytest.raises(rtq.RtqError, match="eps"):
        rtq.rmsnorm_forward(x, gamma, 0.0, **good)
    with pytest.raises(rtq.RtqError, match="multiple of 16"):
        rtq.rmsnorm_forward(e(4, 40), e(40), EPS, y=e(4, 40))
    with pytest.raises(rtq.RtqError, match="dh must not be h"):
        rtq.rmsnorm_backward(e(4, 256), x, gamma, EPS, x)
    with pytest.raises(rtq.RtqError, match="workspace too small"):
        rtq.rmsnorm_backward(x, e(4, 256), gamma, EPS, e(4, 256), dgamma=e(256), workspace=e(16, dt=torch.uint8))
    xc, xs = empty_rows(4, 256)
    w, ws = e(512, 256, dt=E4M3), e(4, 2, dt=F32)
    for change, error, match in (
            (dict(), ValueError, "give either y"), (dict(y=e(4, 256), y_codes=xc, y_scale=xs), ValueError, "give either y"),
            (dict(y=e(4, 256), h_codes=e(4, 512, dt=E4M3)), ValueError, "together"), (dict(y=e(4, 512)), ValueError, "y: shape"),
            (dict(y_codes=xc, y_scale=e(2, 4, dt=torch.uint8).view(E8M0)), TypeError, "y_scale")):
        with pytest.raises(error, match=match):
            rtq.fp8_glu(xc, xs, w, ws, ACTS["silu"], **change)
    with pytest.raises(ValueError, match="two projections"):
        rtq.fp8_glu(xc, xs, e(384, 256, dt=E4M3), e(3, 2, dt=F32), ACTS["silu"], y=e(4, 192))
    with pytest.raises(rtq.RtqError, match="activation"):
        rtq.fp8_glu(xc, xs, w, ws, 9, y=e(4, 256))
    with pytest.raises(ValueError, match="give dh"):
        rtq.glu_fp8_backward(x, e(4, 512, dt=E4M3), e(4, 4, dt=F32), ACTS["silu"])
    flat = torch.zeros(1001, device="cuda")
    with pytest.raises(rtq.RtqError, match="aligned"):                 # a view that begins inside a 16-byte line
        rtq.grad_norm(rtq.TensorList([flat[1:]]), e(1, dt=F32))
    with pytest.raises(TypeError, match="dtype"):
        rtq.TensorList([flat.double()])
    with pytest.raises(ValueError, match="norm: shape"):
        rtq.grad_norm(rtq.TensorList([flat]), e(2, dt=F32))
    with pytest.raises(rtq.RtqError, match="most"):
        rtq.grad_clip(rtq.TensorList([flat]), e(1, dt=F32), -1.0)


def test_replaced_and_overlapping_tensors_are_refused():
    x, y, n = torch.ones(1000, device="cuda"), torch.ones(600, device="cuda"), torch.zeros(1, device="cuda")
    inplace, apart = rtq.TensorList([x, y]), rtq.TensorList([x], [torch.empty_like(x)])
    assert float(rtq.grad_norm(inplace, n)) == 40.0
    x.data = torch.ones(1000, device="cuda")       # the list's memory is gone
    for lst in (inplace, apart):
        with pytest.raises(ValueError, match="replaced"):
            rtq.grad_norm(lst, n)
        with pytest.raises(ValueError, match="replaced"):
            rtq.grad_clip(lst, n, 1.0)
    apart = rtq.TensorList([x], [torch.empty_like(x)])
    apart.outs[0].data = torch.empty_like(x)
    rtq.grad_norm(apart, n)
    with pytest.raises(ValueError, match="replaced"):
        rtq.grad_clip(apart, n, 1.0)
    for tensors, outs in (([x, x], None), ([x, x[500:]], None), ([x[:500], x[500:]], [x[500:], y[:500]]), ([x[:600]], [x[4:604]])):
        with pytest.raises(ValueError, match="overlaps"):
            rtq.TensorList(tensors, outs)
    assert float(rtq.grad_norm(rtq.TensorList([x, x], [torch.empty_like(x), torch.empty_like(x)]), n)) == pytest.approx(2000 ** 0.5, rel=1e-6)


def test_clipping_past_32_bits_of_work_items():
    n = (1 << 36) + 4099                           # in pieces of 4096 elements, 256 threads each: over 2^32 threads
    if torch.cuda.mem_get_info()[0] < 2 * n + (8 << 30):
        pytest.skip("not enough memory")
    x, norm_ = torch.full((n,), 2.0, dtype=BF16, device="cuda"), torch.empty(1, device="cuda")
    lst = rtq.TensorList([x])
    want = 2 * n ** 0.5
    assert float(rtq.grad_norm(lst, norm_)) == pytest.approx(want, rel=1e-6)
    rtq.grad_clip(lst, norm_, want / 2)
    for part in (x[:10000], x[-10000:], x[::1000003]):
        assert bool((part == 1.0).all())
