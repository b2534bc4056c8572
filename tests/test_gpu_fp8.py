"""GPU tests of the 8-bit floating point layer (scales for blocks of 128) against plain 64-bit forms.

Tolerances.  Codes and scales are exact: x / 2^e has no rounding but the code's own.  Products are tested in
two ways.  (1) Operands whose products all lie within 2^13 of each other and whose sums fit 24 bits are exact
through the matrix cores and the fp32 sums, so fp32 outputs equal the 64-bit ones and bf16 outputs are their
roundings.  (2) General operands: an instruction truncates its products to about 2^-13 of the largest; with
magnitudes at most 16 times their root mean square that is at most 16 * 2^-13 = 2^-9 of the result in the
2-norm, and a bf16 output adds half a step, 2^-8."""
import pytest
import torch

import rotation_then_quantize_amd as rtq
from _fp8 import (E4M3, E5M2, E8M0, act, block_values, groups, quantise, rel, row_values, slope)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ACTS = {"gelu_tanh": rtq.RTQ_ACT_GELU_TANH, "gelu": rtq.RTQ_ACT_GELU, "silu": rtq.RTQ_ACT_SILU}
HALF_BF16 = 2.0 ** -8        # largest relative error of one rounding to bf16
GENERAL = 2.0 ** -9          # matrix core alignment, see above


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    rtq.load_library()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows_like(seed, T, d, dtype=BF16):
    """Heavy-tailed rows with a zero group and an outlier, as the CPU reference and the GPU both take them."""
    g = gen(seed)
    x = torch.randn(T, d, generator=g) * torch.exp(torch.randn(T, d, generator=g))
    if T > 2:
        x[1, :128] = 0.0
        x[2, d // 2] = 300.0
    return x.to(dtype)


def empty_rows(T, d, fmt=E4M3, st=F32):
    return (torch.empty(T, d, dtype=fmt, device="cuda"), torch.empty(groups(d), T, dtype=st, device="cuda"))


def int_codes(seed, rows, d, most=4):
    """Small whole numbers: every product and sum below is exact."""
    return torch.randint(-most, most + 1, (rows, d), generator=gen(seed)).float().to(E4M3)


def pow2_scales(seed, a, b, lo=-3, hi=3):
    return torch.exp2(torch.randint(lo, hi + 1, (a, b), generator=gen(seed)).float())


def same(a, b):
    """Bit equality, NaNs in the same places."""
    a, b = a.cpu().double(), b.cpu().double()
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a, 0.0, 9e99, -9e99),
                                                                      torch.nan_to_num(b, 0.0, 9e99, -9e99))


def step(name, *what):
    print(name, *what, flush=True)


# ------------------------------------------------------------------ quantise, dequantise

@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,d", [(1, 16), (1, 4096), (3, 528), (130, 128), (257, 1040)])
def test_quantise_rows(T, d, dtype, st, fmt):
    step("quantise rows", T, d, dtype, st, fmt)
    x = rows_like(T + d, T, d, dtype)
    q, s = quantise(x, fmt)
    codes, scale = empty_rows(T, d, fmt, st)
    rtq.fp8_quantize(x.cuda(), codes, scale)
    assert same(codes, q) and same(scale.float(), s)
    y = torch.empty(T, d, device="cuda")
    rtq.fp8_dequantize(codes, scale, y)
    assert same(y, row_values(codes, scale))
    yb = torch.empty(T, d, dtype=BF16, device="cuda")
    rtq.fp8_dequantize(codes, scale, yb)
    assert same(yb, row_values(codes, scale).float().bfloat16())


@pytest.mark.parametrize("T,d", [(8300, 2064), (4300, 512)])
def test_quantise_rows_many(T, d):
    """Many rows (two a wave) against the one-row form of the same rows."""
    step("quantise rows", T, d)
    x = rows_like(5, T, d).cuda()
    codes, scale = empty_rows(T, d)
    rtq.fp8_quantize(x, codes, scale)
    for i in (0, 1, 2, 15, 16, T - 17, T - 1):
        c1, s1 = empty_rows(1, d)
        rtq.fp8_quantize(x[i:i + 1].contiguous(), c1, s1)
        assert same(codes[i:i + 1], c1) and same(scale[:, i:i + 1], s1)


@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantise_special_values(dtype, fmt):
    """Ties, the largest codes, subnormals, NaN and infinities, blocks of zeros, magnitudes at both ends."""
    step("quantise special", dtype, fmt)
    top = 448.0 if fmt == E4M3 else 57344.0
    base = torch.tensor([top, 1.0625, 1.1875, -1.0625, 17.0, 19.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 0.0, -0.0])
    rows = [base, base * 2.0 ** 100, base * 2.0 ** -100, base * 2.0 ** -130, base * 2.0 ** -140, torch.zeros(11)]
    x = torch.zeros(10, 128)
    for i, r in enumerate(rows):
        x[i, :11] = r
    x[6, 5], x[6, 6], x[6, 7], x[6, 8] = float("nan"), float("inf"), -float("inf"), 3.0
    x[7] = float("nan")
    x[8, :] = 3.3e38
    x[9, :] = torch.linspace(-1.75, 1.7500001, 128)
    x = x.to(dtype)
    q, s = quantise(x, fmt)
    for st in (F32, E8M0):
        codes, scale = empty_rows(10, 128, fmt, st)
        rtq.fp8_quantize(x.cuda(), codes, scale)
        assert same(codes, q) and same(scale.float(), s)


@pytest.mark.parametrize("N,K,dtype,st,fmt", [(1, 16, BF16, F32, E4M3), (129, 272, BF16, E8M0, E4M3),
                                              (300, 528, F32, F32, E5M2), (128, 128, F32, E8M0, E4M3)])
def test_quantise_blocks(N, K, dtype, st, fmt):
    step("quantise blocks", N, K, dtype, st, fmt)
    w = rows_like(N + K, N, K, dtype)
    q, s = quantise(w, fmt, blocks=True)
    codes = torch.empty(N, K, dtype=fmt, device="cuda")
    scale = torch.empty(groups(N), groups(K), dtype=st, device="cuda")
    rtq.fp8_quantize(w.cuda(), codes, scale, blocks=True)
    assert same(codes, q) and same(scale.float(), s)
    y = torch.empty(N, K, device="cuda")
    rtq.fp8_dequantize(codes, scale, y, blocks=True)
    assert same(y, block_values(codes, scale))


# ------------------------------------------------------------------ products

SIZES = [(1, 1, 16), (1, 100, 256), (2, 33, 144), (4, 8200, 400), (16, 16400, 2064), (13, 4096, 2048), (16, 130, 128), (17, 63, 272), (64, 64, 128),
         (65, 129, 400), (200, 1000, 1040), (257, 260, 4096), (391, 1001, 1936), (700, 2304, 640)]


def exact_operands(T, N, K, st, fmt=E4M3, trans=False):
    red = N if trans else K
    a = int_codes(T + K, T, red).float().to(fmt)
    return (a, pow2_scales(3, groups(red), T).to(st), int_codes(N + 1, N, K), pow2_scales(4, groups(N), groups(K)).to(st))


@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_product_exact(T, N, K, fmt, st):
    step("product", T, N, K, fmt, st)
    a, sa, w, sw = exact_operands(T, N, K, st, fmt)
    ref = row_values(a, sa) @ block_values(w, sw).T
    dev = [t.cuda() for t in (a, sa, w, sw)]
    for dtype in (F32, BF16):
        y = torch.full((T + 1, N), 7.0, dtype=dtype, device="cuda")
        rtq.fp8_qgemm(*dev, y[:T])
        assert same(y[:T], ref.float().to(dtype))
        assert (y[T] == 7.0).all()                       # the row behind the last stays as it was
        if T * N < 1 << 16:                              # without a workspace: nothing is split, the same sums
            z = torch.empty(T, N, dtype=dtype, device="cuda")
            ws = torch.empty(16, dtype=torch.uint8, device="cuda")
            rtq.fp8_qgemm(*dev, z, workspace=ws)
            assert same(z, y[:T])


@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("T,N,K", [(1, 16, 16), (1, 256, 128), (5, 144, 272), (64, 128, 64), (130, 400, 1040),
                                   (517, 2064, 1040), (300, 4096, 528), (700, 640, 2304)])
def test_dgrad_exact(T, N, K, fmt, st):
    step("dgrad", T, N, K, fmt, st)
    g, sg, w, sw = exact_operands(T, N, K, st, fmt, trans=True)
    ref = row_values(g, sg) @ block_values(w, sw)
    for dtype in (F32, BF16):
        dx = torch.full((T + 1, K), 7.0, dtype=dtype, device="cuda")
        rtq.fp8_dgrad(*[t.cuda() for t in (g, sg, w, sw)], dx[:T])
        assert same(dx[:T], ref.float().to(dtype))
        assert (dx[T] == 7.0).all()


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("fmt,st", [(E4M3, F32), (E5M2, E8M0), (E4M3, E8M0), (E5M2, F32)])
@pytest.mark.parametrize("T,N,R", [(4100, 1488, 128), (4100, 1488, 144), (4099, 2288, 272), (4608, 4096, 400), (4608, 4096, 640),
                                   (25000, 272, 528), (2500, 2800, 2064)])
def test_large_products_exact(T, N, R, fmt, st, trans):
    """Outputs of many 256 x 256 tiles: whole rounds of them, halves, one to many reduction blocks."""
    step("large product", T, N, R, fmt, st, trans)
    a = int_codes(T + R, T, R).float().to(fmt).cuda()
    sa, w = pow2_scales(3, groups(R), T).to(st).cuda(), int_codes(N + 1, R if trans else N, N if trans else R).cuda()
    sw = pow2_scales(4, groups(w.shape[0]), groups(w.shape[1])).to(st).cuda()
    av = a.double() * sa.double().t().repeat_interleave(128, 1)[:, :R]
    wv = w.double() * sw.double().repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)[:, :w.shape[1]]
    ref = av @ (wv if trans else wv.t().contiguous())
    call = rtq.fp8_dgrad if trans else rtq.fp8_qgemm
    for dtype in (F32, BF16):
        y = torch.full((T + 1, N), 7.0, dtype=dtype, device="cuda")
        call(a, sa, w, sw, y[:T])
        assert torch.equal(y[:T].double(), ref.float().to(dtype).double())
        assert (y[T] == 7.0).all()
    if not trans:                                            # a column count that no store fits
        y = torch.full((T + 1, N - 3), 7.0, dtype=BF16, device="cuda")
        call(a, sa, w[:N - 3].contiguous(), sw, y[:T])
        assert torch.equal(y[:T].double(), ref[:, :N - 3].float().bfloat16().double())
        assert (y[T] == 7.0).all()


@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("T,N,R", [(1000, 4000, 400), (990, 4096, 4176), (64, 4096, 4096), (300, 512, 8240), (40, 1008, 16400),
                                   (512, 4096, 5008), (128, 4096, 16400), (300, 640, 2048), (9, 4096, 2064), (3, 16400, 1040),
                                   (16, 1040, 8208), (1, 4096, 4096)])
def test_product_forms_exact(T, N, R, trans, st):
    """Tiles of 64 and of 128, whole and split reductions, more blocks than a table of scales holds, few rows.
    Codes to 4 and two scales of 1/2 to 2: products are whole quarters up to 64, so every sum is at most 2^20.01
    and a multiple of 1/4, exact in fp32."""
    step("product forms", T, N, R, trans, st)
    a, w = int_codes(T + R, T, R).cuda(), int_codes(N + 1, R if trans else N, N if trans else R).cuda()
    sa = pow2_scales(3, groups(R), T, -1, 1).to(st).cuda()
    sw = pow2_scales(4, groups(w.shape[0]), groups(w.shape[1]), -1, 1).to(st).cuda()
    av = a.double() * sa.double().t().repeat_interleave(128, 1)[:, :R]
    wv = w.double() * sw.double().repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)[:, :w.shape[1]]
    ref = av @ (wv if trans else wv.t().contiguous())
    call, size = (rtq.fp8_dgrad, rtq.fp8_dgrad_workspace) if trans else (rtq.fp8_qgemm, rtq.fp8_qgemm_workspace)
    need = size(T, *((R, N) if trans else (N, R)))
    for dtype in (F32, BF16):
        y = torch.full((T + 1, N), 7.0, dtype=dtype, device="cuda")
        ws = torch.zeros(need + 64, dtype=torch.uint8, device="cuda")
        call(a, sa, w, sw, y[:T], workspace=ws[:need] if need else ws)
        assert torch.equal(y[:T].double(), ref.float().to(dtype).double())
        assert (y[T] == 7.0).all() and not ws[need:].any()      # nothing past the size asked for


@pytest.mark.parametrize("T,N,K", [(1, 300, 2048), (16, 512, 4096), (100, 333, 1040), (300, 512, 2064)])
def test_product_general(T, N, K):
    """General fp32 scales and codes over the whole range."""
    step("product general", T, N, K)
    x, w = rows_like(T, T, K), torch.randn(N, K, generator=gen(N)) * 0.05
    a, sa = [t.cuda() for t in (lambda q: (q[0].float().to(E4M3), q[1].float()))(quantise(x, E4M3))]
    wq, sw = [t.cuda() for t in (lambda q: (q[0].float().to(E4M3), q[1].float()))(quantise(w, E4M3, blocks=True))]
    sa *= 0.75 + 0.5 * torch.rand(sa.shape, generator=gen(1)).cuda()
    sw *= 0.75 + 0.5 * torch.rand(sw.shape, generator=gen(2)).cuda()
    ref = row_values(a, sa) @ block_values(wq, sw).T
    y = torch.empty(T, N, device="cuda")
    rtq.fp8_qgemm(a, sa, wq, sw, y)
    assert rel(y, ref) <= GENERAL
    z = torch.empty(T, N, dtype=BF16, device="cuda")
    rtq.fp8_linear(x.cuda(), wq, sw, z)
    qx, sx = quantise(x, E4M3)
    assert rel(z, row_values(qx, sx) @ block_values(wq, sw).T) <= GENERAL + HALF_BF16


def test_product_spreads_non_finite_values_only_along_their_row_and_column():
    step("product non-finite")
    T, N, K = 70, 200, 528
    a, sa, w, sw = [t.cuda() for t in exact_operands(T, N, K, F32)]
    clean = torch.empty(T, N, device="cuda")
    rtq.fp8_qgemm(a, sa, w, sw, clean)
    a.view(torch.uint8)[3, 500] = 0x7f                      # NaN code
    w.view(torch.uint8)[150, 100] = 0xff
    sa[0, 5] = float("inf")
    y = torch.empty(T, N, device="cuda")
    rtq.fp8_qgemm(a, sa, w, sw, y)
    assert torch.isnan(y[3]).all() and torch.isnan(y[:, 150]).all()
    assert not torch.isfinite(y[5]).any()
    keep = [i for i in range(T) if i not in (3, 5)]
    cols = [j for j in range(N) if j != 150]
    assert same(y[keep][:, cols], clean[keep][:, cols])


@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("T,N,R", [(5, 208, 528), (70, 208, 528), (200, 4096, 1040), (1000, 4000, 400), (4100, 1488, 272)])
def test_not_a_number_scales(T, N, R, trans, st):
    """In every form: one row's and one weight block's scale."""
    step("NaN scales", T, N, R, trans, st)
    a, w = int_codes(1, T, R).cuda(), int_codes(2, R if trans else N, N if trans else R).cuda()
    sa = torch.ones(groups(R), T, device="cuda").to(st)
    sw = torch.ones(groups(w.shape[0]), groups(w.shape[1]), device="cuda").to(st)
    call = rtq.fp8_dgrad if trans else rtq.fp8_qgemm
    clean = torch.empty(T, N, device="cuda")
    call(a, sa, w, sw, clean)
    for s, at in ((sa, (1, 3)), (sw, (1, 0) if trans else (0, 1))):     # the second block of the reduction
        if st == E8M0:
            s.view(torch.uint8)[at] = 255
        else:
            s[at] = float("nan")
    y = torch.empty(T, N, device="cuda")
    call(a, sa, w, sw, y)
    assert torch.isnan(y[3]).all() and torch.isnan(y[:, :128]).all()
    rest = [t for t in range(T) if t != 3]
    assert torch.equal(y[rest][:, 128:], clean[rest][:, 128:])


@pytest.mark.parametrize("T,N,R", [(5, 200, 144), (5, 200, 1040), (16, 4200, 400), (40, 200, 1040), (300, 200, 4112), (4100, 1488, 272)])
def test_infinite_scale_of_the_last_block(T, N, R):
    """Nothing that fills a block, a stage or a turn meets the infinite scale: sums of positive products stay infinite."""
    step("infinite scale", T, N, R)
    a, w = torch.ones(T, R, device="cuda").to(E4M3), torch.ones(N, R, device="cuda").to(E4M3)
    sa, sw = torch.ones(groups(R), T, device="cuda"), torch.ones(groups(N), groups(R), device="cuda")
    sa[-1, T - 1] = float("inf")
    y = torch.empty(T, N, device="cuda")
    rtq.fp8_qgemm(a, sa, w, sw, y)
    assert (y[T - 1] == float("inf")).all() and (y[:T - 1] == float(R)).all()


@pytest.mark.parametrize("T,N,K", [(1, 16, 32), (65, 64, 272), (130, 64, 144), (333, 4096, 4112)])
def test_wgrad_infinite_scale_of_the_last_token(T, N, K):
    step("wgrad infinite scale", T, N, K)
    dy, x = torch.ones(T, N, dtype=BF16, device="cuda"), torch.ones(T, K, device="cuda").to(E4M3)
    sx = torch.ones(groups(K), T, device="cuda")
    sx[0, T - 1] = float("inf")
    dw = torch.empty(N, K, device="cuda")
    rtq.fp8_wgrad(dy, x, sx, dw)
    assert (dw[:, :128] == float("inf")).all() and (dw[:, 128:] == float(T)).all()


def test_product_extreme_scales():
    """Scales at both ends of their range, zero and the smallest E8M0 byte."""
    step("product extreme scales")
    T, N, K = 5, 40, 256
    a, _, w, _ = exact_operands(T, N, K, F32)
    for sa, sw in ((2.0 ** 100, 2.0 ** -100), (2.0 ** -120, 2.0 ** 120), (0.0, 1.0), (2.0 ** -60, 2.0 ** -60)):
        s1, s2 = torch.full((2, T), sa), torch.full((1, 2), sw)
        y = torch.empty(T, N, device="cuda")
        rtq.fp8_qgemm(a.cuda(), s1.cuda(), w.cuda(), s2.cuda(), y)
        assert same(y, (row_values(a, s1) @ block_values(w, s2).T).float())
    b1 = torch.zeros(2, T, dtype=torch.uint8).view(E8M0)     # 2^-127
    b2 = torch.full((1, 2), 127 + 100, dtype=torch.uint8).view(E8M0)
    y = torch.empty(T, N, device="cuda")
    rtq.fp8_qgemm(a.cuda(), b1.cuda(), w.cuda(), b2.cuda(), y)
    assert same(y, (a.double() @ w.double().T * 2.0 ** -27).float())


# ------------------------------------------------------------------ the layer and its gradients

@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("T,N,K", [(1, 256, 512), (7, 1000, 4096), (16, 48, 144), (100, 333, 1040), (600, 512, 256), (13, 4096, 16384),
                                   (5, 8200, 144), (3, 16500, 272), (2, 16, 16)])
def test_linear_equals_its_parts(T, N, K, st):
    step("linear", T, N, K, st)
    x = rows_like(T * K, T, K).cuda()
    w = (torch.randn(N, K, generator=gen(N)) * 0.05).bfloat16().cuda()
    wq, ws = torch.empty(N, K, dtype=E4M3, device="cuda"), torch.empty(groups(N), groups(K), dtype=st, device="cuda")
    rtq.fp8_quantize(w, wq, ws, blocks=True)
    codes, scale = empty_rows(T, K, st=st)
    rtq.fp8_quantize(x, codes, scale)
    ref = row_values(codes, scale) @ block_values(wq, ws).T
    c2, s2 = empty_rows(T, K, st=st)
    y = torch.empty(T, N, device="cuda")
    rtq.fp8_linear(x, wq, ws, y, x_codes=c2, x_scale=s2)
    assert same(c2, codes) and same(s2.float(), scale.float())
    assert rel(y, ref) <= GENERAL
    z = torch.empty(T, N, device="cuda")
    rtq.fp8_linear(x, wq, ws, z, workspace=torch.empty(rtq.fp8_linear_workspace(T, N, K), dtype=torch.uint8, device="cuda"))
    assert rel(z, ref) <= GENERAL
    zb = torch.empty(T, N, dtype=BF16, device="cuda")
    rtq.fp8_linear(x.float(), wq, ws, zb)
    assert rel(zb, ref) <= GENERAL + HALF_BF16
    again = torch.empty(T, N, device="cuda")
    rtq.fp8_linear(x, wq, ws, again)
    assert same(again, z)                                    # equal calls give equal bits


@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("T,N,K", [(1, 8, 16), (3, 40, 144), (31, 136, 128), (64, 64, 64), (517, 264, 1040), (1500, 72, 272), (4200, 136, 400), (129, 8, 16), (65, 640, 656)])
def test_wgrad_exact(T, N, K, st):
    """Whole-number operands: every product and sum is exact in fp32."""
    step("wgrad", T, N, K, st)
    dy = torch.randint(-4, 5, (T, N), generator=gen(T)).to(BF16)
    x, sx = int_codes(K, T, K), pow2_scales(9, groups(K), T, -2, 2).to(st)
    ref = dy.double().T @ row_values(x, sx)
    dev = [t.cuda() for t in (dy, x, sx)]
    for dtype in (F32, BF16):
        dw = torch.full((N + 1, K), 7.0, dtype=dtype, device="cuda")
        rtq.fp8_wgrad(*dev, dw[:N])
        assert same(dw[:N], ref.float().to(dtype))
        assert (dw[N] == 7.0).all()
        start = torch.randint(-8, 9, (N, K), generator=gen(2)).to(dtype).cuda()
        dw = start.clone()
        rtq.fp8_wgrad(*dev, dw, accumulate=True)
        assert same(dw, (ref + start.cpu().double()).float().to(dtype))


@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("T,N,K", [(65, 2568, 2576), (130, 4096, 4112), (333, 2600, 3600), (1000, 2824, 2560), (64, 4096, 4096)])
def test_large_wgrad_exact(T, N, K, st):
    """Outputs of many 256 x 256 tiles: whole rounds of them, halves, two to many stages of tokens."""
    step("large wgrad", T, N, K, st)
    dy = torch.randint(-4, 5, (T, N), generator=gen(T)).to(BF16).cuda()
    x, sx = int_codes(K, T, K).cuda(), pow2_scales(9, groups(K), T, -2, 2).to(st).cuda()
    xv = x.double() * sx.double().t().repeat_interleave(128, 1)[:, :K]
    ref = dy.double().t().contiguous() @ xv
    for dtype in (F32, BF16):
        dw = torch.full((N + 1, K), 7.0, dtype=dtype, device="cuda")
        rtq.fp8_wgrad(dy, x, sx, dw[:N])
        assert torch.equal(dw[:N].double(), ref.float().to(dtype).double())
        assert (dw[N] == 7.0).all()
        start = torch.randint(-8, 9, (N, K), generator=gen(2)).to(dtype).cuda()
        dw = start.clone()
        rtq.fp8_wgrad(dy, x, sx, dw, accumulate=True)
        assert torch.equal(dw.double(), (ref + start.double()).float().to(dtype).double())


def test_wgrad_without_rows_writes_zeros():
    step("wgrad T=0")
    dy, x, sx = torch.empty(0, 16, dtype=BF16, device="cuda"), *empty_rows(0, 32)
    dw = torch.full((16, 32), 7.0, device="cuda")
    rtq.fp8_wgrad(dy, x, sx, dw, accumulate=True)
    assert (dw == 7.0).all()
    rtq.fp8_wgrad(dy, x, sx, dw)
    assert (dw == 0.0).all()


@pytest.mark.parametrize("T,N,K", [(200, 136, 272), (1000, 64, 528)])
def test_wgrad_general(T, N, K):
    """fp32 sums of T exact products: at most (T + 1) 2^-23 of the summed magnitudes, in every element.  General
    fp32 scales round the decoded input to bf16 first, 2^-8 of each term."""
    step("wgrad general", T, N, K)
    dy = rows_like(3, T, N)
    q, s = quantise(rows_like(4, T, K), E4M3)
    x, sx = q.float().to(E4M3), s.float()
    dw = torch.empty(N, K, device="cuda")
    rtq.fp8_wgrad(dy.cuda(), x.cuda(), sx.cuda(), dw)
    ref = dy.double().T @ row_values(x, sx)
    size = dy.double().abs().T @ row_values(x, sx).abs()
    assert ((dw.cpu().double() - ref).abs() <= (T + 1) * 2.0 ** -23 * size).all()
    sx = sx * (0.75 + 0.5 * torch.rand(sx.shape, generator=gen(1)))
    rtq.fp8_wgrad(dy.cuda(), x.cuda(), sx.cuda(), dw)
    ref = dy.double().T @ row_values(x, sx)
    size = dy.double().abs().T @ row_values(x, sx).abs()
    assert ((dw.cpu().double() - ref).abs() <= (2.0 ** -8 + (T + 1) * 2.0 ** -22) * size).all()


@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("st", [F32, E8M0])
def test_linear_dgrad_equals_its_parts(st, fmt):
    T, N, K = 77, 272, 400
    step("linear dgrad", st, fmt)
    dy = (rows_like(8, T, N) * 1e-3).cuda()
    w, sw = int_codes(1, N, K, 8).cuda(), pow2_scales(2, groups(N), groups(K)).to(st).cuda()
    q, s = quantise(dy.cpu(), fmt)
    ref = row_values(q, s) @ block_values(w, sw)
    dx = torch.empty(T, K, device="cuda")
    rtq.fp8_linear_dgrad(dy, w, sw, dx, grad_dtype=fmt)
    assert rel(dx, ref) <= GENERAL
    # against differences: <dx, v> = <dy^, (x + v) W^T - x W^T>
    v = torch.randn(T, K, generator=gen(11)).double()
    x = torch.randn(T, K, generator=gen(12)).double()
    diff = ((x + v) @ block_values(w, sw).T - x @ block_values(w, sw).T)
    want = float((row_values(q, s) * diff).sum())
    got = float((dx.cpu().double() * v).sum())
    # v is independent of dx's error e: |<e, v>| is 4 standard deviations of |e| at most
    assert abs(got - want) <= 4 * GENERAL * float(ref.norm())


# ------------------------------------------------------------------ activation checkpoints

@pytest.mark.parametrize("name", sorted(ACTS))
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,d,st", [(1, 16, F32), (3, 528, E8M0), (130, 1040, F32)])
def test_act_forward(T, d, st, dtype, name):
    """y: fp32 evaluation, whose exponential's argument (at most 60 in magnitude here) costs 60 * 2^-23 and whose
    other steps 4 * 2^-23 in relative terms, 1 + erf's cancellation 2^-22 |h|; then the output's own rounding."""
    step("act forward", T, d, st, dtype, name)
    h = (2.0 * torch.randn(T, d, generator=gen(T + d))).to(dtype)
    h[0, :8] = torch.tensor([0.0, -0.0, 6.0, -6.0, 8.5, -8.5, 1e-20, -1e-20])
    codes, scale = empty_rows(T, d, st=st)
    y = torch.empty(T, d, dtype=dtype, device="cuda")
    rtq.act_fp8_forward(h.cuda(), ACTS[name], codes, scale, y=y)
    q, s = quantise(h, E4M3)
    assert same(codes, q) and same(scale.float(), s)
    ref = act(h.double(), name)
    out = HALF_BF16 if dtype == BF16 else 2.0 ** -24
    tol = ref.abs() * (out + 64 * 2.0 ** -23) + (2.0 ** -22 * h.double().abs() if name == "gelu" else 0.0) + 2.0 ** -126
    assert ((y.cpu().double() - ref).abs() <= tol).all()
    # quantised on the way out: the codes of the same values
    c2, s2 = empty_rows(T, d, st=st)
    yc, ys = empty_rows(T, d, st=st)
    rtq.act_fp8_forward(h.cuda(), ACTS[name], c2, s2, y_codes=yc, y_scale=ys)
    assert same(c2, codes) and same(s2.float(), scale.float())
    if dtype == F32:
        q, s = quantise(y.cpu(), E4M3)
        assert same(yc, q) and same(ys.float(), s)
    else:                                       # within one rounding to a code (half a step, 2^-4) of y,
        v = row_values(yc, ys)                  # or half the smallest code of its group
        small = (ys.cpu().double() * 2.0 ** -10).t().repeat_interleave(128, 1)[:, :d]
        assert ((v - ref).abs() <= ref.abs() * 2.0 ** -4 * (1 + 2.0 ** -10) + small * 1.01 + tol).all()


@pytest.mark.parametrize("name", sorted(ACTS))
@pytest.mark.parametrize("dtype,st", [(BF16, F32), (F32, E8M0)])
@pytest.mark.parametrize("T,d", [(1, 16), (5, 528), (130, 1040)])
def test_act_backward(T, d, dtype, st, name):
    """The slope in fp32: each of its few terms is at most 2 |h| + 2 in size (h (1 - p) p and its factors cut off
    beyond |h| = 10) and costs up to 64 * 2^-23 of itself."""
    step("act backward", T, d, dtype, st, name)
    h = 2.0 * torch.randn(T, d, generator=gen(T))
    h[0, :6] = torch.tensor([0.0, 12.0, -12.0, 6.0, -6.0, 0.5])
    q, s = quantise(h, E4M3)
    codes, scale = q.float().to(E4M3).cuda(), s.float().to(st).cuda()
    dy = rows_like(T, T, d, dtype)
    dh = torch.empty(T, d, dtype=dtype, device="cuda")
    rtq.act_fp8_backward(dy.cuda(), codes, scale, ACTS[name], dh)
    hv = row_values(codes, scale)
    want = dy.double() * slope(hv, name)
    out = HALF_BF16 if dtype == BF16 else 2.0 ** -24
    tol = want.abs() * out + dy.double().abs() * (2 * hv.abs().clamp(max=10.0) + 2) * 64 * 2.0 ** -23
    assert ((dh.cpu().double() - want).abs() <= tol).all()
    # against central differences of the 64-bit function: their own error is f''' eps^2 / 6 < eps^2
    eps = 2.0 ** -12
    diff = (act(hv + eps, name) - act(hv - eps, name)) / (2 * eps)
    assert ((dh.cpu().double() - dy.double() * diff).abs() <= tol + dy.double().abs() * (eps * eps + 2.0 ** -36)).all()
    inplace = dy.cuda()
    rtq.act_fp8_backward(inplace, codes, scale, ACTS[name], inplace)
    assert same(inplace, dh)


@pytest.mark.parametrize("name", sorted(ACTS))
def test_act_far_values(name):
    """Magnitudes whose cube or exponential overflows fp32: f(h) is h or 0 and its slope 1 or 0."""
    step("act far", name)
    h = torch.zeros(2, 128)
    h[0, :6] = torch.tensor([1e4, 1e15, 3e38, 200.0, 129.0, 1e30])
    h[1] = -h[0]
    for dtype in (F32, BF16):
        x = h.to(dtype).cuda()
        codes, scale = empty_rows(2, 128)
        y = torch.empty_like(x)
        rtq.act_fp8_forward(x, ACTS[name], codes, scale, y=y)
        assert same(y[0], x[0]) and (y[1] == 0).all()
        dh = torch.empty_like(x)
        rtq.act_fp8_backward(torch.ones_like(x), codes, scale, ACTS[name], dh)
        v = row_values(codes, scale)
        assert same(dh, torch.where(v > 100, 1.0, torch.where(v < -100, 0.0, 0.5)))


# ------------------------------------------------------------------ used together

def _mlp(T, K, H, seed=0):
    x = torch.randn(T, K, generator=gen(seed)).bfloat16()
    w1 = (torch.randn(H, K, generator=gen(seed + 1)) / K ** 0.5).bfloat16()
    w2 = (torch.randn(K, H, generator=gen(seed + 2)) / H ** 0.5).bfloat16()
    dz = torch.randn(T, K, generator=gen(seed + 3)).bfloat16()
    return [t.cuda() for t in (x, w1, w2, dz)]


def _quantised(w, st=F32):
    q = torch.empty(w.shape, dtype=E4M3, device="cuda")
    s = torch.empty(groups(w.shape[0]), groups(w.shape[1]), dtype=st, device="cuda")
    return rtq.fp8_quantize(w, q, s, blocks=True)


class MlpStep:
    """x -> h = x W1^T -> a = f(h) -> z = a W2^T and back, every buffer kept, as a training program would."""

    def __init__(self, T, K, H, st=F32):
        def rows(d):
            return empty_rows(T, d, st=st)
        self.x_ck, self.h_ck, self.a_ck = rows(K), rows(H), rows(H)
        self.h = torch.empty(T, H, dtype=BF16, device="cuda")
        self.z = torch.empty(T, K, dtype=BF16, device="cuda")
        self.da, self.dx = torch.empty_like(self.h), torch.empty_like(self.z)
        self.dw1 = torch.empty(H, K, device="cuda")
        self.dw2 = torch.empty(K, H, device="cuda")
        size = max(rtq.fp8_linear_workspace(T, H, K), rtq.fp8_qgemm_workspace(T, K, H), rtq.fp8_linear_dgrad_workspace(T, K, H),
                   rtq.fp8_linear_dgrad_workspace(T, H, K), rtq.fp8_wgrad_workspace(T, H, K), rtq.fp8_wgrad_workspace(T, K, H))
        self.ws = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")

    def run(self, x, w1, w2, dz, stream=None):
        kw = dict(workspace=self.ws, stream=stream)
        rtq.fp8_linear(x, *w1, self.h, *self.x_ck, **kw)
        rtq.act_fp8_forward(self.h, ACTS["gelu_tanh"], *self.h_ck, y_codes=self.a_ck[0], y_scale=self.a_ck[1], stream=stream)
        rtq.fp8_qgemm(*self.a_ck, *w2, self.z, **kw)
        rtq.fp8_wgrad(dz, *self.a_ck, self.dw2, **kw)
        rtq.fp8_linear_dgrad(dz, *w2, self.da, **kw)
        rtq.act_fp8_backward(self.da, *self.h_ck, ACTS["gelu_tanh"], self.da, stream=stream)
        rtq.fp8_wgrad(self.da, *self.x_ck, self.dw1, **kw)
        rtq.fp8_linear_dgrad(self.da, *w1, self.dx, **kw)
        return self.z, self.dx, self.dw1, self.dw2


@pytest.mark.parametrize("st", [F32, E8M0])
def test_mlp_training_step(st):
    """The gradients of the unquantised MLP in 64 bits.  A code is off by at most 2^-4 of itself, 2^-4 / sqrt(3)
    (3.6%) in the root mean square at the worst place of a binade (e5m2: 7.2%); at most four quantised operands
    stand between any output and its inputs, two of them e5m2 on the longest chain, which together are off by
    sqrt(3 * 3.6^2 + 2 * 7.2^2) = 12%."""
    T, K, H = 200, 272, 528
    step("mlp", st)
    x, w1, w2, dz = _mlp(T, K, H)
    got = MlpStep(T, K, H, st).run(x, _quantised(w1, st), _quantised(w2, st), dz)
    xd, w1d, w2d = (t.cpu().double().requires_grad_(True) for t in (x, w1, w2))
    z = act(xd @ w1d.T, "gelu_tanh") @ w2d.T
    want = (z, *torch.autograd.grad(z, (xd, w1d, w2d), dz.cpu().double()))
    for g, w, n in zip(got, want, ("z", "dx", "dw1", "dw2")):
        assert rel(g, w.detach()) < 0.12, n


def test_rotation_cancels_between_quantised_operands():
    """x and W rotated by the same RPBH before quantising: the product approximates the unrotated one, each operand
    off by 3.6% at most (above)."""
    step("rotated operands")
    T, N, d = 65, 192, 256
    x = rows_like(1, T, d).cuda()
    w = (torch.randn(N, d, generator=gen(2)) * 0.05).bfloat16().cuda()
    R = rtq.Rpbh.from_seed(5, d)
    xr, wr = torch.empty_like(x), torch.empty_like(w)
    rtq.rpbh_rotate(x, xr, R)
    rtq.rpbh_rotate(w, wr, R)
    y = torch.empty(T, N, dtype=BF16, device="cuda")
    rtq.fp8_linear(xr, *_quantised(wr), y)
    assert rel(y, x.cpu().double() @ w.cpu().double().T) < 0.06


@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("T,N,K", [(1024, 1920, 1920), (1025, 1920, 2000), (1090, 2000, 1920), (2500, 2048, 2048), (2113, 1928, 2032)])
def test_wgrad_many_tokens_exact(T, N, K, st):
    """More tokens in one part than a table of scales holds, one stage and many past it."""
    step("wgrad many tokens", T, N, K, st)
    dy = torch.randint(-4, 5, (T, N), generator=gen(T)).to(BF16).cuda()
    x, sx = int_codes(K, T, K).cuda(), pow2_scales(9, groups(K), T, -2, 2).to(st).cuda()
    ref = dy.double().t().contiguous() @ (x.double() * sx.double().t().repeat_interleave(128, 1)[:, :K])
    dw = torch.full((N + 1, K), 7.0, device="cuda")
    rtq.fp8_wgrad(dy, x, sx, dw[:N])
    assert torch.equal(dw[:N].double(), ref) and (dw[N] == 7.0).all()


@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("T,N,K", [(130, 528, 1040), (391, 1000, 1936), (33, 2064, 272), (512, 256, 2048)])
def test_direct_layer_keeps_the_codes(T, N, K, st):
    """The layers that quantise on the way, at more than 16 rows: what they keep is what the quantiser writes, and
    the gradient's two code types."""
    step("direct layer", T, N, K, st)
    x = rows_like(T * K, T, K).cuda()
    wq, ws = _quantised((torch.randn(N, K, generator=gen(N)) * 0.05).bfloat16().cuda(), st)
    codes, scale = empty_rows(T, K, st=st)
    rtq.fp8_quantize(x, codes, scale)
    c2, s2 = empty_rows(T, K, st=st)
    y = torch.empty(T, N, device="cuda")
    rtq.fp8_linear(x, wq, ws, y, x_codes=c2, x_scale=s2)
    assert same(c2, codes) and same(s2.float(), scale.float())
    assert rel(y, row_values(codes, scale) @ block_values(wq, ws).T) <= GENERAL
    g = rows_like(7, T, (N + 15) // 16 * 16).cuda()[:, :N // 16 * 16].contiguous()
    wg, wgs = _quantised((torch.randn(g.shape[1], K, generator=gen(N)) * 0.05).bfloat16().cuda(), st)
    for fmt in (E4M3, E5M2):
        gc, gs = empty_rows(T, g.shape[1], fmt, st)
        rtq.fp8_quantize(g, gc, gs)
        dx = torch.empty(T, K, device="cuda")
        rtq.fp8_linear_dgrad(g, wg, wgs, dx, grad_dtype=fmt)
        assert rel(dx, row_values(gc, gs) @ block_values(wg, wgs)) <= GENERAL


@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("T,out,R", [(3, 8208, 8192), (3, 304, 5008), (16, 4112, 4096), (7, 9216, 1040), (1, 8208, 1936), (16, 4624, 2064)])
def test_few_row_layers_and_gradients(T, out, R, st):
    """Both sides of the rules for few rows: quantised on the way or before, one to four tiles of columns, forward and
    transposed, against the quantiser's codes."""
    step("few rows", T, out, R, st)
    x = rows_like(T + R, T, R).cuda()
    for trans in (False, True):
        w, ws = _quantised((torch.randn(*((R, out) if trans else (out, R)), generator=gen(out)) * 0.05).bfloat16().cuda(), st)
        wv = block_values(w, ws)
        for fmt in (E4M3, E5M2) if trans else (E4M3,):
            codes, scale = empty_rows(T, R, fmt, st)
            rtq.fp8_quantize(x, codes, scale)
            for dtype in (F32, BF16):
                y = torch.full((T + 1, out), 7.0, dtype=dtype, device="cuda")
                if trans:
                    rtq.fp8_linear_dgrad(x, w, ws, y[:T], grad_dtype=fmt)
                else:
                    rtq.fp8_linear(x, w, ws, y[:T])
                assert rel(y[:T], row_values(codes, scale) @ (wv if trans else wv.T)) <= GENERAL + (HALF_BF16 if dtype == BF16 else 0.0)
                assert (y[T] == 7.0).all()


def test_captured_step_replays():
    """A captured training step, replayed with new inputs in its buffers and eager work between the replays."""
    step("captured step")
    T, K, H = 96, 256, 384
    x, w1, w2, dz = _mlp(T, K, H)
    q1, q2 = _quantised(w1), _quantised(w2)
    kept = MlpStep(T, K, H)
    eager = MlpStep(T, K, H)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kept.run(x, q1, q2, dz)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept.run(x, q1, q2, dz)
    for k in range(4):
        nx, _, _, nz = _mlp(T, K, H, seed=10 + k)
        x.copy_(nx)
        dz.copy_(nz)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (kept.z, kept.dx, kept.dw1, kept.dw2)]
        want = eager.run(x, q1, q2, dz)
        for g, w in zip(got, want):
            assert same(g, w)


def test_two_streams_with_their_own_workspaces():
    step("two streams")
    T, K, H = 33, 512, 640
    x, w1, w2, dz = _mlp(T, K, H)
    q1, q2 = _quantised(w1), _quantised(w2)
    want = [t.clone() for t in MlpStep(T, K, H).run(x, q1, q2, dz)]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    steps = [MlpStep(T, K, H) for _ in range(2)]
    for _ in range(3):
        for s, m in zip((a, b), steps):
            m.run(x, q1, q2, dz, stream=s)
    torch.cuda.synchronize()
    for m in steps:
        for g, w in zip((m.z, m.dx, m.dw1, m.dw2), want):
            assert same(g, w)
    y = torch.empty(T, H, dtype=BF16, device="cuda")     # a temporary workspace, on a stream of its own
    rtq.fp8_linear(x, *q1, y, stream=a)
    torch.cuda.synchronize()
    assert same(y, steps[0].h)


def test_offsets_past_32_bits():
    """More than 2^31 codes, and outputs more than 2^31 elements in."""
    step("big rows")
    T, d = 140000, 16384
    x = torch.zeros(T, d, dtype=BF16, device="cuda")
    x[-1] = torch.arange(d, device="cuda").bfloat16()
    x[-2, 5] = -3.0
    codes, scale = empty_rows(T, d)
    rtq.fp8_quantize(x, codes, scale)
    q, s = quantise(x[-2:].cpu(), E4M3)
    assert same(codes[-2:], q) and same(scale[:, -2:], s) and (scale[:, :-2] == 1.0).all()
    dh = x
    rtq.act_fp8_backward(x, codes, scale, ACTS["silu"], dh)
    want = x.new_zeros(0)
    del want, codes, scale
    step("big product")
    K = 32
    a = torch.zeros(T, K, device="cuda").to(E4M3)
    a[-3:] = int_codes(1, 3, K).cuda()
    w = int_codes(2, d, K).cuda()
    sa, sw = torch.ones(1, T, device="cuda"), torch.ones(groups(d), 1, device="cuda")
    rtq.fp8_qgemm(a, sa, w, sw, x)
    assert same(x[-3:], (a[-3:].cpu().double() @ w.cpu().double().T).bfloat16())
    assert not x[:-3].any()


def test_launches_of_more_than_2_32_work_items():
    """More rows than one dimension of a launch holds threads for."""
    torch.cuda.empty_cache()
    T, d = (1 << 29) + 37, 16
    step("many narrow rows")
    x = torch.zeros(T, d, dtype=BF16, device="cuda")
    tail = rows_like(3, 5, d)
    x[-5:] = tail.cuda()
    codes, scale = empty_rows(T, d)
    codes.view(torch.uint8).fill_(9)
    rtq.fp8_quantize(x, codes, scale)
    q, s = quantise(tail, E4M3)
    assert same(codes[-5:], q) and same(scale[:, -5:], s)
    assert not codes[:-5].view(torch.uint8).any() and (scale[:, :-5] == 1.0).all()
    del x, scale
    step("many narrow tiles")
    T = (1 << 30) + 70
    codes = torch.zeros(T, d, dtype=torch.uint8, device="cuda").view(E4M3)
    a = int_codes(1, 5, d)
    codes[-5:] = a.cuda()
    w, sw = int_codes(2, 8, d), torch.ones(1, 1, device="cuda")
    y = torch.full((T, 8), 7.0, dtype=BF16, device="cuda")
    rtq.fp8_qgemm(codes, torch.ones(1, T, device="cuda"), w.cuda(), sw, y)
    assert same(y[-5:], (a.double() @ w.double().T).bfloat16())
    assert not y[:-5].any()


def before_nans(t):
    """A copy of t on the GPU whose buffer goes on with 64 KB of NaNs."""
    bits = t.contiguous().view(torch.uint8).flatten()
    nan = {E4M3: 0x7f, E5M2: 0x7f, E8M0: 0xff, BF16: 0xff, F32: 0xff}[t.dtype]
    buffer = torch.full((bits.numel() + (1 << 16),), nan, dtype=torch.uint8, device="cuda")
    buffer[:bits.numel()] = bits.cuda()
    return buffer[:bits.numel()].view(t.dtype).view(t.shape)


@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("T,N,R", [(1, 16, 144), (5, 208, 528), (13, 4112, 1040), (16, 8208, 272), (40, 208, 1040), (70, 528, 4112),
                                   (1000, 4000, 400), (4100, 1488, 272)])
def test_products_of_operands_with_nans_behind_them(T, N, R, trans, st):
    """Every form, the last block and tile ragged: what lies behind an operand does not reach the product."""
    step("NaNs behind", T, N, R, trans, st)
    a, w = int_codes(T + R, T, R), int_codes(N + 1, R if trans else N, N if trans else R)
    sa = pow2_scales(3, groups(R), T, -1, 1).to(st)
    sw = pow2_scales(4, groups(w.shape[0]), groups(w.shape[1]), -1, 1).to(st)
    av, wv = row_values(a, sa).cuda(), block_values(w, sw).cuda()
    ref = av @ (wv if trans else wv.t().contiguous())
    y = torch.empty(T, N, device="cuda")
    (rtq.fp8_dgrad if trans else rtq.fp8_qgemm)(*[before_nans(t) for t in (a, sa, w, sw)], y)
    assert torch.equal(y.double(), ref)
    x = torch.randint(-8, 9, (T, R), generator=gen(5)).to(BF16)      # whole numbers: exact codes, any scale
    q, s = quantise(x, E4M3)
    ref = row_values(q, s).cuda() @ (wv if trans else wv.t().contiguous())
    for dtype in (BF16, F32):
        if trans:
            rtq.fp8_linear_dgrad(before_nans(x.to(dtype)), before_nans(w), before_nans(sw), y, grad_dtype=E4M3)
        else:
            rtq.fp8_linear(before_nans(x.to(dtype)), before_nans(w), before_nans(sw), y)
        assert torch.equal(y.double(), ref)


@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("T,N,K", [(1, 8, 16), (77, 136, 272), (517, 264, 1040), (65, 2568, 2576), (333, 2600, 3600)])
def test_wgrad_of_operands_with_nans_behind_them(T, N, K, st):
    step("wgrad NaNs behind", T, N, K, st)
    dy = torch.randint(-4, 5, (T, N), generator=gen(T)).to(BF16)
    x, sx = int_codes(K, T, K), pow2_scales(9, groups(K), T, -2, 2).to(st)
    ref = dy.cuda().double().t().contiguous() @ row_values(x, sx).cuda()
    dw = torch.empty(N, K, device="cuda")
    rtq.fp8_wgrad(*[before_nans(t) for t in (dy, x, sx)], dw)
    assert torch.equal(dw.double(), ref)


def _below_zero(T, d):
    """Groups of 128 that lie wholly in [-8, -4], [-13, -8], [-4, 0] in turn."""
    lo = torch.tensor([-8.0, -13.0, -4.0])[torch.arange(d) // 128 % 3]
    hi = torch.tensor([-4.0, -8.0, 0.0])[torch.arange(d) // 128 % 3]
    return lo + (hi - lo) * torch.rand(T, d, generator=gen(T + d))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,d", [(1, 384), (37, 784)])
def test_gelu_below_zero(T, d, dtype):
    """GELU (erf) keeps its relative accuracy where it is small.  y = h q, q the normal distribution's tail, which falls
    as exp(-h^2 / 2): three roundings of that exponent (the constant's 2^-25, two products' 2^-24) cost at most
    h^2 2^-23, the exponential, a reciprocal and some ten further operations at most 18 * 2^-23; then y's rounding."""
    step("gelu below zero", T, d, dtype)
    h = _below_zero(T, d).to(dtype)
    codes, scale = empty_rows(T, d)
    y = torch.empty(T, d, dtype=dtype, device="cuda")
    rtq.act_fp8_forward(h.cuda(), ACTS["gelu"], codes, scale, y=y)
    ref = act(h.double(), "gelu")
    own = ref.abs() * (h.double() ** 2 + 18) * 2.0 ** -23 + 2.0 ** -126
    tol = own + ref.abs() * (HALF_BF16 if dtype == BF16 else 2.0 ** -24)
    assert ((y.cpu().double() - ref).abs() <= tol).all()
    # as codes: half a step (2^-4) of y, or half the smallest code (2^-10) of a group whose scale follows y's size
    yc, ys = empty_rows(T, d)
    rtq.act_fp8_forward(h.cuda(), ACTS["gelu"], codes, scale, y_codes=yc, y_scale=ys)
    top = torch.nn.functional.pad((ref.abs() + own), (0, groups(d) * 128 - d)).view(T, -1, 128).amax(2).t()
    assert (ys.cpu().double() * 448.0 <= 2 * top * (1 + 2.0 ** -10)).all()      # the smallest power of two that holds it
    small = (ys.cpu().double() * 2.0 ** -10).t().repeat_interleave(128, 1)[:, :d]
    assert ((row_values(yc, ys) - ref).abs() <= own + (ref.abs() + own) * 2.0 ** -4 + small).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,d", [(1, 384), (37, 784)])
def test_gelu_slope_below_zero(T, d, dtype):
    """q + h phi(h): the first term as above, (h^2 + 18) 2^-23 of itself; the density has the same exponential, and two
    products' roundings.  The terms have opposite signs below zero: the bound is on their sum of magnitudes, at most
    (h^2 + 19) 2^-23 of it with the addition's rounding; a density below fp32's normal range may be 0."""
    step("gelu slope below zero", T, d, dtype)
    q, s = quantise(_below_zero(T, d), E4M3)
    codes, scale = q.float().to(E4M3).cuda(), s.float().cuda()
    hv = row_values(codes, scale)
    dy = rows_like(T, T, d, dtype)
    dh = torch.empty(T, d, dtype=dtype, device="cuda")
    rtq.act_fp8_backward(dy.cuda(), codes, scale, ACTS["gelu"], dh)
    want = dy.double() * slope(hv, "gelu")
    first = 0.5 * torch.erfc(-hv / 2.0 ** 0.5)
    second = hv.abs() * torch.exp(-0.5 * hv * hv) / (2 * torch.pi) ** 0.5
    tol = dy.double().abs() * ((first + second) * (hv * hv + 19) * 2.0 ** -23 + 16 * 2.0 ** -126) + 2.0 ** -126
    assert ((dh.cpu().double() - want).abs() <= tol + want.abs() * (HALF_BF16 if dtype == BF16 else 2.0 ** -23)).all()


def _values(codes, scale, blocks=False):
    """What codes stand for, on their device (float64)."""
    s = scale.double()
    s = s.repeat_interleave(128, 0)[:codes.shape[0]] if blocks else s.t()
    return codes.double() * s.repeat_interleave(128, 1)[:, :codes.shape[1]]


def _block_amax(v, dim):
    """Largest magnitude of each 128 along a dimension, which comes last."""
    v = v.abs().movedim(dim, 1)
    return torch.nn.functional.pad(v, (0, groups(v.shape[1]) * 128 - v.shape[1])).view(v.shape[0], -1, 128).amax(2)


# one size for each way a product runs: few rows, small, 64 tiles, split, 128 tiles, 256 tiles, long and 256 tiles
FORMS = [(5, 208, 2064), (100, 336, 1040), (300, 512, 2064), (64, 4096, 4096), (1000, 4000, 400), (2500, 2800, 2064), (2500, 2800, 8208)]


@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("T,N,R", FORMS)
def test_general_operands_in_every_form(T, N, R, trans, fmt, st):
    """Codes over the whole range and, in fp32, scales that are no powers of two.  In the 2-norm as above; in every
    element: an instruction cuts each of 128 products at 2^-13 of the largest, 2^-6 of it in all, which is at most the
    product of the block's largest factors.  (In fp32 sums, or E8M0 ones within the instruction at 2^-20 a block of the
    running sum, which is at most 128 of those products: 2^-13 a block, 2^-6 over 128 blocks: 2^-5 together.)"""
    step("general", T, N, R, trans, fmt, st)
    x = rows_like(T + R, T, R).cuda()
    w = (torch.randn(R if trans else N, N if trans else R, generator=gen(N)) * torch.exp(0.5 * torch.randn(1, generator=gen(3)))).cuda()
    a, sa = empty_rows(T, R, fmt, st)
    rtq.fp8_quantize(x, a, sa)
    wq, sw = torch.empty(w.shape, dtype=E4M3, device="cuda"), torch.empty(groups(w.shape[0]), groups(w.shape[1]), dtype=st, device="cuda")
    rtq.fp8_quantize(w, wq, sw, blocks=True)
    if st == F32:
        sa *= 0.75 + 0.5 * torch.rand(sa.shape, generator=gen(1)).cuda()
        sw *= 0.75 + 0.5 * torch.rand(sw.shape, generator=gen(2)).cuda()
    av, wv = _values(a, sa), _values(wq, sw, blocks=True)
    ref = av @ (wv if trans else wv.t().contiguous())
    each = _block_amax(av, 1) @ _block_amax(wv, 0 if trans else 1).t().contiguous()
    for dtype in (F32, BF16):
        y = torch.empty(T, N, dtype=dtype, device="cuda")
        (rtq.fp8_dgrad if trans else rtq.fp8_qgemm)(a, sa, wq, sw, y)
        out = HALF_BF16 if dtype == BF16 else 0.0
        assert float((y.double() - ref).norm() / ref.norm()) <= GENERAL + out
        assert ((y.double() - ref).abs() <= 2.0 ** -5 * each * (1 + out) + out * ref.abs()).all()


@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("T,N,R", [(4, 512, 2048), (64, 512, 2048), (1000, 4000, 2048), (2500, 2800, 2048)])
def test_small_blocks_behind_a_large_one(T, N, R, st):
    """Block sums of 1 behind one of 2^k: in fp32 every sum here is exact.  E8M0 blocks of the 256 x 256 tiles are added
    by the instruction, which may cut off 2^-20 of the running sum in each of the 15 blocks."""
    step("small blocks behind a large one", T, N, R, st)
    a, w = torch.ones(T, R, device="cuda").to(E4M3), torch.ones(N, R, device="cuda").to(E4M3)
    sw = torch.ones(groups(N), groups(R), device="cuda").to(st)
    for k in (0, 10, 17, 20, 23):
        sa = torch.full((groups(R), T), 2.0 ** -7, device="cuda")
        sa[0] = 2.0 ** (k - 7)
        y = torch.empty(T, N, device="cuda")
        rtq.fp8_qgemm(a, sa.to(st), w, sw, y)
        want = 2.0 ** k + 15
        cut = 15 * 2.0 ** -20 * want if st == E8M0 and T * N > 1 << 22 else 0.0
        assert ((y.double() - want).abs() <= cut).all()


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("T,N,R", [(5, 208, 272), (1000, 4000, 400), (4100, 1488, 272)])
def test_extreme_scales_in_every_form(T, N, R, trans):
    """Scales at both ends of their range, in fp32 and as E8M0 bytes; byte 0 is 2^-127."""
    step("extreme scales", T, N, R, trans)
    a, w = int_codes(1, T, R).cuda(), int_codes(2, R if trans else N, N if trans else R).cuda()
    ref = a.double() @ (w.double() if trans else w.double().t().contiguous())
    call = rtq.fp8_dgrad if trans else rtq.fp8_qgemm

    def product(sa, sw, st):
        s1 = torch.full((groups(R), T), sa, device="cuda").to(st)
        s2 = torch.full((groups(w.shape[0]), groups(w.shape[1])), sw, device="cuda").to(st)
        y = torch.empty(T, N, device="cuda")
        call(a, s1, w, s2, y)
        return y
    for ea, ew in ((100, -100), (-120, 120), (-60, -60), (-127, 100), (100, -127), (60, 50), (-127, 127), (127, -127), (-40, -70)):
        for st in (F32, E8M0):
            assert torch.equal(product(2.0 ** ea, 2.0 ** ew, st).double(), ref * 2.0 ** (ea + ew)), (ea, ew, st)
    assert not product(0.0, 1.0, F32).any()


@pytest.mark.parametrize("T,N,K", [(200, 136, 272), (333, 2600, 3600), (1000, 2824, 2560)])
def test_wgrad_general_scales_in_every_form(T, N, K):
    """Sums of T products in fp32, and with general scales each term's decoded input rounded to bf16: in every element
    2^-8 of the terms' magnitudes and (T + 1) 2^-22 for the sums."""
    step("wgrad general scales", T, N, K)
    dy = rows_like(3, T, N).cuda()
    x, sx = empty_rows(T, K)
    rtq.fp8_quantize(rows_like(4, T, K).cuda(), x, sx)
    for general in (False, True):
        if general:
            sx *= 0.75 + 0.5 * torch.rand(sx.shape, generator=gen(1)).cuda()
        xv, g = _values(x, sx), dy.double().t().contiguous()
        ref, size = g @ xv, g.abs() @ xv.abs()
        tol = ((2.0 ** -8 if general else 0.0) + (T + 1) * 2.0 ** -22) * size
        for dtype in (F32, BF16):
            dw = torch.empty(N, K, dtype=dtype, device="cuda")
            rtq.fp8_wgrad(dy, x, sx, dw)
            assert ((dw.double() - ref).abs() <= tol + (HALF_BF16 * (ref.abs() + tol) if dtype == BF16 else 0.0)).all()


def test_row_passes_past_32_bits():
    """Activations and their gradient, and codes read back, in the last rows of more than 2^31 elements."""
    torch.cuda.empty_cache()
    T, d = 140000, 16384
    step("row passes past 2^31")
    h = torch.zeros(T, d, dtype=BF16, device="cuda")
    tail = rows_like(5, 3, d)
    h[-3:] = tail.cuda()
    codes, scale = empty_rows(T, d)
    y = torch.full((T, d), 7.0, dtype=BF16, device="cuda")
    rtq.act_fp8_forward(h, ACTS["silu"], codes, scale, y=y)
    small, s1 = empty_rows(3, d)
    want = torch.empty(3, d, dtype=BF16, device="cuda")
    rtq.act_fp8_forward(tail.cuda(), ACTS["silu"], small, s1, y=want)       # checked against 64 bits elsewhere
    assert same(y[-3:], want) and not y[:-3].any()
    assert same(codes[-3:], small) and same(scale[:, -3:], s1)
    step("read back past 2^31")
    y.fill_(7.0)
    rtq.fp8_dequantize(codes, scale, y)
    assert same(y[-3:], row_values(small, s1).float().bfloat16()) and not y[:-3].any()
    step("gradient past 2^31")
    h[:] = 1.0
    grad = rows_like(6, 3, d)
    h[-3:] = grad.cuda()
    rtq.act_fp8_backward(h, codes, scale, ACTS["silu"], y)
    rtq.act_fp8_backward(grad.cuda(), small, s1, ACTS["silu"], want)
    assert same(y[-3:], want) and (y[:-3] == 0.5).all()                     # the slope of SiLU at 0
    step("weight blocks past 2^31")
    w = y.fill_(0.0)
    w[-3:] = tail.cuda()
    q, s = quantise(torch.cat([torch.zeros(T % 128 - 3, d), tail.float()]), E4M3, blocks=True)      # the last row of blocks
    bs = torch.empty(groups(T), groups(d), device="cuda")
    rtq.fp8_quantize(w, codes, bs, blocks=True)
    assert same(codes[-3:], q[-3:]) and same(bs[-1], s[0]) and (bs[:-1] == 1.0).all()


@pytest.mark.parametrize("trans", [False, True])
def test_large_products_past_32_bits(trans):
    """256 x 256 tiles: more than 2^31 outputs, and more than 2^31 codes."""
    torch.cuda.empty_cache()
    for T, N, R in ((140000, 16384, 272), (140000, 272, 16384)):
        step("large product past 2^31", T, N, R, trans)
        a = torch.zeros(T, R, device="cuda", dtype=torch.uint8).view(E4M3)
        tail = int_codes(1, 3, R)
        a[-3:] = tail.cuda()
        w = int_codes(2, R if trans else N, N if trans else R).cuda()
        sa, sw = torch.ones(groups(R), T, device="cuda"), torch.ones(groups(w.shape[0]), groups(w.shape[1]), device="cuda")
        y = torch.full((T, N), 7.0, dtype=BF16, device="cuda")
        (rtq.fp8_dgrad if trans else rtq.fp8_qgemm)(a, sa, w, sw, y)
        ref = tail.double().cuda() @ (w.double() if trans else w.double().t().contiguous())
        assert same(y[-3:], ref.float().bfloat16()) and not y[:-3].any()
        del a, y


@pytest.mark.parametrize("T,N,K", [(64, 65544, 32784), (70, 65544, 32784), (270000, 8200, 144)])
def test_wgrad_past_32_bits(T, N, K):
    """Both kernels with more than 2^31 gradients, and with more than 2^31 output gradients."""
    torch.cuda.empty_cache()
    step("wgrad past 2^31", T, N, K)
    dy = torch.zeros(T, N, dtype=BF16, device="cuda")
    dy[-3:, -16:] = torch.randint(-4, 5, (3, 16), generator=gen(1)).to(BF16).cuda()
    x = int_codes(K, 16, K).cuda().view(torch.uint8).repeat(-(-T // 16), 1)[:T].contiguous().view(E4M3)
    sx = torch.ones(groups(K), T, device="cuda")
    dw = torch.full((N, K), 7.0, dtype=BF16, device="cuda")
    rtq.fp8_wgrad(dy, x, sx, dw)
    ref = dy[-3:, -16:].double().t().contiguous() @ x[-3:].double()
    assert same(dw[-16:], ref.float().bfloat16()) and not dw[:-16].any()


@pytest.mark.parametrize("st", [F32, E8M0])
@pytest.mark.parametrize("T,N,R", [(5, 208, 528), (70, 208, 528), (200, 4096, 1040), (1000, 4000, 400), (4100, 1488, 272)])
def test_infinite_gradient_codes(T, N, R, st):
    """An infinite E5M2 code times positive weights, forward and transposed, in every form; and with its opposite: NaN."""
    step("infinite codes", T, N, R, st)
    for trans in (False, True):
        a, w = torch.ones(T, R).to(E5M2), torch.ones(R if trans else N, N if trans else R, device="cuda").to(E4M3)
        a[0, R - 1], a[T // 2, 1], a[T // 2, 2] = -float("inf"), float("inf"), -float("inf")
        sa, sw = torch.ones(groups(R), T, device="cuda").to(st), torch.ones(groups(w.shape[0]), groups(w.shape[1]), device="cuda").to(st)
        y = torch.empty(T, N, device="cuda")
        (rtq.fp8_dgrad if trans else rtq.fp8_qgemm)(a.cuda(), sa, w, sw, y)
        assert (y[0] == -float("inf")).all() and torch.isnan(y[T // 2]).all()
        assert (y[[t for t in range(T) if t not in (0, T // 2)]] == R).all()


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("T,N,R", [(3, 48, 1 << 20), (70, 80, 1 << 20), (2, 1 << 20, 16), (40, 1 << 20, 32), (300, 1 << 20, 272),
                                   (4100, 4112, (1 << 20) - 16)])
def test_longest_rows(T, N, R, trans):
    """The largest reductions and outputs, exact: codes to 1, at most 2^20 of them."""
    torch.cuda.empty_cache()
    step("longest rows", T, N, R, trans)
    g = torch.Generator(device="cuda").manual_seed(T)

    def signs(rows, d):
        return torch.randint(-1, 2, (rows, d), generator=g, device="cuda", dtype=torch.int8).to(BF16).to(E4M3)
    a, w = signs(T, R), signs(R if trans else N, N if trans else R)
    sa, sw = torch.ones(groups(R), T, device="cuda"), torch.ones(groups(w.shape[0]), groups(w.shape[1]), device="cuda")
    y = torch.full((T + 1, N), 7.0, device="cuda")
    (rtq.fp8_dgrad if trans else rtq.fp8_qgemm)(a, sa, w, sw, y[:T])
    rows = [0, T // 2, T - 1]
    ref = torch.zeros(3, N, dtype=torch.float64, device="cuda")
    for k in range(0, R, 1 << 15):
        part = w[k:k + (1 << 15)] if trans else w[:, k:k + (1 << 15)].t().contiguous()
        ref += a[rows, k:k + (1 << 15)].double() @ part.double()
    assert torch.equal(y[rows].double(), ref) and (y[T] == 7.0).all()
    if R <= 272:
        x = torch.empty(T, R, dtype=BF16, device="cuda").copy_(a.to(BF16))
        z = torch.empty(T, N, device="cuda")
        if trans:
            rtq.fp8_linear_dgrad(x, w, sw, z, grad_dtype=E4M3)
        else:
            rtq.fp8_linear(x, w, sw, z)
        assert torch.equal(z[rows].double(), ref)


@pytest.mark.parametrize("T,N,K", [(3, 1 << 20, 16), (70, 1 << 20, 144), (3, 8, 1 << 20), (130, 264, 1 << 20)])
def test_wgrad_longest_rows(T, N, K):
    torch.cuda.empty_cache()
    step("wgrad longest rows", T, N, K)
    dy = torch.randint(-4, 5, (T, N), generator=gen(T)).to(BF16).cuda()
    x, sx = int_codes(1, T, K).cuda(), pow2_scales(9, groups(K), T, -2, 2).cuda()
    dw = torch.full((N + 1, K), 7.0, device="cuda")
    rtq.fp8_wgrad(dy, x, sx, dw[:N])
    xv = _values(x, sx)
    for part in (slice(0, 200), slice(N - 200 if N > 200 else 0, N)):
        assert torch.equal(dw[:N][part].double(), dy[:, part].double().t().contiguous() @ xv)
    assert (dw[N] == 7.0).all()


def test_longest_quantised_rows():
    step("longest quantised rows")
    T, d = 3, 1 << 20
    x = rows_like(1, T, d).cuda()
    codes, scale = empty_rows(T, d)
    rtq.fp8_quantize(x, codes, scale)
    part = x[:, -4096:].contiguous()
    c1, s1 = empty_rows(T, 4096)
    rtq.fp8_quantize(part, c1, s1)
    assert same(codes[:, -4096:], c1) and same(scale[-32:], s1)
    dh = torch.empty_like(x)
    rtq.act_fp8_backward(x, codes, scale, ACTS["gelu"], dh)
    d1 = torch.empty_like(part)
    rtq.act_fp8_backward(part, c1, s1, ACTS["gelu"], d1)
    assert same(dh[:, -4096:], d1)
