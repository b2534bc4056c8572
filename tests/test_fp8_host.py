"""CPU tests of the 8-bit floating point calls: argument checks of the C ABI (run before any HIP call) and
of the Python binding, workspace sizes, and the plain forms the GPU tests compare with."""
import pytest
import torch

import rotation_then_quantize_amd as rtq
from _fp8 import E4M3, E5M2, TOP, quantise, round_to, scale_of

A = 0x10000      # a fake, 16-byte aligned "device" address: never dereferenced by the host checks
OK, INVALID, UNSUPPORTED, MISALIGNED = rtq.RTQ_OK, rtq.RTQ_ERR_INVALID_ARG, rtq.RTQ_ERR_UNSUPPORTED, rtq.RTQ_ERR_MISALIGNED
F32, BF16, I32 = rtq.RTQ_F32, rtq.RTQ_BF16, rtq.RTQ_I32
C4, C5, S8 = rtq.RTQ_E4M3, rtq.RTQ_E5M2, rtq.RTQ_E8M0
BIG = 1 << 40


def call(name, good, **change):
    args = dict(good)
    assert set(change) <= set(args)
    args.update(change)
    return getattr(rtq.load_library(), name)(*args.values())


QUANT = dict(x=A, xt=BF16, rows=4, d=256, layout=0, codes=A, ct=C4, scale=A, st=F32, stream=None)
DEQUANT = dict(codes=A, ct=C4, scale=A, st=F32, rows=4, d=256, layout=0, y=A, yt=BF16, stream=None)
GEMM = dict(a=A, at=C4, a_scale=A, T=4, w=A, w_scale=A, st=F32, N=33, K=256, y=A, yt=BF16, ws=None, nbytes=0, stream=None)
DGRAD = dict(g=A, gt=C5, g_scale=A, T=4, w=A, w_scale=A, st=S8, N=32, K=256, dx=A, dxt=BF16, ws=None, nbytes=0, stream=None)
LINEAR = dict(x=A, xt=BF16, T=4, w=A, w_scale=A, st=F32, N=33, K=256, x_codes=None, x_scale=None, y=A, yt=BF16, ws=A,
              nbytes=BIG, stream=None)
LDGRAD = dict(dy=A, dyt=BF16, gt=C5, T=4, w=A, w_scale=A, st=F32, N=32, K=256, dx=A, dxt=BF16, ws=A, nbytes=BIG, stream=None)
WGRAD = dict(dy=A, T=4, x=A, x_scale=A, st=F32, N=40, K=256, dw=A, dwt=F32, accumulate=0, ws=None, nbytes=0, stream=None)
ACT = dict(h=A, ht=BF16, rows=4, d=256, act=1, h_codes=A, h_scale=A, y=A, y_codes=None, y_scale=None, st=F32, stream=None)
ACTB = dict(dy=A, dyt=BF16, h_codes=A, h_scale=A, st=F32, rows=4, d=256, act=1, dh=A, stream=None)

REFUSALS = [
    ("rtq_fp8_quantize", QUANT, [
        (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scale=None), INVALID), (dict(x=A + 8), MISALIGNED),
        (dict(scale=A + 4), MISALIGNED), (dict(xt=I32), UNSUPPORTED), (dict(xt=C4), UNSUPPORTED), (dict(ct=BF16), UNSUPPORTED),
        (dict(st=BF16), UNSUPPORTED), (dict(st=C4), UNSUPPORTED), (dict(rows=-1), INVALID), (dict(rows=1 << 31), UNSUPPORTED),
        (dict(d=0), INVALID), (dict(d=-16), INVALID), (dict(d=24), UNSUPPORTED), (dict(d=(1 << 20) + 16), UNSUPPORTED),
        (dict(layout=2), INVALID), (dict(layout=-1), INVALID)]),
    ("rtq_fp8_dequantize", DEQUANT, [
        (dict(codes=None), INVALID), (dict(y=None), INVALID), (dict(y=A + 2), MISALIGNED), (dict(ct=F32), UNSUPPORTED),
        (dict(yt=C4), UNSUPPORTED), (dict(st=I32), UNSUPPORTED), (dict(d=100), UNSUPPORTED), (dict(layout=7), INVALID)]),
    ("rtq_fp8_qgemm", GEMM, [
        (dict(a=None), INVALID), (dict(w=None), INVALID), (dict(w_scale=None), INVALID), (dict(y=None), INVALID),
        (dict(a_scale=None), INVALID), (dict(w=A + 8), MISALIGNED), (dict(at=BF16), UNSUPPORTED), (dict(st=BF16), UNSUPPORTED),
        (dict(yt=I32), UNSUPPORTED), (dict(T=-1), INVALID), (dict(N=0), INVALID), (dict(N=(1 << 20) + 1), UNSUPPORTED),
        (dict(K=8), UNSUPPORTED), (dict(K=0), INVALID), (dict(ws=A + 8, nbytes=64), MISALIGNED),
        (dict(T=(1 << 31) - 1, N=1 << 20), UNSUPPORTED)]),
    ("rtq_fp8_dgrad", DGRAD, [
        (dict(g=None), INVALID), (dict(dx=None), INVALID), (dict(N=40), UNSUPPORTED), (dict(K=40), UNSUPPORTED),
        (dict(gt=S8), UNSUPPORTED), (dict(dxt=C5), UNSUPPORTED), (dict(ws=A + 4, nbytes=64), MISALIGNED)]),
    ("rtq_fp8_linear", LINEAR, [
        (dict(x=None), INVALID), (dict(x_codes=A), INVALID), (dict(x_scale=A), INVALID), (dict(ws=None), INVALID),
        (dict(nbytes=16), INVALID), (dict(ws=A + 8), MISALIGNED), (dict(xt=C4), UNSUPPORTED), (dict(K=250), UNSUPPORTED),
        (dict(x_codes=A + 1, x_scale=A), MISALIGNED), (dict(y=None), INVALID), (dict(T=-5), INVALID)]),
    ("rtq_fp8_linear_dgrad", LDGRAD, [
        (dict(dy=None), INVALID), (dict(gt=F32), UNSUPPORTED), (dict(ws=None), INVALID), (dict(nbytes=16), INVALID),
        (dict(N=33), UNSUPPORTED), (dict(dyt=I32), UNSUPPORTED)]),
    ("rtq_fp8_wgrad", WGRAD, [
        (dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(dw=None), INVALID), (dict(N=36), UNSUPPORTED),
        (dict(K=24), UNSUPPORTED), (dict(dwt=C4), UNSUPPORTED), (dict(accumulate=2), INVALID), (dict(st=C4), UNSUPPORTED),
        (dict(ws=A + 8, nbytes=64), MISALIGNED), (dict(T=-1), INVALID)]),
    ("rtq_act_fp8_forward", ACT, [
        (dict(h=None), INVALID), (dict(act=0), INVALID), (dict(act=4), INVALID), (dict(y=None), INVALID),
        (dict(y_codes=A, y_scale=A), INVALID), (dict(y=None, y_codes=A), INVALID), (dict(ht=C4), UNSUPPORTED),
        (dict(d=8), UNSUPPORTED), (dict(y=None, y_codes=A + 8, y_scale=A), MISALIGNED)]),
    ("rtq_act_fp8_backward", ACTB, [
        (dict(dy=None), INVALID), (dict(dh=None), INVALID), (dict(act=9), INVALID), (dict(dyt=I32), UNSUPPORTED),
        (dict(st=BF16), UNSUPPORTED), (dict(h_codes=None), INVALID), (dict(d=20), UNSUPPORTED)]),
]


@pytest.mark.parametrize("name,good,change,want", [(n, g, c, w) for n, g, cs in REFUSALS for c, w in cs],
                         ids=lambda v: str(v) if not isinstance(v, dict) or len(v) < 4 else "")
def test_refused_before_anything_is_enqueued(name, good, change, want):
    assert call(name, good, **change) == want
    assert rtq.last_error() != ""


@pytest.mark.parametrize("name,good,change", [
    ("rtq_fp8_quantize", QUANT, dict(rows=0, x=None, codes=None, scale=None)),
    ("rtq_fp8_dequantize", DEQUANT, dict(rows=0, codes=None, scale=None, y=None)),
    ("rtq_fp8_qgemm", GEMM, dict(T=0, a=None, a_scale=None, y=None)),
    ("rtq_fp8_dgrad", DGRAD, dict(T=0, g=None, g_scale=None, dx=None)),
    ("rtq_fp8_linear", LINEAR, dict(T=0, x=None, y=None, ws=None, nbytes=0)),
    ("rtq_fp8_linear_dgrad", LDGRAD, dict(T=0, dy=None, dx=None, ws=None, nbytes=0)),
    ("rtq_fp8_wgrad", WGRAD, dict(T=0, dy=None, x=None, x_scale=None, accumulate=1)),
    ("rtq_act_fp8_forward", ACT, dict(rows=0, h=None, h_codes=None, h_scale=None, y=None)),
    ("rtq_act_fp8_backward", ACTB, dict(rows=0, dy=None, h_codes=None, h_scale=None, dh=None))])
def test_no_rows_is_a_no_op(name, good, change):
    assert call(name, good, **change) == OK


def test_workspace_sizes():
    for T, N, K in ((1, 100, 256), (37, 4096, 16384), (4608, 16384, 4096)):
        need = T * K + 4 * T * rtq.fp8_groups(K)
        assert rtq.fp8_linear_workspace(T, N, K) >= need + rtq.fp8_qgemm_workspace(T, N, K)
        assert rtq.fp8_linear_dgrad_workspace(T, N, K) >= T * N + 4 * T * rtq.fp8_groups(N) + rtq.fp8_dgrad_workspace(T, N, K)
    lib = rtq.load_library()
    assert lib.rtq_fp8_qgemm_workspace(-1, 64, 64) == 0 and lib.rtq_fp8_linear_workspace(4, 0, 64) == 0
    assert lib.rtq_fp8_wgrad_workspace(4, 64, -64) == 0


def test_binding_refuses_what_the_kernels_do_not_take():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    codes, scale = torch.zeros(4, 256, dtype=E4M3), torch.zeros(2, 4)
    with pytest.raises(ValueError, match="GPU tensor"):
        rtq.fp8_quantize(x, codes, scale)
    with pytest.raises(TypeError, match="dtype"):
        rtq.fp8_quantize(x.half(), codes, scale)
    with pytest.raises(ValueError, match="contiguous"):
        rtq.fp8_quantize(torch.zeros(256, 4, dtype=torch.bfloat16).t(), codes, scale)
    with pytest.raises(ValueError, match="shape"):
        rtq.fp8_quantize(x[0], codes, scale)


def test_plain_rounding_and_scales():
    for fmt in (E4M3, E5M2):
        values = torch.arange(256, dtype=torch.uint8).view(fmt).double()
        values = values[torch.isfinite(values)]
        assert torch.equal(round_to(values, fmt), values)
        mid = (values.unique()[1:] + values.unique()[:-1]) / 2
        assert torch.equal(round_to(mid, fmt), mid.to(torch.float32).to(fmt).double())     # ties to even
    for fmt in (E4M3, E5M2):
        for m in (1e-45, 1e-38, 0.3, 1.0, 447.0, 448.0, 449.0, 896.0, 3e38, 57344.0, 57345.0):
            s = scale_of(m, fmt)
            assert m <= TOP[fmt] * s and (s == 2.0 ** -120 or m > TOP[fmt] * s / 2)
    q, s = quantise(torch.tensor([[0.0] * 128 + [1.0, float("nan"), float("inf")] + [0.0] * 13]), E4M3)
    assert s[0, 0] == 1.0 and s[1, 0] == 2.0 ** -8 and q[0, 128] == 256.0
    assert torch.isnan(q[0, 129]) and torch.isnan(q[0, 130])
