"""CPU tests of the calls around the 8-bit layers of an MLP block: argument checks of the C ABI (run before any HIP call)
and of the Python binding, workspace sizes, and the plain forms the GPU tests compare with."""
import ctypes

import pytest
import torch

import _block
import rotation_then_quantize_amd as rtq
from _fp8 import E4M3, E5M2, E8M0, quantise, scale_of

A = 0x10000      # a fake, 16-byte aligned "device" address: never dereferenced by the host checks
OK, INVALID, UNSUPPORTED, MISALIGNED = rtq.RTQ_OK, rtq.RTQ_ERR_INVALID_ARG, rtq.RTQ_ERR_UNSUPPORTED, rtq.RTQ_ERR_MISALIGNED
F32, BF16, I32 = rtq.RTQ_F32, rtq.RTQ_BF16, rtq.RTQ_I32
C4, C5, S8 = rtq.RTQ_E4M3, rtq.RTQ_E5M2, rtq.RTQ_E8M0
BIG = 1 << 40
NAN, INF = float("nan"), float("inf")


def call(name, good, **change):
    args = dict(good)
    assert set(change) <= set(args)
    args.update(change)
    return getattr(rtq.load_library(), name)(*args.values())


NORM = dict(x=A, xt=BF16, r=A, rt=F32, rows=4, d=256, gamma=A, gt=BF16, eps=1e-6, h=A + 4096, y=None, codes=A, scale=A, st=F32,
            stream=None)
BACK = dict(dn=A, dnt=BF16, h=A, ht=F32, dr=A, rows=4, d=256, gamma=A, gt=BF16, eps=1e-6, dh=A + 4096, dgamma=A, dgt=F32,
            accumulate=0, ws=A, nbytes=BIG, stream=None)
GLU = dict(x=A, x_scale=A, T=4, w=A, w_scale=A, st=F32, N=256, K=272, act=3, h_codes=A, h_scale=A, y=None, yt=BF16, y_codes=A,
           y_scale=A, ws=A, nbytes=BIG, stream=None)
GLUB = dict(dy=A, dyt=BF16, h_codes=A, h_scale=A, st=S8, T=4, N=256, act=3, dh=A, dh_codes=A, gt=C5, dh_scale=A, stream=None)

REFUSALS = [
    ("rtq_rmsnorm_forward", NORM, [
        (dict(x=None), INVALID), (dict(x=A + 8), MISALIGNED), (dict(xt=C4), UNSUPPORTED), (dict(rt=I32), UNSUPPORTED),
        (dict(gt=C5), UNSUPPORTED), (dict(st=BF16), UNSUPPORTED), (dict(r=None), INVALID), (dict(h=None), INVALID),
        (dict(r=A + 4), MISALIGNED), (dict(h=A + 8), MISALIGNED), (dict(gamma=None), INVALID), (dict(gamma=A + 2), MISALIGNED),
        (dict(codes=None), INVALID), (dict(scale=None), INVALID), (dict(codes=None, scale=None), INVALID),
        (dict(codes=A + 8), MISALIGNED), (dict(scale=A + 4), MISALIGNED), (dict(y=A + 8), MISALIGNED), (dict(rows=-1), INVALID),
        (dict(rows=1 << 31), UNSUPPORTED), (dict(d=0), INVALID), (dict(d=40), UNSUPPORTED), (dict(d=(1 << 20) + 16), UNSUPPORTED),
        (dict(eps=0.0), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID),
        (dict(y=A + 4096), INVALID), (dict(h=A), INVALID)]),
    ("rtq_rmsnorm_backward", BACK, [
        (dict(dn=None), INVALID), (dict(h=None), INVALID), (dict(dh=None), INVALID), (dict(gamma=None), INVALID),
        (dict(dn=A + 8), MISALIGNED), (dict(dr=A + 8), MISALIGNED), (dict(dgamma=A + 8), MISALIGNED), (dict(dh=A + 8), MISALIGNED),
        (dict(dh=A), INVALID), (dict(dnt=C4), UNSUPPORTED), (dict(ht=I32), UNSUPPORTED), (dict(gt=S8), UNSUPPORTED),
        (dict(dgt=C4), UNSUPPORTED), (dict(accumulate=2), INVALID), (dict(ws=None), INVALID), (dict(nbytes=16), INVALID),
        (dict(ws=A + 4), MISALIGNED), (dict(d=24), UNSUPPORTED), (dict(rows=-2), INVALID), (dict(eps=0.0), INVALID),
        (dict(dn=A + 4096), INVALID)]),
    ("rtq_fp8_glu", GLU, [
        (dict(x=None), INVALID), (dict(x_scale=None), INVALID), (dict(w=None), INVALID), (dict(w_scale=None), INVALID),
        (dict(w=A + 8), MISALIGNED), (dict(st=BF16), UNSUPPORTED), (dict(N=0), INVALID), (dict(N=192), UNSUPPORTED),
        (dict(N=(1 << 19) + 128), UNSUPPORTED), (dict(K=24), UNSUPPORTED), (dict(K=0), INVALID), (dict(act=0), INVALID),
        (dict(act=4), INVALID), (dict(h_codes=None), INVALID), (dict(h_scale=None), INVALID), (dict(y=A), INVALID),
        (dict(y_codes=None), INVALID), (dict(y_codes=None, y_scale=None), INVALID), (dict(y_codes=A + 8), MISALIGNED),
        (dict(h_scale=A + 4), MISALIGNED), (dict(y=A + 4, y_codes=None, y_scale=None), MISALIGNED), (dict(yt=I32), UNSUPPORTED),
        (dict(ws=A + 4), MISALIGNED), (dict(T=-1), INVALID), (dict(T=1 << 31), UNSUPPORTED),
        (dict(T=(1 << 31) - 1, N=1 << 19), UNSUPPORTED)]),
    ("rtq_glu_fp8_backward", GLUB, [
        (dict(dy=None), INVALID), (dict(h_codes=None), INVALID), (dict(h_scale=None), INVALID), (dict(dyt=C4), UNSUPPORTED),
        (dict(gt=F32), UNSUPPORTED), (dict(st=C4), UNSUPPORTED), (dict(N=64), UNSUPPORTED), (dict(act=7), INVALID),
        (dict(dh_codes=None), INVALID), (dict(dh_scale=None), INVALID), (dict(dh=None, dh_codes=None, dh_scale=None), INVALID),
        (dict(dh=A + 8), MISALIGNED), (dict(dh_codes=A + 8), MISALIGNED), (dict(T=-1), INVALID)]),
]


@pytest.mark.parametrize("name,good,change,want", [(n, g, c, w) for n, g, cs in REFUSALS for c, w in cs],
                         ids=lambda v: str(v) if not isinstance(v, dict) or len(v) < 4 else "")
def test_refused_before_anything_is_enqueued(name, good, change, want):
    assert call(name, good, **change) == want
    assert rtq.last_error() != ""


@pytest.mark.parametrize("name,good,change", [
    ("rtq_rmsnorm_forward", NORM, dict(rows=0, x=None, r=None, h=None, codes=None, scale=None)),
    ("rtq_rmsnorm_backward", BACK, dict(rows=0, dn=None, h=None, dh=None, dr=None, ws=None, nbytes=0, accumulate=1)),
    ("rtq_rmsnorm_backward", BACK, dict(rows=0, dn=None, h=None, dh=None, dr=None, dgamma=None, ws=None, nbytes=0)),
    ("rtq_fp8_glu", GLU, dict(T=0, x=None, x_scale=None, y_codes=None, y_scale=None, h_codes=None, h_scale=None, ws=None, nbytes=0)),
    ("rtq_glu_fp8_backward", GLUB, dict(T=0, dy=None, h_codes=None, h_scale=None, dh=None, dh_codes=None, dh_scale=None))])
def test_no_rows_is_a_no_op(name, good, change):
    assert call(name, good, **change) == OK


def tensors(*entries):
    c = (rtq._Tensor * max(1, len(entries)))()
    for i, e in enumerate(entries):
        c[i] = rtq._Tensor(*e)
    return c


GOOD = (A, 100, F32)


@pytest.mark.parametrize("entry,want", [((None, 5, F32), INVALID), ((A + 8, 5, F32), MISALIGNED), ((A, -1, F32), INVALID),
                                        ((A, (1 << 37) + 1, F32), UNSUPPORTED), ((A, 5, C4), UNSUPPORTED), ((A, 5, I32), UNSUPPORTED)])
def test_tensor_lists_refused(entry, want):
    lib = rtq.load_library()
    c = tensors(GOOD, entry)
    assert lib.rtq_grad_norm(c, 2, A, A, BIG, None) == want
    assert lib.rtq_grad_clip(c, None, 2, A, 1.0, None) == want
    assert lib.rtq_grad_norm_workspace(c, 2) == 0


def test_clip_arguments_refused():
    lib = rtq.load_library()
    c = tensors(GOOD, GOOD)
    outs = (ctypes.c_void_p * 2)(A, A + 8)
    assert lib.rtq_grad_clip(c, outs, 2, A, 1.0, None) == MISALIGNED
    outs = (ctypes.c_void_p * 2)(A, None)
    assert lib.rtq_grad_clip(c, outs, 2, A, 1.0, None) == INVALID
    assert lib.rtq_grad_clip(None, None, 2, A, 1.0, None) == INVALID
    assert lib.rtq_grad_clip(c, None, -1, A, 1.0, None) == INVALID
    assert lib.rtq_grad_clip(c, None, 2, None, 1.0, None) == INVALID
    for most in (-1.0, NAN, INF):
        assert lib.rtq_grad_clip(c, None, 2, A, most, None) == INVALID
    assert lib.rtq_grad_norm(c, 2, None, A, BIG, None) == INVALID
    assert lib.rtq_grad_norm(c, 2, A + 4, A, BIG, None) == MISALIGNED
    assert lib.rtq_grad_norm(c, 2, A, None, 0, None) == INVALID
    assert lib.rtq_grad_norm(c, 2, A, A, 8, None) == INVALID
    assert lib.rtq_grad_norm(c, 2, A, A + 4, BIG, None) == MISALIGNED
    assert lib.rtq_grad_norm((rtq._Tensor * ((1 << 20) + 1))(), (1 << 20) + 1, A, A, BIG, None) == INVALID


def test_workspace_sizes():
    lib = rtq.load_library()
    assert rtq.rmsnorm_backward_workspace(0, 4096) == 0 and lib.rtq_rmsnorm_backward_workspace(-1, 4096) == 0
    assert rtq.rmsnorm_backward_workspace(1, 4096) >= 4096 * 4
    assert lib.rtq_fp8_glu_workspace(4, 100, 256) == 0 and lib.rtq_fp8_glu_workspace(-1, 128, 256) == 0
    assert lib.rtq_grad_norm_workspace(tensors(GOOD, (None, 0, F32)), 2) >= 8


def test_binding_refuses_what_the_kernels_do_not_take():
    bf = torch.bfloat16
    x, gamma = torch.zeros(4, 256, dtype=bf), torch.zeros(256)
    with pytest.raises(ValueError, match="GPU tensor"):
        rtq.rmsnorm_forward(x, gamma, 1e-6, y=torch.zeros_like(x))
    with pytest.raises(TypeError, match="dtype"):
        rtq.rmsnorm_forward(x.half(), gamma, 1e-6, y=torch.zeros_like(x))
    with pytest.raises(ValueError, match="GPU tensor"):
        rtq.rmsnorm_backward(x, x, gamma, 1e-6, torch.zeros_like(x))
    with pytest.raises(ValueError, match="GPU tensor|shape"):
        rtq.glu_fp8_backward(x, torch.zeros(4, 512, dtype=E4M3), torch.zeros(4, 4), rtq.RTQ_ACT_SILU, dh=torch.zeros(4, 512, dtype=bf))
    with pytest.raises(ValueError, match="no tensors"):
        rtq.TensorList([])
    with pytest.raises(ValueError, match="GPU tensor"):
        rtq.TensorList([x])
    with pytest.raises(ValueError, match="outs"):
        rtq.TensorList([x, x], [x])
    with pytest.raises(TypeError, match="tensors"):
        rtq.TensorList([x, None])
    with pytest.raises(ValueError, match="too large"):         # longer than the library's lengths
        rtq.rmsnorm_forward(torch.zeros(0, (1 << 32) + 256, dtype=bf), gamma, 1e-6, y=x)
    with pytest.raises(ValueError, match="too large"):
        rtq.glu_fp8_backward(torch.zeros(0, (1 << 32) + 128, dtype=bf), x, gamma, rtq.RTQ_ACT_SILU, dh=x)


@pytest.mark.parametrize("reads,writes,want", [
    ([], [(0, 8), (8, 16)], False), ([], [(0, 8), (7, 16)], True), ([], [(0, 8), (0, 8)], True), ([(0, 8)], [(8, 16)], False),
    ([(0, 9)], [(8, 16)], True), ([(4, 6)], [(0, 16)], True), ([(0, 8), (0, 8), (2, 20)], [(20, 24)], False),
    ([(0, 30), (2, 4)], [(20, 24)], True), ([(5, 5)], [(0, 8), (3, 3)], False), ([(0, 8)], [(0, 8)], True)])
def test_overlapping_ranges(reads, writes, want):
    assert rtq._overlap(reads, writes) is want


def test_plain_scales_and_gradients():
    for fmt in (E4M3, E5M2):
        m = torch.tensor([0.0, 1e-38, 0.3, 1.0, 447.0, 448.0, 449.0, 896.0, 57344.0, 57345.0, 3e38], dtype=torch.float64)
        assert torch.equal(_block.scales_of(m, fmt), torch.tensor([scale_of(float(v), fmt) for v in m], dtype=torch.float64))
    gen = torch.Generator().manual_seed(3)
    h = torch.randn(5, 48, generator=gen, dtype=torch.float64, requires_grad=True)
    gamma = torch.randn(48, generator=gen, dtype=torch.float64, requires_grad=True)
    dn = torch.randn(5, 48, generator=gen, dtype=torch.float64)
    want = torch.autograd.grad((_block.norm(h, gamma) * dn).sum(), (h, gamma))
    dh, dgamma, _, _ = _block.norm_gradients(dn, h.detach(), gamma.detach())
    assert torch.allclose(dh, want[0], rtol=1e-12, atol=1e-14) and torch.allclose(dgamma, want[1], rtol=1e-12, atol=1e-14)
    step = 1e-6 * torch.randn(5, 48, generator=gen, dtype=torch.float64)       # against differences
    with torch.no_grad():
        diff = ((_block.norm(h + step, gamma) - _block.norm(h - step, gamma)) * dn).sum() / 2
    assert abs(float(diff - (dh * step).sum())) <= 1e-6 * float((dh * step).abs().sum())
    for name in ("silu", "gelu", "gelu_tanh"):
        z = torch.randn(4, 32, generator=gen, dtype=torch.float64, requires_grad=True)
        dy = torch.randn(4, 16, generator=gen, dtype=torch.float64)
        (want,) = torch.autograd.grad(_block.glu(z, name), z, dy)
        assert torch.allclose(_block.glu_gradient(dy, z.detach(), name), want, rtol=1e-10, atol=1e-12)


def test_code_check_finds_a_wrong_code():
    x = torch.randn(3, 272, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    q, s = quantise(x, E4M3)
    off = torch.zeros_like(x)
    _block.check_codes(q.float().to(E4M3), s.to(E8M0).float(), x, off)
    bad = q.clone()
    bad[1, 200] = -bad[1, 200]
    with pytest.raises(AssertionError, match="codes"):
        _block.check_codes(bad, s, x, off)
    worse = s.clone()
    worse[2, 1] *= 2
    with pytest.raises(AssertionError, match="scales"):
        _block.check_codes(q, worse, x, off)
