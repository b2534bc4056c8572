"""CPU tests: the calls around the 8-bit layers of an MLP block refuse outputs that lie over other arrays, where one workgroup
would write over what another has yet to read.  (What may lie on each other, the GPU tests run.)"""
import pytest

import rotation_then_quantize_amd as rtq

F32, BF16, C5, S8 = rtq.RTQ_F32, rtq.RTQ_BF16, rtq.RTQ_E5M2, rtq.RTQ_E8M0


def at(i):
    """Fake, far apart "device" addresses: never dereferenced by the host checks."""
    return (i + 1) << 24


# 4 rows of 256 (and of 2 x 256 channels)
NORM = dict(x=at(0), xt=BF16, r=at(1), rt=F32, rows=4, d=256, gamma=at(2), gt=BF16, eps=1e-6, h=at(3), y=at(4), codes=at(5), scale=at(6),
            st=F32, stream=None)
BACK = dict(dn=at(0), dnt=BF16, h=at(1), ht=F32, dr=at(2), rows=4, d=256, gamma=at(3), gt=BF16, eps=1e-6, dh=at(4), dgamma=at(5), dgt=F32,
            accumulate=0, ws=at(6), nbytes=1 << 20, stream=None)
GLU = dict(x=at(0), x_scale=at(1), T=4, w=at(2), w_scale=at(3), st=F32, N=256, K=256, act=3, h_codes=at(4), h_scale=at(5), y=None, yt=BF16,
           y_codes=at(6), y_scale=at(7), ws=at(8), nbytes=1 << 20, stream=None)
GLUY = dict(GLU, y=at(6), y_codes=None, y_scale=None)
GLUB = dict(dy=at(0), dyt=BF16, h_codes=at(1), h_scale=at(2), st=S8, T=4, N=256, act=3, dh=at(3), dh_codes=at(4), gt=C5, dh_scale=at(5),
            stream=None)

CASES = [("rtq_rmsnorm_forward", NORM, c) for c in [
    dict(y=at(1)),                                              # residual of another type
    dict(h=at(3), y=at(3) + 16), dict(h=at(3), y=at(3) + 4 * 256 * 4 - 16), dict(y=at(0) + 16), dict(h=at(1) - 16), dict(y=at(2)),
    dict(rt=BF16, h=at(0) + 512), dict(codes=at(0)), dict(codes=at(1) + 2048), dict(codes=at(3)), dict(codes=at(4)), dict(codes=at(2)),
    dict(scale=at(0)), dict(scale=at(5) + 1008), dict(scale=at(4) + 2032), dict(h=at(2) - 4096 + 16)]]
CASES += [("rtq_rmsnorm_backward", BACK, c) for c in [
    dict(dh=at(2) + 16), dict(dh=at(1) + 4080), dict(dh=at(0) - 4080), dict(dh=at(3)), dict(dgamma=at(0)), dict(dgamma=at(1)), dict(dgamma=at(3)),
    dict(dgamma=at(4)), dict(ws=at(0)), dict(ws=at(4) + 4080), dict(ws=at(5)), dict(dnt=F32, dh=at(0) + 16)]]
CASES += [("rtq_fp8_glu", GLU, c) for c in [
    dict(y_codes=at(0)), dict(h_codes=at(0)), dict(h_codes=at(2) + 131056), dict(y_codes=at(4) + 2032), dict(h_scale=at(1)),
    dict(y_scale=at(3) + 16), dict(y_scale=at(5) + 48), dict(ws=at(4)), dict(ws=at(0) - 32), dict(h_scale=at(7))]]
CASES += [("rtq_fp8_glu", GLUY, c) for c in [dict(y=at(0)), dict(y=at(2)), dict(y=at(4) + 1024), dict(ws=at(6) + 2032)]]
CASES += [("rtq_glu_fp8_backward", GLUB, c) for c in [
    dict(dh=at(0)), dict(dh=at(1)), dict(dh_codes=at(0)), dict(dh_codes=at(1)), dict(dh_codes=at(3) + 4080), dict(dh_scale=at(2)),
    dict(dh_scale=at(4) + 2032), dict(dh=at(2) - 16)]]


@pytest.mark.parametrize("name,good,change", CASES, ids=lambda v: str(v) if not isinstance(v, dict) or len(v) < 4 else "")
def test_overlapping_outputs_are_refused(name, good, change):
    assert set(change) <= set(good)
    assert getattr(rtq.load_library(), name)(*dict(good, **change).values()) == rtq.RTQ_ERR_INVALID_ARG
    assert "overlaps" in rtq.last_error()
