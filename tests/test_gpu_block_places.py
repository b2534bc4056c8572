"""GPU tests of the norm's outputs on its inputs' places: the same bits as apart from them."""
import pytest
import torch

import rotation_then_quantize_amd as rtq

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("T,d", [(1, 4096), (70, 1040), (300, 4112), (5, 16400)])
@pytest.mark.parametrize("xt,rt", [(F32, F32), (BF16, BF16), (BF16, F32)])
def test_norm_in_place(T, d, xt, rt):
    print("norm in place", T, d, xt, rt, flush=True)
    g = torch.Generator(device="cuda").manual_seed(T + d)
    x, r = (torch.randn(T, d, generator=g, device="cuda").to(t) for t in (xt, rt))
    gamma = torch.rand(d, generator=g, device="cuda") + 0.5
    h, y = torch.empty_like(r), torch.empty_like(x)
    rtq.rmsnorm_forward(x, gamma, 1e-6, residual=r, h=h, y=y)
    for h_on, y_on in (("r", None), ("r", "x"), (None, "x"), ("x", None), ("x", "r"), (None, "r")):
        if xt != rt and (h_on == "x" or y_on == "r"):
            with pytest.raises(rtq.RtqError, match="h must not be|y overlaps residual"):
                own = torch.empty(T, d, dtype=F32, device="cuda")
                over = own.view(BF16).view(-1)[:T * d].view(T, d)      # the first half of an fp32 array, as bf16
                if h_on == "x":
                    rtq.rmsnorm_forward(over, gamma, 1e-6, residual=r, h=own, y=torch.empty_like(x))
                else:
                    rtq.rmsnorm_forward(x, gamma, 1e-6, residual=own, h=torch.empty_like(r), y=over)
            continue
        own = {"x": x.clone(), "r": r.clone()}
        h2 = own[h_on] if h_on else torch.empty_like(r)
        y2 = own[y_on] if y_on else torch.empty_like(x)
        rtq.rmsnorm_forward(own["x"], gamma, 1e-6, residual=own["r"], h=h2, y=y2)
        assert torch.equal(h2, h) and torch.equal(y2, y), (h_on, y_on)


def test_workspaces_that_nothing_uses():
    """A workspace is not looked at where the call needs none."""
    print("unused workspace", flush=True)
    h, gamma = torch.randn(4, 256, device="cuda"), torch.ones(256, device="cuda")
    dh, again = torch.empty_like(h), torch.empty_like(h)
    rtq.rmsnorm_backward(h, h, gamma, 1e-6, dh)
    rtq.rmsnorm_backward(h, h, gamma, 1e-6, again, workspace=dh[1:])
    assert torch.equal(again, dh)
