"""Arguments of the FP8 binding that are right in an unusual form."""
import pytest
import torch

from gpu_common import need_gpu, say
from test_gpu_fp8 import backward_case, to_device_bf16

pytestmark = pytest.mark.gpu


def test_gated_backward_of_a_single_row_has_no_strides():
    """One token: g and u as slices of matrices of different widths, whose row strides say nothing."""
    mx = need_gpu()
    H, n = 200, 130
    dh, g, u, wt, xt, *_ = backward_case(mx, 1, H, n, "silu", 301)
    say("fp8 gated backward, one row")
    want = mx.mxfp4_fp8_gated_backward(to_device_bf16(dh), to_device_bf16(g), to_device_bf16(u), wt, xt, want_ht=True)
    for pads in ((0, 7), (9, 0), (3, 40)):
        got = mx.mxfp4_fp8_gated_backward(to_device_bf16(dh, 5), to_device_bf16(g, pads[0]), to_device_bf16(u, pads[1]),
                                          wt, xt, want_ht=True)
        assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
        assert torch.equal(got[3].codes, want[3].codes) and torch.equal(got[3].exponents().view(torch.uint8),
                                                                        want[3].exponents().view(torch.uint8))


def test_gated_backward_of_rows_wants_one_stride():
    mx = need_gpu()
    dh, g, u, wt, xt, *_ = backward_case(mx, 2, 200, 130, "silu", 302)
    with pytest.raises(ValueError, match="row stride"):
        mx.mxfp4_fp8_gated_backward(to_device_bf16(dh), to_device_bf16(g), to_device_bf16(u, 3), wt, xt)


def test_gated_backward_rows_that_pad_the_weights():
    """Rows n .. np - 1 of either half of dw: zeros, and NaN only in the columns of x that hold one."""
    mx = need_gpu()
    T, H, n = 300, 200, 130
    dh, g, u, wt, xt, *_ = backward_case(mx, T, H, n, "gelu", 303)
    args = [to_device_bf16(t) for t in (dh, g, u)]
    say("fp8 gated backward, padding rows")
    for bad in (None, 7):
        if bad is not None:
            xt.scales[1, bad] = 255
        dwg = mx.mxfp4_fp8_gated_backward(*args, wt, xt, act="gelu")[1]
        dw = torch.as_strided(dwg, (512, H), (H, 1), 0)   # (both halves, 256 rows each)
        for half in (dw[:256], dw[256:]):
            keep = torch.ones(H, dtype=torch.bool, device="cuda")
            if bad is not None:
                keep[bad] = False
            assert not half[n:, keep].any() and bool(torch.isfinite(half[:, keep]).all())
            assert bool(torch.isnan(half[:, ~keep]).all())
