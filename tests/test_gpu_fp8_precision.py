"""How exact the FP8 products are: the matrix instruction cuts products toward
zero, so what a sum loses adds up where the products have one sign."""
import numpy as np
import pytest
import torch

from gpu_common import need_gpu, say, to_device_bf16
from test_gpu_fp8 import BF16, assert_near, exact_product, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("M,N,K", [(16, 48, 16384), (300, 48, 16384), (16, 40, 2048), (40, 33, 65536)])
def test_products_of_one_sign(M, N, K, sign):
    """Long sums of products that all have one sign, in every kernel's form: within the bound of the cut
    (7 * 2^-13 of each eight's largest power of two, and binary32's rounding), and short of the exact sum on average."""
    mx = need_gpu()
    say("fp8 products of one sign", M, N, K, sign)
    a, b = (normal(s, 1.0, 501 + i) & 0x7FFF for i, s in enumerate([(M, K), (N, K)]))   # magnitudes
    if sign < 0:
        b = b | 0x8000
    qa, qb = mx.mxfp4_fp8_quantize(to_device_bf16(a)), mx.mxfp4_fp8_quantize(to_device_bf16(b))
    C, B = exact_product(qa, qb)
    assert (sign * C > 0).all()
    c = mx.mxfp4_fp8_gemm(qa, qb, dtype=torch.float32).cpu().numpy()
    assert_near(c, C, B, "one sign")
    assert 0 < np.mean(1 - c / C) < np.mean(B / np.abs(C))
    assert_near(mx.mxfp4_fp8_gemm(qa, qb).float().cpu().numpy(), C, B * (1 + BF16) + BF16 * np.abs(C), "one sign, bf16")
