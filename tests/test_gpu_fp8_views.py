"""Products and gated blocks of FP8 operands that are views: shards of a
matrix's rows, at offsets that are multiples of 16, the last of them ending where
its buffer ends.  A view's result has the bits that a copy of its own gives
(the bytes around it, NaN scales and NaN codes, reach nothing), and
the value of the 64-bit reference."""
import numpy as np
import pytest
import torch

import fp8_ref as R
import workloads
from gpu_common import need_gpu, say, to_device_bf16
from test_gpu_fp8 import assert_near, exact_product, normal

pytestmark = pytest.mark.gpu


def shard(mx, q, first, rows):
    """Rows first .. first + rows - 1 of q: a view, and a copy in memory of its own."""
    view = mx.Fp8Tensor(rows, q.k, q.codes[first:first + rows], q.scales[:, first:first + rows])
    scales = torch.zeros((q.scales.shape[0], R.up(rows, 16)), dtype=torch.uint8, device="cuda")
    scales[:, :rows] = view.scales
    return view, mx.Fp8Tensor(rows, q.k, view.codes.clone(), scales)


def surrounded(q, first, rows):
    """q with NaN scales and NaN codes in all rows but first .. first + rows - 1."""
    out = type(q)(q.rows, q.k, q.codes.clone(), q.scales.clone())
    for part in (slice(0, first), slice(first + rows, None)):
        out.codes[part] = 0x7F
        out.scales[:, part] = 0xFF
    return out


def matrix(mx, rows, k, seed, std=1.0):
    return mx.mxfp4_fp8_quantize(to_device_bf16(normal((rows, k), std, seed)))


# (rows of the whole matrix, first row, rows of the shard): the last of each kind ends with its buffer
SHARDS = [(160, 16, 16), (160, 144, 16), (400, 128, 33), (400, 384, 16), (1008, 128, 384), (1008, 384, 400), (1008, 624, 384),
          (1008, 880, 128), (816, 240, 573)]


@pytest.mark.parametrize("K", [128, 300, 2500])
@pytest.mark.parametrize("whole,first,rows", SHARDS)
def test_gemm_of_row_shards(whole, first, rows, K):
    mx = need_gpu()
    say("fp8 gemm of shards", whole, first, rows, K)
    q = surrounded(matrix(mx, whole, K, 201), first, rows)
    view, copy = shard(mx, q, first, rows)
    for other in (7, 90, 300):
        o = matrix(mx, other, K, 202, 0.02)
        for a, b, c in ((view, o, copy), (o, view, None)):   # as activations, as weights
            got = mx.mxfp4_fp8_gemm(a, b, dtype=torch.float32)
            assert torch.equal(got, mx.mxfp4_fp8_gemm(c or o, o if c else copy, dtype=torch.float32))
            if K != 300:   # (the reference takes long)
                continue
            C, B = exact_product(copy if c else o, o if c else copy)
            assert_near(got.cpu().numpy(), C, B, f"{whole} {first} {rows} {K} {other}")


@pytest.mark.parametrize("n,k", [(100, 256), (128, 1000), (300, 2300)])
def test_gemm_of_a_pairs_halves(n, k):
    """Either weight of a pair on its own; the second one's lines end where the pair's buffer ends."""
    mx = need_gpu()
    say("fp8 gemm of a pair's halves", n, k)
    g, u = (to_device_bf16(normal((n, k), 0.05, 211 + i)) for i in (0, 1))
    q, np_ = mx.mxfp4_fp8_quantize_pair(g, u), R.up(n, 128)
    for T in (5, 70, 300):
        x = matrix(mx, T, k, 213)
        for i, w in enumerate((g, u)):
            half = mx.Fp8Tensor(n, k, q.codes[i * np_:i * np_ + n], q.scales[:, i * np_:i * np_ + n])
            want = mx.mxfp4_fp8_gemm(x, mx.mxfp4_fp8_quantize(w, block_rows=128))
            assert torch.equal(mx.mxfp4_fp8_gemm(x, half), want)


@pytest.mark.parametrize("whole,first,rows", SHARDS)
def test_gated_of_row_shards(whole, first, rows):
    """The gated block of a shard of its tokens, forward; and backward with the weights' gradient of a shard of x's columns."""
    mx = need_gpu()
    K, n = 300, 200
    say("fp8 gated of shards", whole, first, rows)
    x = workloads.small_t_bf16((whole, K), 4.0, 221)
    q = surrounded(mx.mxfp4_fp8_quantize(to_device_bf16(x)), first, rows)
    view, copy = shard(mx, q, first, rows)
    g, u = (to_device_bf16(normal((n, K), 0.05, 222 + i)) for i in (0, 1))
    w = mx.mxfp4_fp8_quantize_pair(g, u)
    got, want = mx.mxfp4_fp8_gated(view, w, train=True), mx.mxfp4_fp8_gated(copy, w, train=True)
    assert torch.equal(got[0].codes, want[0].codes) and torch.equal(got[0].scales[:, :rows], want[0].scales[:, :rows])
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    # x along the tokens [whole, T]: a shard of it is a shard of x's columns
    T = 90
    dh, gg, uu = (to_device_bf16(normal((T, n), 1.0, 224 + i)) for i in range(3))
    xt = surrounded(matrix(mx, whole, T, 227), first, rows)
    gt, ut = (to_device_bf16(normal((n, rows), 0.05, 228 + i)) for i in (0, 1))
    wt = mx.mxfp4_fp8_quantize_pair(gt, ut, axis=0)
    xv, xc = shard(mx, xt, first, rows)
    a, b = (mx.mxfp4_fp8_gated_backward(dh, gg, uu, wt, t) for t in (xv, xc))
    assert all(torch.equal(s, t) for s, t in zip(a, b)) and torch.isfinite(a[1]).all()


def test_one_line_of_scales():
    """A single 128-block: its line of scales may be a slice of a longer one, whose pitch is then not a pitch."""
    mx = need_gpu()
    q, w = matrix(mx, 304, 128, 231), matrix(mx, 50, 128, 232)
    for first, rows in ((16, 3), (288, 16), (160, 144), (0, 304)):
        view, copy = shard(mx, q, first, rows)
        assert torch.equal(mx.mxfp4_fp8_gemm(view, w), mx.mxfp4_fp8_gemm(copy, w))
        assert torch.equal(mx.mxfp4_fp8_gemm(w, view), mx.mxfp4_fp8_gemm(w, copy))
    assert not np.isnan(mx.mxfp4_fp8_gemm(q, w).float().cpu().numpy()).any()
