"""The longest sides of the block-128 FP8 operators (2^30 rows or columns): more
workgroups than one launch holds."""
import numpy as np
import pytest
import torch

import fp8_ref as R
from gpu_common import need_gpu, say, to_device_bf16
from test_gpu_fp8 import normal

pytestmark = pytest.mark.gpu

SIDE = 1 << 30


def need_memory(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of device memory")


def marked(n):
    """n bf16 values, zeros but for runs of 300 at places all over, the end among them; and where those are."""
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    at = [0, (1 << 26) - 100, (1 << 27) - 100, (1 << 28) - 100, (1 << 28) + 1000, (1 << 29) - 100, n - 300]
    at = [a for a in at if a + 300 <= n]
    for i, a in enumerate(at):
        t[a:a + 300] = to_device_bf16(normal((1, 300), 1.0, 300 + i)).view(-1)
    return t, at


def values(q, rows, cols):
    """Values of q[rows, cols] (slices; cols from a multiple of 128)."""
    k = cols.stop - cols.start
    codes = q.codes[rows, cols.start:cols.start + R.up(k, 128)].cpu().numpy()
    scales = q.scales[cols.start // 128:R.up(cols.stop, 128) // 128, rows].cpu().numpy()
    return R.values(codes, scales, rows.stop - rows.start, k)


def test_quantize_many_rows():
    """[2^28 + 300, 1] along the rows: each row a block of its own."""
    mx = need_gpu()
    need_memory(45)
    n = (1 << 28) + 1300
    say("fp8 max size: rows", n)
    x, at = marked(n)
    q = mx.mxfp4_fp8_quantize(x.view(n, 1))
    for a in at:
        want = R.quantize(x[a:a + 300].double().cpu().numpy()[:, None])[0]
        assert np.array_equal(values(q, slice(a, a + 300), slice(0, 1)), want), a
    live = torch.zeros(n, dtype=torch.bool, device="cuda")
    for a in at:
        live[a:a + 300] = True
    assert not q.codes[:, 0][~live].any() and not q.scales[0, :n][~live].any()


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_longest_contraction_transposed(block_rows):
    """[2^30, 2] along the columns (its transpose): 2^23 tiles."""
    mx = need_gpu()
    need_memory(12)
    say("fp8 max size: transposed", SIDE, block_rows)
    x, at = marked(SIDE)
    both = torch.stack([x, -x], 1)
    q = mx.mxfp4_fp8_quantize(both, axis=0, block_rows=block_rows)
    for a in at:
        lo, hi = a // 128 * 128, min(R.up(a + 300, 128), SIDE)
        want = R.quantize(both[lo:hi].double().cpu().numpy().T)[0]
        assert np.array_equal(values(q, slice(0, 2), slice(lo, hi)), want), a
    assert int(q.codes.count_nonzero()) <= 2 * 300 * len(at) + int(torch.signbit(both).sum())


def test_quantize_longest_rows_in_blocks():
    """[2, 2^30] with a scale per 128 x 128 block: 2^23 tiles."""
    mx = need_gpu()
    need_memory(12)
    say("fp8 max size: blocks", SIDE)
    x, at = marked(SIDE)
    both = torch.stack([x, -x], 0)
    q = mx.mxfp4_fp8_quantize(both, block_rows=128)
    for a in at:
        lo, hi = a // 128 * 128, min(R.up(a + 300, 128), SIDE)
        want = R.quantize(both[:, lo:hi].double().cpu().numpy())[0]
        assert np.array_equal(values(q, slice(0, 2), slice(lo, hi)), want), a


def test_quantize_many_columns_transposed():
    """[3, 2^29 + 300] along the columns: 2^29 rows of the transpose."""
    mx = need_gpu()
    need_memory(90)
    n = (1 << 29) + 300
    say("fp8 max size: many columns", n)
    x, at = marked(n)
    q = mx.mxfp4_fp8_quantize(torch.stack([x, -x, x], 0), axis=0)
    for a in at:
        v = x[a:a + 300].double().cpu().numpy()
        want = R.quantize(np.stack([v, -v, v], 1))[0]
        assert np.array_equal(values(q, slice(a, a + 300), slice(0, 3)), want), a
    del q
    torch.cuda.empty_cache()


def ones_at(mx, rows, at, pair=None):
    """FP8 [rows, 128], scales of 1: zeros, but 1 in the first column of the rows given."""
    codes = torch.zeros((rows, 128), dtype=torch.uint8, device="cuda")
    codes[torch.tensor(at, device="cuda"), 0] = 0x38
    return mx.Fp8Tensor(rows, 128, codes, torch.full((1, R.up(rows, 16)), 127, dtype=torch.uint8, device="cuda"), pair)


def test_gemm_single_row_against_many():
    """[1, 128] x [2^29 + 40, 128]: one output row of more columns than a launch of 32 each holds."""
    mx = need_gpu()
    need_memory(80)
    n = (1 << 29) + 40
    say("fp8 max size: product", n)
    at = [0, 31, (1 << 28) + 5, (1 << 29) - 1, 1 << 29, n - 1]
    b, a = ones_at(mx, n, at), ones_at(mx, 1, [0])
    c = mx.mxfp4_fp8_gemm(a, b)
    assert torch.equal(c[0].nonzero().view(-1).cpu(), torch.tensor(at)) and (c[0, at] == 1).all()
    del b, c
    torch.cuda.empty_cache()


def test_gated_single_row_against_many():
    """One token against 2^28 + 128 gate rows and as many of the up projection."""
    mx = need_gpu()
    need_memory(80)
    n = (1 << 28) + 128
    say("fp8 max size: gated", n)
    at = [0, 17, (1 << 27) + 3, (1 << 28) - 1, 1 << 28, n - 1]
    w, x = ones_at(mx, 2 * n, at + [n + i for i in at], pair=n), ones_at(mx, 1, [0])
    h = mx.mxfp4_fp8_gated(x, w, dtype=torch.bfloat16)
    assert torch.equal(h[0].nonzero().view(-1).cpu(), torch.tensor(at))
    assert (h[0, at].double() - 1 / (1 + np.exp(-1.0))).abs().max().item() < 2.0 ** -9
    q = mx.mxfp4_fp8_gated(x, w)
    assert torch.equal(q.codes[0].nonzero().view(-1).cpu(), torch.tensor(at))
    del w, q, h
    torch.cuda.empty_cache()
