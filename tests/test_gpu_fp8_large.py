"""The forms of the FP8 kernels that only large operands reach: whole tiles,
tiles cut into halves and last rows of tiles together in one launch, and norms
whose workgroups take several rows.

Products: elements are small whole numbers and scales powers of two next to 1, so
every product and every sum of them is exact in binary32 and in the matrix
instruction (|product| <= 2^4 in steps of 1 within a block, well inside its 13 places), in any
order: results equal a binary64 product bit by bit.
Norms: binary64 on the device, with the bounds of test_gpu_fp8.py.
"""
import pytest
import torch

import fp8_ref as R
from gpu_common import need_gpu, say

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def whole_numbers(mx, rows, k, seed, exponents, pair=None):
    """(an Fp8Tensor of elements -4 .. 4 and scales 2^e, e of `exponents`; its values in binary64)"""
    g = gen(seed)
    kp, blocks = R.up(k, 128), R.up(k, 128) // 128
    v = torch.randint(-4, 5, (rows, kp), generator=g, device="cuda").float()
    v[:, k:] = 0
    e = torch.randint(exponents[0], exponents[1] + 1, (blocks, R.up(rows, 16)), generator=g, device="cuda")
    q = mx.Fp8Tensor(rows, k, v.to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8), pair)
    return q, (v.view(rows, blocks, 128) * torch.exp2(e[:, :rows].t().float())[..., None]).view(rows, kp)[:, :k].double()


# (rows, columns, contraction): what one launch holds.  256 compute units; tiles of 256 x 256
PRODUCTS = [
    (4200, 4300, 300),    # 272 tiles: 256 whole, 16 in two halves each, and a last row of 17 halves
    (2900, 6200, 200),    # 275: 256 whole, 19 in halves, 25 in a last row
    (5000, 5100, 130),    # 400 whole tiles, none cut: the halves would not make one round
    (3000, 3000, 260),    # 144 whole tiles
    (4096, 4352, 128),    # 272: no ragged side, one block
    (700, 17000, 1900),   # 201: fewer than compute units, the last row of tiles part filled
    (600, 1100, 4200),    # 10 whole tiles and a last row of 5 halves, their contraction split
]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_products_of_many_tiles(M, N, K):
    mx = need_gpu()
    say("fp8 many tiles", M, N, K)
    (a, av), (b, bv) = whole_numbers(mx, M, K, 401, (-1, 1)), whole_numbers(mx, N, K, 402, (-1, 1))
    want = torch.mm(av, bv.t().contiguous())
    assert want.abs().max().item() * 4 < 2 ** 24   # (sums are whole multiples of a quarter)
    big = torch.full((M + 1, N + 5), 7.0, dtype=torch.float32, device="cuda")
    mx.mxfp4_fp8_gemm(a, b, out=big[:M, :N])
    assert torch.equal(big[:M, :N].double(), want)
    assert (big[M:] == 7).all() and (big[:, N:] == 7).all()
    assert torch.equal(mx.mxfp4_fp8_gemm(a, b), want.float().to(torch.bfloat16))
    assert (mx.mxfp4_fp8_gemm_workspace_bytes(a, b) > 0) == (K == 4200)


def check_quantized(q, want, error, what):
    """q is a quantization of `want` (binary64) that the GPU had within `error` of: its scale is that of a maximum within
    it, its values are within half a step."""
    rows, k = want.shape
    blocks = R.up(k, 128) // 128
    assert (q.rows, q.k) == (rows, k) and not q.codes[:, k:R.up(k, 128)].any(), what

    def tops(v):
        p = torch.zeros((rows, blocks * 128), dtype=torch.float64, device="cuda")
        p[:, :k] = v
        return p.view(rows, blocks, 128).amax(2)

    def exponent(top):   # the least e with 448 2^e >= top
        m, e = torch.frexp(top / 448)
        return torch.where(top > 0, torch.where(m == 0.5, e - 1, e).clamp(-127, 127), -127)
    got = q.scales[:, :rows].t().int() - 127
    lo, hi = exponent(tops((want.abs() - error).clamp(min=0))), exponent(tops(want.abs() + error))
    assert bool(((lo <= got) & (got <= hi)).all()), what
    f = torch.exp2(got.double()).repeat_interleave(128, 1)[:, :k]
    v = q.elements().double() * f
    lim = torch.maximum(2.0 ** -4 * (want.abs() + error), 2.0 ** -10 * f) + error
    assert bool(((v - want).abs() <= lim).all()), what


def activation(name, g):
    if name == "silu":
        return g * torch.sigmoid(g)
    return torch.nn.functional.gelu(g, approximate="none" if name == "gelu" else "tanh")


GATED = [   # tiles of 256 rows x 128 outputs
    (4200, 200, 2100, "silu"),        # 272 tiles: 256 whole, 16 in halves, a last row of 17 halves
    (2600, 130, 5100, "gelu_tanh"),   # 400 whole tiles, none cut, and a last row of 40
    (1800, 300, 2400, "gelu"),        # 133 whole tiles and a last row of 8 tokens
    (4096, 128, 2176, "silu"),        # 272: no ragged side
]


@pytest.mark.parametrize("T,H,n,act", GATED)
def test_gated_of_many_tiles(T, H, n, act):
    mx = need_gpu()
    say("fp8 gated, many tiles", T, H, n, act)
    np_ = R.up(n, 128)
    # projections of about one, the largest of several: steps of 2^-9, exact
    (x, xv), (w, wv) = whole_numbers(mx, T, H, 411, (-4, -3)), whole_numbers(mx, 2 * np_, H, 412, (-5, -3), n)
    both = torch.mm(xv, wv.t().contiguous())
    g, u = both[:, :n], both[:, np_:np_ + n]
    assert both.abs().max().item() * 2 ** 9 < 2 ** 24 and 0.5 < g.std().item() < 20
    # (one rounding each of the exponential, the quotient and the products: a few units of binary32)
    h = activation(act, g) * u
    error = 2e-6 * h.abs() + 1e-6 * u.abs()
    q, gg, gu = mx.mxfp4_fp8_gated(x, w, act=act, train=True)
    assert torch.equal(gg, g.float().to(torch.bfloat16)) and torch.equal(gu, u.float().to(torch.bfloat16))
    check_quantized(q, h, error, "with g and u")
    alone = mx.mxfp4_fp8_gated(x, w, act=act)
    assert torch.equal(alone.codes, q.codes) and torch.equal(alone.scales[:, :T], q.scales[:, :T])
    big = torch.full((T + 1, n + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    mx.mxfp4_fp8_gated(x, w, act=act, dtype=torch.bfloat16, out=big[:T, :n])
    assert bool(((big[:T, :n].double() - h).abs() <= BF16 * (h.abs() + error) + error).all())
    assert (big[T:] == 7).all() and (big[:, n:] == 7).all()


# (rows, width): more rows than workgroups take at once (2048 of one row each, or of four rows up to a width of 2048),
# in every number of waves and chunks, with and without a ragged end
NORMS = [(20000, 136), (9000, 1001), (9000, 1536), (8500, 2047), (4500, 2055), (4300, 4096), (2100, 6145), (2100, 8190),
         (2100, 12288), (2100, 16385), (2100, 20481), (2100, 28000), (2060, 32761)]


def rows(T, H, std, seed):
    return (torch.randn((T, H), generator=gen(seed), device="cuda") * std).to(torch.bfloat16)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,H", NORMS)
def test_rmsnorm_of_many_rows(T, H, residual):
    mx = need_gpu()
    say("fp8 norm, many rows", T, H, residual)
    x, res, w = rows(T, H, 1.0, 421), rows(T, H, 2.0, 422) if residual else None, rows(1, H, 1.0, 423)[0]
    x = x * torch.logspace(-2, 2, T, device="cuda")[:, None].to(torch.bfloat16)   # (no two rows alike in size)
    sums = x if res is None else (x.float() + res.float()).to(torch.bfloat16)
    q, r, y, rstd = mx.mxfp4_fp8_rmsnorm(x, w, R.EPS, res, train=True)
    assert torch.equal(r, sums)
    d = sums.double()
    want_s = (d.square().mean(1) + R.EPS).rsqrt()
    want = d * want_s[:, None] * w.double()
    assert bool(((rstd.double() - want_s).abs() <= 5e-6 * want_s).all())
    assert bool(((y.double() - want).abs() <= (BF16 + 1e-5) * want.abs() + 1e-38).all())
    check_quantized(q, want, 1e-5 * want.abs(), "norm")


@pytest.mark.parametrize("dres", [False, True])
@pytest.mark.parametrize("T,H", NORMS)
def test_rmsnorm_backward_of_many_rows(T, H, dres):
    mx = need_gpu()
    say("fp8 norm backward, many rows", T, H, dres)
    dy, r, e, w = rows(T, H, 1e-3, 431), rows(T, H, 1.0, 432), rows(T, H, 1e-3, 433), rows(1, H, 1.0, 434)[0]
    r = r * torch.logspace(-2, 2, T, device="cuda")[:, None].to(torch.bfloat16)
    rstd = (r.double().square().mean(1) + R.EPS).rsqrt().float()
    dx, dw = mx.mxfp4_fp8_rmsnorm_backward(dy, r, w, rstd, e if dres else None)
    s, a = rstd.double()[:, None], dy.double() * w.double()
    xh = r.double() * s
    want = s * (a - xh * (a * xh).mean(1, keepdim=True)) + (e.double() if dres else 0)
    size = s * (a.abs() + xh.abs() * (a * xh).abs().mean(1, keepdim=True)) + (e.double().abs() if dres else 0)
    assert bool(((dx.double() - want).abs() <= 1e-5 * size * (1 + BF16) + BF16 * want.abs() + 1e-38).all())
    # dw: T terms in at most 512 runs (of four rows' sums, to a width of 2048), then 16 and 32: under 200 u of their size
    t = dy.double() * xh
    assert bool(((dw.double() - t.sum(0)).abs() <= 1.2e-5 * t.abs().sum(0) + 1e-38).all())
