// fp8_internal.h -- launchers of the block-128 FP8 operators, shared between
// their C ABI and their kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxfp4 {

// Where a quantizer writes: element (r, c) of a [rows, k] matrix at
// codes[r * ld + c], the scale of its block at scales[(c / 128) * scale_ld + r].
struct Fp8Out {
  uint8_t* codes;
  uint8_t* scales;
  int64_t ld, scale_ld;
};

// An operand of the products: the same layout, read only.
struct Fp8In {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t ld, scale_ld;
  int64_t rows;
};

// A launch holds fewer than 2^32 threads along x: more are cut off without an
// error just past it, and refused further on.
constexpr int64_t FP8_LAUNCH_THREADS = ((int64_t)1 << 32) - 1;

// Bytes that a product may read from line 0's scale of row `first` of an
// operand, over its kb lines: up to the last line's own last row, in loads of
// `unit` bytes at multiples of it (lines and operands start at multiples of
// 16).  A view's lines start inside those of a wider matrix, whose memory may end
// with the view's last row, a whole line pitch before that of a full matrix.
constexpr int64_t fp8_scale_extent(int64_t kb, int64_t scale_ld, int64_t rows, int64_t first, int unit) {
  return kb > 0 && first < rows ? (kb - 1) * scale_ld + (rows + unit - 1) / unit * unit - first : 0;
}

struct GatedGradArgs {
  const uint16_t *dh, *g, *u;
  int64_t ldd, ldg, ldu;
  int64_t T, n, np;      // rows, columns, columns rounded up to 128
  Fp8Out dgu, dgut, ht;  // [T, 2 np], [2 np, T], [n, T] (ht.codes may be NULL)
};

hipError_t launch_fp8_quantize(const uint16_t* x, int64_t R, int64_t C, int64_t ldx, int axis, int block_rows,
                               const Fp8Out& out, hipStream_t s);
hipError_t launch_fp8_gated_grad(int act, const GatedGradArgs& a, hipStream_t s);
hipError_t launch_fp8_dequantize(const uint8_t* codes, int64_t ld, const uint8_t* scales, int64_t scale_ld,
                                 int64_t rows, int64_t k, float* y, int64_t ldy, hipStream_t s);

struct Fp8NormArgs {
  const uint16_t *x, *res, *w;
  int64_t ldx, ldr;
  int64_t T, H;
  float eps;
  Fp8Out q;
  uint16_t* sum;         // x + res (NULL without a residual)
  int64_t lds;
  uint16_t* y;           // the norm in bf16 (may be NULL)
  int64_t ldy;
  float* rstd;           // may be NULL
};
hipError_t launch_fp8_rmsnorm(const Fp8NormArgs& a, hipStream_t s);

struct Fp8NormGradArgs {
  const uint16_t *dy, *r, *w, *dres;   // dres may be NULL
  int64_t ldd, ldr, lde;
  int64_t T, H;
  const float* rstd;
  uint16_t* dx;
  int64_t ldx;
  float* dw;
  float* parts;          // [groups, H]
};
int64_t fp8_rmsnorm_grad_groups(int64_t T, int64_t H);
hipError_t launch_fp8_rmsnorm_grad(const Fp8NormGradArgs& a, hipStream_t s);

// Products.  What a launch writes:
constexpr int FP8_F32 = 0, FP8_BF16 = 1;
struct Fp8Plan {
  int decode;            // 16-row tiles of A of the decode kernel; 0 = wide tiles
  int half;              // wide tiles of 128 rows
  int splits;            // of the contraction
};
Fp8Plan plan_fp8_gemm(int64_t M, int64_t N, int64_t K);
size_t fp8_gemm_workspace(const Fp8Plan& p, int64_t M, int64_t N);
hipError_t launch_fp8_gemm(const Fp8In& a, const Fp8In& b, int64_t K, void* C, int64_t ldc, int c_type,
                           float* workspace, const Fp8Plan& plan, hipStream_t s);

// Two independent products, the first's result in bf16; together: in one launch.
struct Fp8TwoPlan {
  Fp8Plan first, second;
  int together;
};
Fp8TwoPlan plan_fp8_two(int64_t M0, int64_t N0, int64_t K0, int64_t M1, int64_t N1, int64_t K1);
hipError_t launch_fp8_two(const Fp8In& a0, const Fp8In& b0, int64_t K0, void* C0, int64_t ldc0, const Fp8In& a1,
                          const Fp8In& b1, int64_t K1, void* C1, int64_t ldc1, int c1_type, float* workspace,
                          const Fp8TwoPlan& plan, hipStream_t s);

struct Fp8GatedArgs {
  Fp8In x, w;            // w: rows 0 .. np - 1 the gate's, np .. 2 np - 1 the up projection's
  int64_t K, n, np;
  int act;
  Fp8Out q;              // codes NULL: none
  uint16_t* h;           // bf16 result, may be NULL
  int64_t ldh;
  uint16_t *g, *u;       // both projections in bf16, may be NULL
  int64_t ldgu;
};
size_t fp8_gated_workspace(int64_t M, int64_t np, int64_t K, bool fp8_out);
hipError_t launch_fp8_gated(const Fp8GatedArgs& a, float* workspace, hipStream_t s);

}  // namespace mxfp4
