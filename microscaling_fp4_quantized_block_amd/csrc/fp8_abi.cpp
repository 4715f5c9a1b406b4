// fp8_abi.cpp -- the C ABI of the block-128 FP8 operators: argument checks,
// sizes, dispatch.  As everywhere in the library every argument is checked
// before anything is launched, and nothing is allocated, freed or
// synchronized.  The operations are described in mxfp4.h.
#include "mxfp4.h"

#include <hip/hip_runtime.h>

#include "fp8_internal.h"

namespace {

using mxfp4::Fp8In;
using mxfp4::Fp8Out;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Rows and columns: sizes below stay below 2^63.  (One launch does not hold
// every grid of 128 x 128 tiles: see in_parts and decode_tiles.)
constexpr int64_t kMaxSide = (int64_t)1 << 30;
constexpr int64_t kMaxElems = (int64_t)1 << 40;
// Operands of the products: 128 rows of codes, and all scales, are reached
// through 32-bit offsets of a buffer resource.
constexpr int64_t kMaxLd = (int64_t)1 << 23;
constexpr int64_t kMaxScales = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxNormH = 32768;   // a row stays in the registers of one workgroup

bool sides_ok(int64_t r, int64_t c) { return r <= kMaxSide && c <= kMaxSide && (r == 0 || c <= kMaxElems / r); }

// A descriptor whose buffers a kernel may touch.
mxfp4_status check_tensor(const mxfp4_fp8_tensor* q) {
  if (!q || q->rows < 0 || q->k < 0) return MXFP4_ERR_INVALID_ARG;
  if (!sides_ok(q->rows, q->k)) return MXFP4_ERR_UNSUPPORTED_SHAPE;
  if (q->rows == 0 || q->k == 0) return MXFP4_OK;
  if (q->ld < up(q->k, 128) || q->ld % 16 != 0 || q->scale_ld < q->rows || q->scale_ld % 16 != 0)
    return MXFP4_ERR_INVALID_ARG;
  if (!q->codes || !q->scales || !aligned(q->codes, 16) || !aligned(q->scales, 16)) return MXFP4_ERR_INVALID_ARG;
  return MXFP4_OK;
}

// ... and one that a product reads.
mxfp4_status check_operand(const mxfp4_fp8_tensor* q) {
  const mxfp4_status st = check_tensor(q);
  if (st != MXFP4_OK || q->rows == 0 || q->k == 0) return st;
  if (q->ld > kMaxLd || up(q->k, 128) / 128 > kMaxScales / q->scale_ld) return MXFP4_ERR_UNSUPPORTED_SHAPE;
  return MXFP4_OK;
}

Fp8Out out_of(const mxfp4_fp8_tensor* q) { return Fp8Out{q->codes, q->scales, q->ld, q->scale_ld}; }
Fp8In in_of(const mxfp4_fp8_tensor* q) { return Fp8In{q->codes, q->scales, q->ld, q->scale_ld, q->rows}; }

// A bf16 matrix argument.
bool matrix_ok(const void* p, int64_t cols, int64_t ld) { return p && ld >= cols && ld >= 1 && aligned(p, 2); }
mxfp4_status of(hipError_t e) { return e == hipSuccess ? MXFP4_OK : MXFP4_ERR_HIP; }

mxfp4::Fp8Plan plan_of(const mxfp4_fp8_tensor* A, const mxfp4_fp8_tensor* B) {
  return mxfp4::plan_fp8_gemm(A->rows, B->rows, A->k);
}

mxfp4_status check_pair(const mxfp4_fp8_tensor* A, const mxfp4_fp8_tensor* B) {
  mxfp4_status st = check_operand(A);
  if (st != MXFP4_OK) return st;
  if ((st = check_operand(B)) != MXFP4_OK) return st;
  if (A->k != B->k) return MXFP4_ERR_FORMAT_MISMATCH;
  return MXFP4_OK;
}

}  // namespace

extern "C" {

mxfp4_status mxfp4_fp8_tensor_bytes(int64_t rows, int64_t k, size_t* codes_bytes, size_t* scales_bytes) {
  if (rows < 0 || k < 0 || !codes_bytes || !scales_bytes) return MXFP4_ERR_INVALID_ARG;
  if (!sides_ok(rows, k)) return MXFP4_ERR_UNSUPPORTED_SHAPE;
  *codes_bytes = (size_t)rows * (size_t)up(k, 128);
  *scales_bytes = (size_t)(up(k, 128) / 128) * (size_t)up(rows, 16);
  return MXFP4_OK;
}

mxfp4_status mxfp4_fp8_quantize(const uint16_t* x, int64_t R, int64_t C, int64_t ldx, int axis, int block_rows,
                                mxfp4_fp8_tensor* out, hipStream_t stream) {
  if ((axis != 0 && axis != 1) || (block_rows != 1 && block_rows != 128) || R < 0 || C < 0 || !out)
    return MXFP4_ERR_INVALID_ARG;
  if (!sides_ok(R, C)) return MXFP4_ERR_UNSUPPORTED_SHAPE;
  if (out->rows != (axis ? R : C) || out->k != (axis ? C : R)) return MXFP4_ERR_INVALID_ARG;
  const mxfp4_status st = check_tensor(out);
  if (st != MXFP4_OK || R == 0 || C == 0) return st;
  if (!matrix_ok(x, C, ldx)) return MXFP4_ERR_INVALID_ARG;
  return of(mxfp4::launch_fp8_quantize(x, R, C, ldx, axis, block_rows, out_of(out), stream));
}

mxfp4_status mxfp4_fp8_dequantize(const mxfp4_fp8_tensor* q, float* y, int64_t ldy, hipStream_t stream) {
  const mxfp4_status st = check_tensor(q);
  if (st != MXFP4_OK || q->rows == 0 || q->k == 0) return st;
  if (!y || ldy < q->k || !aligned(y, 4)) return MXFP4_ERR_INVALID_ARG;
  return of(mxfp4::launch_fp8_dequantize(q->codes, q->ld, q->scales, q->scale_ld, q->rows, q->k, y, ldy, stream));
}

mxfp4_status mxfp4_fp8_gemm_workspace_bytes(const mxfp4_fp8_tensor* A, const mxfp4_fp8_tensor* B, size_t* bytes) {
  if (!bytes) return MXFP4_ERR_INVALID_ARG;
  const mxfp4_status st = check_pair(A, B);
  if (st != MXFP4_OK) return st;
  *bytes = A->rows && B->rows ? mxfp4::fp8_gemm_workspace(plan_of(A, B), A->rows, B->rows) : 0;
  return MXFP4_OK;
}

mxfp4_status mxfp4_fp8_gemm(const mxfp4_fp8_tensor* A, const mxfp4_fp8_tensor* B, void* C, int64_t ldc, int c_type,
                            void* workspace, size_t ws_bytes, hipStream_t stream) {
  if (c_type != MXFP4_C_F32 && c_type != MXFP4_C_BF16) return MXFP4_ERR_INVALID_ARG;
  const mxfp4_status st = check_pair(A, B);
  if (st != MXFP4_OK || A->rows == 0 || B->rows == 0) return st;
  if (!C || ldc < B->rows || !aligned(C, c_type == MXFP4_C_F32 ? 4 : 2)) return MXFP4_ERR_INVALID_ARG;
  const mxfp4::Fp8Plan plan = plan_of(A, B);
  const size_t need = mxfp4::fp8_gemm_workspace(plan, A->rows, B->rows);
  if (need && (!workspace || ws_bytes < need || !aligned(workspace, 16))) return MXFP4_ERR_WORKSPACE;
  return of(mxfp4::launch_fp8_gemm(in_of(A), in_of(B), A->k, C, ldc,
                                   c_type == MXFP4_C_BF16 ? mxfp4::FP8_BF16 : mxfp4::FP8_F32, (float*)workspace, plan,
                                   stream));
}

mxfp4_status mxfp4_fp8_rmsnorm(const uint16_t* x, int64_t T, int64_t H, int64_t ldx, const uint16_t* residual,
                               int64_t ldr, const uint16_t* weight, float eps, mxfp4_fp8_tensor* out, uint16_t* sum,
                               int64_t lds, uint16_t* y, int64_t ldy, float* rstd, hipStream_t stream) {
  if (T < 0 || H < 0 || !out || !(eps >= 0.0f)) return MXFP4_ERR_INVALID_ARG;
  if (H > kMaxNormH || !sides_ok(T, H)) return MXFP4_ERR_UNSUPPORTED_SHAPE;
  if (out->rows != T || out->k != H || (residual == nullptr) != (sum == nullptr)) return MXFP4_ERR_INVALID_ARG;
  const mxfp4_status st = check_tensor(out);
  if (st != MXFP4_OK || T == 0 || H == 0) return st;
  if (!matrix_ok(x, H, ldx) || !weight || !aligned(weight, 2)) return MXFP4_ERR_INVALID_ARG;
  if (residual && (!matrix_ok(residual, H, ldr) || !matrix_ok(sum, H, lds))) return MXFP4_ERR_INVALID_ARG;
  if ((y && !matrix_ok(y, H, ldy)) || !aligned(rstd, 4)) return MXFP4_ERR_INVALID_ARG;
  mxfp4::Fp8NormArgs a{};
  a.x = x; a.ldx = ldx; a.res = residual; a.ldr = ldr; a.w = weight; a.T = T; a.H = H; a.eps = eps;
  a.q = out_of(out); a.sum = sum; a.lds = lds; a.y = y; a.ldy = ldy; a.rstd = rstd;
  return of(mxfp4::launch_fp8_rmsnorm(a, stream));
}

mxfp4_status mxfp4_fp8_rmsnorm_backward_workspace_bytes(int64_t T, int64_t H, size_t* bytes) {
  if (T < 0 || H < 0 || !bytes) return MXFP4_ERR_INVALID_ARG;
  if (H > kMaxNormH || !sides_ok(T, H)) return MXFP4_ERR_UNSUPPORTED_SHAPE;
  *bytes = (size_t)mxfp4::fp8_rmsnorm_grad_groups(T, H) * (size_t)H * sizeof(float);
  return MXFP4_OK;
}

mxfp4_status mxfp4_fp8_rmsnorm_backward(const uint16_t* dy, int64_t T, int64_t H, int64_t ldd, const uint16_t* r,
                                        int64_t ldr, const uint16_t* weight, const float* rstd, const uint16_t* dres,
                                        int64_t lde, uint16_t* dx, int64_t ldx, float* dw, void* workspace,
                                        size_t ws_bytes, hipStream_t stream) {
  if (T < 0 || H < 0) return MXFP4_ERR_INVALID_ARG;
  if (H > kMaxNormH || !sides_ok(T, H)) return MXFP4_ERR_UNSUPPORTED_SHAPE;
  if (H == 0) return MXFP4_OK;
  if (!dw || !aligned(dw, 4) || !weight || !aligned(weight, 2)) return MXFP4_ERR_INVALID_ARG;
  if (T > 0) {
    if (!matrix_ok(dy, H, ldd) || !matrix_ok(r, H, ldr) || !matrix_ok(dx, H, ldx) || !rstd || !aligned(rstd, 4))
      return MXFP4_ERR_INVALID_ARG;
    if (dres && !matrix_ok(dres, H, lde)) return MXFP4_ERR_INVALID_ARG;
  }
  const size_t need = (size_t)mxfp4::fp8_rmsnorm_grad_groups(T, H) * (size_t)H * sizeof(float);
  if (need && (!workspace || ws_bytes < need || !aligned(workspace, 16))) return MXFP4_ERR_WORKSPACE;
  mxfp4::Fp8NormGradArgs a{};
  a.dy = dy; a.ldd = ldd; a.r = r; a.ldr = ldr; a.w = weight; a.dres = dres; a.lde = lde; a.T = T; a.H = H;
  a.rstd = rstd; a.dx = dx; a.ldx = ldx; a.dw = dw; a.parts = (float*)workspace;
  return of(mxfp4::launch_fp8_rmsnorm_grad(a, stream));
}

// The gated block's operands: x [T, k] and w [2 np, k], np = n rounded up to 128.
static mxfp4_status check_gated(const mxfp4_fp8_tensor* x, const mxfp4_fp8_tensor* w, int64_t n, int act) {
  if (n < 0 || act < MXFP4_ACT_SILU || act > MXFP4_ACT_GELU_TANH) return MXFP4_ERR_INVALID_ARG;
  if (n > kMaxSide / 2) return MXFP4_ERR_UNSUPPORTED_SHAPE;
  const mxfp4_status st = check_pair(x, w);
  if (st != MXFP4_OK) return st;
  return w->rows == 2 * up(n, 128) ? MXFP4_OK : MXFP4_ERR_INVALID_ARG;
}

mxfp4_status mxfp4_fp8_gated_workspace_bytes(const mxfp4_fp8_tensor* x, const mxfp4_fp8_tensor* w, int64_t n,
                                             int fp8_out, size_t* bytes) {
  if (!bytes || (fp8_out != 0 && fp8_out != 1)) return MXFP4_ERR_INVALID_ARG;
  const mxfp4_status st = check_gated(x, w, n, MXFP4_ACT_SILU);
  if (st != MXFP4_OK) return st;
  *bytes = x->rows ? mxfp4::fp8_gated_workspace(x->rows, up(n, 128), x->k, fp8_out) : 0;
  return MXFP4_OK;
}

mxfp4_status mxfp4_fp8_gated(const mxfp4_fp8_tensor* x, const mxfp4_fp8_tensor* w, int64_t n, int act,
                             mxfp4_fp8_tensor* out, uint16_t* h, int64_t ldh, uint16_t* g, uint16_t* u, int64_t ldgu,
                             void* workspace, size_t ws_bytes, hipStream_t stream) {
  mxfp4_status st = check_gated(x, w, n, act);
  if (st != MXFP4_OK) return st;
  if ((!out && !h) || (g == nullptr) != (u == nullptr)) return MXFP4_ERR_INVALID_ARG;
  const int64_t T = x->rows, np = up(n, 128);
  if (out) {
    if (out->rows != T || out->k != n) return MXFP4_ERR_INVALID_ARG;
    if ((st = check_tensor(out)) != MXFP4_OK) return st;
  }
  if (T == 0 || n == 0) return MXFP4_OK;
  if (x->k == 0) return MXFP4_ERR_UNSUPPORTED_SHAPE;
  if ((h && !matrix_ok(h, n, ldh)) || (g && (!matrix_ok(g, n, ldgu) || !aligned(u, 2)))) return MXFP4_ERR_INVALID_ARG;
  const size_t need = mxfp4::fp8_gated_workspace(T, np, x->k, out != nullptr);
  if (need && (!workspace || ws_bytes < need || !aligned(workspace, 16))) return MXFP4_ERR_WORKSPACE;
  mxfp4::Fp8GatedArgs a{};
  a.x = in_of(x); a.w = in_of(w); a.K = x->k; a.n = n; a.np = np; a.act = act;
  if (out) a.q = out_of(out);
  a.h = h; a.ldh = ldh; a.g = g; a.u = u; a.ldgu = ldgu;
  return of(mxfp4::launch_fp8_gated(a, (float*)workspace, stream));
}

// Workspace of the backward pass: dgu and its transpose, then what the larger
// of the two products needs.
struct GatedBackward {
  mxfp4_fp8_tensor dgu, dgut;
  mxfp4::Fp8TwoPlan plan;   // dx = dgu wt, dw = dgut xt
  size_t at[4], gemm, gemm_at, bytes;
};
static GatedBackward layout_gated_backward(int64_t T, int64_t n, const mxfp4_fp8_tensor* wt,
                                           const mxfp4_fp8_tensor* xt) {
  const int64_t np = up(n, 128);
  GatedBackward b{};
  b.dgu = mxfp4_fp8_tensor{T, 2 * np, 2 * np, up(T, 16), nullptr, nullptr};
  b.dgut = mxfp4_fp8_tensor{2 * np, T, up(T, 128), 2 * np, nullptr, nullptr};
  size_t at = 0;
  auto take = [&](size_t n) { const size_t was = at; at += (n + 255) / 256 * 256; return was; };
  b.at[0] = take((size_t)T * (size_t)b.dgu.ld);
  b.at[1] = take((size_t)(2 * np / 128) * (size_t)b.dgu.scale_ld);
  b.at[2] = take((size_t)(2 * np) * (size_t)b.dgut.ld);
  b.at[3] = take((size_t)(b.dgut.ld / 128) * (size_t)b.dgut.scale_ld);
  b.plan = mxfp4::plan_fp8_two(T, wt->rows, 2 * np, 2 * np, xt->rows, T);
  const size_t g1 = mxfp4::fp8_gemm_workspace(b.plan.first, T, wt->rows);
  const size_t g2 = mxfp4::fp8_gemm_workspace(b.plan.second, 2 * np, xt->rows);
  b.gemm = g1 > g2 ? g1 : g2;
  b.gemm_at = take(b.gemm);
  b.bytes = at;
  return b;
}

static mxfp4_status check_gated_backward(int64_t T, int64_t n, const mxfp4_fp8_tensor* wt,
                                         const mxfp4_fp8_tensor* xt) {
  if (T < 0 || n < 0) return MXFP4_ERR_INVALID_ARG;
  if (n > kMaxSide / 2 || !sides_ok(T, 2 * up(n, 128))) return MXFP4_ERR_UNSUPPORTED_SHAPE;
  mxfp4_status st = check_operand(wt);
  if (st != MXFP4_OK) return st;
  if ((st = check_operand(xt)) != MXFP4_OK) return st;
  if (wt->k != 2 * up(n, 128) || xt->k != T || wt->rows != xt->rows) return MXFP4_ERR_FORMAT_MISMATCH;
  // the gradients are operands themselves
  if (up(T, 128) > kMaxLd || 2 * up(n, 128) > kMaxLd ||
      (n > 0 && T > 0 && up(T, 128) / 128 + 1 > kMaxScales / (2 * up(n, 128))))
    return MXFP4_ERR_UNSUPPORTED_SHAPE;
  return MXFP4_OK;
}

mxfp4_status mxfp4_fp8_gated_backward_workspace_bytes(int64_t T, int64_t n, const mxfp4_fp8_tensor* wt,
                                                      const mxfp4_fp8_tensor* xt, size_t* bytes) {
  if (!bytes) return MXFP4_ERR_INVALID_ARG;
  const mxfp4_status st = check_gated_backward(T, n, wt, xt);
  if (st != MXFP4_OK) return st;
  *bytes = layout_gated_backward(T, n, wt, xt).bytes;
  return MXFP4_OK;
}

mxfp4_status mxfp4_fp8_gated_backward(const uint16_t* dh, int64_t ldd, const uint16_t* g, const uint16_t* u,
                                      int64_t ldgu, int64_t T, int64_t n, int act, const mxfp4_fp8_tensor* wt,
                                      const mxfp4_fp8_tensor* xt, uint16_t* dx, int64_t ldx, void* dw, int64_t ldw,
                                      int dw_type, mxfp4_fp8_tensor* ht, void* workspace, size_t ws_bytes,
                                      hipStream_t stream) {
  if (act < MXFP4_ACT_SILU || act > MXFP4_ACT_GELU_TANH || (dw_type != MXFP4_C_F32 && dw_type != MXFP4_C_BF16))
    return MXFP4_ERR_INVALID_ARG;
  mxfp4_status st = check_gated_backward(T, n, wt, xt);
  if (st != MXFP4_OK) return st;
  if (ht) {
    if (ht->rows != n || ht->k != T) return MXFP4_ERR_INVALID_ARG;
    if ((st = check_tensor(ht)) != MXFP4_OK) return st;
  }
  const int64_t H = wt->rows;
  const bool tokens = T > 0 && H > 0, weights = n > 0 && H > 0, grads = T > 0 && n > 0;
  if (grads && (!matrix_ok(dh, n, ldd) || !matrix_ok(g, n, ldgu) || !matrix_ok(u, n, ldgu)))
    return MXFP4_ERR_INVALID_ARG;
  if (tokens && !matrix_ok(dx, H, ldx)) return MXFP4_ERR_INVALID_ARG;
  if (weights && (!dw || ldw < H || !aligned(dw, dw_type == MXFP4_C_F32 ? 4 : 2))) return MXFP4_ERR_INVALID_ARG;
  GatedBackward b = layout_gated_backward(T, n, wt, xt);
  if (b.bytes && (!workspace || ws_bytes < b.bytes || !aligned(workspace, 256))) return MXFP4_ERR_WORKSPACE;
  uint8_t* base = (uint8_t*)workspace;
  if (grads) {
    b.dgu.codes = base + b.at[0];
    b.dgu.scales = base + b.at[1];
    b.dgut.codes = base + b.at[2];
    b.dgut.scales = base + b.at[3];
    mxfp4::GatedGradArgs a{};
    a.dh = dh; a.g = g; a.u = u; a.ldd = ldd; a.ldg = ldgu; a.ldu = ldgu;
    a.T = T; a.n = n; a.np = up(n, 128);
    a.dgu = out_of(&b.dgu);
    a.dgut = out_of(&b.dgut);
    if (ht) a.ht = out_of(ht);
    if (mxfp4::launch_fp8_gated_grad(act, a, stream) != hipSuccess) return MXFP4_ERR_HIP;
  }
  void* gemm_ws = b.gemm ? base + b.gemm_at : nullptr;
  const int c_type = dw_type == MXFP4_C_BF16 ? mxfp4::FP8_BF16 : mxfp4::FP8_F32;
  if (tokens && weights)
    return of(mxfp4::launch_fp8_two(in_of(&b.dgu), in_of(wt), b.dgu.k, dx, ldx, in_of(&b.dgut), in_of(xt), T, dw, ldw,
                                    c_type, (float*)gemm_ws, b.plan, stream));
  // (no tokens, or no columns: the product over them is zero)
  st = tokens ? mxfp4_fp8_gemm(&b.dgu, wt, dx, ldx, MXFP4_C_BF16, gemm_ws, b.gemm, stream) : MXFP4_OK;
  if (st != MXFP4_OK) return st;
  return weights ? mxfp4_fp8_gemm(&b.dgut, xt, dw, ldw, dw_type, gemm_ws, b.gemm, stream) : MXFP4_OK;
}

}  // extern "C"
