// fp8_quantize.hip -- bf16 to block-128 FP8 (E4M3 elements, E8M0 scales), along
// rows, along columns (written transposed), in 128 x 128 blocks, and the gated
// block's gradients quantized both ways in one pass.
//
// All of it is bound by memory: a quantizer reads 2 bytes and writes 1 per
// element, the gated gradient reads 6 and writes 4.  16384 x 11008 takes 93 us
// along rows and 102 us along columns (5.8 and 5.3 TB/s; a large copy reaches
// 5.2).  Two kernels:
//   rows   16 lanes hold one 128-block (16 bytes per lane), so the block's
//          maximum takes four DPP rotations and no LDS.
//   tile   128 x 128 elements per workgroup of 512 threads, thread t holding
//          rows 4 (t / 16) .. + 3 of columns 8 (t % 16) .. + 7: row maxima over
//          16 lanes, column maxima over a thread's 4 rows, the wave's four row
//          groups and, through LDS, the eight waves.  Codes along the columns
//          turn around in LDS, so both layouts are written in whole
//          128-byte lines.
#include "fp8_device.h"
#include "fp8_internal.h"

namespace mxfp4 {

// ---------------------------------------------------------------------------
// Along rows
// ---------------------------------------------------------------------------
// Workgroup: 16 rows x ROWS_NB blocks; 16-lane group i takes row i of them, so a
// lane has 64 bytes in flight and a row's group writes 512 bytes of codes.
constexpr int ROWS_NB = 4;

__global__ void __launch_bounds__(256) fp8_rows_kernel(const uint16_t* __restrict__ x, int64_t R, int64_t C,
                                                       int64_t ldx, int64_t blocks, int64_t groups,
                                                       Fp8Out out) {
  const int64_t bg = blockIdx.x % groups, rg = blockIdx.x / groups;
  const int64_t row = rg * 16 + (threadIdx.x >> 4);
  const int l = threadIdx.x & 15;
  if (row >= R) return;
  const uint16_t* src = x + row * ldx;
  u32v4 p[ROWS_NB];
#pragma unroll
  for (int j = 0; j < ROWS_NB; j++) {
    const int64_t b = bg * ROWS_NB + j;
    if (b < blocks) p[j] = fetch8(src, b * FP8_BLOCK + 8 * l, C);
  }
  uint32_t mine = 0;
#pragma unroll
  for (int j = 0; j < ROWS_NB; j++) {
    const int64_t b = bg * ROWS_NB + j;
    if (b >= blocks) break;
    settle8(p[j], b * FP8_BLOCK + 8 * l, C);
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < 4; q++) m = pk_max_u16(m, p[j][q] & 0x7FFF7FFFu);
    m = max16(max(m & 0xFFFFu, m >> 16) << 16);
    const uint32_t byte = fp8_scale_byte(m);
    float v[8];
    bf16x8_to_f32(p[j], v);
    *(u32v2*)(out.codes + row * out.ld + b * FP8_BLOCK + 8 * l) = fp8_encode8(v, byte);
    if (l == j) mine = byte;
  }
  if (l < ROWS_NB && bg * ROWS_NB + l < blocks) out.scales[(bg * ROWS_NB + l) * out.scale_ld + row] = (uint8_t)mine;
}

// ---------------------------------------------------------------------------
// 128 x 128 tiles
// ---------------------------------------------------------------------------
constexpr int TILE_THREADS = 512;

struct TileShared {
  uint8_t turn[128 * 128];            // codes along the columns: column c at 128 c, 8-byte chunks swizzled
  uint32_t top[3][128];               // maxima of each column (SQUARE: of the tile, in [0][0]), one line per tile
};

// (maxima do not depend on the order in which the waves bring theirs)
__device__ __forceinline__ void clear_tops(TileShared& sh) {
  if (threadIdx.x < 3 * 128) sh.top[0][threadIdx.x] = 0;
  __syncthreads();
}

// Chunk (8 rows) q of column c sits at position q ^ (c / 8 & 14): the eight
// columns of a thread and its neighbours' then fall on different banks, and
// chunk pairs stay 16 contiguous bytes.
__device__ __forceinline__ int turn_at(int c, int q) { return c * 128 + ((q ^ ((c >> 3) & 14)) << 3); }

// Writes the tile v (this thread's 4 rows x 8 columns, rows r0 + 4 rg + i,
// columns c0 + 8 cg + j) into either output that is asked for.  rows: codes
// along the rows at out row r0 + .., out column c0 + .., rows up to R.
// cols: the transpose, out row c0 + .., out column r0 + .., out rows up to
// CR.  SQUARE: one scale for the whole tile.  WHOLE: every row and column of the
// tile is there.  sh.top[n] has been cleared.
template <bool ROWS, bool COLS, bool SQUARE, bool WHOLE>
__device__ __forceinline__ void quantize_tile(TileShared& sh, int n, const float (&v)[4][8], int64_t r0, int64_t c0,
                                              const Fp8Out& rows, int64_t R, const Fp8Out& cols, int64_t CR) {
  const int t = threadIdx.x, cg = t & 15, rg = t >> 4;
  uint32_t rm[4], cm[8];
#pragma unroll
  for (int i = 0; i < 4; i++) rm[i] = 0;
#pragma unroll
  for (int j = 0; j < 8; j++) cm[j] = 0;
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const uint32_t a = abs_bits(v[i][j]);
      if (ROWS || SQUARE) rm[i] = max(rm[i], a);
      if (COLS && !SQUARE) cm[j] = max(cm[j], a);
    }
  if constexpr (SQUARE) {
    uint32_t m = max16(max(max(rm[0], rm[1]), max(rm[2], rm[3])));
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if ((t & 63) == 0) atomicMax(&sh.top[n][0], m);
    __syncthreads();
    m = sh.top[n][0];
#pragma unroll
    for (int i = 0; i < 4; i++) rm[i] = m;
#pragma unroll
    for (int j = 0; j < 8; j++) cm[j] = m;
  } else {
    if constexpr (ROWS) {
#pragma unroll
      for (int i = 0; i < 4; i++) rm[i] = max16(rm[i]);
    }
    if constexpr (COLS) {
#pragma unroll
      for (int j = 0; j < 8; j++) {
        cm[j] = max(cm[j], (uint32_t)__shfl_xor((int)cm[j], 16));
        cm[j] = max(cm[j], (uint32_t)__shfl_xor((int)cm[j], 32));
      }
      if ((t & 63) < 16) {
#pragma unroll
        for (int j = 0; j < 8; j++) atomicMax(&sh.top[n][8 * cg + j], cm[j]);
      }
    }
  }
  if constexpr (ROWS) {
    const int64_t lane = WHOLE ? (int64_t)((uint32_t)(4 * rg) * (uint32_t)rows.ld + 8 * cg) : 4 * rg * rows.ld + 8 * cg;
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint32_t byte = fp8_scale_byte(rm[i]);
      const u32v2 o = fp8_encode8(v[i], byte);
      if (WHOLE || r0 + 4 * rg + i < R) *(u32v2*)(rows.codes + ((r0 + i) * rows.ld + c0) + lane) = o;
      if (cg == i) mine = byte;
    }
    const int64_t row = r0 + 4 * rg + cg;
    if (cg < 4 && (WHOLE || row < R)) rows.scales[(c0 / FP8_BLOCK) * rows.scale_ld + row] = (uint8_t)mine;
  }
  if constexpr (COLS) {
    if constexpr (!SQUARE) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; j++) cm[j] = sh.top[n][8 * cg + j];
    }
#pragma unroll
    for (int j = 0; j < 8; j++) {
      *(uint32_t*)(sh.turn + turn_at(8 * cg + j, rg >> 1) + 4 * (rg & 1)) =
          fp8_encode4(v[0][j], v[1][j], v[2][j], v[3][j], fp8_scale_byte(cm[j]));
    }
    if (rg == 0) {
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (WHOLE || c0 + 8 * cg + j < CR)
          cols.scales[(r0 / FP8_BLOCK) * cols.scale_ld + c0 + 8 * cg + j] = (uint8_t)fp8_scale_byte(cm[j]);
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 2; m++) {
      const int c = (t >> 3) + 64 * m, q = t & 7;
      const u32v4 o = *(const u32v4*)(sh.turn + turn_at(c, 2 * q));
      if (WHOLE || c0 + c < CR) *(u32v4*)(cols.codes + (c0 + c) * cols.ld + r0 + 16 * q) = o;
    }
  }
}

// This thread's part of the tile of x [R, C] at (r0, c0); past R and C zeros.
// Whole tiles take a uniform base per row and one 32-bit lane offset, and no
// checks; RAGGED = false: C is a multiple of 8.
template <bool WHOLE, bool RAGGED>
__device__ __forceinline__ void load_tile(const uint16_t* x, int64_t ld, int64_t r0, int64_t c0, int64_t R, int64_t C,
                                          u32v4 (&p)[4]) {
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
  if constexpr (WHOLE) {
    const uint32_t lane = (uint32_t)(4 * rg) * (uint32_t)ld + 8 * cg;
#pragma unroll
    for (int i = 0; i < 4; i++) p[i] = *(const u32v4_any*)(x + ((r0 + i) * ld + c0) + lane);
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int64_t row = r0 + 4 * rg + i;
      p[i] = (u32v4){0u, 0u, 0u, 0u};
      if (row < R) p[i] = fetch8<RAGGED>(x + row * ld, c0 + 8 * cg, C);
    }
#pragma unroll
    for (int i = 0; i < 4; i++) settle8<RAGGED>(p[i], c0 + 8 * cg, r0 + 4 * rg + i < R ? C : 0);
  }
}
constexpr int64_t TILE_LD_MAX = (int64_t)1 << 23;   // row strides that a 32-bit lane offset reaches over

// Tile of x [R, C]: out along rows (COLS false) or transposed.
template <bool COLS, bool SQUARE, bool WHOLE, bool RAGGED>
__device__ __forceinline__ void tile_body(TileShared& sh, const uint16_t* x, int64_t R, int64_t C, int64_t ldx,
                                          int64_t r0, int64_t c0, const Fp8Out& out) {
  u32v4 p[4];
  load_tile<WHOLE, RAGGED>(x, ldx, r0, c0, R, C, p);
  float v[4][8];
#pragma unroll
  for (int i = 0; i < 4; i++) bf16x8_to_f32(p[i], v[i]);
  clear_tops(sh);
  quantize_tile<!COLS, COLS, SQUARE, WHOLE>(sh, 0, v, r0, c0, out, R, out, C);
}
template <bool COLS, bool SQUARE, bool RAGGED>
__global__ void __launch_bounds__(TILE_THREADS) fp8_tile_kernel(const uint16_t* __restrict__ x, int64_t R, int64_t C,
                                                                int64_t ldx, int64_t tiles_c, Fp8Out out) {
  __shared__ __attribute__((aligned(16))) TileShared sh;
  const int64_t c0 = (blockIdx.x % tiles_c) * 128, r0 = (blockIdx.x / tiles_c) * 128;
  if (r0 + 128 <= R && c0 + 128 <= C && max(ldx, out.ld) <= TILE_LD_MAX)
    tile_body<COLS, SQUARE, true, RAGGED>(sh, x, R, C, ldx, r0, c0, out);
  else
    tile_body<COLS, SQUARE, false, RAGGED>(sh, x, R, C, ldx, r0, c0, out);
}

// ---------------------------------------------------------------------------
// Gradient of h = act(g) * u for dh: dg = dh u act'(g), du = dh act(g), each
// quantized along its rows (for dx = dg Wg + du Wu) and along its columns (for
// dWg = dg^T x, dWu = du^T x), and h itself along its columns when `ht` is
// wanted (for the down projection's weight).  Columns n .. np - 1 of both
// halves (np: n rounded up to 128) are written as zeros.
//
// One pass instead of five: the three inputs are read once and each product is
// rounded once from binary32, in both orientations.  10 bytes an element (11 with
// `ht`): 8192 x 11008 silu takes 175 us (5.1 TB/s), 12608 x 2048 gelu 61 us (4.2
// TB/s: 1584 workgroups end in a part-filled round, and gelu's evaluation is the
// longest).
// ---------------------------------------------------------------------------
template <int ACT, bool WHOLE, bool RAGGED>
__device__ __forceinline__ void gated_grad_body(TileShared& sh, const GatedGradArgs& a, int64_t r0, int64_t c0) {
  u32v4 pg[4], pu[4], pd[4];
  load_tile<WHOLE, RAGGED>(a.g, a.ldg, r0, c0, a.T, a.n, pg);
  load_tile<WHOLE, RAGGED>(a.u, a.ldu, r0, c0, a.T, a.n, pu);
  load_tile<WHOLE, RAGGED>(a.dh, a.ldd, r0, c0, a.T, a.n, pd);
  Fp8Out up_rows = a.dgu, up_cols = a.dgut;
  up_rows.codes += a.np;
  up_rows.scales += (a.np / FP8_BLOCK) * up_rows.scale_ld;
  up_cols.codes += a.np * up_cols.ld;
  up_cols.scales += a.np;
  // both gradients from one evaluation of the activation, which costs more than
  // all else here; pinned, or the compiler moves the second product to its use
  // and keeps its factors instead
  float v[4][8], vu[4][8];
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const float g = bf16_of(pg[i][j >> 1], j & 1), u = bf16_of(pu[i][j >> 1], j & 1);
      const float d = bf16_of(pd[i][j >> 1], j & 1);
      float h, dact;
      act_grad<ACT>(g, h, dact);
      v[i][j] = d * u * dact;
      vu[i][j] = d * h;
      asm volatile("" : "+v"(v[i][j]), "+v"(vu[i][j]));
    }
  clear_tops(sh);
  quantize_tile<true, true, false, WHOLE>(sh, 0, v, r0, c0, a.dgu, a.T, a.dgut, a.np);
  __syncthreads();   // LDS is free for the next tile
  quantize_tile<true, true, false, WHOLE>(sh, 1, vu, r0, c0, up_rows, a.T, up_cols, a.np);
  if (a.ht.codes) {
    // (from the caches: kept in registers they would cost every call)
    load_tile<WHOLE, RAGGED>(a.g, a.ldg, r0, c0, a.T, a.n, pg);
    load_tile<WHOLE, RAGGED>(a.u, a.ldu, r0, c0, a.T, a.n, pu);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      float g[8], u[8];
      bf16x8_to_f32(pg[i], g);
      bf16x8_to_f32(pu[i], u);
#pragma unroll
      for (int j = 0; j < 8; j++) v[i][j] = act_value<ACT>(g[j]) * u[j];
    }
    __syncthreads();
    quantize_tile<false, true, false, WHOLE>(sh, 2, v, r0, c0, a.ht, a.T, a.ht, a.n);
  }
}

template <int ACT, bool RAGGED>
__global__ void __launch_bounds__(TILE_THREADS, 4) fp8_gated_grad_kernel(GatedGradArgs a) {
  __shared__ __attribute__((aligned(16))) TileShared sh;
  const int64_t tiles_c = a.np / 128;
  const int64_t c0 = (blockIdx.x % tiles_c) * 128, r0 = (blockIdx.x / tiles_c) * 128;
  const int64_t ld = max(max(a.ldg, a.ldu), a.ldd);
  if (r0 + 128 <= a.T && c0 + 128 <= a.n && ld <= TILE_LD_MAX) gated_grad_body<ACT, true, RAGGED>(sh, a, r0, c0);
  else gated_grad_body<ACT, false, RAGGED>(sh, a, r0, c0);
}

// ---------------------------------------------------------------------------
// FP8 to binary32 (validation)
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) fp8_dequantize_kernel(const uint8_t* __restrict__ codes, int64_t ld,
                                                             const uint8_t* __restrict__ scales, int64_t scale_ld,
                                                             int64_t rows, int64_t k, float* __restrict__ y,
                                                             int64_t ldy) {
  const int64_t total = rows * k, stride = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += stride) {
    const int64_t r = i / k, c = i - r * k;
    const float v = __builtin_amdgcn_cvt_f32_fp8((int)codes[r * ld + c], 0);
    y[r * ldy + c] = v * e8m0_value(scales[(c / FP8_BLOCK) * scale_ld + r]);
  }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
template <bool RAGGED>
static void launch_tile(const uint16_t* x, int64_t R, int64_t C, int64_t ldx, int axis, int block_rows, int64_t tc,
                        const Fp8Out& out, int64_t n, hipStream_t s) {
  const dim3 grid((unsigned)n), wg(TILE_THREADS);
  if (axis == 1)
    hipLaunchKernelGGL((fp8_tile_kernel<false, true, RAGGED>), grid, wg, 0, s, x, R, C, ldx, tc, out);
  else if (block_rows == 128)
    hipLaunchKernelGGL((fp8_tile_kernel<true, true, RAGGED>), grid, wg, 0, s, x, R, C, ldx, tc, out);
  else
    hipLaunchKernelGGL((fp8_tile_kernel<true, false, RAGGED>), grid, wg, 0, s, x, R, C, ldx, tc, out);
}

// f(first row, rows, first column, columns) for parts of [R, C] of which each
// takes one launch: workgroups of `threads` (at most 512) for tr x tc elements
// (at least 16 x 128).  Parts start at multiples of 128.
template <typename F>
static void in_parts(int64_t R, int64_t C, int64_t tr, int64_t tc, int64_t threads, F f) {
  constexpr int64_t COLS = (int64_t)1 << 26;
  const int64_t most = FP8_LAUNCH_THREADS / threads;
  for (int64_t c0 = 0; c0 < C; c0 += COLS) {
    const int64_t cols = C - c0 < COLS ? C - c0 : COLS;
    const int64_t rows = most / ((cols + tc - 1) / tc) * tr / 128 * 128;
    for (int64_t r0 = 0; r0 < R; r0 += rows) f(r0, R - r0 < rows ? R - r0 : rows, c0, cols);
  }
}

hipError_t launch_fp8_quantize(const uint16_t* x, int64_t R, int64_t C, int64_t ldx, int axis, int block_rows,
                               const Fp8Out& out, hipStream_t s) {
  auto part = [&](int64_t r0, int64_t c0) {
    return axis ? Fp8Out{out.codes + r0 * out.ld + c0, out.scales + c0 / FP8_BLOCK * out.scale_ld + r0, out.ld, out.scale_ld}
                : Fp8Out{out.codes + c0 * out.ld + r0, out.scales + r0 / FP8_BLOCK * out.scale_ld + c0, out.ld, out.scale_ld};
  };
  if (axis == 1 && block_rows == 1) {
    in_parts(R, C, 16, ROWS_NB * FP8_BLOCK, 256, [&](int64_t r0, int64_t rows, int64_t c0, int64_t cols) {
      const int64_t blocks = (cols + 127) / 128, groups = (blocks + ROWS_NB - 1) / ROWS_NB;
      const int64_t n = groups * ((rows + 15) / 16);
      hipLaunchKernelGGL(fp8_rows_kernel, dim3((unsigned)n), dim3(256), 0, s, x + r0 * ldx + c0, rows, cols, ldx, blocks,
                         groups, part(r0, c0));
    });
    return hipGetLastError();
  }
  in_parts(R, C, 128, 128, TILE_THREADS, [&](int64_t r0, int64_t rows, int64_t c0, int64_t cols) {
    const int64_t tc = (cols + 127) / 128, n = tc * ((rows + 127) / 128);
    const uint16_t* p = x + r0 * ldx + c0;
    if (C % 8) launch_tile<true>(p, rows, cols, ldx, axis, block_rows, tc, part(r0, c0), n, s);
    else launch_tile<false>(p, rows, cols, ldx, axis, block_rows, tc, part(r0, c0), n, s);
  });
  return hipGetLastError();
}

template <int ACT>
static void launch_grad(const GatedGradArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.np / 128) * ((a.T + 127) / 128))), wg(TILE_THREADS);
  if (a.n % 8) hipLaunchKernelGGL((fp8_gated_grad_kernel<ACT, true>), grid, wg, 0, s, a);
  else hipLaunchKernelGGL((fp8_gated_grad_kernel<ACT, false>), grid, wg, 0, s, a);
}

hipError_t launch_fp8_gated_grad(int act, const GatedGradArgs& a, hipStream_t s) {
  if (act == ACT_SILU) launch_grad<ACT_SILU>(a, s);
  else if (act == ACT_GELU) launch_grad<ACT_GELU>(a, s);
  else launch_grad<ACT_GELU_TANH>(a, s);
  return hipGetLastError();
}

hipError_t launch_fp8_dequantize(const uint8_t* codes, int64_t ld, const uint8_t* scales, int64_t scale_ld,
                                 int64_t rows, int64_t k, float* y, int64_t ldy, hipStream_t s) {
  int64_t n = (rows * k + 255) / 256;
  if (n > 65536) n = 65536;
  hipLaunchKernelGGL(fp8_dequantize_kernel, dim3((unsigned)n), dim3(256), 0, s, codes, ld, scales, scale_ld, rows, k,
                     y, ldy);
  return hipGetLastError();
}

}  // namespace mxfp4
