// fp8_gemm.hip -- products of block-128 FP8 operands, C[M,N] = A[M,K] B[N,K]^T,
// and the gated block's h = act(x Wg^T) * (x Wu^T), for gfx950.
//
// Both run on the block-scaled matrix instructions with E4M3 operands, whose
// E8M0 scale per 32 contraction elements of a row is given the byte of the
// 128-block that they lie in: scaling costs no vector instruction and the
// accumulators stay in binary32 registers over the whole contraction.  Within a
// 128-block the order of the contraction is free as long as A and B agree.
//
// What the instruction adds to them is less exact than binary32: it takes eight
// consecutive products at a time, each cut toward zero to a multiple of
// 2^-13 of the largest one's power of two.  As measured, products of either
// sign leave a sum off by 1.5e-5 of the root of the sum of their squares; products of
// one sign leave it 2.5e-6 short.  Taken for its speed: a bf16 output's
// rounding is 100 times the first and 800 times the second.
//
// Bound by the matrix pipe and the clock that its power leaves: 4096 x 14336 x
// 8192 takes 328 - 368 us from card to card (2.6 - 2.9 PF, 316 us being what a
// library's E4M3 product with one scale per tensor takes), the pipe busy for 79 %
// of the cycles at 1.63 GHz (53 % at 1.92 GHz before the half-stage pipeline).
//
// Wide tiles: 256 x 256 outputs per workgroup of four waves (128 x 128 per
// wave: 4 x 4 tiles of 32x32x64, 256 accumulators per lane).  A stage is one
// 128-block: 128 bytes, one whole line, of every operand row, and one scale
// byte per row.  Two stages (64.5 KB each) alternate in LDS, filled by
// buffer->LDS loads, half a stage at a time (see fp8_mainloop).  Codes sit in
// LDS as 16-byte chunks at chunk ^ (row / 2 & 7), so that 16 consecutive rows at
// one chunk fall on different banks.  The gated kernel is the same tile with 128
// rows of the gate's weight and the 128 rows of the up projection's that belong
// to them as its B rows: each wave then holds both factors of its outputs.
// Few rows of A take the decode kernel (see decode_tiles): 16 columns per
// workgroup, whose waves split the contraction.
#include <type_traits>

#include "fp8_device.h"
#include "fp8_internal.h"

namespace mxfp4 {

constexpr uint32_t kRsrcWord3 = 0x00020000u;      // raw buffer, 32-bit data format
constexpr uint32_t kOutOfRange = 0x80000000u;     // a buffer offset past every operand
constexpr int F8_OPND = 256 * 128;                // one operand's codes per stage: 32 KB
constexpr int F8_SCALE = 2 * F8_OPND;             // scale bytes: A's 256, then B's 256
constexpr int F8_STAGE = 2 * F8_OPND + 512;
constexpr int F8_LDS = 2 * F8_STAGE;
constexpr int F8_ROW_GU = 1184, F8_ROW_H = 608;   // LDS rows of the gated epilogue (store_gated)
constexpr int F8_LDS_GATED = 2 * 2 * 32 * F8_ROW_GU;
static_assert(F8_LDS_GATED >= F8_LDS && F8_LDS_GATED <= 160 * 1024 && 2 * 2 * 32 * F8_ROW_H <= F8_LDS, "LDS");

// what a kernel writes
constexpr int OUT_F32 = FP8_F32, OUT_BF16 = FP8_BF16, OUT_PART = 2, OUT_GATED = 3, OUT_GATED_TRAIN = 4;


struct Fp8Args {
  Fp8In a, b;
  int64_t M, N;             // outputs (gated: N = np)
  int kb;                   // contraction blocks of 128
  int splits;
  int ntm, ntn, rem;        // 256-row tiles; the last `rem` of them run as two 128-row halves
  int tails;                // tiles of a last row of at most 128: a first half each
  void* C;
  int64_t ldc, split_stride;
  // gated
  int64_t n, np;
  Fp8Out q;
  uint16_t *h, *g, *u;
  float* hf;                // decode: binary32 result [M, np] for the quantizing pass
  int64_t ldh, ldgu;
};

template <int VM, int LGKM>
__device__ __forceinline__ void wait_cnt() {
  static_assert(VM < 64 && LGKM < 16, "counter range");
  __builtin_amdgcn_s_waitcnt((VM & 0xF) | ((VM >> 4) << 14) | (0x7 << 4) | (LGKM << 8));
}
__device__ __forceinline__ void block_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
// LDS operations of this wave done
__device__ __forceinline__ void lds_done() {
  asm volatile("" ::: "memory");
  wait_cnt<63, 0>();
  __builtin_amdgcn_wave_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const uint8_t* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, kRsrcWord3);
}

// ---------------------------------------------------------------------------
// Wide tiles
// ---------------------------------------------------------------------------
// This wave's share of an operand: ROWS rows from r0, 8 per load.  The resource
// ends with the operand's last row, so rows past it read as zeros (their
// products are never stored).
struct Share {
  __amdgpu_buffer_rsrc_t codes;
};
template <int ROWS>
__device__ __forceinline__ Share make_share(const Fp8In& o, int64_t r0, int kb) {
  int64_t rows = o.rows - r0;
  rows = rows < 0 ? 0 : rows > ROWS ? ROWS : rows;
  // (rows = 0: nothing is in range)
  return Share{resource(o.codes + (rows ? r0 : 0) * o.ld, rows ? (rows - 1) * o.ld + (int64_t)kb * FP8_BLOCK : 0)};
}

// Lane offsets of loads 0 and 1 of a share that starts at a multiple of 16
// rows (load j adds (j >> 1) steps of 16 rows): lane l fills position l & 7 of
// row 8 j + l / 8 with chunk (l & 7) ^ (row / 2 & 7).
struct Lanes {
  uint32_t off[2], rows16;
};
__device__ __forceinline__ Lanes make_lanes(int64_t ld, int l) {
  Lanes s;
#pragma unroll
  for (int j = 0; j < 2; j++) {
    const int r = 8 * j + (l >> 3);
    s.off[j] = (uint32_t)(r * ld) + (uint32_t)(((l & 7) ^ ((r >> 1) & 7)) << 4);
  }
  s.rows16 = (uint32_t)(16 * ld);
  return s;
}

template <int L>
__device__ __forceinline__ void issue_share(const Share& s, const Lanes& n, uint8_t* lds, int kt) {
#pragma unroll
  for (int j = 0; j < L; j++)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(s.codes, (lds_void*)(lds + 8 * j * 128), 16,
                                             n.off[j & 1] + (uint32_t)(j >> 1) * n.rows16, kt * 128, 0, 0);
}

// A half of a wave's rows of an operand: T 32-row tiles, whole 128-blocks (both
// halves of the contraction).
template <int T>
struct Frag {
  v8i k[T][2];
};

// A quarter's NM MFMAs: its ND LDS reads go ahead of the first half of them, its
// NV loads between those of the second half.  (Both spread over all of the
// MFMAs, so that loads fill LDS while fragments are read from it, took 384 us
// on 4096 x 14336 x 8192; the loads first 362 us; this order 338 us.)
template <int NM, int ND, int NV>
__device__ __forceinline__ void spread() {
  constexpr int D = 2 * ((ND + NM - 1) / NM);
#pragma unroll
  for (int q = 0; q < NM; q++) {
    if (q * D < ND) __builtin_amdgcn_sched_group_barrier(0x100, D, 0);                        // LDS reads
    if (q >= NM / 2 && q - NM / 2 < NV) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);    // a buffer->LDS load
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                                        // an MFMA
  }
  __builtin_amdgcn_sched_barrier(0);
}

// One output tile of 64 TM rows and 256 B rows, contraction blocks kt0 ..
// kt1 - 1.  A wave's rows of A and of B come in halves (A0, A1; B0, B1; gated:
// B0 is the gate's weight, B1 the up projection's), and the quarters of its
// outputs are taken in an order in which each needs one new half:
//   step 0   A0 Bx, reading By        A0 By, reading A1
//   step 1   A1 By, reading A0'       A1 Bx, reading By'      (' : of stage a + 1)
// with x = 0 and 1 in turn, so four halves of registers hold everything.  Step
// 0 loads stage a + 2's A0 and Bx, which have been read in the step before, and
// step 1 its By and A1.  A barrier ends each step: what the next step reads has
// then been loaded by every wave, and what it loads over has been read by every
// wave.  A load thus has two to three steps (about 1000 cycles each) to land.
// Loads past the end fetch the last block again: they land in buffers that are
// not read any more.  (Whole stages in turn, with one barrier per stage: 410 us on
// 4096 x 14336 x 8192, this 338 us on the same card.)
template <int TM, bool GATED>
__device__ __forceinline__ void fp8_mainloop(const Fp8Args& p, uint8_t* smem, int64_t m0, int64_t n0, int kt0, int kt1,
                                             v16f (&acc)[TM][4]) {
  constexpr int TH = TM / 2;                      // 32-row tiles of half a wave's A rows
  constexpr int LA = 2 * TH, LB = 4;              // loads per wave of half of A (16 TH rows) and half of B (32 rows)
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = threadIdx.x & 63, h = l >> 5;
  const int wm = w >> 1, wn = w & 1;
  // LDS rows of B: wave column wn's half 0 starts at BW wn, its half 1 BH further
  constexpr int BW = GATED ? 64 : 128, BH = GATED ? 128 : 64;
  constexpr int AW = 32 * TM, AH = 32 * TH;
  const int ra0 = wm * AW + (l & 31), rb0 = wn * BW + (l & 31);
  int pos[4];
#pragma unroll
  for (int c = 0; c < 4; c++) pos[c] = ((2 * c + h) ^ ((l >> 1) & 7)) << 4;
#pragma unroll
  for (int i = 0; i < TM; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) acc[i][j] = (v16f){};
  if (kt1 <= kt0) return;

  // this wave loads half of the rows of each half of one wave row's A and one wave column's B
  const int la0 = (w >> 1) * AW + (w & 1) * (AH / 2), lb0 = (w >> 1) * BW + (w & 1) * 32;
  const Share sa0 = make_share<AH / 2>(p.a, m0 + la0, p.kb), sa1 = make_share<AH / 2>(p.a, m0 + la0 + AH, p.kb);
  const Share sb0 = make_share<32>(p.b, n0 + lb0, p.kb);
  const Share sb1 = make_share<32>(p.b, n0 + lb0 + (GATED ? p.np : BH), p.kb);
  const Lanes la = make_lanes(p.a.ld, l), lb = make_lanes(p.b.ld, l);
  // scale bytes: even waves bring A's 256 rows, odd waves B's, 4 per lane.
  // Rows past the matrix read the next line's bytes or, past the last line's
  // last row, zeros.
  const Fp8In& so = (w & 1) ? p.b : p.a;
  const int64_t s0 = (w & 1) ? n0 : m0;
  const __amdgpu_buffer_rsrc_t sres = resource(so.scales + s0, fp8_scale_extent(p.kb, so.scale_ld, so.rows, s0, 4));
  const uint32_t soff = 4 * l + ((GATED && (w & 1) && l >= 32) ? (uint32_t)(p.np - 128) : 0u);
  const uint32_t sld = (uint32_t)so.scale_ld;
  auto stage = [&](int a) { return smem + (a & 1) * F8_STAGE; };
  auto clamp = [&](int a) { return a < kt1 ? a : kt1 - 1; };
  auto issue_a = [&](int a, const Share& s, int half) {
    issue_share<LA>(s, la, stage(a) + (la0 + half * AH) * 128, clamp(a));
  };
  auto issue_b = [&](int a, const Share& s, int half) {
    issue_share<LB>(s, lb, stage(a) + F8_OPND + (lb0 + half * BH) * 128, clamp(a));
  };
  auto issue_scales = [&](int a) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(sres, (lds_void*)(stage(a) + F8_SCALE + 256 * (w & 1)), 4,
                                             soff + (uint32_t)clamp(a) * sld, 0, 0, 0);
  };
  auto row = [&](const uint8_t* r, v8i (&k)[2]) {
#pragma unroll
    for (int s = 0; s < 2; s++)
      k[s] = __builtin_shufflevector(*(const v4i*)(r + pos[2 * s]), *(const v4i*)(r + pos[2 * s + 1]), 0, 1, 2, 3, 4, 5,
                                     6, 7);
  };
  auto read_a = [&](int a, int half, Frag<TH>& f) {
#pragma unroll
    for (int t = 0; t < TH; t++) row(stage(a) + (ra0 + half * AH + 32 * t) * 128, f.k[t]);
  };
  auto read_b = [&](int a, int half, Frag<2>& f) {
#pragma unroll
    for (int t = 0; t < 2; t++) row(stage(a) + F8_OPND + (rb0 + half * BH + 32 * t) * 128, f.k[t]);
  };
  auto scales = [&](int a, int (&ea)[TM], int (&eb)[4]) {
    const uint8_t* s = stage(a) + F8_SCALE;
#pragma unroll
    for (int t = 0; t < TM; t++) ea[t] = s[ra0 + 32 * t];
#pragma unroll
    for (int t = 0; t < 4; t++) eb[t] = s[256 + rb0 + (t >> 1) * BH + 32 * (t & 1)];
  };
  Frag<TH> fa[2];
  Frag<2> fb[2];
  int ea[TM], eb[4];
  auto quarter = [&](int ha, int hb) {
#pragma unroll
    for (int s = 0; s < 2; s++)
#pragma unroll
      for (int i = 0; i < TH; i++)
#pragma unroll
        for (int j = 0; j < 2; j++) {
          v16f& c = acc[ha * TH + i][2 * hb + j];
          c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[ha].k[i][s], fb[hb].k[j][s], c, 0, 0, 0,
                                                              ea[ha * TH + i], 0, eb[2 * hb + j]);
        }
  };
  constexpr int NM = 4 * TH;                      // MFMAs of a quarter
  constexpr int RA = 4 * TH, RB = 8;              // LDS reads of half of A, of half of B
  constexpr int ND = 2 * (LA + LB) + 1;           // loads of one stage

  issue_a(kt0, sa0, 0);
  issue_b(kt0, sb0, 0);
  issue_scales(kt0);
  issue_b(kt0, sb1, 1);
  issue_a(kt0, sa1, 1);
  issue_a(kt0 + 1, sa0, 0);
  issue_b(kt0 + 1, sb1, 1);
  issue_scales(kt0 + 1);
  issue_b(kt0 + 1, sb0, 0);
  issue_a(kt0 + 1, sa1, 1);
  wait_cnt<LA + LB + ND, 15>();
  block_barrier();
  scales(kt0, ea, eb);
  read_a(kt0, 0, fa[0]);
  read_b(kt0, 0, fb[0]);
  wait_cnt<ND, 0>();
  block_barrier();
  auto one = [&](int a, auto xc) {
    constexpr int X = decltype(xc)::value, Y = X ^ 1;
    const Share& sx = X ? sb1 : sb0;
    const Share& sy = X ? sb0 : sb1;
    read_b(a, Y, fb[Y]);
    issue_a(a + 2, sa0, 0);
    issue_scales(a + 2);
    quarter(0, X);
    spread<NM, RB, LA + 1>();
    read_a(a, 1, fa[1]);
    issue_b(a + 2, sx, X);
    quarter(0, Y);
    spread<NM, RA, LB>();
    wait_cnt<ND, 0>();
    block_barrier();
    read_a(a + 1, 0, fa[0]);
    issue_b(a + 2, sy, Y);
    quarter(1, Y);
    spread<NM, RA, LB>();
    int ean[TM], ebn[4];
    const int live = a + 1 < kt1 ? 255 : 0;
    read_b(a + 1, Y, fb[Y]);
    scales(a + 1, ean, ebn);
    issue_a(a + 2, sa1, 1);
    quarter(1, X);
    spread<NM, RB + TM + 4, LA>();
    wait_cnt<ND, 0>();
    block_barrier();
#pragma unroll
    for (int t = 0; t < TM; t++) ea[t] = ean[t] & live;
#pragma unroll
    for (int t = 0; t < 4; t++) eb[t] = ebn[t] & live;
  };
  // (stages come in pairs; one past the end multiplies with scales of zero)
  for (int a = kt0; a < kt1; a += 2) {
    one(a, std::integral_constant<int, 0>{});
    one(a + 1, std::integral_constant<int, 1>{});
  }
  wait_cnt<0, 0>();   // nothing may still write LDS when the tile's LDS is used again
  block_barrier();
}

// In an accumulator lane l holds column l % 32 and rows 8 (v / 4) + 4 (l / 32)
// + v % 4, v = 0 .. 15.
__device__ __forceinline__ int acc_row(int v, int l) { return 8 * (v >> 2) + 4 * (l >> 5) + (v & 3); }

// Stores a wave's 32 TM x 128 outputs through its own slice of LDS, 32 rows at
// a time, so that each lane stores 16 bytes and a wave whole row segments.
// The split sums are read again right after, so they are stored plainly; C is
// not, and is stored past the caches.
template <int TM, int OUT>
__device__ __forceinline__ void store_tile(const Fp8Args& p, uint8_t* smem, void* C, int64_t mb, int64_t nb,
                                           const v16f (&acc)[TM][4]) {
  constexpr int RB = 512 + 32;                     // LDS row: 128 floats, padded against bank conflicts
  constexpr int V = OUT == OUT_BF16 ? 8 : 4;       // outputs per lane and store
  constexpr int LPR = 128 / V;                     // lanes per row
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
  uint8_t* slab = smem + w * 32 * RB;
#pragma unroll
  for (int tm = 0; tm < TM; tm++) {
#pragma unroll
    for (int v = 0; v < 16; v++)
#pragma unroll
      for (int j = 0; j < 4; j++) *(float*)(slab + acc_row(v, l) * RB + 4 * (32 * j + (l & 31))) = acc[tm][j][v];
    lds_done();
#pragma unroll
    for (int i = 0; i < 32 * LPR / 64; i++) {
      const int r = i * (64 / LPR) + l / LPR, c = V * (l % LPR);
      float o[V];
#pragma unroll
      for (int q = 0; q < V / 4; q++) {
        const v4f x = *(const v4f*)(slab + r * RB + 4 * c + 16 * q);
#pragma unroll
        for (int e = 0; e < 4; e++) o[4 * q + e] = x[e];
      }
      const int64_t row = mb + 32 * tm + r, col = nb + c;
      if (row >= p.M) continue;
      if constexpr (OUT == OUT_BF16) {
        uint16_t* dst = (uint16_t*)C + row * p.ldc;
        const u32v4 b = f32_to_bf16x8(o);
        if (col + 8 <= p.N) __builtin_nontemporal_store(b, (u32v4_any*)(dst + col));
        else store8(dst, col, p.N, b);
      } else {
        float* dst = (float*)C + row * p.ldc + col;
        const v4f x = {o[0], o[1], o[2], o[3]};
        if (col + 4 <= p.N) {
          if (OUT == OUT_PART) *(v4f_any*)dst = x;
          else __builtin_nontemporal_store(x, (v4f_any*)dst);
        } else {
#pragma unroll
          for (int e = 0; e < 4; e++)
            if (col + e < p.N) dst[e] = o[e];
        }
      }
    }
    lds_done();   // the slice is read before the next rows overwrite it
  }
}

// The gated epilogue.  32 rows at a time go through LDS, where the two waves of a
// row meet, and come back with 16 lanes holding a row's 128 outputs, eight
// consecutive ones each: one FP8 block (its maximum is four lane rotations
// away) and 16-byte stores of whole bf16 segments.  Without a backward pass h =
// act(g) u is what goes through; with one, g and u do, and h is computed on the
// way out.  While rows are read back and stored, the next 32 go into the
// other half of the space: one barrier per 32 rows.
//
// It has to move 7 bytes an output with a backward pass (16384 x 4096 x 11008:
// 1183 us; 1396 us when each lane stored its own accumulators in two-byte pieces).
//
// LDS row: float column x sits in 16-byte chunk x / 4; even chunks come
// first, odd ones 320 bytes on, so that both a wave's writes (32 columns of
// rows r and r + 4) and its reads (every other chunk of a row) fall on different
// banks; u follows g after 592 bytes.
template <int TM, int ACT, bool TRAIN>
__device__ __forceinline__ void store_gated(const Fp8Args& p, uint8_t* smem, int64_t m0, int64_t n0,
                                            const v16f (&acc)[TM][4]) {
  constexpr int RB = TRAIN ? F8_ROW_GU : F8_ROW_H, U = 592, ODD = 320;
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6, wm = w >> 1, wn = w & 1;
  uint8_t* const half = smem + wm * 32 * RB;
  // this lane's columns 64 wn + 32 j + l % 32 (j: 8 chunks, 64 bytes of either parity, apart) and rows
  uint8_t* const put_at = half + 4 * (l >> 5) * RB + (64 * wn + (l & 31)) / 8 * 16 + ((l >> 2) & 1) * ODD + 4 * (l & 3);
  auto put = [&](int tm) {
#pragma unroll
    for (int v = 0; v < 16; v++)
#pragma unroll
      for (int j = 0; j < 2; j++) {
        uint8_t* at = put_at + (tm & 1) * 64 * RB + acc_row(v, 0) * RB + 64 * j;
        if constexpr (TRAIN) {
          *(float*)at = acc[tm][j][v];
          *(float*)(at + U) = acc[tm][j + 2][v];
        } else {
          *(float*)at = act_value<ACT>(acc[tm][j][v]) * acc[tm][j + 2][v];
        }
      }
  };
  // read back: rows 16 wn + 4 i + l / 16, columns 8 (l % 16) ..
  const int r0 = 16 * wn + (l >> 4), c = 8 * (l & 15);
  const uint8_t* const get_at = half + r0 * RB + 16 * (l & 15);
  int64_t row = m0 + 32 * TM * wm + r0;
  const int64_t col = n0 + c;
  uint8_t* qp = p.q.codes + row * p.q.ld + col;
  uint8_t* sp = p.q.scales + (n0 / FP8_BLOCK) * p.q.scale_ld + row;
  uint16_t *hp = p.h + row * p.ldh, *gp = p.g + row * p.ldgu, *up = p.u + row * p.ldgu;
  auto get = [&](const uint8_t* at, float (&o)[8]) {
#pragma unroll
    for (int q = 0; q < 2; q++) {
      const v4f x = *(const v4f*)(at + q * ODD);
#pragma unroll
      for (int e = 0; e < 4; e++) o[4 * q + e] = x[e];
    }
  };
  auto store = [&](uint16_t* dst, const float (&o)[8]) {
    const u32v4 b = f32_to_bf16x8(o);
    if (col + 8 <= p.n) __builtin_nontemporal_store(b, (u32v4_any*)(dst + col));
    else store8(dst, col, p.n, b);
  };
  put(0);
  wait_cnt<63, 0>();
  block_barrier();
#pragma unroll
  for (int tm = 0; tm < TM; tm++) {
    if (tm + 1 < TM) put(tm + 1);
#pragma unroll 2
    for (int i = 0; i < 4; i++) {
      const uint8_t* at = get_at + (tm & 1) * 64 * RB + 4 * i * RB;
      float o[8];
      get(at, o);
      if constexpr (TRAIN) {
        float u[8];
        get(at + U, u);
        if (row < p.M) {
          store(gp, o);
          store(up, u);
        }
#pragma unroll
        for (int e = 0; e < 8; e++) o[e] = act_value<ACT>(o[e]) * u[e];
      }
      if (n0 + 128 > p.n) {   // (the columns that pad the weights may hold anything)
#pragma unroll
        for (int e = 0; e < 8; e++) o[e] = col + e < p.n ? o[e] : 0.0f;
      }
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; e++) m = max(m, abs_bits(o[e]));
      const uint32_t byte = fp8_scale_byte(max16(m));
      if (row < p.M) {
        if (p.q.codes) {
          *(u32v2*)qp = fp8_encode8(o, byte);
          if ((l & 15) == 0) *sp = (uint8_t)byte;
        }
        if (p.h) store8(hp, col, p.n, f32_to_bf16x8(o));
      }
      const int64_t step = i < 3 ? 4 : 32 - 12;
      row += step;
      qp += step * p.q.ld;
      sp += step;
      hp += step * p.ldh;
      gp += step * p.ldgu;
      up += step * p.ldgu;
    }
    wait_cnt<63, 0>();
    block_barrier();
  }
}

// Work items: [R first halves] [T - R full tiles] [R second halves] [tails] over T
// tiles, R of them cut into two 128-row halves (see lay_tiles), so that every
// compute unit ends at about the same time.  When at most 128 rows are
// left for the last row of tiles, those are halves without a second one.  Consecutive ids go to
// consecutive XCDs: the ids of one XCD are gathered into a contiguous run of
// tiles, walked in groups of four tile rows, so that they share its L2.
__device__ __forceinline__ int xcd_gather(int id, int n) {
  return (n & 7) == 0 ? (id & 7) * (n >> 3) + (id >> 3) : id;
}
__device__ __forceinline__ int walk(const Fp8Args& p, int t, int& tn) {
  constexpr int GROUP_M = 4;
  const int group = t / (GROUP_M * p.ntn), first = group * GROUP_M;
  const int gm = min(p.ntm - first, GROUP_M), in = t - group * GROUP_M * p.ntn;
  tn = in / gm;
  return first + in % gm;
}

template <int TM, int OUT, int ACT>
__device__ __forceinline__ void fp8_tile(const Fp8Args& p, uint8_t* smem, int64_t m0, int64_t n0, int kt0, int kt1,
                                         void* C) {
  v16f acc[TM][4];
  fp8_mainloop<TM, OUT >= OUT_GATED>(p, smem, m0, n0, kt0, kt1, acc);
  const int w = threadIdx.x >> 6;
  if constexpr (OUT >= OUT_GATED) {
    store_gated<TM, ACT, OUT == OUT_GATED_TRAIN>(p, smem, m0, n0, acc);
  } else {
    store_tile<TM, OUT>(p, smem, C, m0 + 32 * TM * (w >> 1), n0 + 128 * (w & 1), acc);
  }
}

// Work item id of a launch of per items for each of p.splits ranges of the
// contraction.
template <int OUT, int ACT>
__device__ __forceinline__ void fp8_item(const Fp8Args& p, uint8_t* smem, int id, int per) {
  constexpr int BN = OUT >= OUT_GATED ? 128 : 256;
  int b = id, z = 0;
  if (p.splits > 1) {   // (split, tile) pairs in split-major order, cut into eight runs, one per XCD
    const int total = per * p.splits, base = total >> 3, extra = total & 7, x = id & 7, slot = id >> 3;
    const int pos = (x < extra ? x * (base + 1) : extra * (base + 1) + (x - extra) * base) + slot;
    z = pos / per;
    b = pos - z * per;
  }
  const int kt0 = (int)((int64_t)p.kb * z / p.splits), kt1 = (int)((int64_t)p.kb * (z + 1) / p.splits);
  void* C = OUT == OUT_PART ? (void*)((float*)p.C + (int64_t)z * p.split_stride) : p.C;
  const int R = p.rem, F = p.ntm * p.ntn - R;
  int tm, tn;
  if (b >= F + 2 * R) {
    fp8_tile<2, OUT, ACT>(p, smem, (int64_t)p.ntm * 256, (int64_t)(b - F - 2 * R) * BN, kt0, kt1, C);
  } else if (b >= R && b < R + F) {
    tm = walk(p, p.splits > 1 ? b : xcd_gather(b - R, F), tn);
    fp8_tile<4, OUT, ACT>(p, smem, (int64_t)tm * 256, (int64_t)tn * BN, kt0, kt1, C);
  } else {
    const int second = b >= R + F;
    tm = walk(p, F + xcd_gather(second ? b - R - F : b, R), tn);
    fp8_tile<2, OUT, ACT>(p, smem, (int64_t)tm * 256 + 128 * second, (int64_t)tn * BN, kt0, kt1, C);
  }
}

template <int OUT, int ACT>
__global__ void __launch_bounds__(256, 1) fp8_gemm_kernel(Fp8Args p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[OUT == OUT_GATED_TRAIN ? F8_LDS_GATED : F8_LDS];
  fp8_item<OUT, ACT>(p, smem, blockIdx.x, gridDim.x / p.splits);
}

// Two products in one launch, the first (bf16) in items 0 .. first - 1.
template <int OUT>
__global__ void __launch_bounds__(256, 1) fp8_two_kernel(Fp8Args p, Fp8Args q, int first) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[F8_LDS];
  if ((int)blockIdx.x < first) fp8_item<OUT_BF16, 0>(p, smem, blockIdx.x, first);
  else fp8_item<OUT, 0>(q, smem, blockIdx.x - first, (gridDim.x - first) / q.splits);
}

// ---------------------------------------------------------------------------
// Decode
// ---------------------------------------------------------------------------
// Few rows of A against the weights, which stream from HBM once, so the kernel
// is built for bytes in flight.  A workgroup takes 16 TMR rows of A and owns 16
// TN weight rows (gated: 16 of the gate's and the same 16 of the up
// projection's) over the whole contraction; its four waves take contiguous ranges of 128-blocks and
// their sums meet in LDS, in wave order.  Each wave fills R slots of one
// 128-block by buffer->LDS loads of whole lines (8 rows x 128 bytes) and
// reads its fragments back from them: no barrier in the loop.  (16 x 4096 x 14336
// 12.0 us, 4.9 TB/s; gated 1 x 14336 x 4096 20 us, 5.9 TB/s.  Two or eight waves
// are slower on both, and so are workgroups of 128 gated columns that quantize
// their own block: 32 us, for too few of them share the memory.)
//
// 16x16x128: lane l holds row l % 16 and chunks l / 16 and 4 + l / 16 of the
// 128-block; the weights are the first operand, so the result's lane l holds
// columns 4 (l / 16) + v of row l % 16.
constexpr int DEC_NW = 4;

template <int TMR, int TN, int R>
struct DecodeShape {
  static constexpr int ROWS = 16 * (TN + TMR);
  static constexpr int SLOT = ROWS * 128;
  static constexpr int LDS = DEC_NW * R * SLOT;
};

__device__ __forceinline__ void line_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, offset, 0, 0, 0);
}

struct Rows16 {
  __amdgpu_buffer_rsrc_t codes, scales;
};

template <int TMR, int TN, int R, int OUT, int ACT>
__global__ void __launch_bounds__(64 * DEC_NW) fp8_decode_kernel(Fp8Args p) {
  typedef DecodeShape<TMR, TN, R> Shape;
  constexpr bool GATED = OUT == OUT_GATED;
  static_assert(!GATED || TN == 2, "a gate tile and an up tile");
  constexpr int SLOT = Shape::SLOT, NDMA = Shape::ROWS / 8, NB = 2 * TN;
  constexpr int VM = NDMA + TN + TMR;            // vector memory operations per 128-block
  static_assert((R - 1) * VM < 64, "vmcnt is 6 bits");
  static_assert(DEC_NW * TMR * TN * 64 * 16 <= Shape::LDS, "the wave sums reuse the slots");
  __shared__ __attribute__((aligned(16))) uint8_t smem[Shape::LDS];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = threadIdx.x & 63, r = l & 15, g = l >> 4;
  constexpr int COLS = GATED ? 16 : 16 * TN;
  const int64_t n0 = (int64_t)blockIdx.x * COLS, m0 = (int64_t)blockIdx.y * (16 * TMR);
  const int64_t rows_a = p.M - m0 < 16 * TMR ? p.M - m0 : 16 * TMR;
  const int c0 = (int)((int64_t)p.kb * w / DEC_NW), c1 = (int)((int64_t)p.kb * (w + 1) / DEC_NW);
  const int64_t kp = (int64_t)p.kb * FP8_BLOCK;
  // weight tile j: 16 rows from n0 + 16 j (gated: from n0, and from np + n0)
  Rows16 bt[TN];
#pragma unroll
  for (int j = 0; j < TN; j++) {
    const int64_t first = n0 + (GATED ? j * p.np : 16 * j);
    int64_t rows = p.b.rows - first;
    rows = rows < 0 ? 0 : rows > 16 ? 16 : rows;
    bt[j].codes = resource(p.b.codes + (rows ? first : 0) * p.b.ld, rows ? (rows - 1) * p.b.ld + kp : 0);
    bt[j].scales = resource(p.b.scales + (rows ? first : 0), fp8_scale_extent(p.kb, p.b.scale_ld, p.b.rows, first, 1));
  }
  Rows16 at;
  at.codes = resource(p.a.codes + m0 * p.a.ld, (rows_a - 1) * p.a.ld + kp);
  at.scales = resource(p.a.scales + m0, fp8_scale_extent(p.kb, p.a.scale_ld, p.a.rows, m0, 1));
  uint8_t* const ring = smem + w * (R * SLOT);

  // load q of a slot moves slot rows 8 q .. + 7 (weight rows first); lane l
  // fills position l & 7 of its row with chunk (l & 7) ^ (row / 2 & 7)
  uint32_t off[NDMA];
#pragma unroll
  for (int q = 0; q < NDMA; q++) {
    const int row = 8 * (q < NB ? (q & 1) : q - NB) + (l >> 3);   // within its tile, or within A
    const uint32_t chunk = (uint32_t)((l & 7) ^ ((4 * (q & 1) + (l >> 4)) & 7));
    off[q] = (uint32_t)(row * (q < NB ? p.b.ld : p.a.ld)) + 16 * chunk;
  }
  const int pos0 = (g ^ ((r >> 1) & 7)) << 4, pos1 = ((4 + g) ^ ((r >> 1) & 7)) << 4;

  v4f acc[TMR][TN];
#pragma unroll
  for (int t = 0; t < TMR; t++)
#pragma unroll
    for (int j = 0; j < TN; j++) acc[t][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  int eb[R][TN], ea[R][TMR];

  // block c into slot k (past the wave's range: zeros, which add nothing)
  auto issue = [&](int k, int c) {
    const bool live = c < c1;
    uint8_t* sl = ring + k * SLOT;
#pragma unroll
    for (int q = 0; q < NDMA; q++) {
      const uint32_t at_byte = live ? off[q] + 128u * (uint32_t)c : kOutOfRange;
      line_to_lds(q < NB ? bt[q >> 1].codes : at.codes, sl + q * 1024, at_byte);
    }
#pragma unroll
    for (int j = 0; j < TN; j++)
      eb[k][j] = __builtin_amdgcn_raw_buffer_load_b8(
          bt[j].scales, live ? (uint32_t)c * (uint32_t)p.b.scale_ld + (uint32_t)r : kOutOfRange, 0, 0);
#pragma unroll
    for (int t = 0; t < TMR; t++)
      ea[k][t] = __builtin_amdgcn_raw_buffer_load_b8(
          at.scales, live ? (uint32_t)c * (uint32_t)p.a.scale_ld + (uint32_t)(16 * t + r) : kOutOfRange, 0, 0);
  };
#pragma unroll
  for (int k = 0; k < R; k++) {
    issue(k, c0 + k);
    __builtin_amdgcn_sched_barrier(0);
  }
  for (int base = c0; base < c1; base += R) {
#pragma unroll
    for (int k = 0; k < R; k++) {
      wait_cnt<(R - 1) * VM, 15>();              // this slot has landed
      asm volatile("" ::: "memory");
      const uint8_t* sl = ring + k * SLOT;
      v8i fb[TN];
#pragma unroll
      for (int j = 0; j < TN; j++) {
        const uint8_t* s = sl + (16 * j + r) * 128;
        fb[j] = __builtin_shufflevector(*(const v4i*)(s + pos0), *(const v4i*)(s + pos1), 0, 1, 2, 3, 4, 5, 6, 7);
      }
#pragma unroll
      for (int t = 0; t < TMR; t++) {
        const uint8_t* s = sl + (16 * TN + 16 * t + r) * 128;
        const v8i fa = __builtin_shufflevector(*(const v4i*)(s + pos0), *(const v4i*)(s + pos1), 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
        for (int j = 0; j < TN; j++)
          acc[t][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[j], fa, acc[t][j], 0, 0, 0, eb[k][j], 0,
                                                                       ea[k][t]);
      }
      wait_cnt<63, 0>();                          // the slot's reads are done before it is filled again
      asm volatile("" ::: "memory");
      issue(k, base + k + R);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  wait_cnt<0, 0>();   // nothing may still write LDS

  __syncthreads();
  v4f(*red)[TMR][TN][64] = (v4f(*)[TMR][TN][64])smem;
#pragma unroll
  for (int t = 0; t < TMR; t++)
#pragma unroll
    for (int j = 0; j < TN; j++) red[w][t][j][l] = acc[t][j];
  __syncthreads();
  for (int t = w; t < TMR; t += DEC_NW) {
    const int64_t m = m0 + 16 * t + r;
    if (m >= p.M) continue;
    v4f s[TN];
#pragma unroll
    for (int j = 0; j < TN; j++) {
      s[j] = red[0][t][j][l];
#pragma unroll
      for (int q = 1; q < DEC_NW; q++) s[j] += red[q][t][j][l];
    }
    if constexpr (GATED) {
      const int64_t n = n0 + 4 * g;
      v4f h;
#pragma unroll
      for (int v = 0; v < 4; v++) h[v] = n + v < p.n ? act_value<ACT>(s[0][v]) * s[1][v] : 0.0f;
      if (p.hf) *(v4f*)(p.hf + m * p.np + n) = h;
#pragma unroll
      for (int v = 0; v < 4; v++) {
        const float o = h[v];
        if (n + v < p.n) {
          if (p.h) p.h[m * p.ldh + n + v] = __builtin_bit_cast(uint16_t, (__bf16)o);
          if (p.g) {
            p.g[m * p.ldgu + n + v] = __builtin_bit_cast(uint16_t, (__bf16)s[0][v]);
            p.u[m * p.ldgu + n + v] = __builtin_bit_cast(uint16_t, (__bf16)s[1][v]);
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < TN; j++) {
        const int64_t n = n0 + 16 * j + 4 * g;
        if constexpr (OUT == OUT_BF16) {
          uint16_t* dst = (uint16_t*)p.C + m * p.ldc + n;
          const u32v2 o = {__builtin_bit_cast(uint32_t, (bf16x2){(__bf16)s[j][0], (__bf16)s[j][1]}),
                           __builtin_bit_cast(uint32_t, (bf16x2){(__bf16)s[j][2], (__bf16)s[j][3]})};
          if (n + 4 <= p.N) {
            *(u32v2_any*)dst = o;
          } else {
#pragma unroll
            for (int v = 0; v < 4; v++)
              if (n + v < p.N) dst[v] = (uint16_t)(o[v >> 1] >> (16 * (v & 1)));
          }
        } else {
          float* dst = (float*)p.C + m * p.ldc + n;
          if (n + 4 <= p.N) {
            *(v4f_any*)dst = s[j];
          } else {
#pragma unroll
            for (int v = 0; v < 4; v++)
              if (n + v < p.N) dst[v] = s[j][v];
          }
        }
      }
    }
  }
}

// The decode form's FP8 output: h [M, np] binary32 to codes and scales, 16
// lanes per block.  A launch of its own (3.9 us), because a block of 128 outputs
// comes from eight workgroups.
__global__ void __launch_bounds__(256) fp8_quantize_f32_kernel(const float* __restrict__ h, int64_t M, int64_t np,
                                                               Fp8Out q) {
  const int64_t i = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int64_t blocks = np / FP8_BLOCK;
  const int64_t row = i / blocks, b = i - row * blocks;
  if (row >= M) return;
  const int64_t c = b * FP8_BLOCK + 8 * (threadIdx.x & 15);
  float o[8];
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; e++) o[e] = h[row * np + c + e];
#pragma unroll
  for (int e = 0; e < 8; e++) m = max(m, abs_bits(o[e]));
  const uint32_t byte = fp8_scale_byte(max16(m));
  *(u32v2*)(q.codes + row * q.ld + c) = fp8_encode8(o, byte);
  if ((threadIdx.x & 15) == 0) q.scales[b * q.scale_ld + row] = (uint8_t)byte;
}

// ---------------------------------------------------------------------------
// C = sum over splits, in split order
// ---------------------------------------------------------------------------
template <bool BF16>
__global__ void __launch_bounds__(256) fp8_reduce_kernel(const float* __restrict__ ws, int splits, int64_t M, int64_t N,
                                                         void* __restrict__ C, int64_t ldc) {
  const int64_t total = M * N, stride = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += stride) {
    float s = ws[i];
#pragma unroll 4
    for (int z = 1; z < splits; z++) s += ws[(int64_t)z * total + i];
    const int64_t m = i / N, n = i - m * N;
    if (BF16) ((uint16_t*)C)[m * ldc + n] = __builtin_bit_cast(uint16_t, (__bf16)s);
    else ((float*)C)[m * ldc + n] = s;
  }
}

// ---------------------------------------------------------------------------
// Planning and launch
// ---------------------------------------------------------------------------
constexpr int64_t CUS = 256;

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// From 6144 columns on there are enough workgroups for several per compute unit:
// two slots each, and two weight tiles so that A's rows come through L2 half as
// often (16 x 14336 x 4096: 13.7 us against 15.9 with one tile and four slots;
// gated 1 x 14336 x 4096 25.4 against 30.6).  Below that one workgroup per compute
// unit keeps more in flight (16 x 4096 x 14336: 13.8 against 15.5).
constexpr int64_t DEC_MANY_COLUMNS = 6144;

// 128-blocks in LDS per wave (four of more rows do not fit)
constexpr int dec_slots(int tiles, bool many_columns) { return many_columns || tiles > 2 ? 2 : 4; }

// Time of the decode kernel in us, and the 16-row tiles per workgroup that it
// is shortest with: 2 for each round of the workgroups that the compute units
// hold, and 17 for a MB of the codes that one unit's workgroups bring.  (The
// gated form's quantizer is a launch of 3.)
struct DecodeTime {
  int tiles;
  double us;
};
static DecodeTime decode_time(int64_t M, int64_t N, int64_t kb, bool gated) {
  const bool many = N >= DEC_MANY_COLUMNS;
  const int b_tiles = gated || many ? 2 : 1;
  const int64_t cols = gated ? 16 : 16 * b_tiles;
  DecodeTime best{0, 0.0};
  for (int t = 8; t >= 1; t /= 2) {
    const int64_t rows = 16 * (b_tiles + t), held = 160 * 1024 / (DEC_NW * dec_slots(t, many) * rows * 128);
    const int64_t wgs = ceil_div(N, cols) * ceil_div(M, 16 * t);
    const double us = (gated ? 5.0 : 2.0) + 2.0 * (double)ceil_div(wgs, CUS * held) +
                      17e-6 * (double)(ceil_div(wgs, CUS) * rows * kb * FP8_BLOCK);
    if (!best.tiles || us < best.us) best = DecodeTime{t, us};
  }
  return best;
}

// Time of wide tiles in us: 8 for a tile and 1.3 for each of its blocks, half a
// tile 5 and 0.9 (0.75 where half of the compute units have none); 4 and 5 TB/s
// for the reduction of a split contraction.
static double wide_time(int64_t M, int64_t cols, int64_t kb, int half, int splits) {
  const int64_t tiles = ceil_div(M, 256) * cols, parts = ceil_div(M, 128) * cols;
  const double blocks = (double)kb;
  if (splits > 1) return 8.0 + 1.3 * blocks / splits;
  if (half) return 5.0 + (parts <= CUS / 2 ? 0.75 : 0.9) * blocks;
  return (8.0 + 1.3 * blocks) * (double)(tiles > CUS ? tiles / (double)CUS : 1.0);
}
static double reduce_time(int64_t M, int64_t N, int splits) {
  return splits > 1 ? 4.0 + 8.0e-6 * (double)M * (double)N * splits / 5.0 : 0.0;
}

// Decode kernel or wide tiles: decode up to 32 rows, and up to 256 where its
// time is the shorter one.  As measured with the weights in memory, decode and
// wide tiles: 64 x 4096 x 4096 9.9 and 17.0 us, 256 x 1024 x 8192 12.4 and 25.8,
// 128 x 4096 x 14336 38.7 and 27.9; gated 64 x 4096 x 4096 15.9 and 30.5, 256 x
// 1024 x 8192 19.2 and 50.1, 64 x 14336 x 4096 46.5 and 37.2.  (With more rows it
// would still be for narrow outputs, 400 x 1024 x 8192 18.6 and 28.2, and not
// for others, 400 x 4096 x 4096 35.3 and 26.5: those are left to the wide tiles,
// as are outputs of more columns than one launch of this kernel holds.)
static int decode_tiles(int64_t M, int64_t N, int64_t kb, bool gated, double wide) {
  if (M > 256 || ceil_div(N, gated ? 16 : 32) > FP8_LAUNCH_THREADS / (64 * DEC_NW)) return 0;
  const DecodeTime d = decode_time(M, N, kb, gated);
  return M <= 32 || d.us < wide ? d.tiles : 0;
}

static Fp8Plan plan_wide(int64_t M, int64_t N, int64_t K, double* us) {
  Fp8Plan pl{0, 0, 1};
  const int64_t kb = ceil_div(K, FP8_BLOCK), cols = ceil_div(N, 256), tiles = ceil_div(M, 256) * cols;
  pl.half = ceil_div(M, 128) * cols <= CUS;
  *us = wide_time(M, cols, kb, pl.half, 1);
  if (tiles == 0 || tiles >= CUS || kb < 16) return pl;
  int64_t most = CUS / tiles;
  if (most > kb / 8) most = kb / 8;
  if (most > 32) most = 32;
  for (int s = 2; s <= most; s++) {
    const double t = wide_time(M, cols, kb, 0, s) + reduce_time(M, N, s);
    if (t < *us) {
      *us = t;
      pl.splits = s;
    }
  }
  return pl;
}

Fp8Plan plan_fp8_gemm(int64_t M, int64_t N, int64_t K) {
  double us;
  Fp8Plan pl = plan_wide(M, N, K, &us);
  // (over no contraction the wide tiles write their zeros)
  if (K > 0 && M > 0 && N > 0) pl.decode = decode_tiles(M, N, ceil_div(K, FP8_BLOCK), false, us);
  if (pl.decode) pl.splits = 1;
  return pl;
}

size_t fp8_gemm_workspace(const Fp8Plan& p, int64_t M, int64_t N) {
  return p.splits > 1 ? (size_t)p.splits * (size_t)M * (size_t)N * sizeof(float) : 0;
}

template <int TMR, int TN, int R, int OUT, int ACT>
static void launch_decode_one(const Fp8Args& p, int64_t groups, hipStream_t s) {
  static_assert(DecodeShape<TMR, TN, R>::LDS <= 160 * 1024, "LDS");
  hipLaunchKernelGGL((fp8_decode_kernel<TMR, TN, R, OUT, ACT>), dim3((unsigned)groups, (unsigned)ceil_div(p.M, 16 * TMR)),
                     dim3(64 * DEC_NW), 0, s, p);
}

template <int TMR, int OUT, int ACT>
static void launch_decode_tmr(const Fp8Args& p, hipStream_t s) {
  constexpr int R0 = dec_slots(TMR, false), R1 = dec_slots(TMR, true);
  if constexpr (OUT == OUT_GATED) {
    if (p.np < DEC_MANY_COLUMNS) launch_decode_one<TMR, 2, R0, OUT, ACT>(p, p.np / 16, s);
    else launch_decode_one<TMR, 2, R1, OUT, ACT>(p, p.np / 16, s);
  } else {
    if (p.N < DEC_MANY_COLUMNS) launch_decode_one<TMR, 1, R0, OUT, ACT>(p, ceil_div(p.N, 16), s);
    else launch_decode_one<TMR, 2, R1, OUT, ACT>(p, ceil_div(p.N, 32), s);
  }
}

// The wide launch's tiles; returns its work items per range of the contraction.
// The tiles that are left over after whole rounds of the compute units are cut
// into halves while those, with the tails, make one round: half a tile takes 0.6
// of a whole one's time, so a second round of them would be later than the
// uncut tiles (4096 x 11008 x 16384, 176 left over: 540 us cut, 509 whole; gated
// 1000 x 4096 x 14336, 192: 108 and 99.  4096 x 14336 x 8192, 128: 343 cut, 354
// whole; 4096 x 5120 x 4096, 64: 74 and 88).
static int lay_tiles(Fp8Args& p, const Fp8Plan& plan, int bn) {
  p.ntm = (int)((p.M + 127) / 256);
  p.ntn = (int)((p.N + bn - 1) / bn);
  p.tails = (int64_t)p.ntm * 256 < p.M ? p.ntn : 0;
  p.splits = plan.splits;
  const int64_t tiles = (int64_t)p.ntm * p.ntn;
  const int over = tiles > CUS ? (int)(tiles % CUS) : 0;
  p.rem = plan.splits > 1 ? 0 : plan.half ? (int)tiles : 2 * over + p.tails <= CUS ? over : 0;
  return (int)(tiles + p.rem + p.tails);
}

template <int OUT, int ACT>
static void launch_products(Fp8Args p, const Fp8Plan& plan, hipStream_t s) {
  if (plan.decode) {
    if constexpr (OUT != OUT_PART && OUT != OUT_GATED_TRAIN) {
      switch (plan.decode) {
        case 1: return launch_decode_tmr<1, OUT, ACT>(p, s);
        case 2: return launch_decode_tmr<2, OUT, ACT>(p, s);
        case 4: return launch_decode_tmr<4, OUT, ACT>(p, s);
        default: return launch_decode_tmr<8, OUT, ACT>(p, s);
      }
    }
    return;
  }
  const int per = lay_tiles(p, plan, OUT >= OUT_GATED ? 128 : 256);
  hipLaunchKernelGGL((fp8_gemm_kernel<OUT, ACT>), dim3((unsigned)per * (unsigned)plan.splits), dim3(256), 0, s, p);
}

static Fp8Args gemm_args(const Fp8In& a, const Fp8In& b, int64_t K, void* C, int64_t ldc, float* workspace,
                         const Fp8Plan& plan) {
  Fp8Args p{};
  p.a = a;
  p.b = b;
  p.M = a.rows;
  p.N = b.rows;
  p.kb = (int)((K + FP8_BLOCK - 1) / FP8_BLOCK);
  p.splits = plan.splits;
  p.C = plan.splits > 1 ? workspace : C;
  p.ldc = plan.splits > 1 ? p.N : ldc;
  p.split_stride = plan.splits > 1 ? p.M * p.N : 0;
  return p;
}

static void launch_reduce(const Fp8Args& p, void* C, int64_t ldc, int c_type, const float* workspace, hipStream_t s) {
  int64_t n = (p.M * p.N + 255) / 256;
  if (n > 8192) n = 8192;
  if (c_type == FP8_BF16)
    hipLaunchKernelGGL(fp8_reduce_kernel<true>, dim3((unsigned)n), dim3(256), 0, s, workspace, p.splits, p.M, p.N, C, ldc);
  else
    hipLaunchKernelGGL(fp8_reduce_kernel<false>, dim3((unsigned)n), dim3(256), 0, s, workspace, p.splits, p.M, p.N, C,
                       ldc);
}

hipError_t launch_fp8_gemm(const Fp8In& a, const Fp8In& b, int64_t K, void* C, int64_t ldc, int c_type,
                           float* workspace, const Fp8Plan& plan, hipStream_t s) {
  const Fp8Args p = gemm_args(a, b, K, C, ldc, workspace, plan);
  if (plan.splits > 1) {
    launch_products<OUT_PART, 0>(p, plan, s);
    launch_reduce(p, C, ldc, c_type, workspace, s);
  } else if (c_type == FP8_BF16) {
    launch_products<OUT_BF16, 0>(p, plan, s);
  } else {
    launch_products<OUT_F32, 0>(p, plan, s);
  }
  return hipGetLastError();
}

// Two products that depend on nothing of each other: where both together fit the
// compute units at once, one launch runs them side by side, the second split
// over what the first leaves free, if that is sooner than one after the other.
// (12608 x 768 x 4096 in 150 tiles and 4096 x 768 x 12608 in 48 tiles of three
// times their length: 105 us one after the other, 88 in one launch.)
Fp8TwoPlan plan_fp8_two(int64_t M0, int64_t N0, int64_t K0, int64_t M1, int64_t N1, int64_t K1) {
  Fp8TwoPlan t{plan_fp8_gemm(M0, N0, K0), plan_fp8_gemm(M1, N1, K1), 0};
  const int64_t c0 = ceil_div(N0, 256), c1 = ceil_div(N1, 256), n0 = ceil_div(M0, 256) * c0, n1 = ceil_div(M1, 256) * c1;
  const int64_t kb0 = ceil_div(K0, FP8_BLOCK), kb1 = ceil_div(K1, FP8_BLOCK);
  if (n0 == 0 || n1 == 0 || n0 + n1 > CUS || t.first.decode || t.second.decode || t.first.splits > 1) return t;
  int64_t s = (CUS - n0) / n1;
  if (s > kb1 / 8) s = kb1 / 8;
  if (s < 1) s = 1;
  const int half = s == 1 && ceil_div(M0, 128) * c0 + ceil_div(M1, 128) * c1 <= CUS;
  const Fp8Plan first{0, half, 1}, second{0, half, (int)s};
  const double a = wide_time(M0, c0, kb0, half, 1);
  const double b = wide_time(M1, c1, kb1, half, (int)s) + reduce_time(M1, N1, (int)s);
  const double one = wide_time(M0, c0, kb0, t.first.half, 1);
  const double two = wide_time(M1, c1, kb1, t.second.half, t.second.splits) + reduce_time(M1, N1, t.second.splits);
  if ((a > b ? a : b) < one + two) t = Fp8TwoPlan{first, second, 1};
  return t;
}

hipError_t launch_fp8_two(const Fp8In& a0, const Fp8In& b0, int64_t K0, void* C0, int64_t ldc0, const Fp8In& a1,
                          const Fp8In& b1, int64_t K1, void* C1, int64_t ldc1, int c1_type, float* workspace,
                          const Fp8TwoPlan& plan, hipStream_t s) {
  if (!plan.together) {
    const hipError_t e = launch_fp8_gemm(a0, b0, K0, C0, ldc0, FP8_BF16, workspace, plan.first, s);
    return e != hipSuccess ? e : launch_fp8_gemm(a1, b1, K1, C1, ldc1, c1_type, workspace, plan.second, s);
  }
  Fp8Args p = gemm_args(a0, b0, K0, C0, ldc0, nullptr, plan.first);
  Fp8Args q = gemm_args(a1, b1, K1, C1, ldc1, workspace, plan.second);
  const int first = lay_tiles(p, plan.first, 256), per = lay_tiles(q, plan.second, 256);
  const dim3 grid((unsigned)(first + per * plan.second.splits)), wg(256);
  if (plan.second.splits > 1) {
    hipLaunchKernelGGL(fp8_two_kernel<OUT_PART>, grid, wg, 0, s, p, q, first);
    launch_reduce(q, C1, ldc1, c1_type, workspace, s);
  } else if (c1_type == FP8_BF16) {
    hipLaunchKernelGGL(fp8_two_kernel<OUT_BF16>, grid, wg, 0, s, p, q, first);
  } else {
    hipLaunchKernelGGL(fp8_two_kernel<OUT_F32>, grid, wg, 0, s, p, q, first);
  }
  return hipGetLastError();
}

// The gated block: the decode form for few rows, else wide tiles (256 rows x 128
// outputs), as halves of 128 rows when there are few of them.
static Fp8Plan plan_fp8_gated(int64_t M, int64_t np, int64_t K) {
  Fp8Plan pl{0, 0, 1};
  const int64_t kb = ceil_div(K, FP8_BLOCK), cols = np / 128;
  pl.half = ceil_div(M, 128) * cols <= CUS;
  // (its epilogue takes 1.2 us longer than the product's: 64 x 512 x 512 decode 6.4 us, wide 9.2)
  if (M > 0) pl.decode = decode_tiles(M, np, kb, true, 1.2 + wide_time(M, cols, kb, pl.half, 1));
  return pl;
}

size_t fp8_gated_workspace(int64_t M, int64_t np, int64_t K, bool fp8_out) {
  return plan_fp8_gated(M, np, K).decode && fp8_out ? (size_t)M * (size_t)np * sizeof(float) : 0;
}

template <int ACT>
static void launch_gated(const Fp8Args& p, const Fp8Plan& plan, hipStream_t s) {
  if (p.g && !plan.decode) launch_products<OUT_GATED_TRAIN, ACT>(p, plan, s);
  else launch_products<OUT_GATED, ACT>(p, plan, s);
}

hipError_t launch_fp8_gated(const Fp8GatedArgs& a, float* workspace, hipStream_t s) {
  Fp8Args p{};
  p.a = a.x;
  p.b = a.w;
  p.M = a.x.rows;
  p.N = a.np;
  p.kb = (int)((a.K + FP8_BLOCK - 1) / FP8_BLOCK);
  p.splits = 1;
  p.n = a.n;
  p.np = a.np;
  p.q = a.q;
  p.h = a.h;
  p.g = a.g;
  p.u = a.u;
  p.ldh = a.ldh;
  p.ldgu = a.ldgu;
  const Fp8Plan plan = plan_fp8_gated(p.M, p.np, a.K);
  const bool quantize = plan.decode && a.q.codes;
  p.hf = quantize ? workspace : nullptr;
  if (a.act == ACT_SILU) launch_gated<ACT_SILU>(p, plan, s);
  else if (a.act == ACT_GELU) launch_gated<ACT_GELU>(p, plan, s);
  else launch_gated<ACT_GELU_TANH>(p, plan, s);
  if (quantize)
    hipLaunchKernelGGL(fp8_quantize_f32_kernel, dim3((unsigned)((p.M * (p.np / FP8_BLOCK) + 15) / 16)), dim3(256), 0, s,
                       workspace, p.M, p.np, a.q);
  return hipGetLastError();
}

}  // namespace mxfp4
