// kq_mx4_gemm.hip — the product of two microscaled 4-bit matrices:
// y[m][n] = sum_k a'[m][k] w'[n][k].
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 4-bit codes directly and applies
// one scale byte per 32 of them, so nothing is unpacked: a lane's operand is
// the 16 bytes of one block and its scale byte. The products are exact (codes
// have at most two significant bits) and are summed in fp32.
//
// Weight rows are the instruction's A operand and activation rows its B
// operand, so a lane's results are runs of four consecutive n for one m.
//
// Many rows are bound by the operands' way through LDS (64 bytes a clock) and the
// barrier between a K tile's copies and its products: 4096 x 2560 x 9728 runs
// 60 to 75 us, 2.7 to 3.4 PFLOP/s, of which neither the copies alone (51 to 57)
// nor the products alone (53 to 57, 27 from registers) account for all. Its
// 124000 clocks hold 68000 of LDS reads and 34000 of copies into LDS, and the
// matrix cores are busy for 39 % of them.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq_internal.h"
#include "kq_mx4_dev.h"

namespace kqd {

constexpr int GEMM_KB = 8;   // blocks of 32 per K tile: 128 bytes of codes per row, a line (64 bytes: half the rate of copies)
constexpr int GEMM_KS = 4;   // K tiles per group of scales: 32 bytes per row

// The lane's 16-byte pieces of one operand's K tiles: piece p of row r goes to
// LDS slot 8 r + (p ^ (r >> 1 & 7)), so that the 16 rows of a quarter-wave read
// at one piece cover every bank. The byte offsets of K tile 0 stay in
// registers; a K tile is 128 bytes further for every row. Rows past the matrix
// and pieces past a row's end read zero.
template <int ROWS, int THREADS>
struct CodePieces {
  static constexpr int N = ROWS * GEMM_KB / THREADS;
  static_assert(N * THREADS == ROWS * GEMM_KB && THREADS % 128 == 0, "whole copies, one piece index per lane");
  uint32_t off[N];
  __device__ __forceinline__ static int piece() { return ((int)threadIdx.x & 7) ^ (((int)threadIdx.x >> 4) & 7); }
  __device__ __forceinline__ void init(int nblk) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int slot = i * THREADS + (int)threadIdx.x;
      off[i] = ((uint32_t)(slot >> 3) * (uint32_t)nblk + (uint32_t)piece()) * 16u;
    }
  }
  __device__ __forceinline__ void copy(rsrc_t rc, uint8_t* lds, int kt, int nblk) const {
    const bool in = piece() < nblk - kt * GEMM_KB;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint32_t o = off[i];
      if (!in) o = OOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rc, (lds_void_t*)(lds + (i * THREADS + wave_id() * 64) * 16), 16, o,
                                               kt * 128, 0, 0);
    }
  }
};

// Scales of one operand for a group of K tiles, 32 bytes per row as two 16-byte
// pieces, piece q of row r at slot q ROWS + r. A lane that took its scales from
// memory at each K tile would touch a line per row, 1500 lines per workgroup
// and K tile (4096 x 2560 x 9728: 98 us against 84 with the scales in LDS).
// AL: rows of scales are dword-aligned (K a multiple of 128) and are copied;
// otherwise each dword is put together from bytes. What lies past a row's end
// is masked where it is read.
template <int ROWS, int THREADS, bool AL>
__device__ __forceinline__ void copy_scales(rsrc_t rs, uint8_t* lds, int group, int nblk) {
  const int b0 = group * (GEMM_KS * GEMM_KB);
  if constexpr (AL) {
#pragma unroll
    for (int i = 0; i < (ROWS * 2 + THREADS - 1) / THREADS; ++i) {
      const int first = i * THREADS + wave_id() * 64, slot = first + (int)(threadIdx.x & 63);
      if (ROWS * 2 % THREADS != 0 && first >= ROWS * 2) break;   // whole waves leave
      const int q = slot / ROWS, r = slot - q * ROWS, b = b0 + q * 16;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)(lds + first * 16), 16,
                                               b < nblk ? (uint32_t)(r * nblk + b) : OOB, 0, 0, 0);
    }
  } else {
    for (int i = threadIdx.x; i < ROWS * 8; i += THREADS) {
      const int slot = i >> 2, q = slot / ROWS, r = slot - q * ROWS, b = b0 + q * 16 + (i & 3) * 4;
      uint32_t d = 0;
#pragma unroll
      for (int s = 0; s < 4; ++s) d |= ld8(rs, b + s < nblk ? (uint32_t)(r * nblk + b + s) : OOB) << (8 * s);
      reinterpret_cast<uint32_t*>(lds)[i] = d;
    }
  }
}

template <int S>
__device__ __forceinline__ v16f mfma_fp4(u32x4 a, u32x4 b, v16f c, uint32_t sa, uint32_t sb) {
  const v8i av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const v8i bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, S, (int)sa, S, (int)sb);
}

template <int T> struct OutT;
template <> struct OutT<T_F32> { typedef float t; };
template <> struct OutT<T_F16> { typedef _Float16 t; };
template <> struct OutT<T_BF16> { typedef __bf16 t; };

// The lane's operands of one step: ROWS tiles of 32 rows from `row` on, at the
// piece at byte offset p.
template <int TILES>
__device__ __forceinline__ void read_pieces(const uint8_t* lds, int row, int p, u32x4 (&f)[TILES]) {
#pragma unroll
  for (int i = 0; i < TILES; ++i) f[i] = *reinterpret_cast<const u32x4*>(lds + (row + 32 * i) * 128 + p);
}

// The lane's four scale bytes of K tile kt (blocks 4 h .. 4 h + 3 of it) of the
// same rows of an operand with ROWS rows; `in`: all ones, or zero for blocks
// past the end of the rows.
template <int ROWS, int TILES>
__device__ __forceinline__ void read_scales(const uint8_t* lds, int row, int kt, int h, uint32_t in, uint32_t (&s)[TILES]) {
  const uint8_t* p = lds + (((kt % GEMM_KS) >> 1) * ROWS + row) * 16 + (kt & 1) * 8 + 4 * h;
#pragma unroll
  for (int i = 0; i < TILES; ++i) s[i] = *reinterpret_cast<const uint32_t*>(p + 32 * 16 * i) & in;
}

// One step of a wave's tiles.
template <int S, int TN, int TM>
__device__ __forceinline__ void multiply_step(const u32x4 (&fw)[TN], const u32x4 (&fa)[TM], const uint32_t (&sw)[TN],
                                              const uint32_t (&sa)[TM], v16f (&acc)[TN][TM]) {
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = mfma_fp4<S>(fw[i], fa[j], acc[i][j], sw[i], sa[j]);
}

// A workgroup of WN x WM waves computes BN weight rows x BM activation rows;
// each wave TN x TM tiles of 32 x 32. Two K tiles of codes in LDS, one being
// multiplied while the other lands, and one barrier per K tile. Each step's
// operands are read from LDS ahead of it (a quarter of a K tile; 63 us against
// 69 for 4096 x 2560 x 9728 where they are read in the step itself).
template <int WN, int WM, int TN, int TM>
struct GemmTile {
  static constexpr int BN = 32 * WN * TN, BM = 32 * WM * TM, THREADS = 64 * WN * WM;
  static constexpr int CODES = (BN + BM) * 128, SCALES = (BN + BM) * 32;   // bytes of a K tile, of a group
  static constexpr int LDS = 2 * (CODES + SCALES);
};

// Every copy of this wave has landed and every LDS read has returned, for all
// waves. A barrier alone waits for neither: copies are loads to the compiler.
__device__ __forceinline__ void meet() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <int T, int WN, int WM, int TN, int TM, bool AL>
__global__ __launch_bounds__(64 * WN * WM) void k_mx4_gemm(const uint8_t* __restrict__ ac, const uint8_t* __restrict__ as,
                                                          const uint8_t* __restrict__ wc, const uint8_t* __restrict__ ws,
                                                          void* __restrict__ y, int64_t M, int64_t N, int nblk,
                                                          uint32_t tiles_m) {
  typedef GemmTile<WN, WM, TN, TM> G;
  constexpr int BN = G::BN, BM = G::BM, THREADS = G::THREADS;
  extern __shared__ u32x4 lds4[];   // two K tiles of codes, two groups of scales; weight rows first in each
  uint8_t* lds = reinterpret_cast<uint8_t*>(lds4);
  uint8_t* lds_s = lds + 2 * G::CODES;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int r = lane & 31, h = lane >> 5;
  const int wn = (wave % WN) * 32 * TN, wm = (wave / WN) * 32 * TM;
  const uint32_t tn = blockIdx.x / tiles_m, tm = blockIdx.x - tn * tiles_m;
  const int64_t n0 = (int64_t)tn * BN, m0 = (int64_t)tm * BM;
  const int rows_n = __builtin_amdgcn_readfirstlane((int)min<int64_t>(BN, N - n0));
  const int rows_m = __builtin_amdgcn_readfirstlane((int)min<int64_t>(BM, M - m0));
  rsrc_t rwc, rws, rac, ras;
  mx4_rows(wc, ws, n0, rows_n, nblk, rwc, rws);
  mx4_rows(ac, as, m0, rows_m, nblk, rac, ras);
  CodePieces<BN, THREADS> pw;
  CodePieces<BM, THREADS> pa;
  pw.init(nblk);
  pa.init(nblk);
  const int nkt = (nblk + GEMM_KB - 1) / GEMM_KB;
  v16f acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.0f;
  u32x4 fw[2][TN], fa[2][TM];
  uint32_t sw[TN], sa[TM], swn[TN], san[TM];
#define KQ_COPY_CODES(KT)                                          \
  {                                                                \
    uint8_t* st = lds + ((KT) & 1) * G::CODES;                     \
    pw.copy(rwc, st, KT, nblk);                                    \
    pa.copy(rac, st + BN * 128, KT, nblk);                         \
  }
#define KQ_COPY_SCALES(GROUP)                                      \
  {                                                                \
    uint8_t* st = lds_s + ((GROUP) & 1) * G::SCALES;               \
    copy_scales<BN, THREADS, AL>(rws, st, GROUP, nblk);            \
    copy_scales<BM, THREADS, AL>(ras, st + BN * 32, GROUP, nblk);  \
  }
  // step S of a K tile takes block 4 h + S
#define KQ_READ(KT, S)                                             \
  {                                                                \
    const uint8_t* st = lds + ((KT) & 1) * G::CODES;               \
    const int p = ((4 * h + (S)) ^ (r >> 1 & 7)) * 16;             \
    read_pieces<TN>(st, wn + r, p, fw[(S) & 1]);                   \
    read_pieces<TM>(st + BN * 128, wm + r, p, fa[(S) & 1]);        \
  }
#define KQ_READ_SCALES(KT, SW, SA)                                           \
  {                                                                          \
    const uint8_t* st = lds_s + (((KT) / GEMM_KS) & 1) * G::SCALES;          \
    const uint32_t in = (KT) * GEMM_KB + 4 * h < nblk ? 0xffffffffu : 0u;    \
    read_scales<BN, TN>(st, wn + r, KT, h, in, SW);                          \
    read_scales<BM, TM>(st + BN * 32, wm + r, KT, h, in, SA);                \
  }
#define KQ_MULTIPLY(S) multiply_step<S>(fw[(S) & 1], fa[(S) & 1], sw, sa, acc);
  KQ_COPY_SCALES(0)
  KQ_COPY_CODES(0)
  meet();
  KQ_COPY_CODES(1)
  KQ_READ(0, 0)
  KQ_READ_SCALES(0, sw, sa)
  for (int kt = 0; kt < nkt - 1;) {
    // The next group's scales (none: zeros) take the place of the group before
    // this one, which every wave is done with.
    const int group = kt / GEMM_KS + 1;
    KQ_COPY_SCALES(group)
    const int end = min(kt + GEMM_KS, nkt - 1);
    for (; kt < end; ++kt) {
      KQ_READ(kt, 1)
      KQ_MULTIPLY(0)
      KQ_READ(kt, 2)
      KQ_MULTIPLY(1)
      KQ_READ(kt, 3)
      KQ_MULTIPLY(2)
      meet();   // K tile kt + 1 has landed, K tile kt has been read
      const int k1 = kt + 1, k2 = kt + 2;
      KQ_COPY_CODES(k2)   // past the last: zeros
      KQ_READ(k1, 0)
      KQ_READ_SCALES(k1, swn, san)
      KQ_MULTIPLY(3)
#pragma unroll
      for (int i = 0; i < TN; ++i) sw[i] = swn[i];
#pragma unroll
      for (int j = 0; j < TM; ++j) sa[j] = san[j];
    }
  }
  const int last = nkt - 1;
  KQ_READ(last, 1)
  KQ_MULTIPLY(0)
  KQ_READ(last, 2)
  KQ_MULTIPLY(1)
  KQ_READ(last, 3)
  KQ_MULTIPLY(2)
  KQ_MULTIPLY(3)
#undef KQ_MULTIPLY
#undef KQ_READ_SCALES
#undef KQ_READ
#undef KQ_COPY_SCALES
#undef KQ_COPY_CODES
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no copy outlives the workgroup
  typedef typename OutT<T>::t out_t;
  typedef out_t out4 __attribute__((ext_vector_type(4)));
  out_t* yo = static_cast<out_t*>(y);
  const bool whole = (N & 3) == 0;   // then four consecutive n of a row are aligned together
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int64_t m = m0 + wm + 32 * j + r;
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      // The stores are conditional; a matrix instruction moved into such a
      // branch would read registers that its idle lanes never wrote.
      asm volatile("" : "+v"(acc[i][j]));
      if (m < M) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t n = n0 + wn + 32 * i + 8 * q + 4 * h;
          out_t* p = yo + m * N + n;
          const out4 v = {(out_t)acc[i][j][4 * q], (out_t)acc[i][j][4 * q + 1], (out_t)acc[i][j][4 * q + 2],
                          (out_t)acc[i][j][4 * q + 3]};
          if (whole && n + 4 <= N) {
            *reinterpret_cast<out4*>(p) = v;
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (n + k < N) p[k] = v[k];
          }
        }
      }
    }
  }
}

// The product for few tiles: a workgroup computes 32 x 32, its waves split K and
// take their operands straight from memory. Such loads (a lane's 16 bytes of a
// row of its own) run at a quarter of the rate of whole lines, but nothing waits
// for anything else until the waves' sums meet in LDS, where they are added in
// wave order. A lane (r, h) takes blocks 4 h .. 4 h + 3 of each 8 of its wave's,
// so that their scales are one dword.
constexpr int SMALL_WAVES = 16;

template <bool AL>
struct SmallOperand {
  u32x4 codes[4];
  uint32_t scales;
  __device__ __forceinline__ void load(rsrc_t rc, rsrc_t rs, int c, int nblk, int r, int h) {
    const int b = c * GEMM_KB + 4 * h;
    const uint32_t o = (uint32_t)r * (uint32_t)nblk + (uint32_t)b;
#pragma unroll
    for (int s = 0; s < 4; ++s) codes[s] = ld128(rc, b + s < nblk ? (o + s) * 16u : OOB);
    if constexpr (AL) {
      scales = ld32(rs, b < nblk ? o : OOB);
    } else {
      scales = 0;
#pragma unroll
      for (int s = 0; s < 4; ++s) scales |= ld8(rs, b + s < nblk ? o + s : OOB) << (8 * s);
    }
  }
};

template <int T, bool AL>
__global__ __launch_bounds__(64 * SMALL_WAVES) void k_mx4_gemm_small(const uint8_t* __restrict__ ac, const uint8_t* __restrict__ as,
                                                                    const uint8_t* __restrict__ wc, const uint8_t* __restrict__ ws,
                                                                    void* __restrict__ y, int64_t M, int64_t N, int nblk,
                                                                    uint32_t tiles_m, int waves) {
  __shared__ v16f red[SMALL_WAVES][64];
  const int lane = threadIdx.x & 63, wave = wave_id(), r = lane & 31, h = lane >> 5;
  const uint32_t tn = blockIdx.x / tiles_m, tm = blockIdx.x - tn * tiles_m;
  const int64_t n0 = (int64_t)tn * 32, m0 = (int64_t)tm * 32;
  const int rows_n = __builtin_amdgcn_readfirstlane((int)min<int64_t>(32, N - n0));
  const int rows_m = __builtin_amdgcn_readfirstlane((int)min<int64_t>(32, M - m0));
  rsrc_t rwc, rws, rac, ras;
  mx4_rows(wc, ws, n0, rows_n, nblk, rwc, rws);
  mx4_rows(ac, as, m0, rows_m, nblk, rac, ras);
  const int nc = (nblk + GEMM_KB - 1) / GEMM_KB, c0 = nc * wave / waves, c1 = nc * (wave + 1) / waves;
  v16f acc = {};
  SmallOperand<AL> w, a, wn, an;
  wn.load(rwc, rws, c0 < c1 ? c0 : nc, nblk, r, h);
  an.load(rac, ras, c0 < c1 ? c0 : nc, nblk, r, h);
  for (int c = c0; c < c1; ++c) {
    w = wn;
    a = an;
    wn.load(rwc, rws, c + 1 < c1 ? c + 1 : nc, nblk, r, h);
    an.load(rac, ras, c + 1 < c1 ? c + 1 : nc, nblk, r, h);
    acc = mfma_fp4<0>(w.codes[0], a.codes[0], acc, w.scales, a.scales);
    acc = mfma_fp4<1>(w.codes[1], a.codes[1], acc, w.scales, a.scales);
    acc = mfma_fp4<2>(w.codes[2], a.codes[2], acc, w.scales, a.scales);
    acc = mfma_fp4<3>(w.codes[3], a.codes[3], acc, w.scales, a.scales);
  }
  red[wave][lane] = acc;
  __syncthreads();
  typedef typename OutT<T>::t out_t;
  for (int t = threadIdx.x; t < 1024; t += 64 * waves) {
    // weight row n is element 4 (n >> 3) + (n & 3) of lane m + 32 (n >> 2 & 1)
    const int n = t & 31, m = t >> 5, i = 4 * (n >> 3) + (n & 3), l = m + 32 * (n >> 2 & 1);
    if (n < rows_n && m < rows_m) {
      const float* p = reinterpret_cast<const float*>(&red[0][l]) + i;
      float v = p[0];
      for (int k = 1; k < waves; ++k) v += p[k * 1024];
      static_cast<out_t*>(y)[(m0 + m) * N + n0 + n] = (out_t)v;
    }
  }
}

}  // namespace kqd

namespace kq {

using namespace kqd;

namespace {

template <int T, int WN, int WM, int TN, int TM>
int gemm_cfg(const Mx4GemmArgs& a) {
  typedef GemmTile<WN, WM, TN, TM> G;
  static_assert(G::LDS <= 160 * 1024, "a compute unit's LDS");
  const int64_t tiles_m = (a.M + G::BM - 1) / G::BM, tiles_n = (a.N + G::BN - 1) / G::BN;
  const unsigned grid = (unsigned)(tiles_m * tiles_n);
  dispatch_log("k_mx4_gemm", -1, a.N, a.K, (int)a.M, grid, 1, G::THREADS, G::LDS, "type=%d tile=%dx%d", T, G::BN, G::BM);
  auto* k = a.K % 128 == 0 ? k_mx4_gemm<T, WN, WM, TN, TM, true> : k_mx4_gemm<T, WN, WM, TN, TM, false>;
  hipLaunchKernelGGL(k, dim3(grid), dim3(G::THREADS), G::LDS, a.stream, a.a_codes, a.a_scales, a.w_codes, a.w_scales,
                     a.y, a.M, a.N, (int)(a.K / 32), (uint32_t)tiles_m);
  return (int)hipGetLastError();
}

// Rounds of the grid over the compute units, in microseconds per K tile, from
// runs with at least one tile per unit (64 x 64 tiles share a unit: 0.3 each,
// 0.5 for one alone). M x N x K, the tile chosen and the next best:
//   4096 x 2560 x 9728: 160 x 256 (256 tiles) 68.6 us, 256 x 256 (160) 76.0
//   4096 x 19456 x 2560: 256 x 256 157 us, 160 x 256 193
//   2048 x 2560 x 9728: 192 x 128 (224 tiles) 40.9 us, 160 x 256 55.6
//   300 x 6144 x 2560: 64 x 64 11.0 us, 192 x 128 14.5
// Where 32 x 32 tiles do not outnumber the compute units and K is not short,
// the direct kernel: 64 x 2560 x 9728 14.9 us (64 x 64: 20.2), 17 x 1570 x 5856
// 8.8 (17.1), 3 x 520 x 14272 14.9 (33.8); with more, 128 x 2560 x 2560 9.5 (7.2).
enum GemmShape { G256X256, G160X256, G192X128, G64X64, G32X32 };
GemmShape gemm_shape(int64_t M, int64_t N, int64_t K) {
  const int64_t cus = device_cus();
  if (K > 3 * 32 * GEMM_KB && ((M + 31) / 32) * ((N + 31) / 32) <= cus) return G32X32;
  const auto rounds = [&](int bn, int bm) {
    return (double)((((M + bm - 1) / bm) * ((N + bn - 1) / bn) + cus - 1) / cus);
  };
  const double cost[4] = {rounds(256, 256) * 1.79, rounds(160, 256) * 1.66, rounds(192, 128) * 1.08,
                          rounds(64, 64) * 0.3 > 0.5 ? rounds(64, 64) * 0.3 : 0.5};
  int best = 0;
  for (int i = 1; i < 4; ++i)
    if (cost[i] < cost[best]) best = i;
  return (GemmShape)best;
}

template <int T>
int gemm_small(const Mx4GemmArgs& a) {
  const int64_t tiles_m = (a.M + 31) / 32;
  const unsigned grid = (unsigned)(tiles_m * ((a.N + 31) / 32));
  const int nc = (int)((a.K / 32 + GEMM_KB - 1) / GEMM_KB), waves = nc < SMALL_WAVES ? nc : SMALL_WAVES;
  dispatch_log("k_mx4_gemm_small", -1, a.N, a.K, (int)a.M, grid, 1, (unsigned)(64 * waves), SMALL_WAVES * 4096, "type=%d", T);
  auto* k = a.K % 128 == 0 ? k_mx4_gemm_small<T, true> : k_mx4_gemm_small<T, false>;
  hipLaunchKernelGGL(k, dim3(grid), dim3((unsigned)(64 * waves)), 0, a.stream, a.a_codes, a.a_scales, a.w_codes,
                     a.w_scales, a.y, a.M, a.N, (int)(a.K / 32), (uint32_t)tiles_m, waves);
  return (int)hipGetLastError();
}

template <int T>
int gemm_type(const Mx4GemmArgs& a) {
  switch (gemm_shape(a.M, a.N, a.K)) {
    case G256X256: return gemm_cfg<T, 4, 2, 2, 4>(a);
    case G160X256: return gemm_cfg<T, 1, 4, 5, 2>(a);
    case G192X128: return gemm_cfg<T, 2, 2, 3, 2>(a);
    case G32X32: return gemm_small<T>(a);
    default: return gemm_cfg<T, 2, 2, 1, 1>(a);
  }
}

}  // namespace

bool mx4_gemm_fits(int64_t M, int64_t N) {
  // Less than 2^32 threads in a grid: 512 for each 256 x 256 tile, and no more
  // for the same area of the others (up to 4096) while there are few tiles.
  return ((M + 255) / 256) * ((N + 255) / 256) <= 1 << 19;
}

int launch_mx4_gemm(const Mx4GemmArgs& a) {
  return a.type == KQ_F32 ? gemm_type<T_F32>(a) : a.type == KQ_F16 ? gemm_type<T_F16>(a) : gemm_type<T_BF16>(a);
}

}  // namespace kq
