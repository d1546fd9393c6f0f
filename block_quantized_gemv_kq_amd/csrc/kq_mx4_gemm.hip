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
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq_internal.h"
#include "kq_mx4_dev.h"

namespace kqd {

constexpr int GEMM_KB = 8;   // blocks of 32 per K tile: 128 bytes of codes per row

// Copy ROWS x 128 bytes of codes (K tile kt) to LDS: 16-byte piece p of row r
// sits at slot 8 r + (p ^ (r & 7)), so that eight consecutive rows read at one
// piece cover every bank. Pieces past the row's end or the matrix read zero.
template <int ROWS, int THREADS>
__device__ __forceinline__ void stage_codes(rsrc_t rc, uint8_t* lds, int kt, int nblk) {
  const int lane = threadIdx.x & 63, wave = wave_id();
#pragma unroll
  for (int i = 0; i < ROWS * 8 / THREADS; ++i) {
    const int first = (i * (THREADS / 64) + wave) * 64;   // first slot of this wave's copy
    const int slot = first + lane, r = slot >> 3, p = (slot & 7) ^ (r & 7);
    const int b = kt * GEMM_KB + p;
    const uint32_t off = b < nblk ? ((uint32_t)r * (uint32_t)nblk + (uint32_t)b) * 16u : OOB;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rc, (lds_void_t*)(lds + first * 16), 16, off, 0, 0, 0);
  }
}

// The four scale bytes of blocks 8 kt + 4 h .. + 3 of row r.
template <bool AL>
__device__ __forceinline__ uint32_t load_scales(rsrc_t rs, int r, int kt, int h, int nblk) {
  const int b = kt * GEMM_KB + 4 * h;
  const uint32_t o = (uint32_t)r * (uint32_t)nblk + (uint32_t)b;
  if constexpr (AL) return ld32(rs, b < nblk ? o : OOB);
  uint32_t d = 0;
#pragma unroll
  for (int s = 0; s < 4; ++s) d |= ld8(rs, b + s < nblk ? o + s : OOB) << (8 * s);
  return d;
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

// A workgroup of WN x WM waves computes BN weight rows x BM activation rows;
// each wave TN x TM tiles of 32 x 32. Two K tiles in LDS: the copies of the
// next are in flight while this one is multiplied, one barrier per K tile.
template <int T, int WN, int WM, int TN, int TM, bool AL>
__global__ __launch_bounds__(64 * WN * WM) void k_mx4_gemm(const uint8_t* __restrict__ ac, const uint8_t* __restrict__ as,
                                                          const uint8_t* __restrict__ wc, const uint8_t* __restrict__ ws,
                                                          void* __restrict__ y, int64_t M, int64_t N, int nblk,
                                                          uint32_t tiles_m) {
  constexpr int BN = 32 * WN * TN, BM = 32 * WM * TM, THREADS = 64 * WN * WM;
  extern __shared__ uint8_t lds[];   // two of (BN + BM) * 128 bytes
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int r = lane & 31, h = lane >> 5;
  const int wn = (wave % WN) * 32 * TN, wm = (wave / WN) * 32 * TM;
  const uint32_t tn = blockIdx.x / tiles_m, tm = blockIdx.x - tn * tiles_m;
  const int64_t n0 = (int64_t)tn * BN, m0 = (int64_t)tm * BM;
  const int rows_n = (int)min<int64_t>(BN, N - n0), rows_m = (int)min<int64_t>(BM, M - m0);
  rsrc_t rwc, rws, rac, ras;
  mx4_rows(wc, ws, n0, rows_n, nblk, rwc, rws);
  mx4_rows(ac, as, m0, rows_m, nblk, rac, ras);
  v16f acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.0f;
  const int nkt = (nblk + GEMM_KB - 1) / GEMM_KB;
  uint32_t sw[TN], sa[TM], swn[TN], san[TM];
  stage_codes<BN, THREADS>(rwc, lds, 0, nblk);
  stage_codes<BM, THREADS>(rac, lds + BN * 128, 0, nblk);
#pragma unroll
  for (int i = 0; i < TN; ++i) swn[i] = load_scales<AL>(rws, wn + 32 * i + r, 0, h, nblk);
#pragma unroll
  for (int j = 0; j < TM; ++j) san[j] = load_scales<AL>(ras, wm + 32 * j + r, 0, h, nblk);
  for (int kt = 0; kt < nkt; ++kt) {
    uint8_t* cur = lds + (kt & 1) * ((BN + BM) * 128);
    uint8_t* nxt = lds + ((kt + 1) & 1) * ((BN + BM) * 128);
#pragma unroll
    for (int i = 0; i < TN; ++i) sw[i] = swn[i];
#pragma unroll
    for (int j = 0; j < TM; ++j) sa[j] = san[j];
    // This tile's copies have landed (a barrier alone does not wait for them:
    // they are loads to the compiler), and every wave has read the other buffer.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (kt + 1 < nkt) {
      stage_codes<BN, THREADS>(rwc, nxt, kt + 1, nblk);
      stage_codes<BM, THREADS>(rac, nxt + BN * 128, kt + 1, nblk);
#pragma unroll
      for (int i = 0; i < TN; ++i) swn[i] = load_scales<AL>(rws, wn + 32 * i + r, kt + 1, h, nblk);
#pragma unroll
      for (int j = 0; j < TM; ++j) san[j] = load_scales<AL>(ras, wm + 32 * j + r, kt + 1, h, nblk);
    }
    const uint8_t* lw = cur + (wn + r) * 128;
    const uint8_t* la = cur + BN * 128 + (wm + r) * 128;
#define KQ_STEP(S)                                                                                              \
  {                                                                                                             \
    const int p = ((4 * h + S) ^ (r & 7)) * 16;                                                                 \
    u32x4 fw[TN], fa[TM];                                                                                       \
    _Pragma("unroll") for (int i = 0; i < TN; ++i) fw[i] = *reinterpret_cast<const u32x4*>(lw + i * 4096 + p);  \
    _Pragma("unroll") for (int j = 0; j < TM; ++j) fa[j] = *reinterpret_cast<const u32x4*>(la + j * 4096 + p);  \
    _Pragma("unroll") for (int i = 0; i < TN; ++i)                                                              \
      _Pragma("unroll") for (int j = 0; j < TM; ++j) acc[i][j] = mfma_fp4<S>(fw[i], fa[j], acc[i][j], sw[i], sa[j]); \
  }
    KQ_STEP(0)
    KQ_STEP(1)
    KQ_STEP(2)
    KQ_STEP(3)
#undef KQ_STEP
  }
  // The stores below are conditional; a matrix instruction moved into such a
  // branch would read registers that its idle lanes never wrote.
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) asm volatile("" : "+v"(acc[i][j]));
  typedef typename OutT<T>::t out_t;
  out_t* yo = static_cast<out_t*>(y);
  const bool whole = (N & 3) == 0;   // then four consecutive n of a row are aligned together
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int64_t m = m0 + wm + 32 * j + r;
    if (m >= M) continue;
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t n = n0 + wn + 32 * i + 8 * q + 4 * h;
        out_t* p = yo + m * N + n;
        typedef out_t out4 __attribute__((ext_vector_type(4)));
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

}  // namespace kqd

namespace kq {

using namespace kqd;

namespace {

template <int T, int WN, int WM, int TN, int TM>
int gemm_cfg(const Mx4GemmArgs& a) {
  constexpr int BN = 32 * WN * TN, BM = 32 * WM * TM;
  const int64_t tiles_m = (a.M + BM - 1) / BM, tiles_n = (a.N + BN - 1) / BN;
  const unsigned grid = (unsigned)(tiles_m * tiles_n);
  const size_t lds = 2 * (BN + BM) * 128;
  dispatch_log("k_mx4_gemm", -1, a.N, a.K, (int)a.M, grid, 1, 64 * WN * WM, lds, "type=%d tile=%dx%d", T, BN, BM);
  const bool al = a.K % 128 == 0;
  auto* k = al ? k_mx4_gemm<T, WN, WM, TN, TM, true> : k_mx4_gemm<T, WN, WM, TN, TM, false>;
  hipLaunchKernelGGL(k, dim3(grid), dim3(64 * WN * WM), lds, a.stream, a.a_codes, a.a_scales, a.w_codes, a.w_scales,
                     a.y, a.M, a.N, (int)(a.K / 32), (uint32_t)tiles_m);
  return (int)hipGetLastError();
}

template <int T>
int gemm_type(const Mx4GemmArgs& a) {
  const int64_t big = ((a.M + 255) / 256) * ((a.N + 255) / 256);
  if (big >= 128) return gemm_cfg<T, 2, 4, 4, 2>(a);     // 256 x 256
  return gemm_cfg<T, 2, 2, 1, 1>(a);                      // 64 x 64
}

}  // namespace

bool mx4_gemm_fits(int64_t M, int64_t N) {
  // 512 threads for each 256 x 256 tile, and less than 2^32 threads in a grid
  return ((M + 255) / 256) * ((N + 255) / 256) <= 1 << 22;
}

int launch_mx4_gemm(const Mx4GemmArgs& a) {
  return a.type == KQ_F32 ? gemm_type<T_F32>(a) : a.type == KQ_F16 ? gemm_type<T_F16>(a) : gemm_type<T_BF16>(a);
}

}  // namespace kq
