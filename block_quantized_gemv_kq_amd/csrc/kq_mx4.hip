// kq_mx4.hip — microscaled 4-bit matrices: quantising, dequantising, and the
// product with a few activation columns (decode and verify passes).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq_internal.h"
#include "kq_mx4_dev.h"

namespace kqd {

// Eight consecutive values of type T at p as fp32 (exact). VEC: p is aligned
// for 16-byte loads.
template <int T, bool VEC>
__device__ __forceinline__ void load8(const void* p, float (&f)[8]) {
  if constexpr (T == T_F32) {
    const float* q = static_cast<const float*>(p);
    if constexpr (VEC) {
      const v4f a = *reinterpret_cast<const v4f*>(q), b = *reinterpret_cast<const v4f*>(q + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = a[j], f[4 + j] = b[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = q[j];
    }
  } else {
    uint16_t h[8];
    const uint16_t* q = static_cast<const uint16_t*>(p);
    if constexpr (VEC) {
      const u32x4 a = *reinterpret_cast<const u32x4*>(q);
#pragma unroll
      for (int j = 0; j < 4; ++j) h[2 * j] = (uint16_t)a[j], h[2 * j + 1] = (uint16_t)(a[j] >> 16);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = q[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      f[j] = T == T_F16 ? (float)__builtin_bit_cast(_Float16, h[j]) : __builtin_bit_cast(float, (uint32_t)h[j] << 16);
  }
}

// Quantise: four lanes per block of 32, eight values each. The scale byte is
// the exponent field of the block's largest magnitude less two, not below
// zero: floor(log2(amax)) - 2 with the bias of 127, so the largest value lands
// in [4, 8) (a denormal or zero amax gives byte 0). The conversion instruction
// divides by the scale exactly, rounds to the nearest code (even on ties) and
// saturates at 6. Magnitudes are compared as integers, which orders NaN above
// infinity above every number, so one comparison finds a block that has any.
// Bound by memory: 19456 x 2560 fp32 in 46 us, 4.9 TB/s read and written (a large
// copy reaches 4.8); 16 x 2560 is a launch, 2.0 us.
template <int T, bool VEC>
__global__ __launch_bounds__(256) void k_mx4_quantize(const uint8_t* __restrict__ x, int64_t ldx_bytes,
                                                      uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                      int64_t row_groups, uint32_t chunks) {
  const uint32_t row = blockIdx.x / chunks, chunk = blockIdx.x - row * chunks;
  const int64_t i = (int64_t)chunk * 256 + threadIdx.x;   // group of eight values within the row
  if (i >= row_groups) return;                            // whole blocks leave together (row_groups % 4 == 0)
  float f[8];
  load8<T, VEC>(x + (int64_t)row * ldx_bytes + i * (8 * TypeSize<T>::v), f);
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = max(amax, __builtin_bit_cast(uint32_t, f[j]) & 0x7fffffffu);
  amax = max(amax, (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, 0xB1, 0xF, 0xF, true));   // lane ^ 1
  amax = max(amax, (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, 0x4E, 0xF, 0xF, true));   // lane ^ 2
  const bool finite = amax < 0x7f800000u;
  const uint32_t e = amax >> 23;
  const uint32_t s = finite ? (e > 2u ? e - 2u : 0u) : 255u;
  const float sc = scale_of(finite ? s : 127u);
  uint32_t d = 0;
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, f[0], f[1], sc, 0);
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, f[2], f[3], sc, 1);
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, f[4], f[5], sc, 2);
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, f[6], f[7], sc, 3);
  const int64_t o = (int64_t)row * row_groups + i;
  reinterpret_cast<uint32_t*>(codes)[o] = finite ? d : 0u;
  if ((threadIdx.x & 3) == 0) scales[o >> 2] = (uint8_t)s;
}

// Dequantise: eight values per lane, each code times its scale rounded to T
// (exact in fp32 and bf16 up to their largest finite value). Bound by memory:
// 19456 x 2560 to bf16 in 19 us, 6.6 TB/s (part of it stays in the last cache).
template <int T, bool VEC>
__global__ __launch_bounds__(256) void k_mx4_dequantize(const uint8_t* __restrict__ codes,
                                                        const uint8_t* __restrict__ scales, uint8_t* __restrict__ out,
                                                        int64_t ldo_bytes, int64_t row_groups, uint32_t chunks) {
  const uint32_t row = blockIdx.x / chunks, chunk = blockIdx.x - row * chunks;
  const int64_t i = (int64_t)chunk * 256 + threadIdx.x;
  if (i >= row_groups) return;
  const int64_t o = (int64_t)row * row_groups + i;
  const uint32_t d = reinterpret_cast<const uint32_t*>(codes)[o];
  const float sc = scale_of(scales[o >> 2]);
  uint8_t* p = out + (int64_t)row * ldo_bytes + i * (8 * TypeSize<T>::v);
  if constexpr (T == T_BF16) {
    const v8b v = codes_bf16(d, sc);
    if constexpr (VEC) {
      *reinterpret_cast<v8b*>(p) = v;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) reinterpret_cast<__bf16*>(p)[j] = v[j];
    }
  } else {
    float f[8];
    const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, sc, 0);
    const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, sc, 1);
    const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, sc, 2);
    const v2f e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, sc, 3);
    f[0] = a[0], f[1] = a[1], f[2] = b[0], f[3] = b[1], f[4] = c[0], f[5] = c[1], f[6] = e[0], f[7] = e[1];
    if constexpr (T == T_F32) {
      if constexpr (VEC) {
        reinterpret_cast<v4f*>(p)[0] = v4f{f[0], f[1], f[2], f[3]};
        reinterpret_cast<v4f*>(p)[1] = v4f{f[4], f[5], f[6], f[7]};
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) reinterpret_cast<float*>(p)[j] = f[j];
      }
    } else {
      v8h v;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (_Float16)f[j];
      if constexpr (VEC) {
        *reinterpret_cast<v8h*>(p) = v;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) reinterpret_cast<_Float16*>(p)[j] = v[j];
      }
    }
  }
}

// Buffers of RT tiles of 16 weight rows from row0 on (rows past N read zero).
template <int RT>
__device__ __forceinline__ void mx4_tiles(const uint8_t* codes, const uint8_t* scales, int64_t row0, int N, int nblk,
                                          rsrc_t (&rc)[RT], rsrc_t (&rs)[RT]) {
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int64_t left = (int64_t)N - row0 - 16 * t;
    const int rows = left < 0 ? 0 : left < 16 ? (int)left : 16;
    mx4_rows(codes, scales, rows ? row0 + 16 * t : 0, rows, nblk, rc[t], rs[t]);
  }
}

// The waves' partial sums, added in wave order, to y.
template <int RT, int CT>
__device__ __forceinline__ void store_sums(const v4f (&acc)[RT][CT], v4f* red, int wave, int waves,
                                           float* __restrict__ y, int64_t row0, int N, int M) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int u = 0; u < CT; ++u) red[((wave * RT + t) * CT + u) * 64 + lane] = acc[t][u];
  __syncthreads();
  for (int i = threadIdx.x; i < RT * CT * 64; i += 64 * waves) {
    v4f s = red[i];
    for (int w = 1; w < waves; ++w) s += red[w * (RT * CT * 64) + i];
    const int l = i & 63, u = (i >> 6) % CT, t = (i >> 6) / CT;
    const int64_t n = row0 + 16 * t + (l & 15);
    if (n >= N) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = 16 * u + 4 * (l >> 4) + j;
      if (m < M) y[(int64_t)m * N + n] = s[j];
    }
  }
}

// y[m][n] for RT tiles of 16 weight rows and up to 16 CT columns. The waves of
// a workgroup share the rows and split K; their partial sums meet in LDS and
// are added in wave order. Grid y: groups of 16 CT columns. Dynamic LDS: waves *
// (the columns' and the weights' regions), then (CT 1) or in their place (CT >
// 1) waves * RT * CT KiB of partial sums. One column is bound by memory and the
// launch (19456 x 2560, bf16: 26.5 MB in 6.9 us, 7.3 where none of it is in the last
// cache; a kernel that only reads it takes 5.3); many columns by what each
// workgroup brings through LDS, a byte of it written and read once at 64 bytes a
// clock (2560 x 9728 at 48: 15 us, 33000 clocks, of which reads and writes take
// 16000 each).
template <int XT, int CT, int RT, int U, bool AL>
__global__ __launch_bounds__(1024) void k_mx4_gemv(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                   const void* __restrict__ x, float* __restrict__ y, int N, int K,
                                                   int M, int waves) {
  extern __shared__ u32x4 lds4[];
  uint8_t* lds = reinterpret_cast<uint8_t*>(lds4);
  const int wave = wave_id();
  const int nblk = K / 32, nchunk = (nblk + 3) / 4;
  const int64_t row0 = (int64_t)blockIdx.x * (16 * RT);
  rsrc_t rc[RT], rs[RT];
  mx4_tiles<RT>(codes, scales, row0, N, nblk, rc, rs);
  const uint32_t xrow = (uint32_t)K * TypeSize<XT>::v;
  const rsrc_t rx = make_rsrc(x, (uint32_t)M * xrow);
  v4f acc[RT][CT];
  const int c0 = nchunk * wave / waves, c1 = nchunk * (wave + 1) / waves;
  const int m0 = (int)blockIdx.y * (16 * CT);
  const int cols = min(M - m0, 16 * CT), xbytes = x_region_bytes<XT, U>(min(M, 16 * CT)), region = xbytes + w_region_bytes<RT, U>();
  uint8_t* xl = lds + wave * region;
  mx4_tile<XT, CT, RT, U, AL>(rc, rs, rx, xl, xl + xbytes, cols,
                              [=](int row) { return (uint32_t)(m0 + row) * xrow; }, nblk, c0, c1, acc);
  if constexpr (CT > 1) __syncthreads();   // every wave has read its region
  store_sums<RT, CT>(acc, reinterpret_cast<v4f*>(lds + (CT == 1 ? waves * region : 0)), wave, waves, y + (int64_t)m0 * N, row0, N, cols);
}

}  // namespace kqd

namespace kq {

using namespace kqd;

namespace {

// Rows as the kernels walk them: contiguous rows are one long row.
struct Walk {
  int64_t rows, groups;
  bool contiguous;
};
Walk walk_of(int64_t R, int64_t K, int64_t ld) {
  return ld == K ? Walk{1, R * K / 8, true} : Walk{R, K / 8, false};
}
int64_t blocks_of(int64_t rows, int64_t groups) { return rows * ((groups + 255) / 256); }

// A grid has less than 2^32 threads: contiguous rows of more than 2^34 elements
// (8 a thread, half of what would fit) are several launches, one after another.
constexpr int64_t PIECE_GROUPS = (int64_t)1 << 31;

// launch(first group, groups, blocks) for each piece; the first error ends it.
template <class Launch>
int each_piece(const Walk& w, Launch launch) {
  const int64_t step = w.contiguous ? PIECE_GROUPS : w.groups;
  for (int64_t first = 0; first < w.groups; first += step) {
    const int64_t groups = w.groups - first < step ? w.groups - first : step;
    const int err = launch(first, groups, (unsigned)blocks_of(w.rows, groups));
    if (err) return err;
  }
  return 0;
}

}  // namespace

bool mx4_walk_fits(int64_t R, int64_t K, int64_t ld) {
  const Walk w = walk_of(R, K, ld);
  return w.contiguous || blocks_of(w.rows, w.groups) <= 0xffffffffll / 256;
}

int launch_mx4_quantize(int type, const void* x, int64_t ldx, void* codes, void* scales, int64_t R, int64_t K,
                        hipStream_t stream) {
  const Walk w = walk_of(R, K, ldx);
  const int size = type == KQ_F32 ? 4 : 2;
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && (w.rows == 1 || ldx * size % 16 == 0);
  return each_piece(w, [&](int64_t first, int64_t groups, unsigned blocks) {
    dispatch_log("k_mx4_quantize", -1, R, K, 0, blocks, 1, 256, 0, "type=%d vec=%d", type, (int)vec);
#define KQ_LAUNCH(T, V)                                                                                        \
  hipLaunchKernelGGL((k_mx4_quantize<T, V>), dim3(blocks), dim3(256), 0, stream,                               \
                     static_cast<const uint8_t*>(x) + first * 8 * size, ldx* size,                             \
                     static_cast<uint8_t*>(codes) + first * 4, static_cast<uint8_t*>(scales) + first / 4, groups, \
                     (uint32_t)((groups + 255) / 256))
    if (type == KQ_F32) { if (vec) KQ_LAUNCH(T_F32, true); else KQ_LAUNCH(T_F32, false); }
    else if (type == KQ_F16) { if (vec) KQ_LAUNCH(T_F16, true); else KQ_LAUNCH(T_F16, false); }
    else { if (vec) KQ_LAUNCH(T_BF16, true); else KQ_LAUNCH(T_BF16, false); }
#undef KQ_LAUNCH
    return (int)hipGetLastError();
  });
}

int launch_mx4_dequantize(const void* codes, const void* scales, int type, void* out, int64_t ldo, int64_t R,
                          int64_t K, hipStream_t stream) {
  const Walk w = walk_of(R, K, ldo);
  const int size = type == KQ_F32 ? 4 : 2;
  const bool vec = (reinterpret_cast<uintptr_t>(out) & 15) == 0 && (w.rows == 1 || ldo * size % 16 == 0);
  return each_piece(w, [&](int64_t first, int64_t groups, unsigned blocks) {
    dispatch_log("k_mx4_dequantize", -1, R, K, 0, blocks, 1, 256, 0, "type=%d vec=%d", type, (int)vec);
#define KQ_LAUNCH(T, V)                                                                                        \
  hipLaunchKernelGGL((k_mx4_dequantize<T, V>), dim3(blocks), dim3(256), 0, stream,                             \
                     static_cast<const uint8_t*>(codes) + first * 4, static_cast<const uint8_t*>(scales) + first / 4, \
                     static_cast<uint8_t*>(out) + first * 8 * size, ldo* size, groups, (uint32_t)((groups + 255) / 256))
    if (type == KQ_F32) { if (vec) KQ_LAUNCH(T_F32, true); else KQ_LAUNCH(T_F32, false); }
    else if (type == KQ_F16) { if (vec) KQ_LAUNCH(T_F16, true); else KQ_LAUNCH(T_F16, false); }
    else { if (vec) KQ_LAUNCH(T_BF16, true); else KQ_LAUNCH(T_BF16, false); }
#undef KQ_LAUNCH
    return (int)hipGetLastError();
  });
}

namespace {

constexpr int LDS_BYTES = 160 * 1024;   // of a compute unit

// Waves of a workgroup, one batch of loads each while LDS lasts, and its LDS.
template <int XT, int CT, int RT, int U>
int gemv_waves(const Mx4GemvArgs& a, int* lds) {
  const int nchunk = (int)((a.K / 32 + 3) / 4);
  const int region = x_region_bytes<XT, U>(a.M < 16 * CT ? a.M : 16 * CT) + w_region_bytes<RT, U>(), sums = RT * CT * 1024;
  const int per_wave = CT == 1 ? region + sums : region > sums ? region : sums;
  int waves = (nchunk + U - 1) / U;
  const int most = LDS_BYTES / per_wave < 16 ? LDS_BYTES / per_wave : 16;
  waves = waves > most ? most : waves;
  *lds = waves * per_wave;
  return waves;
}

template <int XT, int CT, int RT, int U>
int gemv_cfg(const Mx4GemvArgs& a) {
  int bytes;
  const int waves = gemv_waves<XT, CT, RT, U>(a, &bytes);
  const unsigned grid = (unsigned)((a.N + 16 * RT - 1) / (16 * RT));
  const unsigned parts = (unsigned)((a.M + 16 * CT - 1) / (16 * CT));
  const size_t lds = (size_t)bytes;
  dispatch_log("k_mx4_gemv", -1, a.N, a.K, a.M, grid, parts, (unsigned)(64 * waves), lds, "type=%d ct=%d rt=%d u=%d", XT, CT, RT, U);
  auto* k = a.K % 128 == 0 ? k_mx4_gemv<XT, CT, RT, U, true> : k_mx4_gemv<XT, CT, RT, U, false>;
  hipLaunchKernelGGL(k, dim3(grid, parts), dim3(64 * waves), lds, a.stream, a.codes, a.scales, a.x, a.y, (int)a.N, (int)a.K,
                     a.M, waves);
  return (int)hipGetLastError();
}

// bf16 and fp16 columns. More than 16 are most of what a workgroup reads, so a
// workgroup takes them all, and two row tiles where that leaves a workgroup per
// compute unit (19456 x 2560 at 48 bf16 columns: 21.6 us against 27.2 with one
// tile and 41 with 16 columns each; 8192 x 4096 at 32: 9.8 against 12.9; 2560 x
// 9728 at 48: 17.8 against 14.9; the rule's edge is late: 6144 x 2560 at 32, 48 and
// 64 7.1, 8.0 and 9.8 with two, 10.4, 11.2 and 15.6 with one). Nine to 16 columns
// take two tiles from 384 tiles on, unless a compute unit's LDS holds two
// workgroups of one (6144 x 2560 at 16 bf16 columns: 4.7 us against 6.5, 19456 x
// 2560 12.5 against 15.5; but 19456 x 2048 at nine, where it does, 11.0 against
// 9.6, fp16 12.8 against 10.0, and 12288 x 1024 at 16 4.7 against 4.6). That is
// less sure where the tiles fill the compute units just past a whole number of
// times: 12288 x 4096 at nine fp16 columns 13.3 against 12.4.
// Where the row tiles are few, groups of columns go to workgroups of their own
// as far as the compute units take them at once (1000 x 14080 at 64 fp16
// columns: 13.4 us against 31.5).
template <int XT, int CT>
int gemv_wide(const Mx4GemvArgs& a) {
  if (a.N >= 32 * 256) return gemv_cfg<XT, CT, 2, 1>(a);
  return gemv_cfg<XT, CT, 1, 1>(a);
}

template <int XT>
int gemv_half(const Mx4GemvArgs& a) {
  const int64_t tiles = (a.N + 15) / 16, parts = (a.M + 15) / 16;
  if (a.M <= 8) return gemv_cfg<XT, 1, 1, 4>(a);
  if (a.M <= 16 && tiles >= 384) {
    int one;   // LDS of a workgroup of one tile
    gemv_waves<XT, 1, 1, 2>(a, &one);
    if (2 * one > LDS_BYTES) return gemv_cfg<XT, 1, 2, 2>(a);
  }
  if (a.M <= 16 || tiles * parts <= 256) return gemv_cfg<XT, 1, 1, 2>(a);
  if (a.M <= 32 || tiles * ((parts + 1) / 2) <= 256) return gemv_wide<XT, 2>(a);
  return a.M <= 48 ? gemv_wide<XT, 3>(a) : gemv_wide<XT, 4>(a);
}

// fp32 columns. Splitting them into pieces is the work: row tiles share it, as
// many as leave the compute units about one workgroup each, and columns past 16
// go to other workgroups (11000 x 4096 at 64 columns: 45 us with four tiles, 91
// with one, 122 with one of all columns; 2551 x 12000 at 36: 30 with two, 40, 43
// and 55).
int gemv_f32(const Mx4GemvArgs& a) {
  const int64_t groups = (a.N + 15) / 16 * ((a.M + 15) / 16);
  if (groups >= 4 * 192) return gemv_cfg<T_F32, 1, 4, 1>(a);
  if (groups >= 2 * 192) return gemv_cfg<T_F32, 1, 2, 1>(a);
  return gemv_cfg<T_F32, 1, 1, 1>(a);
}

}  // namespace

int launch_mx4_gemv(const Mx4GemvArgs& a) {
  return a.type == KQ_F32 ? gemv_f32(a) : a.type == KQ_F16 ? gemv_half<T_F16>(a) : gemv_half<T_BF16>(a);
}

}  // namespace kq
