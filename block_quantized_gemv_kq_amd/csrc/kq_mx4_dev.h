// kq_mx4_dev.h — device-side building blocks of the microscaled 4-bit kernels.
//
// A microscaled matrix is two planes: codes [R][K/2] (element 2i in the low
// nibble of byte i; sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5,
// 2, 3, 4, 6) and scales [R][K/32], one byte s per 32 elements of a row that
// stands for 2^(s-127) (255: NaN). The value of an element is code * scale.
//
// gfx950 converts pairs of codes to fp32, fp16 or bf16 with a scale in one
// instruction. Its scale operand is an fp32 whose exponent field is read, so
// s << 23 is the scale for every byte: 0 stands for 2^-127 and 255 gives NaN.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq_dev.h"

namespace kqd {

enum { T_F32 = 0, T_F16 = 1, T_BF16 = 2 };   // kq_type
template <int T> struct TypeSize { static constexpr int v = T == T_F32 ? 4 : 2; };

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef double v4d __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint32_t ld8(rsrc_t r, uint32_t off) {
  return (uint32_t)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(r, off, 0, 0);
}

// By value: this compiler takes element 0 for every element when a vector's
// element is bit-cast in place.
__device__ __forceinline__ float bits_f32(uint32_t v) { return __builtin_bit_cast(float, v); }

__device__ __forceinline__ float scale_of(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }

// fp32 value of a scale byte (NaN for 255), through the code of 1.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  const v2f one = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(0x22u, scale_of(byte), 0);
  return one[0];
}

// Eight codes (one dword) times their scale as bf16: exact as far as bf16
// reaches (4 times 2^126 and 2 times 2^127, scale bytes 253 and 254, do not fit).
__device__ __forceinline__ v8b codes_bf16(uint32_t d, float scale) {
  const v2b a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 0);
  const v2b b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 1);
  const v2b c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 2);
  const v2b e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 3);
  return v8b{a[0], a[1], b[0], b[1], c[0], c[1], e[0], e[1]};
}

// Eight codes times a quarter of their scale as bf16: exact for every scale
// byte (at most 1.5 * 2^127; the least, 2^-130, is a multiple of bf16's 2^-133).
__device__ __forceinline__ v8b codes_quarter_bf16(uint32_t d, uint32_t byte) {
  const float scale = scale_of(byte < 2u || byte == 255u ? byte : byte - 2u), rest = byte < 2u ? 0.25f : 1.0f;
  const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, scale, 0);
  const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, scale, 1);
  const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, scale, 2);
  const v2f e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, scale, 3);
  const float f[8] = {a[0] * rest, a[1] * rest, b[0] * rest, b[1] * rest, c[0] * rest, c[1] * rest, e[0] * rest, e[1] * rest};
  u32x4 h;   // the upper halves: a value has two significant bits
#pragma unroll
  for (int j = 0; j < 4; ++j)
    h[j] = perm(__builtin_bit_cast(uint32_t, f[2 * j + 1]), __builtin_bit_cast(uint32_t, f[2 * j]), 0x07060302u);
  return __builtin_bit_cast(v8b, h);
}

// Eight codes as fp16, unscaled (exact).
__device__ __forceinline__ v8h codes_f16(uint32_t d) {
  const v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 0);
  const v2h b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 1);
  const v2h c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 2);
  const v2h e = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 3);
  return v8h{a[0], a[1], b[0], b[1], c[0], c[1], e[0], e[1]};
}

// 4x4 transposition between the four 16-lane groups of a wave and the four
// dwords each lane holds: afterwards dword s of a lane in group g is dword g
// of the lane 16 s + (lane & 15). The swaps are written out with their wait
// states: the compiler does not track them through inline assembly.
__device__ __forceinline__ void transpose_groups(uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm("s_nop 1\n\t"
      "v_permlane32_swap_b32 %0, %2\n\t"
      "v_permlane32_swap_b32 %1, %3\n\t"
      "s_nop 1\n\t"
      "v_permlane16_swap_b32 %0, %1\n\t"
      "v_permlane16_swap_b32 %2, %3\n\t"
      "s_nop 1"
      : "+v"(a), "+v"(b), "+v"(c), "+v"(d));
}

// ---- The product of a weight tile with a few columns, one wave's share.
//
// v_mfma_f32_16x16x32 with the columns' values as its A operand and 16 weight
// rows as B: lane (r = lane & 15, g = lane >> 4) supplies column r and weight
// row r, and result element i of the lane is y[column 4 g + i][row r].
// K is walked in chunks of 128 (four blocks); a lane loads the 16 bytes of
// block 4c + g of its weight row, so a wave reads 64 contiguous bytes of each
// row per load.
//
// bf16 columns: the four matrix instructions of a chunk take dword s of every
// lane, so lane group g contributes elements 8s..8s+7 of block 4c + g, and the
// conversion applies each lane's own scale: the operand is the exact weight.
// The largest scales pass bf16: a wave that has met a scale byte of 192 or more
// (no weights in earnest have one) walks its chunks again, with a quarter of
// every weight and four times each chunk's sum. Compiled into the ordinary way
// it would take its registers (78 -> 128 for four column tiles). Looking for such
// bytes takes two instructions per chunk and tile: 19456 x 2560 at 64 bf16
// columns 25.7 and 25.3 us, at 64 fp32 columns 54.1 without and 55.5 with it.
// fp32 columns: the same with the value split into three bf16 pieces of eight
// bits each (24 in all: exact), three matrix instructions each.
// fp16 columns: bf16 cannot hold them and fp16 cannot hold the scales, so the
// codes go in unscaled and the scale multiplies each block's fp32 result; for
// that the codes are transposed among the lane groups first, and matrix
// instruction s covers the 32 elements of block 4c + s.
//
// The columns of a wave's K range come through LDS, in a region of the wave's
// own (no barrier): loads straight into the operand layout take four
// instructions per chunk and column tile whether its columns exist or not, each
// touching 16 rows (2560 x 9728 at 48 bf16 columns: 33 us, at any number of
// waves, against 15), here one instruction per KiB of real columns. A row of the
// region holds U chunks; its 16-byte piece p lies at p ^ (row & 7), so that
// the operand reads of eight consecutive rows touch every bank. Lanes whose
// column does not exist read an existing row: their results are never used.
template <int XT> struct Pieces { static constexpr int v = 8 * TypeSize<XT>::v; };   // of a row's chunk: 16 or 32

// LDS bytes of a wave's region for `rows` columns, U chunks at a time.
template <int XT, int U>
__host__ __device__ constexpr int x_region_bytes(int rows) { return (rows * Pieces<XT>::v * U + 63) / 64 * 1024; }

// Copy chunks c.. of `rows` columns into the region; off(row): byte offset of a
// column in rx. Pieces from `end` (counted along a column) on read zero.
template <int XT, int U, class Off>
__device__ __forceinline__ void stage_x(rsrc_t rx, uint8_t* xl, int rows, Off off, int c, int end) {
  constexpr int PR = Pieces<XT>::v * U;
  const int lane = threadIdx.x & 63;
  for (int first = 0; first < rows * PR; first += 64) {
    const int slot = first + lane, row = slot / PR;
    const int piece = c * Pieces<XT>::v + ((slot % PR) ^ (row & 7));
    const uint32_t o = off(row < rows ? row : 0) + 16u * (uint32_t)piece;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void_t*)(xl + first * 16), 16,
                                             row < rows && piece < end ? o : OOB, 0, 0, 0);
  }
}

// The weights come through LDS too, in the wave's region: a wave's lanes in
// operand order are 16 rows, and loads of 16 bytes each by lanes of different
// rows run at a quarter of the rate of loads whose neighbouring lanes take the
// pieces of one row (19456 x 2560 at one bf16 column: 7.8 us against 6.8; gate and
// up of 16 tokens of 128 experts: 40 against 31). Row
// r of tile t holds U chunks, its piece p at p ^ r (its low bits for U < 4);
// behind the codes, a dword of four scale bytes per row and chunk.
template <int RT, int U>
__host__ __device__ constexpr int w_region_bytes() { return RT * (U * 1024 + U * 64); }

// Chunks c .. c + U - 1 of a tile: codes to cl, scale bytes to sl. AL: rows hold
// whole chunks (K a multiple of 128), so a chunk's scale bytes are one aligned
// dword; otherwise it is put together from bytes. Blocks from `end` on read zero.
template <int U, bool AL>
__device__ __forceinline__ void stage_w(rsrc_t rc, rsrc_t rs, uint8_t* cl, uint8_t* sl, int c, int end, int nblk) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int slot = i * 64 + lane, row = slot / (4 * U), b = 4 * c + ((slot % (4 * U)) ^ (row & (4 * U - 1)));
    const uint32_t o = ((uint32_t)row * (uint32_t)nblk + (uint32_t)b) * 16u;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rc, (lds_void_t*)(cl + i * 1024), 16, b < end ? o : +OOB, 0, 0, 0);
  }
  const int row = lane / U, b = 4 * (c + lane % U);   // lanes past 16 U: rows past the tile
  const uint32_t o = (uint32_t)row * (uint32_t)nblk + (uint32_t)b;
  if constexpr (AL) {
    if (lane < 16 * U)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)sl, 4, b < end ? o : +OOB, 0, 0, 0);
  } else {
    uint32_t d = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) d |= ld8(rs, lane < 16 * U && b + k < end ? o + k : +OOB) << (8 * k);
    if (lane < 16 * U) reinterpret_cast<uint32_t*>(sl)[lane] = d;
  }
}

// bf16 pieces of eight fp32 values: each is the leading eight significant bits
// of what the earlier ones leave, so hi + mid + lo is the value (truncating
// keeps the largest finite values finite). An infinity goes into hi alone.
__device__ __forceinline__ void split3(const float (&x)[8], v8b& hi, v8b& mid, v8b& lo) {
  u32x4 h, m, l;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t b0[2], b1[2], b2[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float v = x[2 * j + k];
      b0[k] = __builtin_bit_cast(uint32_t, v);
      const float vh = __builtin_bit_cast(float, b0[k] & 0xffff0000u);
      const float r1 = v == vh ? 0.0f : v - vh;
      b1[k] = __builtin_bit_cast(uint32_t, r1);
      b2[k] = __builtin_bit_cast(uint32_t, r1 - __builtin_bit_cast(float, b1[k] & 0xffff0000u));
    }
    h[j] = perm(b0[1], b0[0], 0x07060302u);   // the upper halves of both
    m[j] = perm(b1[1], b1[0], 0x07060302u);
    l[j] = perm(b2[1], b2[0], 0x07060302u);
  }
  hi = __builtin_bit_cast(v8b, h);
  mid = __builtin_bit_cast(v8b, m);
  lo = __builtin_bit_cast(v8b, l);
}

// The bf16 pieces, the smallest first, of the eight bf16 or fp32 activations of
// step s that a lane of group g takes from its region row at piece `base` on.
template <int XT>
__device__ __forceinline__ void x_pieces(const uint8_t* xrow, int base, int swz, int g, int s, v8b (&x)[XT == T_F32 ? 3 : 1]) {
  if constexpr (XT == T_F32) {
    const v4f a = *reinterpret_cast<const v4f*>(xrow + (base + ((8 * g + 2 * s) ^ swz)) * 16);
    const v4f b = *reinterpret_cast<const v4f*>(xrow + (base + ((8 * g + 2 * s + 1) ^ swz)) * 16);
    const float f[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    split3(f, x[2], x[1], x[0]);
  } else {
    x[0] = *reinterpret_cast<const v8b*>(xrow + (base + ((4 * g + s) ^ swz)) * 16);
  }
}

// acc += the products of chunk u of the regions. xrow[t]: the region row of the
// lane's column in column tile t; swz: its row & 7, the same for every t.
// Bit 7 of a byte of `seen` is set where a scale byte has been 192 or more (bf16
// and fp32 columns).
template <int XT, int CT, int RT, int U>
__device__ __forceinline__ void chunk_products(const uint8_t* (&xrow)[CT], int swz, int u, const uint8_t* wl, int r, int g,
                                               v4f (&acc)[RT][CT], uint32_t& seen) {
  constexpr int XP = XT == T_F32 ? 3 : 1;
  const int base = u * Pieces<XT>::v;
  u32x4 codes[RT];
  uint32_t scale[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    codes[t] = *reinterpret_cast<const u32x4*>(wl + t * U * 1024 + (r * (4 * U) + ((4 * u + g) ^ (r & (4 * U - 1)))) * 16);
    scale[t] = *reinterpret_cast<const uint32_t*>(wl + RT * U * 1024 + t * U * 64 + (r * U + u) * 4);
  }
  if constexpr (XT == T_F16) {
    v8h x[4][CT];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int c = 0; c < CT; ++c) x[s][c] = *reinterpret_cast<const v8h*>(xrow[c] + (base + ((4 * s + g) ^ swz)) * 16);
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      uint32_t e[4] = {codes[t].x, codes[t].y, codes[t].z, codes[t].w};
      transpose_groups(e[0], e[1], e[2], e[3]);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const v8h wb = codes_f16(e[s]);
        const float sc = scale_value((scale[t] >> (8 * s)) & 255u);
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const v4f p = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[s][c], wb, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][c][i] = __builtin_fmaf(sc, p[i], acc[t][c][i]);
        }
      }
    }
  } else {
    float sc[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      sc[t] = scale_of((scale[t] >> (8 * g)) & 255u);
      seen |= scale[t] & (scale[t] << 1);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      v8b wb[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) wb[t] = codes_bf16(codes[t][s], sc[t]);
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        v8b x[XP];
        x_pieces<XT>(xrow[c], base, swz, g, s, x);
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int p = 0; p < XP; ++p) acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[p], wb[t], acc[t][c], 0, 0, 0);
      }
    }
  }
}

// Regions filled: this wave's copies have landed, and its LDS stores are done.
__device__ __forceinline__ void regions_filled() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory"); }
// Regions read: the next copies may take their place.
__device__ __forceinline__ void regions_read() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// acc += the products of the first n chunks of the regions, the way that fits
// every scale. Loops stay loops, one sum at a time, to take few registers.
template <int XT, int CT, int RT, int U>
__device__ __forceinline__ void large_products(const uint8_t* (&xrow)[CT], int swz, int n, const uint8_t* wl, int r, int g,
                                               v4f (&acc)[RT][CT]) {
  constexpr int XP = XT == T_F32 ? 3 : 1;
#pragma unroll 1
  for (int u = 0; u < n; ++u)
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const uint8_t* codes = wl + t * U * 1024 + (r * (4 * U) + ((4 * u + g) ^ (r & (4 * U - 1)))) * 16;
      const uint32_t byte = wl[RT * U * 1024 + t * U * 64 + (r * U + u) * 4 + g];
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        v4f quarter = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          __builtin_amdgcn_sched_barrier(0);
          const v8b wb = codes_quarter_bf16(*reinterpret_cast<const uint32_t*>(codes + 4 * s), byte);
          v8b x[XP];
          x_pieces<XT>(xrow[c], u * Pieces<XT>::v, swz, g, s, x);
#pragma unroll
          for (int p = 0; p < XP; ++p) quarter = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[p], wb, quarter, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][c][i] = __builtin_fmaf(4.0f, quarter[i], acc[t][c][i]);
      }
    }
}

// acc += the products of the first n (up to U) chunks of the filled regions.
template <bool LARGE, int XT, int CT, int RT, int U>
__device__ __forceinline__ void step_products(const uint8_t* (&xrow)[CT], int swz, int n, const uint8_t* wl, int r, int g,
                                              v4f (&acc)[RT][CT], uint32_t& seen) {
  if constexpr (LARGE && XT != T_F16) {
    large_products<XT, CT, RT, U>(xrow, swz, min(n, U), wl, r, g, acc);
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < n) chunk_products<XT, CT, RT, U>(xrow, swz, u, wl, r, g, acc, seen);
  }
}

template <bool L> struct Large { static constexpr bool value = L; };
// Whether the wave has to walk its chunks again (wave-uniform): see above.
template <int XT>
__device__ __forceinline__ bool again(uint32_t seen) {
  return XT != T_F16 && __builtin_amdgcn_ballot_w64((seen & 0x80808080u) != 0) != 0;
}

// acc = the products of chunks [c0, c1) (wave-uniform) with `rows` columns
// (1 to 16 CT). rc[t], rs[t]: the code and scale rows of tile t (rows past the
// matrix read zero); xl, wl: the wave's regions; off: see stage_x.
template <int XT, int CT, int RT, int U, bool AL, class Off>
__device__ __forceinline__ void mx4_tile(const rsrc_t (&rc)[RT], const rsrc_t (&rs)[RT], rsrc_t rx, uint8_t* xl,
                                         uint8_t* wl, int rows, Off off, int nblk, int c0, int c1,
                                         v4f (&acc)[RT][CT]) {
  constexpr int PR = Pieces<XT>::v * U;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const uint8_t* xrow[CT];
  int swz = 0;
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int row = 16 * c + r, have = row < rows ? row : rows > 7 ? row & 7 : 0;
    xrow[c] = xl + have * (PR * 16);
    if (c == 0) swz = have & 7;
  }
  const int end = min(c1 * Pieces<XT>::v, nblk * (Pieces<XT>::v / 4));
  const auto walk = [&](auto large) {
    uint32_t seen = 0;
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int u = 0; u < CT; ++u) acc[t][u] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int c = c0; c < c1; c += U) {
#pragma unroll
      for (int t = 0; t < RT; ++t)
        stage_w<U, AL>(rc[t], rs[t], wl + t * U * 1024, wl + RT * U * 1024 + t * U * 64, c, min(4 * c1, nblk), nblk);
      stage_x<XT, U>(rx, xl, rows, off, c, end);
      regions_filled();
      step_products<decltype(large)::value, XT, CT, RT, U>(xrow, swz, c1 - c, wl, r, g, acc, seen);
      regions_read();
    }
    return seen;
  };
  if (again<XT>(walk(Large<false>()))) walk(Large<true>());
}

// Rows [row0, row0 + rows) of the planes of a matrix as buffers.
__device__ __forceinline__ void mx4_rows(const uint8_t* codes, const uint8_t* scales, int64_t row0, int rows, int nblk,
                                         rsrc_t& rc, rsrc_t& rs) {
  rc = make_rsrc(codes + row0 * ((int64_t)nblk * 16), (uint32_t)rows * (uint32_t)nblk * 16u);
  rs = make_rsrc(scales + row0 * (int64_t)nblk, (uint32_t)rows * (uint32_t)nblk);
}

}  // namespace kqd
