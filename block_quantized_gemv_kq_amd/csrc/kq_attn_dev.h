// kq_attn_dev.h — what the two attention kernels share: operands from the
// cache's pages, the split of a weight into two 16-bit parts, the join of
// partial results.
//
// With t_j = scale * log2(e) * (q . k_j) over the keys a query sees, a walk keeps
// m = max t_j and l = sum 2^(t_j - m) in 32 bits and o = sum 2^(t_j - m) v_j in
// the matrix instructions' 32-bit sums; results of parts of the keys join as
// m = max m_i, l = sum 2^(m_i - m) l_i, o = sum 2^(m_i - m) o_i.
#pragma once

#include "kq_kv_dev.h"

namespace kqd {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

enum { A_F16 = 1, A_BF16 = 2 };   // kq_type of q and out

struct AttnArgs {
  Batch b;
  Cache c;
  Split w;
  const uint16_t* q;
  uint16_t* out;
  const uint64_t* tree;
  float* part;      // [slots][tile][D] o, not divided by l
  float2* ml;       // [slots][tile]
  int64_t ldq, ldo;
  float scale;      // scale * log2(e)
};

__device__ __forceinline__ v16f zero16() {
  v16f z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.0f;
  return z;
}
__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ uint32_t bits_of(float v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ float float_of(uint32_t v) { return __builtin_bit_cast(float, v); }

// The larger of v and lane ^ 32's v (permlane32 swap, written out as in add_lane_xor32).
__device__ __forceinline__ float max_lane_xor32(float v) {
  uint32_t x = bits_of(v), y = x;
  asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(x), "+v"(y));
  return fmaxf(float_of(x), float_of(y));
}

__device__ __forceinline__ float max_lane_xor16(float v) {
  uint32_t x = bits_of(v), y = x;
  asm volatile("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(x), "+v"(y));
  return fmaxf(float_of(x), float_of(y));
}

// What a column's weights 2^(t - m) are relative to: m is its largest t, for fp16
// weights SHIFT below it: weights are up to 2^15, so one that is a 2^-29th of the
// largest keeps all its bits, and one below a 2^-40th none. (With weights up to 1 in
// decode and 2^7 in prompts, keys with scores 14.9 below one other came out 0.1 to
// 0.6 % wrong, 21 below it 4 to 6 %.) Not where t is FAR from zero or further:
// nearer, m is off by at most 0.5 (two roundings) and no weight passes 2^15.5,
// which fp16 holds; there, the shift itself would be rounded.
template <int T> constexpr float SHIFT = T == A_F16 ? 15.0f : 0.0f;
constexpr float FAR = 0x1p22f;
template <int T>
__device__ __forceinline__ float lowered(float top) {
  return __builtin_fabsf(top) < FAR ? top - SHIFT<T> : top;
}

// A pair of fp32 as two 16-bit values of type T, nearest even.
template <int T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (T == A_F16) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, h2{(_Float16)a, (_Float16)b});
  } else {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, b2{(__bf16)a, (__bf16)b});
  }
}
template <int T>
__device__ __forceinline__ float low_half(uint32_t v) { return T == A_F16 ? h2f(v) : float_of(v << 16); }
template <int T>
__device__ __forceinline__ float high_half(uint32_t v) { return T == A_F16 ? h2f(v >> 16) : float_of(v & 0xffff0000u); }

// hi + lo = the pair to twice the type's bits (finite values; fp16 to 2^-25, which
// is fewer below 2^-3: see SHIFT).
template <int T>
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack2<T>(a, b);
  lo = pack2<T>(a - low_half<T>(hi), b - high_half<T>(hi));
}

template <int T>
__device__ __forceinline__ v4f mfma16(u32x4 a, u32x4 b, v4f c) {
  if constexpr (T == A_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
}
template <int T>
__device__ __forceinline__ v16f mfma32(u32x4 a, u32x4 b, v16f c) {
  if constexpr (T == A_F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
}

// a + b of a packed pair, added to c.
template <int T>
__device__ __forceinline__ float add_pair(uint32_t p, float c) {
  if constexpr (T == A_F16) {
    return dot2(p, ONES, c);
  } else {
    typedef short s2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, p), __builtin_bit_cast(b2, 0x3f803f80u), c, false);
  }
}

// Eight int8 codes as 16-bit values (exact in both types).
template <int T>
__device__ __forceinline__ u32x4 codes16(uint32_t c0, uint32_t c1) {
  u32x4 r;
  const uint32_t u[2] = {c0 ^ 0x80808080u, c1 ^ 0x80808080u};   // code + 128
  if constexpr (T == A_F16) {
    const half2_t off = {(_Float16)-1152.0f, (_Float16)-1152.0f};   // 1024 + 128 + code is exact in fp16
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, perm(MAGIC, u[i], SEL_LO)) + off);
      r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, perm(MAGIC, u[i], SEL_HI)) + off);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = (float)((u[i] >> (8 * j)) & 0xffu) - 128.0f;
      r[2 * i] = perm(bits_of(f[1]), bits_of(f[0]), 0x07060302u);       // the upper halves: 8 bits are exact there
      r[2 * i + 1] = perm(bits_of(f[3]), bits_of(f[2]), 0x07060302u);
    }
  }
  return r;
}

// Eight int8 codes as 16-bit values of code + BIAS, exact: fp16 1024 + (code +
// 128) by its bits, bf16 code + 128.
template <int T> struct Bias { static constexpr float v = T == A_F16 ? 1152.0f : 128.0f; };
template <int T>
__device__ __forceinline__ u32x4 biased16(uint32_t c0, uint32_t c1) {
  u32x4 r;
  const uint32_t u[2] = {c0 ^ 0x80808080u, c1 ^ 0x80808080u};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (T == A_F16) {
      r[2 * i] = perm(MAGIC, u[i], SEL_LO);
      r[2 * i + 1] = perm(MAGIC, u[i], SEL_HI);
    } else {
      float f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = (float)((u[i] >> (8 * j)) & 0xffu);
      r[2 * i] = perm(bits_of(f[1]), bits_of(f[0]), 0x07060302u);   // the upper halves: 8 bits are exact there
      r[2 * i + 1] = perm(bits_of(f[3]), bits_of(f[2]), 0x07060302u);
    }
  }
  return r;
}
// Eight equal 16-bit values.
template <int T>
__device__ __forceinline__ u32x4 splat16(float v) {
  const uint32_t p = pack2<T>(v, v);
  return u32x4{p, p, p, p};
}

// Where a 16-bit element is infinite or NaN.
template <int T>
__device__ __forceinline__ bool any_not_finite(u32x4 v) {
  constexpr uint32_t E = T == A_F16 ? 0x7c00u : 0x7f80u;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) bad |= (v[i] & E) == E || (v[i] & E << 16) == E << 16;
  return bad;
}
// The finite elements of v; plus and minus get 1 where it is +infinity or NaN,
// and where it is -infinity or NaN.
template <int T>
__device__ __forceinline__ u32x4 take_finite(u32x4 v, u32x4& plus, u32x4& minus) {
  constexpr uint32_t E = T == A_F16 ? 0x7c00u : 0x7f80u, ONE = T == A_F16 ? 0x3c00u : 0x3f80u;
  u32x4 r = {0u, 0u, 0u, 0u};
  plus = minus = r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t e = (v[i] >> (16 * h)) & 0xffffu, mag = e & 0x7fffu;
      if (mag < E) r[i] |= e << (16 * h);
      if (mag > E || (mag == E && e == mag)) plus[i] |= ONE << (16 * h);
      if (mag > E || (mag == E && e != mag)) minus[i] |= ONE << (16 * h);
    }
  return r;
}

// Eight 16-bit elements of a row; 16-byte loads where rows allow it.
__device__ __forceinline__ u32x4 row_piece(const uint16_t* p, bool wide) {
  if (wide) return *reinterpret_cast<const u32x4*>(p);
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (uint32_t)p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
  return r;
}
__device__ __forceinline__ bool wide_rows(const void* p, int64_t ld) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * 2)) & 15) == 0;
}
// Four elements of an output row.
template <int T>
__device__ __forceinline__ void put_4(uint16_t* p, bool wide, v4f v) {
  const uint32_t a = pack2<T>(v[0], v[1]), b = pack2<T>(v[2], v[3]);
  if (wide) {
    *reinterpret_cast<u32x2v*>(p) = u32x2v{a, b};
  } else {
    p[0] = (uint16_t)a;
    p[1] = (uint16_t)(a >> 16);
    p[2] = (uint16_t)b;
    p[3] = (uint16_t)(b >> 16);
  }
}

}  // namespace kqd

namespace kq {
kqd::AttnArgs attn_args(const AttnCall& p, const AttnPlan& w);
void finish_plan(const kq_kv_cache& c, const kq_kv_batch& b, int heads, AttnPlan& w);
// Joins the partial results of split tiles (kq_attn.hip).
int launch_attn_join(const kqd::AttnArgs& a, int type, int D, hipStream_t stream);
int launch_attn_join_tiles(const kqd::AttnArgs& a, int type, int D, hipStream_t stream);
}  // namespace kq
