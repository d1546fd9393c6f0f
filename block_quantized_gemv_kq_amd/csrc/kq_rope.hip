// kq_rope.hip — rotary positions, and the write of new tokens into the paged
// key-value cache (and its inverse).
//
// Rotation: pair i of a head turns by th = position * freqs[i]:
//   a' = m (a cos th - b sin th), b' = m (a sin th + b cos th).
// Angles, their reduction, cos, sin and the products are 64-bit: an angle of a
// far position keeps its fraction of a turn, and the rotated value is rounded
// once, so what is stored in 8 bits does not depend on how 32-bit steps round.
//
// Tokens are taken 8 at a time: their cos and sin are computed once per workgroup
// and serve all its heads, and 8 positions of a channel are what V keeps together.
// Bound by memory where there are many tokens: kq_rope of 6001 x 32 x 128 bf16 24 us
// (4.1 TB/s read and written; a copy of as much 20); seven prompts of up to 1100
// tokens (4879), 32 + 8 + 8 heads x 128, into bf16 pages 39 us (3.1 TB/s; vector
// instructions take 69 % of the cycles), read back in 21 (V in single elements). Few
// tokens: kq_rope of 16 5.5 us, most of it the launch and the sines; 16 tokens into
// 8-bit pages 8.9 us, one after another the batch's arrays, the page table, the sines
// and the rows.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq_kv_dev.h"

namespace kqd {

enum { T_F32 = 0, T_F16 = 1, T_BF16 = 2 };   // kq_type

__device__ __forceinline__ float f32_of(uint32_t v) { return __builtin_bit_cast(float, v); }
__device__ __forceinline__ float bf16_f32(uint32_t h) { return __builtin_bit_cast(float, h << 16); }
// fp32 to bf16, round to nearest even; NaN stays one.
__device__ __forceinline__ uint32_t f32_bf16(float v) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v);
}
template <int T>
__device__ __forceinline__ int type_size() { return T == T_F32 ? 4 : 2; }
template <int T>
__device__ __forceinline__ float load_one(const void* x, int64_t i) {
  if constexpr (T == T_F32) return static_cast<const float*>(x)[i];
  const uint32_t h = static_cast<const uint16_t*>(x)[i];
  return T == T_F16 ? h2f(h) : bf16_f32(h);
}
// 16-bit pattern of v.
template <int T>
__device__ __forceinline__ uint32_t to_16(float v) { return T == T_F16 ? f2h_bits(v) : f32_bf16(v); }
template <int T>
__device__ __forceinline__ void store_one(void* y, int64_t i, float v) {
  if constexpr (T == T_F32) static_cast<float*>(y)[i] = v;
  else static_cast<uint16_t*>(y)[i] = (uint16_t)to_16<T>(v);
}
template <int T>
__device__ __forceinline__ bool is_aligned(const void* p, int64_t ld) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * type_size<T>())) & 15) == 0;
}
// Eight elements at x + i (i a multiple of 8), in 16-byte loads where `wide`.
template <int T>
__device__ __forceinline__ void load_8(const void* x, int64_t i, bool wide, float (&v)[8]) {
  if (!wide) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = load_one<T>(x, i + j);
  } else if constexpr (T == T_F32) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const float*>(x) + i);
    const u32x4 a = p[0], b = p[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = f32_of(a[j]), v[4 + j] = f32_of(b[j]);
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + i);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t h = (a[j / 2] >> (16 * (j & 1))) & 0xffffu;
      v[j] = T == T_F16 ? h2f(h) : bf16_f32(h);
    }
  }
}
template <int T>
__device__ __forceinline__ u32x4 pack_8(const float (&v)[8]) {
  u32x4 a;
#pragma unroll
  for (int j = 0; j < 4; ++j) a[j] = to_16<T>(v[2 * j]) | to_16<T>(v[2 * j + 1]) << 16;
  return a;
}
template <int T>
__device__ __forceinline__ void store_8(void* y, int64_t i, bool wide, const float (&v)[8]) {
  if (!wide) {
#pragma unroll
    for (int j = 0; j < 8; ++j) store_one<T>(y, i + j, v[j]);
  } else if constexpr (T == T_F32) {
    u32x4* p = reinterpret_cast<u32x4*>(static_cast<float*>(y) + i);
    u32x4 a, b;
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = __builtin_bit_cast(uint32_t, v[j]), b[j] = __builtin_bit_cast(uint32_t, v[4 + j]);
    p[0] = a;
    p[1] = b;
  } else {
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(y) + i) = pack_8<T>(v);
  }
}

// cos and sin of position * freq, times m. The turns are taken off in 64 bits
// (2 pi in two parts, each step one fused multiply-add), which leaves at most
// half a turn: the error is that of the product's rounding.
__device__ __forceinline__ double2 cos_sin(int position, double freq, double m) {
  const double angle = (double)position * freq;
  const double n = rint(angle * 0.15915494309189535);                 // 1 / (2 pi)
  double r = __builtin_fma(-n, 6.283185307179586, angle);             // 2 pi rounded to 64 bits
  r = __builtin_fma(-n, 2.4492935982947064e-16, r);                   // the rest of 2 pi
  double s, c;
  sincos(r, &s, &c);
  return double2{c * m, s * m};
}

struct RopeArgs {
  const double* freqs;        // [rot / 2] or null: no rotation
  const int32_t* positions;   // [tokens] or null: the cache's
  double m;
  int rot;
  int interleaved;
};

constexpr int ROPE_WAVES = 4, OCT = 8;
constexpr int ROW_PAD = 4;   // floats after each token's row in LDS (16-byte pieces stay aligned)
typedef float v4f __attribute__((ext_vector_type(4)));
// LDS: OCT tables of rot / 2 (cos, sin), then per wave OCT rows of D floats.
__host__ __device__ constexpr int rope_lds(int D, int rot) {
  return OCT * (rot / 2) * 16 + ROPE_WAVES * OCT * (D + ROW_PAD) * 4;
}

// Rows [tokens t0, t0 + n) of one head, on their way into the wave's LDS region:
// the loads are issued in one place and waited for in another.
template <int T>
struct Rows {
  static constexpr int EACH = 4;   // pieces of 8 elements per lane: 8 tokens of up to 256
  float v[EACH][8];
  int n8, pieces;
  __device__ __forceinline__ void load(const void* x, int64_t ld, int64_t col, int t0, int n, int D) {
    const bool wide = is_aligned<T>(static_cast<const uint8_t*>(x) + col * type_size<T>(), ld);
    pieces = D / 8;
    n8 = n * pieces;
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
      const int i = (threadIdx.x & 63) + 64 * k;
      if (i < n8) load_8<T>(x, (int64_t)(t0 + i / pieces) * ld + col + 8 * (i % pieces), wide, v[k]);
    }
  }
  __device__ __forceinline__ void put(float* rows) const {
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
      const int i = (threadIdx.x & 63) + 64 * k;
      if (i < n8) {
        v4f* p = reinterpret_cast<v4f*>(rows + (i / pieces) * (8 * pieces + ROW_PAD) + 8 * (i % pieces));
        p[0] = v4f{v[k][0], v[k][1], v[k][2], v[k][3]};
        p[1] = v4f{v[k][4], v[k][5], v[k][6], v[k][7]};
      }
    }
    wave_sync();
  }
};

// Turns the pairs of n rows in LDS; neighbouring lanes have neighbouring pairs.
__device__ __forceinline__ void turn_rows(float* rows, const double2* cs, const RopeArgs& a, int n, int D) {
  if (a.freqs == nullptr) return;
  const int lane = threadIdx.x & 63, half = a.rot / 2;
  for (int i = lane; i < half; i += 64) {
    const int ia = a.interleaved ? 2 * i : i, ib = a.interleaved ? 2 * i + 1 : i + half;
    for (int t = 0; t < n; ++t) {
      float* row = rows + t * (D + ROW_PAD);
      const double2 w = cs[t * half + i];
      const double x = (double)row[ia], y = (double)row[ib];
      row[ia] = (float)__builtin_fma(-y, w.y, x * w.x);
      row[ib] = (float)__builtin_fma(x, w.y, y * w.x);
    }
  }
  wave_sync();
}

// Eight elements of a row in LDS.
__device__ __forceinline__ void row_8(const float* p, float (&v)[8]) {
  const v4f a = reinterpret_cast<const v4f*>(p)[0], b = reinterpret_cast<const v4f*>(p)[1];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
}

// Rows out.
template <int T>
__device__ __forceinline__ void rows_out(void* y, int64_t ld, int64_t col, int t0, int n, int D, const float* rows) {
  const int lane = threadIdx.x & 63, pieces = D / 8;
  const bool wide = is_aligned<T>(static_cast<const uint8_t*>(y) + col * type_size<T>(), ld);
  for (int i = lane; i < n * pieces; i += 64) {
    const int t = i / pieces, o = i % pieces;
    float v[8];
    row_8(rows + t * (D + ROW_PAD) + 8 * o, v);
    store_8<T>(y, (int64_t)(t0 + t) * ld + col + 8 * o, wide, v);
  }
  wave_sync();
}

// ---- kq_rope: a workgroup takes up to 8 tokens and a part of the heads, its
// waves a head at a time. The first rows' loads run while the angles are computed.
template <int XT, int YT>
__global__ __launch_bounds__(64 * ROPE_WAVES) void k_rope(RopeArgs a, const void* x, int64_t ldx, void* y, int64_t ldy,
                                                         int T, int heads, int D) {
  extern __shared__ u32x4 lds4[];
  double2* cs = reinterpret_cast<double2*>(lds4);
  const int half = a.rot / 2, wave = wave_id();
  float* rows = reinterpret_cast<float*>(cs + OCT * half) + wave * OCT * (D + ROW_PAD);
  const int t0 = blockIdx.x * OCT, n = min(OCT, T - t0), step = ROPE_WAVES * gridDim.y;
  Rows<XT> next;
  int h = blockIdx.y * ROPE_WAVES + wave;
  if (h < heads) next.load(x, ldx, (int64_t)h * D, t0, n, D);
  for (int i = threadIdx.x; i < n * half; i += 64 * ROPE_WAVES)
    cs[i] = cos_sin(a.positions[t0 + i / half], a.freqs[i % half], a.m);
  __syncthreads();
  for (; h < heads; h += step) {
    next.put(rows);
    if (h + step < heads) next.load(x, ldx, (int64_t)(h + step) * D, t0, n, D);
    turn_rows(rows, cs, a, n, D);
    rows_out<YT>(y, ldy, (int64_t)h * D, t0, n, D, rows);
  }
}

// ---- Q8_0 of a value whose block has the largest magnitude `bits` (as fp32
// bits: a NaN's are above infinity's): the scale as fp16 bits, and the code.
// The steps of kq_pack; a block that has no finite scale becomes NaN.
__device__ __forceinline__ uint32_t q8_scale(uint32_t bits) {
  if (bits >= 0x7f800000u) return 0x7e00u;
  const uint32_t d = f2h_bits(__builtin_bit_cast(float, bits) / 127.0f);
  return d == 0x7c00u ? 0x7e00u : d;
}
// The code is round(x / d), halves away from zero, of the quotient in fp32: the
// largest c with (c - 1/2) d <= |x|. (That product is exact, 8 bits by 11; and
// where x is below it, x / d is below c - 1/2 by 2^-24 of it at least, which is
// more than half an fp32 step there, so the quotient does not round up to it.) An
// approximate quotient is at most one off.
struct Q8Scale {
  float d, inverse;   // 0: every code is 0
};
__device__ __forceinline__ Q8Scale q8_of(uint32_t scale) {
  const float d = h2f(scale);
  const bool none = scale == 0u || scale == 0x7e00u;
  return Q8Scale{none ? 0.0f : d, none ? 0.0f : __builtin_amdgcn_rcpf(d)};
}
__device__ __forceinline__ int q8_code(float x, const Q8Scale& s) {
  const float m = fabsf(x);
  float c = truncf(fminf(__builtin_fmaf(m, s.inverse, 0.5f), 127.0f));
  if ((c - 0.5f) * s.d > m) c -= 1.0f;
  else if ((c + 0.5f) * s.d <= m && s.d > 0.0f) c += 1.0f;
  c = fminf(c, 127.0f);
  return (int)(x < 0.0f ? -c : c);
}
// The largest of the 32 lanes of a half wave (neighbours, quads, eights, rows of
// 16 through DPP; the neighbouring row by a permlane swap), in every lane.
template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ uint32_t max_xor16(uint32_t v) {
  uint32_t x = v, y = v;
  asm volatile("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(x), "+v"(y));
  return max(x, y);
}
__device__ __forceinline__ uint32_t max_32(uint32_t v) {
  return max_xor16(max_dpp<0x140>(max_dpp<0x141>(max_dpp<0x4E>(max_dpp<0xB1>(v)))));
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }

// The positions of a sequence's new tokens in runs that lie in one aligned
// octet: V keeps 8 positions of a channel together.
__device__ __forceinline__ int octets_of(const Seq& q) {
  const int first = max(q.len - q.n, 0);
  return q.n > 0 && q.len > 0 ? (q.len - 1) / OCT - first / OCT + 1 : 0;
}
struct Run {
  int s, token, n, position;   // `n` tokens from `token` on, at `position` on; s < 0: none
};
__device__ __forceinline__ Run run_of(const Batch& b, int id) {
  const int lane = threadIdx.x & 63;
  Run r{-1, 0, 0, 0};
  int before = 0;   // at most 2^20 tokens: sums stay below 2^31
  for (int s0 = 0; s0 < b.n_seqs; s0 += 64) {
    const Seq mine_of = s0 + lane < b.n_seqs ? seq_of(b, s0 + lane) : Seq{0, 0, 0};
    const int mine = octets_of(mine_of);
    const int upto = wave_scan(mine) + before;
    const uint64_t hit = __ballot(id < upto);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
      const Seq q{of(mine_of.begin), of(mine_of.n), of(mine_of.len)};
      const int local = id - of(upto - mine);
      const int first = max(q.len - q.n, 0);
      const int from = max((first / OCT + local) * OCT, first), to = min((first / OCT + local + 1) * OCT, q.len);
      r.s = s0 + l;
      r.position = from;
      r.n = to - from;
      r.token = q.begin + (from - (q.len - q.n));
      return r;
    }
    before = __builtin_amdgcn_readlane(upto, 63);
  }
  return r;
}

struct AppendArgs {
  Batch b;
  Cache c;
  RopeArgs rope;
  const void* k;
  const void* v;
  const void* q;
  void* q_out;
  int64_t ldk, ldv, ldq, ldo;
  int heads, D;
};

// K rows of a run (rotated) into a page: a lane has the 8 channels of one
// position, positions next to each other, so 4 lanes fill 64 bytes.
template <int CT>
__device__ __forceinline__ void put_k(uint8_t* region, int p0, int n, int D, const float* rows) {
  const int lane = threadIdx.x & 63;
  for (int i = lane; i < OCT * (D / 8); i += 64) {   // D / 8 is a multiple of 4: lanes of a block take part together
    const int t = i & 7, o = i >> 3, p = p0 + t;
    const bool have = t < n;
    float v[8];
    row_8(rows + t * (D + ROW_PAD) + 8 * o, v);   // rows that there are none of hold anything, and are not used
    uint32_t big = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) big = max(big, abs_bits(v[j]));
    if constexpr (CT == KQ_KV_Q8_0) {
      big = max_xor16(max_dpp<0x128>(big));   // the lanes 8 (row_ror:8) and 16 away: the block's other pieces
      const uint32_t scale = q8_scale(big);
      const Q8Scale by = q8_of(scale);
      u32x2v c = {0u, 0u};
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j / 4] |= ((uint32_t)q8_code(v[j], by) & 0xffu) << (8 * (j & 3));
      if (have) {
        *reinterpret_cast<u32x2v*>(region + k_index(true, p, 8 * o)) = c;
        if ((o & 3) == 0) reinterpret_cast<uint16_t*>(region + 32 * D)[(o >> 2) * 32 + p] = (uint16_t)scale;
      }
    } else if (have) {
      *reinterpret_cast<u32x4*>(region + 2 * k_index(false, p, 8 * o)) = pack_8<CT>(v);
    }
  }
}

// V rows of a run into a page: a lane has one channel of all its positions.
template <int CT>
__device__ __forceinline__ void put_v(uint8_t* region, int p0, int n, int D, const float* rows) {
  const int lane = threadIdx.x & 63;
  for (int d = lane; d < D; d += 64) {   // D is a multiple of 32: the lanes of a block take part together
    float v[OCT];
#pragma unroll
    for (int t = 0; t < OCT; ++t) v[t] = t < n ? rows[t * (D + ROW_PAD) + d] : 0.0f;
    if constexpr (CT == KQ_KV_Q8_0) {
      uint8_t* at = region + v_index(true, p0, d);
      u32x2v c = {0u, 0u};
#pragma unroll
      for (int t = 0; t < OCT; ++t) {
        const uint32_t scale = q8_scale(max_32(abs_bits(v[t]))), code = (uint32_t)q8_code(v[t], q8_of(scale)) & 0xffu;
        c[t / 4] |= code << (8 * (t & 3));
        if (t < n) {
          if ((d & 31) == 0) reinterpret_cast<uint16_t*>(region + 32 * D)[(d >> 5) * 32 + p0 + t] = (uint16_t)scale;
          if (n < OCT) at[t] = (uint8_t)code;
        }
      }
      if (n == OCT) *reinterpret_cast<u32x2v*>(at) = c;
    } else {
      uint8_t* at = region + 2 * v_index(false, p0, d);
      if (n == OCT) {
        *reinterpret_cast<u32x4*>(at) = pack_8<CT>(v);
      } else {
#pragma unroll
        for (int t = 0; t < OCT; ++t)
          if (t < n) reinterpret_cast<uint16_t*>(at)[t] = (uint16_t)to_16<CT>(v[t]);
      }
    }
  }
}

// ---- kq_kv_append: a workgroup takes one run and a part of the head rows (the
// heads of q, then those of k, then those of v), its waves a row at a time.
template <int XT, int CT, int OT>
__global__ __launch_bounds__(64 * ROPE_WAVES) void k_kv_append(AppendArgs a) {
  extern __shared__ u32x4 lds4[];
  const Run run = run_of(a.b, blockIdx.x);
  if (run.s < 0) return;
  double2* cs = reinterpret_cast<double2*>(lds4);
  const int half = a.rope.rot / 2, wave = wave_id(), D = a.D, Hk = a.c.kv_heads;
  float* rows = reinterpret_cast<float*>(cs + OCT * half) + wave * OCT * (D + ROW_PAD);
  const int H = a.q != nullptr ? a.heads : 0, rows_in_all = H + 2 * Hk, step = ROPE_WAVES * gridDim.y;
  Rows<XT> next;
  const auto load = [&](int row) {
    if (row < H) next.load(a.q, a.ldq, (int64_t)row * D, run.token, run.n, D);
    else if (row < H + Hk) next.load(a.k, a.ldk, (int64_t)(row - H) * D, run.token, run.n, D);
    else next.load(a.v, a.ldv, (int64_t)(row - H - Hk) * D, run.token, run.n, D);
  };
  int row = blockIdx.y * ROPE_WAVES + wave;
  if (row < rows_in_all) load(row);
  const int32_t page = scalar(page_id(a.b, a.c.n_pages, run.s, run.position / PAGE));
  if (a.rope.freqs != nullptr) {
    for (int i = threadIdx.x; i < run.n * half; i += 64 * ROPE_WAVES) {
      const int t = i / half;
      const int position = a.rope.positions != nullptr ? a.rope.positions[run.token + t] : run.position + t;
      cs[i] = cos_sin(position, a.rope.freqs[i % half], a.rope.m);
    }
  }
  __syncthreads();
  const int p0 = run.position % PAGE;
  const int64_t region = region_bytes(CT == KQ_KV_Q8_0, D);
  for (; row < rows_in_all; row += step) {
    next.put(rows);
    if (row + step < rows_in_all) load(row + step);
    if (row < H + Hk) turn_rows(rows, cs, a.rope, run.n, D);
    if (row < H) {
      rows_out<OT>(a.q_out, a.ldo, (int64_t)row * D, run.token, run.n, D, rows);
    } else if (page >= 0) {
      const bool is_v = row >= H + Hk;
      uint8_t* at = (is_v ? a.c.v : a.c.k) + ((int64_t)page * Hk + (row - H - (is_v ? Hk : 0))) * region;
      // V's pieces start at position 8 (p / 8); a run that starts inside one has fewer than 8 positions
      if (is_v) put_v<CT>(at, p0, run.n, D, rows);
      else put_k<CT>(at, p0, run.n, D, rows);
      wave_sync();
    }
  }
}

// ---- kq_kv_read: the rows of the new tokens as the cache holds them.
template <int CT, int YT>
__global__ __launch_bounds__(64 * ROPE_WAVES) void k_kv_read(Batch b, Cache c, void* k, int64_t ldk, void* v, int64_t ldv,
                                                            int D) {
  constexpr bool Q8 = CT == KQ_KV_Q8_0;
  const Run run = run_of(b, blockIdx.x);
  if (run.s < 0) return;
  const int32_t page = scalar(page_id(b, c.n_pages, run.s, run.position / PAGE));
  const int p0 = run.position % PAGE, Hk = c.kv_heads, lane = threadIdx.x & 63;
  const int64_t bytes = region_bytes(Q8, D);
  for (int row = blockIdx.y * ROPE_WAVES + wave_id(); row < 2 * Hk; row += ROPE_WAVES * gridDim.y) {
    const bool is_v = row >= Hk;
    const int h = is_v ? row - Hk : row;
    const uint8_t* region = (is_v ? c.v : c.k) + ((int64_t)(page < 0 ? 0 : page) * Hk + h) * bytes;
    const uint16_t* scales = reinterpret_cast<const uint16_t*>(region + 32 * D);
    const auto value = [&](int index, int p, int d) {
      if (page < 0) return __builtin_nanf("");
      if constexpr (Q8) return h2f(scales[(d >> 5) * 32 + p]) * (float)reinterpret_cast<const int8_t*>(region)[index];
      const uint32_t e = reinterpret_cast<const uint16_t*>(region)[index];
      return CT == KQ_KV_F16 ? h2f(e) : bf16_f32(e);
    };
    if (is_v) {
      for (int d = lane; d < D; d += 64)
#pragma unroll
        for (int t = 0; t < OCT; ++t)
          if (t < run.n)
            store_one<YT>(v, (int64_t)(run.token + t) * ldv + (int64_t)h * D + d, value(v_index(Q8, p0 + t, d), p0 + t, d));
    } else {
      const bool wide = is_aligned<YT>(static_cast<const uint8_t*>(k) + (int64_t)h * D * type_size<YT>(), ldk);
      for (int i = lane; i < OCT * (D / 8); i += 64) {
        const int t = i & 7, o = i >> 3;
        if (t >= run.n) continue;
        float e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = value(k_index(Q8, p0 + t, 8 * o) + j, p0 + t, 8 * o + j);
        store_8<YT>(k, (int64_t)(run.token + t) * ldk + (int64_t)h * D + 8 * o, wide, e);
      }
    }
  }
}

}  // namespace kqd

namespace kq {
using namespace kqd;

namespace {

RopeArgs rope_args(const kq_rope_spec* r) {
  if (r == nullptr) return RopeArgs{nullptr, nullptr, 1.0, 0, 0};
  return RopeArgs{r->freqs, r->positions, r->mscale, r->rot_dim, r->pairs == KQ_ROPE_INTERLEAVED};
}

// Runs of a batch: at most one per token, and at most two more per sequence
// than its tokens fill.
unsigned most_runs(const kq_kv_batch& b) {
  const int64_t octets = ((int64_t)b.n_tokens + OCT - 1) / OCT + 2ll * b.n_seqs;
  return (unsigned)(octets < b.n_tokens ? octets : b.n_tokens);
}

// Workgroups that share `rows` head rows: a wave per row where there are few
// runs, else enough to fill the chip.
unsigned row_parts(int64_t runs, int rows) {
  const int64_t most = (rows + ROPE_WAVES - 1) / ROPE_WAVES, want = (2048 + runs - 1) / runs;
  return (unsigned)(want < most ? (want < 1 ? 1 : want) : most);
}

Batch batch_view(const kq_kv_batch& b) {
  return Batch{b.page_table, b.table_width, b.q_start, b.lens, b.n_seqs, b.n_tokens};
}
Cache cache_view(const kq_kv_cache& c) {
  return Cache{static_cast<uint8_t*>(c.k), static_cast<uint8_t*>(c.v), c.n_pages, c.kv_heads};
}

template <int XT>
int rope_out(const kq_rope_spec* r, const void* x, int64_t ldx, int otype, void* y, int64_t ldy, int T, int heads, int D,
             hipStream_t stream) {
  const RopeArgs a = rope_args(r);
  const unsigned runs = (unsigned)((T + OCT - 1) / OCT);
  const dim3 grid(runs, row_parts(runs, heads));
  const size_t lds = (size_t)rope_lds(D, a.rot);
  dispatch_log("k_rope", -1, heads, D, T, grid.x, grid.y, 64 * ROPE_WAVES, lds, "rot=%d", a.rot);
  auto* k = otype == KQ_F32 ? k_rope<XT, T_F32> : otype == KQ_F16 ? k_rope<XT, T_F16> : k_rope<XT, T_BF16>;
  hipLaunchKernelGGL(k, grid, dim3(64 * ROPE_WAVES), lds, stream, a, x, ldx, y, ldy, T, heads, D);
  return (int)hipGetLastError();
}

template <int XT, int CT>
int append_out(const AppendArgs& a, int otype, dim3 grid, size_t lds, hipStream_t stream) {
  auto* k = otype == KQ_F32 ? k_kv_append<XT, CT, T_F32> : otype == KQ_F16 ? k_kv_append<XT, CT, T_F16> : k_kv_append<XT, CT, T_BF16>;
  hipLaunchKernelGGL(k, grid, dim3(64 * ROPE_WAVES), lds, stream, a);
  return (int)hipGetLastError();
}
template <int XT>
int append_cache(const AppendArgs& a, int ctype, int otype, dim3 grid, size_t lds, hipStream_t stream) {
  return ctype == KQ_KV_F16    ? append_out<XT, KQ_KV_F16>(a, otype, grid, lds, stream)
         : ctype == KQ_KV_BF16 ? append_out<XT, KQ_KV_BF16>(a, otype, grid, lds, stream)
                               : append_out<XT, KQ_KV_Q8_0>(a, otype, grid, lds, stream);
}

template <int CT>
int read_out(const kq_kv_cache& c, const kq_kv_batch& b, int otype, void* k, int64_t ldk, void* v, int64_t ldv, dim3 grid,
             hipStream_t stream) {
  auto* f = otype == KQ_F32 ? k_kv_read<CT, T_F32> : otype == KQ_F16 ? k_kv_read<CT, T_F16> : k_kv_read<CT, T_BF16>;
  hipLaunchKernelGGL(f, grid, dim3(64 * ROPE_WAVES), 0, stream, batch_view(b), cache_view(c), k, ldk, v, ldv, c.head_dim);
  return (int)hipGetLastError();
}

}  // namespace

int launch_rope(const kq_rope_spec* r, int xtype, const void* x, int64_t ldx, int otype, void* y, int64_t ldy, int T,
                int heads, int D, hipStream_t stream) {
  return xtype == KQ_F32   ? rope_out<T_F32>(r, x, ldx, otype, y, ldy, T, heads, D, stream)
         : xtype == KQ_F16 ? rope_out<T_F16>(r, x, ldx, otype, y, ldy, T, heads, D, stream)
                           : rope_out<T_BF16>(r, x, ldx, otype, y, ldy, T, heads, D, stream);
}

int launch_kv_append(const KvAppendArgs& p) {
  const kq_kv_cache& c = *p.cache;
  const kq_kv_batch& b = *p.batch;
  AppendArgs a{batch_view(b), cache_view(c), rope_args(p.rope), p.k, p.v, p.q, p.q_out, p.ldk, p.ldv, p.ldq, p.ldo, p.heads,
               c.head_dim};
  const int rows = (p.q != nullptr ? p.heads : 0) + 2 * c.kv_heads;
  const unsigned runs = most_runs(b);
  const dim3 grid(runs, row_parts(runs, rows));
  const size_t lds = (size_t)rope_lds(c.head_dim, a.rope.rot);
  dispatch_log("k_kv_append", -1, rows, c.head_dim, b.n_tokens, grid.x, grid.y, 64 * ROPE_WAVES, lds, "cache=%d", c.type);
  return p.xtype == KQ_F32   ? append_cache<T_F32>(a, c.type, p.otype, grid, lds, p.stream)
         : p.xtype == KQ_F16 ? append_cache<T_F16>(a, c.type, p.otype, grid, lds, p.stream)
                             : append_cache<T_BF16>(a, c.type, p.otype, grid, lds, p.stream);
}

int launch_kv_read(const kq_kv_cache& c, const kq_kv_batch& b, int otype, void* k, int64_t ldk, void* v, int64_t ldv,
                   hipStream_t stream) {
  const unsigned runs = most_runs(b);
  const dim3 grid(runs, row_parts(runs, 2 * c.kv_heads));
  dispatch_log("k_kv_read", -1, 2 * c.kv_heads, c.head_dim, b.n_tokens, grid.x, grid.y, 64 * ROPE_WAVES, 0, "cache=%d", c.type);
  return c.type == KQ_KV_F16    ? read_out<KQ_KV_F16>(c, b, otype, k, ldk, v, ldv, grid, stream)
         : c.type == KQ_KV_BF16 ? read_out<KQ_KV_BF16>(c, b, otype, k, ldk, v, ldv, grid, stream)
                                : read_out<KQ_KV_Q8_0>(c, b, otype, k, ldk, v, ldv, grid, stream);
}

}  // namespace kq
