// kq_attn_prompt.hip — attention of many new tokens per sequence (prompts, or
// the next part of one) over the paged cache.
//
// A workgroup has a tile of columns: the queries of one key-value head, token
// by token, so the heads of a group share what is read and a tile spans few
// tokens, which keeps the masked corner small. Its waves have 32 columns each
// and walk the tile's pages together: the pages' regions come into LDS by
// direct copies, in the order in which the operands of the 32 x 32 x 16 matrix
// instructions are read back (16 lanes read 256 bytes in a row: no bank
// conflicts, nothing to transpose).
//   S^T = K Q^T: keys on the rows, queries on the columns, so a lane has 16
//   scores of one query per page and shares the column with one other lane;
//   they are the operand of O^T += V^T P^T as they stand.
//
// Bound by the matrix instructions and, nearly as long, the softmax's arithmetic
// between them: 8191 bf16 tokens of 32 heads x 128 555 to 605 us with the clock
// (991 to 909 TFLOP/s of visible products; a plain 8192^3 product of the library
// 1255), 500 tokens behind 32000 285 to 310 us (926 to 850 TFLOP/s). In 8 bits every
// wave converts the codes that it reads, and V takes two products: twelve prompts of
// up to 2500 tokens of 16 heads x 64 190 us, bound by that arithmetic. Five prompts
// of up to 150 tokens 14.5 us, bound by the latency of one step after another.
// Two waves to a SIMD leave each 256 registers. Heads of 192 and more pass them in
// 16 bits (45, 138 and 260 of a wave's in scratch, in the loop without masks 1, 15
// and 14 loads of 16 bytes and 8 stores a step): 4000 bf16 tokens of 32 heads x 160
// 223 us (733 TFLOP/s), of 192 302 (651), of 224 907 to 990 (253), of 256 700 (374).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq_attn_dev.h"

// The kernel's parts: a call would put all that they share into memory.
#define INLINE __attribute__((always_inline))

namespace kqd {

// A step is PP pages. Step i of a wave is two phases: the matrix instructions
// (the scores of step i, then V of step i - 1) and the arithmetic (the weights
// of step i), each ended by a barrier. With 8 waves two share a SIMD; the second
// four are one phase behind, so one of the two has matrix instructions while
// the other has arithmetic: left alone they fall into step and take turns.
// K and V of three steps are in LDS: in the phase in which the first half of
// the waves begins step i, K of step i + 2 and V of step i + 1 take the places
// of K of step i - 1 and V of step i - 2, which the second half last read in the
// phase before; they are waited for two phases later.
template <bool V> struct Flag { static constexpr bool value = V; };
template <int N> struct Count { static constexpr int value = N; };

template <bool Q8, int DB, int WAVES_>
struct Prompt {
  static constexpr int WAVES = WAVES_, TILE = WAVES * 32;
  static constexpr int PP = DB <= 4 ? 2 : 1;
  static constexpr int REGION = (int)region_bytes(Q8, 32 * DB);
  static constexpr int STEP = PP * REGION, RING = 3;
  static constexpr int LDS = 2 * RING * STEP;
};

// Copies a region from memory into LDS, the workgroup's waves a part each; no
// bytes: zeros. (Not through global_load_lds: with those in flight the compiler
// waits for all reads of LDS at each use of one.)
template <int REGION, int WAVES>
__device__ __forceinline__ void copy_in(uint8_t* dst, const uint8_t* src, int bytes, int wave) {
  constexpr int PIECES = REGION / 16, EACH = WAVES * 64;
  const rsrc_t rs = make_rsrc(src, (uint32_t)bytes);
  const int piece = threadIdx.x;
#pragma unroll
  for (int t = 0; t < (PIECES + EACH - 1) / EACH; ++t)
    if ((t + 1) * EACH <= PIECES || t * EACH + piece < PIECES)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)(dst + (t * EACH + wave * 64) * 16), 16, piece * 16,
                                               t * EACH * 16, 0, 0);
}

template <int QT, bool Q8, int DB, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void k_attn_prompt(AttnArgs a) {
  typedef Prompt<Q8, DB, WAVES> Sh;
  constexpr int D = 32 * DB, VT = Q8 ? A_BF16 : QT, PP = Sh::PP;
  // In 8 bits m follows the largest score only in steps of 2^GROWTH, each column by
  // itself, and most steps leave o as it is (twelve prompts of 16 x 64: 189 us, with
  // every step 193). Weights that are rounded to 16 bits keep 1 for the largest one,
  // which is exact: following in steps costs them a third more error and gains nothing
  // with heads of 128.
  constexpr float GROWTH = Q8 ? 8.0f : 0.0f;
  extern __shared__ u32x4 lds4[];
  uint8_t* kring = reinterpret_cast<uint8_t*>(lds4);
  uint8_t* vring = kring + Sh::RING * Sh::STEP;

  const Part p = part_of(a.b, a.w, blockIdx.x);
  if (p.s < 0) return;
  const int lane = threadIdx.x & 63, wave = wave_id(), r = lane & 31, H = lane >> 5;
  const int G = a.w.G, cols = p.seq.n * G, col0 = p.tile * Sh::TILE, start = p.seq.len - p.seq.n;

  // the tile's pages, and this chunk's part of them
  const int tile_last = start + (min(cols, col0 + Sh::TILE) - 1) / G;
  int first = p.first, np = p.np;
  if (first < a.b.width || np == 0) {   // not behind the table
    const int lo = a.w.window > 0 ? max(start + col0 / G - a.w.window + 1, 0) : 0;
    first = lo / PAGE;
    np = tile_last < 0 ? 0 : max(tile_last / PAGE + 1 - first, 0);
  }
  const int base = np / p.chunks, rest = np % p.chunks;
  const int p0 = first + p.chunk * base + min(p.chunk, rest), p1 = p0 + base + (p.chunk < rest ? 1 : 0);

  // the wave's columns
  const int wcol = col0 + wave * 32;
  const bool works = wcol < cols;
  const int from = start + wcol / G, to = start + (min(cols, wcol + 32) - 1) / G;   // positions
  const int col = wcol + r;
  const bool have = col < cols;
  const int token = have ? col / G : 0, qhead = p.head * G + (have ? col - token * G : 0);
  const int at = have ? start + token : -1;
  u32x4 qf[2 * DB];
  const auto load_q = [&]() INLINE {
    const bool wide = wide_rows(a.q, a.ldq);
    const uint16_t* q = a.q + (int64_t)(p.seq.begin + token) * a.ldq + (int64_t)qhead * D + 8 * H;
#pragma unroll
    for (int c = 0; c < 2 * DB; ++c) {
      qf[c] = row_piece(q + 16 * c, wide);
      if (!have) qf[c] = u32x4{0u, 0u, 0u, 0u};
    }
  };
  load_q();

  v16f o[DB], s[PP];
  u32x4 pf[Q8 ? 1 : PP][2];      // packed weights (Q8_0: s itself holds them)
  uint32_t seen = 0xffffffffu;   // what the lane's column sees of a step: bit 16 g + 8 h + element of operand h
  float m = -__builtin_inff(), l = 0.0f;
  bool poison = false;           // infinities or NaN were left out of V
#pragma unroll
  for (int d = 0; d < DB; ++d) o[d] = zero16();

  // Where the lane's operands lie in a region. Row r of a K tile is piece row
  // r % 16 of tile r / 16, so 16 lanes read 256 bytes in a row; register i of
  // lane half H then holds key 16 (i / 4 % 2) + 8 H + 4 (i / 8) + i % 4, and
  // registers 4 h .. and 8 + 4 h .. are the 8 keys of the second product's
  // operand h.
  const int at_lds = Q8 ? (H * 16 + (r & 15)) * 16 + (r >> 4) * 8 : ((r >> 4) * 64 + H * 16 + (r & 15)) * 16;
  // 16 channels of K; 32 channels and 16 keys of V
  const auto k_operand = [&](const uint8_t* region, int c) INLINE {
    if constexpr (Q8) {
      const u32x2v e = *reinterpret_cast<const u32x2v*>(region + at_lds + (c >> 1) * 1024 + (c & 1) * 512);
      return codes16<QT>(e[0], e[1]);
    } else {
      return *reinterpret_cast<const u32x4*>(region + at_lds + (c >> 1) * 2048 + (c & 1) * 512);
    }
  };
  const auto v_operand = [&](const uint8_t* region, int d, int h) INLINE {
    if constexpr (Q8) {
      const u32x2v e = *reinterpret_cast<const u32x2v*>(region + at_lds + d * 1024 + h * 512);
      return codes16<VT>(e[0], e[1]);
    } else {
      return *reinterpret_cast<const u32x4*>(region + at_lds + d * 2048 + h * 512);
    }
  };

  // s = scores of a step (16-bit caches): f[first] holds the first page's
  // operands. Operands are read 2 DB ahead of their products, one read behind each
  // matrix instruction: left to itself the compiler reads each one just before its
  // use and waits for it.
  const auto score_products = [&](u32x4 (&f)[2][2 * DB], int first, const uint8_t* stage) INLINE {
#pragma unroll
    for (int g = 0; g < PP; ++g) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int c = 0; c < 2 * DB; ++c) {
        if (g + 1 < PP) f[(first + g + 1) & 1][c] = k_operand(stage + (g + 1) * Sh::REGION, c);
        s[g] = mfma32<QT>(f[(first + g) & 1][c], qf[c], c == 0 ? zero16() : s[g]);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                   // a matrix instruction
        if (g + 1 < PP) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // a read from LDS
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // s = scores of a step, or of one page.
  const auto scores = [&](const uint8_t* stage, auto pages) INLINE {
    constexpr int N = decltype(pages)::value;
    if constexpr (Q8) {
#pragma unroll
      for (int g = 0; g < N; ++g) {
        const uint8_t* region = stage + g * Sh::REGION;
        const u32x4* scales = reinterpret_cast<const u32x4*>(region + 32 * D);
        s[g] = zero16();
#pragma unroll
        for (int b = 0; b < DB; ++b) {
          const u32x4 k0 = k_operand(region, 2 * b), k1 = k_operand(region, 2 * b + 1);
          const u32x4 sc[2] = {scales[4 * b + H], scales[4 * b + 2 + H]};
          const v16f d = mfma32<QT>(k1, qf[2 * b + 1], mfma32<QT>(k0, qf[2 * b], zero16()));
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t w = sc[(i >> 2) & 1][2 * (i >> 3) + ((i & 3) >> 1)];
            s[g][i] = __builtin_fmaf(h2f(i & 1 ? w >> 16 : w), d[i], s[g][i]);
          }
        }
      }
    } else if constexpr (N == PP) {
      u32x4 f[2][2 * DB];
#pragma unroll
      for (int c = 0; c < 2 * DB; ++c) f[0][c] = k_operand(stage, c);
      score_products(f, 0, stage);
    } else {
#pragma unroll
      for (int c = 0; c < 2 * DB; ++c) s[0] = mfma32<QT>(k_operand(stage, c), qf[c], c == 0 ? zero16() : s[0]);
    }
  };

  // Masks of a step that not every column sees whole: of a page's keys, element j
  // of the lane's operands is key 2 (j & 8) + 8 H + (j & 7).
  const auto mask = [&](int page, const int32_t (&id)[PP]) INLINE {
#pragma unroll
    for (int g = 0; g < PP; ++g) {
      // the column sees keys above `below` and up to `last` of this page
      int last = at - (page + g) * PAGE - 8 * H, below = a.w.window > 0 ? last - a.w.window : -64;
      if (id[g] == -3) last = -64;
      if (id[g] == -2) last = 64, below = -64;
      const uint32_t span = (uint32_t)max(min(last, 64) - max(below, -64), 0);
      below = max(below, -64);
      uint32_t bits = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int j = 8 * ((i >> 2) & 1) + 4 * (i >> 3) + (i & 3);   // register i's place
        const bool ok = (uint32_t)(2 * (j & 8) + (j & 7) - below - 1) < span;
        if constexpr (Q8) bits |= (ok ? 1u : 0u) << j;
        s[g][i] = ok ? s[g][i] : -__builtin_inff();
      }
      if (id[g] == -1 || id[g] == -2) {   // no such page: what sees it becomes NaN
#pragma unroll
        for (int i = 0; i < 16; ++i) s[g][i] = s[g][i] == -__builtin_inff() ? s[g][i] : __builtin_nanf("");
      }
      if constexpr (Q8) seen = (seen & ~(0xffffu << (16 * g))) | bits << (16 * g);
    }
  };

  // Scores to weights; o to the new m. t = scale * s: the hot loop's are exact
  // products, and m is a product that was rounded, so where they are far from zero
  // (see again below) t - m is off by many powers of two; there t is rounded as m is.
  const auto weigh = [&](auto far_) INLINE {
    constexpr bool ROUNDED = decltype(far_)::value;
    float top = s[0][0];
#pragma unroll
    for (int g = 0; g < PP; ++g)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[g][i]);
    top = max_lane_xor32(top);
    top = ROUNDED ? lowered<VT>(top * a.scale) : __builtin_fmaf(top, a.scale, -SHIFT<VT>);   // scale > 0
    const bool grows = top > m + (ROUNDED ? 0.0f : GROWTH);
    const float by = grows ? exp2_fast(m - top) : 1.0f;
    m = grows ? top : m;
    l *= by;
    // 16 bits, always: a branch around it cost more than it saved
    if (!Q8 || __any(grows)) {
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= by;
    }
    const float sub = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
    for (int g = 0; g < PP; ++g) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if constexpr (ROUNDED) {
#pragma clang fp contract(off)
          const float t = s[g][i] * a.scale;
          s[g][i] = exp2_fast(t - sub);
        } else {
          s[g][i] = exp2_fast(__builtin_fmaf(s[g][i], a.scale, -sub));
        }
      }
      if constexpr (Q8) {
#pragma unroll
        for (int i = 0; i < 16; ++i) l += s[g][i];
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int i = 8 * (j >> 1) + 4 * h + 2 * (j & 1);
            pf[g][h][j] = pack2<VT>(s[g][i], s[g][i + 1]);
            // the sum is of the rounded weights: where one weight is most of it,
            // its rounding leaves the quotient again
            l = add_pair<VT>(pf[g][h][j], l);
          }
      }
    }
  };

  // o += V^T P^T of a step, or of one page.
  const auto add_v = [&](const uint8_t* stage, auto masked_, auto pages) INLINE {
    constexpr bool MASKED = decltype(masked_)::value;
    constexpr int N = decltype(pages)::value;
    if constexpr (Q8) {
      // The scale of V's block goes to the weight, in two parts of 8 bits (bf16 has
      // the range of the scales); the codes stay whole numbers.
#pragma unroll
      for (int g = 0; g < N; ++g) {
        const uint8_t* region = stage + g * Sh::REGION;
        const u32x4* scales = reinterpret_cast<const u32x4*>(region + 32 * D);
#pragma unroll
        for (int b = 0; b < DB; ++b) {
          const u32x4 sc[2] = {scales[4 * b + H], scales[4 * b + 2 + H]};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const u32x4 vf = v_operand(region, b, h);
            u32x4 hi, lo;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t w = sc[h][j];
              const int i = 8 * (j >> 1) + 4 * h + 2 * (j & 1), bit = 16 * g + 8 * h + 2 * j;
              float e0 = s[g][i] * h2f(w), e1 = s[g][i + 1] * h2f(w >> 16);
              if constexpr (MASKED) {   // a masked key's scale may be NaN
                e0 = seen >> bit & 1 ? e0 : 0.0f;
                e1 = seen >> bit & 2 ? e1 : 0.0f;
              }
              uint32_t x, y;
              split2<VT>(e0, e1, x, y);
              hi[j] = x;
              lo[j] = y;
            }
            o[b] = mfma32<VT>(vf, hi, o[b]);
            o[b] = mfma32<VT>(vf, lo, o[b]);
          }
        }
      }
    } else {
      // Infinities and NaN of keys that a column does not see must not reach it
      // (0 times them is NaN): they are left out here and added at the end.
#pragma unroll
      for (int g = 0; g < N; ++g) {
        u32x4 v[2 * DB];
#pragma unroll
        for (int c = 0; c < 2 * DB; ++c) v[c] = v_operand(stage + g * Sh::REGION, c % DB, c / DB);
        if constexpr (MASKED) {
          bool bad = false;
#pragma unroll
          for (int c = 0; c < 2 * DB; ++c) bad |= any_not_finite<VT>(v[c]);
          if (__any(bad)) {
            poison = true;
#pragma unroll
            for (int c = 0; c < 2 * DB; ++c) {
              u32x4 plus, minus;
              v[c] = take_finite<VT>(v[c], plus, minus);
            }
          }
        }
#pragma unroll
        for (int c = 0; c < 2 * DB; ++c) o[c % DB] = mfma32<VT>(v[c], pf[g][c / DB], o[c % DB]);
      }
    }
  };

  // The matrix instructions of a step between steps that need no masks, V of
  // the step before first (its weights make room for the scores). The first
  // operands of V were read in the phase before.
  u32x4 ahead[Q8 ? 1 : 2 * DB];
  const auto read_ahead = [&](const uint8_t* stage) INLINE {
    if constexpr (!Q8) {
#pragma unroll
      for (int c = 0; c < 2 * DB; ++c) ahead[c] = v_operand(stage, c % DB, c / DB);
    }
  };
  const auto products = [&](const uint8_t* kstage, const uint8_t* vstage) INLINE {
    if constexpr (Q8) {
      add_v(vstage, Flag<false>(), Count<PP>());
      scores(kstage, Count<PP>());
    } else {
      u32x4 f[2][2 * DB];
#pragma unroll
      for (int c = 0; c < 2 * DB; ++c) f[0][c] = ahead[c];
#pragma unroll
      for (int g = 0; g < PP; ++g) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int c = 0; c < 2 * DB; ++c) {
          f[(g + 1) & 1][c] = g + 1 < PP ? v_operand(vstage + (g + 1) * Sh::REGION, c % DB, c / DB) : k_operand(kstage, c);
          o[c % DB] = mfma32<VT>(f[g & 1][c], pf[g][c / DB], o[c % DB]);
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
      }
      score_products(f, PP & 1, kstage);
    }
  };

  const int steps = (p1 - p0 + PP - 1) / PP;
  if (steps > 0) {
    // Where the regions of 64 steps' pages begin, held by the lanes, from step
    // held_from on (the cache's first region stands in for pages that there are
    // none of: any_bad says that there was one).
    int64_t held[PP];
    int held_from = 0;
    bool any_bad = false;
    const auto fill = [&](int from_step) INLINE {
#pragma unroll
      for (int g = 0; g < PP; ++g) {
        const int64_t page = (int64_t)p0 + (int64_t)(from_step + lane) * PP + g;
        const int32_t id = page >= p1 ? 0 : page_id(a.b, a.c.n_pages, p.s, (int)page);
        any_bad |= __any(id < 0);
        held[g] = ((int64_t)max(id, 0) * a.c.kv_heads + p.head) * Sh::REGION;
      }
      held_from = from_step;
    };
    struct Step {
      int64_t at[PP];
    };
    const auto step_at = [&](int i) INLINE {
      Step st;
#pragma unroll
      for (int g = 0; g < PP; ++g)
        st.at[g] = (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)held[g], i - held_from) |
                   (int64_t)__builtin_amdgcn_readlane((int)(held[g] >> 32), i - held_from) << 32;
      return st;
    };
    const auto copy_step = [&](uint8_t* stage, const uint8_t* plane, const Step& st, int i) INLINE {
#pragma unroll
      for (int g = 0; g < PP; ++g)
        copy_in<Sh::REGION, WAVES>(stage + g * Sh::REGION, plane + st.at[g], p0 + i * PP + g < p1 ? Sh::REGION : 0, wave);
    };
    fill(0);
    // Barriers of their own: __syncthreads would wait for every copy in flight.
    // A phase's arithmetic stays in it.
    const auto phase_ends = [] {
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("s_barrier" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    // This wave's copies have landed (they are loads to the compiler).
    const auto copies_landed = [] { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); };
    const Step st0 = step_at(0);
    Step st1 = step_at(1), st2 = step_at(2);
    copy_step(kring, a.c.k, st0, 0);
    copy_step(vring, a.c.v, st0, 0);
    copy_step(kring + Sh::STEP, a.c.k, st1, 1);
    copies_landed();
    phase_ends();
    const bool behind = WAVES == 8 && wave >= 4;
    if (behind) phase_ends();
    int now = 0, i = 0;   // step, and its place in both rings
    bool had = false, had_mask = false;
    // pages that every column sees whole: a step of them needs no masks
    const int whole_from = a.w.window > 0 ? max((to - a.w.window + PAGE) / PAGE, 0) : 0;
    const int whole_to = works ? min(p1, (from + 1) / PAGE) : 0;
    const auto whole = [&]() INLINE { return p0 + i * PP >= whole_from && p0 + (i + 1) * PP <= whole_to && !any_bad; };
    const auto walk = [&](auto fast) INLINE {
      const int next = now == 2 ? 0 : now + 1, last = now == 0 ? 2 : now - 1;
      copy_step(kring + last * Sh::STEP, a.c.k, st2, i + 2);
      copy_step(vring + next * Sh::STEP, a.c.v, st1, i + 1);
      if constexpr (decltype(fast)::value) {
        products(kring + now * Sh::STEP, vring + last * Sh::STEP);
        phase_ends();
        weigh(Flag<false>());
        read_ahead(vring + now * Sh::STEP);
      } else {
        const int page = p0 + i * PP;
        int32_t id[PP];
#pragma unroll
        for (int g = 0; g < PP; ++g)
          id[g] = page + g >= p1 ? -3 : any_bad ? scalar(page_id(a.b, a.c.n_pages, p.s, page + g)) : 0;
        const bool beyond = page * PAGE > to || (a.w.window > 0 && (page + PP) * PAGE <= from - a.w.window + 1);
        const bool does = works && (!beyond || id[0] == -2), unmasked = whole();
        // V of a step that needed no masks is also multiplied this way here
        if (had) add_v(vring + last * Sh::STEP, Flag<true>(), Count<PP>());
        if (does) scores(kring + now * Sh::STEP, Count<PP>());
        phase_ends();
        if (does) {
          seen = 0xffffffffu;
          if (!unmasked) mask(page, id);
          weigh(Flag<false>());
          read_ahead(vring + now * Sh::STEP);
        }
        had = does;
        had_mask = !unmasked;
      }
      // the next step's pages in this phase: these reads of lanes would queue behind
      // the other wave's arithmetic in the next one
      st1 = st2;
      if constexpr (!decltype(fast)::value)
        if (i + 3 - held_from > 63) fill(i + 3);
      st2 = step_at(i + 3);
      copies_landed();
      phase_ends();
      now = next;
      ++i;
    };
    while (i < steps) {
      if (had && !had_mask && whole()) {
        // as far as steps are whole, and before the one that moves on to the next 64
        const int end = min((whole_to - p0) / PP, held_from + 61);
        while (i < end) walk(Flag<true>());
      }
      if (i < steps) walk(Flag<false>());
    }
    if (WAVES == 8 && !behind) phase_ends();
    if (had) add_v(vring + (now == 0 ? 2 : now - 1) * Sh::STEP, Flag<true>(), Count<PP>());
  }

  // Where scores are far from zero the walk is taken again, by the waves that have
  // such columns, a page at a time from memory. (m only rises: what it passed on its
  // way up from below -FAR has no weight, or left l or o infinite or NaN. 4000 bf16
  // tokens of 32 x 128 that all have such scores 452 us, 178 without. A branch in
  // every step instead: 8191 tokens 568 -> 619 us, heads of 256 870 -> 1400.)
  float zero[4] = {l * 0.0f, 0.0f, 0.0f, 0.0f};   // NaN where one of l and o is infinite or NaN
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) zero[i & 3] = __builtin_fmaf(o[d][i], 0.0f, zero[i & 3]);
  const bool finite = (zero[0] + zero[1]) + (zero[2] + zero[3]) == 0.0f;
  if (__any(have && m != -__builtin_inff() && !(finite && __builtin_fabsf(m) < FAR))) {
    m = -__builtin_inff();
    l = 0.0f;
#pragma unroll
    for (int d = 0; d < DB; ++d) o[d] = zero16();
    // Heads of 256 are short of registers: there q does not outlast the loop above
    // (4000 bf16 tokens of 32 x 256 737 us, 950 with q kept; of 32 x 224 1262, 875).
    if constexpr (DB == 8) load_q();
    for (int page = p0; page < p1; ++page) {
      int32_t id[PP];
#pragma unroll
      for (int g = 0; g < PP; ++g) id[g] = g == 0 ? scalar(page_id(a.b, a.c.n_pages, p.s, page)) : -3;
      const int64_t region = ((int64_t)max(id[0], 0) * a.c.kv_heads + p.head) * Sh::REGION;
      scores(a.c.k + region, Count<1>());
      mask(page, id);
      weigh(Flag<true>());
      add_v(a.c.v + region, Flag<true>(), Count<1>());
    }
  }

  if constexpr (!Q8) {
    if (poison) {
      // What was left out of V: a column that sees plus and minus infinity, or
      // NaN, gets NaN, whatever the weights (they are above 0).
      constexpr uint32_t ONE = VT == A_F16 ? 0x3c00u : 0x3f80u;
      for (int page = p0; page < p1; ++page) {
        const int32_t id = scalar(page_id(a.b, a.c.n_pages, p.s, page));
        if (id < 0) continue;
        const uint8_t* region = a.c.v + ((int64_t)id * a.c.kv_heads + p.head) * Sh::REGION;
        for (int h = 0; h < 2; ++h) {
          u32x4 one = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int key = page * PAGE + 16 * h + 8 * H + j;
            if (key <= at && (a.w.window <= 0 || key > at - a.w.window)) one[j / 2] |= ONE << (16 * (j & 1));
          }
#pragma unroll
          for (int d = 0; d < DB; ++d) {
            u32x4 plus, minus;
            take_finite<VT>(v_operand(region, d, h), plus, minus);
            const v16f up = mfma32<VT>(plus, one, zero16()), down = mfma32<VT>(minus, one, zero16());
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[d][i] += (up[i] > 0.0f ? __builtin_inff() : 0.0f) + (down[i] > 0.0f ? -__builtin_inff() : 0.0f);
          }
        }
      }
    }
  }

  l += __shfl_xor(l, 32, 64);
  if (!have) return;
  const int64_t row = (int64_t)p.slot * Sh::TILE + wave * 32 + r;
  if (p.chunks > 1 && H == 0) a.ml[row] = float2{m, l};
  const bool wide = wide_rows(a.out, a.ldo);
  uint16_t* out = a.out + (int64_t)(p.seq.begin + token) * a.ldo + (int64_t)qhead * D + 4 * H;
  const float by = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v4f v = {o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2], o[d][4 * e + 3]};
      if (p.chunks > 1) *reinterpret_cast<v4f*>(a.part + row * D + 32 * d + 8 * e + 4 * H) = v;
      else put_4<QT>(out + 32 * d + 8 * e, wide, l == 0.0f ? v4f{0.f, 0.f, 0.f, 0.f} : v * by);
    }
}

}  // namespace kqd

namespace kq {
using namespace kqd;

namespace {

template <int QT, bool Q8, int DB, int WAVES>
int prompt_launch(const AttnCall& p, const AttnPlan& w) {
  typedef Prompt<Q8, DB, WAVES> Sh;
  const AttnArgs a = attn_args(p, w);
  dispatch_log("k_attn_prompt", -1, p.heads, 32 * DB, p.batch->n_tokens, (unsigned)w.grid, 1, 64 * WAVES, Sh::LDS,
               "cache=%d tile=%d slots=%lld", p.cache->type, w.tile, (long long)w.slots);
  hipLaunchKernelGGL((k_attn_prompt<QT, Q8, DB, WAVES>), dim3((unsigned)w.grid), dim3(64 * WAVES), Sh::LDS, p.stream, a);
  int err = (int)hipGetLastError();
  if (err || w.slots == 0) return err;
  return launch_attn_join_tiles(a, p.type, 32 * DB, p.stream);
}
template <int QT, bool Q8, int DB>
int prompt_tile(const AttnCall& p, const AttnPlan& w) {
  if constexpr (!Q8 && DB > 3)   // (prompt_plan)
    if (w.tile == 256) return prompt_launch<QT, Q8, DB, 8>(p, w);
  return prompt_launch<QT, Q8, DB, 4>(p, w);
}
template <int QT, bool Q8>
int prompt_dim(const AttnCall& p, const AttnPlan& w) {
  switch (p.cache->head_dim / 32) {
    case 1: return prompt_tile<QT, Q8, 1>(p, w);
    case 2: return prompt_tile<QT, Q8, 2>(p, w);
    case 3: return prompt_tile<QT, Q8, 3>(p, w);
    case 4: return prompt_tile<QT, Q8, 4>(p, w);
    case 5: return prompt_tile<QT, Q8, 5>(p, w);
    case 6: return prompt_tile<QT, Q8, 6>(p, w);
    case 7: return prompt_tile<QT, Q8, 7>(p, w);
    default: return prompt_tile<QT, Q8, 8>(p, w);
  }
}

}  // namespace

AttnPlan prompt_plan(const kq_kv_cache& c, const kq_kv_batch& b, int heads) {
  AttnPlan w;
  w.search = 1;
  // Tiles of 256 columns, 8 waves that share what is read, two of them to a SIMD,
  // where a workgroup of 4 waves would leave a SIMD one (three steps of 16-bit
  // heads of more than 96 are above half of LDS) and sequences have the columns:
  // 8191 bf16 tokens of 32 x 128 579 us (128 columns 709). Prompts of up to 300
  // tokens have fewer tiles than the chip has places even with 128 columns, which
  // the others take too: 4000 fp16 tokens of 32 x 64 102 us (256 columns 114), twelve
  // prompts of 16 x 64 in 8 bits 189 (265).
  const int64_t cols = (int64_t)b.n_tokens * (heads / c.kv_heads) / b.n_seqs;   // of a mean sequence
  w.tile = cols >= 1024 && c.type != KQ_KV_Q8_0 && c.head_dim > 96 ? 256 : 128;
  w.target = 256;
  w.places = 256;
  w.least = 16;
  finish_plan(c, b, heads, w);
  return w;
}

int launch_attn_prompt(const AttnCall& p) {
  const AttnPlan w = prompt_plan(*p.cache, *p.batch, p.heads);
  const bool q8 = p.cache->type == KQ_KV_Q8_0;
  if (p.type == KQ_F16) return q8 ? prompt_dim<A_F16, true>(p, w) : prompt_dim<A_F16, false>(p, w);
  return q8 ? prompt_dim<A_BF16, true>(p, w) : prompt_dim<A_BF16, false>(p, w);
}

}  // namespace kq
