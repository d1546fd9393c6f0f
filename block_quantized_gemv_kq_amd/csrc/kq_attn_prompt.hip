// kq_attn_prompt.hip — attention of many new tokens per sequence (prompts, or
// the next part of one) over the paged cache.
//
// A workgroup has a tile of columns: the queries of one key-value head, token
// by token, so the heads of a group share what is read and a tile spans few
// tokens, which keeps the masked corner small. Its waves have 32 columns (or
// 64) each and walk the tile's pages together: the pages' regions come into
// LDS by direct copies, one step ahead, in the order in which the operands of
// the 32 x 32 x 16 matrix instructions are read back (64 lanes, 16 bytes each,
// in runs of 256 bytes: no bank conflicts, nothing to transpose).
//   S^T = K Q^T: keys on the rows, queries on the columns, so a lane has 16
//   scores of one query per page and shares the column with one other lane;
//   they are the operand of O^T += V^T P^T as they stand.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq_attn_dev.h"

namespace kqd {

constexpr int PR_WAVES = 4, PR_PAGES = 2;   // pages per step

template <bool V> struct Flag { static constexpr bool value = V; };

template <bool Q8, int DB, int NC>
struct PromptShape {
  static constexpr int REGION = (int)region_bytes(Q8, 32 * DB);
  static constexpr int STAGE = PR_PAGES * 2 * REGION;
  static constexpr int TILE = PR_WAVES * 32 * NC;
};

// Copies `bytes` (a multiple of 16) from memory into LDS by the whole workgroup.
__device__ __forceinline__ void copy_in(uint8_t* dst, const uint8_t* src, int bytes) {
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const rsrc_t rs = make_rsrc(src, (uint32_t)bytes);
  for (int i = wave * 64; i < bytes / 16; i += 64 * PR_WAVES)
    if (i + lane < bytes / 16)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)(dst + 16 * i), 16, (i + lane) * 16, 0, 0, 0);
}

template <int QT, bool Q8, int DB, int NC>
__global__ __launch_bounds__(64 * PR_WAVES) void k_attn_prompt(AttnArgs a) {
  typedef PromptShape<Q8, DB, NC> Sh;
  constexpr int D = 32 * DB, VT = Q8 ? A_BF16 : QT;
  extern __shared__ u32x4 lds4[];
  uint8_t* lds = reinterpret_cast<uint8_t*>(lds4);

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
  const int wcol = col0 + wave * 32 * NC;
  const bool works = wcol < cols;
  const int from = start + wcol / G, to = start + (min(cols, wcol + 32 * NC) - 1) / G;   // positions
  u32x4 qf[NC][2 * DB];
  int at[NC];
  const bool qwide = wide_rows(a.q, a.ldq);
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const int col = wcol + 32 * n + r;
    const bool have = col < cols;
    const int i = have ? col / G : 0, h = p.head * G + (have ? col - i * G : 0);
    at[n] = have ? start + i : -1;
    const uint16_t* q = a.q + (int64_t)(p.seq.begin + i) * a.ldq + (int64_t)h * D + 8 * H;
#pragma unroll
    for (int c = 0; c < 2 * DB; ++c) {
      qf[n][c] = row_piece(q + 16 * c, qwide);
      if (!have) qf[n][c] = u32x4{0u, 0u, 0u, 0u};
    }
  }

  v16f o[NC][DB];
  float m[NC], l[NC];
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    m[n] = -__builtin_inff();
    l[n] = 0.0f;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[n][d][i] = 0.0f;
  }

  // where the lane's operands lie in a region: row r of a K tile is key
  // 16 (r / 16) + 8 (r / 4 % 2) + 4 (r / 8 % 2) + r % 4, so that register i of
  // lane half H holds key 16 (i / 8) + 8 H + i % 8
  const int krow = (4 * (2 * (r >> 4) + ((r >> 2) & 1)) + (r & 3)), kt = (r >> 3) & 1;
  const int k_at = Q8 ? (H * 16 + krow) * 16 + kt * 8 : (kt * 64 + H * 16 + krow) * 16;
  const int v_at = Q8 ? (H * 16 + (r & 15)) * 16 + (r >> 4) * 8 : ((r >> 4) * 64 + H * 16 + (r & 15)) * 16;

  const auto k_operand = [&](const uint8_t* region, int c) {   // 16 channels
    if constexpr (Q8) {
      const u32x2v e = *reinterpret_cast<const u32x2v*>(region + k_at + (c >> 1) * 1024 + (c & 1) * 512);
      return codes16<QT>(e[0], e[1]);
    } else {
      return *reinterpret_cast<const u32x4*>(region + k_at + (c >> 1) * 2048 + (c & 1) * 512);
    }
  };
  const auto v_operand = [&](const uint8_t* region, int d, int s) {   // 32 channels, 16 keys
    if constexpr (Q8) {
      const u32x2v e = *reinterpret_cast<const u32x2v*>(region + v_at + d * 1024 + s * 512);
      return codes16<VT>(e[0], e[1]);
    } else {
      return *reinterpret_cast<const u32x4*>(region + v_at + d * 2048 + s * 512);
    }
  };

  const auto step = [&](const uint8_t* stage, int page, const int32_t (&id)[PR_PAGES], auto masked_) {
    constexpr bool MASKED = decltype(masked_)::value;
    v16f s[NC][PR_PAGES];
#pragma unroll
    for (int g = 0; g < PR_PAGES; ++g) {
      const uint8_t* region = stage + g * Sh::REGION;
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[n][g][i] = 0.0f;
      if constexpr (Q8) {
        const u32x4* scales = reinterpret_cast<const u32x4*>(region + 32 * D);
#pragma unroll
        for (int b = 0; b < DB; ++b) {
          const u32x4 k0 = k_operand(region, 2 * b), k1 = k_operand(region, 2 * b + 1);
          const u32x4 sc[2] = {scales[4 * b + H], scales[4 * b + 2 + H]};
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            v16f d;
#pragma unroll
            for (int i = 0; i < 16; ++i) d[i] = 0.0f;
            d = mfma32<QT>(k0, qf[n][2 * b], d);
            d = mfma32<QT>(k1, qf[n][2 * b + 1], d);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint32_t w = sc[i >> 3][(i & 7) >> 1];
              s[n][g][i] = __builtin_fmaf(h2f(i & 1 ? w >> 16 : w), d[i], s[n][g][i]);
            }
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < 2 * DB; ++c) {
          const u32x4 k = k_operand(region, c);
#pragma unroll
          for (int n = 0; n < NC; ++n) s[n][g] = mfma32<QT>(k, qf[n][c], s[n][g]);
        }
      }
    }
    uint32_t seen[NC];   // bit 16 g + i
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      seen[n] = 0xffffffffu;
      if constexpr (MASKED) {
        seen[n] = 0;
#pragma unroll
        for (int g = 0; g < PR_PAGES; ++g)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int key = (page + g) * PAGE + 16 * (i >> 3) + 8 * H + (i & 7);
            bool ok = key <= at[n] && (a.w.window <= 0 || key > at[n] - a.w.window);
            if (id[g] == -2) ok = true;
            if (id[g] == -3) ok = false;
            seen[n] |= (ok ? 1u : 0u) << (16 * g + i);
            s[n][g][i] = !ok ? -__builtin_inff() : id[g] < 0 ? __builtin_nanf("") : s[n][g][i];
          }
      }
      float top = s[n][0][0];
#pragma unroll
      for (int g = 0; g < PR_PAGES; ++g)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[n][g][i]);
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      top *= a.scale;   // scale > 0
      if (__any(top > m[n])) {
        const float now = fmaxf(m[n], top), by = m[n] == now ? 1.0f : exp2_fast(m[n] - now);
        m[n] = now;
        l[n] *= by;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[n][d][i] *= by;
      }
      const float sub = m[n] == -__builtin_inff() ? 0.0f : m[n];
#pragma unroll
      for (int g = 0; g < PR_PAGES; ++g)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[n][g][i] = exp2_fast(__builtin_fmaf(s[n][g][i], a.scale, -sub));
          l[n] += s[n][g][i];
        }
    }
#pragma unroll
    for (int g = 0; g < PR_PAGES; ++g) {
      const uint8_t* region = stage + (PR_PAGES + g) * Sh::REGION;
      if constexpr (Q8) {
        const u32x4* scales = reinterpret_cast<const u32x4*>(region + 32 * D);
#pragma unroll
        for (int b = 0; b < DB; ++b) {
          const u32x4 sc[2] = {scales[4 * b + H], scales[4 * b + 2 + H]};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const u32x4 v = v_operand(region, b, h);
#pragma unroll
            for (int n = 0; n < NC; ++n) {
              u32x4 hi, lo;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t w = sc[h][j];
                const int i = 8 * h + 2 * j;
                // a masked key's scale may be NaN
                const float e0 = !MASKED || (seen[n] >> (16 * g + i) & 1) ? s[n][g][i] * h2f(w) : 0.0f;
                const float e1 = !MASKED || (seen[n] >> (16 * g + i + 1) & 1) ? s[n][g][i + 1] * h2f(w >> 16) : 0.0f;
                uint32_t x, y;
                split2<VT>(e0, e1, x, y);
                hi[j] = x;
                lo[j] = y;
              }
              o[n][b] = mfma32<VT>(v, hi, o[n][b]);
              o[n][b] = mfma32<VT>(v, lo, o[n][b]);
            }
          }
        }
      } else {
        u32x4 pf[NC][2];
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) pf[n][h][j] = pack2<VT>(s[n][g][8 * h + 2 * j], s[n][g][8 * h + 2 * j + 1]);
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            u32x4 v = v_operand(region, d, h);
            if constexpr (MASKED) {
              if (__any(any_not_finite<VT>(v))) {
                // infinities and NaN of keys that a column does not see must not
                // reach it: the finite part is multiplied, and what a column sees
                // of the rest is counted and added as it is
                u32x4 plus, minus;
                v = take_finite<VT>(v, plus, minus);
                constexpr uint32_t ONE = VT == A_F16 ? 0x3c00u : 0x3f80u;
#pragma unroll
                for (int n = 0; n < NC; ++n) {
                  u32x4 one;
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    const uint32_t w = seen[n] >> (16 * g + 8 * h + 2 * j);
                    one[j] = (w & 1 ? ONE : 0u) | (w & 2 ? ONE << 16 : 0u);
                  }
                  v16f zero;
#pragma unroll
                  for (int i = 0; i < 16; ++i) zero[i] = 0.0f;
                  const v16f up = mfma32<VT>(plus, one, zero), down = mfma32<VT>(minus, one, zero);
#pragma unroll
                  for (int i = 0; i < 16; ++i)
                    o[n][d][i] += (up[i] > 0.0f ? __builtin_inff() : 0.0f) + (down[i] > 0.0f ? -__builtin_inff() : 0.0f);
                }
              }
            }
#pragma unroll
            for (int n = 0; n < NC; ++n) o[n][d] = mfma32<VT>(v, pf[n][h], o[n][d]);
          }
      }
    }
  };

  const auto ids_at = [&](int page, int32_t (&id)[PR_PAGES]) {
#pragma unroll
    for (int g = 0; g < PR_PAGES; ++g)
      id[g] = page + g < p1 ? scalar(page_id(a.b, a.c.n_pages, p.s, page + g)) : -3;
  };
  const auto copy_step = [&](uint8_t* stage, const int32_t (&id)[PR_PAGES]) {
#pragma unroll
    for (int g = 0; g < PR_PAGES; ++g) {
      if (id[g] == -3) continue;
      const int64_t off = ((int64_t)(id[g] < 0 ? 0 : id[g]) * a.c.kv_heads + p.head) * Sh::REGION;
      copy_in(stage + g * Sh::REGION, a.c.k + off, Sh::REGION);
      copy_in(stage + (PR_PAGES + g) * Sh::REGION, a.c.v + off, Sh::REGION);
    }
  };

  if (p0 < p1) {
    int32_t id[PR_PAGES], next[PR_PAGES];
    ids_at(p0, id);
    ids_at(p0 + PR_PAGES, next);
    copy_step(lds, id);
    int buf = 0;
    for (int page = p0; page < p1; page += PR_PAGES) {
      // this step's copies have landed (they are loads to the compiler), and
      // every wave is done with the other buffer
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      int32_t after[PR_PAGES];
      ids_at(page + 2 * PR_PAGES, after);
      if (page + PR_PAGES < p1) copy_step(lds + (buf ^ 1) * Sh::STAGE, next);
      const bool beyond = page * PAGE > to || (a.w.window > 0 && (page + PR_PAGES) * PAGE <= from - a.w.window + 1);
      bool whole = (page + PR_PAGES) * PAGE - 1 <= from && (a.w.window <= 0 || page * PAGE > to - a.w.window);
#pragma unroll
      for (int g = 0; g < PR_PAGES; ++g) whole &= id[g] >= 0;
      if (works && whole) step(lds + buf * Sh::STAGE, page, id, Flag<false>());
      else if (works && (!beyond || id[0] == -2)) step(lds + buf * Sh::STAGE, page, id, Flag<true>());
#pragma unroll
      for (int g = 0; g < PR_PAGES; ++g) id[g] = next[g], next[g] = after[g];
      buf ^= 1;
    }
  }
  if (!works) return;

  const bool owide = wide_rows(a.out, a.ldo);
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    l[n] += __shfl_xor(l[n], 32, 64);
    const int in_tile = wave * 32 * NC + 32 * n + r, col = col0 + in_tile;
    if (col >= cols) continue;
    const int64_t row = (int64_t)p.slot * Sh::TILE + in_tile;
    if (p.chunks > 1 && H == 0) a.ml[row] = float2{m[n], l[n]};
    const int tok = col / G, h = p.head * G + col % G;
    uint16_t* out = a.out + (int64_t)(p.seq.begin + tok) * a.ldo + (int64_t)h * D + 4 * H;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v4f v = {o[n][d][4 * e], o[n][d][4 * e + 1], o[n][d][4 * e + 2], o[n][d][4 * e + 3]};
        if (p.chunks > 1) {
          *reinterpret_cast<v4f*>(a.part + row * D + 32 * d + 8 * e + 4 * H) = v;
        } else {
          v = l[n] == 0.0f ? v4f{0.f, 0.f, 0.f, 0.f} : v / l[n];
          put_4<QT>(out + 32 * d + 8 * e, owide, v);
        }
      }
  }
}

}  // namespace kqd

namespace kq {
using namespace kqd;

namespace {

template <int QT, bool Q8, int DB, int NC>
int prompt_launch(const AttnCall& p, const AttnPlan& w) {
  typedef PromptShape<Q8, DB, NC> Sh;
  const AttnArgs a = attn_args(p, w);
  dispatch_log("k_attn_prompt", -1, p.heads, 32 * DB, p.batch->n_tokens, (unsigned)w.grid, 1, 64 * PR_WAVES, 2 * Sh::STAGE,
               "cache=%d tile=%d slots=%lld", p.cache->type, w.tile, (long long)w.slots);
  hipLaunchKernelGGL((k_attn_prompt<QT, Q8, DB, NC>), dim3((unsigned)w.grid), dim3(64 * PR_WAVES), 2 * Sh::STAGE, p.stream, a);
  int err = (int)hipGetLastError();
  if (err || w.slots == 0) return err;
  return launch_attn_join(a, p.type, 32 * DB, p.stream);
}
template <int QT, bool Q8>
int prompt_dim(const AttnCall& p, const AttnPlan& w) {
  switch (p.cache->head_dim / 32) {
    case 1: return prompt_launch<QT, Q8, 1, 1>(p, w);
    case 2: return prompt_launch<QT, Q8, 2, 1>(p, w);
    case 3: return prompt_launch<QT, Q8, 3, 1>(p, w);
    case 4: return prompt_launch<QT, Q8, 4, 1>(p, w);
    case 5: return prompt_launch<QT, Q8, 5, 1>(p, w);
    case 6: return prompt_launch<QT, Q8, 6, 1>(p, w);
    case 7: return prompt_launch<QT, Q8, 7, 1>(p, w);
    default: return prompt_launch<QT, Q8, 8, 1>(p, w);
  }
}

}  // namespace

AttnPlan prompt_plan(const kq_kv_cache& c, const kq_kv_batch& b, int heads) {
  AttnPlan w;
  w.tile = 128;
  w.target = 512;
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
