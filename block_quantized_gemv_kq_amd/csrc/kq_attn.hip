// kq_attn.hip — attention of a few new tokens per sequence over the paged
// cache (decode and verify passes), and the join of partial results.
//
// A wave takes a page (32 keys) at a time, straight from memory to registers:
// S^T = K Q^T on matrix instructions, 16 keys by 16 columns (the queries of one
// key-value head, token by token); the scores of a lane are 8 consecutive keys
// of one column, which is the operand of O^T += V^T P^T as it stands.
// Every byte of K and V is read once per column tile, so there are as few tiles
// as the registers carry (1 or 2 of 16 columns), and where that leaves few
// workgroups the walk is split over the pages. V's loads run under the scores,
// the next K's under the softmax.
//
// Bound by memory where the cache is long: one token of 32 heads over 131071
// bf16 positions of 8 key-value heads x 128 100 us (5.4 TB/s; a plain read of as
// much 87), 48 such tokens over up to 8000 positions in 8 bits 102 us (4.6 TB/s:
// the conversion of codes shares the time), 64 over 500 in fp16 17 us (4.2 TB/s).
// Three trees of 16 rows x 32 heads (8 of keys) over up to 6000 positions are bound
// by the two parts of the weights and the softmax of 64 columns a page, in four
// tiles that each read it (22.7 us; the bytes alone 7.5), a token at 1000 positions
// by two launches and the latency of one page after another (10.9 us). Above heads
// of 192 registers run out: one token at 131071 bf16 positions 147 us with heads of
// 192 (5.5 TB/s), 181 with 224 (5.2), 265 with 256 (4.1; 8 scratch stores and 11
// loads of 16 bytes a page).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq_attn_dev.h"

namespace kqd {

constexpr int DEC_WAVES = 4;

// A wave's page of one head, as operands.
template <bool Q8, int DB>
struct Page {
  u32x4 k[Q8 ? DB : 2 * DB];
  u32x4 v[Q8 ? DB : 2 * DB];
  u32x4 ks[Q8 ? DB : 1];   // scales of the lane's 8 keys, per block of 32 channels
  u32x4 vs[Q8 ? DB : 1];
};

template <bool Q8, int DB>
__device__ __forceinline__ void load_half(u32x4 (&x)[Q8 ? DB : 2 * DB], u32x4 (&scales)[Q8 ? DB : 1], const uint8_t* plane,
                                          const Cache& c, int32_t id, int head) {
  const int lane = threadIdx.x & 63;
  const u32x4* p = reinterpret_cast<const u32x4*>(
      plane + ((int64_t)(id < 0 ? 0 : id) * c.kv_heads + head) * region_bytes(Q8, 32 * DB));
#pragma unroll
  for (int i = 0; i < (Q8 ? DB : 2 * DB); ++i) x[i] = p[i * 64 + lane];
  if constexpr (Q8) {
#pragma unroll
    for (int i = 0; i < DB; ++i) scales[i] = p[64 * DB + 4 * i + (lane >> 4)];
  }
}

// CT: tiles of 16 columns that every wave carries.
template <int QT, bool Q8, int DB, int CT>
__global__ __launch_bounds__(64 * DEC_WAVES, DB * CT <= 2 ? 4 : DB * CT <= 4 || (!Q8 && DB * CT <= 8) ? 2 : 1) void k_attn_decode(AttnArgs a) {
  constexpr int D = 32 * DB, DT = 2 * DB, VT = Q8 ? A_BF16 : QT;
  // d-tiles per round of the sum over the waves: 64 KB of LDS
  constexpr int ROUND = DT * CT * DEC_WAVES <= 64 ? DT : 64 / (CT * DEC_WAVES);
  __shared__ v4f sum[DEC_WAVES * ROUND * CT * 64];
  __shared__ float s_m[DEC_WAVES][CT * 16], s_l[DEC_WAVES][CT * 16];

  const Part p = part_of(a.b, a.w, blockIdx.x);
  if (p.s < 0) return;
  const int lane = threadIdx.x & 63, wave = wave_id(), r = lane & 15, g = lane >> 4;
  const int G = a.w.G, cols = p.seq.n * G, col0 = p.tile * (16 * CT);

  // this lane's columns: token, position, what of the newest tokens it sees
  u32x4 qf[CT][DB];
  int at[CT];            // position, or -1: no column
  uint64_t tree[CT];
  const bool qwide = wide_rows(a.q, a.ldq);
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int col = col0 + 16 * ct + r;
    const bool have = col < cols;
    const int i = have ? col / G : 0, h = p.head * G + (have ? col - i * G : 0);
    at[ct] = have ? p.seq.len - p.seq.n + i : -1;
    tree[ct] = a.tree != nullptr && have ? a.tree[p.seq.begin + i] : ~0ull;
    const uint16_t* q = a.q + (int64_t)(p.seq.begin + i) * a.ldq + (int64_t)h * D + 8 * g;
#pragma unroll
    for (int c = 0; c < DB; ++c) {
      qf[ct][c] = row_piece(q + 32 * c, qwide);
      if (!have) qf[ct][c] = u32x4{0u, 0u, 0u, 0u};
    }
  }
  // Codes come with a bias added (see biased16); it leaves the scores through
  // what the products start from, and o through the sums z of the weights.
  v4f kbias[Q8 ? CT : 1][Q8 ? DB : 1], z[Q8 ? CT : 1][Q8 ? DB : 1];
  if constexpr (Q8) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int c = 0; c < DB; ++c) {
        kbias[ct][c] = mfma16<QT>(splat16<QT>(-Bias<QT>::v), qf[ct][c], v4f{0.f, 0.f, 0.f, 0.f});
        z[ct][c] = v4f{0.f, 0.f, 0.f, 0.f};
      }
  }
  // a page that every column sees whole needs no mask
  const int newest = p.seq.len - p.seq.n;   // position of the first new token
  const int whole_to = a.tree != nullptr ? newest : newest + 1;   // keys below are seen by every query
  const int whole_from = a.w.window > 0 ? p.seq.len - a.w.window : 0;

  v4f o[CT][DT];
  float m[CT], l[CT];
  const auto reset = [&] {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      m[ct] = -__builtin_inff();
      l[ct] = 0.0f;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) o[ct][dt] = v4f{0.f, 0.f, 0.f, 0.f};
    }
  };
  reset();
  // Pages that every column sees whole are multiplied as they are. Where that
  // leaves something infinite or NaN, the walk is taken again with care for each
  // infinity and NaN of V (see below).
  bool careful = false;

  // the chunk's pages, one in DEC_WAVES for this wave
  const int base = p.np / p.chunks, rest = p.np % p.chunks;
  const int p0 = p.first + p.chunk * base + min(p.chunk, rest);
  const int p1 = p0 + base + (p.chunk < rest ? 1 : 0);
  const int steps = (p1 - p0 - wave + DEC_WAVES - 1) / DEC_WAVES;

  const auto step = [&](Page<Q8, DB>& pg, int32_t id, int page, bool more, int32_t id_next) {
    const int key0 = page * PAGE + 8 * g;    // this lane's keys: key0 + j
    const bool masked = page * PAGE + PAGE > whole_to || page * PAGE < whole_from || id < 0;
    // V comes in while the scores are computed, the next K from then on
    load_half<Q8, DB>(pg.v, pg.vs, a.c.v, a.c, id, p.head);
    u32x4 ph[CT][Q8 ? DB : 1], pl[CT][Q8 ? DB : 1], seen1[CT];
    v4f sc[CT][2];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      sc[ct][0] = sc[ct][1] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < DB; ++c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (Q8) {
            const u32x4 kf = biased16<QT>(pg.k[c][2 * h], pg.k[c][2 * h + 1]);
            const v4f d = mfma16<QT>(kf, qf[ct][c], kbias[ct][c]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t w = pg.ks[c][2 * h + i / 2];
              sc[ct][h][i] = __builtin_fmaf(h2f(i & 1 ? w >> 16 : w), d[i], sc[ct][h][i]);
            }
          } else {
            sc[ct][h] = mfma16<QT>(pg.k[2 * c + h], qf[ct][c], sc[ct][h]);
          }
        }
      }
    }
    if (more) load_half<Q8, DB>(pg.k, pg.ks, a.c.k, a.c, id_next, p.head);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      float t[8];
      {
#pragma clang fp contract(off)   // t as m has it
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = sc[ct][j >> 2][j & 3] * a.scale;
      }
      uint32_t seen = 0xff;
      if (masked) {
        seen = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int key = key0 + j, among = key - newest;
          bool ok = key <= at[ct] && (a.w.window <= 0 || key > at[ct] - a.w.window);
          if (a.tree != nullptr && among >= 0) ok &= among < 64 && (tree[ct] >> (among & 63) & 1) != 0;
          if (id == -2) ok = true;
          seen |= (ok ? 1u : 0u) << j;
          t[j] = !ok ? -__builtin_inff() : id < 0 ? __builtin_nanf("") : t[j];
        }
      }
      float top = fmaxf(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])), fmaxf(fmaxf(t[4], t[5]), fmaxf(t[6], t[7])));
      top = lowered<VT>(max_lane_xor32(max_lane_xor16(top)));
      if (__any(top > m[ct])) {
        const float now = fmaxf(m[ct], top), by = m[ct] == now ? 1.0f : exp2_fast(m[ct] - now);
        m[ct] = now;
        l[ct] *= by;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[ct][dt] *= by;
        if constexpr (Q8) {
#pragma unroll
          for (int c = 0; c < DB; ++c) z[ct][c] *= by;
        }
      }
      const float sub = m[ct] == -__builtin_inff() ? 0.0f : m[ct];   // nothing seen yet: weights 0
      float e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        e[j] = exp2_fast(t[j] - sub);
        l[ct] += e[j];
      }
      if constexpr (Q8) {
        // The scale of V's block goes to the weight, the codes stay whole numbers.
        // A masked key's scale may be NaN.
        u32x4 vs[DB];
#pragma unroll
        for (int c = 0; c < DB; ++c) vs[c] = pg.vs[c];
        if (masked) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t keep = (seen >> (2 * j) & 1 ? 0xffffu : 0u) | (seen >> (2 * j + 1) & 1 ? 0xffff0000u : 0u);
#pragma unroll
            for (int c = 0; c < DB; ++c) vs[c][j] &= keep;
          }
        }
#pragma unroll
        for (int c = 0; c < DB; ++c) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t w = vs[c][j];
            uint32_t hi, lo;
            split2<A_BF16>(e[2 * j] * h2f(w), e[2 * j + 1] * h2f(w >> 16), hi, lo);
            ph[ct][c][j] = hi;
            pl[ct][c][j] = lo;
          }
          z[ct][c] = mfma16<A_BF16>(splat16<A_BF16>(1.0f), ph[ct][c], z[ct][c]);
          z[ct][c] = mfma16<A_BF16>(splat16<A_BF16>(1.0f), pl[ct][c], z[ct][c]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t hi, lo;
          split2<VT>(e[2 * j], e[2 * j + 1], hi, lo);
          ph[ct][0][j] = hi;
          pl[ct][0][j] = lo;
          const uint32_t one = VT == A_F16 ? 0x3c00u : 0x3f80u;
          seen1[ct][j] = (seen >> (2 * j) & 1 ? one : 0u) | (seen >> (2 * j + 1) & 1 ? one << 16 : 0u);
        }
      }
    }
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      if constexpr (Q8) {
        const u32x4 vf = biased16<VT>(pg.v[dt / 2][2 * (dt & 1)], pg.v[dt / 2][2 * (dt & 1) + 1]);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          o[ct][dt] = mfma16<VT>(vf, ph[ct][dt / 2], o[ct][dt]);
          o[ct][dt] = mfma16<VT>(vf, pl[ct][dt / 2], o[ct][dt]);
        }
      } else {
        u32x4 vf = pg.v[dt];
        if ((masked || careful) && __any(any_not_finite<VT>(vf))) {
          // Infinities and NaN of V must not reach columns that do not see
          // them (0 times them is NaN), nor meet the two parts of a weight: the
          // finite part is multiplied, and what a column sees of the rest is
          // counted and added as it is.
          u32x4 plus, minus;
          vf = take_finite<VT>(vf, plus, minus);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) {
            const v4f up = mfma16<VT>(plus, seen1[ct], v4f{0.f, 0.f, 0.f, 0.f});
            const v4f down = mfma16<VT>(minus, seen1[ct], v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int i = 0; i < 4; ++i)
              o[ct][dt][i] += (up[i] > 0.0f ? __builtin_inff() : 0.0f) + (down[i] > 0.0f ? -__builtin_inff() : 0.0f);
          }
        }
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          o[ct][dt] = mfma16<VT>(vf, ph[ct][0], o[ct][dt]);
          o[ct][dt] = mfma16<VT>(vf, pl[ct][0], o[ct][dt]);
        }
      }
    }
  };

  if (steps > 0) {
    Page<Q8, DB> pg;
    PageIds ids;
    ids.fill(a.b, a.c.n_pages, p.s, p0 + wave, DEC_WAVES, 0);
    int32_t id = ids.at(a.b, a.c.n_pages, p.s, p0 + wave, DEC_WAVES, 0);
    for (;;) {
      load_half<Q8, DB>(pg.k, pg.ks, a.c.k, a.c, id, p.head);
      for (int i = 0; i < steps; ++i) {
        const bool more = i + 1 < steps;
        const int32_t id_next = more ? ids.at(a.b, a.c.n_pages, p.s, p0 + wave, DEC_WAVES, i + 1) : 0;
        step(pg, id, p0 + wave + i * DEC_WAVES, more, id_next);
        id = id_next;
      }
      if (Q8 || careful) break;
      bool bad = false;
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
          for (int i = 0; i < 4; ++i) bad |= !(__builtin_fabsf(o[ct][dt][i]) < __builtin_inff());
      if (!__any(bad)) break;
      careful = true;
      reset();
      ids.fill(a.b, a.c.n_pages, p.s, p0 + wave, DEC_WAVES, 0);
      id = ids.at(a.b, a.c.n_pages, p.s, p0 + wave, DEC_WAVES, 0);
    }
  }

  if constexpr (Q8) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[ct][dt][i] = __builtin_fmaf(-Bias<VT>::v, z[ct][dt / 2][i], o[ct][dt][i]);
  }
  // join the waves
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    l[ct] += __shfl_xor(l[ct], 16, 64);
    l[ct] += __shfl_xor(l[ct], 32, 64);
    if (g == 0) {
      s_m[wave][16 * ct + r] = m[ct];
      s_l[wave][16 * ct + r] = l[ct];
    }
  }
  __syncthreads();
  float by[CT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    float top = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < DEC_WAVES; ++w) top = fmaxf(top, s_m[w][16 * ct + r]);
    by[ct] = m[ct] == -__builtin_inff() ? (l[ct] == 0.0f ? 0.0f : 1.0f) : exp2_fast(m[ct] - top);
  }
  const bool owide = wide_rows(a.out, a.ldo);
#pragma unroll
  for (int d0 = 0; d0 < DT; d0 += ROUND) {
    if (d0 > 0) __syncthreads();
#pragma unroll
    for (int dt = d0; dt < d0 + ROUND && dt < DT; ++dt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) sum[((wave * ROUND + dt - d0) * CT + ct) * 64 + lane] = o[ct][dt] * by[ct];
    __syncthreads();
    const int here = DT - d0 < ROUND ? DT - d0 : ROUND;
    for (int i = wave; i < here * CT; i += DEC_WAVES) {
      const int dt = d0 + i / CT, ct = i % CT;
      v4f v = sum[i * 64 + lane];
#pragma unroll
      for (int w = 1; w < DEC_WAVES; ++w) v += sum[(w * ROUND * CT + i) * 64 + lane];
      const int col = col0 + 16 * ct + r;
      if (col >= cols) continue;
      float top = -__builtin_inff(), total = 0.0f;
#pragma unroll
      for (int w = 0; w < DEC_WAVES; ++w) top = fmaxf(top, s_m[w][16 * ct + r]);
#pragma unroll
      for (int w = 0; w < DEC_WAVES; ++w) {
        const float mw = s_m[w][16 * ct + r], lw = s_l[w][16 * ct + r];
        total += mw == -__builtin_inff() ? lw : exp2_fast(mw - top) * lw;   // NaN scores leave m, and l is NaN
      }
      if (p.chunks > 1) {
        const int64_t row = (int64_t)p.slot * (16 * CT) + 16 * ct + r;
        *reinterpret_cast<v4f*>(a.part + row * D + 16 * dt + 4 * g) = v;
        if (dt == 0 && g == 0) a.ml[row] = float2{top, total};
      } else {
        const int tok = col / G, h = p.head * G + col % G;
        v = total == 0.0f ? v4f{0.f, 0.f, 0.f, 0.f} : v / total;
        put_4<QT>(a.out + (int64_t)(p.seq.begin + tok) * a.ldo + (int64_t)h * D + 16 * dt + 4 * g, owide, v);
      }
    }
  }
}

// ---- The join of split tiles. Parts [first, chunks) of a row, every `step`-th:
// lanes over its channels in fours, groups of lanes over the parts, several of
// each group's in flight. Returns the lane's channels' sum and the weights' sum
// over the wave's parts, relative to the largest m of the row.
struct Joined {
  v4f v;
  float l;
};
__device__ __forceinline__ Joined join_row(const AttnArgs& a, int64_t row0, int64_t stride, int chunks, int first, int step,
                                           int D) {
  const int lane = threadIdx.x & 63, quads = D / 4;
  const int per = quads <= 8 ? 8 : quads <= 16 ? 16 : quads <= 32 ? 32 : 64;   // lanes of a row's channels
  const int lanes = 64 / per, quad = min(lane % per, quads - 1);
  const int part = first * lanes + lane / per, all = step * lanes;
  constexpr int FLY = 4;
  float2 ml[FLY];
  v4f o[FLY];
  const auto fetch = [&](int c0) {
#pragma unroll
    for (int i = 0; i < FLY; ++i) {
      const int64_t row = row0 + min(c0 + i * all, chunks - 1) * stride;
      ml[i] = a.ml[row];
      o[i] = *reinterpret_cast<const v4f*>(a.part + row * D + 4 * quad);
    }
  };
  fetch(part);
  float top = -__builtin_inff();
  for (int c = lane; c < chunks; c += 64) top = fmaxf(top, a.ml[row0 + c * stride].x);
  for (int off = 32; off > 0; off /= 2) top = fmaxf(top, __shfl_xor(top, off, 64));
  Joined j{v4f{0.f, 0.f, 0.f, 0.f}, 0.0f};
  for (int c0 = part; c0 < chunks; c0 += FLY * all) {
    if (c0 > part) fetch(c0);
#pragma unroll
    for (int i = 0; i < FLY; ++i) {
      if (c0 + i * all >= chunks) continue;
      // a part that saw nothing holds zeros, or what scores of NaN made of it
      const float by = ml[i].x == -__builtin_inff() ? (ml[i].y == 0.0f ? 0.0f : 1.0f) : exp2_fast(ml[i].x - top);
      j.l += by * ml[i].y;
      j.v += by * o[i];
    }
  }
  for (int off = per; off < 64; off *= 2) {
    j.l += __shfl_xor(j.l, off, 64);
#pragma unroll
    for (int i = 0; i < 4; ++i) j.v[i] += __shfl_xor(j.v[i], off, 64);
  }
  return j;
}
template <int QT>
__device__ __forceinline__ void put_joined(const AttnArgs& a, int64_t token, int h, int D, const Joined& j) {
  const int lane = threadIdx.x & 63;
  if (lane < D / 4)
    put_4<QT>(a.out + token * a.ldo + (int64_t)h * D + 4 * lane, wide_rows(a.out, a.ldo),
              j.l == 0.0f ? v4f{0.f, 0.f, 0.f, 0.f} : j.v / j.l);
}

// Few rows: a workgroup per (token, head), its waves sharing the parts.
template <int QT>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a, int D) {
  __shared__ v4f sum[4][64];
  __shared__ float sum_l[4];
  const int token = blockIdx.x, lane = threadIdx.x & 63, wave = wave_id();
  const Row w = row_of(a.b, a.w, token);
  const int G = a.w.G, Hk = a.w.kv_heads;
  if (w.s < 0 || w.chunks == 1 || w.slot0 + Hk * w.chunks * w.tiles > a.w.slots) return;   // the last for starts that do not ascend
  const int h = blockIdx.y, col = (token - w.begin) * G + h % G, head = h / G, tile = col / a.w.tile;
  // slot of chunk c: slot0 + (tile * chunks + c) * kv_heads + head
  const int64_t row0 = ((int64_t)w.slot0 + (int64_t)tile * w.chunks * Hk + head) * a.w.tile + col % a.w.tile;
  Joined j = join_row(a, row0, (int64_t)Hk * a.w.tile, w.chunks, wave, 4, D);
  sum[wave][lane] = j.v;
  if (lane == 0) sum_l[wave] = j.l;
  __syncthreads();
  if (wave > 0) return;
  j.l = sum_l[0] + sum_l[1] + sum_l[2] + sum_l[3];
  j.v = sum[0][lane] + sum[1][lane] + sum[2][lane] + sum[3][lane];
  put_joined<QT>(a, token, h, D, j);
}

// Many rows, few of them split: workgroups by split tile (there are at most half
// as many as slots), a wave per column.
template <int QT>
__global__ __launch_bounds__(256) void k_attn_join_tiles(AttnArgs a, int D) {
  const SplitTile t = split_tile(a.b, a.w, blockIdx.x);
  if (t.begin < 0) return;
  const int G = a.w.G;
  for (int c = blockIdx.y * 4 + wave_id(); c < a.w.tile; c += 4 * gridDim.y) {
    const int col = t.tile * a.w.tile + c;
    if (col >= t.n * G) return;
    const Joined j = join_row(a, (int64_t)t.slot * a.w.tile + c, (int64_t)a.w.kv_heads * a.w.tile, t.chunks, 0, 1, D);
    put_joined<QT>(a, t.begin + col / G, t.head * G + col % G, D, j);
  }
}

}  // namespace kqd

namespace kq {
using namespace kqd;

int launch_attn_join(const AttnArgs& a, int type, int D, hipStream_t stream) {
  const dim3 grid((unsigned)a.b.n_tokens, (unsigned)(a.w.G * a.w.kv_heads));
  dispatch_log("k_attn_join", -1, a.w.G * a.w.kv_heads, D, a.b.n_tokens, grid.x, grid.y, 256, 0, "-");
  if (type == KQ_F16) hipLaunchKernelGGL(k_attn_join<A_F16>, grid, dim3(256), 0, stream, a, D);
  else hipLaunchKernelGGL(k_attn_join<A_BF16>, grid, dim3(256), 0, stream, a, D);
  return (int)hipGetLastError();
}
int launch_attn_join_tiles(const AttnArgs& a, int type, int D, hipStream_t stream) {
  const dim3 grid((unsigned)(a.w.slots / 2), (unsigned)(a.w.tile / 16));
  dispatch_log("k_attn_join_tiles", -1, a.w.G * a.w.kv_heads, D, a.b.n_tokens, grid.x, grid.y, 256, 0, "-");
  if (type == KQ_F16) hipLaunchKernelGGL(k_attn_join_tiles<A_F16>, grid, dim3(256), 0, stream, a, D);
  else hipLaunchKernelGGL(k_attn_join_tiles<A_BF16>, grid, dim3(256), 0, stream, a, D);
  return (int)hipGetLastError();
}

AttnArgs attn_args(const AttnCall& p, const AttnPlan& w) {
  AttnArgs a;
  const kq_kv_batch& b = *p.batch;
  const kq_kv_cache& c = *p.cache;
  a.b = Batch{b.page_table, b.table_width, b.q_start, b.lens, b.n_seqs, b.n_tokens};
  a.c = Cache{static_cast<uint8_t*>(c.k), static_cast<uint8_t*>(c.v), c.n_pages, c.kv_heads};
  a.w = Split{p.heads / c.kv_heads, c.kv_heads, w.tile, p.window, w.target, w.least, w.places, w.search, (int)w.slots};
  a.q = static_cast<const uint16_t*>(p.q);
  a.out = static_cast<uint16_t*>(p.out);
  a.tree = p.tree;
  a.part = static_cast<float*>(p.ws);
  a.ml = reinterpret_cast<float2*>(a.part + w.slots * w.tile * c.head_dim);
  a.ldq = p.ldq;
  a.ldo = p.ldo;
  a.scale = p.scale * 1.4426950408889634f;
  return a;
}

namespace {

template <int QT, bool Q8, int DB, int CT>
int decode_launch(const AttnCall& p, const AttnPlan& w) {
  const AttnArgs a = attn_args(p, w);
  dispatch_log("k_attn_decode", -1, p.heads, 32 * DB, p.batch->n_tokens, (unsigned)w.grid, 1, 64 * DEC_WAVES, 0,
               "cache=%d tile=%d slots=%lld", p.cache->type, w.tile, (long long)w.slots);
  hipLaunchKernelGGL((k_attn_decode<QT, Q8, DB, CT>), dim3((unsigned)w.grid), dim3(64 * DEC_WAVES), 0, p.stream, a);
  int err = (int)hipGetLastError();
  if (err || w.slots == 0) return err;
  return launch_attn_join(a, p.type, 32 * DB, p.stream);
}
template <int QT, bool Q8, int DB>
int decode_cols(const AttnCall& p, const AttnPlan& w) {
  if constexpr (!Q8 || DB <= 2)   // (decode_plan)
    if (w.tile == 32) return decode_launch<QT, Q8, DB, 2>(p, w);
  return decode_launch<QT, Q8, DB, 1>(p, w);
}
template <int QT, bool Q8>
int decode_dim(const AttnCall& p, const AttnPlan& w) {
  switch (p.cache->head_dim / 32) {
    case 1: return decode_cols<QT, Q8, 1>(p, w);
    case 2: return decode_cols<QT, Q8, 2>(p, w);
    case 3: return decode_cols<QT, Q8, 3>(p, w);
    case 4: return decode_cols<QT, Q8, 4>(p, w);
    case 5: return decode_cols<QT, Q8, 5>(p, w);
    case 6: return decode_cols<QT, Q8, 6>(p, w);
    case 7: return decode_cols<QT, Q8, 7>(p, w);
    default: return decode_cols<QT, Q8, 8>(p, w);
  }
}

}  // namespace

// Partial results take part in a call only where a table row is longer than
// the shortest chunk.
void finish_plan(const kq_kv_cache& c, const kq_kv_batch& b, int heads, AttnPlan& w) {
  const int64_t G = heads / c.kv_heads;
  const int64_t tiles = c.kv_heads * ((b.n_tokens * G + w.tile - 1) / w.tile + b.n_seqs);
  w.grid = w.target + tiles;
  const bool split = b.table_width > w.least;
  w.slots = split ? (w.grid < 2ll * w.target ? w.grid : 2ll * w.target) : 0;
  if (!split) w.grid = tiles;
  w.bytes = w.slots * w.tile * ((int64_t)c.head_dim + 2) * 4;
}

AttnPlan decode_plan(const kq_kv_cache& c, const kq_kv_batch& b, int heads) {
  AttnPlan w;
  w.search = 0;
  const int64_t cols = ((int64_t)b.n_tokens * (heads / c.kv_heads) + b.n_seqs - 1) / b.n_seqs;   // of a mean sequence
  // Tiles of 32 columns read the cache half as often, tiles of 16 have half the
  // latency per page and fill the chip better; what is read again comes out of the
  // caches unless there is much of it. So 32 where a mean sequence has the columns
  // and the table's pages are above 160 MB: 8 rows x 32 heads (8 of keys) of 131000
  // bf16 positions 107 us (16: 158), of 48000 49 (60); 16 rows of 4 sequences to 8000
  // (131 MB) 34 (33), three trees of 16 rows to 6000 25.3 (22.7). In 8 bits the
  // conversions bound it, and 32 columns of heads above 64 leave the registers of
  // one workgroup: 8 rows of 131000 105 (92), with heads of 64 of 260000 86 (96).
  // The host knows the table's width, not the lengths. With room for 131072
  // positions, as a captured graph keeps it, short sequences pay for it: those trees
  // 25.3, eight sequences of 8 rows at 500 18.3 (a table of their length 15.8), one
  // row at 100 9.3 (6.9, and no workspace).
  const int64_t read = 2ll * b.n_seqs * b.table_width * c.kv_heads * region_bytes(c.type == KQ_KV_Q8_0, c.head_dim);
  const bool wide = cols > 16 && read > 160000000 && (c.type != KQ_KV_Q8_0 || c.head_dim <= 64);
  w.tile = wide ? 32 : 16;
  // Two workgroups to a compute unit, four with heads up to 64, one for wide tiles
  // and heads above 128 in 8 bits (the kernel's launch bounds). With heads of 64: one
  // token at 131071 positions 55.2 us, 53.1 with two, in 8 bits 33.6 (34.7), eight at
  // 8000 18.1 (18.5), in 8 bits 15.5 (16.0). Not all of it fits the registers: 16-bit
  // heads of 224 and 256 keep 12 and 64 of a wave's in scratch (32 columns of 32,
  // 128 and 256: 12, 2 and 50; 8 bits of 256: 67).
  const int work = c.head_dim / 32 * (w.tile / 16);
  w.places = work <= 2 ? 1024 : work <= 4 || (c.type != KQ_KV_Q8_0 && work <= 8) ? 512 : 256;
  // Where tiles alone fill more than a quarter of the places: 64 tokens over 4000
  // positions of 8 heads 119 us, 512 parts 124.
  w.target = w.places > 768 ? w.places : 768;
  // One page per wave is the least; where tiles alone fill half the chip, shorter
  // chunks cost more in the join than they spread: 64 tokens over 500 positions of
  // 8 heads 17.2 us with 16, 27.3 with 4 (one token at 1000 10.8 with 4, 13.1 with 16).
  const int64_t tiles = c.kv_heads * ((b.n_tokens * (int64_t)(heads / c.kv_heads) + w.tile - 1) / w.tile + b.n_seqs);
  w.least = tiles >= 256 ? 16 : 4;
  finish_plan(c, b, heads, w);
  return w;
}

int launch_attn_decode(const AttnCall& p) {
  const AttnPlan w = decode_plan(*p.cache, *p.batch, p.heads);
  const bool q8 = p.cache->type == KQ_KV_Q8_0;
  if (p.type == KQ_F16) return q8 ? decode_dim<A_F16, true>(p, w) : decode_dim<A_F16, false>(p, w);
  return q8 ? decode_dim<A_BF16, true>(p, w) : decode_dim<A_BF16, false>(p, w);
}

}  // namespace kq
