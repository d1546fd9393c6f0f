// kq_mx4_moe.hip — the router of a mixture of experts, and the whole layer
// (router, chosen experts' gated FFN with microscaled 4-bit weights, weighted
// sum) for a few tokens.
//
// Only the experts in use are read (kinfer page, "Models bigger than the
// machine"; Kinetic docs, "What makes it fast").
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq_internal.h"
#include "kq_mx4_dev.h"

namespace kqd {

// ---- Router logits: l[m][e] = sum_k x[m][k] W[e][k], in 64 bits throughout,
// so the choice of experts does not depend on the order of summation unless
// two logits agree to about 50 bits. v_mfma_f64_16x16x4 takes 16 experts
// and 16 tokens; a lane (r = lane & 15, g = lane >> 4) supplies elements
// 32 it + 8 g + j of expert row r and token row r to instruction j of step it.
// A workgroup is one such tile and a part of K (blockIdx.z); its waves split that
// and meet in LDS in wave order, and the choice adds the parts in their order.
// Bound by one round trip to memory, which is why K is split over workgroups as
// well: 128 experts of 2048 fp16 inputs 4.7 us (in one part 7), 512 experts of
// 2048 bf16 inputs at 48 tokens 5.6.
template <int T>
__device__ __forceinline__ void to_f64(const u32x4 (&v)[T == T_F32 ? 2 : 1], double (&d)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float f;
    if constexpr (T == T_F32) {
      f = bits_f32(v[j / 4][j % 4]);
    } else {
      const uint32_t h = (v[0][j / 2] >> (16 * (j & 1))) & 0xffffu;
      f = T == T_F16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)h) : __builtin_bit_cast(float, h << 16);
    }
    d[j] = (double)f;
  }
}

constexpr int ROUTE_WAVES = 8, ROUTE_SPLITS = 8;

template <int XT, int WT>
__global__ __launch_bounds__(64 * ROUTE_WAVES) void k_route_logits(const void* __restrict__ x,
                                                                  const uint8_t* __restrict__ W,
                                                                  double* __restrict__ part, int M, int K, int E) {
  __shared__ v4d red[ROUTE_WAVES][64];
  const int lane = threadIdx.x & 63, wave = wave_id(), r = lane & 15, g = lane >> 4;
  const int e0 = blockIdx.x * 16, m0 = blockIdx.y * 16, nit = K / 32;
  const int i0 = nit * (int)blockIdx.z / (int)gridDim.z, i1 = nit * ((int)blockIdx.z + 1) / (int)gridDim.z;
  const uint32_t xrow = (uint32_t)K * TypeSize<XT>::v, wrow = (uint32_t)K * TypeSize<WT>::v;
  const int erows = E - e0 < 16 ? E - e0 : 16, mrows = M - m0 < 16 ? M - m0 : 16;
  const rsrc_t rw = make_rsrc(W + (int64_t)e0 * wrow, (uint32_t)erows * wrow);
  const rsrc_t rx = make_rsrc(static_cast<const uint8_t*>(x) + (int64_t)m0 * xrow, (uint32_t)mrows * xrow);
  const uint32_t wo = r < erows ? (uint32_t)r * wrow : OOB, xo = r < mrows ? (uint32_t)r * xrow : OOB;
  v4d acc = {0., 0., 0., 0.};
  for (int it = i0 + wave; it < i1; it += ROUTE_WAVES) {
    const int k = 32 * it + 8 * g;
    u32x4 xv[XT == T_F32 ? 2 : 1], wv[WT == T_F32 ? 2 : 1];
#pragma unroll
    for (int i = 0; i < (WT == T_F32 ? 2 : 1); ++i) wv[i] = ld128(rw, wo + (uint32_t)k * TypeSize<WT>::v + 16u * i);
#pragma unroll
    for (int i = 0; i < (XT == T_F32 ? 2 : 1); ++i) xv[i] = ld128(rx, xo + (uint32_t)k * TypeSize<XT>::v + 16u * i);
    double xd[8], wd[8];
    to_f64<XT>(xv, xd);
    to_f64<WT>(wv, wd);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc = __builtin_amdgcn_mfma_f64_16x16x4f64(wd[j], xd[j], acc, 0, 0, 0);
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (threadIdx.x < 256) {
    const int l = threadIdx.x >> 2, i = threadIdx.x & 3;
    double s = red[0][l][i];
    for (int w = 1; w < ROUTE_WAVES; ++w) s += red[w][l][i];
    // result element i of lane l: expert 4 i + (l >> 4), token l & 15
    const int e = 4 * i + (l >> 4), m = l & 15;
    if (e < erows && m < mrows) part[((int64_t)blockIdx.z * M + m0 + m) * E + e0 + e] = s;
  }
}

// ---- Choice of a token's top_k largest logits by one workgroup, a thread per
// expert: the larger first, the lower index on ties, NaN below every number.
// A wave ranks its 64 experts against each other (64 comparisons a lane, the
// other keys through scalar registers) and passes on its top_k best in order;
// these candidates are ranked against each other in the same way. Logits are
// compared as integers that order like them; 0 is below every logit. Bound by
// latency: 3.6 us for one token of 128 experts (picking them one at a time 8.6),
// 7.3 for 48 tokens of 512 (15.2).
__device__ __forceinline__ uint64_t logit_key(double v) {
  if (!(v == v)) v = -__builtin_inf();
  if (v == 0.0) v = 0.0;   // -0 and +0 are equal
  const int64_t b = __builtin_bit_cast(int64_t, v);
  return (uint64_t)b ^ ((uint64_t)(b >> 63) | 0x8000000000000000ull);
}

// Scratch of a workgroup's choice, for `waves` waves.
struct SelectLds {
  uint64_t* key;    // [waves * top_k]
  double* raw;      // [waves * top_k]
  double* best;     // [64]
  double* sum;      // [16]
  int* id;          // [waves * top_k]
  int* chosen;      // [64]
  __device__ __forceinline__ SelectLds(void* lds, int waves, int top_k) {
    key = static_cast<uint64_t*>(lds);
    raw = reinterpret_cast<double*>(key + waves * top_k);
    best = raw + waves * top_k;
    sum = best + 64;
    id = reinterpret_cast<int*>(sum + 16);
    chosen = id + waves * top_k;
  }
};
__host__ __device__ constexpr int select_lds_bytes(int waves, int top_k) { return waves * top_k * 20 + 64 * 8 + 16 * 8 + 64 * 4; }

// The choice for token m by a workgroup of `waves` waves, at least a thread per
// expert: S.chosen has it for every thread on return; ids and weights are
// written where `write` is set.
__device__ __forceinline__ void select_experts(const double* __restrict__ part, int splits, int m, int M, int E,
                                               int top_k, int renorm, int waves, const SelectLds& S, bool write,
                                               int32_t* __restrict__ ids, float* __restrict__ weights) {
  const int e = threadIdx.x, lane = threadIdx.x & 63, wave = wave_id();
  double raw = 0.0;
  if (e < E) {
    double p[ROUTE_SPLITS];
#pragma unroll
    for (int s = 0; s < ROUTE_SPLITS; ++s) p[s] = s < splits ? part[((int64_t)s * M + m) * E + e] : 0.0;
    raw = p[0];
#pragma unroll
    for (int s = 1; s < ROUTE_SPLITS; ++s)
      if (s < splits) raw += p[s];
  }
  const uint64_t key = e < E ? logit_key(raw) : 0ull;
  const uint32_t klo = (uint32_t)key, khi = (uint32_t)(key >> 32);
  // Upper halves first; whole keys where two of the wave's agree in them.
  int rank = 0, same = 0;
#pragma unroll 16
  for (int j = 0; j < 64; ++j) {
    const uint32_t hj = (uint32_t)__builtin_amdgcn_readlane((int)khi, j);
    rank += hj > khi;
    same += hj == khi;
  }
  if (__any(e < E && same > 1)) {
    rank = 0;
    for (int j = 0; j < 64; ++j) {
      const uint64_t kj = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)klo, j) |
                          (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)khi, j) << 32;
      rank += kj > key || (kj == key && j < lane);
    }
  }
  // lanes past the experts all have key 0 and the same rank: they come after
  // the experts in lane order
  if (e >= E && wave * 64 < E) rank = lane;
  if (rank < top_k) {
    const int at = wave * top_k + rank;
    S.key[at] = key;
    S.raw[at] = raw;
    S.id[at] = e;
  }
  __syncthreads();
  const int C = (E + 63) / 64 * top_k;   // waves past the experts have no candidates
  if ((int)threadIdx.x < C) {
    const uint64_t mine = S.key[threadIdx.x];
    int at = (int)threadIdx.x;
    if (C > top_k) {
      at = 0;
#pragma unroll 8
      for (int j = 0; j < C; ++j) {
        const uint64_t kj = S.key[j];
        at += kj > mine || (kj == mine && j < (int)threadIdx.x);
      }
    }
    if (at < top_k) {
      S.best[at] = S.raw[threadIdx.x];
      S.chosen[at] = S.id[threadIdx.x];
    }
  }
  __syncthreads();
  if (!write) return;
  const double first = S.best[0];
  if (!renorm) {
    double p = e < E ? exp(raw - first) : 0.0;
    for (int off = 32; off > 0; off >>= 1) p += __shfl_xor(p, off, 64);
    if (lane == 0) S.sum[wave] = p;
    __syncthreads();
  }
  if (wave > 0) return;
  const double mine = lane < top_k ? exp(S.best[lane] - first) : 0.0;
  double sum = 0.0;
  if (renorm) {
    sum = mine;
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
  } else {
    for (int w = 0; w < waves; ++w) sum += S.sum[w];
  }
  if (lane < top_k) {
    ids[m * top_k + lane] = S.chosen[lane];
    weights[m * top_k + lane] = (float)(mine / sum);
  }
}

__global__ __launch_bounds__(1024) void k_route_select(const double* __restrict__ part, int splits, int M, int E,
                                                       int top_k, int renorm, int32_t* __restrict__ ids,
                                                       float* __restrict__ weights) {
  extern __shared__ u32x4 lds4[];
  const int waves = blockDim.x >> 6;
  select_experts(part, splits, blockIdx.x, M, E, top_k, renorm, waves, SelectLds(lds4, waves, top_k), true, ids, weights);
}

// ---- Slots (token * top_k + rank) of one expert, found by a wave among the P
// ids in LDS: their number, and their indices in increasing order in list.
__device__ __forceinline__ int gather_slots(const uint16_t* ids, int P, int e, uint16_t* list) {
  const int lane = threadIdx.x & 63;
  int n = 0;
  for (int p0 = 0; p0 < P; p0 += 64) {
    const bool hit = p0 + lane < P && ids[p0 + lane] == e;
    const uint64_t mask = __ballot(hit);
    if (hit) list[n + __popcll(mask & ((1ull << lane) - 1ull))] = (uint16_t)(p0 + lane);
    n += __popcll(mask);
  }
  return n;
}

// Whether an earlier slot has the expert of slot p (wave-uniform).
__device__ __forceinline__ bool earlier_slot(const uint16_t* ids, int p, int e) {
  const int lane = threadIdx.x & 63;
  for (int p0 = 0; p0 < p; p0 += 64)
    if (__any(p0 + lane < p && ids[p0 + lane] == e)) return true;
  return false;
}

// The down projection takes up to DOWN_SLOTS slots of an expert at a time. The
// first of each group leads it: its entry of `groups` has the group's size in
// the upper half, others 0; the lower half is the next slot with the expert.
constexpr int DOWN_SLOTS = 3;
__device__ __forceinline__ void write_groups(const uint16_t* list, int cnt, int32_t* __restrict__ groups) {
  for (int t = threadIdx.x & 63; t < cnt; t += 64) {
    const int size = t % DOWN_SLOTS == 0 ? min(DOWN_SLOTS, cnt - t) : 0;
    groups[list[t]] = size << 16 | (t + 1 < cnt ? list[t + 1] : 0);
  }
}

// Three bf16 pieces of an fp32 value (as split3).
__device__ __forceinline__ void split3_one(float v, uint16_t& hi, uint16_t& mid, uint16_t& lo) {
  const uint32_t b0 = __builtin_bit_cast(uint32_t, v);
  const float vh = __builtin_bit_cast(float, b0 & 0xffff0000u);
  const float r1 = v == vh ? 0.0f : v - vh;
  const uint32_t b1 = __builtin_bit_cast(uint32_t, r1);
  hi = (uint16_t)(b0 >> 16);
  mid = (uint16_t)(b1 >> 16);
  lo = (uint16_t)(__builtin_bit_cast(uint32_t, r1 - __builtin_bit_cast(float, b1 & 0xffff0000u)) >> 16);
}

// ---- Gate and up rows of one expert for the tokens routed to it:
// h[slot][n] = silu(gate_n . x) * (up_n . x), silu(z) = z / (1 + e^-z), kept
// as three bf16 planes whose sum is the fp32 value (no rounding of h), ready
// as operands of the down projection. Grid (inter / 16 TILES, min(E, P), Z):
// workgroup z takes the expert's passes of columns z, z + Z, ...; row y is
// expert y, or, with fewer slots than experts, the expert of slot y unless an
// earlier slot has it. One token: its experts differ, and where a workgroup
// has a thread per expert (splits > 0) each makes the choice itself, the first
// one writing ids and weights, which saves a launch between two others.
// The waves split K; each stages its part of the tokens once and walks TILES
// tiles of 16 gate and 16 up rows. The partial sums meet in LDS in wave order,
// where the regions were. 16 tokens of 128 experts of 768 x 2048, top 8, read 137
// MB of weights of some 82 experts in 31 us, 4.4 TB/s, where a kernel that only
// reads them takes 22: a wave's region is filled, waited for and then multiplied,
// with the other waves' copies in flight meanwhile. One token takes 8.7 us for
// 13.4 MB, most of it the latency of the choice, the copies and the launch. An
// expert's weights come again for each pass of its slots: 64 tokens of 16
// experts of 1536 x 4096, top 4, are far from their bytes (layer 153 us, 26).
// Dynamic LDS: waves * PER_WAVE, then ids and list (P uint16 each).
template <int XT, int TILES, int COLS>   // COLS: columns in a pass
struct GateUp {
  static constexpr int CHUNKS = XT == T_F32 ? 2 : 4;   // of K in a wave's region
  static constexpr int X = x_region_bytes<XT, CHUNKS>(COLS), REGION = X + w_region_bytes<2, CHUNKS>();
  static constexpr int PER_WAVE = TILES * 2048 > REGION ? TILES * 2048 : REGION;
  static constexpr int MAX_WAVES = 8;
};

template <int XT, int TILES, int COLS, bool AL>
__global__ __launch_bounds__((GateUp<XT, TILES, COLS>::MAX_WAVES * 64)) void k_mx4_gate_up(
    const uint8_t* __restrict__ gc, const uint8_t* __restrict__ gs, const uint8_t* __restrict__ uc,
    const uint8_t* __restrict__ us, const void* __restrict__ x, int32_t* __restrict__ ids, uint16_t* __restrict__ h,
    int hidden, int inter, int M, int top_k, int E, int waves, const double* __restrict__ part, int splits, int renorm,
    float* __restrict__ weights, int32_t* __restrict__ groups) {
  constexpr int U = GateUp<XT, TILES, COLS>::CHUNKS, PER_WAVE = GateUp<XT, TILES, COLS>::PER_WAVE;
  extern __shared__ u32x4 lds4[];
  uint8_t* lds = reinterpret_cast<uint8_t*>(lds4);
  uint16_t* s_ids = reinterpret_cast<uint16_t*>(lds + waves * PER_WAVE);
  const int P = M * top_k, y = blockIdx.y;
  uint16_t* list = s_ids + P;
  const int lane = threadIdx.x & 63, wave = wave_id(), r = lane & 15, g = lane >> 4;
  int e, cnt;
  if (M == 1) {
    if (splits > 0) {
      const SelectLds S(lds, waves, top_k);
      select_experts(part, splits, 0, 1, E, top_k, renorm, waves, S, blockIdx.x == 0 && y == 0, ids, weights);
      e = __builtin_amdgcn_readfirstlane(S.chosen[y]);
      __syncthreads();   // read before the regions take its place
    } else {
      e = __builtin_amdgcn_readfirstlane(ids[y]);
    }
    cnt = 1;
    if (lane == 0) list[0] = (uint16_t)y;   // every wave writes the same
  } else {
    for (int p = threadIdx.x; p < P; p += 64 * waves) s_ids[p] = (uint16_t)ids[p];
    __syncthreads();
    e = P <= E ? __builtin_amdgcn_readfirstlane(s_ids[y]) : y;
    if (P <= E && earlier_slot(s_ids, y, e)) return;
    cnt = gather_slots(s_ids, P, e, list);   // every wave writes the same list
    if (cnt == 0) return;
  }
  if (blockIdx.x == 0 && blockIdx.z == 0 && wave == 0) write_groups(list, cnt, groups);
  const int nblk = hidden / 32, nchunk = (nblk + 3) / 4, tile0 = blockIdx.x * TILES;
  const uint32_t xrow = (uint32_t)hidden * TypeSize<XT>::v;
  const rsrc_t rx = make_rsrc(x, (uint32_t)M * xrow);
  const int c0 = nchunk * wave / waves, c1 = nchunk * (wave + 1) / waves;
  const int64_t plane = (int64_t)P * inter;
  uint8_t* xl = lds + wave * PER_WAVE;
  uint8_t* wl = xl + GateUp<XT, TILES, COLS>::X;
  for (int t0 = COLS * (int)blockIdx.z; t0 < cnt; t0 += COLS * (int)gridDim.z) {
    if (t0 >= COLS * (int)gridDim.z) __syncthreads();   // the previous pass has read the sums
    const int cols = min(COLS, cnt - t0);
    const uint32_t xoff = lane < cols ? (uint32_t)(list[t0 + lane] / top_k) * xrow : 0u;   // of column `lane`
    const auto off = [=](int c) { return (uint32_t)__shfl((int)xoff, c, 64); };
    const int have = r < cols ? r : 0;
    const uint8_t* xr[1] = {xl + have * (Pieces<XT>::v * U * 16)};
    v4f acc[TILES][2][1];
    const auto walk = [&](auto large) {
      uint32_t seen = 0;
#pragma unroll
      for (int t = 0; t < TILES; ++t) acc[t][0][0] = acc[t][1][0] = v4f{0.f, 0.f, 0.f, 0.f};
      for (int c = c0; c < c1; c += U) {   // once, unless K is longer than the waves' regions
        stage_x<XT, U>(rx, xl, cols, off, c, min(c1 * Pieces<XT>::v, nblk * (Pieces<XT>::v / 4)));
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          rsrc_t rc[2], rs[2];
          const int rows = 16 * (tile0 + t) < inter ? 16 : 0;
          const int64_t row = (int64_t)e * inter + (rows ? 16 * (tile0 + t) : 0);
          mx4_rows(gc, gs, row, rows, nblk, rc[0], rs[0]);
          mx4_rows(uc, us, row, rows, nblk, rc[1], rs[1]);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            stage_w<U, AL>(rc[i], rs[i], wl + i * U * 1024, wl + 2 * U * 1024 + i * U * 64, c, min(4 * c1, nblk), nblk);
          regions_filled();
          step_products<decltype(large)::value, XT, 1, 2, U>(xr, have & 7, c1 - c, wl, r, g, acc[t], seen);
          regions_read();
        }
      }
      return seen;
    };
    if (again<XT>(walk(Large<false>()))) walk(Large<true>());
    __syncthreads();   // the sums take the regions' place
    v4f* red = reinterpret_cast<v4f*>(lds);   // [wave][tile][gate, up][64]
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      red[((wave * TILES + t) * 2 + 0) * 64 + lane] = acc[t][0][0];
      red[((wave * TILES + t) * 2 + 1) * 64 + lane] = acc[t][1][0];
    }
    __syncthreads();
    for (int j = threadIdx.x; j < TILES * 256; j += 64 * waves) {
      // result element i of lane l of tile t: column 4 (l >> 4) + i, row l & 15
      const int i = j & 3, l = (j >> 2) & 63, t = j >> 8, col = 4 * (l >> 4) + i;
      const int n = 16 * (tile0 + t) + (l & 15);
      if (col < cols && n < inter) {
        float gv = 0.f, uv = 0.f;
        for (int w = 0; w < waves; ++w) {
          gv += red[((w * TILES + t) * 2 + 0) * 64 + l][i];
          uv += red[((w * TILES + t) * 2 + 1) * 64 + l][i];
        }
        uint16_t* o = h + (int64_t)list[t0 + col] * inter + n;
        split3_one(gv / (1.0f + expf(-gv)) * uv, o[0], o[plane], o[2 * plane]);
      }
    }
  }
}

// ---- Down projection and weighted sum: y[m] = sum_j w[m][j] Down_e h[m][j].
// A workgroup owns 16 rows of y for every token; its waves take the experts in
// use in turn, up to SLOTS slots of one at a time (of all gridDim.y workgroups'
// waves, wave w the groups led by slots w, w + all waves, ...), each into sums
// of its own in LDS, and the waves' sums are added in wave order, so the result
// does not depend on timing. With more than one workgroup for the rows, out is
// theirs in turn and k_mx4_down_sum adds them. The operand columns are the
// three pieces of h of a group's slots. Bound by a wave's own copies, which it
// waits for with nothing else in flight, three times per group at 768 inputs: 16
// tokens of 128 experts of 768 to 2048, top 8, 22.4 us and 4.8 for the sum of the
// parts (68 MB of weights, 3.0 TB/s; reading them alone takes 11.8), one token 5.7.
// Dynamic LDS: per wave a region, then per wave M x 16 sums, then the route
// weights (P fp32), groups (P int32) and ids (P uint16).
template <int U, int SLOTS, bool AL>
__global__ __launch_bounds__(1024) void k_mx4_down(const uint8_t* __restrict__ dc, const uint8_t* __restrict__ ds,
                                                  const uint16_t* __restrict__ h, const int32_t* __restrict__ ids,
                                                  const float* __restrict__ weights,
                                                  const int32_t* __restrict__ groups, float* __restrict__ out,
                                                  int hidden, int inter, int M, int top_k, int waves) {
  constexpr int X = x_region_bytes<T_BF16, U>(3 * SLOTS), REGION = X + w_region_bytes<1, U>(), PR = Pieces<T_BF16>::v * U;
  static_assert(X >= 1024, "the region serves the results too");
  extern __shared__ u32x4 lds4[];
  const int lane = threadIdx.x & 63, wave = wave_id(), P = M * top_k, r = lane & 15, g = lane >> 4;
  uint8_t* xl = reinterpret_cast<uint8_t*>(lds4) + wave * REGION;
  uint8_t* wl = xl + X;
  float* sums = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(lds4) + waves * REGION);
  float* ys = sums + wave * M * 16;
  float* s_w = sums + waves * M * 16;
  int32_t* s_groups = reinterpret_cast<int32_t*>(s_w + P);
  uint16_t* s_ids = reinterpret_cast<uint16_t*>(s_groups + P);
  const int nblk = inter / 32, nchunk = (nblk + 3) / 4;
  const uint32_t hrow = (uint32_t)inter * 2u;
  const rsrc_t rh = make_rsrc(h, 3u * (uint32_t)P * hrow);
  const int all = waves * (int)gridDim.y;
  const int first = (int)blockIdx.y * waves + wave;
  int e = first < P ? __builtin_amdgcn_readfirstlane(ids[first]) : 0;
  for (int i = threadIdx.x; i < P; i += 64 * waves) {
    s_ids[i] = (uint16_t)ids[i];
    s_w[i] = weights[i];
    s_groups[i] = groups[i];
  }
  for (int i = lane; i < M * 16; i += 64) ys[i] = 0.0f;
  __syncthreads();
  // e: the expert of the wave's first group
  const auto walk = [&](auto large, int p, int e) {
    uint32_t seen = 0;
    while (p < P) {
      int pn = p + all;
      while (pn < P && s_groups[pn] < 1 << 16) pn += all;
      const int en = pn < P ? __builtin_amdgcn_readfirstlane(s_ids[pn]) : 0;
      // column piece * n + m: that piece of h of slot m of this group
      const int n = __builtin_amdgcn_readfirstlane(s_groups[p] >> 16), piece = r / n, m = r - piece * n;
      int slots[SLOTS];
      slots[0] = p;
#pragma unroll
      for (int k = 1; k < SLOTS; ++k) slots[k] = k < n ? __builtin_amdgcn_readfirstlane(s_groups[slots[k - 1]] & 0xffff) : p;
      int mine = p;   // slot of this lane's column
#pragma unroll
      for (int k = 1; k < SLOTS; ++k) mine = m == k ? slots[k] : mine;
      const uint32_t xoff = piece < 3 ? (uint32_t)(piece * P + mine) * hrow : 0u;
      const auto off = [=](int row) { return (uint32_t)__shfl((int)xoff, row, 64); };
      const int have = piece < 3 ? r : 0;
      const uint8_t* xr[1] = {xl + have * (PR * 16)};
      v4f acc[1][1] = {};
      rsrc_t rc[1], rs[1];
      mx4_rows(dc, ds, (int64_t)e * hidden + blockIdx.x * 16, 16, nblk, rc[0], rs[0]);
      for (int c = 0; c < nchunk; c += U) {
        stage_w<U, AL>(rc[0], rs[0], wl, wl + U * 1024, c, nblk, nblk);
        stage_x<T_BF16, U>(rh, xl, 3 * n, off, c, nblk * (Pieces<T_BF16>::v / 4));
        regions_filled();
        step_products<decltype(large)::value, T_BF16, 1, 1, U>(xr, have & 7, nchunk - c, wl, r, g, acc, seen);
        regions_read();
      }
      // the results take the region's place, 16 rows (columns of h) of 16
      float* res = reinterpret_cast<float*>(xl);
#pragma unroll
      for (int i = 0; i < 4; ++i) res[(4 * g + i) * 16 + r] = acc[0][0][i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      for (int i = lane; i < n * 16; i += 64) {
        int slot = p;
#pragma unroll
        for (int k = 1; k < SLOTS; ++k) slot = (i >> 4) == k ? slots[k] : slot;
        const float v = res[2 * n * 16 + i] + res[n * 16 + i] + res[i];
        float* o = ys + (slot / top_k) * 16 + (i & 15);
        *o = __builtin_fmaf(s_w[slot], v, *o);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read before the next copies land there
      p = pn;
      e = en;
    }
    return seen;
  };
  int p0 = first;
  if (M > 1) {
    while (p0 < P && s_groups[p0] < 1 << 16) p0 += all;
    if (p0 < P) e = __builtin_amdgcn_readfirstlane(s_ids[p0]);
  }
  if (again<T_BF16>(walk(Large<false>(), p0, e))) {
    for (int i = lane; i < M * 16; i += 64) ys[i] = 0.0f;
    walk(Large<true>(), p0, e);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < M * 16; i += 64 * waves) {
    float s = sums[i];
    for (int w = 1; w < waves; ++w) s += sums[w * M * 16 + i];
    out[((int64_t)blockIdx.y * M + (i >> 4)) * hidden + blockIdx.x * 16 + (i & 15)] = s;
  }
}

// y = the parts' sum in their order, four values a thread (hidden % 32 == 0).
__global__ __launch_bounds__(256) void k_mx4_down_sum(const v4f* __restrict__ parts, v4f* __restrict__ y, int n4,
                                                      int count) {
  const int i = (int)blockIdx.x * 256 + (int)threadIdx.x;
  if (i >= n4) return;
  v4f s = parts[i];
  for (int z = 1; z < count; ++z) s += parts[(int64_t)z * n4 + i];
  y[i] = s;
}

}  // namespace kqd

namespace kq {

using namespace kqd;

namespace {

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

// Parts K is split into: one step of 32 per wave, so that a workgroup's loads
// are one round trip.
int route_splits(int64_t K) {
  const int64_t s = K / 32 / ROUTE_WAVES;
  return s < 1 ? 1 : s > ROUTE_SPLITS ? ROUTE_SPLITS : (int)s;
}

template <int XT>
int logits_x(const RouteArgs& a, double* part) {
  const dim3 grid((unsigned)((a.E + 15) / 16), (unsigned)((a.M + 15) / 16), (unsigned)route_splits(a.K)), block(64 * ROUTE_WAVES);
  const uint8_t* W = static_cast<const uint8_t*>(a.W);
  dispatch_log("k_route_logits", -1, a.E, a.K, a.M, grid.x, grid.y, block.x, 0, "x=%d w=%d splits=%u", XT, a.wtype, grid.z);
#define KQ_LAUNCH(WT) hipLaunchKernelGGL((k_route_logits<XT, WT>), grid, block, 0, a.stream, a.x, W, part, a.M, (int)a.K, a.E)
  if (a.wtype == KQ_F32) KQ_LAUNCH(T_F32);
  else if (a.wtype == KQ_F16) KQ_LAUNCH(T_F16);
  else KQ_LAUNCH(T_BF16);
#undef KQ_LAUNCH
  return (int)hipGetLastError();
}

}  // namespace

int64_t route_workspace_bytes(int M, int E) { return (int64_t)ROUTE_SPLITS * M * E * 8; }

namespace {

int launch_logits(const RouteArgs& a) {
  double* part = static_cast<double*>(a.ws);
  return a.xtype == KQ_F32 ? logits_x<T_F32>(a, part) : a.xtype == KQ_F16 ? logits_x<T_F16>(a, part) : logits_x<T_BF16>(a, part);
}

}  // namespace

int launch_route(const RouteArgs& a) {
  double* part = static_cast<double*>(a.ws);
  const int err = launch_logits(a);
  if (err) return err;
  int threads = 64;   // a thread per expert, whole waves in a power of two
  while (threads < a.E) threads *= 2;
  const size_t lds = (size_t)select_lds_bytes(threads / 64, a.top_k);
  dispatch_log("k_route_select", -1, a.E, a.K, a.M, (unsigned)a.M, 1, (unsigned)threads, lds, "top_k=%d", a.top_k);
  hipLaunchKernelGGL(k_route_select, dim3((unsigned)a.M), dim3((unsigned)threads), lds, a.stream, part, route_splits(a.K),
                     a.M, a.E, a.top_k, a.renorm, a.ids, a.weights);
  return (int)hipGetLastError();
}

namespace {

constexpr int MOE_LDS_BYTES = 160 * 1024;   // of a compute unit

// One token's experts are chosen in the gate and up kernel where a workgroup of
// up to 8 waves has a thread per expert.
bool chooses_itself(const Mx4MoeArgs& a) {
  return a.route.M == 1 && a.route.E <= 512 && (a.inter / 32) * a.route.top_k < 512;
}

template <int XT, int TILES, int COLS>
int gate_up_cfg(const Mx4MoeArgs& a, uint16_t* h, int32_t* groups) {
  typedef GateUp<XT, TILES, COLS> G;
  constexpr int U = G::CHUNKS;
  const RouteArgs& r = a.route;
  const int P = r.M * r.top_k, nchunk = (int)((r.K / 32 + 3) / 4);
  int waves = (nchunk + U - 1) / U;   // a wave's part of K in its region, while the waves last
  waves = waves > G::MAX_WAVES ? G::MAX_WAVES : waves;
  const int splits = chooses_itself(a) ? route_splits(r.K) : 0;
  if (splits)   // a thread per expert, and the choice's scratch
    while (waves * 64 < r.E || waves * G::PER_WAVE < select_lds_bytes(waves, r.top_k)) ++waves;
  // passes of twice an expert's mean number of slots (54 tokens, 15 experts of
  // 480 x 896, top 11: 15.5 us against 56.5 with one workgroup walking all passes)
  const int mean2 = (2 * P + r.E - 1) / r.E, z = (mean2 + COLS - 1) / COLS;
  const dim3 grid((unsigned)((a.inter / 16 + TILES - 1) / TILES), (unsigned)(P < r.E ? P : r.E), (unsigned)(z > 8 ? 8 : z));
  const size_t lds = (size_t)waves * G::PER_WAVE + (size_t)P * 4;
  dispatch_log("k_mx4_gate_up", -1, a.inter, r.K, r.M, grid.x, grid.y, (unsigned)(64 * waves), lds, "type=%d tiles=%d cols=%d chooses=%d", XT, TILES, COLS, splits > 0);
  auto* k = r.K % 128 == 0 ? k_mx4_gate_up<XT, TILES, COLS, true> : k_mx4_gate_up<XT, TILES, COLS, false>;
  hipLaunchKernelGGL(k, grid, dim3((unsigned)(64 * waves)), lds, r.stream, a.codes[0], a.scales[0], a.codes[1],
                     a.scales[1], r.x, r.ids, h, (int)r.K, (int)a.inter, r.M, r.top_k, r.E, waves,
                     static_cast<const double*>(r.ws), splits, r.renorm, r.weights, groups);
  return (int)hipGetLastError();
}

// Two tiles per workgroup spread what a workgroup does once over more rows
// where the slots still fill the compute units (16 fp32 tokens, 128 experts of
// 768 x 2048, top 8: layer 88 us against 96 with one and 92 with four; bf16 66,
// 66 and 70). Passes of four
// columns leave room for three workgroups per compute unit (those 16 tokens: 31
// us against 35); experts with four slots and more on average take eight in
// bf16 and fp16 (64 tokens, 16 experts of 1536 x 4096, top 4: layer 169 us
// against 219).
template <int XT>
int gate_up_x(const Mx4MoeArgs& a, uint16_t* h, int32_t* groups) {
  const int P = a.route.M * a.route.top_k;
  const bool two = (a.inter / 32) * (P < a.route.E ? P : a.route.E) >= 512;
  if constexpr (XT != T_F32)
    if (P >= 4 * a.route.E) return two ? gate_up_cfg<XT, 2, 8>(a, h, groups) : gate_up_cfg<XT, 1, 8>(a, h, groups);
  return two ? gate_up_cfg<XT, 2, 4>(a, h, groups) : gate_up_cfg<XT, 1, 4>(a, h, groups);
}

// Workgroups that share the down projection's rows: with many slots, or few
// rows, one workgroup per 16 rows leaves compute units idle (and each reads all
// of h). Two per compute unit, four slots and more each; the sum of the parts
// costs a launch of 4.8 us. Layers of 128 experts with 768 inner values, top 8, in
// us with one part, two, four and eight: 2048 rows, 4 tokens 30.9, 31.5, 30.0,
// 31.4; 8 tokens 48.5, 47.7, 43.0, 46.4; 16 tokens 68.9, 68.6, 61.8, 65.1; 1024
// rows, 4 tokens 26.1, 25.9, 24.0, 25.4; 16 tokens 55.8, 52.5, 43.8, 40.6; 4096
// rows, 16 tokens 118, 121, 124, 130 (the rule's two cost 2 % there).
int down_parts(int64_t hidden, int P) {
  if (P < 64 && hidden > 1024) return 1;
  const int64_t fill = 512 / (hidden / 16), most = P / 4;
  const int64_t n = fill < most ? fill : most;
  return n < 2 ? 1 : n > 16 ? 16 : (int)n;
}

template <int U, int SLOTS>
int down_cfg(const Mx4MoeArgs& a, const uint16_t* h, const int32_t* groups, float* parts, int count) {
  const RouteArgs& r = a.route;
  const int P = r.M * r.top_k;
  // a wave per slot up to what LDS holds; two workgroups to a compute unit where there are parts
  const int shared = P * 10, per_wave = x_region_bytes<T_BF16, U>(3 * SLOTS) + w_region_bytes<1, U>() + r.M * 64;
  int waves = (MOE_LDS_BYTES / (count > 1 ? 2 : 1) - shared) / per_wave;
  const int most = count > 1 ? 8 : 16;
  waves = waves > most ? most : waves < 1 ? 1 : waves;
  waves = waves > P ? P : waves;
  const dim3 grid((unsigned)(r.K / 16), (unsigned)count);
  const size_t lds = (size_t)(shared + waves * per_wave);
  dispatch_log("k_mx4_down", -1, r.K, a.inter, r.M, grid.x, grid.y, (unsigned)(64 * waves), lds, "u=%d slots=%d", U, SLOTS);
  auto* k = a.inter % 128 == 0 ? k_mx4_down<U, SLOTS, true> : k_mx4_down<U, SLOTS, false>;
  hipLaunchKernelGGL(k, grid, dim3((unsigned)(64 * waves)), lds, r.stream, a.codes[2], a.scales[2], h, r.ids,
                     r.weights, groups, count > 1 ? parts : a.y, (int)r.K, (int)a.inter, r.M, r.top_k, waves);
  int err = (int)hipGetLastError();
  if (err || count == 1) return err;
  const int n4 = (int)(r.M * r.K / 4);
  dispatch_log("k_mx4_down_sum", -1, r.K, a.inter, r.M, (unsigned)((n4 + 255) / 256), 1, 256, 0, "parts=%d", count);
  hipLaunchKernelGGL(k_mx4_down_sum, dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, r.stream,
                     reinterpret_cast<const v4f*>(parts), reinterpret_cast<v4f*>(a.y), n4, count);
  return (int)hipGetLastError();
}

}  // namespace

namespace {

// Byte offsets in the workspace, after the logits' parts.
struct MoeLayout {
  int64_t h, groups, parts, total;
};
MoeLayout moe_layout(int64_t hidden, int64_t inter, int M, int top_k, int E) {
  const int64_t P = (int64_t)M * top_k, n = down_parts(hidden, (int)P);
  MoeLayout L;
  L.h = up256(route_workspace_bytes(M, E));
  L.groups = L.h + up256(3 * P * inter * 2);
  L.parts = L.groups + up256(P * 4);
  L.total = L.parts + (n > 1 ? n * M * hidden * 4 : 0);
  return L;
}

}  // namespace

int64_t mx4_moe_workspace_bytes(int64_t hidden, int64_t inter, int M, int top_k, int E) {
  return moe_layout(hidden, inter, M, top_k, E).total;
}

int launch_mx4_moe(const Mx4MoeArgs& a) {
  const RouteArgs& r = a.route;
  const MoeLayout L = moe_layout(r.K, a.inter, r.M, r.top_k, r.E);
  uint8_t* ws = static_cast<uint8_t*>(r.ws);
  uint16_t* h = reinterpret_cast<uint16_t*>(ws + L.h);
  int32_t* groups = reinterpret_cast<int32_t*>(ws + L.groups);
  float* parts = reinterpret_cast<float*>(ws + L.parts);
  int err = chooses_itself(a) ? launch_logits(r) : launch_route(r);
  if (err) return err;
  err = r.xtype == KQ_F32   ? gate_up_x<T_F32>(a, h, groups)
        : r.xtype == KQ_F16 ? gate_up_x<T_F16>(a, h, groups)
                            : gate_up_x<T_BF16>(a, h, groups);
  if (err) return err;
  return r.M == 1 ? down_cfg<4, 1>(a, h, groups, parts, 1)
                  : down_cfg<2, DOWN_SLOTS>(a, h, groups, parts, down_parts(r.K, r.M * r.top_k));
}

}  // namespace kq
