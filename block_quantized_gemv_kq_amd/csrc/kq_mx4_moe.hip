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

constexpr int ROUTE_WAVES = 16, ROUTE_SPLITS = 8;

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
// compared as integers that order like them; 0 is below every logit.
__device__ __forceinline__ uint64_t logit_key(double v) {
  if (!(v == v)) v = -__builtin_inf();
  if (v == 0.0) v = 0.0;   // -0 and +0 are equal
  const int64_t b = __builtin_bit_cast(int64_t, v);
  return (uint64_t)b ^ ((uint64_t)(b >> 63) | 0x8000000000000000ull);
}

__global__ __launch_bounds__(1024) void k_route_select(const double* __restrict__ part, int splits, int M, int E,
                                                       int top_k, int renorm, int32_t* __restrict__ ids,
                                                       float* __restrict__ weights) {
  __shared__ uint64_t s_key[1024];
  __shared__ double s_raw[1024];
  __shared__ int s_id[1024];
  __shared__ double s_best[64], s_sum[16];
  const int m = blockIdx.x, e = threadIdx.x, lane = threadIdx.x & 63, wave = wave_id(), waves = blockDim.x >> 6;
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
  int rank = 0;
#pragma unroll 8
  for (int j = 0; j < 64; ++j) {
    const uint64_t kj = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)klo, j) |
                        (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)khi, j) << 32;
    rank += kj > key || (kj == key && j < lane);
  }
  if (rank < top_k) {
    const int at = wave * top_k + rank;
    s_key[at] = key;
    s_raw[at] = raw;
    s_id[at] = e;
  }
  __syncthreads();
  const int C = waves * top_k;
  if (threadIdx.x < (unsigned)C) {
    const uint64_t mine = s_key[threadIdx.x];
    int at = (int)threadIdx.x;
    if (waves > 1) {
      at = 0;
      for (int j = 0; j < C; ++j) {
        const uint64_t kj = s_key[j];
        at += kj > mine || (kj == mine && j < (int)threadIdx.x);
      }
    }
    if (at < top_k) {
      s_best[at] = s_raw[threadIdx.x];
      ids[m * top_k + at] = s_id[threadIdx.x];
    }
  }
  __syncthreads();
  const double first = s_best[0];
  if (!renorm) {
    double p = e < E ? exp(raw - first) : 0.0;
    for (int off = 32; off > 0; off >>= 1) p += __shfl_xor(p, off, 64);
    if (lane == 0) s_sum[wave] = p;
    __syncthreads();
  }
  if (wave > 0) return;
  const double mine = lane < top_k ? exp(s_best[lane] - first) : 0.0;
  double sum = 0.0;
  if (renorm) {
    sum = mine;
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
  } else {
    for (int w = 0; w < waves; ++w) sum += s_sum[w];
  }
  if (lane < top_k) weights[m * top_k + lane] = (float)(mine / sum);
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
// as operands of the down projection. Grid (inter / 16, min(E, P)): row y is
// expert y, or, with fewer slots than experts, the expert of slot y unless an
// earlier slot has it. The waves split K and meet in LDS in wave order.
// Dynamic LDS: ids and list, P uint16 each.
constexpr int GU_WAVES = 4;

template <int XT, bool AL>
__global__ __launch_bounds__(64 * GU_WAVES) void k_mx4_gate_up(const uint8_t* __restrict__ gc, const uint8_t* __restrict__ gs,
                                                              const uint8_t* __restrict__ uc, const uint8_t* __restrict__ us,
                                                              const void* __restrict__ x, const int32_t* __restrict__ ids,
                                                              uint16_t* __restrict__ h, int hidden, int inter, int M,
                                                              int top_k, int E) {
  constexpr int US = XT == T_F32 ? 2 : 4, UL = US / 2;   // chunks in flight with up to 8 and up to 16 columns
  constexpr int REGION = x_region_bytes<XT, US>(8);
  static_assert(REGION == x_region_bytes<XT, UL>(16), "one region for both");
  extern __shared__ uint16_t s_ids[];
  __shared__ v4f red[GU_WAVES][2][64];
  __shared__ u32x4 xl4[GU_WAVES][REGION / 16];
  const int P = M * top_k, y = blockIdx.y;
  uint16_t* list = s_ids + P;
  const int lane = threadIdx.x & 63, wave = wave_id();
  for (int p = threadIdx.x; p < P; p += 64 * GU_WAVES) s_ids[p] = (uint16_t)ids[p];
  __syncthreads();
  const int e = P <= E ? __builtin_amdgcn_readfirstlane(s_ids[y]) : y;
  if (P <= E && earlier_slot(s_ids, y, e)) return;
  const int cnt = gather_slots(s_ids, P, e, list);   // every wave writes the same list
  if (cnt == 0) return;
  const int nblk = hidden / 32, nchunk = (nblk + 3) / 4;
  const int64_t row = (int64_t)e * inter + blockIdx.x * 16;
  rsrc_t rc[2], rs[2];
  mx4_rows(gc, gs, row, 16, nblk, rc[0], rs[0]);
  mx4_rows(uc, us, row, 16, nblk, rc[1], rs[1]);
  const uint32_t xrow = (uint32_t)hidden * TypeSize<XT>::v;
  const rsrc_t rx = make_rsrc(x, (uint32_t)M * xrow);
  const int c0 = nchunk * wave / GU_WAVES, c1 = nchunk * (wave + 1) / GU_WAVES;
  const int64_t plane = (int64_t)P * inter;
  uint8_t* xl = reinterpret_cast<uint8_t*>(xl4[wave]);
  for (int t0 = 0; t0 < cnt; t0 += 16) {
    if (t0 > 0) __syncthreads();   // the previous pass has read red
    const int t = t0 + (lane & 15), rows = min(16, cnt - t0);
    const uint32_t xoff = t < cnt ? (uint32_t)(list[t] / top_k) * xrow : 0u;   // of column lane & 15
    const auto off = [=](int c) { return (uint32_t)__shfl((int)xoff, c, 64); };
    v4f acc[2][1] = {{v4f{0.f, 0.f, 0.f, 0.f}}, {v4f{0.f, 0.f, 0.f, 0.f}}};
    if (rows <= 8) mx4_tile<XT, 1, 2, US, AL>(rc, rs, rx, xl, rows, off, nblk, c0, c1, acc);
    else mx4_tile<XT, 1, 2, UL, AL>(rc, rs, rx, xl, rows, off, nblk, c0, c1, acc);
    red[wave][0][lane] = acc[0][0];
    red[wave][1][lane] = acc[1][0];
    __syncthreads();
    // thread: result element i of lane l
    const int l = threadIdx.x >> 2, i = threadIdx.x & 3;
    float g = red[0][0][l][i], u = red[0][1][l][i];
    for (int w = 1; w < GU_WAVES; ++w) g += red[w][0][l][i], u += red[w][1][l][i];
    const int col = t0 + 4 * (l >> 4) + i;
    if (col < cnt) {
      uint16_t* o = h + (int64_t)list[col] * inter + blockIdx.x * 16 + (l & 15);
      split3_one(g / (1.0f + expf(-g)) * u, o[0], o[plane], o[2 * plane]);
    }
  }
}

// ---- Down projection and weighted sum: y[m] = sum_j w[m][j] Down_e h[m][j].
// A workgroup owns 16 rows of y for every token; its waves take the experts in
// use in turn (wave w those first named by slots w, w + waves, ...), each into
// sums of its own in LDS, and the waves' sums are added in wave order, so the
// result does not depend on timing. Four slots at a time: the operand columns
// are their three pieces of h (12 of 16).
// Dynamic LDS: per wave a region, then per wave M x 16 sums, then the route
// weights (P fp32), ids (P uint16) and a list of slots per wave (P uint16).
constexpr int DOWN_SLOTS = 4, DOWN_REGION = x_region_bytes<T_BF16, 2>(3 * DOWN_SLOTS);
static_assert(DOWN_REGION >= x_region_bytes<T_BF16, 4>(6) && DOWN_REGION >= 1024, "the region serves both widths and the results");

template <bool AL>
__global__ __launch_bounds__(1024) void k_mx4_down(const uint8_t* __restrict__ dc, const uint8_t* __restrict__ ds,
                                                  const uint16_t* __restrict__ h, const int32_t* __restrict__ ids,
                                                  const float* __restrict__ weights, float* __restrict__ y, int hidden,
                                                  int inter, int M, int top_k, int waves) {
  extern __shared__ u32x4 lds4[];
  const int lane = threadIdx.x & 63, wave = wave_id(), P = M * top_k;
  uint8_t* xl = reinterpret_cast<uint8_t*>(lds4) + wave * DOWN_REGION;
  float* sums = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(lds4) + waves * DOWN_REGION);
  float* ys = sums + wave * M * 16;
  float* s_w = sums + waves * M * 16;
  uint16_t* s_ids = reinterpret_cast<uint16_t*>(s_w + P);
  uint16_t* list = s_ids + P + wave * P;
  for (int p = threadIdx.x; p < P; p += 64 * waves) {
    s_ids[p] = (uint16_t)ids[p];
    s_w[p] = weights[p];
  }
  for (int i = lane; i < M * 16; i += 64) ys[i] = 0.0f;
  __syncthreads();
  const int nblk = inter / 32, nchunk = (nblk + 3) / 4;
  const uint32_t hrow = (uint32_t)inter * 2u;
  const rsrc_t rh = make_rsrc(h, 3u * (uint32_t)P * hrow);
  const int r = lane & 15;
  for (int p = wave; p < P; p += waves) {
    const int e = __builtin_amdgcn_readfirstlane(s_ids[p]);
    if (earlier_slot(s_ids, p, e)) continue;
    const int cnt = gather_slots(s_ids, P, e, list);
    rsrc_t rc[1], rs[1];
    mx4_rows(dc, ds, (int64_t)e * hidden + blockIdx.x * 16, 16, nblk, rc[0], rs[0]);
    for (int t0 = 0; t0 < cnt; t0 += DOWN_SLOTS) {
      // column piece * n + m: that piece of h of slot m of this group
      const int n = min(DOWN_SLOTS, cnt - t0), piece = r / n, m = r - piece * n;
      const uint32_t xoff = piece < 3 ? (uint32_t)(piece * P + list[t0 + m]) * hrow : 0u;
      const auto off = [=](int row) { return (uint32_t)__shfl((int)xoff, row, 64); };
      v4f acc[1][1] = {{v4f{0.f, 0.f, 0.f, 0.f}}};
      if (n <= 2) mx4_tile<T_BF16, 1, 1, 4, AL>(rc, rs, rh, xl, 3 * n, off, nblk, 0, nchunk, acc);
      else mx4_tile<T_BF16, 1, 1, 2, AL>(rc, rs, rh, xl, 3 * n, off, nblk, 0, nchunk, acc);
      // the results take the region's place, 16 rows (columns of h) of 16
      float* out = reinterpret_cast<float*>(xl);
#pragma unroll
      for (int i = 0; i < 4; ++i) out[(4 * (lane >> 4) + i) * 16 + r] = acc[0][0][i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (lane < n * 16) {
        const int slot = list[t0 + (lane >> 4)];
        const float v = out[2 * n * 16 + lane] + out[n * 16 + lane] + out[lane];
        float* o = ys + (slot / top_k) * 16 + r;
        *o = __builtin_fmaf(s_w[slot], v, *o);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read before the next copies land there
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < M * 16; i += 64 * waves) {
    float s = sums[i];
    for (int w = 1; w < waves; ++w) s += sums[w * M * 16 + i];
    y[(int64_t)(i >> 4) * hidden + blockIdx.x * 16 + (i & 15)] = s;
  }
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

int launch_route(const RouteArgs& a) {
  double* part = static_cast<double*>(a.ws);
  const int err = a.xtype == KQ_F32 ? logits_x<T_F32>(a, part) : a.xtype == KQ_F16 ? logits_x<T_F16>(a, part) : logits_x<T_BF16>(a, part);
  if (err) return err;
  int threads = 64;   // a thread per expert, whole waves in a power of two
  while (threads < a.E) threads *= 2;
  dispatch_log("k_route_select", -1, a.E, a.K, a.M, (unsigned)a.M, 1, (unsigned)threads, 0, "top_k=%d", a.top_k);
  hipLaunchKernelGGL(k_route_select, dim3((unsigned)a.M), dim3((unsigned)threads), 0, a.stream, part, route_splits(a.K),
                     a.M, a.E, a.top_k, a.renorm, a.ids, a.weights);
  return (int)hipGetLastError();
}

namespace {

constexpr int MOE_LDS_BYTES = 160 * 1024;   // of a compute unit

template <int XT>
int gate_up_x(const Mx4MoeArgs& a, uint16_t* h) {
  const RouteArgs& r = a.route;
  const int P = r.M * r.top_k;
  const dim3 grid((unsigned)(a.inter / 16), (unsigned)(P < r.E ? P : r.E));
  const size_t lds = (size_t)P * 4;
  dispatch_log("k_mx4_gate_up", -1, a.inter, r.K, r.M, grid.x, grid.y, 64 * GU_WAVES, lds, "type=%d", XT);
#define KQ_LAUNCH(AL)                                                                                            \
  hipLaunchKernelGGL((k_mx4_gate_up<XT, AL>), grid, dim3(64 * GU_WAVES), lds, r.stream, a.codes[0], a.scales[0], \
                     a.codes[1], a.scales[1], r.x, r.ids, h, (int)r.K, (int)a.inter, r.M, r.top_k, r.E)
  if (r.K % 128 == 0) KQ_LAUNCH(true);
  else KQ_LAUNCH(false);
#undef KQ_LAUNCH
  return (int)hipGetLastError();
}

}  // namespace

// The logits' parts, then the three planes of h.
int64_t mx4_moe_workspace_bytes(int64_t hidden, int64_t inter, int M, int top_k, int E) {
  (void)hidden;
  return up256(route_workspace_bytes(M, E)) + 3 * (int64_t)M * top_k * inter * 2;
}

int launch_mx4_moe(const Mx4MoeArgs& a) {
  const RouteArgs& r = a.route;
  uint16_t* h = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(r.ws) + up256(route_workspace_bytes(r.M, r.E)));
  int err = launch_route(r);
  if (err) return err;
  err = r.xtype == KQ_F32 ? gate_up_x<T_F32>(a, h) : r.xtype == KQ_F16 ? gate_up_x<T_F16>(a, h) : gate_up_x<T_BF16>(a, h);
  if (err) return err;
  const int P = r.M * r.top_k;
  // a wave per slot up to what LDS holds
  const int shared = P * 6, per_wave = DOWN_REGION + r.M * 64 + P * 2;
  int waves = (MOE_LDS_BYTES - shared) / per_wave;
  waves = waves > 16 ? 16 : waves;
  waves = waves > P ? P : waves;
  const unsigned grid = (unsigned)(r.K / 16);
  const size_t lds = (size_t)(shared + waves * per_wave);
  dispatch_log("k_mx4_down", -1, r.K, a.inter, r.M, grid, 1, (unsigned)(64 * waves), lds, "top_k=%d", r.top_k);
#define KQ_LAUNCH(AL)                                                                                            \
  hipLaunchKernelGGL(k_mx4_down<AL>, dim3(grid), dim3((unsigned)(64 * waves)), lds, r.stream, a.codes[2],        \
                     a.scales[2], h, r.ids, r.weights, a.y, (int)r.K, (int)a.inter, r.M, r.top_k, waves)
  if (a.inter % 128 == 0) KQ_LAUNCH(true);
  else KQ_LAUNCH(false);
#undef KQ_LAUNCH
  return (int)hipGetLastError();
}

}  // namespace kq
