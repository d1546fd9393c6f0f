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
// A workgroup is one such tile; its waves split K and meet in LDS in wave order.
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

constexpr int ROUTE_WAVES = 16;

template <int XT, int WT>
__global__ __launch_bounds__(64 * ROUTE_WAVES) void k_route_logits(const void* __restrict__ x,
                                                                  const uint8_t* __restrict__ W,
                                                                  double* __restrict__ logits, int M, int K, int E) {
  __shared__ v4d red[ROUTE_WAVES][64];
  const int lane = threadIdx.x & 63, wave = wave_id(), r = lane & 15, g = lane >> 4;
  const int e0 = blockIdx.x * 16, m0 = blockIdx.y * 16;
  const uint32_t xrow = (uint32_t)K * TypeSize<XT>::v, wrow = (uint32_t)K * TypeSize<WT>::v;
  const int erows = E - e0 < 16 ? E - e0 : 16, mrows = M - m0 < 16 ? M - m0 : 16;
  const rsrc_t rw = make_rsrc(W + (int64_t)e0 * wrow, (uint32_t)erows * wrow);
  const rsrc_t rx = make_rsrc(static_cast<const uint8_t*>(x) + (int64_t)m0 * xrow, (uint32_t)mrows * xrow);
  const uint32_t wo = r < erows ? (uint32_t)r * wrow : OOB, xo = r < mrows ? (uint32_t)r * xrow : OOB;
  v4d acc = {0., 0., 0., 0.};
  for (int it = wave; it < K / 32; it += ROUTE_WAVES) {
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
    if (e < erows && m < mrows) logits[(int64_t)(m0 + m) * E + e0 + e] = s;
  }
}

// ---- Choice of the top_k largest logits of one token by one wave: the larger
// first, the lower index on ties, NaN below every number. ids and softmax
// weights of the chosen go out in that order; the softmax is over the chosen
// (renorm) or over all experts. Lane l holds experts l, l + 64, ...
template <int NR>
__device__ __forceinline__ void select_experts(const double* __restrict__ l, int E, int top_k, int renorm,
                                               int32_t* __restrict__ ids, float* __restrict__ weights, int* s_ids) {
  const int lane = threadIdx.x & 63;
  const double ninf = -__builtin_inf();
  double v[NR], raw[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int e = lane + 64 * i;
    raw[i] = e < E ? l[e] : ninf;
    v[i] = raw[i] == raw[i] ? raw[i] : ninf;
  }
  uint32_t taken = 0;
  double first = 0.0, sum = 0.0, mine = 0.0;
  int mine_id = 0;
  for (int k = 0; k < top_k; ++k) {
    double best = 0.0, braw = 0.0;
    int bi = INT32_MAX;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int e = lane + 64 * i;
      const bool open = e < E && !((taken >> i) & 1u);
      if (open && (bi == INT32_MAX || v[i] > best)) best = v[i], braw = raw[i], bi = e;
    }
    for (int off = 32; off > 0; off >>= 1) {
      const double ob = __shfl_xor(best, off, 64), orw = __shfl_xor(braw, off, 64);
      const int oi = __shfl_xor(bi, off, 64);
      if (oi != INT32_MAX && (bi == INT32_MAX || ob > best || (ob == best && oi < bi))) best = ob, braw = orw, bi = oi;
    }
    if ((bi & 63) == lane) taken |= 1u << (bi >> 6);
    if (k == 0) first = braw;
    const double p = exp(braw - first);
    sum += p;
    if (lane == k) mine = p, mine_id = bi;
  }
  if (!renorm) {
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < NR; ++i)
      if (lane + 64 * i < E) sum += exp(raw[i] - first);
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
  }
  if (lane < top_k) {
    ids[lane] = mine_id;
    weights[lane] = (float)(mine / sum);
    if (s_ids) s_ids[lane] = mine_id;
  }
}

template <int NR>
__global__ __launch_bounds__(64) void k_route_select(const double* __restrict__ logits, int E, int top_k, int renorm,
                                                     int32_t* __restrict__ ids, float* __restrict__ weights) {
  const int m = blockIdx.x;
  select_experts<NR>(logits + (int64_t)m * E, E, top_k, renorm, ids + m * top_k, weights + m * top_k, nullptr);
}

// What the expert kernels read: the experts in use in ascending order, with
// the slots (token * top_k + rank) routed to each. The order of one expert's
// slots is not fixed; it decides only which matrix column holds a slot.
struct Groups {
  int32_t* n_active;   // [1]
  int32_t* expert;     // [min(E, P)]
  int32_t* start;      // [min(E, P) + 1] into list
  int32_t* list;       // [P]
};

constexpr int MOE_E_MAX = 1024, MOE_P_MAX = 64 * 64;

// The choice for every token of the layer and the grouping, in one workgroup.
template <int NR>
__global__ __launch_bounds__(1024) void k_moe_select(const double* __restrict__ logits, int M, int E, int top_k,
                                                     int renorm, int32_t* __restrict__ ids,
                                                     float* __restrict__ weights, Groups G) {
  __shared__ int s_ids[MOE_P_MAX];
  __shared__ int s_cnt[MOE_E_MAX];
  const int lane = threadIdx.x & 63, wave = wave_id(), P = M * top_k;
  for (int e = threadIdx.x; e < E; e += 1024) s_cnt[e] = 0;
  for (int m = wave; m < M; m += 16)
    select_experts<NR>(logits + (int64_t)m * E, E, top_k, renorm, ids + m * top_k, weights + m * top_k,
                       s_ids + m * top_k);
  __syncthreads();
  for (int p = threadIdx.x; p < P; p += 1024) atomicAdd(&s_cnt[s_ids[p]], 1);
  __syncthreads();
  if (wave == 0) {
    int n = 0, at = 0;   // experts in use and slots before this step's 64 experts
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane;
      const int c = e < E ? s_cnt[e] : 0;
      int incl = c;
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(incl, off, 64);
        if (lane >= off) incl += o;
      }
      const uint64_t used = __ballot(c > 0);
      const int start = at + incl - c;
      if (c > 0) {
        const int a = n + __popcll(used & ((1ull << lane) - 1ull));
        G.expert[a] = e;
        G.start[a] = start;
      }
      if (e < E) s_cnt[e] = start;
      n += __popcll(used);
      at += __shfl(incl, 63, 64);
    }
    if (lane == 0) {
      G.start[n] = at;
      *G.n_active = n;
    }
  }
  __syncthreads();
  for (int p = threadIdx.x; p < P; p += 1024) G.list[atomicAdd(&s_cnt[s_ids[p]], 1)] = p;
}

// ---- Gate and up rows of one expert for the tokens routed to it:
// h[slot][n] = silu(gate_n . x) * (up_n . x), silu(z) = z / (1 + e^-z), kept
// as three bf16 planes whose sum is the fp32 value (no rounding of h), ready
// as operands of the down projection. Grid (inter / 16, min(E, P)); the waves
// split K and meet in LDS in wave order.
constexpr int GU_WAVES = 4;

template <int XT, bool AL>
__global__ __launch_bounds__(64 * GU_WAVES) void k_mx4_gate_up(const uint8_t* __restrict__ gc, const uint8_t* __restrict__ gs,
                                                              const uint8_t* __restrict__ uc, const uint8_t* __restrict__ us,
                                                              const void* __restrict__ x, Groups G,
                                                              uint16_t* __restrict__ h, int hidden, int inter, int M,
                                                              int top_k) {
  __shared__ v4f red[GU_WAVES][2][64];
  constexpr int U = XT == T_F32 ? 1 : 2;
  __shared__ u32x4 xl4[GU_WAVES][x_region_bytes<XT, U>(16) / 16];
  const int a = blockIdx.y;
  if (a >= *G.n_active) return;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int e = G.expert[a], s0 = G.start[a], cnt = G.start[a + 1] - s0;
  const int nblk = hidden / 32, nchunk = (nblk + 3) / 4;
  const int64_t row = (int64_t)e * inter + blockIdx.x * 16;
  rsrc_t rc[2], rs[2];
  mx4_rows(gc, gs, row, 16, nblk, rc[0], rs[0]);
  mx4_rows(uc, us, row, 16, nblk, rc[1], rs[1]);
  const uint32_t xrow = (uint32_t)hidden * TypeSize<XT>::v;
  const rsrc_t rx = make_rsrc(x, (uint32_t)M * xrow);
  const int c0 = nchunk * wave / GU_WAVES, c1 = nchunk * (wave + 1) / GU_WAVES;
  const int64_t plane = (int64_t)M * top_k * inter;
  for (int t0 = 0; t0 < cnt; t0 += 16) {
    if (t0 > 0) __syncthreads();   // the previous pass has read red
    const int t = t0 + (lane & 15), rows = min(16, cnt - t0);
    const uint32_t xoff = t < cnt ? (uint32_t)(G.list[s0 + t] / top_k) * xrow : 0u;   // of column lane & 15
    v4f acc[2][1] = {{v4f{0.f, 0.f, 0.f, 0.f}}, {v4f{0.f, 0.f, 0.f, 0.f}}};
    mx4_tile<XT, 1, 2, U, AL>(rc, rs, rx, reinterpret_cast<uint8_t*>(xl4[wave]), rows,
                              [=](int row) { return (uint32_t)__shfl((int)xoff, row, 64); }, nblk, c0, c1, acc);
    red[wave][0][lane] = acc[0][0];
    red[wave][1][lane] = acc[1][0];
    __syncthreads();
    // thread: result element i of lane l
    const int l = threadIdx.x >> 2, i = threadIdx.x & 3;
    float g = red[0][0][l][i], u = red[0][1][l][i];
    for (int w = 1; w < GU_WAVES; ++w) g += red[w][0][l][i], u += red[w][1][l][i];
    const int col = t0 + 4 * (l >> 4) + i;
    if (col < cnt) {
      const float hv = g / (1.0f + expf(-g)) * u;
      const uint32_t b0 = __builtin_bit_cast(uint32_t, hv);
      const float vh = __builtin_bit_cast(float, b0 & 0xffff0000u);
      const float r1 = hv == vh ? 0.0f : hv - vh;
      const uint32_t b1 = __builtin_bit_cast(uint32_t, r1);
      const uint32_t b2 = __builtin_bit_cast(uint32_t, r1 - __builtin_bit_cast(float, b1 & 0xffff0000u));
      uint16_t* o = h + (int64_t)G.list[s0 + col] * inter + blockIdx.x * 16 + (l & 15);
      o[0] = (uint16_t)(b0 >> 16);
      o[plane] = (uint16_t)(b1 >> 16);
      o[2 * plane] = (uint16_t)(b2 >> 16);
    }
  }
}

// ---- Down projection and weighted sum: y[m] = sum_j w[m][j] Down_e h[m][j].
// A workgroup owns 16 rows of y for every token; its waves take the experts in
// use in turn, each into sums of its own in LDS, and the waves' sums are added
// in wave order, so the result does not depend on timing. Five slots at a
// time: the 16 operand columns are their three pieces of h (15 in use).
constexpr int DOWN_WAVES = 8, DOWN_SLOTS = 5;

template <bool AL>
__global__ __launch_bounds__(64 * DOWN_WAVES) void k_mx4_down(const uint8_t* __restrict__ dc, const uint8_t* __restrict__ ds,
                                                             const uint16_t* __restrict__ h, Groups G,
                                                             const float* __restrict__ weights, float* __restrict__ y,
                                                             int hidden, int inter, int M, int top_k) {
  extern __shared__ float lds_f[];   // [waves][M][16] sums, then [waves][16][16] scratch
  constexpr int U = 2;
  __shared__ u32x4 xl4[DOWN_WAVES][x_region_bytes<T_BF16, U>(3 * DOWN_SLOTS) / 16];
  const int lane = threadIdx.x & 63, wave = wave_id();
  float* ys = lds_f + wave * M * 16;
  float* scratch = lds_f + DOWN_WAVES * M * 16 + wave * 256;
  for (int i = lane; i < M * 16; i += 64) ys[i] = 0.0f;
  const int n_active = *G.n_active, P = M * top_k;
  const int nblk = inter / 32, nchunk = (nblk + 3) / 4;
  const uint32_t hrow = (uint32_t)inter * 2u;
  const rsrc_t rh = make_rsrc(h, 3u * (uint32_t)P * hrow);
  const int r = lane & 15;
  for (int a = wave; a < n_active; a += DOWN_WAVES) {
    const int e = __builtin_amdgcn_readfirstlane(G.expert[a]), s0 = __builtin_amdgcn_readfirstlane(G.start[a]);
    const int cnt = __builtin_amdgcn_readfirstlane(G.start[a + 1]) - s0;
    rsrc_t rc[1], rs[1];
    mx4_rows(dc, ds, (int64_t)e * hidden + blockIdx.x * 16, 16, nblk, rc[0], rs[0]);
    for (int t0 = 0; t0 < cnt; t0 += DOWN_SLOTS) {
      // column piece * n + m: that piece of h of slot m of this group
      const int n = min(DOWN_SLOTS, cnt - t0), piece = r / n, m = r - piece * n;
      const uint32_t xoff = piece < 3 ? (uint32_t)(piece * P + G.list[s0 + t0 + m]) * hrow : 0u;
      v4f acc[1][1] = {{v4f{0.f, 0.f, 0.f, 0.f}}};
      mx4_tile<T_BF16, 1, 1, U, AL>(rc, rs, rh, reinterpret_cast<uint8_t*>(xl4[wave]), 3 * n,
                                    [=](int row) { return (uint32_t)__shfl((int)xoff, row, 64); }, nblk, 0, nchunk, acc);
#pragma unroll
      for (int i = 0; i < 4; ++i) scratch[(4 * (lane >> 4) + i) * 16 + r] = acc[0][0][i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      for (int i = lane; i < n * 16; i += 64) {
        const int slot = G.list[s0 + t0 + (i >> 4)];
        const float v = scratch[2 * n * 16 + i] + scratch[n * 16 + i] + scratch[i];
        float* o = ys + (slot / top_k) * 16 + (i & 15);
        *o = __builtin_fmaf(weights[slot], v, *o);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < M * 16; i += 64 * DOWN_WAVES) {
    float s = lds_f[i];
    for (int w = 1; w < DOWN_WAVES; ++w) s += lds_f[w * M * 16 + i];
    y[(int64_t)(i >> 4) * hidden + blockIdx.x * 16 + (i & 15)] = s;
  }
}

}  // namespace kqd

namespace kq {

using namespace kqd;

namespace {

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

template <int XT>
int logits_x(const RouteArgs& a, double* logits) {
  const dim3 grid((unsigned)((a.E + 15) / 16), (unsigned)((a.M + 15) / 16)), block(64 * ROUTE_WAVES);
  const uint8_t* W = static_cast<const uint8_t*>(a.W);
#define KQ_LAUNCH(WT) hipLaunchKernelGGL((k_route_logits<XT, WT>), grid, block, 0, a.stream, a.x, W, logits, a.M, (int)a.K, a.E)
  if (a.wtype == KQ_F32) KQ_LAUNCH(T_F32);
  else if (a.wtype == KQ_F16) KQ_LAUNCH(T_F16);
  else KQ_LAUNCH(T_BF16);
#undef KQ_LAUNCH
  dispatch_log("k_route_logits", -1, a.E, a.K, a.M, grid.x, grid.y, block.x, 0, "x=%d w=%d", XT, a.wtype);
  return (int)hipGetLastError();
}

int launch_logits(const RouteArgs& a, double* logits) {
  return a.xtype == KQ_F32 ? logits_x<T_F32>(a, logits) : a.xtype == KQ_F16 ? logits_x<T_F16>(a, logits) : logits_x<T_BF16>(a, logits);
}

// Experts a lane holds: E / 64 rounded up to a power of two.
#define KQ_BY_EXPERTS(E, CALL)       \
  if ((E) <= 64) CALL(1);            \
  else if ((E) <= 128) CALL(2);      \
  else if ((E) <= 256) CALL(4);      \
  else if ((E) <= 512) CALL(8);      \
  else CALL(16);

}  // namespace

int64_t route_workspace_bytes(int M, int E) { return (int64_t)M * E * 8; }

int launch_route(const RouteArgs& a) {
  double* logits = static_cast<double*>(a.ws);
  const int err = launch_logits(a, logits);
  if (err) return err;
  dispatch_log("k_route_select", -1, a.E, a.K, a.M, (unsigned)a.M, 1, 64, 0, "top_k=%d", a.top_k);
#define KQ_LAUNCH(NR) \
  hipLaunchKernelGGL(k_route_select<NR>, dim3((unsigned)a.M), dim3(64), 0, a.stream, logits, a.E, a.top_k, a.renorm, a.ids, a.weights)
  KQ_BY_EXPERTS(a.E, KQ_LAUNCH)
#undef KQ_LAUNCH
  return (int)hipGetLastError();
}

namespace {

struct MoeLayout {
  int64_t h, n_active, expert, start, list, total;   // byte offsets; the logits come first
};
MoeLayout moe_layout(int64_t inter, int M, int top_k, int E) {
  const int64_t P = (int64_t)M * top_k, A = P < E ? P : E;
  MoeLayout L;
  L.h = up256(route_workspace_bytes(M, E));
  L.n_active = L.h + up256(3 * P * inter * 2);
  L.expert = L.n_active + 256;
  L.start = L.expert + up256(4 * A);
  L.list = L.start + up256(4 * (A + 1));
  L.total = L.list + up256(4 * P);
  return L;
}

template <int XT>
int gate_up_x(const Mx4MoeArgs& a, Groups G, uint16_t* h, dim3 grid) {
  const RouteArgs& r = a.route;
#define KQ_LAUNCH(AL)                                                                                               \
  hipLaunchKernelGGL((k_mx4_gate_up<XT, AL>), grid, dim3(64 * GU_WAVES), 0, r.stream, a.codes[0], a.scales[0],      \
                     a.codes[1], a.scales[1], r.x, G, h, (int)r.K, (int)a.inter, r.M, r.top_k)
  if (r.K % 128 == 0) KQ_LAUNCH(true);
  else KQ_LAUNCH(false);
#undef KQ_LAUNCH
  return (int)hipGetLastError();
}

}  // namespace

int64_t mx4_moe_workspace_bytes(int64_t hidden, int64_t inter, int M, int top_k, int E) {
  (void)hidden;
  return moe_layout(inter, M, top_k, E).total;
}

int launch_mx4_moe(const Mx4MoeArgs& a) {
  const RouteArgs& r = a.route;
  const MoeLayout L = moe_layout(a.inter, r.M, r.top_k, r.E);
  uint8_t* ws = static_cast<uint8_t*>(r.ws);
  double* logits = reinterpret_cast<double*>(ws);
  uint16_t* h = reinterpret_cast<uint16_t*>(ws + L.h);
  Groups G{reinterpret_cast<int32_t*>(ws + L.n_active), reinterpret_cast<int32_t*>(ws + L.expert),
           reinterpret_cast<int32_t*>(ws + L.start), reinterpret_cast<int32_t*>(ws + L.list)};
  int err = launch_logits(r, logits);
  if (err) return err;
  dispatch_log("k_moe_select", -1, r.E, r.K, r.M, 1, 1, 1024, 0, "top_k=%d", r.top_k);
#define KQ_LAUNCH(NR) \
  hipLaunchKernelGGL(k_moe_select<NR>, dim3(1), dim3(1024), 0, r.stream, logits, r.M, r.E, r.top_k, r.renorm, r.ids, r.weights, G)
  KQ_BY_EXPERTS(r.E, KQ_LAUNCH)
#undef KQ_LAUNCH
  if ((err = (int)hipGetLastError())) return err;
  const int P = r.M * r.top_k, A = P < r.E ? P : r.E;
  const dim3 gu((unsigned)(a.inter / 16), (unsigned)A);
  dispatch_log("k_mx4_gate_up", -1, a.inter, r.K, r.M, gu.x, gu.y, 64 * GU_WAVES, 0, "type=%d", r.xtype);
  err = r.xtype == KQ_F32 ? gate_up_x<T_F32>(a, G, h, gu) : r.xtype == KQ_F16 ? gate_up_x<T_F16>(a, G, h, gu) : gate_up_x<T_BF16>(a, G, h, gu);
  if (err) return err;
  const unsigned gd = (unsigned)(r.K / 16);
  const size_t lds = (size_t)DOWN_WAVES * (r.M * 16 + 256) * 4;
  dispatch_log("k_mx4_down", -1, r.K, a.inter, r.M, gd, 1, 64 * DOWN_WAVES, lds, "top_k=%d", r.top_k);
#define KQ_LAUNCH(AL)                                                                                          \
  hipLaunchKernelGGL(k_mx4_down<AL>, dim3(gd), dim3(64 * DOWN_WAVES), lds, r.stream, a.codes[2], a.scales[2],  \
                     h, G, r.weights, a.y, (int)r.K, (int)a.inter, r.M, r.top_k)
  if (a.inter % 128 == 0) KQ_LAUNCH(true);
  else KQ_LAUNCH(false);
#undef KQ_LAUNCH
  return (int)hipGetLastError();
}

}  // namespace kq
