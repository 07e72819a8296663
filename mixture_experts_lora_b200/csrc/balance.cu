// The router's balance loss per sequence, the per-expert counts, and the gradient into
// the logits.
//
// With p = softmax(logits[t]), counts[s,e] the pairs of sequence s routed to expert e and
// n_s its valid rows:
//   loss[s]      = E / (k n_s^2) sum_e counts[s,e] sum_t p[t,e]
//   dlogits[t,e] = g_s p[t,e] (counts[s,e] - sum_j p[t,j] counts[s,j]),
//   g_s          = dloss[s] E / (k n_s^2)
//
// Both directions read every logit once and are bound by HBM (the backward writes as much).
// Rows are cut into windows; forward a block takes the rows of one sequence in one window (131072 x
// 128 in 64 sequences: 18 us; 3 us more with a block per window, where one with rows of two
// sequences took them one after the other), backward a window.  A row is spread over L lanes (a
// power of two, 32 from 128 experts on: fewer lanes leave room for several rows in a warp), each
// holding NQ groups of V experts, V = 4 where rows are 16-byte aligned.  A warp loads U rows per
// lane group before it works on the first, so that enough bytes are on their way.
// Forward: the lanes sum their experts' probabilities over the rows, the block's warps are
// summed in a fixed order through shared memory, and each (window, sequence) pair writes one
// partial row; a second launch sums a sequence's partials in a fixed order.  A batch of one
// window needs no second launch.  Everything is fp32 (counts: integers).
#include <climits>

#include "common.cuh"
#include "internal.h"
#include "sequences.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct BalanceArgs {
  const float* logits;
  const int32_t* ids;
  const int32_t* off;      // nullptr: one sequence [0, T)
  const uint8_t* mask;     // nullptr: every row counts
  int64_t T;
  int E, k, S;
  int rows;                // rows per window
  // forward: partial rows of the (window, sequence) slots
  // partials, or (one window) the outputs themselves
  float* psum;             // [slots][E]
  int32_t* pcnt;           // [slots][E]
  int32_t* pn;             // [slots]
  float* loss;             // outputs; balance_partial_kernel writes them itself if loss is set
  int32_t* out_counts;
  int32_t* out_n;
  int lanes;               // lanes per row
  int sum_ranks;           // blocks per sequence of balance_sum_kernel
  int* err;
  // backward
  const int32_t* counts;
  const int32_t* n_tokens;
  const float* dloss;
  float* dlogits;
  int accumulate;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// How a row lies in a warp: V consecutive experts at a time, NQ times, over LANES lanes (0: as
// many as the launch says).
template <int V_, int NQ_, int LANES_>
struct RowCfg {
  static constexpr int V = V_, NQ = NQ_, N = V * NQ, LANES = LANES_;
  static constexpr bool FULL = LANES == 32;
  static constexpr int U = N <= 4 ? 4 : N <= 8 ? 2 : 1;      // rows loaded at once
};

// The lanes of a row.
struct Lanes {
  int L, sub, group, groups;     // lanes per row, lane within its row, row within the warp, rows
  __device__ __forceinline__ Lanes(int fixed, int l) : L(fixed != 0 ? fixed : l) {
    sub = lane_id() & (L - 1);
    groups = 32 / L;
    group = lane_id() / L;
  }
};
template <class C>
__device__ __forceinline__ float row_max(float v, const Lanes& ln) {
  if constexpr (C::FULL) {
    float r;                     // (a NaN loses)
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
  } else {
    if constexpr (C::LANES != 0) {
#pragma unroll
      for (int o = C::LANES / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    } else {
      for (int o = ln.L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    }
    return v;
  }
}
template <class C>
__device__ __forceinline__ float row_sum(float v, const Lanes& ln) {
  if constexpr (C::LANES != 0) {
#pragma unroll
    for (int o = C::LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  } else {
    for (int o = ln.L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}

// First expert of the lane's group q.
template <class C>
__device__ __forceinline__ int expert_of(const Lanes& ln, int q) { return (q * ln.L + ln.sub) * C::V; }

// The lane's experts of a row (px: the row's first of them), -inf past E and where !live.
template <class C>
__device__ __forceinline__ void load_row(const float* __restrict__ px, int E, const Lanes& ln, bool live,
                                         float (&v)[C::N]) {
#pragma unroll
  for (int q = 0; q < C::NQ; ++q) {
    const bool in = live && expert_of<C>(ln, q) < E;
    if constexpr (C::V == 4) {
      const float4 t = in ? __ldg(reinterpret_cast<const float4*>(px + q * ln.L * 4))
                          : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      v[4 * q] = t.x; v[4 * q + 1] = t.y; v[4 * q + 2] = t.z; v[4 * q + 3] = t.w;
    } else {
      v[q] = in ? __ldg(px + q * ln.L) : -INFINITY;
    }
  }
}

// exp(x - max) in place, 0 for -inf.  2^y to 2 ulp with y = (x - max) log2(e) rounded: a term is
// off by |x - max| u and a few u more, u = 2^-24 (two issue slots in three are taken, and an
// exponential good to the last bit costs four times as many instructions).
template <class C>
__device__ __forceinline__ void row_exp(float (&v)[C::N], const Lanes& ln) {
  float mx = v[0];
#pragma unroll
  for (int i = 1; i < C::N; ++i) mx = fmaxf(mx, v[i]);
  mx = row_max<C>(mx, ln);
  if (mx == -INFINITY) mx = 0.f;          // nothing finite: every term 2^-inf = 0
  const f32x2 nm = pack2(-mx, -mx), l2e = pack2(1.4426950408889634f, 1.4426950408889634f);
#pragma unroll
  for (int i = 0; i < C::N; i += 2) {
    const bool two = i + 1 < C::N;
    const float2 y = unpack2(mul2(add2(pack2(v[i], two ? v[i + 1] : 0.f), nm), l2e));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(v[i]) : "f"(y.x));
    if (two) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(v[i + 1]) : "f"(y.y));
  }
}
template <class C>
__device__ __forceinline__ float lane_sum(const float (&v)[C::N]) {
  float sum = v[0];
#pragma unroll
  for (int i = 1; i < C::N; ++i) sum += v[i];
  return sum;
}
// 1 / (a row's sum of exponentials: at least 1, 0 or not a number), 0 for 0
__device__ __forceinline__ float row_inverse(float sum) { return sum == 0.f ? 0.f : rcp_approx(sum); }

__device__ __forceinline__ float loss_factor(int E, int k, int n) {
  return n > 0 ? (float)E / ((float)k * (float)n) / (float)n : 0.f;
}

// The sum of one float per thread over the block (any multiple of 32 threads), in thread 0.
__device__ __forceinline__ float block_sum(float v, float* s_part) {
  v = warp_sum(v);
  __syncthreads();
  if (lane_id() == 0) s_part[warp_id()] = v;
  __syncthreads();
  float all = 0.f;
  if (threadIdx.x == 0)
    for (int i = 0; i < (int)blockDim.x / 32; ++i) all += s_part[i];
  return all;
}

template <class C>
__global__ void __launch_bounds__(kThreads, C::N <= 8 ? 4 : 2) balance_partial_kernel(const BalanceArgs a) {
  pdl_begin();
  extern __shared__ float s_dyn[];            // [kWarps][E] sums, then E counts
  float* s_sum = s_dyn;
  int* s_cnt = reinterpret_cast<int*>(s_dyn + kWarps * a.E);
  __shared__ int s_n;
  __shared__ float s_part[kWarps];
  const int warp = warp_id(), E = a.E;
  const Lanes ln(C::LANES, a.lanes);
  // the block's slot: rows [r0, r1) of sequence s in window w
  const int slot = (int)blockIdx.x;
  int s = 0;
  int64_t r0 = 0, r1 = a.T;
  if (a.off != nullptr) {
    check_offsets(a.off, a.S, a.T, a.err);
    s = slot;                                  // (one window: the outputs of sequence s, empty or not)
    if (a.loss == nullptr) s = block_count_le(a.S, slot, [&](int i) { return (long long)(a.off[i] / a.rows) + i; }) - 1;
    if (s < 0 || s > slot) return;             // (no sequence; or offsets below 0)
    r0 = a.off[s];
    r1 = a.off[s + 1];
  }
  const int64_t t0 = (int64_t)(slot - s) * a.rows;
  r0 = r0 > t0 ? r0 : t0;
  r1 = r1 < t0 + a.rows ? r1 : t0 + a.rows;
  if (r1 > a.T) r1 = a.T;
  if (r0 >= r1) {
    if (a.loss == nullptr) return;
    r0 = r1 = 0;
  }
  for (int e = threadIdx.x; e < E; e += kThreads) s_cnt[e] = 0;
  if (threadIdx.x == 0) s_n = 0;
  __syncthreads();
  float acc[C::N];
#pragma unroll
  for (int i = 0; i < C::N; ++i) acc[i] = 0.f;
  int n = 0;
  const int per = ln.groups * C::U;          // rows of a warp at a time
  const int rows = (int)(r1 - r0), step = kWarps * per;
  int t = warp * per + ln.group;             // the lane group's first row, from r0
  const float* px = a.logits + (r0 + t) * E + ln.sub * C::V;
  const uint8_t* pmask = a.mask != nullptr ? a.mask + r0 : nullptr;
  // the next rows' logits are on their way while a row's softmax is computed
  float next[C::U][C::N];
  uint32_t next_live = 0;
  const auto fetch = [&]() {
    next_live = 0;
#pragma unroll
    for (int u = 0; u < C::U; ++u) {
      const bool live = t + u * ln.groups < rows && (pmask == nullptr || pmask[t + u * ln.groups] != 0);
      next_live |= (uint32_t)live << u;
      load_row<C>(px + u * ln.groups * E, E, ln, live, next[u]);
    }
    t += step;
    px += (int64_t)step * E;
  };
  // pairs per expert, eight ids on their way at a time, the first of them ahead of the logits: the
  // counting ends while those arrive (131072 x 128: 1.7 us less than with four ids at a time
  // behind the logits)
  constexpr int IDS = 8;
  const int pairs = rows * a.k;
  const int32_t* ids = a.ids + r0 * a.k;
  int id[IDS];
  uint32_t valid = 0;
  const auto load_ids = [&](int first) {
    valid = 0;
#pragma unroll
    for (int q = 0; q < IDS; ++q) {
      if (first + q * kThreads >= pairs) break;                // (the same for the block)
      const int i = first + q * kThreads + threadIdx.x;
      const bool in = i < pairs && (pmask == nullptr || pmask[(uint32_t)i / (uint32_t)a.k] != 0);
      valid |= (uint32_t)in << q;
      if (in) id[q] = __ldg(ids + i);
    }
  };
  load_ids(0);
  fetch();
  for (int first = 0; first < pairs;) {
#pragma unroll
    for (int q = 0; q < IDS; ++q) {
      if (first + q * kThreads >= pairs) break;
      if (((valid >> q) & 1) == 0) continue;
      if ((uint32_t)id[q] < (uint32_t)E) atomicAdd(&s_cnt[id[q]], 1);
      else report_error(a.err, MOE_ERR_DEVICE_INDEX);
    }
    first += IDS * kThreads;
    load_ids(first);
  }
  for (int tw = warp * per; tw < rows; tw += step) {
    float v[C::U][C::N];
#pragma unroll
    for (int u = 0; u < C::U; ++u)
#pragma unroll
      for (int i = 0; i < C::N; ++i) v[u][i] = next[u][i];
    n += __popc(next_live);
    fetch();
#pragma unroll
    for (int u = 0; u < C::U; ++u) {
      row_exp<C>(v[u], ln);
      const float inv = row_inverse(row_sum<C>(lane_sum<C>(v[u]), ln));
#pragma unroll
      for (int i = 0; i < C::N; ++i) acc[i] += v[u][i] * inv;
    }
  }
  // rows of one warp side by side: the lanes of the same experts
  if constexpr (!C::FULL) {
    for (int o = ln.L; o < 32; o <<= 1) {
#pragma unroll
      for (int i = 0; i < C::N; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    }
  }
  if (C::FULL || ln.group == 0) {
#pragma unroll
    for (int q = 0; q < C::NQ; ++q) {
      const int e = expert_of<C>(ln, q);
#pragma unroll
      for (int i = 0; i < C::V; ++i)
        if (e + i < E) s_sum[warp * E + e + i] = acc[q * C::V + i];
    }
  }
  if (ln.sub == 0 && n > 0) atomicAdd(&s_n, n);
  __syncthreads();
  float part = 0.f;
  for (int e = threadIdx.x; e < E; e += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += s_sum[i * E + e];
    const int cnt = s_cnt[e];
    if (a.loss != nullptr) {
      a.out_counts[(int64_t)s * E + e] = cnt;
      part += (float)cnt * v;
    } else {
      a.psum[(int64_t)slot * E + e] = v;
      a.pcnt[(int64_t)slot * E + e] = cnt;
    }
  }
  if (a.loss != nullptr) {
    const float all = block_sum(part, s_part);
    if (threadIdx.x == 0) {
      a.loss[s] = all * loss_factor(E, a.k, s_n);
      a.out_n[s] = s_n;
    }
  } else if (threadIdx.x == 0) {
    a.pn[slot] = s_n;
  }
}

// A cluster per sequence sums its partial rows.  Experts are taken in groups of 128, four a lane;
// the cluster's CTAs share the groups and, where there are more CTAs, each group's windows.  A warp
// sums every so-manyth window, then the CTA's warps and the CTAs are summed, all in a fixed
// order.  Four windows of a warp are on their way at once, so that up to 1024 windows of 128 experts
// need one wait for memory (131072 x 128, 592 windows: 3.8 us less than where each of four CTAs took
// all windows of 32 experts).
constexpr int kSumThreads = 1024, kGroup = 128, kMaxRanks = 8;
template <bool V4>
__global__ void __launch_bounds__(kSumThreads) balance_sum_kernel(const BalanceArgs a) {
  __shared__ __align__(16) float s_sum[32][kGroup];
  __shared__ __align__(16) int s_cnt[32][kGroup];
  __shared__ float r_sum[kMaxRanks][kGroup];     // the other CTAs' parts
  __shared__ int r_cnt[kMaxRanks][kGroup];
  __shared__ float s_part[32], s_loss[kMaxRanks];
  __shared__ int s_n;
  const int warps = (int)blockDim.x / 32, warp = warp_id(), lane = lane_id(), tid = (int)threadIdx.x, E = a.E;
  const int rank = (int)cluster_ctarank(), ranks = a.sum_ranks, s = (int)blockIdx.x / ranks;
  // CTA (re, wr): groups re, re + rE, ... and of their windows the wr-th part; with rW > 1 one group
  const int groups = (E + kGroup - 1) / kGroup;
  int rE = 1;
  while (rE < ranks && rE < groups) rE *= 2;
  const int rW = ranks / rE, re = rank % rE, wr = rank / rE;
  const int n_win = (int)((uint32_t)(a.T + a.rows - 1) / (uint32_t)a.rows);     // (T < 2^31)
  if (tid == 0) s_n = 0;
  if (ranks > 1) cluster_arrive();
  pdl_begin();
  const int64_t r0 = a.off != nullptr ? a.off[s] : 0, r1 = a.off != nullptr ? a.off[s + 1] : a.T;
  // first and last window of the sequence (none if it is empty), within the table whatever
  // the offsets hold
  int64_t w0 = 0, w1 = 0;
  if (a.off == nullptr) {
    w1 = n_win;
  } else if (r0 >= 0 && r1 > r0) {
    w0 = (uint32_t)r0 / (uint32_t)a.rows;
    w1 = (uint32_t)(r1 - 1) / (uint32_t)a.rows + 1;
    if (w1 > n_win) w1 = n_win;
  }
  int n = 0;                                     // (added up below, with the sums on their way)
  if (rank == 0)
    for (int64_t w = w0 + tid; w < w1; w += blockDim.x) n += a.pn[w + s];
  float part = 0.f;
  const auto finish = [&](int e, float v, int c) {
    if (e >= E) return;
    a.out_counts[(int64_t)s * E + e] = c;
    part += (float)c * v;
  };
  bool started = ranks == 1;
  for (int g = re; g < groups; g += rE) {
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    int cnt[4] = {0, 0, 0, 0};
    const int e0 = g * kGroup + (V4 ? 4 * lane : lane);
    const int64_t step = (int64_t)rW * warps;
    for (int64_t w = w0 + wr * warps + warp; w < w1; w += 4 * step) {
      float v[4][4];
      int c[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t at = (w + i * step + s) * E + e0;
        const bool in = w + i * step < w1;
        if constexpr (V4) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          int4 y = make_int4(0, 0, 0, 0);
          if (in && e0 < E) {
            x = *reinterpret_cast<const float4*>(a.psum + at);
            y = *reinterpret_cast<const int4*>(a.pcnt + at);
          }
          v[i][0] = x.x; v[i][1] = x.y; v[i][2] = x.z; v[i][3] = x.w;
          c[i][0] = y.x; c[i][1] = y.y; c[i][2] = y.z; c[i][3] = y.w;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool here = in && e0 + 32 * j < E;
            v[i][j] = here ? a.psum[at + 32 * j] : 0.f;
            c[i][j] = here ? a.pcnt[at + 32 * j] : 0;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sum[j] += v[i][j];
          cnt[j] += c[i][j];
        }
    }
    __syncthreads();                             // the last group's sums are read
    if (n != 0) atomicAdd(&s_n, n);
    n = 0;
    if constexpr (V4) {
      *reinterpret_cast<float4*>(&s_sum[warp][4 * lane]) = make_float4(sum[0], sum[1], sum[2], sum[3]);
      *reinterpret_cast<int4*>(&s_cnt[warp][4 * lane]) = make_int4(cnt[0], cnt[1], cnt[2], cnt[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s_sum[warp][lane + 32 * j] = sum[j];
        s_cnt[warp][lane + 32 * j] = cnt[j];
      }
    }
    __syncthreads();
    if (!started) {                              // (long past: the CTAs of the cluster run)
      cluster_wait();
      started = true;
    }
    if (tid < kGroup) {
      float v = 0.f;
      int c = 0;
#pragma unroll 8
      for (int i = 0; i < warps; ++i) {
        v += s_sum[i][tid];
        c += s_cnt[i][tid];
      }
      if (rW == 1) {
        finish(g * kGroup + tid, v, c);
      } else {                                   // to the group's first CTA
        const uint32_t dv = mapa_smem(smem_u32(&r_sum[wr][tid]), (uint32_t)re);
        const uint32_t dc = mapa_smem(smem_u32(&r_cnt[wr][tid]), (uint32_t)re);
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dv), "f"(v) : "memory");
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dc), "r"(c) : "memory");
      }
    }
  }
  if (!started) cluster_wait();                  // (a CTA without a group)
  if (rW > 1) {
    __syncwarp();
    cluster_sync();
    if (wr == 0 && re < groups && tid < kGroup) {
      float v = 0.f;
      int c = 0;
      for (int i = 0; i < rW; ++i) {
        v += r_sum[i][tid];
        c += r_cnt[i][tid];
      }
      finish(re * kGroup + tid, v, c);
    }
  }
  const float mine = block_sum(part, s_part);
  if (rE > 1) {
    if (tid == 0 && wr == 0) {
      const uint32_t dst = mapa_smem(smem_u32(&s_loss[re]), 0u);
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst), "f"(mine) : "memory");
    }
    __syncwarp();
    cluster_sync();
  }
  if (rank == 0 && tid == 0) {
    float all = mine;
    if (rE > 1) {
      all = 0.f;
      for (int i = 0; i < rE; ++i) all += s_loss[i];
    }
    a.loss[s] = all * loss_factor(E, a.k, s_n);
    a.out_n[s] = s_n;
  }
}

template <class C>
__global__ void __launch_bounds__(kThreads) balance_backward_kernel(const BalanceArgs a) {
  pdl_begin();
  const int warp = warp_id(), E = a.E;
  const Lanes ln(C::LANES, a.lanes);
  const int64_t t0 = (int64_t)blockIdx.x * a.rows;
  const int64_t t1 = t0 + a.rows < a.T ? t0 + a.rows : a.T;
  int s = 0;
  if (a.off != nullptr) {
    check_offsets(a.off, a.S, a.T, a.err);
    s = block_count_le(a.S, t0, [&](int i) { return a.off[i + 1]; });
  }
  // everything from t0 on: rows of the window, and of the lane group's sequence s
  const int rows = (int)(t1 - t0);
  int s_lo = 0, s_hi = a.off != nullptr ? -1 : rows;
  int held = -1;                               // the sequence whose f is held
  float f[C::N];
  const int per = ln.groups * C::U;
  const int64_t skip = (int64_t)kWarps * per * E;
  int t = warp * per + ln.group;
  const int64_t first = (t0 + t) * E + ln.sub * C::V;
  const float* px = a.logits + first;
  float* po = a.dlogits + first;
  const uint8_t* pmask = a.mask != nullptr ? a.mask + t0 : nullptr;
  for (int tw = warp * per; tw < rows; tw += kWarps * per, t += kWarps * per, px += skip, po += skip) {
    float v[C::U][C::N];
    bool live[C::U];
    int seq[C::U];
#pragma unroll
    for (int u = 0; u < C::U; ++u) {
      const int tu = t + u * ln.groups;
      live[u] = tu < rows && (pmask == nullptr || pmask[tu] != 0);
      if (tu < rows && tu >= s_hi) {           // on to the row's sequence
        if (s < a.S && a.off[s + 1] <= t0 + tu) ++s;
        if (s < a.S && a.off[s + 1] <= t0 + tu) {        // (past empty sequences, by halves)
          int lo = s + 1, hi = a.S;
          while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (a.off[mid + 1] <= t0 + tu) lo = mid + 1;
            else hi = mid;
          }
          s = lo;
        }
        s_lo = s < a.S ? (int)(a.off[s] - t0) : rows;
        s_hi = s < a.S ? (int)(a.off[s + 1] - t0) : rows;
      }
      live[u] = live[u] && tu >= s_lo;
      seq[u] = s;
      load_row<C>(px + u * ln.groups * E, E, ln, live[u], v[u]);
      // what is added to is on its way to L2 meanwhile (131072 x 128 added: 36 us, 5 us
      // more without; asking for the next rows too took 43 to 46 us)
      if (a.accumulate && live[u]) {
#pragma unroll
        for (int q = 0; q < C::NQ; ++q)
          if (expert_of<C>(ln, q) < E)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(po + u * ln.groups * E + q * ln.L * C::V));
      }
    }
#pragma unroll
    for (int u = 0; u < C::U; ++u) {
      if (live[u] && seq[u] != held) {
        held = seq[u];
        const int n = a.n_tokens[held];
        const float g = a.dloss[held] * loss_factor(E, a.k, n);
        // counts less the least of them: sum_j p_j = 1 lets any constant be taken off the counts, and
        // small differences keep the digits that counts - sum_j p_j counts_j would cancel.  (Less
        // their mean, experts without any pair would cancel against it in rows that one expert has:
        // 2 experts, p = 1.4e-4: 7e-5 of the gradient.)
        int c[C::N], least = INT_MAX;
#pragma unroll
        for (int q = 0; q < C::NQ; ++q) {
          const int e = expert_of<C>(ln, q);
#pragma unroll
          for (int i = 0; i < C::V; ++i) {
            c[q * C::V + i] = e + i < E ? a.counts[(int64_t)held * E + e + i] : INT_MAX;
            least = min(least, c[q * C::V + i]);
          }
        }
        const uint32_t row = ln.L == 32 ? 0xffffffffu : ((1u << ln.L) - 1) << (ln.group * ln.L);
        for (int o = ln.L / 2; o > 0; o >>= 1) least = min(least, __shfl_xor_sync(row, least, o));
#pragma unroll
        for (int i = 0; i < C::N; ++i) f[i] = c[i] != INT_MAX ? (float)(c[i] - least) * g : 0.f;
      }
      row_exp<C>(v[u], ln);
      float dot = 0.f;
      if (live[u]) {
#pragma unroll
        for (int i = 0; i < C::N; ++i) dot += v[u][i] * f[i];
      }
      const float inv = row_inverse(row_sum<C>(lane_sum<C>(v[u]), ln));
      dot = row_sum<C>(dot, ln) * inv;
      if (t + u * ln.groups >= rows || (!live[u] && a.accumulate)) continue;
      float* out = po + u * ln.groups * E;
#pragma unroll
      for (int q = 0; q < C::NQ; ++q) {
        if (expert_of<C>(ln, q) >= E) continue;
        float d[C::V];
#pragma unroll
        for (int i = 0; i < C::V; ++i)
          d[i] = live[u] ? v[u][q * C::V + i] * inv * (f[q * C::V + i] - dot) : 0.f;
        if constexpr (C::V == 4) {
          float4* p = reinterpret_cast<float4*>(out + q * ln.L * 4);
          float4 o = make_float4(d[0], d[1], d[2], d[3]);
          if (a.accumulate) {
            const float4 b = *p;
            o = make_float4(b.x + o.x, b.y + o.y, b.z + o.z, b.w + o.w);
          }
          *p = o;
        } else {
          float* p = out + q * ln.L;
          *p = a.accumulate ? *p + d[0] : d[0];
        }
      }
    }
  }
}

struct Forward {
  template <class C>
  static cudaError_t launch(const BalanceArgs& a, int64_t slots, cudaStream_t st) {
    ProfScope ps(K_BALANCE, st);
    return launch_pdl(balance_partial_kernel<C>, dim3((unsigned)slots), dim3(kThreads),
                      (size_t)(kWarps + 1) * a.E * 4, st, 1, a);
  }
};
struct Backward {
  template <class C>
  static cudaError_t launch(const BalanceArgs& a, int64_t n_win, cudaStream_t st) {
    ProfScope ps(K_BALANCE_BWD, st);
    return launch_pdl(balance_backward_kernel<C>, dim3((unsigned)n_win), dim3(kThreads), 0, st, 1, a);
  }
};

// Four experts at a time where every row of logits (and of the gradient) is 16-byte aligned.
template <class K>
cudaError_t launch_rows(BalanceArgs& a, int64_t blocks, cudaStream_t s) {
  const bool v4 = a.E % 4 == 0 && aligned16(a.logits) && (a.dlogits == nullptr || aligned16(a.dlogits));
  const int groups = v4 ? a.E / 4 : a.E;
  a.lanes = 1;
  while (a.lanes < 32 && a.lanes < groups) a.lanes *= 2;
  const int nq = (groups + a.lanes - 1) / a.lanes;
  if (v4) {
    if (a.lanes == 16) return K::template launch<RowCfg<4, 1, 16>>(a, blocks, s);
    if (a.lanes == 8) return K::template launch<RowCfg<4, 1, 8>>(a, blocks, s);
    if (a.lanes < 32) return K::template launch<RowCfg<4, 1, 0>>(a, blocks, s);
    if (nq <= 1) return K::template launch<RowCfg<4, 1, 32>>(a, blocks, s);
    if (nq <= 2) return K::template launch<RowCfg<4, 2, 32>>(a, blocks, s);
    if (nq <= 4) return K::template launch<RowCfg<4, 4, 32>>(a, blocks, s);
    return K::template launch<RowCfg<4, 8, 32>>(a, blocks, s);
  }
  if (a.lanes < 32) return K::template launch<RowCfg<1, 1, 0>>(a, blocks, s);
  if (nq <= 1) return K::template launch<RowCfg<1, 1, 32>>(a, blocks, s);
  if (nq <= 2) return K::template launch<RowCfg<1, 2, 32>>(a, blocks, s);
  if (nq <= 4) return K::template launch<RowCfg<1, 4, 32>>(a, blocks, s);
  if (nq <= 8) return K::template launch<RowCfg<1, 8, 32>>(a, blocks, s);
  if (nq <= 16) return K::template launch<RowCfg<1, 16, 32>>(a, blocks, s);
  return K::template launch<RowCfg<1, 32, 32>>(a, blocks, s);
}

// Rows of a window where `blocks` of them are to cover T: 32 at least.
int rows_for(int64_t T, int64_t blocks) {
  const int64_t per = (T + blocks - 1) / blocks;
  return (int)(per < 32 ? 32 : per);
}
// Four blocks per SM of 148, two above 256 experts.  (A constant: the workspace's size follows from
// it and is asked for without a device.)
int64_t wanted_blocks(int E) { return E <= 256 ? 592 : 296; }
// Rows per window, forward.  Batches of up to 1024 rows and 32768 logits in few sequences: one window,
// which needs no second launch.  Otherwise as many (window, sequence) pairs as blocks are wanted
// if sequences are few (a block writes, and the second launch reads, a partial row per pair).
int window_rows(int64_t T, int E, int S) {
  if (T * E <= 32768 && T <= 1024 && S <= 4) return T > 0 ? (int)T : 1;
  const int64_t blocks = wanted_blocks(E);
  return rows_for(T, S < blocks / 2 ? blocks + 1 - S : blocks / 2);
}

moe_status_t check_shape(int64_t T, int32_t E, int32_t k, const int32_t* off, int32_t S) {
  if (T < 0 || S < 1) return MOE_ERR_INVALID_ARG;
  if (k < 1 || k > 32 || E < k || E > 1024 || S >= (1 << 24)) return MOE_ERR_UNSUPPORTED;
  if (T * (int64_t)k >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  if (off == nullptr && S != 1) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Slots for any batch of up to T rows: windows get longer where T passes what their number covers, so
// a shorter batch may have more of them.  (The last summand: nor does it shrink when S grows.)
int64_t most_slots(int64_t T, int E, int S) {
  const int64_t blocks = wanted_blocks(E), most = S < blocks / 2 ? blocks + 1 - S : blocks / 2 + 1;
  const int64_t shortest = (T + 31) / 32;
  return (shortest < most ? shortest : most) + S;
}

struct BalanceLayout {
  int64_t n_win;
  size_t psum, pcnt, pn, total;
};
BalanceLayout make_layout(int64_t T, int E, int S) {
  BalanceLayout L{};
  const int rows = window_rows(T, E, S);
  L.n_win = (T + rows - 1) / rows;
  const int64_t slots = most_slots(T, E, S);
  const size_t row = ((size_t)slots * E * 4 + 255) & ~size_t(255);
  L.psum = 0;
  L.pcnt = row;
  L.pn = 2 * row;
  L.total = 2 * row + (((size_t)slots * 4 + 255) & ~size_t(255));
  return L;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_balance_workspace_bytes(int64_t T, int32_t E, int32_t S) {
  if (T < 0 || E < 1 || E > 1024 || S < 1 || S >= (1 << 24) || T >= (int64_t(1) << 31)) return 0;
  return make_layout(T, E, S).total;
}

moe_status_t moe_balance_loss(const float* logits, const int32_t* topk_ids, int64_t T, int32_t E,
                              int32_t k, const int32_t* seq_offsets, int32_t S,
                              const uint8_t* token_mask, float* loss, int32_t* counts,
                              int32_t* n_tokens, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nr("moe_balance_loss");
  moe_status_t st = check_shape(T, E, k, seq_offsets, S);
  if (st != MOE_OK) return st;
  if (loss == nullptr || counts == nullptr || n_tokens == nullptr || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (logits == nullptr || topk_ids == nullptr)) return MOE_ERR_INVALID_ARG;
  const BalanceLayout L = make_layout(T, E, S);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  BalanceArgs a{};
  a.logits = logits;
  a.ids = topk_ids;
  a.off = seq_offsets;
  a.mask = token_mask;
  a.T = T;
  a.E = E;
  a.k = k;
  a.S = S;
  a.rows = window_rows(T, E, S);
  char* base = static_cast<char*>(ws);
  a.psum = reinterpret_cast<float*>(base + L.psum);
  a.pcnt = reinterpret_cast<int32_t*>(base + L.pcnt);
  a.pn = reinterpret_cast<int32_t*>(base + L.pn);
  a.err = moe_status_word();
  if (a.err == nullptr) return MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  a.out_counts = counts;
  a.out_n = n_tokens;
  const bool one = L.n_win == 1;
  a.loss = one ? loss : nullptr;
  if (T > 0 && launch_rows<Forward>(a, L.n_win + S - 1, s) != cudaSuccess) return MOE_ERR_CUDA;
  if (!one) {
    a.loss = loss;
    ProfScope ps(K_BALANCE_SUM, s);
    // many windows per sequence: large blocks; as many of them as find work, while there are SMs
    const bool many = L.n_win > 32 * (int64_t)S;
    const int64_t parts = ((E + kGroup - 1) / kGroup) * (L.n_win / S / 32 + 1);
    a.sum_ranks = 1;
    while (a.sum_ranks < kMaxRanks && a.sum_ranks < parts && S * (int64_t)a.sum_ranks < device_sms()) a.sum_ranks *= 2;
    const dim3 grid((unsigned)S * a.sum_ranks), block(many ? kSumThreads : kThreads);
    const cudaError_t e = E % 4 == 0 ? launch_pdl(balance_sum_kernel<true>, grid, block, 0, s, a.sum_ranks, a)
                                     : launch_pdl(balance_sum_kernel<false>, grid, block, 0, s, a.sum_ranks, a);
    if (e != cudaSuccess)
      return MOE_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t moe_balance_loss_backward(const float* logits, const int32_t* counts,
                                       const int32_t* n_tokens, const float* dloss, int64_t T,
                                       int32_t E, int32_t k, const int32_t* seq_offsets, int32_t S,
                                       const uint8_t* token_mask, float* dlogits,
                                       int32_t accumulate, void* stream) {
  NvtxRange nr("moe_balance_loss_backward");
  moe_status_t st = check_shape(T, E, k, seq_offsets, S);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (logits == nullptr || counts == nullptr || n_tokens == nullptr || dloss == nullptr || dlogits == nullptr)
    return MOE_ERR_INVALID_ARG;
  BalanceArgs a{};
  a.logits = logits;
  a.off = seq_offsets;
  a.mask = token_mask;
  a.T = T;
  a.E = E;
  a.k = k;
  a.S = S;
  a.rows = rows_for(T, wanted_blocks(E));
  a.counts = counts;
  a.n_tokens = n_tokens;
  a.dloss = dloss;
  a.dlogits = dlogits;
  a.accumulate = accumulate;
  a.err = moe_status_word();
  if (a.err == nullptr) return MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (launch_rows<Backward>(a, (T + a.rows - 1) / a.rows, s) != cudaSuccess) return MOE_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
