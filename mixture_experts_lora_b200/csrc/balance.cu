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
// Forward: a block per window of rows, a warp per row (softmax in registers, lane l holds
// experts l, l + 32, ...); the lanes sum their experts' probabilities over the warp's rows,
// the block's warps are summed in a fixed order through shared memory, and each
// (window, sequence) pair writes one partial row; a second launch sums a sequence's
// partials in window order.  Everything is fp32 (counts: integers).
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
  float* psum;             // [slots][E]
  int32_t* pcnt;           // [slots][E]
  int32_t* pn;             // [slots]
  int* err;
  // backward
  const int32_t* counts;
  const int32_t* n_tokens;
  const float* dloss;
  float* dlogits;
  int accumulate;
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The row's softmax, lane l's experts l + 32 q in p[q] (0 past E; all 0 for a row of -inf).
template <int PL>
__device__ __forceinline__ void row_softmax(const float* __restrict__ x, int E, int lane,
                                            float (&p)[PL]) {
  float mx = -INFINITY;
#pragma unroll
  for (int q = 0; q < PL; ++q) {
    const int e = lane + 32 * q;
    p[q] = e < E ? x[e] : -INFINITY;
    mx = fmaxf(mx, p[q]);
  }
  mx = warp_max(mx);
  float sum = 0.f;
#pragma unroll
  for (int q = 0; q < PL; ++q) {
    p[q] = p[q] == -INFINITY ? 0.f : expf(p[q] - mx);
    sum += p[q];
  }
  sum = warp_sum(sum);
  // (a NaN logit may lose the maximum's comparison; the sum carries it)
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
  for (int q = 0; q < PL; ++q) p[q] *= inv;
}

template <int PL>
__global__ void __launch_bounds__(kThreads) balance_partial_kernel(const BalanceArgs a) {
  pdl_begin();
  extern __shared__ float s_dyn[];            // [kWarps][E] sums, then E counts
  float* s_sum = s_dyn;
  int* s_cnt = reinterpret_cast<int*>(s_dyn + kWarps * a.E);
  __shared__ int s_n;
  const int warp = warp_id(), lane = lane_id(), E = a.E;
  const int64_t w = blockIdx.x, t0 = w * a.rows;
  const int64_t t1 = t0 + a.rows < a.T ? t0 + a.rows : a.T;
  int s = 0;
  if (a.off != nullptr) {
    check_offsets(a.off, a.S, a.T, a.err);
    s = block_count_le(a.S, t0, [&](int i) { return a.off[i + 1]; });
  }
  for (; s < a.S; ++s) {
    int64_t r0 = a.off != nullptr ? a.off[s] : 0, r1 = a.off != nullptr ? a.off[s + 1] : a.T;
    if (r0 >= t1) break;
    r0 = r0 > t0 ? r0 : t0;
    r1 = r1 < t1 ? r1 : t1;
    if (r0 >= r1) continue;
    for (int e = threadIdx.x; e < E; e += kThreads) s_cnt[e] = 0;
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    float acc[PL];
#pragma unroll
    for (int q = 0; q < PL; ++q) acc[q] = 0.f;
    int n = 0;
    for (int64_t t = r0 + warp; t < r1; t += kWarps) {
      if (a.mask != nullptr && a.mask[t] == 0) continue;
      ++n;
      float p[PL];
      row_softmax<PL>(a.logits + t * E, E, lane, p);
#pragma unroll
      for (int q = 0; q < PL; ++q) acc[q] += p[q];
      if (lane < a.k) {
        const int e = a.ids[t * a.k + lane];
        if (e >= 0 && e < E) atomicAdd(&s_cnt[e], 1);
        else report_error(a.err, MOE_ERR_DEVICE_INDEX);
      }
    }
#pragma unroll
    for (int q = 0; q < PL; ++q)
      if (lane + 32 * q < E) s_sum[warp * E + lane + 32 * q] = acc[q];
    if (lane == 0) atomicAdd(&s_n, n);
    __syncthreads();
    const int64_t slot = w + s;
    for (int e = threadIdx.x; e < E; e += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) v += s_sum[i * E + e];
      a.psum[slot * E + e] = v;
      a.pcnt[slot * E + e] = s_cnt[e];
    }
    if (threadIdx.x == 0) a.pn[slot] = s_n;
    __syncthreads();
  }
}

// One block per sequence: its partial rows summed in window order.
__global__ void __launch_bounds__(kThreads)
    balance_sum_kernel(const BalanceArgs a, float* __restrict__ loss, int32_t* __restrict__ counts,
                       int32_t* __restrict__ n_tokens) {
  pdl_begin();
  __shared__ float s_part[kWarps];
  const int s = blockIdx.x, E = a.E;
  const int64_t n_win = (a.T + a.rows - 1) / a.rows;
  int64_t r0 = a.off != nullptr ? a.off[s] : 0, r1 = a.off != nullptr ? a.off[s + 1] : a.T;
  // first and last window of the sequence (none if it is empty), within the table whatever
  // the offsets hold
  int64_t w0 = 0, w1 = 0;
  if (r0 >= 0 && r1 > r0) {
    w0 = r0 / a.rows;
    w1 = (r1 - 1) / a.rows + 1;
    if (w1 > n_win) w1 = n_win;
  }
  int n = 0;
  for (int64_t w = w0; w < w1; ++w) n += a.pn[w + s];
  float part = 0.f;
  for (int e = threadIdx.x; e < E; e += kThreads) {
    float sum = 0.f;
    int cnt = 0;
    for (int64_t w = w0; w < w1; ++w) {
      sum += a.psum[(w + s) * E + e];
      cnt += a.pcnt[(w + s) * E + e];
    }
    counts[(int64_t)s * E + e] = cnt;
    part += (float)cnt * sum;
  }
  part = warp_sum(part);
  if (lane_id() == 0) s_part[warp_id()] = part;
  __syncthreads();
  if (threadIdx.x == 0) {
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) all += s_part[i];
    const float fn = (float)n;
    loss[s] = n > 0 ? all * ((float)E / ((float)a.k * fn)) / fn : 0.f;
    n_tokens[s] = n;
  }
}

template <int PL>
__global__ void __launch_bounds__(kThreads) balance_backward_kernel(const BalanceArgs a) {
  pdl_begin();
  const int warp = warp_id(), lane = lane_id(), E = a.E;
  const int64_t t0 = (int64_t)blockIdx.x * a.rows;
  const int64_t t1 = t0 + a.rows < a.T ? t0 + a.rows : a.T;
  int s = 0;
  if (a.off != nullptr) {
    check_offsets(a.off, a.S, a.T, a.err);
    s = block_count_le(a.S, t0, [&](int i) { return a.off[i + 1]; });
  }
  for (int64_t t = t0 + warp; t < t1; t += kWarps) {
    bool live = a.mask == nullptr || a.mask[t] != 0;
    if (a.off != nullptr) {
      while (s < a.S && a.off[s + 1] <= t) ++s;
      live = live && s < a.S && a.off[s] <= t;
    }
    float* out = a.dlogits + t * E;
    if (!live) {
      if (!a.accumulate)
        for (int e = lane; e < E; e += 32) out[e] = 0.f;
      continue;
    }
    float p[PL], f[PL];
    row_softmax<PL>(a.logits + t * E, E, lane, p);
    const float n = (float)a.n_tokens[s];
    const float g = n > 0.f ? a.dloss[s] * ((float)E / ((float)a.k * n)) / n : 0.f;
    float dot = 0.f;
#pragma unroll
    for (int q = 0; q < PL; ++q) {
      const int e = lane + 32 * q;
      f[q] = e < E ? (float)a.counts[(int64_t)s * E + e] * g : 0.f;
      dot += p[q] * f[q];
    }
    dot = warp_sum(dot);
#pragma unroll
    for (int q = 0; q < PL; ++q) {
      const int e = lane + 32 * q;
      if (e >= E) continue;
      const float d = p[q] * (f[q] - dot);
      out[e] = a.accumulate ? out[e] + d : d;
    }
  }
}

template <int PL>
cudaError_t launch_forward(const BalanceArgs& a, int64_t n_win, cudaStream_t st) {
  ProfScope ps(K_BALANCE, st);
  return launch_pdl(balance_partial_kernel<PL>, dim3((unsigned)n_win), dim3(kThreads),
                    (size_t)(kWarps + 1) * a.E * 4, st, 1, a);
}
template <int PL>
cudaError_t launch_backward(const BalanceArgs& a, int64_t n_win, cudaStream_t st) {
  ProfScope ps(K_BALANCE_BWD, st);
  return launch_pdl(balance_backward_kernel<PL>, dim3((unsigned)n_win), dim3(kThreads), 0, st, 1, a);
}

// Rows per window: at most about two windows per SM, so that a sequence's partial rows stay
// few, and at least four rows per warp.
int window_rows(int64_t T) {
  const int64_t per = (T + 295) / 296;
  return (int)(per < 32 ? 32 : per);
}

moe_status_t check_shape(int64_t T, int32_t E, int32_t k, const int32_t* off, int32_t S) {
  if (T < 0 || S < 1) return MOE_ERR_INVALID_ARG;
  if (k < 1 || k > 32 || E < k || E > 1024 || S >= (1 << 24)) return MOE_ERR_UNSUPPORTED;
  if (T * (int64_t)k >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  if (off == nullptr && S != 1) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

struct BalanceLayout {
  int64_t slots, n_win;
  size_t psum, pcnt, pn, total;
};
BalanceLayout make_layout(int64_t T, int E, int S) {
  BalanceLayout L{};
  const int rows = window_rows(T);
  L.n_win = (T + rows - 1) / rows;
  L.slots = L.n_win + S;
  const size_t row = ((size_t)L.slots * E * 4 + 255) & ~size_t(255);
  L.psum = 0;
  L.pcnt = row;
  L.pn = 2 * row;
  L.total = 2 * row + (((size_t)L.slots * 4 + 255) & ~size_t(255));
  return L;
}

}  // namespace
}  // namespace moe

using namespace moe;

#define MOE_BY_EXPERTS(E, CALL)                 \
  ((E) <= 32 ? CALL<1> : (E) <= 64 ? CALL<2>    \
   : (E) <= 128 ? CALL<4> : (E) <= 256 ? CALL<8> \
   : (E) <= 512 ? CALL<16> : CALL<32>)

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
  a.rows = window_rows(T);
  char* base = static_cast<char*>(ws);
  a.psum = reinterpret_cast<float*>(base + L.psum);
  a.pcnt = reinterpret_cast<int32_t*>(base + L.pcnt);
  a.pn = reinterpret_cast<int32_t*>(base + L.pn);
  a.err = moe_status_word();
  if (a.err == nullptr) return MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T > 0 && MOE_BY_EXPERTS(E, launch_forward)(a, L.n_win, s) != cudaSuccess) return MOE_ERR_CUDA;
  {
    ProfScope ps(K_BALANCE_SUM, s);
    if (launch_pdl(balance_sum_kernel, dim3((unsigned)S), dim3(kThreads), 0, s, 1, a, loss, counts,
                   n_tokens) != cudaSuccess)
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
  a.rows = window_rows(T);
  a.counts = counts;
  a.n_tokens = n_tokens;
  a.dloss = dloss;
  a.dlogits = dlogits;
  a.accumulate = accumulate;
  a.err = moe_status_word();
  if (a.err == nullptr) return MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (MOE_BY_EXPERTS(E, launch_backward)(a, (T + a.rows - 1) / a.rows, s) != cudaSuccess) return MOE_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
