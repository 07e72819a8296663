// Low-rank adapters of many requests beside a shared projection, in place on its output:
//   Y[t] += c_a (X[t] A_a) B_a,   a the adapter of t's request.
//
// Reads X once, the adapters in use once, reads and writes Y once: bound by HBM for long
// prompts, by latency for a few tokens.  A block owns the rows of one request within one
// window of kRows rows: it sums X A over K in fp32 (each thread eight rank columns of every
// blockDim-th row of A, joined through shared memory in a fixed order), then adds the
// product with B to its rows of Y.
#include "common.cuh"
#include "internal.h"
#include "sequences.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 8;

struct LoraArgs {
  const __nv_bfloat16* X;
  int64_t ldx;
  const int32_t* off;      // nullptr: request s is row s
  const int32_t* adapters;
  int64_t T;
  int S;
  const __nv_bfloat16* A;
  const __nv_bfloat16* B;
  const float* scale;
  int n_adapters, K, N, r;
  __nv_bfloat16* Y;
  int64_t ldy;
  int* err;
};

__global__ void __launch_bounds__(kThreads) lora_rows_kernel(const LoraArgs a) {
  pdl_begin();
  __shared__ float s_red[kThreads * 8];
  __shared__ float s_xa[kRows * 128];
  int s = blockIdx.x;
  int64_t r0 = s, r1 = s + 1;
  if (a.off != nullptr) {
    check_offsets(a.off, a.S, a.T, a.err);
    // the slot's sequence: the last whose first slot is not past it
    s = block_count_le(a.S, blockIdx.x, [&](int i) { return (long long)a.off[i] / kRows + i; }) - 1;
    if (s < 0) return;
    const int64_t w = (int64_t)blockIdx.x - s, lo = a.off[s], hi = a.off[s + 1];
    r0 = w * kRows > lo ? w * kRows : lo;
    r1 = (w + 1) * kRows < hi ? (w + 1) * kRows : hi;
    if (lo < 0 || r1 > a.T || r0 >= r1) return;
  }
  const int ad = a.adapters[s];
  if (ad < 0) return;
  if (ad >= a.n_adapters) {
    if (threadIdx.x == 0) report_error(a.err, MOE_ERR_DEVICE_INDEX);
    return;
  }
  const int nr = (int)(r1 - r0), tid = threadIdx.x;
  const int groups = a.r / 8, lanes = kThreads / groups;     // rank groups of 8, rows of A at a time
  const int g = tid % groups, kl = tid / groups;
  const __nv_bfloat16* A = a.A + (int64_t)ad * a.K * a.r;
  const __nv_bfloat16* B = a.B + (int64_t)ad * a.r * a.N;
  const __nv_bfloat16* X = a.X + r0 * a.ldx;
  float acc[kRows][8];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[i][c] = 0.f;
  if (kl < lanes) {
    for (int k = kl; k < a.K; k += lanes) {
      float v[8];
      unpack8(*reinterpret_cast<const uint4*>(A + (int64_t)k * a.r + g * 8), v);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (i >= nr) break;
        const float x = __bfloat162float(X[i * a.ldx + k]);
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[i][c] += x * v[c];
      }
    }
  }
  const float scale = a.scale[ad];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (i >= nr) break;
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 8; ++c) s_red[tid * 8 + c] = acc[i][c];
    __syncthreads();
    if (tid < a.r) {
      float sum = 0.f;
      for (int l = 0; l < lanes; ++l) sum += s_red[(l * groups + tid / 8) * 8 + (tid & 7)];
      s_xa[i * 128 + tid] = sum * scale;
    }
  }
  __syncthreads();
  for (int n = tid * 8; n < a.N; n += kThreads * 8) {
    float y[kRows][8];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int c = 0; c < 8; ++c) y[i][c] = 0.f;
    for (int j = 0; j < a.r; ++j) {
      float v[8];
      unpack8(*reinterpret_cast<const uint4*>(B + (int64_t)j * a.N + n), v);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (i >= nr) break;
        const float x = s_xa[i * 128 + j];
#pragma unroll
        for (int c = 0; c < 8; ++c) y[i][c] += x * v[c];
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (i >= nr) break;
      uint4* p = reinterpret_cast<uint4*>(a.Y + (r0 + i) * a.ldy + n);
      float v[8];
      unpack8(*p, v);
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] += y[i][c];
      *p = pack8(v);
    }
  }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_lora_requests(const moe_bf16_t* X, int64_t ldx, const int32_t* seq_offsets,
                                          const int32_t* adapters, int64_t T, int32_t S,
                                          const moe_bf16_t* A, const moe_bf16_t* B, const float* scale,
                                          int32_t n_adapters, int32_t K, int32_t N, int32_t r,
                                          moe_bf16_t* Y, int64_t ldy, void* stream) {
  NvtxRange nr("moe_lora_requests");
  if (T < 0 || S < 0 || n_adapters < 0) return MOE_ERR_INVALID_ARG;
  if (K < 16 || N < 16 || K % 16 != 0 || N % 16 != 0 || K > (1 << 19) || N > (1 << 19)) return MOE_ERR_UNSUPPORTED;
  if (r < 8 || r > 128 || r % 8 != 0 || T >= (1 << 24) || S >= (1 << 24)) return MOE_ERR_UNSUPPORTED;
  if (seq_offsets == nullptr && S != T) return MOE_ERR_INVALID_ARG;
  if (ldx < K || ldy < N || ldx % 8 != 0 || ldy % 8 != 0) return MOE_ERR_INVALID_ARG;
  if (T == 0 || S == 0) return MOE_OK;
  if (!aligned16(X) || !aligned16(Y) || adapters == nullptr) return MOE_ERR_INVALID_ARG;
  if (n_adapters > 0 && (!aligned16(A) || !aligned16(B) || scale == nullptr)) return MOE_ERR_INVALID_ARG;
  LoraArgs a{};
  a.X = reinterpret_cast<const __nv_bfloat16*>(X);
  a.ldx = ldx;
  a.off = seq_offsets;
  a.adapters = adapters;
  a.T = T;
  a.S = S;
  a.A = reinterpret_cast<const __nv_bfloat16*>(A);
  a.B = reinterpret_cast<const __nv_bfloat16*>(B);
  a.scale = scale;
  a.n_adapters = n_adapters;
  a.K = K;
  a.N = N;
  a.r = r;
  a.Y = reinterpret_cast<__nv_bfloat16*>(Y);
  a.ldy = ldy;
  a.err = moe_status_word();
  if (a.err == nullptr) return MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t blocks = seq_offsets == nullptr ? S : (T + kRows - 1) / kRows + S;
  ProfScope ps(K_LORA_REQUESTS, s);
  if (launch_pdl(lora_rows_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, 1, a) != cudaSuccess)
    return MOE_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
