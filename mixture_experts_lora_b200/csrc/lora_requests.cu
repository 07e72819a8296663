// Low-rank adapters of many requests beside a shared projection, in place on its output:
//   Y[t] += c_a (X[t] A_a) B_a,   a the adapter of t's request.
//
// Reads X once, reads and writes Y once, and reads a row's or a tile's adapter for each of them (from
// L2 where several share one): bound by HBM for long prompts, by latency for a few tokens.  Two forms:
//
// lora_tiles_kernel, for larger batches of requests of any length.  Rows are cut into windows of 128; a
// cluster of 1 to 8 CTAs owns the rows of one request within one window and runs both
// products in one launch, so that X A never leaves the chip:
//   1. X A: each CTA sums its share of K, 64 columns a stage: TMA brings the rows of X and
//      64 rows of A, tcgen05.mma adds S[128 x RP] in TMEM;
//   2. each CTA receives the partial S of its share of the rows in its shared memory and sums them
//      in rank order; c S, split into two bf16 (its rounding and what the rounding left), goes to
//      every CTA as rows of the K-major operand of the second product, K = 2 RP.  Both ways by stores
//      that count their bytes at the receiver's mbarrier (128 rows, rank 16: 1.2 us less than with
//      stores, arrivals and a bulk copy of the operand);
//   3. each CTA takes its share of the columns, 64 a stage: TMA brings the rows of Y and 64
//      columns of B, tcgen05.mma forms S B in TMEM, the epilogue warps add it to Y in
//      shared memory, and TMA stores the rows back.
// A stage of either product is 16 KB of rows and RP x 64 of the adapter, so both run through
// one ring of slots, and the first stages of Y and B arrive while X A is still being
// summed.  The split over a cluster is for batches of few windows: it spreads one window's
// bytes over as many SMs.  Only 32-row boxes that hold rows of the request are copied; a box
// that it shares with another request is stored row by row.
//
// lora_single_kernel, for one row per request and for small batches: a cluster per row.
#include <climits>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "sequences.cuh"
#include "tmap.cuh"

namespace moe {
namespace {


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

__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// 16 bytes to another CTA's shared memory (dst and bar as mapa_smem gives them), counted there.
__device__ __forceinline__ void st_async_u4(uint32_t dst, uint4 v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
               "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void st_async_f32(uint32_t dst, float v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(dst),
               "r"(__float_as_uint(v)), "r"(bar)
               : "memory");
}

// For mbarriers that other CTAs of the cluster complete: the waiter sees what they stored.
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, int* err) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((i & 31u) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) {
      report_error(err, MOE_ERR_TIMEOUT);
      return false;
    }
  }
}

// ---------------------------------------------------------------- one row
// One row x by a cluster.  CTA j sums x A over its share of K in fp32, then adds its share of
// the columns.  Both operands stream through one ring of shared-memory slots by bulk copies that
// one warp issues, so that the memory is busy from the first cycle on and B arrives while the
// CTAs exchange their sums (registers as buffers held too few bytes: 64 rows at 7168 x 2048, rank
// 32 took 1.3 us more):
//   * a slot of A is 16 KB of the adapter's share of K rows as they lie, and those rows' x.  A
//     thread takes 16 bytes (eight ranks of one K row), GP = 2^k >= r / 8 threads side by side
//     on a K row, so that lanes GP apart hold the same ranks: a warp is summed by shuffles, the
//     warps and then the CTAs (through distributed shared memory) in a fixed order;
//   * a slot of B is some of its rows, cut to the CTA's columns.  A thread takes eight columns
//     of every parts-th row, the parts are summed in order.
constexpr int kConsumers = 256;             // and one warp that issues the copies
constexpr int kSingleThreads = kConsumers + 32;
constexpr int kSlotBytes = 16384, kSlotX = 2048, kSlots = 5;
constexpr int kMaxCluster = 8;

struct RowSmem {
  uint8_t slot[kSlots][kSlotBytes + kSlotX];
  float4 out[2][kConsumers];                // partial sums of eight columns
  float warp[kConsumers / 32][128];
  float part[kMaxCluster][128];             // every CTA's sum over its share of K
  float xa[128];
  uint64_t full[kSlots], empty[kSlots];
  uint64_t met;                             // every CTA's sum is here
};

// Bytes from global to this CTA's shared memory, counted by one of its mbarriers.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void add_scaled(float (&y)[8], uint4 w, float x) {
  float v[8];
  unpack8(w, v);
#pragma unroll
  for (int c = 0; c < 8; ++c) y[c] += x * v[c];
}

// A cluster per row: request s is row s, or the row's request is looked up.
__global__ void __launch_bounds__(kSingleThreads) lora_single_kernel(const LoraArgs a) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  RowSmem& sm = *reinterpret_cast<RowSmem*>(smem_raw);
  const int tid = threadIdx.x, warp = warp_id(), lane = lane_id();
  const int rank = (int)cluster_ctarank(), CL = (int)cluster_nctarank();
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_u32(&sm.full[i]), 1);
      mbar_init(smem_u32(&sm.empty[i]), kConsumers / 32);
    }
    mbar_init(smem_u32(&sm.met), 1);
    mbar_fence_init();
  }
  pdl_begin();
  const int row = (int)blockIdx.x / CL;
  int s = row;
  if (a.off != nullptr) {
    check_offsets(a.off, a.S, a.T, a.err);
    s = block_count_le(a.S, row, [&](int i) { return a.off[i + 1]; });       // the first that ends past the row
    if (s >= a.S) return;
    const int lo = a.off[s], hi = a.off[s + 1];
    if (row < lo || lo < 0 || hi > a.T) return;
  }
  const int ad = a.adapters[s];
  if (ad < 0) return;                          // (the same for the cluster)
  if (ad >= a.n_adapters) {
    if (tid == 0) report_error(a.err, MOE_ERR_DEVICE_INDEX);
    return;
  }
  const int r = a.r;
  // ---- this CTA's share of K (a multiple of 8 rows), in chunks of whole groups of 8 rows
  const int kc = ((a.K + CL - 1) / CL + 7) / 8 * 8;
  const int k0 = rank * kc < a.K ? rank * kc : a.K, k1 = k0 + kc < a.K ? k0 + kc : a.K;
  const int rows_c = kSlotBytes / (r * 2) / 8 * 8;                    // (r = 8: 1024 rows, 2 KB of x)
  const int na = (k1 - k0 + rows_c - 1) / rows_c;
  // ---- this CTA's groups of eight columns, in passes of cp, each in chunks of rb rows of B
  const int ng = a.N / 8, ng_c = (ng + CL - 1) / CL;
  const int g0 = rank * ng_c < ng ? rank * ng_c : ng, g1 = g0 + ng_c < ng ? g0 + ng_c : ng;
  int cp = 32;
  while (cp < kConsumers && cp < ng_c) cp *= 2;
  const int passes = (g1 - g0 + cp - 1) / cp;
  const int rb = kSlotBytes / (cp * 16) < r ? kSlotBytes / (cp * 16) : r;
  const int nb = (r + rb - 1) / rb;
  __syncthreads();
  bool ok = true;
  // Every CTA's barriers are set up and its shared memory may be written.  (Only in a cluster:
  // without one a barrier would make the consumers wait for the copy warp, which waits for them.)
  if (CL > 1) cluster_arrive();

  if (warp == kConsumers / 32) {
    // ------------------------------------------------------------ copies
    const __nv_bfloat16* A = a.A + ((int64_t)ad * a.K + k0) * r;
    const __nv_bfloat16* X = a.X + (int64_t)row * a.ldx + k0;
    const __nv_bfloat16* B = a.B + (int64_t)ad * r * a.N + (int64_t)g0 * 8;
    const int total = na + passes * nb;
    int it = 0;
    for (; it < total; ++it) {
      const int st = it % kSlots;
      if (it >= kSlots) ok = mbar_wait(smem_u32(&sm.empty[st]), (it / kSlots - 1) & 1, a.err);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t bar = smem_u32(&sm.full[st]), dst = smem_u32(sm.slot[st]);
      if (it < na) {
        const int o = it * rows_c, n = k1 - k0 - o < rows_c ? k1 - k0 - o : rows_c;
        if (elect_one()) {
          mbar_arrive_expect_tx(bar, (uint32_t)n * (r * 2 + 2));
          bulk_load(dst, A + (int64_t)o * r, (uint32_t)n * r * 2, bar);
          bulk_load(dst + kSlotBytes, X + o, (uint32_t)n * 2, bar);
        }
      } else {
        const int p = (it - na) / nb, j0 = (it - na) % nb * rb;
        const int seg = g1 - g0 - p * cp < cp ? g1 - g0 - p * cp : cp;
        const int n = r - j0 < rb ? r - j0 : rb;
        if (elect_one()) mbar_arrive_expect_tx(bar, (uint32_t)(n * seg) * 16);
        __syncwarp();
        for (int j = lane; j < n; j += 32)
          bulk_load(dst + j * cp * 16, B + (int64_t)(j0 + j) * a.N + (int64_t)p * cp * 8, (uint32_t)seg * 16, bar);
      }
      __syncwarp();
    }
    // after a failed wait, the copies on their way land before the CTA ends
    for (int j = it < kSlots ? 0 : it - kSlots; !ok && j < it; ++j)
      mbar_wait(smem_u32(&sm.full[j % kSlots]), (j / kSlots) & 1, a.err);
    __syncwarp();
    if (CL > 1) cluster_wait();
    return;
  }

  // -------------------------------------------------------------- consumers
  const float scale = a.scale[ad];
  const auto meet = [&]() {                    // (whole warps: what came before may have split them)
    __syncwarp();
    named_bar(1, kConsumers);
  };
  int it = 0;
  const auto wait_full = [&]() {
    if (ok) ok = mbar_wait(smem_u32(&sm.full[it % kSlots]), (it / kSlots) & 1, a.err);
  };
  const auto release = [&]() {                 // (the slot's reads of this warp are done)
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm.empty[it % kSlots]));
    __syncwarp();
    ++it;
  };
  int gp = 1;
  while (gp < r / 8) gp *= 2;
  const int g = tid & (gp - 1), kl = tid / gp, lanes = kConsumers / gp;
  const bool has = g * 8 < r;
  float acc[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) acc[c] = 0.f;
  for (int c = 0; c < na; ++c) {
    const int o = c * rows_c, n = k1 - k0 - o < rows_c ? k1 - k0 - o : rows_c;
    wait_full();
    const uint8_t* p = sm.slot[it % kSlots];
    const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(p + kSlotBytes);
    if (has) {
#pragma unroll 4
      for (int k = kl; k < n; k += lanes)
        add_scaled(acc, *reinterpret_cast<const uint4*>(p + (k * r + g * 8) * 2), __bfloat162float(x[k]));
    }
    release();
  }
  for (int o = gp; o < 32; o <<= 1) {
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] += __shfl_xor_sync(0xffffffffu, acc[c], o);
  }
  if (lane < gp && has) {
#pragma unroll
    for (int c = 0; c < 8; ++c) sm.warp[warp][g * 8 + c] = acc[c];
  }
  // the eight elements of Y that this thread finishes in a pass
  uint4* yp = reinterpret_cast<uint4*>(a.Y + (int64_t)row * a.ldy) + g0 + tid;
  const auto ends = [&](int pass) { return tid < cp && g0 + pass * cp + tid < g1; };
  uint4 yv = make_uint4(0u, 0u, 0u, 0u);
  if (ends(0)) yv = *yp;
  meet();
  // the sums to every CTA, by stores that count their bytes there (64 rows at 7168 x 2048, rank 32:
  // 9.5 us, 0.7 us more with plain stores and a cluster barrier)
  if (CL > 1) cluster_wait();
  if (tid == 0 && CL > 1) mbar_arrive_expect_tx(smem_u32(&sm.met), (uint32_t)(CL * r) * 4);
  if (tid < r) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kConsumers / 32; ++i) v += sm.warp[i][tid];
    const uint32_t mine = smem_u32(&sm.part[rank][tid]), met = smem_u32(&sm.met);
    if (CL == 1) sm.part[0][tid] = v;
    else
      for (int q = 0; q < CL; ++q) st_async_f32(mapa_smem(mine, (uint32_t)q), v, mapa_smem(met, (uint32_t)q));
  }
  __syncwarp();
  if (CL > 1 && !mbar_wait_cluster(smem_u32(&sm.met), 0, a.err)) ok = false;
  if (tid < r) {                               // (without a cluster, each thread's own value)
    float v = 0.f;
    for (int i = 0; i < CL; ++i) v += sm.part[i][tid];
    sm.xa[tid] = v * scale;
  }
  meet();
  const int col = tid & (cp - 1), part = tid / cp, parts = kConsumers / cp;
  for (int pass = 0; pass < passes; ++pass) {
    float y[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) y[c] = 0.f;
    const bool in = g0 + pass * cp + col < g1;
    for (int c = 0; c < nb; ++c) {
      const int j0 = c * rb, n = r - j0 < rb ? r - j0 : rb;
      wait_full();
      const uint8_t* p = sm.slot[it % kSlots] + col * 16;
      if (in) {
#pragma unroll 4
        for (int j = part; j < n; j += parts)
          add_scaled(y, *reinterpret_cast<const uint4*>(p + j * cp * 16), sm.xa[j0 + j]);
      }
      release();
    }
    // the parts of a column group, summed in order
    sm.out[0][tid] = make_float4(y[0], y[1], y[2], y[3]);
    sm.out[1][tid] = make_float4(y[4], y[5], y[6], y[7]);
    meet();
    if (ends(pass)) {
      float v[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] = 0.f;
      for (int q = 0; q < parts; ++q) {
        const float4 lo = sm.out[0][q * cp + tid], hi = sm.out[1][q * cp + tid];
        v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
        v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
      }
      float old[8];
      unpack8(yv, old);
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] += old[c];
      if (ok) yp[pass * cp] = pack8(v);
      if (ends(pass + 1)) yv = yp[(pass + 1) * cp];
    }
    if (pass + 1 < passes) meet();
  }
}

cudaError_t launch_single(const LoraArgs& a, int64_t rows, int CL, cudaStream_t s) {
  const cudaError_t st = ensure_smem(lora_single_kernel, (int)sizeof(RowSmem));
  if (st != cudaSuccess) return st;
  ProfScope ps(K_LORA_REQUESTS, s);
  return launch_pdl(lora_single_kernel, dim3((unsigned)(rows * CL)), dim3(kSingleThreads), sizeof(RowSmem), s, CL, a);
}

// ---------------------------------------------------------------- rows of one adapter
template <int RP_>
struct TilesCfg {
  static constexpr int RP = RP_;
  static constexpr int BM = 128, BK = 64, BN = 64;
  static constexpr int ROWS_BYTES = BM * 64 * 2;          // X or Y rows of a stage
  static constexpr int AD_BYTES = RP * 64 * 2;            // A or B of a stage
  static constexpr int STAGE_BYTES = ROWS_BYTES + AD_BYTES;
  // two CTAs per SM up to rank 32 beside a cluster's PART buffer (a fourth stage at rank 32 would
  // leave one), what fits above
  static constexpr int STAGES = RP == 32 || RP == 128 ? 3 : 4;
  static constexpr int OP_ATOMS = RP <= 32 ? 1 : 2 * RP / 64;   // 64-column atoms of [hi | lo]
  static constexpr int OP_BYTES = OP_ATOMS * BM * 128;
  static constexpr int PART_BYTES = BM * RP * 4;          // exchanged partial (clusters only)
  static constexpr int BAR_BYTES = 256;
  static constexpr int ND = 4, TMEM_COLS = ND * 64;       // accumulators of 64 columns; S before them
  // S as the sum of NS accumulators that the stages take in turn: the tensor cores cut off what lies
  // below an accumulator's last bits instead of rounding it, an error of one sign that grows with the
  // accumulator and with the length of its chain (16384 products of one sign: 8.2e-5 of the sum in
  // one chain, 1.4e-5 in four; 16384 rows at 7168 x 4096, rank 32: 100 us both ways)
  static constexpr int NS = RP == 128 ? 2 : 4;
  // two groups of four epilogue warps (the second stage by stage in turn with the first), two loaders
  // (one issues about one copy in 150 cycles), MMA issuer
  static constexpr int THREADS = 352;
  static constexpr int LOADER = 8, ISSUER = 9, ADAPTER = 10;
  static int smem_bytes(bool cluster) {
    return STAGES * STAGE_BYTES + OP_BYTES + (cluster ? PART_BYTES : 0) + BAR_BYTES + 1024;
  }
  // A chunk [64 K rows][RP], rank innermost: rows of up to 128 bytes, two atoms at rank 128
  static constexpr uint32_t A_SW = RP == 16 ? kSw32 : RP == 32 ? kSw64 : kSw128;
  static constexpr int A_ROWB = (RP < 64 ? RP : 64) * 2;
  static constexpr int A_ATOMS = RP > 64 ? 2 : 1;
  static constexpr int A_ATOM_BYTES = BK * A_ROWB;
};

// (Registers are given to warps in fours: two blocks of eleven warps hold as many as two of twelve.)
template <class C>
__global__ void __launch_bounds__((C::THREADS + 127) / 128 * 128, 2)
    lora_tiles_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmA,
                      const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmY,
                      const LoraArgs a) {
  constexpr int RP = C::RP, S = C::STAGES;
  extern __shared__ __align__(1024) uint8_t smem_tiles[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_tiles) + 1023) & ~uintptr_t(1023));
  uint8_t* op = smem + S * C::STAGE_BYTES;                 // [hi | lo] operand of the second product
  uint64_t* bars = reinterpret_cast<uint64_t*>(op + C::OP_BYTES);
  float* recv = reinterpret_cast<float*>(op + C::OP_BYTES + C::BAR_BYTES);   // clusters only
  uint64_t* full = bars;                 // [S] TMA bytes of the stage landed
  uint64_t* xfree = bars + S;            // [S] the MMAs of an X stage completed
  uint64_t* yfree = bars + 2 * S;        // [S] a Y stage's rows are stored (4 warps)
  uint64_t* dfull = bars + 3 * S;        // [ND] product ready in TMEM
  uint64_t* dfree = dfull + C::ND;       // [ND] product read (4 warps)
  uint64_t* acc_done = dfree + C::ND;
  uint64_t* op_ready = acc_done + 1;         // S is read (and without a cluster the operand written)
  uint64_t* drain = acc_done + 2;
  uint64_t* recv_ready = acc_done + 3;       // every CTA's partial of this CTA's rows is here
  uint64_t* op_full = acc_done + 4;          // every CTA's rows of the operand are here
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_done + 5);

  const int tid = threadIdx.x, warp = warp_id(), lane = lane_id();
  const int rank = (int)cluster_ctarank(), CL = (int)cluster_nctarank();
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&full[i]), 2);
      mbar_init(smem_u32(&xfree[i]), 1);
      mbar_init(smem_u32(&yfree[i]), 4);
    }
    for (int i = 0; i < C::ND; ++i) {
      mbar_init(smem_u32(&dfull[i]), 1);
      mbar_init(smem_u32(&dfree[i]), 4);
    }
    mbar_init(smem_u32(acc_done), 1);
    mbar_init(smem_u32(op_ready), C::BM);
    mbar_init(smem_u32(op_full), 1);
    mbar_init(smem_u32(drain), 1);
    mbar_init(smem_u32(recv_ready), 1);
    mbar_fence_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmY);
  }
  // (The dependents are let in only when this CTA holds its TMEM columns, below: other kernels take theirs
  // before they wait for this grid to end, and would then wait for each other.)
  pdl_wait();
  check_offsets(a.off, a.S, a.T, a.err);
  // the cluster's tile, the same for all its CTAs: slot -> (window, request) -> rows, adapter
  const int slot = (int)blockIdx.x / CL;
  int s, ad;
  int64_t lo, hi;
  if (a.S <= C::THREADS) {
    // a thread per request: one of them finds the slot among its own (one wait for memory)
    __shared__ int found[4];
    if (tid == 0) found[0] = -1;
    int f0 = 0, f1 = 0, o0 = 0, o1 = 0, my_ad = 0;
    if (tid < a.S) {
      o0 = a.off[tid];
      o1 = a.off[tid + 1];
      my_ad = a.adapters[tid];
      f0 = o0 / C::BM + tid;
      f1 = tid + 1 < a.S ? o1 / C::BM + tid + 1 : INT_MAX;
    }
    __syncthreads();
    // (offsets that decrease give a slot to several requests: every CTA of the cluster takes the last)
    if (tid < a.S && f0 <= slot && slot < f1) atomicMax(&found[0], tid);
    __syncthreads();
    s = found[0];
    if (s < 0) return;
    if (tid == s) {
      found[1] = o0; found[2] = o1; found[3] = my_ad;
    }
    __syncthreads();
    lo = found[1]; hi = found[2]; ad = found[3];
  } else {
    s = block_count_le(a.S, slot, [&](int i) { return (long long)a.off[i] / C::BM + i; }) - 1;
    if (s < 0) return;
    lo = a.off[s]; hi = a.off[s + 1]; ad = a.adapters[s];
  }
  const int64_t w = slot - s;
  const int64_t row0 = w * C::BM;
  const int64_t r0 = row0 > lo ? row0 : lo, r1 = row0 + C::BM < hi ? row0 + C::BM : hi;
  if (lo < 0 || r1 > a.T || r0 >= r1 || ad < 0) return;
  if (ad >= a.n_adapters) {
    if (tid == 0) report_error(a.err, MOE_ERR_DEVICE_INDEX);
    return;
  }
  // 32-row boxes that hold rows of the request
  const int box0 = (int)(r0 - row0) / 32, box1 = (int)(r1 - 1 - row0) / 32 + 1;
  const int nk = (a.K + C::BK - 1) / C::BK, nn = (a.N + C::BN - 1) / C::BN;
  const int n_x = (nk - rank + CL - 1) / CL;      // this CTA's stages: rank, rank + CL, ...
  const int n_y = rank < nn ? (nn - rank + CL - 1) / CL : 0;
  // rows in such boxes among the 128 / CL that this CTA sums up
  const int own = C::BM / CL, own_rows = max(0, min(box1 * 32, (rank + 1) * own) - max(box0 * 32, rank * own));

  if (warp == C::ISSUER) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;
  // Two cluster barriers: this CTA's barriers are set up; all that it sends is on its way, and what
  // comes is waited for (so that no CTA ends before).  Warps that do not send pass from the first to
  // the second when they have time, for the last arrival takes a microsecond to be seen.
  const auto pass = [&]() {
    cluster_wait();
    cluster_arrive();
  };
  if (CL > 1) {
    cluster_arrive();
    if (warp == C::ISSUER || (warp >= 4 && warp < 8)) pass();
  }

  if (warp == C::LOADER || warp == C::ADAPTER) {
    // ------------------------------------------------------------ loaders: rows of X and Y; the adapter
    if (elect_one()) {
      const bool ofrows = warp == C::LOADER;
      const uint32_t bytes = ofrows ? (uint32_t)(box1 - box0) * 32 * 128 : C::AD_BYTES;
      const uint32_t part = smem_u32(smem) + (ofrows ? box0 * 4096 : C::ROWS_BYTES);
      const int y_lap = n_x / S, y_st = n_x % S;   // the first Y stage's lap of the ring and slot
      int it = 0, st = 0, lap = 0, col = rank * 64;
      for (; it < n_x + n_y; ++it) {
        if (lap > 0) {
          // the slot's last stage was an X stage (its MMAs read it) or a Y stage (stored)
          const bool stored = it - S >= n_x;
          const int uses = stored ? y_lap + (st < y_st ? 1 : 0) : 0;     // laps before the first of that kind
          ok = mbar_wait(smem_u32(stored ? &yfree[st] : &xfree[st]), (lap - 1 - uses) & 1, a.err);
          if (!ok) break;
        }
        const uint32_t dst = part + st * C::STAGE_BYTES, fb = smem_u32(&full[st]);
        mbar_arrive_expect_tx(fb, bytes);
        if (it == n_x) col = rank * 64;
        if (ofrows) {
          const CUtensorMap* map = it < n_x ? &tmX : &tmY;
          for (int b = 0; b < box1 - box0; ++b) tma_load_2d(map, fb, dst + b * 4096, col, (int)row0 + (box0 + b) * 32);
        } else if (it < n_x) {
#pragma unroll
          for (int x = 0; x < C::A_ATOMS; ++x) tma_load_3d(&tmA, fb, dst + x * C::A_ATOM_BYTES, x * 64, col, ad);
        } else {
          tma_load_3d(&tmB, fb, dst, col, 0, ad);
        }
        col += CL * 64;
        if (++st == S) {
          st = 0;
          ++lap;
        }
      }
      // after a failed wait, the copies on their way land before the CTA ends
      for (int j = it < S ? 0 : it - S; !ok && j < it; ++j) mbar_wait(smem_u32(&full[j % S]), (j / S) & 1, a.err);
    }
    __syncwarp();
  } else if (warp == C::ISSUER) {
    // ------------------------------------------------------------ MMA issuer
    // (one thread's instructions set the pace of a short chain: 340 ns a stage with one loader,
    // lane 0 and descriptors built per MMA, 190 ns with two, elected lanes and sums)
    if (elect_one()) {
      const uint32_t id1 = idesc_bf16(128, RP, 0, 1), id2 = idesc_bf16(128, C::BN, 0, 1);
      if (CL > 1) {
        // a row of S and a row of the operand are RP floats long, [hi | lo] in bf16
        if (own_rows > 0) mbar_arrive_expect_tx(smem_u32(recv_ready), (uint32_t)(CL * own_rows) * RP * 4);
        mbar_arrive_expect_tx(smem_u32(op_full), (uint32_t)(box1 - box0) * 32 * RP * 4);
      }
      // (an address counts in 16 bytes in a descriptor's low bits: stages and columns are added)
      const uint32_t adp = smem_u32(smem) + C::ROWS_BYTES;
      const uint64_t drows = smem_desc(smem_u32(smem), 16, 1024, kSw128), dop = smem_desc(smem_u32(op), 16, 1024, kSw128);
      const uint64_t da = smem_desc(adp, C::A_ATOM_BYTES, 8 * C::A_ROWB, C::A_SW);
      const uint64_t db = smem_desc(adp, RP * 128, 1024, kSw128);
      for (int it = 0; it < n_x && ok; ++it) {
        const int st = it % S;
        ok = mbar_wait(smem_u32(&full[st]), (it / S) & 1, a.err);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < C::BK / 16; ++kk)
          umma_bf16(tmem + it % C::NS * RP, drows + (uint32_t)(st * C::STAGE_BYTES + kk * 32) / 16,
                    da + (uint32_t)(st * C::STAGE_BYTES + kk * 16 * C::A_ROWB) / 16, id1, it >= C::NS || kk ? 1u : 0u);
        umma_commit(smem_u32(&xfree[st]));
      }
      umma_commit(smem_u32(acc_done));
      if (ok) ok = mbar_wait(smem_u32(op_ready), 0, a.err);
      if (CL > 1 && ok) {
        ok = mbar_wait_cluster(smem_u32(op_full), 0, a.err);
        fence_proxy_async_smem();              // (stored by threads, read by the MMAs)
      }
      tc_fence_after();
      for (int j = 0; j < n_y && ok; ++j) {
        const int it = n_x + j, st = it % S, d = j % C::ND;
        ok = mbar_wait(smem_u32(&full[st]), (it / S) & 1, a.err);
        if (ok && j >= C::ND) ok = mbar_wait(smem_u32(&dfree[d]), (j / C::ND - 1) & 1, a.err);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int kk = 0; kk < RP / 16; ++kk) {
            const int col = h * RP + kk * 16;
            umma_bf16(tmem + d * C::BN, dop + ((col / 64) * (C::BM * 128) + (col % 64) * 2) / 16,
                      db + (uint32_t)(st * C::STAGE_BYTES + kk * 16 * 128) / 16, id2, (h | kk) ? 1u : 0u);
          }
        umma_commit(smem_u32(&dfull[d]));
      }
      if (!ok) {       // the MMAs on their way are done before TMEM is freed
        umma_commit(smem_u32(drain));
        mbar_wait(smem_u32(drain), 0, a.err);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue warps: tile row = tid % 128
    const int group = warp / 4, quarter = warp % 4, trow = tid % C::BM;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const bool mine = quarter >= box0 && quarter < box1;   // this warp's box holds rows
    if (group == 0) {
      ok = mbar_wait(smem_u32(acc_done), 0, a.err);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      const float c = a.scale[ad];
      // 16 columns of S from c0 on: the accumulators in use, summed in fp32
      const auto load_s = [&](int c0, float (&x)[16]) {
        uint32_t v[16];
        tmem_ld16(lanes + c0, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(v[i]);
#pragma unroll
        for (int q = 1; q < C::NS; ++q) {
          if (q >= n_x) break;
          tmem_ld16(lanes + q * RP + c0, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] += __uint_as_float(v[i]);
        }
      };
      // c S of a row's eight columns from c0 on, split into two bf16: pieces of an operand row
      const auto write_op = [&](int t, int c0, const float (&x)[8], auto&& store) {
        float h[8], l[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // (ranks past r are zeros of A and B; a row that is not finite would bring 0 x inf into them)
          const float v = c0 < a.r ? x[i] * c : 0.f;
          h[i] = __bfloat162float(__float2bfloat16_rn(v));
          l[i] = isinf(h[i]) ? 0.f : v - h[i];
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int col = p * RP + c0, chunk = (col % 64) / 8;
          store(op + (col / 64) * (C::BM * 128) + t * 128 + ((chunk ^ (t & 7)) << 4), pack8(p == 0 ? h : l));
        }
      };
      if (CL == 1) {
#pragma unroll 1
        for (int c0 = 0; c0 < RP; c0 += 16) {
          float v[16];
          load_s(c0, v);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = v[8 * g + i];
            write_op(tid, c0 + 8 * g, x, [](uint8_t* at, uint4 v) { *reinterpret_cast<uint4*>(at) = v; });
          }
        }
        tc_fence_before();
        fence_proxy_async_smem();
        mbar_arrive(smem_u32(op_ready));
      } else {
        // Each CTA owns 128 / CL rows.  Every CTA stores its partial of them in the owner's memory
        // (row major, 16-byte pieces of row t at piece ^ t, so that rows differ in their banks) ...
        constexpr int PIECES = RP / 4;
        const int owner = tid / own;
        cluster_wait();                  // (long past: every CTA has set up its barriers)
        if (mine) {
          const uint32_t dst = mapa_smem(smem_u32(recv + (rank * own + tid % own) * RP), (uint32_t)owner);
          const uint32_t bar = mapa_smem(smem_u32(recv_ready), (uint32_t)owner);
#pragma unroll
          for (int c0 = 0; c0 < RP; c0 += 16) {
            float v[16];
            load_s(c0, v);
#pragma unroll
            for (int g = 0; g < 4; ++g)
              st_async_u4(dst + ((c0 / 4 + g) ^ (tid & (PIECES - 1))) * 16,
                          make_uint4(__float_as_uint(v[4 * g]), __float_as_uint(v[4 * g + 1]),
                                     __float_as_uint(v[4 * g + 2]), __float_as_uint(v[4 * g + 3])), bar);
          }
        }
        tc_fence_before();
        mbar_arrive(smem_u32(op_ready));
        __syncwarp();
        // ... and sums what it received for its own rows, in rank order, for all CTAs' operands
        if (own_rows > 0 && !mbar_wait_cluster(smem_u32(recv_ready), 0, a.err)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        for (int i = tid; i < own * (RP / 8); i += C::BM) {
          const int tl = i % own, g = i / own, t = rank * own + tl;
          if (t / 32 < box0 || t / 32 >= box1) continue;
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = 0.f;
          for (int q = 0; q < CL; ++q) {
            const float* src = recv + (q * own + tl) * RP;
            const float4 u = *reinterpret_cast<const float4*>(src + ((2 * g) ^ (t & (PIECES - 1))) * 4);
            const float4 v = *reinterpret_cast<const float4*>(src + ((2 * g + 1) ^ (t & (PIECES - 1))) * 4);
            x[0] += u.x; x[1] += u.y; x[2] += u.z; x[3] += u.w;
            x[4] += v.x; x[5] += v.y; x[6] += v.z; x[7] += v.w;
          }
          write_op(t, 8 * g, x, [&](uint8_t* at, uint4 v) {
            for (int q = 0; q < CL; ++q)
              st_async_u4(mapa_smem(smem_u32(at), (uint32_t)q), v, mapa_smem(smem_u32(op_full), (uint32_t)q));
          });
        }
        __syncwarp();
        cluster_arrive();
      }
    }
    const int64_t brow = row0 + quarter * 32;              // first row of this warp's box
    const bool whole = mine && brow >= r0 && brow + 32 <= r1;
    for (int j = group; j < n_y; j += 2) {
      const int it = n_x + j, st = it % S, d = j % C::ND;
      if (ok) ok = mbar_wait(smem_u32(&dfull[d]), (j / C::ND) & 1, a.err);
      if (ok) ok = mbar_wait(smem_u32(&full[st]), (it / S) & 1, a.err);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      uint8_t* rows = smem + st * C::STAGE_BYTES;
      const int n0 = (rank + j * CL) * C::BN;
      if (mine) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t v[32];
          tmem_ld32(lanes + d * C::BN + half * 32, v);
          uint4* p[4];
          uint4 old[4];
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            p[g] = reinterpret_cast<uint4*>(rows + trow * 128 + (((half * 4 + g) ^ (trow & 7)) << 4));
            old[g] = *p[g];
          }
          tmem_wait_ld();
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float y[8];
            unpack8(old[g], y);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] += __uint_as_float(v[8 * g + i]);
            *p[g] = pack8(y);
          }
        }
      }
      tc_fence_before();
      if (whole) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&dfree[d]));
          tma_store_2d(&tmY, smem_u32(rows + quarter * 4096), n0, (int)brow);
          bulk_commit_group();
          bulk_wait_read<0>();
          mbar_arrive(smem_u32(&yfree[st]));
        }
      } else {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&dfree[d]));
        if (mine) {
          // four rows at a time, eight lanes a row
#pragma unroll 4
          for (int i = 0; i < 32; i += 4) {
            const int t = quarter * 32 + i + lane / 8, g = lane & 7, n = n0 + g * 8;
            const int64_t row = row0 + t;
            if (row >= r0 && row < r1 && n < a.N)
              *reinterpret_cast<uint4*>(a.Y + row * a.ldy + n) =
                  *reinterpret_cast<const uint4*>(rows + t * 128 + ((g ^ (t & 7)) << 4));
          }
          fence_proxy_async_smem();        // (the slot's next bytes come by a bulk copy)
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(smem_u32(&yfree[st]));
      }
      __syncwarp();                      // (the TMEM loads that follow are for whole warps)
    }
    if (lane == 0) bulk_wait<0>();
    __syncwarp();
  }
  if (CL > 1) {
    if (warp == C::LOADER || warp == C::ADAPTER) pass();
    cluster_wait();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::ISSUER) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int RP>
cudaError_t launch_tiles(const LoraArgs& a, int CL, cudaStream_t s) {
  using C = TilesCfg<RP>;
  CUtensorMap tx, ta, tb, ty;
  // (without adapters nothing reads the maps of A and B: any valid tensor does)
  const bool none = a.n_adapters == 0;
  const uint64_t n = none ? 1 : (uint64_t)a.n_adapters;
  const void* A = none ? a.X : a.A;
  const void* B = none ? a.X : a.B;
  if (!encode2d(&tx, a.X, (uint64_t)a.T, (uint64_t)a.K, (uint64_t)a.ldx, 32, 64) ||
      !encode2d(&ty, a.Y, (uint64_t)a.T, (uint64_t)a.N, (uint64_t)a.ldy, 32, 64) ||
      !encode3d(&ta, A, n, (uint64_t)a.K, (uint64_t)a.r, 64, RP < 64 ? RP : 64) ||
      !encode3d(&tb, B, n, (uint64_t)a.r, (uint64_t)a.N, RP, 64))
    return cudaErrorInvalidValue;
  const int smem = C::smem_bytes(CL > 1);
  auto kern = lora_tiles_kernel<C>;
  cudaError_t st = ensure_smem(kern, C::smem_bytes(true));
  if (st != cudaSuccess) return st;
  const int64_t slots = (a.T + C::BM - 1) / C::BM + a.S - 1;
  ProfScope ps(K_LORA_REQUESTS, s);
  return launch_pdl(kern, dim3((unsigned)(slots * CL)), dim3(C::THREADS), smem, s, CL, tx, ta, tb, ty, a);
}

// CTAs per cluster, 1 to 8: what finishes the tiles soonest if a tile takes 1 / CL and the clusters
// that run at once are as many as measured: two CTAs per SM up to rank 32, one above, and on 148 SMs
// places for 33 clusters of four and 15 of eight (3 tiles, 7168 x 4096, rank 32: 15.4 us with 8, 23.8
// with 4, 40 with 2, 70 us with 1; 20 tiles, rank 64: 34.6 us with 8, 26.2 us with 4; 8 tiles, rank 128:
// 24, 32, 53, 88 us).  A last wave of a few clusters costs as much as a full one (rank 64, 35 tiles at
// 7168 x 4096: 52 us with 2, 59 us with 4), unless two CTAs share an SM, clusters are small and it holds
// less than a seventh (rank 16, 67 tiles at 2048 x 2048: 18.3 us with 4, 19.0 with 2, 27.6 us with 1).
int cluster_size(int64_t T, int S, int K, int r) {
  const double tiles = (double)((T + 127) / 128) + (S - 1);      // (requests cut windows)
  const int per_sm = r <= 32 ? 2 : 1;
  int best = 1;
  double most = 0.;
  for (int cl = 1; cl <= 8 && cl <= (K + 63) / 64; cl *= 2) {
    const double places = cl < 4 ? 1. / cl : cl == 4 ? 33. / 148. : 15. / 148.;      // per SM
    const double room = std::floor(device_sms() * places + 1e-6) * per_sm;
    if (cl == 8 && tiles > room) break;    // (35 tiles, rank 64: 60.7 us)
    const double waves = std::ceil(tiles / room - (per_sm == 2 ? 0.15 : 0.));
    const double gain = cl / (waves < 1. ? 1. : waves);
    if (gain > most * 1.1) {               // (a cluster has its own cost)
      most = gain;
      best = cl;
    }
  }
  return best;
}

// Whether an element of the T rows of K from x on, ldx apart, is one of the T rows of N from y on.
bool rows_overlap(const moe_bf16_t* x, int64_t ldx, int64_t K, const moe_bf16_t* y, int64_t ldy, int64_t N, int64_t T) {
  const int64_t d = (reinterpret_cast<intptr_t>(y) - reinterpret_cast<intptr_t>(x)) / (int64_t)sizeof(moe_bf16_t);
  if (d >= (T - 1) * ldx + K || -d >= (T - 1) * ldy + N) return false;
  // interleaved rows of one buffer: their columns must lie apart
  if (ldx != ldy) return true;
  const int64_t c = ((d % ldx) + ldx) % ldx;      // Y's first column within X's rows
  return c < K || c + N > ldx;
}

// CTAs per row of lora_single_kernel: 8 while all clusters find a place at once (15 of 8 CTAs),
// then what keeps the CTAs within two per SM (at 7168 x 2048, rank 32, an adapter each, with 8, 4, 2
// and 1: 15 rows 5.7, 7.0, 10.3, 16.7 us; 64 rows 14.8, 9.5, 10.6, 16.8 us; 128 rows 26.4, 17.8, 14.4,
// 17.2 us; 296 rows 64, 44, 37, 31.6 us.  The same wins at 2048 x 2048, rank 16, and at 7168 x 4096,
// rank 128: 61 us with 2 and 67 with 4 for 128 rows; at 512 x 512, rank 8 one CTA does, by 0.3 us at
// 15 rows and 1.2 us at 128).
int single_cluster(int64_t rows) {
  if (rows <= 15) return 8;
  int cl = 4;
  while (cl > 1 && rows * cl > 2 * (int64_t)device_sms()) cl /= 2;
  return cl;
}

// Rows of a batch of packed requests up to which it is worked through row by row, each row reading
// its adapter (rows and tiles, us: 15 rows at 7168 x 4096 6.7, 14.2 at rank 32, 8.8, 15.4 at rank 64 and
// 14.8, 19.7 at rank 128; 64 rows 10.8, 13.8 at rank 32, 16.8, 15.2 at rank 64 and 30, 20 at rank 128; at
// 512 x 512 64 rows 5.3, 6.1 at rank 16 and 7.3, 8.8 at rank 64).  Longer where the requests may be more
// tiles than clusters of eight find places for (96 rows in 40 requests: 16.6, 28.4 at rank 32 and 55, 60
// at rank 128).
int few_rows(int S, int r) {
  if (S > (r <= 32 ? 30 : 15)) return 128;
  return r <= 32 ? 64 : 24;
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
  if (rows_overlap(X, ldx, K, Y, ldy, N, T)) return MOE_ERR_INVALID_ARG;
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
  cudaError_t e;
  if (seq_offsets == nullptr || T <= few_rows(S, r)) {
    e = launch_single(a, T, single_cluster(T), s);
  } else {
    const int cl = cluster_size(T, S, K, r);
    e = r <= 16 ? launch_tiles<16>(a, cl, s) : r <= 32 ? launch_tiles<32>(a, cl, s)
        : r <= 64 ? launch_tiles<64>(a, cl, s) : launch_tiles<128>(a, cl, s);
  }
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
