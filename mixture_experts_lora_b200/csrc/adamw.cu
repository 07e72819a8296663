// One AdamW step over many tensors in one launch, states in fp32 or in 8 bits.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   w = w (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Every element is read and written once: the step is bound by HBM.  The tensors' table
// travels in the kernel's parameters, so a call needs no copy to the device and a captured
// call keeps its own table.  A warp takes 256 consecutive elements at a time, which is also the
// block of elements that shares a scale in 8 bits, so its maximum is a warp reduction.  Each
// tensor is cut into chunks of eight warps' work, one such block a warp, in 8 bits up to 32
// in a row; thread blocks walk the chunks.
//
// 8 bits: e4m3 codes of m and of sqrt(v) (the root halves the exponent range that a block
// has to span), scaled so that the block's largest value is 448.  A code is the value with
// 3 mantissa bits; the bits below are rounded up with probability equal to their value
// (random bits: a 32-bit integer mix of the element's index and t), so that the averages
// move as they should although one step changes them by less than a code.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kBlockElems = 256;     // elements that share a scale, and a warp's share
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRun = 32;                            // blocks per warp and chunk: a lane holds each's scales
constexpr int kChunk = kWarps * kBlockElems;            // elements of a chunk, times blocks per warp

struct Tensor {
  void* p;
  const void* g;
  float* w;
  void* m;
  void* v;
  float* ms;
  float* vs;
  int64_t n;
  uint32_t d1, d2;         // strided views: sizes of the two inner dimensions; d2 = 0: contiguous
  bool vec;                // groups of eight elements lie together, 16-byte aligned
  int64_t ps[3], gs[3];
};

template <int NT>
struct AdamwArgs {
  Tensor t[NT];
  int32_t chunk0[NT + 1];  // first chunk of each tensor
  int n;
  float lr, b1, b2, eps, wd, one_b1, one_b2, ln_b1, ln_b2;
  float one;               // 1, see update8
  const float* lr_dev;
  const float* grad_scale;
  long long* step;
  int advance;
  int blocks;              // blocks of 256 elements per warp and chunk
};

// A 32-bit integer mix (xor-shifts and odd multipliers: the fractional parts of the golden
// ratio and of the square root of 3).
__device__ __forceinline__ uint32_t mix_end(uint32_t x) {   // from x ^ (x >> 16)
  x *= 0x9E3779B9u;
  return (x ^ (x >> 15)) * 0xBB67AE85u;                     // (the last x ^= x >> 16 is the caller's)
}
__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x = mix_end(x ^ (x >> 16));
  return x ^ (x >> 16);
}

__device__ __forceinline__ float max_nan_abs(float a, float b) {   // a NaN wins
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// e4m3 code of |y|, |y| <= 448, in bits 20 to 27 (and y's sign in bit 31), from z = y 2^-120: that
// moves e4m3's exponents to the bottom of fp32's and makes e4m3's subnormals fp32's own, after
// which the low 20 mantissa bits are what is rounded: up if they and 20 random bits (16 and zeros)
// carry.
__device__ __forceinline__ uint32_t encode_bits(float z, uint32_t rnd16) {
  return __float_as_uint(z) + rnd16 * 16u;
}
// The codes of four such words as four bytes, and bytes with their signs in bit 7.
__device__ __forceinline__ uint32_t code_bytes(const uint32_t (&t)[4], uint32_t& signs) {
  const uint32_t lo = __byte_perm(t[0], t[1], 0x7632), hi = __byte_perm(t[2], t[3], 0x7632);
  signs = __byte_perm(lo, hi, 0x7531);
  return __byte_perm(lo << 4, hi << 4, 0x7531);
}
// 0x80 in every byte that is not zero (bytes up to 0x80).
__device__ __forceinline__ uint32_t nonzero_bytes(uint32_t w) { return (w + 0x7f7f7f7fu) & 0x80808080u; }

__device__ __forceinline__ float rsqrt_normal(float v) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// Two codes (the low bytes) as floats; e4m3 to fp16 and fp32 is exact.
__device__ __forceinline__ float2 decode2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

template <bool BF16>
__device__ __forceinline__ float load_one(const void* p, int64_t i) {
  if constexpr (BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ void store_one(void* p, int64_t i, float v) {
  if constexpr (BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<float*>(p)[i] = v;
}
// Eight consecutive elements from a 16-byte aligned place.
template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&x)[8]) {
  if constexpr (BF16) {
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i), x);
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 u = q[0], v = q[1];
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
  }
}
template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&x)[8]) {
  if constexpr (BF16) {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) = pack8(x);
  } else {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(x[0], x[1], x[2], x[3]);
    q[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// Offset of element i (row-major index of the view) under strides st.
__device__ __forceinline__ int64_t view_offset(const Tensor& t, int64_t i, const int64_t (&st)[3]) {
  if (t.d2 == 0) return i;
  const uint32_t u = (uint32_t)i, r = u / t.d2, c = u - r * t.d2, a = r / t.d1, b = r - a * t.d1;
  return a * st[0] + b * st[1] + c * st[2];
}

// The scalars of a step.
struct Step {
  float b1, b2, one_b1, one_b2, eps, gscale, c1, rbc2, keep, one;
};

// One element.  The moments are rounded operation by operation (no fused multiply-adds), as
// separate fp32 operations elsewhere round them: 8-bit codes then agree bit for bit.
__device__ __forceinline__ void moments(const Step& q, float g, float& m, float& v) {
  g = __fmul_rn(g, q.gscale);
  m = __fadd_rn(__fmul_rn(q.b1, m), __fmul_rn(q.one_b1, g));
  v = __fadd_rn(__fmul_rn(q.b2, v), __fmul_rn(q.one_b2, __fmul_rn(g, g)));
}
// The weight; the quotient by an approximate reciprocal (1 ulp).
__device__ __forceinline__ void weight(const Step& q, float m, float root, float& w) {
  w = w * q.keep - q.c1 * (m * rcp_approx(root * q.rbc2 + q.eps));
}

// Eight elements two at a time: m, v, sqrt(v), w from m, v, g, w.  The moments' sums are written as
// x * 1 + y with a 1 that the assembler cannot see: it makes one rounding of a packed product and
// a packed sum.  Returns whether every v is
// finite and at least 2^-100.  Their roots are one Newton step (v - s^2) / (2 s) from
// s = v rsqrt(v): equal to __fsqrt_rn for all 2^24 values of [1, 4), and so for their scalings
// by 4^k down to 2^-100 (below 2^-102 the bits of v - s^2 leave fp32's range), in half its
// instructions (the 8-bit step is bound by instruction issue).
__device__ __forceinline__ bool update8(const Step& q, const float (&g)[8], float (&m)[8], float (&v)[8],
                                        float (&u)[8], float (&w)[8]) {
  const f32x2 b1 = pack2(q.b1, q.b1), b2 = pack2(q.b2, q.b2), o1 = pack2(q.one_b1, q.one_b1),
              o2 = pack2(q.one_b2, q.one_b2), gs = pack2(q.gscale, q.gscale), rb = pack2(q.rbc2, q.rbc2),
              ep = pack2(q.eps, q.eps), kp = pack2(q.keep, q.keep), nc = pack2(-q.c1, -q.c1),
              one = pack2(q.one, q.one), mone = pack2(-1.f, -1.f), mhalf = pack2(-0.5f, -0.5f);
  f32x2 M[4], V[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const f32x2 G = mul2(pack2(g[2 * j], g[2 * j + 1]), gs);
    M[j] = fma2(mul2(b1, pack2(m[2 * j], m[2 * j + 1])), one, mul2(o1, G));
    V[j] = fma2(mul2(b2, pack2(v[2 * j], v[2 * j + 1])), one, mul2(o2, mul2(G, G)));
    const float2 x = unpack2(M[j]), y = unpack2(V[j]);
    m[2 * j] = x.x; m[2 * j + 1] = x.y;
    v[2 * j] = y.x; v[2 * j + 1] = y.y;
  }
  uint32_t low = __float_as_uint(v[0]), high = low;
#pragma unroll
  for (int j = 1; j < 8; ++j) {
    low = min(low, __float_as_uint(v[j]));
    high = max(high, __float_as_uint(v[j]));
  }
  const bool normal = low >= 0x0d800000u && high < 0x7f800000u;
  if (normal) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f32x2 r = pack2(rsqrt_normal(v[2 * j]), rsqrt_normal(v[2 * j + 1]));
      const f32x2 s = mul2(V[j], r);
      const float2 x = unpack2(fma2(fma2(s, s, mul2(V[j], mone)), mul2(r, mhalf), s));
      u[2 * j] = x.x; u[2 * j + 1] = x.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = __fsqrt_rn(v[j]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 den = unpack2(fma2(pack2(u[2 * j], u[2 * j + 1]), rb, ep));
    const f32x2 t = mul2(M[j], pack2(rcp_approx(den.x), rcp_approx(den.y)));
    const float2 x = unpack2(fma2(t, nc, mul2(pack2(w[2 * j], w[2 * j + 1]), kp)));
    w[2 * j] = x.x; w[2 * j + 1] = x.y;
  }
  return normal;
}

__device__ __forceinline__ void decode_m(uint2 c, float scale, float (&m)[8]) {
  const f32x2 s2 = pack2(scale, scale);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = decode2((j < 2 ? c.x : c.y) >> (16 * (j & 1)) & 0xffffu);
    const float2 y = unpack2(mul2(pack2(x.x, x.y), s2));
    m[2 * j] = y.x;
    m[2 * j + 1] = y.y;
  }
}
__device__ __forceinline__ void decode_v(uint2 c, float scale, float (&v)[8]) {
  const f32x2 s2 = pack2(scale, scale);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = decode2((j < 2 ? c.x : c.y) >> (16 * (j & 1)) & 0xffffu);
    const f32x2 r = mul2(pack2(x.x, x.y), s2);
    const float2 y = unpack2(mul2(r, r));
    v[2 * j] = y.x;
    v[2 * j + 1] = y.y;
  }
}

// The codes of a warp's block of 256 elements and its scales.  Lane's elements: index, index +
// step, ...; normal: all its v are positive and finite.
__device__ __forceinline__ void encode_block(const float (&m)[8], const float (&v)[8], const float (&u)[8],
                                             uint32_t index, uint32_t step, uint32_t seed, bool normal,
                                             uint2& cm, uint2& cv, float& ms, float& vs) {
  float mt = fabsf(m[0]);
  uint32_t vb = __float_as_uint(v[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) {
    mt = max_nan_abs(mt, m[j]);
    vb = max(vb, __float_as_uint(v[j]));
  }
  // non-negative floats order as their bits, a NaN above all; the root keeps the order
  float mtop = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mt) & 0x7fffffffu));
  float vtop = __fsqrt_rn(__uint_as_float(__reduce_max_sync(0xffffffffu, vb)));
  if (mtop < 0x1p-100f) mtop = 0.f;
  if (vtop < 0x1p-100f) vtop = 0.f;
  const float minv = mtop == 0.f ? 0.f : __fmul_rn(__frcp_rn(mtop), 448.0f);
  const float vinv = vtop == 0.f ? 0.f : __fmul_rn(__frcp_rn(vtop), 448.0f);
  ms = __fmul_rn(mtop, 1.0f / 448.0f);
  vs = __fmul_rn(vtop, 1.0f / 448.0f);
  const f32x2 mi = pack2(minv, minv), vi = pack2(vinv, vinv), down = pack2(0x1p-120f, 0x1p-120f);
  // The mix of index ^ seed begins with x ^ (x >> 16).  A lane's indexes in a row differ in
  // their low three bits only, which the shift does not reach.
  const uint32_t x0 = index ^ seed, y0 = x0 ^ (x0 >> 16);
  uint32_t wm[2], wv[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t tm[4], tv[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const int j = 4 * k + i;
      const float2 zm = unpack2(mul2(mul2(pack2(m[j], m[j + 1]), mi), down));
      const float2 zv = unpack2(mul2(mul2(pack2(u[j], u[j + 1]), vi), down));
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t y = y0 ^ (uint32_t)(j + e);
        if (step != 1) {
          const uint32_t x = (index + (j + e) * step) ^ seed;
          y = x ^ (x >> 16);
        }
        const uint32_t h = mix_end(y), hi = h >> 16;
        tm[i + e] = encode_bits(e ? zm.y : zm.x, (h ^ hi) & 0xffffu);
        tv[i + e] = encode_bits(e ? zv.y : zv.x, hi);
      }
    }
    uint32_t sign, none;
    wm[k] = code_bytes(tm, sign);
    wm[k] |= sign & nonzero_bytes(wm[k]);              // (zero has no sign)
    // a positive root is never stored as zero
    wv[k] = code_bytes(tv, none);
    uint32_t least = 0x01010101u;
    if (!normal) {
      least = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) least |= (u[4 * k + i] > 0.f ? 1u : 0u) << (8 * i);
    }
    if (vinv != 0.f) wv[k] |= least & ((nonzero_bytes(wv[k]) ^ 0x80808080u) >> 7);
  }
  cm = make_uint2(wm[0], wm[1]);
  cv = make_uint2(wv[0], wv[1]);
}

// One warp's block of 256 elements of any tensor: 16-byte accesses where the lane's eight
// elements lie together and are there, else element by element (every 32nd element a lane, so
// that the warp's accesses are consecutive).
template <bool PBF16, bool GBF16, bool MASTER, bool BITS8>
__device__ __forceinline__ void any_block(const Tensor& t, int64_t base, const Step& q, uint32_t seed) {
  const int lane = lane_id();
  const int64_t blk = base / kBlockElems;
  float msc = 0.f, vsc = 0.f;
  if constexpr (BITS8) { msc = t.ms[blk]; vsc = t.vs[blk]; }
  const int64_t first = t.vec ? base + 8 * lane : base + lane;
  const int step = t.vec ? 1 : 32;
  float m[8], v[8], u[8], w[8], g[8];
  bool normal = false;
  if (t.vec && first + 8 <= t.n) {
    const int64_t po = view_offset(t, first, t.ps);
    load8<GBF16>(t.g, view_offset(t, first, t.gs), g);
    if constexpr (MASTER) load8<false>(t.w, first, w);
    else load8<PBF16>(t.p, po, w);
    if constexpr (BITS8) {
      decode_m(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.m) + first), msc, m);
      decode_v(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.v) + first), vsc, v);
    } else {
      load8<false>(t.m, first, m);
      load8<false>(t.v, first, v);
    }
    normal = update8(q, g, m, v, u, w);
    if constexpr (MASTER) store8<false>(t.w, first, w);
    store8<PBF16>(t.p, po, w);
    if constexpr (!BITS8) {
      store8<false>(t.m, first, m);
      store8<false>(t.v, first, v);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t i = first + j * step;
      m[j] = v[j] = u[j] = 0.f;
      if (i >= t.n) continue;
      const int64_t po = view_offset(t, i, t.ps);
      const float gj = load_one<GBF16>(t.g, view_offset(t, i, t.gs));
      float wj;
      if constexpr (MASTER) wj = t.w[i];
      else wj = load_one<PBF16>(t.p, po);
      if constexpr (BITS8) {
        m[j] = __fmul_rn(decode2(static_cast<const uint8_t*>(t.m)[i]).x, msc);
        v[j] = __fmul_rn(decode2(static_cast<const uint8_t*>(t.v)[i]).x, vsc);
        v[j] = __fmul_rn(v[j], v[j]);
      } else {
        m[j] = static_cast<const float*>(t.m)[i];
        v[j] = static_cast<const float*>(t.v)[i];
      }
      moments(q, gj, m[j], v[j]);
      u[j] = __fsqrt_rn(v[j]);
      weight(q, m[j], u[j], wj);
      if constexpr (MASTER) t.w[i] = wj;
      store_one<PBF16>(t.p, po, wj);
      if constexpr (!BITS8) {
        static_cast<float*>(t.m)[i] = m[j];
        static_cast<float*>(t.v)[i] = v[j];
      }
    }
  }
  if constexpr (BITS8) {
    uint2 cm, cv;
    float ms, vs;
    encode_block(m, v, u, (uint32_t)first, (uint32_t)step, seed, normal, cm, cv, ms, vs);
    // (the codes' memory is whole blocks: no end to look at)
    uint8_t* dm = static_cast<uint8_t*>(t.m) + first;
    uint8_t* dv = static_cast<uint8_t*>(t.v) + first;
    if (t.vec) {
      *reinterpret_cast<uint2*>(dm) = cm;
      *reinterpret_cast<uint2*>(dv) = cv;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dm[32 * j] = (uint8_t)((j < 4 ? cm.x : cm.y) >> (8 * (j & 3)));
        dv[32 * j] = (uint8_t)((j < 4 ? cv.x : cv.y) >> (8 * (j & 3)));
      }
    }
    if (lane == 0) {
      t.ms[blk] = ms;
      t.vs[blk] = vs;
    }
  }
}

// Eight consecutive elements as they lie in memory.
template <bool BF16>
struct Raw8 {
  uint4 q[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* p) {
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) q[i] = static_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (BF16) {
      unpack8(q[0], x);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[4 * i] = __uint_as_float(q[i].x); x[4 * i + 1] = __uint_as_float(q[i].y);
        x[4 * i + 2] = __uint_as_float(q[i].z); x[4 * i + 3] = __uint_as_float(q[i].w);
      }
    }
  }
};

template <int NT, bool PBF16, bool GBF16, bool MASTER, bool BITS8>
__global__ void __launch_bounds__(kThreads, BITS8 ? 3 : 5) adamw_kernel(const __grid_constant__ AdamwArgs<NT> a) {
  pdl_begin();
  const int lane = lane_id();
  const long long t_step = a.step[0] + 1;
  const float lr = a.lr_dev != nullptr ? *a.lr_dev : a.lr;
  // 1 - b^t = -expm1(t ln b): relative accuracy even where b^t is near 1
  const float tf = (float)t_step;
  const Step q = {a.b1, a.b2, a.one_b1, a.one_b2, a.eps, a.grad_scale != nullptr ? *a.grad_scale : 1.0f,
                  lr / -expm1f(tf * a.ln_b1), 1.0f / sqrtf(-expm1f(tf * a.ln_b2)), 1.0f - lr * a.wd,
                  a.one};
  const uint32_t seed = mix32((uint32_t)t_step);
  const int n_chunks = a.chunk0[a.n], blocks = a.blocks;
  for (int c = blockIdx.x; c < n_chunks; c += gridDim.x) {
    int lo = 0, hi = a.n;                      // the chunk's tensor: chunk0[lo] <= c < chunk0[lo + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.chunk0[mid] <= c) lo = mid; else hi = mid;
    }
    const Tensor& t = a.t[lo];
    // this warp's `blocks` blocks of the chunk
    int64_t base = ((int64_t)(c - a.chunk0[lo]) * kWarps + warp_id()) * blocks * kBlockElems;
    int left = blocks;
    if (BITS8 && t.vec && t.d2 == 0) {
      const int64_t first = base + 8 * lane;
      // whole blocks among them
      const int64_t room = t.n - base - kBlockElems;
      int whole = room < 0 ? 0 : room >= (int64_t)(blocks - 1) * kBlockElems ? blocks : (int)(room / kBlockElems) + 1;
      uint8_t* pp = static_cast<uint8_t*>(t.p) + first * (PBF16 ? 2 : 4);
      const uint8_t* pg = static_cast<const uint8_t*>(t.g) + first * (GBF16 ? 2 : 4);
      float* pw = MASTER ? t.w + first : nullptr;
      uint8_t* pm = static_cast<uint8_t*>(t.m) + first;
      uint8_t* pv = static_cast<uint8_t*>(t.v) + first;
      // lane b holds the old, and after its turn the new, scales of block b
      const int64_t blk = base / kBlockElems + lane;
      float lms = 0.f, lvs = 0.f;
      if (lane < whole) {
        lms = t.ms[blk];
        lvs = t.vs[blk];
      }
      Raw8<GBF16> rg;
      Raw8<PBF16 && !MASTER> rw;
      uint2 rm, rv;
      const auto fetch = [&](int b) {
        const int i = b * kBlockElems;
        rg.load(pg + i * (GBF16 ? 2 : 4));
        if constexpr (MASTER) rw.load(pw + i);
        else rw.load(pp + i * (PBF16 ? 2 : 4));
        rm = *reinterpret_cast<const uint2*>(pm + i);
        rv = *reinterpret_cast<const uint2*>(pv + i);
      };
      if (whole > 0) fetch(0);
#pragma unroll 1
      for (int b = 0; b < whole; ++b) {
        const int i = b * kBlockElems;
        float m[8], v[8], u[8], w[8], g[8];
        rg.get(g);
        rw.get(w);
        decode_m(rm, __shfl_sync(0xffffffffu, lms, b), m);
        decode_v(rv, __shfl_sync(0xffffffffu, lvs, b), v);
        // the next block's bytes are on their way while this one is computed
        if (b + 1 < whole) fetch(b + 1);
        const bool normal = update8(q, g, m, v, u, w);
        if constexpr (MASTER) store8<false>(pw, i, w);
        store8<PBF16>(pp, i, w);
        uint2 cm, cv;
        float ms, vs;
        encode_block(m, v, u, (uint32_t)first + i, 1u, seed, normal, cm, cv, ms, vs);
        *reinterpret_cast<uint2*>(pm + i) = cm;
        *reinterpret_cast<uint2*>(pv + i) = cv;
        if (lane == b) {
          lms = ms;
          lvs = vs;
        }
      }
      if (lane < whole) {
        t.ms[blk] = lms;
        t.vs[blk] = lvs;
      }
      base += (int64_t)whole * kBlockElems;
      left -= whole;
    }
    for (; left > 0 && base < t.n; --left, base += kBlockElems)
      any_block<PBF16, GBF16, MASTER, BITS8>(t, base, q, seed);
  }
  if (a.advance) {
    // every block has read the step before it arrives; the last one moves it on
    __syncthreads();
    if (threadIdx.x == 0) {
      unsigned long long* arrived = reinterpret_cast<unsigned long long*>(a.step + 1);
      if (atomicAdd(arrived, 1ull) == gridDim.x - 1) {
        a.step[1] = 0;
        a.step[0] = t_step;
      }
    }
  }
}

// Tensors per launch: a short table for few (kernel parameters are copied at every launch),
// a long one that fills the 32764 bytes that a kernel's parameters may take.
constexpr int kShort = 16, kLong = 240;
static_assert(sizeof(AdamwArgs<kLong>) <= 32764, "kernel parameters");

template <int NT, bool P, bool G, bool M, bool B8>
cudaError_t launch(const moe_adamw_tensor_t* src, int n, const moe_adamw_config_t& c, const float* lr,
                   const float* gscale, int64_t* step, bool advance, cudaStream_t s) {
  AdamwArgs<NT> a;
  // 8 bits: resident thread blocks that walk chunks of up to 32 blocks a warp, since a chunk's
  // first block waits for its bytes (eight layers' adapters, 206 us: 16 blocks a warp 6 us more than
  // 32, 8 blocks 21 us more); the length evens out the chunks per thread block.  Not longer than an
  // average tensor, nor than keeps every SM busy.  32 bits: one block a warp and a thread block
  // for every chunk up to 64 per SM (bound by HBM: 57 us for one layer with master weights, 98% of
  // the measured copy bandwidth; 6 us more as a loop over longer chunks).
  const int64_t resident = (int64_t)device_sms() * (B8 ? 3 : 64);
  int64_t blocks = 0;
  for (int i = 0; i < n; ++i)
    blocks += (src[i].size[0] * src[i].size[1] * src[i].size[2] + kBlockElems - 1) / kBlockElems;
  int64_t run = 1;
  if (B8 && n > 0) {
    const int64_t each = (blocks + resident * kWarps - 1) / (resident * kWarps);   // blocks per warp in all
    const int64_t rounds = (each + kMaxRun - 1) / kMaxRun;
    run = rounds > 0 ? (each + rounds - 1) / rounds : 1;
    const int64_t most = blocks / (kWarps * (int64_t)n);
    run = run < most ? run : most;
    run = run < 1 ? 1 : run;
  }
  a.blocks = (int)run;
  const int64_t per = (int64_t)kChunk * run;
  int64_t chunks = 0;
  for (int i = 0; i < n; ++i) {
    const moe_adamw_tensor_t& t = src[i];
    Tensor& d = a.t[i];
    d.p = t.param; d.g = t.grad; d.w = t.master; d.m = t.exp_avg; d.v = t.exp_avg_sq;
    d.ms = t.exp_avg_scale; d.vs = t.exp_avg_sq_scale;
    d.n = t.size[0] * t.size[1] * t.size[2];
    const bool flat = t.size[0] == 1 && t.size[1] == 1 && t.param_stride[2] == 1 && t.grad_stride[2] == 1;
    d.d1 = (uint32_t)t.size[1];
    d.d2 = flat ? 0u : (uint32_t)t.size[2];
    for (int k = 0; k < 3; ++k) { d.ps[k] = t.param_stride[k]; d.gs[k] = t.grad_stride[k]; }
    // 16-byte accesses to groups of eight: aligned bases, and in a strided view rows of whole
    // groups that begin aligned
    const int pe = P ? 8 : 4, ge = G ? 8 : 4;             // elements in 16 bytes
    d.vec = aligned16(t.param) && aligned16(t.grad) &&
            (flat || (t.size[2] % 8 == 0 && t.param_stride[2] == 1 && t.grad_stride[2] == 1 &&
                      t.param_stride[0] % pe == 0 && t.param_stride[1] % pe == 0 &&
                      t.grad_stride[0] % ge == 0 && t.grad_stride[1] % ge == 0));
    a.chunk0[i] = (int32_t)chunks;
    chunks += (d.n + per - 1) / per;
  }
  if (chunks >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  a.chunk0[n] = (int32_t)chunks;
  a.n = n;
  a.lr = (float)c.lr; a.b1 = (float)c.beta1; a.b2 = (float)c.beta2; a.eps = (float)c.eps;
  a.wd = (float)c.weight_decay;
  a.one_b1 = (float)(1.0 - c.beta1); a.one_b2 = (float)(1.0 - c.beta2);
  a.one = 1.0f;
  a.ln_b1 = (float)std::log(c.beta1); a.ln_b2 = (float)std::log(c.beta2);
  a.lr_dev = lr; a.grad_scale = gscale;
  a.step = reinterpret_cast<long long*>(step);
  a.advance = advance ? 1 : 0;
  const unsigned grid = (unsigned)(chunks < 1 ? 1 : chunks < resident ? chunks : resident);
  ProfScope ps(K_ADAMW, s);
  return launch_pdl(adamw_kernel<NT, P, G, M, B8>, dim3(grid), dim3(kThreads), 0, s, 1, a);
}

template <bool P, bool G, bool M, bool B8>
cudaError_t launch_all(const moe_adamw_tensor_t* src, int n, const moe_adamw_config_t& c, const float* lr,
                       const float* gscale, int64_t* step, bool advance, cudaStream_t s) {
  for (int i = 0; i == 0 || i < n; i += kLong) {
    const int k = n - i < kLong ? n - i : kLong;
    const bool last = advance && i + kLong >= n;
    const cudaError_t e = k <= kShort ? launch<kShort, P, G, M, B8>(src + i, k, c, lr, gscale, step, last, s)
                                      : launch<kLong, P, G, M, B8>(src + i, k, c, lr, gscale, step, last, s);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

// Whether two elements of the parameter may lie in one place (they would race): a dimension that steps
// inside the reach of those of smaller strides.
bool places_meet(const moe_adamw_tensor_t& t) {
  int by[3] = {0, 1, 2};
  std::sort(by, by + 3, [&](int a, int b) { return t.param_stride[a] < t.param_stride[b]; });
  int64_t reach = 1;
  for (int k : by) {
    if (t.size[k] <= 1) continue;
    if (t.param_stride[k] < reach) return true;
    // (a stride beyond what any memory holds ends the sum before it can overflow)
    if (t.param_stride[k] > (int64_t(1) << 60) / t.size[k]) return false;
    reach += t.param_stride[k] * (t.size[k] - 1);
  }
  return false;
}

bool aligned_to(const void* p, size_t a) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_adamw_step(const moe_adamw_tensor_t* tensors, int32_t n_tensors,
                                       const moe_adamw_config_t* cfg, const float* lr,
                                       const float* grad_scale, int64_t* step, int32_t advance,
                                       void* stream) {
  NvtxRange nr("moe_adamw_step");
  if (cfg == nullptr || n_tensors < 0 || (n_tensors > 0 && tensors == nullptr)) return MOE_ERR_INVALID_ARG;
  const moe_adamw_config_t& c = *cfg;
  if (!std::isfinite(c.lr) || !std::isfinite(c.weight_decay) || !(c.eps >= 0) || !std::isfinite(c.eps) ||
      !(c.beta1 >= 0 && c.beta1 < 1) || !(c.beta2 >= 0 && c.beta2 < 1))
    return MOE_ERR_INVALID_ARG;
  // (the quotient's reciprocal takes a subnormal divisor for zero: 0 / eps would be no number)
  if (c.eps > 0 && c.eps < 0x1p-126) return MOE_ERR_INVALID_ARG;
  if (c.state_bits != 8 && c.state_bits != 32) return MOE_ERR_UNSUPPORTED;
  const bool p16 = c.param_bf16 != 0, g16 = c.grad_bf16 != 0, master = c.has_master != 0, b8 = c.state_bits == 8;
  if (master && !p16) return MOE_ERR_UNSUPPORTED;
  if (!aligned16(step)) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < n_tensors; ++i) {
    const moe_adamw_tensor_t& t = tensors[i];
    int64_t n = 1;
    for (int k = 0; k < 3; ++k) {
      if (t.size[k] < 0 || t.param_stride[k] < 0 || t.grad_stride[k] < 0) return MOE_ERR_INVALID_ARG;
      if (t.size[k] > (int64_t(1) << 40) || n > (int64_t(1) << 40)) return MOE_ERR_UNSUPPORTED;
      n *= t.size[k];
    }
    if (n == 0) continue;
    if (n > (int64_t(1) << 40)) return MOE_ERR_UNSUPPORTED;
    if (places_meet(t)) return MOE_ERR_INVALID_ARG;
    const bool flat = t.size[0] == 1 && t.size[1] == 1 && t.param_stride[2] == 1 && t.grad_stride[2] == 1;
    if (!flat && n >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
    if (!aligned_to(t.param, p16 ? 2 : 4) || !aligned_to(t.grad, g16 ? 2 : 4)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(t.exp_avg) || !aligned16(t.exp_avg_sq)) return MOE_ERR_INVALID_ARG;
    if (b8 && (!aligned_to(t.exp_avg_scale, 4) || !aligned_to(t.exp_avg_sq_scale, 4))) return MOE_ERR_INVALID_ARG;
    if (master && !aligned16(t.master)) return MOE_ERR_INVALID_ARG;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool adv = advance != 0;
#define MOE_ADAMW(P, G, M) \
  (b8 ? launch_all<P, G, M, true>(tensors, n_tensors, c, lr, grad_scale, step, adv, s) \
      : launch_all<P, G, M, false>(tensors, n_tensors, c, lr, grad_scale, step, adv, s))
  cudaError_t e;
  if (p16 && master) e = g16 ? MOE_ADAMW(true, true, true) : MOE_ADAMW(true, false, true);
  else if (p16) e = g16 ? MOE_ADAMW(true, true, false) : MOE_ADAMW(true, false, false);
  else e = g16 ? MOE_ADAMW(false, true, false) : MOE_ADAMW(false, false, false);
#undef MOE_ADAMW
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
