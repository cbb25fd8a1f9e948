// AdamW over many tensors in one launch, states in 32 or 8 bits (the formula and
// the order of its fp32 operations stand in dictproj.h).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "dictproj_internal.h"
#include "kernels.h"

namespace dictproj {
namespace {

constexpr int kBlock = DICTPROJ_ADAMW_BLOCK;
constexpr float kTinyScale = 0x1p-126f;
constexpr float kScalePerAmax = 1.f / 448.f;

__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_f32x2(uint32_t two) {
  const uint32_t h = e4m3x2_to_f16x2(two);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// x / s for many x and one s, correctly rounded. Markstein (1990): with y the correctly
// rounded 1 / s, q = x y and q + y (x - q s), the residual by fma, is the rounded
// quotient as long as the residual is exact. With 2^-90 <= s <= 2^100 that holds for every
// quotient from 2^-11 on: the residual is a multiple of ulp(q) ulp(s) >= 2^-34 2^-113 = 2^-147.
// A smaller quotient, right in its last bit or not, is code 0 for m (2^-10 is half the smallest
// code) and code 1 for r > 0 (its bits are below 2^18 and the dither's below 2^20: 0 or 1, and r > 0
// has at least 1). Other scales (a block of zeros, of overflowing moments) divide.
struct Divisor {
  float s, y;
  bool fast;
};
__device__ __forceinline__ Divisor divisor(float s) {
  return Divisor{s, __fdiv_rn(1.f, s), s >= 0x1p-90f && s <= 0x1p100f};
}
template <bool FAST>
__device__ __forceinline__ float quotient(float x, const Divisor& d) {
  if (!FAST) return __fdiv_rn(x, d.s);
  const float q = __fmul_rn(x, d.y);
  return __fmaf_rn(__fmaf_rn(-q, d.s, x), d.y, q);
}

__device__ __forceinline__ uint32_t dither20(uint32_t i, uint32_t step) {
  uint32_t h = i * 0x9E3779B9u + step * 0x6A09E667u;
  h ^= h >> 16;
  h *= 0xBB67AE85u;
  h ^= h >> 15;
  h *= 0x6A09E667u;
  return h >> 12;
}

struct Updated {
  float p, m, v, r;
};
// Every operation is rounded on its own (no contraction to fma), so that the
// result is the formula's in any implementation of it.
__device__ __forceinline__ Updated adamw_element(float p, float grad, float m, float v, const AdamwFactors& f) {
  Updated u;
  const float g = __fmul_rn(grad, f.grad_scale);
  u.m = __fadd_rn(__fmul_rn(m, f.b1), __fmul_rn(g, f.omb1));
  u.v = __fadd_rn(__fmul_rn(v, f.b2), __fmul_rn(__fmul_rn(g, f.omb2), g));
  u.r = __fsqrt_rn(u.v);
  const float d = __fadd_rn(__fmul_rn(u.r, f.rbc2), f.eps);
  u.p = __fsub_rn(__fmul_rn(p, f.decay), __fmul_rn(__fdiv_rn(u.m, d), f.alpha));
  return u;
}

// The scale of a block from a lane's four values: amax / 448, at least kTinyScale. Magnitudes
// order as their bits do, a NaN above the infinities, so that it is the maximum and the scale.
__device__ __forceinline__ float block_scale(float a, float b, float c, float d) {
  const uint32_t m = max(max(__float_as_uint(fabsf(a)), __float_as_uint(fabsf(b))), max(__float_as_uint(fabsf(c)), __float_as_uint(fabsf(d))));
  const float s = __fmul_rn(__uint_as_float(__reduce_max_sync(0xffffffffu, m)), kScalePerAmax);
  return s < kTinyScale ? kTinyScale : s;
}

// Four consecutive values of a lane, zeros past n; one load where the arrays allow it.
// MODE 2: a whole chunk of aligned arrays; 1: aligned, with a ragged end; 0: neither.
template <int MODE, class V, class E>
__device__ __forceinline__ V load4(const E* p, int i, int n) {
  V v = {};
  if (MODE == 2 || (MODE == 1 && i + 4 <= n)) return *reinterpret_cast<const V*>(p + i);
  E* e = reinterpret_cast<E*>(&v);
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (i + q < n) e[q] = p[i + q];
  return v;
}
template <int MODE, class V, class E>
__device__ __forceinline__ void store4(E* p, int i, int n, V v) {
  if (MODE == 2 || (MODE == 1 && i + 4 <= n)) {
    *reinterpret_cast<V*>(p + i) = v;
    return;
  }
  const E* e = reinterpret_cast<const E*>(&v);
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (i + q < n) p[i + q] = e[q];
}

// The codes of four elements of one block.
template <bool FAST>
__device__ __forceinline__ uint2 encode4(const Updated (&u)[4], const Divisor& dm, const Divisor& dr, uint32_t first, uint32_t step) {
  uint2 c;
  c.x = f32x2_to_e4m3x2(quotient<FAST>(u[0].m, dm), quotient<FAST>(u[1].m, dm)) |
        f32x2_to_e4m3x2(quotient<FAST>(u[2].m, dm), quotient<FAST>(u[3].m, dm)) << 16;
  c.y = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t code = (__float_as_uint(__fmul_rn(quotient<FAST>(u[q].r, dr), 0x1p-120f)) + dither20(first + (uint32_t)q, step)) >> 20;
    code = max(min(code, 0x7Eu), u[q].r > 0.f ? 1u : 0u);
    c.y |= code << (8 * q);
  }
  return c;
}

// A warp takes a block of 128 at a time, four elements a lane.
template <int BITS, int MODE>
__device__ __forceinline__ void adamw_chunk(const AdamwChunk& c, const AdamwFactors& f) {
  constexpr int kPer = kAdamwChunk / kBlock / 8;  // blocks of a warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = (int)c.count;
  float4 p[kPer], g[kPer], m[kPer], v[kPer];
  uint32_t mc[kPer], vc[kPer];
  float sm[kPer], sr[kPer];
#pragma unroll
  for (int b = 0; b < kPer; ++b) {  // all loads first
    const int blk = warp + 8 * b, i = blk * kBlock + 4 * lane;
    p[b] = load4<MODE, float4>(c.p, i, n);
    g[b] = load4<MODE, float4>(c.g, i, n);
    if (BITS == 8) {
      mc[b] = load4<MODE, uint32_t>(static_cast<const uint8_t*>(c.m), i, n);
      vc[b] = load4<MODE, uint32_t>(static_cast<const uint8_t*>(c.v), i, n);
      sm[b] = MODE == 2 || blk * kBlock < n ? c.m_scale[blk] : 0.f;
      sr[b] = MODE == 2 || blk * kBlock < n ? c.v_scale[blk] : 0.f;
    } else {
      m[b] = load4<MODE, float4>(static_cast<const float*>(c.m), i, n);
      v[b] = load4<MODE, float4>(static_cast<const float*>(c.v), i, n);
    }
  }
#pragma unroll
  for (int b = 0; b < kPer; ++b) {
    const int blk = warp + 8 * b, i = blk * kBlock + 4 * lane;
    if (MODE < 2 && blk * kBlock >= n) break;
    if (BITS == 8) {
      const float2 m0 = e4m3x2_to_f32x2(mc[b]), m1 = e4m3x2_to_f32x2(mc[b] >> 16);
      const float2 r0 = e4m3x2_to_f32x2(vc[b]), r1 = e4m3x2_to_f32x2(vc[b] >> 16);
      m[b] = make_float4(__fmul_rn(m0.x, sm[b]), __fmul_rn(m0.y, sm[b]), __fmul_rn(m1.x, sm[b]), __fmul_rn(m1.y, sm[b]));
      const float x = __fmul_rn(r0.x, sr[b]), y = __fmul_rn(r0.y, sr[b]), z = __fmul_rn(r1.x, sr[b]), w = __fmul_rn(r1.y, sr[b]);
      v[b] = make_float4(__fmul_rn(x, x), __fmul_rn(y, y), __fmul_rn(z, z), __fmul_rn(w, w));
    }
    const Updated u[4] = {adamw_element(p[b].x, g[b].x, m[b].x, v[b].x, f), adamw_element(p[b].y, g[b].y, m[b].y, v[b].y, f),
                          adamw_element(p[b].z, g[b].z, m[b].z, v[b].z, f), adamw_element(p[b].w, g[b].w, m[b].w, v[b].w, f)};
    store4<MODE>(c.p, i, n, make_float4(u[0].p, u[1].p, u[2].p, u[3].p));
    if (c.copy) {
      const __half2 lo = __floats2half2_rn(u[0].p, u[1].p), hi = __floats2half2_rn(u[2].p, u[3].p);
      store4<MODE>(reinterpret_cast<unsigned short*>(c.copy), i, n,
                  make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi)));
    }
    if (BITS == 32) {
      store4<MODE>(static_cast<float*>(c.m), i, n, make_float4(u[0].m, u[1].m, u[2].m, u[3].m));
      store4<MODE>(static_cast<float*>(c.v), i, n, make_float4(u[0].v, u[1].v, u[2].v, u[3].v));
      continue;
    }
    // past n nothing decides a scale (a zero code times a scale that is not finite would)
    const int left = MODE == 2 ? 4 : n - i;
    const Divisor dm = divisor(block_scale(left > 0 ? u[0].m : 0.f, left > 1 ? u[1].m : 0.f, left > 2 ? u[2].m : 0.f, left > 3 ? u[3].m : 0.f));
    const Divisor dr = divisor(block_scale(left > 0 ? u[0].r : 0.f, left > 1 ? u[1].r : 0.f, left > 2 ? u[2].r : 0.f, left > 3 ? u[3].r : 0.f));
    if (lane == 0) {
      c.m_scale[blk] = dm.s;
      c.v_scale[blk] = dr.s;
    }
    const uint32_t e = c.first + (uint32_t)i;
    const uint2 codes = dm.fast && dr.fast ? encode4<true>(u, dm, dr, e, f.step) : encode4<false>(u, dm, dr, e, f.step);
    store4<MODE>(static_cast<uint8_t*>(c.m), i, n, codes.x);
    store4<MODE>(static_cast<uint8_t*>(c.v), i, n, codes.y);
  }
}

// One CTA per chunk; its record holds the pointers, so that the data is one load away.
// Bound by the bytes (30 a weight with 32-bit states, 18 with 8-bit ones) as long as the
// arithmetic of an 8-bit step, some 80 instructions a weight, hides behind them: five
// CTAs an SM (48 registers) measured 136 us for 44 M weights (5.9 TB/s), four 149 us, six
// (40 registers, spills) 150 us; divisions by the compiler's sequence and maxima by
// shuffles 177 us. With 32-bit states the registers serve loads in flight instead
// (14 tensors of 65536: 4.2 us without a limit, 4.9 us at 48).
template <int BITS>
__global__ void __launch_bounds__(256, BITS == 8 ? 5 : 1) k_adamw(const AdamwChunk* __restrict__ chunks, AdamwFactors f) {
  grid_dependency_wait();
  trigger_dependents();
  const AdamwChunk c = chunks[blockIdx.x];
  if (c.vec && c.count == kAdamwChunk) adamw_chunk<BITS, 2>(c, f);
  else if (c.vec) adamw_chunk<BITS, 1>(c, f);
  else adamw_chunk<BITS, 0>(c, f);
}

}  // namespace

cudaError_t launch_adamw(const dictproj_adamw* w, const AdamwFactors& f, cudaStream_t stream) {
  if (w->chunks == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)w->chunks);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  AdamwFactors ff = f;
  void* args[] = {(void*)&w->table, &ff};
  return cudaLaunchKernelExC(&cfg, w->bits == 8 ? (const void*)k_adamw<8> : (const void*)k_adamw<32>, args);
}

}  // namespace dictproj
