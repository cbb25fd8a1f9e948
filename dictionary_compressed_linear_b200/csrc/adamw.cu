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

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int off = 16; off; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

// One CTA per chunk of kAdamwChunk elements; a warp takes a block of 128 at a time.
template <int BITS>
__global__ void __launch_bounds__(256)
    k_adamw(const dictproj_adamw_tensor* __restrict__ tensors, const long long* __restrict__ first, int n_tensors,
            AdamwFactors f) {
  grid_dependency_wait();
  const long long c = blockIdx.x;
  int lo = 0, hi = n_tensors - 1;  // the last tensor whose first chunk is <= c (an empty tensor owns none)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  const dictproj_adamw_tensor T = tensors[lo];
  const long long e0 = (c - first[lo]) * kAdamwChunk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __half* copy = static_cast<__half*>(T.copy);
  for (int b = warp; b < kAdamwChunk / kBlock; b += 8) {
    const long long base = e0 + (long long)b * kBlock;
    if (base >= T.n) break;
    float sm = 0.f, sr = 0.f;
    if (BITS == 8) {
      sm = T.m_scale[base / kBlock];
      sr = T.v_scale[base / kBlock];
    }
    Updated u[4];
    float am = 0.f, ar = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const long long i = base + 32 * q + lane;
      u[q] = Updated{0.f, 0.f, 0.f, 0.f};
      if (i < T.n) {
        float m, v;
        if (BITS == 8) {
          m = __fmul_rn(e4m3_to_f32(static_cast<const uint8_t*>(T.m)[i]), sm);
          const float r = __fmul_rn(e4m3_to_f32(static_cast<const uint8_t*>(T.v)[i]), sr);
          v = __fmul_rn(r, r);
        } else {
          m = static_cast<const float*>(T.m)[i];
          v = static_cast<const float*>(T.v)[i];
        }
        u[q] = adamw_element(T.p[i], T.g[i], m, v, f);
        T.p[i] = u[q].p;
        if (copy) copy[i] = __float2half_rn(u[q].p);
        if (BITS == 32) {
          static_cast<float*>(T.m)[i] = u[q].m;
          static_cast<float*>(T.v)[i] = u[q].v;
        }
        am = fmaxf(am, fabsf(u[q].m));
        ar = fmaxf(ar, u[q].r);
      }
    }
    if (BITS == 8) {
      sm = fmaxf(__fmul_rn(warp_max(am), kScalePerAmax), kTinyScale);
      sr = fmaxf(__fmul_rn(warp_max(ar), kScalePerAmax), kTinyScale);
      if (lane == 0) {
        T.m_scale[base / kBlock] = sm;
        T.v_scale[base / kBlock] = sr;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const long long i = base + 32 * q + lane;
        if (i >= T.n) continue;
        static_cast<uint8_t*>(T.m)[i] = (uint8_t)f32x2_to_e4m3x2(__fdiv_rn(u[q].m, sm), 0.f);
        uint32_t code = (__float_as_uint(__fmul_rn(__fdiv_rn(u[q].r, sr), 0x1p-120f)) + dither20((uint32_t)i, f.step)) >> 20;
        code = min(code, 0x7Eu);
        if (u[q].r > 0.f) code = max(code, 1u);
        static_cast<uint8_t*>(T.v)[i] = (uint8_t)code;
      }
    }
  }
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
  int n = w->n_tensors;
  AdamwFactors ff = f;
  void* args[] = {(void*)&w->tensors, (void*)&w->first, &n, &ff};
  return cudaLaunchKernelExC(&cfg, w->bits == 8 ? (const void*)k_adamw<8> : (const void*)k_adamw<32>, args);
}

}  // namespace dictproj
