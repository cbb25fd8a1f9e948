// What the adapter kernels share: arguments, T's two parts, distributed shared memory.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "dictproj_internal.h"

namespace dictproj {

constexpr int kFewRows = 4, kWideRows = 64, kTallRows = 128;  // rows of a tile
constexpr int kGradCols = 128;                                // columns of a weight gradient's CTA

struct RowsPass {
  const __half* in;
  const __half* P;
  const __half* Q;
  const __half* base;
  __half* out;
  // many rows: the two parts of scale * T, [tile][kWideRows][rp], zeros past a tile's
  // rows, and what the parts of a tile are multiplied with
  __half* hi;
  __half* lo;
  float* unit;
  int K, N, ld_p, ld_q;
};
struct RowsArgs {
  RowsPass pass[2];
  const int* n_tiles;
  const int4* tiles;
  const int* perm;
  const int* rank;
  const float* scale;
  int rp, n_slots, rows, cluster;
};

struct GradPass {
  const __half* in;
  const __half* hi;
  const __half* lo;
  const float* unit;
  float* g;
  int K, blocks;
};
struct GradArgs {
  GradPass pass[2];
  const int* start;
  const int* first64;
  const int* perm;
  const int* rank;
  int rp, max_rank, accumulate, n_rows;
};

// ---- clusters and distributed shared memory
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t peer_smem(uint32_t local, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_peer_v4f(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_peer_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_peer_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ uint32_t half2_bits(__half a, __half b) {
  const __half2 h = __halves2half2(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// T in two fp16 parts: t * unit = high + low with |t * unit| < 2^14, so that the two
// together keep 22 bits of it, or 2^-24 absolute (2^-38 of the tile's largest): the
// MMA's fp16 operands then carry T as exactly as the fp32 sums that made it, whatever
// its size. unit is a power of two.
struct Split {
  __half hi, lo;
};
__device__ __forceinline__ Split split_half(float t) {
  Split s;
  s.hi = __float2half_rn(t);
  s.lo = __hisinf(s.hi) ? __float2half_rn(0.f) : __float2half_rn(t - __half2float(s.hi));
  return s;
}
// 2^13 / 2^floor(log2 m), within fp32's normal range; 1 for m = 0.
__device__ __forceinline__ float split_unit(float m) {
  if (m == 0.f) return 1.f;
  const int e = (int)((__float_as_uint(m) >> 23) & 255) - 127;  // -127 for a subnormal
  return __uint_as_float((uint32_t)(min(13 - e, 126) + 127) << 23);
}

// Largest of the warp's finite non-negative values.
__device__ __forceinline__ float warp_max_bits(float m) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
}

}  // namespace dictproj
