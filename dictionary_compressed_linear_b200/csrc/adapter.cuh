// What the adapter kernels share: arguments, T's two parts, distributed shared memory.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "dictproj_internal.h"

namespace dictproj {

constexpr int kFewRows = 4, kWideRows = 64, kTallRows = 128;  // rows of a tile
constexpr int kCrowd = 32;  // a slot of more rows is a crowd: its tiles carry kCrowdTile with their row count
constexpr int kCrowdTile = 1 << 16;
constexpr int kGradCols = 128;                                // columns of a weight gradient's CTA

struct RowsPass {
  const __half* in;
  const __half* P;
  const __half* Q;
  const __half* base;
  __half* out;
  // many rows: scale * T in two parts, [64-row tile][kWideRows][high pp | low pp], zeros past a
  // tile's rows, and what the parts are multiplied with: for the expansion, which sums over the
  // ranks, a number for each row; for the weight gradients, which sum over the rows, one for each
  // tile and rank ([tile][pp]). Null: not wanted.
  __half* parts;
  float* unit;
  __half* gparts;
  float* gunit;
  float* sums;  // few rows, backward: scale * T in plan order, [rows][pp], or null
  int K, N, ld_p, ld_q;
};
struct RowsArgs {
  RowsPass pass[2];
  const int* n_tiles;
  const int* planned;  // the plan's rows, on the device
  const int4* tiles;
  const int* runs;  // 128-row tiles: the first row of a tile whose rows follow one another, else -1
  const int* perm;
  const int* rank;
  const float* scale;
  int rp, pp, n_slots, rows, cluster;
  int only;  // -1: every tile; 0: no crowds' tiles; 1: crowds' tiles alone
};

struct GradPass {
  const __half* in;
  const __half* parts;
  const float* unit;
  const float* sums;  // few rows
  float* g;
  int K, blocks;
};
struct GradArgs {
  GradPass pass[2];
  const int* start;
  const int* first64;
  const int* runs;  // of the 64-row tiles
  const int* perm;
  const int* rank;
  const int* used;    // the slots that have rows
  const int* n_used;
  const int* planned;
  int rp, pp, max_rank, accumulate, n_rows;
  int zeroed;         // several slots: those without rows or rank are zeroed by a launch of their own
};

// The slot of a gradient CTA (blockIdx.y counts the slots that have rows), -1: none.
__device__ __forceinline__ int grad_slot(const GradArgs& g) {
  if (__ldcg(g.planned) > g.n_rows) return -1;
  if (!g.zeroed) return blockIdx.y;
  return (int)blockIdx.y < __ldcg(g.n_used) ? __ldcg(g.used + blockIdx.y) : -1;
}

// Kernels that start before the launch ahead of them has ended read what was there before
// the call through L2 (__ldcg, cp.async.cg, TMA): a line of an earlier launch that an SM's L1
// may still hold is not what they want.

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
// Four floats of every CTA of the cluster, summed in rank order (the loads go out together).
__device__ __forceinline__ float4 sum_peers(uint32_t local, int cluster) {
  float4 v[8];
#pragma unroll
  for (int c = 0; c < 8; ++c)
    if (c < cluster) v[c] = ld_peer_v4f(peer_smem(local, c));
#pragma unroll
  for (int c = 1; c < 8; ++c)
    if (c < cluster) v[0].x += v[c].x, v[0].y += v[c].y, v[0].z += v[c].z, v[0].w += v[c].w;
  return v[0];
}
__device__ __forceinline__ void st_peer_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t half2_bits(__half a, __half b) {
  const __half2 h = __halves2half2(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// T in two fp16 parts: t * unit = high + low, unit a power of two that brings the largest
// of the values it serves (a row's, or a rank's in a tile) to 2^13 or more, below 2^14. The
// two parts keep 22 bits of a value down to 2^-16 of that largest one; below, what they
// leave out is at most 2^-38 of the largest (half of fp16's smallest step, 2^-25, of 2^13).
// With one unit for all of a tile, rows or ranks 2^-26 below the largest kept 12 bits.
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

// Rows of a length that is no multiple of 8 start at any even byte. Eight elements from
// `src` are then two aligned 16-byte loads and a shift, as long as both lie inside the array
// (which ends at `end`).
__device__ __forceinline__ const uint4* window_of(const __half* src) {
  return reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(src) & ~(uintptr_t)15);
}
__device__ __forceinline__ bool window_inside(const __half* src, const __half* end) {
  return reinterpret_cast<uintptr_t>(window_of(src) + 2) <= reinterpret_cast<uintptr_t>(end);
}
// The first `left` of the eight elements, zeros behind them.
__device__ __forceinline__ uint4 shift_window(const uint4& a, const uint4& b, const __half* src, int left) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(src);
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  const uint32_t words = (uint32_t)(at >> 2) & 3u, shift = 8u * ((uint32_t)at & 2u);
  if (words & 2) w[0] = w[2], w[1] = w[3], w[2] = w[4], w[3] = w[5], w[4] = w[6], w[5] = w[7];
  if (words & 1) w[0] = w[1], w[1] = w[2], w[2] = w[3], w[3] = w[4], w[4] = w[5];
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = __funnelshift_r(w[i], w[i + 1], shift) & (left >= 2 * i + 2 ? 0xFFFFFFFFu : left == 2 * i + 1 ? 0xFFFFu : 0u);
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ uint4 single_elements(const __half* src, int left) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned short* h = reinterpret_cast<const unsigned short*>(src) + 2 * i;
    const unsigned short a = 2 * i < left ? __ldcg(h) : 0, b = 2 * i + 1 < left ? __ldcg(h + 1) : 0;
    w[i] = (uint32_t)a | ((uint32_t)b << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// 8 elements from column c of a row of n elements, zeros past the end (vec: n % 8 == 0).
__device__ __forceinline__ uint4 read_piece(const __half* row, int c, int n, bool vec, const __half* end) {
  if (vec) return c < n ? __ldcg(reinterpret_cast<const uint4*>(row + c)) : make_uint4(0, 0, 0, 0);
  if (!window_inside(row + c, end)) return single_elements(row + c, n - c);
  const uint4* q = window_of(row + c);
  return shift_window(__ldcg(q), __ldcg(q + 1), row + c, n - c);
}
// The same column of several unaligned rows (in: whether a row is wanted), all loads
// together: one after the other they took 2 us a stage.
template <int N>
__device__ __forceinline__ void read_pieces(uint4 (&out)[N], const __half* const (&row)[N], const bool (&in)[N], int c, int n,
                                            const __half* end) {
  bool all = true;
#pragma unroll
  for (int i = 0; i < N; ++i) all = all && (!in[i] || window_inside(row[i] + c, end));
  if (all) {
    uint4 a[N], b[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      a[i] = b[i] = make_uint4(0, 0, 0, 0);
      if (in[i]) {
        a[i] = __ldcg(window_of(row[i] + c));
        b[i] = __ldcg(window_of(row[i] + c) + 1);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = shift_window(a[i], b[i], row[i] + c, in[i] ? n - c : 0);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = in[i] ? read_piece(row[i], c, n, false, end) : make_uint4(0, 0, 0, 0);
  }
}
__device__ __forceinline__ void write_piece(__half* row, int c, int n, bool vec, const uint4& v) {
  if (vec) {
    if (c < n) *reinterpret_cast<uint4*>(row + c) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (c + 8 <= n) {
    unsigned short* h = reinterpret_cast<unsigned short*>(row + c);
    if ((reinterpret_cast<uintptr_t>(h) & 2) == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t*>(h)[i] = w[i];
    } else {
      h[0] = (unsigned short)w[0];
#pragma unroll
      for (int i = 0; i < 3; ++i) *reinterpret_cast<uint32_t*>(h + 1 + 2 * i) = __funnelshift_r(w[i], w[i + 1], 16);
      h[7] = (unsigned short)(w[3] >> 16);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + e < n) row[c + e] = __ushort_as_half((unsigned short)(w[e >> 1] >> (16 * (e & 1))));
}

// base alone, for rows without an adapter: pieces [lo, hi) of the columns
__device__ __forceinline__ void copy_rows(const RowsPass& a, int n_rows, const int* rows, int count, int lo, int hi) {
  const bool vec = (a.N & 7) == 0;
  const int n = hi - lo;
  for (int i = threadIdx.x; i < count * n; i += blockDim.x) {
    const size_t at = (size_t)rows[i / n] * a.N;
    const int c = 8 * (lo + i % n);
    write_piece(a.out + at, c, a.N, vec, a.base ? read_piece(a.base + at, c, a.N, vec, a.base + (size_t)n_rows * a.N) : make_uint4(0, 0, 0, 0));
  }
}

// Whether a launch is to take a tile (slots' and, unless the output is in place, those of
// rows without an adapter). A captured call may meet a plan of more rows than it was made
// for, whose row numbers reach past its arrays: it takes none of them.
__device__ __forceinline__ bool takes_tile(const RowsArgs& g, int tile_no, const int4& tile, bool in_place) {
  return __ldcg(g.planned) <= g.rows && tile_no < __ldcg(g.n_tiles + (in_place ? 0 : 1)) && (g.only < 0 || g.only == (tile.z >= kCrowdTile ? 1 : 0));
}

// Zeros over `width` columns of rows [0, n) of a gradient, shared by `parts` CTAs.
__device__ __forceinline__ void zero_columns(float* out, int K, int width, int n, int part, int parts) {
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const bool vec = (K & 3) == 0 && (width & 3) == 0;
  for (int j = part * warps + warp; j < n; j += parts * warps) {
    float* row = out + (size_t)j * K;
    if (vec)
      for (int c = 4 * lane; c < width; c += 128) *reinterpret_cast<float4*>(row + c) = make_float4(0.f, 0.f, 0.f, 0.f);
    else
      for (int c = lane; c < width; c += 32) row[c] = 0.f;
  }
}

// The magnitude's bits, which order as it does; an infinity or NaN does not decide the others'
// digits.
__device__ __forceinline__ uint32_t finite_bits(float x) {
  return fabsf(x) <= 3.0e38f ? __float_as_uint(fabsf(x)) : 0u;
}
__device__ __forceinline__ uint4 finite_bits(const float4& x) {
  return make_uint4(finite_bits(x.x), finite_bits(x.y), finite_bits(x.z), finite_bits(x.w));
}
__device__ __forceinline__ uint32_t largest(const uint4& x) { return max(max(x.x, x.y), max(x.z, x.w)); }
__device__ __forceinline__ uint4 larger(const uint4& a, const uint4& b) {
  return make_uint4(max(a.x, b.x), max(a.y, b.y), max(a.z, b.z), max(a.w, b.w));
}
__device__ __forceinline__ void atomic_larger(uint32_t* at, const uint4& x) {
  atomicMax(at, x.x);
  atomicMax(at + 1, x.y);
  atomicMax(at + 2, x.z);
  atomicMax(at + 3, x.w);
}
// The unit of a rank from the largest values that n CTAs found, `stride` apart.
__device__ __forceinline__ float rank_unit(const uint32_t* maxima, int stride, int n) {
  uint32_t m = 0;
  for (int c = 0; c < n; ++c) m = max(m, maxima[c * stride]);
  return split_unit(__uint_as_float(m));
}
// Four values of T times their units, in two parts.
__device__ __forceinline__ void write_parts(__half* at, int pp, const float4& x, const float4& u) {
  const Split s0 = split_half(x.x * u.x), s1 = split_half(x.y * u.y), s2 = split_half(x.z * u.z), s3 = split_half(x.w * u.w);
  *reinterpret_cast<uint2*>(at) = make_uint2(half2_bits(s0.hi, s1.hi), half2_bits(s2.hi, s3.hi));
  *reinterpret_cast<uint2*>(at + pp) = make_uint2(half2_bits(s0.lo, s1.lo), half2_bits(s2.lo, s3.lo));
}

}  // namespace dictproj
