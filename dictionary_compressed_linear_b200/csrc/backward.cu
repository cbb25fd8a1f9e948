// Input gradient of the frozen projection: dZ = s_C dY C^T and dX = s_D dZ D^T as tcgen05
// GEMMs on densified factors.
//
// The forward's factors are stored along the reductions of the forward: Cd[d_out][k],
// D codes [k][d_in]. The gradients contract over the row index instead, so each product is
// A[M][K] B[K][N] with B row-major: a stage's B tile is bn / 64 boxes of 64 columns x 64
// reduction rows (128-byte rows, 128-byte swizzle), which the tensor cores read as an
// MN-major operand. No transposed copy of a factor exists.
//
// At 2048 rows the dense products (127 GFLOP for 4096 <- 2048 <- 11008) are what the time
// goes to; with few rows it is the chain of stages, which a cluster then splits.
//
// Between the products dZ is kept as a sum of bf16 parts, the second product's reduction running
// over them: bf16 has fp32's range, so that neither small nor large gradients leave it, and the
// dense dictionary (a product of E2M1 and E4M3 has at most six bits) is exact in it. Two parts
// hold 16 bits (2^-16 of an element at most beside dX's own 2^-11). One fp16 part made dX's
// error 2.9e-4 (2.1e-4 now: its own rounding), lost what lay below 2^-24 and gave NaN above
// 65504; it took 40 us where two take 42 (128 rows, 4096 <- 2048 <- 4096), and 130 where they
// take 161 (2048 rows, 4096 <- 2048 <- 11008). Up to
// kFineRows rows, where the second product waits for its loads and not for the tensor cores,
// a third part makes it fp32's 24 bits.
//
// Every spin-wait is bounded; a wait that gives up sets the file's device error word and
// the kernel unwinds (frees its tensor memory) without hanging.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "adapter.cuh"
#include "common.cuh"
#include "dictproj_internal.h"
#include "kernels.h"
#include "tcgen05.cuh"

namespace dictproj {
namespace {

__device__ __forceinline__ uint32_t bf16x2_bits(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }

// Dense bf16 copy of D^ (Dd[j][i], E2M1 x E4M3 exact in fp16 and in bf16, without s_D): a
// thread per 16-value block, 8 + 1 bytes in, 32 bytes out.
struct DictCopy {
  const uint8_t* codes;
  const uint8_t* scales;
  __nv_bfloat16* dd;
  long n_blocks;
};
// N blocks, `step` apart; those past the end are left out.
template <int N>
__device__ __forceinline__ void densify_blocks(const DictCopy& d, long b, long step) {
  uint2 c[N];
  uint32_t sc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const long at = min(b + i * step, d.n_blocks - 1);
    c[i] = ld_stream_v2(d.codes + 8 * at);
    sc[i] = d.scales[at];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (b + i * step >= d.n_blocks) break;
    const uint32_t sv = dup_lo(e4m3x2_to_f16x2(sc[i]));
    uint32_t v[8];
    e2m1x8_to_f16x2x4(c[i].x, *reinterpret_cast<uint32_t(*)[4]>(v));
    e2m1x8_to_f16x2x4(c[i].y, *reinterpret_cast<uint32_t(*)[4]>(v + 4));
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t h = hmul2_u32(v[e], sv);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      v[e] = bf16x2_bits(f.x, f.y);
    }
    uint4* dst = reinterpret_cast<uint4*>(d.dd + 16 * (b + i * step));
    dst[0] = make_uint4(v[0], v[1], v[2], v[3]);
    dst[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}
__global__ void __launch_bounds__(256) k_densify_dict(DictCopy d) {
  grid_dependency_wait();  // Dd may still be read by the previous input-gradient GEMM
  trigger_dependents();
  const long b = (long)blockIdx.x * blockDim.x + threadIdx.x;
  if (b < d.n_blocks) densify_blocks<1>(d, b, 0);
}

constexpr int kNnM = 128, kNnK = 64, kNnMaxN = 256, kNnStages = 4;
constexpr int kNnThreads = 320;  // warp 0 TMA, warp 1 MMA + tensor memory, warps 2..9 epilogue
constexpr int kNnABytes = kNnM * kNnK * 2, kNnBBytes = kNnMaxN * kNnK * 2;
constexpr size_t kNnSmem = (size_t)kNnStages * (kNnABytes + kNnBBytes) + 1024 + 256;
constexpr int kNnSplitN = 128;  // widest tile of a split product: its fp32 sums fit the ring
static_assert(kNnM * (kNnSplitN + 4) * 4 <= kNnStages * (kNnABytes + kNnBBytes), "partial sums");

// dZ's parts, each bf16 [M][k]: a part is the bf16 value nearest to what the parts before it leave.
constexpr int kZParts = 3;
struct ZParts {
  __nv_bfloat16* p[kZParts];
  int n;
};
__device__ __forceinline__ void store_parts(const ZParts& z, size_t at, float (&f)[8]) {
#pragma unroll
  for (int q = 0; q < kZParts; ++q) {
    if (q >= z.n) break;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[e] = bf16x2_bits(f[2 * e], f[2 * e + 1]);
      const float a = bf16_value(w[e]), b = bf16_value(w[e] >> 16);
      // nothing is left of an infinity or NaN
      f[2 * e] = fabsf(a) <= 3.4e38f ? f[2 * e] - a : 0.f;
      f[2 * e + 1] = fabsf(b) <= 3.4e38f ? f[2 * e + 1] - b : 0.f;
    }
    *reinterpret_cast<uint4*>(z.p[q] + at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
__device__ __forceinline__ void store_half(__half* out, const float (&f)[8]) {
  uint32_t h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = half2_bits(__float2half_rn(f[2 * e]), __float2half_rn(f[2 * e + 1]));
  *reinterpret_cast<uint4*>(out) = make_uint4(h[0], h[1], h[2], h[3]);
}

// A's parts (the first product has one), 128 rows by 64 columns, and B, 64 by 64.
struct NnMaps {
  CUtensorMap a[kZParts], b;
};
struct NnShape {
  int M, N, K;
  int parts;  // of A
  int bn, nx, tiles;
  float scale;
};

// One 128 x bn tile (bn a multiple of 64) of out = scale A B. With gridDim.z = S > 1 the S
// CTAs of a cluster (1, 1, S) take consecutive ranges of the reduction's stages; the fp32
// partial tiles meet through distributed shared memory, in rank order, each CTA writing its
// share of the rows. CTAs past the tiles (only without a split, on SMs that the tiles leave
// idle) make the dense dictionary that the next product reads.
// FIRST: dZ = s_C dY Cd, fp16 operands, into z. Otherwise dX = s_D z Dd, bf16 operands, into out.
template <bool FIRST>
__global__ void __launch_bounds__(kNnThreads, 1)
    k_gemm_nn(const __grid_constant__ NnMaps maps, const __grid_constant__ NnShape shape, const __grid_constant__ ZParts z,
              __half* __restrict__ out, const __grid_constant__ DictCopy copy) {
  const int M = shape.M, N = shape.N, K = shape.K, bn = shape.bn, nx = shape.nx, tiles = shape.tiles;
  const float scale = shape.scale;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sb = smem + kNnStages * kNnABytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sb + kNnStages * kNnBBytes);
  uint64_t* empty = full + kNnStages;
  uint64_t* accf = empty + kNnStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accf + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((int)blockIdx.x >= tiles) {
    grid_dependency_wait();
    trigger_dependents();
    const long step = (long)(gridDim.x - tiles) * kNnThreads;
    // four blocks at a time, their loads together
    for (long b = (long)(blockIdx.x - tiles) * kNnThreads + threadIdx.x; b < copy.n_blocks; b += 4 * step) densify_blocks<4>(copy, b, step);
    return;
  }
  const int n0 = blockIdx.x % nx * bn, m0 = blockIdx.x / nx * kNnM, split = blockIdx.z, nsplit = gridDim.z;
  const int nk_one = (K + kNnK - 1) / kNnK, nk_all = shape.parts * nk_one;  // A's parts in turn
  const int s_lo = (int)((long)nk_all * split / nsplit);
  const int nk = (int)((long)nk_all * (split + 1) / nsplit) - s_lo;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kNnStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(accf, 1);
    fence_mbar_init();
    tma_prefetch_map(&maps.a[0]);
    tma_prefetch_map(&maps.b);
  }
  if (warp == 1) tmem_alloc(tmem_slot, kNnMaxN);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();  // A and B may be the previous kernels' output
  trigger_dependents();    // after the tensor memory is ours

  if (warp == 0) {
    if (lane == 0) {
      RingPos at;
      // A's part and column of a stage, advanced without a division (one took 10 us of 82, a
      // stage waiting for its coordinates)
      int part = FIRST ? 0 : s_lo / nk_one, kx = (s_lo - part * nk_one) * kNnK;
      const CUtensorMap* tm_a = FIRST || part == 0 ? &maps.a[0] : part == 1 ? &maps.a[1] : &maps.a[2];
      for (int s = 0; s < nk; ++s, at.next(kNnStages), kx += kNnK) {
        if (!FIRST && kx >= K) {
          tm_a = ++part == 1 ? &maps.a[1] : &maps.a[2];
          kx = 0;
        }
        if (s >= kNnStages && !mbar_wait_bounded(&empty[at.slot], at.phase ^ 1)) {
          drain(full, kNnStages, s);
          break;
        }
        mbar_arrive_expect_tx(&full[at.slot], kNnABytes + bn * kNnK * 2);
        tma_load_2d(smem_u32(smem + at.slot * kNnABytes), tm_a, kx, m0, &full[at.slot]);
        for (int c = 0; c < bn / 64; ++c)
          tma_load_2d(smem_u32(sb + at.slot * kNnBBytes + c * kMnChunk), &maps.b, n0 + 64 * c, kx, &full[at.slot]);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // kind::f16, A (K-major) and B (MN-major) fp16 or bf16, D fp32, M = 128, N = bn
      const uint32_t idesc = (1u << 4) | (FIRST ? 0u : (1u << 7) | (1u << 10)) | (1u << 16) | ((uint32_t)(bn >> 3) << 17) | ((uint32_t)(kNnM >> 4) << 24);
      const uint64_t a0 = smem_desc_sw128(smem_u32(smem)), b0 = smem_desc_mn_sw128(smem_u32(sb));
      RingPos at;
      for (int s = 0; s < nk; ++s, at.next(kNnStages)) {
        if (!mbar_wait_bounded(&full[at.slot], at.phase)) break;
        tc_fence_after();
        const uint64_t a = desc_at(a0, at.slot * kNnABytes), b = desc_at(b0, at.slot * kNnBBytes);
#pragma unroll
        for (int j = 0; j < kNnK / 16; ++j)
          mma_f16_ss(tmem, desc_at(a, 32 * j), desc_at(b, 2048 * j), idesc, (s | j) != 0);
        mma_commit(&empty[at.slot]);
      }
      mma_commit(accf);
    }
  }
  __syncwarp();
  const int pitch = bn + 4;  // floats of a row of the partial sums, over the drained ring
  float* part = reinterpret_cast<float*>(smem);
  if (warp >= 2) {
    const int q = warp & 3, half = (warp - 2) >> 2, row = 32 * q + lane;
    const bool ok = mbar_wait_bounded(accf, 0);
    tc_fence_after();
#pragma unroll 1
    for (int c = half; 32 * c < bn; c += 2) {
      uint32_t v[32];
      tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + 32 * c, v);
      if (nsplit > 1) {
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          *reinterpret_cast<float4*>(part + row * pitch + 32 * c + e) = make_float4(
              __uint_as_float(v[e]), __uint_as_float(v[e + 1]), __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
        continue;
      }
      if (!ok || m0 + row >= M) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int gc = n0 + 32 * c + 8 * j;
        if (gc >= N) break;  // N % 8 == 0
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(v[8 * j + e]) * scale;
        const size_t o = (size_t)(m0 + row) * N + gc;
        if (FIRST) store_parts(z, o, f);
        else store_half(out + o, f);
      }
    }
  }
  tc_fence_before();
  if (nsplit > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kNnMaxN);
  }
  if (nsplit > 1) {
    const uint32_t pbase = smem_u32(part);
    const int pieces = bn / 8, rows = kNnM / nsplit;
    for (int i = threadIdx.x; i < rows * pieces; i += kNnThreads) {
      const int row = split * rows + i / pieces, c = 8 * (i % pieces);
      if (m0 + row >= M || n0 + c >= N) continue;
      const uint32_t at = pbase + 4 * (row * pitch + c);
      const float4 x = sum_peers(at, nsplit), y = sum_peers(at + 16, nsplit);
      float f[8] = {x.x * scale, x.y * scale, x.z * scale, x.w * scale, y.x * scale, y.y * scale, y.z * scale, y.w * scale};
      const size_t o = (size_t)(m0 + row) * N + n0 + c;
      if (FIRST) store_parts(z, o, f);
      else store_half(out + o, f);
    }
    cluster_arrive();  // no CTA leaves while its sums are read
    cluster_wait();
  }
}

// Self-test of this file's bounded-wait error path (its own device error word).
__global__ void k_wait_probe_backward(long long cycles) {
  __shared__ __align__(8) uint64_t bar;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 2);
    fence_mbar_init();
  }
  __syncwarp();
  if (threadIdx.x == 0) {
    mbar_arrive(&bar);
    mbar_wait_bounded(&bar, 0, cycles);
  }
  __syncwarp();
}

void set_pdl(cudaLaunchAttribute& a) {
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
}
void set_cluster_z(cudaLaunchAttribute& a, int s) {
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = 1;
  a.val.clusterDim.y = 1;
  a.val.clusterDim.z = (unsigned)s;
}

// Clusters of S CTAs of k_gemm_nn (one CTA an SM) that the device holds at once; cached.
int nn_clusters_that_fit(int S, int n_sm) {
  static std::atomic<int> cache[16][9];  // the answer + 1; zero: not asked yet
  if (S == 1) return n_sm;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 16 || S > 8) return 0;
  if (const int known = cache[dev][S].load(std::memory_order_relaxed)) return known - 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, 1, S);
  cfg.blockDim = dim3(kNnThreads);
  cfg.dynamicSmemBytes = kNnSmem;
  cudaLaunchAttribute attr[1];
  set_cluster_z(attr[0], S);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, (const void*)k_gemm_nn<true>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  cache[dev][S].store(n + 1, std::memory_order_relaxed);
  return n;
}

// Tile width and split of one product, by a model of its time in us: waves of tiles, each a
// fixed part, its stages (0.1 + 0.0014 per column each) and, split, the sum over the cluster.
struct NnPlan {
  int bn, split;
  double us;
};
NnPlan nn_plan(int M, int N, int K, int n_sm) {
  const int nk = (K + kNnK - 1) / kNnK, rows = (M + kNnM - 1) / kNnM;
  NnPlan best = {256, 1, 0.0};
  double cost = 1e30;
  for (int bn = 64; bn <= kNnMaxN; bn += 64) {
    const long tiles = (long)rows * ((N + bn - 1) / bn);
    for (int S = 1; S <= 8 && (S == 1 || (bn <= kNnSplitN && nk / S >= 2)); S *= 2) {
      const int fit = nn_clusters_that_fit(S, n_sm);
      if (fit < 1) continue;
      const double t = (double)((tiles + fit - 1) / fit) * (3.0 + (double)((nk + S - 1) / S) * (0.1 + 0.0014 * bn) + (S > 1 ? 2.5 : 0.0));
      if (t < cost) cost = t, best = {bn, S, t};
    }
  }
  return best;
}

}  // namespace

cudaError_t prepare_backward_kernels(int device) {
  (void)device;
  const cudaError_t e = cudaFuncSetAttribute(k_gemm_nn<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kNnSmem);
  return e != cudaSuccess ? e : cudaFuncSetAttribute(k_gemm_nn<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kNnSmem);
}

// A: the product's left operand in shape.parts parts, [M][K] each; B [K][N].
template <bool FIRST>
static cudaError_t launch_nn(const void* const* A, const void* B, NnShape shape, const ZParts& z, __half* out, const NnPlan& plan,
                             const DictCopy& copy, int helpers, cudaStream_t stream) {
  const CUtensorMapDataType type = FIRST ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const uint64_t M = shape.M, N = shape.N, K = shape.K;
  NnMaps maps;
  cudaError_t e;
  for (int p = 0; p < shape.parts; ++p)
    if ((e = encode_tiled_2d(&maps.a[p], type, A[p], K, M, K * 2, kNnK, kNnM, CU_TENSOR_MAP_SWIZZLE_128B))) return e;
  for (int p = shape.parts; p < kZParts; ++p) maps.a[p] = maps.a[0];  // not used
  if ((e = encode_tiled_2d(&maps.b, type, B, N, K, N * 2, 64, kNnK, CU_TENSOR_MAP_SWIZZLE_128B))) return e;
  shape.bn = plan.bn;
  shape.nx = (shape.N + plan.bn - 1) / plan.bn;
  shape.tiles = shape.nx * ((shape.M + kNnM - 1) / kNnM);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(shape.tiles + helpers, 1, plan.split);
  cfg.blockDim = dim3(kNnThreads);
  cfg.dynamicSmemBytes = kNnSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  set_pdl(attr[0]);
  set_cluster_z(attr[1], plan.split);
  cfg.attrs = attr;
  cfg.numAttrs = plan.split > 1 ? 2 : 1;
  void* args[] = {(void*)&maps, (void*)&shape, (void*)&z, (void*)&out, (void*)&copy};
  return cudaLaunchKernelExC(&cfg, (const void*)k_gemm_nn<FIRST>, args);
}

cudaError_t launch_backward_input(const dictproj_group* g, const dictproj_layer* l, const __half* dY, int M, const __half* Cd,
                                  __half* dX, cudaStream_t stream) {
  cudaError_t e;
  const DictCopy copy = {g->codes, g->scales, reinterpret_cast<__nv_bfloat16*>(g->ddense), (long)g->k * (g->d_in / 16)};
  const NnPlan p = nn_plan(M, g->k, l->d_out, g->n_sm);
  // SMs that the first product leaves idle make the dense dictionary, where they can in its
  // time (41 bytes a block at some 60 GB/s an SM): 2048 rows (4096 <- 2048 <- 11008) took 119 us
  // with a launch for it and one part of dZ.
  const int tiles = (g->k + p.bn - 1) / p.bn * ((M + kNnM - 1) / kNnM), idle = g->n_sm - tiles;
  int helpers = p.split == 1 && idle >= 8 && copy.n_blocks * 41e-3 / 60 / idle < 0.7 * p.us ? idle : 0;
  if (!helpers) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((copy.n_blocks + 255) / 256));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    set_pdl(attr[0]);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {(void*)&copy};
    if ((e = cudaLaunchKernelExC(&cfg, (const void*)k_densify_dict, args))) return e;
  }
  __nv_bfloat16* more = reinterpret_cast<__nv_bfloat16*>(g->zmore);
  const ZParts z = {{reinterpret_cast<__nv_bfloat16*>(g->z16), more, more + (size_t)g->max_tokens * g->k}, M <= kFineRows ? 3 : 2};
  const void* dy[] = {dY};
  if ((e = launch_nn<true>(dy, Cd, NnShape{M, g->k, l->d_out, 1, 0, 0, 0, l->s}, z, nullptr, p, copy, helpers, stream))) return e;
  const void* parts[] = {z.p[0], z.p[1], z.p[2]};
  return launch_nn<false>(parts, g->ddense, NnShape{M, g->d_in, g->k, z.n, 0, 0, 0, g->s}, z, dX,
                          nn_plan(M, g->d_in, z.n * g->k, g->n_sm), copy, 0, stream);
}

cudaError_t launch_wait_probe_backward(long long cycles, cudaStream_t stream) {
  k_wait_probe_backward<<<1, 32, 0, stream>>>(cycles);
  return cudaGetLastError();
}

cudaError_t take_backward_error(unsigned int* out) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_dictproj_error, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_dictproj_error, &zero, sizeof(unsigned int));
}

}  // namespace dictproj
