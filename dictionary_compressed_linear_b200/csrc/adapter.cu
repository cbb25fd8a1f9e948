// Low-rank adapters beside a projection (forward, input gradient, weight gradients).
//
//   T[m] = X[m] A_s^T,  Y[m] = base[m] + scale_s T[m] B_s          s = slot of row m
//   U[m] = dY[m] B_s^T, dX[m] = base[m] + scale_s U[m] A_s
//   dA_s = scale_s sum_m U[m]^T X[m],  dB_s = scale_s sum_m T[m]^T dY[m]
//
// A and B are stored rank-major ([rank][d_in], [rank][d_out]), so the forward and
// the input gradient are one kernel with A and B exchanged: a contraction along
// the rows of the first, an expansion along the rows of the second.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "dictproj_internal.h"
#include "kernels.h"

namespace dictproj {
namespace {

// ---- plan: a stable counting sort of the rows by slot ---------------------------
// One CTA. Warp w owns a contiguous range of rows and counts its slots in its own
// histogram (equal lanes found by match), a scan over (slot, warp) turns the counts
// into positions, and the second pass over the ids scatters in row order, so the
// result does not depend on timing. Bucket n_slots takes the rows without a slot.
constexpr int kPlanWarps = 32;

__device__ __forceinline__ int plan_bucket(const int* ids, int m, int n_slots) {
  const int id = ids[m];
  return id >= 0 && id < n_slots ? id : n_slots;
}

__global__ void __launch_bounds__(kPlanWarps * 32)
    k_rows_plan(const int* __restrict__ ids, int M, int n_slots, int* __restrict__ perm, int* __restrict__ start) {
  extern __shared__ int hist[];  // [kPlanWarps][n_slots + 1]
  __shared__ int wsum[kPlanWarps];
  const int nb = n_slots + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  for (int i = threadIdx.x; i < kPlanWarps * nb; i += blockDim.x) hist[i] = 0;
  __syncthreads();
  const int per = (M + kPlanWarps - 1) / kPlanWarps;
  const int lo = warp * per, hi = min(M, lo + per);
  int* h = hist + warp * nb;
  for (int base = lo; base < hi; base += 32) {
    const int m = base + lane;
    const bool in = m < hi;
    const int b = in ? plan_bucket(ids, m, n_slots) : -1;
    const unsigned eq = __match_any_sync(0xffffffffu, b);
    if (in && lane == __ffs(eq) - 1) h[b] += __popc(eq);
    __syncwarp();
  }
  __syncthreads();
  // counts -> positions: per bucket over the warps, then over the buckets. The last
  // bucket (no slot) starts where the slots' total ends.
  int total = 0;
  if ((int)threadIdx.x < n_slots)
    for (int w = 0; w < kPlanWarps; ++w) {
      const int c = hist[w * nb + threadIdx.x];
      hist[w * nb + threadIdx.x] = total;
      total += c;
    }
  int incl = total;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += t;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int s = wsum[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, s, off);
      if (lane >= off) s += t;
    }
    wsum[lane] = s;
  }
  __syncthreads();
  const int first = incl - total + (warp ? wsum[warp - 1] : 0);
  if ((int)threadIdx.x < n_slots) {
    start[threadIdx.x] = first;
    for (int w = 0; w < kPlanWarps; ++w) hist[w * nb + threadIdx.x] += first;
  }
  if (threadIdx.x == 0) {
    int at = wsum[kPlanWarps - 1];
    start[n_slots] = at;
    start[n_slots + 1] = M;
    for (int w = 0; w < kPlanWarps; ++w) {
      const int c = hist[w * nb + n_slots];
      hist[w * nb + n_slots] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int base = lo; base < hi; base += 32) {
    const int m = base + lane;
    const bool in = m < hi;
    const int b = in ? plan_bucket(ids, m, n_slots) : -1;
    const unsigned eq = __match_any_sync(0xffffffffu, b);
    if (in) perm[h[b] + __popc(eq & ((1u << lane) - 1u))] = m;
    __syncwarp();
    if (in && lane == __ffs(eq) - 1) h[b] += __popc(eq);
    __syncwarp();
  }
}

// Slot that owns plan position p (n_slots: no adapter): the last s with start[s] <= p.
__device__ __forceinline__ int slot_at(const int* start, int n_slots, int p) {
  int lo = 0, hi = n_slots;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= p) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Copy an adapter into its slot, with zeros past its rank and past d_out.
__global__ void __launch_bounds__(256)
    k_adapter_set(const __half* __restrict__ A, const __half* __restrict__ B, int rank, float scale, int rp, int d_in,
                  int d_out, int ld_b, __half* __restrict__ sa, __half* __restrict__ sb, int* __restrict__ srank,
                  float* __restrict__ sscale) {
  grid_dependency_wait();
  const int j = blockIdx.x;
  const __half zero = __float2half_rn(0.f);
  for (int i = threadIdx.x; i < d_in; i += blockDim.x)
    sa[(size_t)j * d_in + i] = j < rank ? A[(size_t)j * d_in + i] : zero;
  for (int o = threadIdx.x; o < ld_b; o += blockDim.x)
    sb[(size_t)j * ld_b + o] = j < rank && o < d_out ? B[(size_t)j * d_out + o] : zero;
  if (j == 0 && threadIdx.x == 0) {
    *srank = rank;
    *sscale = scale;
  }
}

// ---- simple kernels -----------------------------------------------------------------
// T[p][j] = factor * In[row p] . P_s[j], one warp per (position, j)
__global__ void __launch_bounds__(256)
    k_contract(const __half* __restrict__ in, int K, const __half* __restrict__ P, int ld_p, int rp, int n_slots,
               const int* __restrict__ rank, const float* __restrict__ scale, const int* __restrict__ perm,
               const int* __restrict__ start, float* __restrict__ t) {
  grid_dependency_wait();
  const int p = blockIdx.x, s = slot_at(start, n_slots, p);
  if (s >= n_slots) return;
  const int r = rank[s], warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const __half* x = in + (size_t)perm[p] * K;
  for (int j = warp; j < rp; j += 8) {
    float acc = 0.f;
    const __half* w = P + ((size_t)s * rp + j) * ld_p;
    if (j < r)
      for (int i = lane; i < K; i += 32) acc = fmaf(__half2float(x[i]), __half2float(w[i]), acc);
#pragma unroll
    for (int off = 16; off; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (lane == 0) t[(size_t)p * rp + j] = acc * scale[s];
  }
}

// out[row p][n] = base + sum_j T[p][j] Q_s[j][n]
__global__ void __launch_bounds__(256)
    k_expand(const float* __restrict__ t, const __half* __restrict__ Q, int ld_q, int N, int rp, int n_slots,
             const int* __restrict__ rank, const int* __restrict__ perm, const int* __restrict__ start,
             const __half* __restrict__ base, __half* __restrict__ out) {
  grid_dependency_wait();
  const int p = blockIdx.x, s = slot_at(start, n_slots, p), n = blockIdx.y * 256 + threadIdx.x;
  if (n >= N) return;
  const size_t at = (size_t)perm[p] * N + n;
  const int r = s < n_slots ? rank[s] : 0;
  if (r == 0 && base == out) return;
  float acc = base ? __half2float(base[at]) : 0.f;
  for (int j = 0; j < r; ++j)
    acc = fmaf(t[(size_t)p * rp + j], __half2float(Q[((size_t)s * rp + j) * ld_q + n]), acc);
  out[at] = __float2half_rn(acc);
}

// G_s[j][i] (+)= sum over the slot's rows of T[p][j] In[row p][i]
__global__ void __launch_bounds__(256)
    k_weight_grad(const float* __restrict__ t, const __half* __restrict__ in, int K, int rp, int max_rank, int n_slots,
                  const int* __restrict__ rank, const int* __restrict__ perm, const int* __restrict__ start,
                  int accumulate, float* __restrict__ g) {
  grid_dependency_wait();
  const int i = blockIdx.x * 256 + threadIdx.x, j = blockIdx.y, s = blockIdx.z;
  if (i >= K) return;
  float acc = 0.f;
  if (j < rank[s])
    for (int p = start[s]; p < start[s + 1]; ++p)
      acc = fmaf(t[(size_t)p * rp + j], __half2float(in[(size_t)perm[p] * K + i]), acc);
  float* o = g + ((size_t)s * max_rank + j) * K + i;
  *o = accumulate ? *o + acc : acc;
}

cudaError_t launch_pdl(const void* fn, dim3 grid, dim3 block, size_t smem, cudaStream_t stream, void** args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

cudaError_t contract(const dictproj_adapters* a, const dictproj_rows* r, const __half* in, int K, const uint16_t* P,
                     int ld_p, float* t, cudaStream_t stream) {
  int rp = a->rp, ns = a->n_slots;
  void* args[] = {&in, &K, &P, &ld_p, &rp, &ns, (void*)&a->rank, (void*)&a->scale, (void*)&r->perm, (void*)&r->start, &t};
  return launch_pdl((const void*)k_contract, dim3(r->M), dim3(256), 0, stream, args);
}
cudaError_t expand(const dictproj_adapters* a, const dictproj_rows* r, const float* t, const uint16_t* Q, int ld_q,
                   int N, const __half* base, __half* out, cudaStream_t stream) {
  int rp = a->rp, ns = a->n_slots;
  void* args[] = {&t, &Q, &ld_q, &N, &rp, &ns, (void*)&a->rank, (void*)&r->perm, (void*)&r->start, &base, &out};
  return launch_pdl((const void*)k_expand, dim3(r->M, (N + 255) / 256), dim3(256), 0, stream, args);
}
cudaError_t weight_grad(const dictproj_adapters* a, const dictproj_rows* r, const float* t, const __half* in, int K,
                        bool accumulate, float* g, cudaStream_t stream) {
  int rp = a->rp, ns = a->n_slots, mr = a->max_rank, acc = accumulate;
  void* args[] = {&t, &in, &K, &rp, &mr, &ns, (void*)&a->rank, (void*)&r->perm, (void*)&r->start, &acc, &g};
  return launch_pdl((const void*)k_weight_grad, dim3((K + 255) / 256, a->max_rank, a->n_slots), dim3(256), 0, stream, args);
}

}  // namespace

cudaError_t prepare_adapter_kernels(int device) {
  (void)device;
  return cudaFuncSetAttribute(k_rows_plan, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kPlanWarps * (DICTPROJ_MAX_SLOTS + 1) * (int)sizeof(int));
}

cudaError_t launch_adapter_set(const dictproj_adapters* a, int slot, int rank, float scale, const __half* A,
                               const __half* B, cudaStream_t stream) {
  uint16_t* sa = a->A + (size_t)slot * a->rp * a->d_in;
  uint16_t* sb = a->B + (size_t)slot * a->rp * a->ld_b;
  int* sr = a->rank + slot;
  float* ss = a->scale + slot;
  int rp = a->rp, d_in = a->d_in, d_out = a->d_out, ld_b = a->ld_b;
  void* args[] = {&A, &B, &rank, &scale, &rp, &d_in, &d_out, &ld_b, &sa, &sb, &sr, &ss};
  return launch_pdl((const void*)k_adapter_set, dim3(a->rp), dim3(256), 0, stream, args);
}

cudaError_t launch_rows_plan(const dictproj_rows* r, const int* ids, int M, cudaStream_t stream) {
  int ns = r->n_slots;
  void* args[] = {&ids, &M, &ns, (void*)&r->perm, (void*)&r->start};
  return launch_pdl((const void*)k_rows_plan, dim3(1), dim3(kPlanWarps * 32),
                    (size_t)kPlanWarps * (ns + 1) * sizeof(int), stream, args);
}

cudaError_t launch_adapter_forward(const dictproj_adapters* a, const dictproj_rows* r, const __half* X,
                                   const __half* base, __half* Y, cudaStream_t stream) {
  cudaError_t e = contract(a, r, X, a->d_in, a->A, a->d_in, a->t, stream);
  if (e != cudaSuccess) return e;
  return expand(a, r, a->t, a->B, a->ld_b, a->d_out, base, Y, stream);
}

cudaError_t launch_adapter_backward(const dictproj_adapters* a, const dictproj_rows* r, const __half* X,
                                    const __half* dY, const __half* base, __half* dX, float* dA, float* dB,
                                    bool accumulate, cudaStream_t stream) {
  cudaError_t e = contract(a, r, dY, a->d_out, a->B, a->ld_b, a->u, stream);
  if (e != cudaSuccess) return e;
  if (dX && (e = expand(a, r, a->u, a->A, a->d_in, a->d_in, base, dX, stream))) return e;
  if (!dA) return cudaSuccess;
  if ((e = contract(a, r, X, a->d_in, a->A, a->d_in, a->t, stream))) return e;
  if ((e = weight_grad(a, r, a->u, X, a->d_in, accumulate, dA, stream))) return e;
  return weight_grad(a, r, a->t, dY, a->d_out, accumulate, dB, stream);
}

}  // namespace dictproj
