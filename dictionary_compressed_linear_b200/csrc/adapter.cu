// Low-rank adapters beside a projection (forward, input gradient, weight gradients).
//
//   T[m] = X[m] A_s^T,  Y[m] = base[m] + scale_s T[m] B_s          s = slot of row m
//   U[m] = dY[m] B_s^T, dX[m] = base[m] + scale_s U[m] A_s
//   dA_s = scale_s sum_m U[m]^T X[m],  dB_s = scale_s sum_m T[m]^T dY[m]
//
// A and B are stored rank-major ([rank][d_in], [rank][d_out]), so the forward and
// the input gradient are the same kernels with A and B exchanged: a contraction along
// the rows of the first, an expansion along the rows of the second. Both weight
// gradients are one kernel as well.
//
// Here are the plan, the kernels of few rows (CUDA cores) and those of many rows on
// mma.sync, which serve any row length; adapter_tall.cu has those on tcgen05 for row
// lengths that TMA can read.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "adapter.cuh"
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
// Then the slots' rows are cut into tiles of kFewRows, kWideRows and kTallRows.
constexpr int kPlanWarps = 32;

__device__ __forceinline__ int plan_bucket(const int* ids, int m, int n_slots) {
  const int id = ids[m];
  return id >= 0 && id < n_slots ? id : n_slots;
}

__device__ __forceinline__ int plan_rows(int q) { return q == 0 ? kFewRows : q == 1 ? kWideRows : kTallRows; }

// Exclusive sum over the CTA's threads; *total gets the whole sum.
__device__ __forceinline__ int block_exclusive_sum(int x, int* wsum, int* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int incl = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += t;
  }
  __syncthreads();  // wsum may still be read
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kPlanWarps; ++w) {
    const int s = wsum[w];
    before += w < warp ? s : 0;
    all += s;
  }
  *total = all;
  return before + incl - x;
}

__global__ void __launch_bounds__(kPlanWarps * 32)
    k_rows_plan(const int* __restrict__ ids, int M, int n_slots, int* __restrict__ perm, int* __restrict__ start,
                int* __restrict__ n_tiles, int4* __restrict__ tiles4, int4* __restrict__ tiles64,
                int4* __restrict__ tiles128, int* __restrict__ runs64, int* __restrict__ runs128,
                int* __restrict__ first64, int* __restrict__ used) {
  extern __shared__ int plan_smem[];
  __shared__ int wsum[kPlanWarps];
  const int nb = n_slots + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* hist = plan_smem;                    // [kPlanWarps][nb]
  int* begin = hist + kPlanWarps * nb;      // [nb + 1] first position of each bucket
  int* tfirst = begin + nb + 1;             // [3][nb + 1] first tile of each bucket
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
  // counts -> positions: per bucket over the warps, then over the buckets; the
  // bucket without a slot comes last, behind the total of the others
  const int s = threadIdx.x;
  int count = 0;
  if (s < n_slots)
    for (int w = 0; w < kPlanWarps; ++w) {
      const int c = hist[w * nb + s];
      hist[w * nb + s] = count;
      count += c;
    }
  int live;
  const int first = block_exclusive_sum(count, wsum, &live);
  if (s < n_slots) {
    start[s] = begin[s] = first;
    for (int w = 0; w < kPlanWarps; ++w) hist[w * nb + s] += first;
  }
  if (threadIdx.x == 0) {
    start[n_slots] = begin[n_slots] = live;
    start[n_slots + 1] = begin[nb] = M;
    int at = live;
    for (int w = 0; w < kPlanWarps; ++w) {
      const int c = hist[w * nb + n_slots];
      hist[w * nb + n_slots] = at;
      at += c;
    }
  }
  int n_used;
  const int at_used = block_exclusive_sum(count > 0 ? 1 : 0, wsum, &n_used);
  if (count > 0) used[at_used] = s;
  if (threadIdx.x == 0) {
    n_tiles[6] = n_used;
    n_tiles[7] = M;
  }
#pragma unroll 1
  for (int q = 0; q < 3; ++q) {
    const int T = plan_rows(q);
    int last;
    const int f = block_exclusive_sum((count + T - 1) / T, wsum, &last);
    if (s < n_slots) {
      tfirst[q * (nb + 1) + s] = f;
      if (q == 1) first64[s] = f;
    }
    if (threadIdx.x == 0) {
      const int all = last + (M - live + T - 1) / T;
      tfirst[q * (nb + 1) + n_slots] = last;
      tfirst[q * (nb + 1) + nb] = all;
      n_tiles[2 * q] = last;
      n_tiles[2 * q + 1] = all;
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
  __syncthreads();  // the tiles name row numbers of perm
#pragma unroll 1
  for (int q = 0; q < 3; ++q) {
    const int T = plan_rows(q);
    const int* tf = tfirst + q * (nb + 1);
    int4* tiles = q == 0 ? tiles4 : q == 1 ? tiles64 : tiles128;
    for (int t = threadIdx.x; t < tf[nb]; t += blockDim.x) {
      int a = 0, z = n_slots;  // the last bucket whose first tile is <= t (an empty bucket owns none)
      while (a < z) {
        const int mid = (a + z + 1) >> 1;
        if (tf[mid] <= t) a = mid;
        else z = mid - 1;
      }
      const int p = begin[a] + (t - tf[a]) * T, n = min(T, begin[a + 1] - p), row = perm[p];
      const int crowd = a < n_slots && begin[a + 1] - begin[a] > kCrowd ? kCrowdTile : 0;
      tiles[t] = make_int4(a, p, n | crowd, q == 2 ? tfirst[nb + 1 + a] + 2 * (t - tf[a]) : row);
      // a bucket's rows ascend: they follow one another when the last is n - 1 further
      if (q) (q == 1 ? runs64 : runs128)[t] = perm[p + n - 1] - row == n - 1 ? row : -1;
    }
  }
}

// Copy an adapter into its slot, with zeros past its rank and past d_out.
constexpr int kSetCols = 1024;  // columns of a CTA

__global__ void __launch_bounds__(256)
    k_adapter_set(const __half* __restrict__ A, const __half* __restrict__ B, int rank, float scale, int rp, int d_in,
                  int d_out, int ld_b, __half* __restrict__ sa, __half* __restrict__ sb, int* __restrict__ srank,
                  float* __restrict__ sscale) {
  grid_dependency_wait();
  const int j = blockIdx.x, c0 = blockIdx.y * kSetCols + threadIdx.x;
  const __half zero = __float2half_rn(0.f);
#pragma unroll
  for (int q = 0; q < kSetCols / 256; ++q) {
    const int c = c0 + 256 * q;
    if (c < d_in) sa[(size_t)j * d_in + c] = j < rank ? A[(size_t)j * d_in + c] : zero;
    if (c < ld_b) sb[(size_t)j * ld_b + c] = j < rank && c < d_out ? B[(size_t)j * d_out + c] : zero;
  }
  if (j == 0 && c0 == 0) {
    *srank = rank;
    *sscale = scale;
  }
}

// 16 bytes global -> shared, the last 16 - bytes of them zeros
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// Byte offset of 16-byte piece p of row `row` in a tile of PITCH-byte rows whose
// pieces are permuted so that 8 rows' pieces of one column lie in different banks.
template <int PITCH>
__device__ __forceinline__ uint32_t swz(int row, int p) {
  constexpr int per = PITCH / 16, shift = PITCH >= 128 ? 0 : PITCH == 64 ? 1 : 2, mask = per >= 8 ? 7 : per - 1;
  return (uint32_t)(row * PITCH + 16 * (p ^ ((row >> shift) & mask)));
}

// ---- contraction and expansion -------------------------------------------------------------
constexpr int kCluster = 8;
constexpr int kRowThreads = 256;

// ---- few rows of a slot: serving ----------------------------------------------------------
// A cluster of kCluster CTAs takes one tile of up to four rows of one slot and walks the
// weights once, 16 bytes a lane straight from memory, on the CUDA cores (a weight meets
// at most four rows: the tensor cores would have nothing to reuse).
//   1. CTA c contracts its share of the K columns: warp w owns the ranks w, w + 8, ...;
//   2. the CTAs' partial sums meet through distributed shared memory, in rank order;
//   3. CTA c expands T into its share of the N columns: four lanes split the ranks of
//      eight columns. Its part of Q is on its way to L2 since before 1.
// Bound by latency: the chain is plan -> rank and rows -> X and P -> cluster -> Q. One row of
// rank 16 (4096 -> 4096) takes 4.2 us, 64 requests with an adapter each (4096 -> 11008, 34 MB)
// 12.1 us: 2.8 TB/s. With tiles of 16 rows on mma.sync, staged through shared memory, they
// took 7.0 and 29.9 us; without the prefetch of the first ranks the second took 17.0 us.
__device__ __forceinline__ void dot2(float& acc, uint32_t x2, uint32_t w2) {
  asm("{\n\t.reg .f16 a, b, c, d;\n\tmov.b32 {a, b}, %1;\n\tmov.b32 {c, d}, %2;\n\t"
      "fma.rn.f32.f16 %0, a, c, %0;\n\tfma.rn.f32.f16 %0, b, d, %0;\n\t}" : "+f"(acc) : "r"(x2), "r"(w2));
}
__device__ __forceinline__ void dot8(float& acc, const uint4& x, const uint4& w) {
  dot2(acc, x.x, w.x);
  dot2(acc, x.y, w.y);
  dot2(acc, x.z, w.z);
  dot2(acc, x.w, w.w);
}
struct FewTile {
  int row[kFewRows];
  int first, count, r, rankc;  // first: the tile's first position in the plan
  float scale;
  const __half* P;
  const __half* Q;
};

// Rows [r_lo, r_hi) of pieces [lo, hi) to L2, by 128-byte lines.
__device__ __forceinline__ void prefetch_rows(const __half* w, int ld, int lo, int hi, int r_lo, int r_hi) {
  const int lines = (hi - lo + 7) / 8;
  for (int i = threadIdx.x; i < (r_hi - r_lo) * lines; i += kRowThreads) {
    const __half* q = w + (size_t)(r_lo + i / lines) * ld + 8 * (lo + 8 * (i % lines));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
  }
}

template <int R, int NR, bool VEC>
__device__ __forceinline__ void few_rows(const RowsPass& a, int n_rows, int pp, const FewTile& f, float* part, float* full) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kp = (a.K + 7) / 8, np = a.out ? (a.N + 7) / 8 : 0;
  const int n_lo = np * f.rankc / kCluster, n_hi = np * (f.rankc + 1) / kCluster;
  if (R > 16) prefetch_rows(f.Q, a.ld_q, n_lo, n_hi, 16, f.r);
  float acc[R / 8][NR];
#pragma unroll
  for (int j = 0; j < R / 8; ++j)
#pragma unroll
    for (int m = 0; m < NR; ++m) acc[j][m] = 0.f;
  const int k_hi = kp * (f.rankc + 1) / kCluster;
#pragma unroll 2
  for (int p = kp * f.rankc / kCluster + lane; p < k_hi; p += 32) {
    uint4 x[NR];
#pragma unroll
    for (int m = 0; m < NR; ++m) x[m] = read_piece(a.in + (size_t)f.row[m] * a.K, 8 * p, a.K, VEC, a.in + (size_t)n_rows * a.K);
    // Ranks past the slot's repeat its last (their T is zeroed below), so that no branch
    // stands between the loads: with one they went out one after the other, and a row of
    // 10288 columns and 93 ranks took 42 us. Eight at a time bounds the registers.
#pragma unroll
    for (int j0 = 0; j0 < R / 8; j0 += 8) {
      if (warp + 8 * j0 >= f.r) break;
      uint4 w[R / 8 < 8 ? R / 8 : 8];
#pragma unroll
      for (int j = 0; j < 8 && j0 + j < R / 8; ++j)
        w[j] = *reinterpret_cast<const uint4*>(f.P + (size_t)min(warp + 8 * (j0 + j), f.r - 1) * a.ld_p + 8 * p);
#pragma unroll
      for (int j = 0; j < 8 && j0 + j < R / 8; ++j)
#pragma unroll
        for (int m = 0; m < NR; ++m) dot8(acc[j0 + j][m], x[m], w[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < R / 8; ++j)
#pragma unroll
    for (int m = 0; m < NR; ++m) {
      float x = acc[j][m];
#pragma unroll
      for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
      if (lane == 0) part[m * R + warp + 8 * j] = x;
    }
  cluster_arrive();
  cluster_wait();
  const uint32_t pbase = smem_u32(part);
  for (int i = tid; i < NR * R; i += kRowThreads) {
    float x[kCluster];
#pragma unroll
    for (int c = 0; c < kCluster; ++c) x[c] = ld_peer_f32(peer_smem(pbase + 4 * i, c));
#pragma unroll
    for (int c = 1; c < kCluster; ++c) x[0] += x[c];
    full[i] = i % R < f.r ? x[0] * f.scale : 0.f;
  }
  cluster_arrive();  // waited for at the end: no CTA leaves while its sums are read
  __syncthreads();
  if (a.sums && f.rankc < f.count)  // a row each for the weight gradients
    for (int j = tid; j < ((f.r + 7) & ~7); j += kRowThreads) a.sums[(size_t)(f.first + f.rankc) * pp + j] = full[f.rankc * R + j];
  const int js = lane >> 3;
  for (int p0 = n_lo + 8 * warp; p0 < n_hi; p0 += 8 * (kRowThreads / 32)) {  // the warp's lanes stay together
    const int p = p0 + (lane & 7);
    const bool in = p < n_hi;
    float y[NR][8];
#pragma unroll
    for (int m = 0; m < NR; ++m)
#pragma unroll
      for (int e = 0; e < 8; ++e) y[m][e] = 0.f;
    uint4 b = make_uint4(0, 0, 0, 0);
    const int row = f.row[0];
    const bool mine = in && js < f.count && js < NR;
    const __half* brow = nullptr;
    __half* orow = nullptr;
    if (mine) {
      int mr = row;
#pragma unroll
      for (int m = 1; m < NR; ++m) mr = js == m ? f.row[m] : mr;
      brow = a.base + (size_t)mr * a.N;
      orow = a.out + (size_t)mr * a.N;
      if (a.base) b = read_piece(brow, 8 * p, a.N, VEC, a.base + (size_t)n_rows * a.N);
    }
    if (in)
#pragma unroll 4
      for (int j = js; j < f.r; j += 4) {
        const uint4 w = *reinterpret_cast<const uint4*>(f.Q + (size_t)j * a.ld_q + 8 * p);
        const float2 w0 = __half22float2(*reinterpret_cast<const __half2*>(&w.x)), w1 = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
        const float2 w2 = __half22float2(*reinterpret_cast<const __half2*>(&w.z)), w3 = __half22float2(*reinterpret_cast<const __half2*>(&w.w));
#pragma unroll
        for (int m = 0; m < NR; ++m) {
          const float t = full[m * R + j];
          y[m][0] = fmaf(t, w0.x, y[m][0]), y[m][1] = fmaf(t, w0.y, y[m][1]);
          y[m][2] = fmaf(t, w1.x, y[m][2]), y[m][3] = fmaf(t, w1.y, y[m][3]);
          y[m][4] = fmaf(t, w2.x, y[m][4]), y[m][5] = fmaf(t, w2.y, y[m][5]);
          y[m][6] = fmaf(t, w3.x, y[m][6]), y[m][7] = fmaf(t, w3.y, y[m][7]);
        }
      }
    float o[8];
#pragma unroll
    for (int m = 0; m < NR; ++m)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float x = y[m][e];
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        o[e] = m == 0 || js == m ? x : o[e];
      }
    if (mine) {
      const float2 b0 = __half22float2(*reinterpret_cast<const __half2*>(&b.x)), b1 = __half22float2(*reinterpret_cast<const __half2*>(&b.y));
      const float2 b2 = __half22float2(*reinterpret_cast<const __half2*>(&b.z)), b3 = __half22float2(*reinterpret_cast<const __half2*>(&b.w));
      const __half2 h0 = __floats2half2_rn(b0.x + o[0], b0.y + o[1]), h1 = __floats2half2_rn(b1.x + o[2], b1.y + o[3]);
      const __half2 h2 = __floats2half2_rn(b2.x + o[4], b2.y + o[5]), h3 = __floats2half2_rn(b3.x + o[6], b3.y + o[7]);
      write_piece(orow, 8 * p, a.N, VEC,
                  make_uint4(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1),
                             *reinterpret_cast<const uint32_t*>(&h2), *reinterpret_cast<const uint32_t*>(&h3)));
    }
  }
  cluster_wait();
}

// VEC: K and N are multiples of 8, every row 16-byte aligned.
template <int R, bool VEC>
__global__ void __launch_bounds__(kRowThreads, R <= 32 ? 4 : 2) k_adapter_few(const __grid_constant__ RowsArgs g) {
  __shared__ __align__(16) float part[kFewRows * R], full[kFewRows * R];
  const RowsPass& a = g.pass[blockIdx.y];
  const int tile_no = blockIdx.x / kCluster;
  grid_dependency_wait();
  trigger_dependents();
  const bool in_place = a.out == nullptr || a.base == a.out;
  const int4 tile = g.tiles[tile_no];
  if (!takes_tile(g, tile_no, tile, in_place)) return;  // the whole cluster
  FewTile f;
  f.first = tile.y;
  f.count = tile.z & (kCrowdTile - 1);
  f.rankc = blockIdx.x % kCluster;
  if (tile.x < g.n_slots) {
    f.P = a.P + (size_t)tile.x * g.rp * a.ld_p;
    f.Q = a.Q + (size_t)tile.x * g.rp * a.ld_q;
    // the first 16 ranks (every slot holds as many rows) start before the rank is known
    const int kp = (a.K + 7) / 8, np = a.out ? (a.N + 7) / 8 : 0;
    prefetch_rows(f.P, a.ld_p, kp * f.rankc / kCluster, kp * (f.rankc + 1) / kCluster, 0, 16);
    prefetch_rows(f.Q, a.ld_q, np * f.rankc / kCluster, np * (f.rankc + 1) / kCluster, 0, 16);
  }
  f.r = tile.x < g.n_slots ? g.rank[tile.x] : 0;
  f.row[0] = tile.w;
#pragma unroll
  for (int m = 1; m < kFewRows; ++m) f.row[m] = m < f.count ? g.perm[tile.y + m] : tile.w;
  if (f.r == 0) {
    const int np = (a.N + 7) / 8;
    if (!in_place)
      copy_rows(a, g.rows, g.perm + tile.y, f.count, np * f.rankc / kCluster, np * (f.rankc + 1) / kCluster);
    return;
  }
  f.scale = g.scale[tile.x];
  if (f.count == 1) few_rows<R, 1, VEC>(a, g.rows, g.pp, f, part, full);
  else few_rows<R, kFewRows, VEC>(a, g.rows, g.pp, f, part, full);
}

// ---- many rows of a slot: prefill and training ----------------------------------------------
// Two launches, so that each has a grid of its own: tiles x K-splits for the contraction,
// tiles x column blocks for the expansion (one launch for both, a cluster a tile, left
// each CTA a chain of eight loads and two cluster barriers, and at 2048 rows of rank 32
// took 27 us). T passes through the pool's workspace in two fp16 parts, with a
// unit per row for the expansion and once more with one per rank for the weight gradients.
//
// Contraction: a cluster splits the K columns of one tile of up to kWideRows rows; every
// CTA streams its share in 64-column stages (cp.async) through mma.sync, the partial sums
// meet through distributed shared memory, in rank order, and each CTA writes its share of
// the tile's rows.
template <int R>
struct ContractShape {
  static constexpr int TM = kWideRows, CW = 64;  // rows, columns of a stage
  static constexpr int kPitch = 2 * CW;
  static constexpr int kStages = 4;
  static constexpr int kInBytes = TM * kPitch, kStageBytes = (TM + R) * kPitch;
  static constexpr int kPart = kStages * kStageBytes;
  static constexpr int smem = kPart + TM * R * 4;
};

template <int R>
__global__ void __launch_bounds__(kRowThreads) k_adapter_contract(const __grid_constant__ RowsArgs g) {
  using S = ContractShape<R>;
  constexpr int TM = S::TM, CW = S::CW, PITCH = S::kPitch, PIECES = PITCH / 16, STEP = kRowThreads / PIECES;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int srow[TM];
  // largest values (bits) of the share's rows, of the ranks in it, and of the ranks by CTA
  __shared__ uint32_t rowmax[TM], rankmax[R], allmax[8][R];
  __shared__ __align__(16) float units[R];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cluster = g.cluster, rankc = blockIdx.x % cluster, tile_no = blockIdx.x / cluster;
  const RowsPass& a = g.pass[blockIdx.y];
  float* part = reinterpret_cast<float*>(smem + S::kPart);
  const uint32_t ring = smem_u32(smem);

  grid_dependency_wait();
  trigger_dependents();
  const int4 tile = g.tiles[tile_no];
  if (!takes_tile(g, tile_no, tile, true)) return;  // the whole cluster
  const int count = tile.z & (kCrowdTile - 1), slot = tile.x, r = g.rank[slot], r16 = (r + 15) & ~15;
  if (r == 0) return;
  if (tid < TM) srow[tid] = tid < count ? g.perm[tile.y + tid] : tile.w;
  for (int i = tid; i < TM + R; i += kRowThreads) (i < TM ? rowmax[i] : rankmax[i - TM]) = 0;
  const bool vec = (a.K & 7) == 0;
  const int kc = (a.K + CW - 1) / CW, nk = (kc - rankc + cluster - 1) / cluster;  // blocks in turn
  const float scale = g.scale[slot];
  __syncthreads();
  // this thread's 16-byte column and rows of a stage
  const int piece = tid % PIECES, row0 = tid / PIECES;
  const uint32_t spot = swz<PITCH>(row0, piece);
  const __half* wp = a.P + ((size_t)slot * g.rp + row0) * a.ld_p + 8 * piece;
  const __half* line[TM / STEP];
#pragma unroll
  for (int i = 0; i < TM / STEP; ++i) line[i] = a.in + (size_t)srow[row0 + STEP * i] * a.K;
  auto issue = [&](int i) {
    if (i < nk) {
      const uint32_t st = ring + (uint32_t)(i % S::kStages) * S::kStageBytes + spot;
      const int col = (i * cluster + rankc) * CW, c = col + 8 * piece;
      bool want[TM / STEP];
#pragma unroll
      for (int q = 0; q < TM / STEP; ++q) {
        want[q] = row0 + STEP * q < count && c < a.K;
        if (vec) cp_async16(st + STEP * q * PITCH, line[q] + (want[q] ? c : 0), want[q] ? 16 : 0);
      }
      if (!vec) {
        uint4 v[TM / STEP];
        read_pieces(v, line, want, c, a.K, a.in + (size_t)g.rows * a.K);
#pragma unroll
        for (int q = 0; q < TM / STEP; ++q) sts16(st + STEP * q * PITCH, v[q]);
      }
      const bool in = c < a.ld_p;
#pragma unroll
      for (int j = 0; j < (R + STEP - 1) / STEP; ++j)
        if (row0 + STEP * j < r16)
          cp_async16(st + S::kInBytes + STEP * j * PITCH, in ? wp + (size_t)(STEP * j) * a.ld_p + col : wp, in ? 16 : 0);
    }
    cp_async_commit();
  };
  for (int i = 0; i < S::kStages - 1; ++i) issue(i);

  const int rg = warp & 3, half = warp >> 2, g0 = lane >> 2, c0 = 2 * (lane & 3);
  // a long accumulation on the tensor cores is less exact than fp32 sums: every eight steps
  // the accumulators are added to sums of their own
  float acc[R / 8][4], sum[R / 8][4];
#pragma unroll
  for (int t = 0; t < R / 8; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[t][q] = sum[t][q] = 0.f;
  for (int i = 0; i < nk; ++i) {
    cp_async_wait<S::kStages - 2>();
    __syncthreads();
    issue(i + S::kStages - 1);
    const uint32_t st = ring + (uint32_t)(i % S::kStages) * S::kStageBytes;
#pragma unroll
    for (int kk = 0; kk < CW / 32; ++kk) {
      const int k16 = half * (CW / 32) + kk;
      uint32_t af[4];
      ldmatrix4(af, st + swz<PITCH>(rg * 16 + (lane & 15), 2 * k16 + (lane >> 4)));
#pragma unroll
      for (int t = 0; t < R / 16; ++t) {
        if (16 * t >= r16) break;
        uint32_t bf[4];
        ldmatrix4(bf, st + S::kInBytes + swz<PITCH>(16 * t + (lane & 7) + (lane >> 4) * 8, 2 * k16 + ((lane >> 3) & 1)));
        mma_16816(acc[2 * t], af, bf);
        mma_16816(acc[2 * t + 1], af, bf + 2);
      }
    }
    if ((i & 3) == 3 || i == nk - 1)
#pragma unroll
      for (int t = 0; t < R / 8; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) sum[t][q] += acc[t][q], acc[t][q] = 0.f;
  }
  // the CTA's sum: the second half of the steps, then the first on top
  float* mine = part + (rg * 16) * R;
#pragma unroll 1
  for (int h = 1; h >= 0; --h) {
    if (half == h)
#pragma unroll
      for (int t = 0; t < R / 8; ++t) {
        if (8 * t >= r16) break;
        float2* lo = reinterpret_cast<float2*>(mine + g0 * R + 8 * t + c0);
        float2* hi = reinterpret_cast<float2*>(mine + (g0 + 8) * R + 8 * t + c0);
        const float2 x = h ? make_float2(0.f, 0.f) : *lo, y = h ? make_float2(0.f, 0.f) : *hi;
        *lo = make_float2(sum[t][0] + x.x, sum[t][1] + x.y);
        *hi = make_float2(sum[t][2] + y.x, sum[t][3] + y.y);
      }
    __syncthreads();
  }
  cp_async_wait<0>();
  cluster_arrive();
  cluster_wait();
  // the cluster's sum of this CTA's share, CTAs in order: scale * T, zero past the rank
  float* own = reinterpret_cast<float*>(smem);  // [TM / cluster][R], over the drained ring
  const uint32_t pbase = smem_u32(part);
  const int share = TM / cluster, row_lo = rankc * share;
  // a thread's ranks are always the same four
  static_assert(4 * kRowThreads % R == 0, "ranks of a thread");
  const int j = 4 * tid % R;
  uint4 most = make_uint4(0, 0, 0, 0);
  for (int i = 4 * tid; i < share * R; i += 4 * kRowThreads) {
    const int row = row_lo + i / R;
    if (j >= r16 || row >= count) continue;
    const float4 x = sum_peers(pbase + 4 * (row * R + j), cluster);
    const float4 t = make_float4(j < r ? x.x * scale : 0.f, j + 1 < r ? x.y * scale : 0.f, j + 2 < r ? x.z * scale : 0.f,
                                 j + 3 < r ? x.w * scale : 0.f);
    *reinterpret_cast<float4*>(own + i) = t;
    const uint4 bits = finite_bits(t);
    if (a.parts) atomicMax(&rowmax[i / R], largest(bits));
    most = larger(most, bits);
  }
  if (a.gparts && j < r16) atomic_larger(rankmax + j, most);
  __syncthreads();
  if (a.gparts)
    for (int i = tid; i < r16 * cluster; i += kRowThreads)
      st_peer_u32(peer_smem(smem_u32(&allmax[rankc][i % r16]), i / r16), rankmax[i % r16]);
  cluster_arrive();
  auto value = [&](int i) { return row_lo + i / R < count ? *reinterpret_cast<const float4*>(own + i) : make_float4(0.f, 0.f, 0.f, 0.f); };
  auto at = [&](__half* parts, int i) { return parts + (size_t)(tile_no * TM + row_lo + i / R) * (2 * g.pp) + j; };
  if (a.parts) {
    for (int i = 4 * tid; i < share * R && j < r16; i += 4 * kRowThreads) {
      const float u = split_unit(__uint_as_float(rowmax[i / R]));
      write_parts(at(a.parts, i), g.pp, value(i), make_float4(u, u, u, u));
    }
    if (tid < share) a.unit[(size_t)tile_no * TM + row_lo + tid] = 1.f / split_unit(__uint_as_float(rowmax[tid]));
  }
  cluster_wait();
  if (a.gparts) {
    if (tid < r16) {
      units[tid] = rank_unit(&allmax[0][tid], R, cluster);
      if (rankc == 0) a.gunit[(size_t)tile_no * g.pp + tid] = 1.f / units[tid];
    }
    __syncthreads();
    const float4 u = *reinterpret_cast<const float4*>(units + j);
    for (int i = 4 * tid; i < share * R && j < r16; i += 4 * kRowThreads) write_parts(at(a.gparts, i), g.pp, value(i), u);
  }
}

// Expansion: a CTA takes some 128-column blocks of one tile; T's parts sit in MMA
// fragments throughout, the base tile and r rows of Q of the next blocks arrive (cp.async)
// while one is computed. The launches before are the contraction of the same call and, in a
// backward pass, the weight gradients: each lets the next one start only after its own dependency
// wait. All that was written before the call (plan, weights, base) is complete then, so it is
// read before this kernel's wait, and only T and the output come after it.
template <int R>
struct ExpandShape {
  static constexpr int TM = kWideRows, CW = 128, kPitch = 2 * CW;
  static constexpr int kStages = R <= 64 ? 3 : 2, kStageBytes = (TM + R) * kPitch;
  static constexpr int smem = kStages * kStageBytes;
};

template <int R>
__global__ void __launch_bounds__(kRowThreads, R <= 32 ? 3 : 2) k_adapter_expand(const __grid_constant__ RowsArgs g) {
  using S = ExpandShape<R>;
  constexpr int TM = S::TM, CW = S::CW, PITCH = S::kPitch;
  static_assert(kRowThreads == 16 * PITCH / 16, "a thread loads one 16-byte column of every 16th row");
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const RowsPass& a = g.pass[0];
  trigger_dependents();
  const int tile_no = blockIdx.y;
  const bool in_place = a.base == a.out;
  const int4 tile = __ldcg(g.tiles + tile_no);
  if (!takes_tile(g, tile_no, tile, in_place)) {
    grid_dependency_wait();
    return;
  }
  const int count = tile.z & (kCrowdTile - 1), slot = tile.x;
  const int r = slot < g.n_slots ? __ldcg(g.rank + slot) : 0, r16 = (r + 15) & ~15;
  const bool vec = (a.N & 7) == 0;
  // the CTAs of a tile take its column blocks in turn, so that they read and write
  // neighbouring parts of the rows at the same time
  const int blocks = (a.N + CW - 1) / CW, b0 = blockIdx.x, parts = gridDim.x, nb = (blocks - b0 + parts - 1) / parts;
  if (r == 0) {  // base alone
    grid_dependency_wait();
    if (!in_place)
      for (int b = b0; b < blocks; b += parts)
        copy_rows(a, g.rows, g.perm + tile.y, count, b * (CW / 8), min((b + 1) * (CW / 8), (a.N + 7) / 8));
    return;
  }
  const int piece = tid & 15, row0 = tid >> 4;
  const uint32_t spot = smem_u32(smem) + swz<PITCH>(row0, piece);
  int row[TM / 16];
#pragma unroll
  for (int i = 0; i < TM / 16; ++i) row[i] = row0 + 16 * i < count ? __ldcg(g.perm + tile.y + row0 + 16 * i) : -1;
  const __half* wq = a.Q + ((size_t)slot * g.rp + row0) * a.ld_q;
  auto issue = [&](int i) {
    if (i < nb) {
      const uint32_t dst = spot + (uint32_t)(i % S::kStages) * S::kStageBytes;
      const int c = (b0 + i * parts) * CW + 8 * piece;
      const bool inq = c < a.ld_q;
#pragma unroll
      for (int j = 0; j < R / 16; ++j)
        if (16 * j < r16) cp_async16(dst + (TM + 16 * j) * PITCH, wq + (inq ? (size_t)(16 * j) * a.ld_q + c : 0), inq ? 16 : 0);
      if (a.base) {
        const __half* line[TM / 16];
        bool want[TM / 16];
#pragma unroll
        for (int q = 0; q < TM / 16; ++q) {
          want[q] = row[q] >= 0 && c < a.N;
          line[q] = a.base + (size_t)max(row[q], 0) * a.N;
          if (vec) cp_async16(dst + 16 * q * PITCH, line[q] + (want[q] ? c : 0), want[q] ? 16 : 0);
        }
        if (!vec) {
          uint4 v[TM / 16];
          read_pieces(v, line, want, c, a.N, a.base + (size_t)g.rows * a.N);
#pragma unroll
          for (int q = 0; q < TM / 16; ++q) sts16(dst + 16 * q * PITCH, v[q]);
        }
      }
    }
    cp_async_commit();
  };
  for (int i = 0; i < S::kStages - 1; ++i) issue(i);
  grid_dependency_wait();
  const int rg = warp & 3, half = warp >> 2, g0 = rg * 16 + (lane >> 2), c0 = 2 * (lane & 3);
  uint32_t thi[R / 16][4], tlo[R / 16][4];
#pragma unroll
  for (int t = 0; t < R / 16; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const __half* at = a.parts + (size_t)(tile_no * TM + g0 + 8 * (q & 1)) * (2 * g.pp) + 16 * t + c0 + 8 * (q >> 1);
      const bool in = 16 * t < r16;
      thi[t][q] = in ? __ldcg(reinterpret_cast<const uint32_t*>(at)) : 0u;
      tlo[t][q] = in ? __ldcg(reinterpret_cast<const uint32_t*>(at + g.pp)) : 0u;
    }
  const float back[2] = {__ldcg(a.unit + (size_t)tile_no * TM + g0), __ldcg(a.unit + (size_t)tile_no * TM + g0 + 8)};
  constexpr int NT = CW / 16;  // 8-column tiles of a warp
  const int cw = 8 * NT * half;
  for (int i = 0; i < nb; ++i) {
    cp_async_wait<S::kStages - 2>();
    __syncthreads();
    issue(i + S::kStages - 1);
    const uint32_t off = (uint32_t)(i % S::kStages) * S::kStageBytes, st = smem_u32(smem) + off;
    float acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
#pragma unroll
    for (int t = 0; t < R / 16; ++t) {
      if (16 * t >= r16) break;
#pragma unroll
      for (int n = 0; n < NT / 2; ++n) {
        uint32_t bf[4];
        ldmatrix4_t(bf, st + swz<PITCH>(TM + 16 * t + (lane & 15), cw / 8 + 2 * n + (lane >> 4)));
        mma_16816(acc[2 * n], tlo[t], bf);
        mma_16816(acc[2 * n + 1], tlo[t], bf + 2);
        mma_16816(acc[2 * n], thi[t], bf);
        mma_16816(acc[2 * n + 1], thi[t], bf + 2);
      }
    }
    // base + acc, rounded once, over the base tile, then out in 16-byte pieces
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t at = st + swz<PITCH>(g0 + 8 * q, cw / 8 + n) + 2 * c0;
        const uint32_t bw = a.base ? lds_u32(at) : 0u;
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&bw));
        const __half2 o = __floats2half2_rn(fmaf(acc[n][2 * q], back[q], b.x), fmaf(acc[n][2 * q + 1], back[q], b.y));
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(*reinterpret_cast<const uint32_t*>(&o)) : "memory");
      }
    __syncthreads();
    const int c = (b0 + i * parts) * CW + 8 * piece;
#pragma unroll
    for (int q = 0; q < TM / 16; ++q)
      if (row[q] >= 0) write_piece(a.out + (size_t)row[q] * a.N, c, a.N, vec, lds_u32x4(spot + off + 16 * q * PITCH));
  }
  cp_async_wait<0>();
}

// ---- weight gradients --------------------------------------------------------------------
// G_s[j][i] (+)= sum over the slot's rows of (scale T)[p][j] In[row p][i]: r x rows by
// rows x kGradCols. A CTA owns kGradCols columns of one slot's gradient; a cluster
// splits the slot's 64-row tiles and sums through distributed shared memory in rank
// order. Per tile the products of T's two parts are accumulated by the MMA and then
// added, times the rank's unit, to fp32 sums: a long sum is rounded to nearest once a
// tile, not truncated at each MMA.
constexpr int kGradThreads = 256;

template <int R>
struct GradShape {
  static constexpr int kStages = 3, kInPitch = 2 * kGradCols, kTPitch = 2 * R;
  static constexpr int kInBytes = 64 * kInPitch, kTBytes = 64 * kTPitch;
  static constexpr int kStageBytes = kInBytes + 2 * kTBytes;
  static constexpr int smem = kStages * kStageBytes > R * kGradCols * 4 ? kStages * kStageBytes : R * kGradCols * 4;
};

template <int R>
__global__ void __launch_bounds__(kGradThreads) k_adapter_grad(const __grid_constant__ GradArgs g) {
  using S = GradShape<R>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = blockIdx.z, nsplit = gridDim.z, slot = grad_slot(g);
  const int which = (int)blockIdx.x < g.pass[0].blocks ? 0 : 1;
  const GradPass& a = g.pass[which];
  const int col0 = ((int)blockIdx.x - (which ? g.pass[0].blocks : 0)) * kGradCols;
  const uint32_t ring = smem_u32(smem);
  if (slot < 0) {
    grid_dependency_wait();
    return;
  }
  const int p0 = __ldcg(g.start + slot), rows = __ldcg(g.start + slot + 1) - p0, tile0 = __ldcg(g.first64 + slot);
  const int r = rows ? __ldcg(g.rank + slot) : 0, r16 = (r + 15) & ~15;
  float* out = a.g + (size_t)slot * g.max_rank * a.K;
  const int width = min(kGradCols, a.K - col0);
  if (r == 0) {
    grid_dependency_wait();
    if (!g.zeroed && !g.accumulate) zero_columns(out + col0, a.K, width, g.max_rank, split, nsplit);
    return;
  }
  const int nt_all = (rows + 63) / 64, t_lo = (int)((long)nt_all * split / nsplit);
  const int nt = (int)((long)nt_all * (split + 1) / nsplit) - t_lo;
  const bool vec = (a.K & 7) == 0;
  // this thread's 16-byte column and rows of a stage; the row numbers of the next stage
  // to be issued are loaded one stage ahead
  const int piece = tid & 15, row0 = tid >> 4, col = col0 + 8 * piece;
  const uint32_t spot = swz<S::kInPitch>(row0, piece);
  int next[4];
  auto fetch = [&](int i) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int p = (t_lo + i) * 64 + row0 + 16 * q;
      next[q] = i < nt && p < rows ? __ldcg(g.perm + p0 + p) : -1;
    }
  };
  auto issue_in = [&](int i) {
    if (i < nt) {
      const uint32_t st = ring + (uint32_t)(i % S::kStages) * S::kStageBytes;
      const __half* line[4];
      bool want[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        want[q] = next[q] >= 0 && col < a.K;
        line[q] = a.in + (size_t)max(next[q], 0) * a.K;
        if (vec) cp_async16(st + spot + 16 * q * S::kInPitch, line[q] + (want[q] ? col : 0), want[q] ? 16 : 0);
      }
      if (!vec) {
        uint4 v[4];
        read_pieces(v, line, want, col, a.K, a.in + (size_t)g.n_rows * a.K);
#pragma unroll
        for (int q = 0; q < 4; ++q) sts16(st + spot + 16 * q * S::kInPitch, v[q]);
      }
      fetch(i + 1);
    }
  };
  auto issue_t = [&](int i) {
    if (i < nt) {
      const uint32_t st = ring + (uint32_t)(i % S::kStages) * S::kStageBytes;
      constexpr int pieces = R / 8;
#pragma unroll
      for (int q = tid; q < 64 * pieces; q += kGradThreads) {
        const int row = q / pieces, c = q % pieces;
        if (8 * c >= r16) continue;
        const __half* at = a.parts + (size_t)((tile0 + t_lo + i) * kWideRows + row) * (2 * g.pp) + 8 * c;
        const uint32_t dst = st + S::kInBytes + swz<S::kTPitch>(row, c);
        cp_async16(dst, at, 16);
        cp_async16(dst + S::kTBytes, at + g.pp, 16);
      }
    }
    cp_async_commit();
  };
  fetch(0);
  for (int i = 0; i < S::kStages - 1; ++i) issue_in(i);
  grid_dependency_wait();  // T is the call's own; the rest was there before the call
  trigger_dependents();    // the expansion's first loads may go out
  for (int i = 0; i < S::kStages - 1; ++i) issue_t(i);
  float ahead[R / 16][2];  // the units of this thread's ranks, a tile ahead
  auto fetch_units = [&](int i) {
#pragma unroll
    for (int t = 0; t < R / 16; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        ahead[t][h] = i < nt && 16 * t < r16 ? __ldcg(a.unit + (size_t)(tile0 + t_lo + i) * g.pp + 16 * t + 8 * h + (lane >> 2)) : 0.f;
  };
  fetch_units(0);
  float sum[R / 16][2][4];
#pragma unroll
  for (int t = 0; t < R / 16; ++t)
#pragma unroll
    for (int n = 0; n < 2; ++n) sum[t][n][0] = sum[t][n][1] = sum[t][n][2] = sum[t][n][3] = 0.f;
  for (int i = 0; i < nt; ++i) {
    cp_async_wait<S::kStages - 2>();
    __syncthreads();
    issue_in(i + S::kStages - 1);
    issue_t(i + S::kStages - 1);
    const uint32_t st = ring + (uint32_t)(i % S::kStages) * S::kStageBytes;
    float back[R / 16][2];
#pragma unroll
    for (int t = 0; t < R / 16; ++t) back[t][0] = ahead[t][0], back[t][1] = ahead[t][1];
    fetch_units(i + 1);
    uint32_t bf[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      ldmatrix4_t(bf[k], st + swz<S::kInPitch>(16 * k + (lane & 15), 2 * warp + (lane >> 4)));
#pragma unroll
    for (int t = 0; t < R / 16; ++t) {
      if (16 * t >= r16) break;
      float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t hi[4], lo[4];
        const uint32_t at = st + S::kInBytes + swz<S::kTPitch>(16 * k + (lane & 7) + 8 * (lane >> 4), 2 * t + ((lane >> 3) & 1));
        ldmatrix4_t(hi, at);
        ldmatrix4_t(lo, at + S::kTBytes);
        mma_16816(acc[0], lo, bf[k]);
        mma_16816(acc[1], lo, bf[k] + 2);
        mma_16816(acc[0], hi, bf[k]);
        mma_16816(acc[1], hi, bf[k] + 2);
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) sum[t][n][q] = fmaf(acc[n][q], back[t][q >> 1], sum[t][n][q]);
    }
  }
  cp_async_wait<0>();
  __syncthreads();
  float* part = reinterpret_cast<float*>(smem);  // [R][kGradCols], over the drained ring
  const int g0 = lane >> 2, c0 = 16 * warp + 2 * (lane & 3);
#pragma unroll
  for (int t = 0; t < R / 16; ++t)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        *reinterpret_cast<float2*>(part + (16 * t + g0 + 8 * q) * kGradCols + c0 + 8 * n) =
            make_float2(sum[t][n][2 * q], sum[t][n][2 * q + 1]);
  if (nsplit > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  // this CTA's share of the gradient's rows; rows past the rank are zero
  const uint32_t pbase = smem_u32(part);
  for (int i = split * kGradThreads + tid; i < g.max_rank * (kGradCols / 4); i += nsplit * kGradThreads) {
    const int j = i / (kGradCols / 4), c = 4 * (i % (kGradCols / 4));
    if (c >= width) continue;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (j < r)
      for (int s = 0; s < nsplit; ++s) {
        const float4 y = nsplit > 1 ? ld_peer_v4f(peer_smem(pbase + 4 * (j * kGradCols + c), s)) : *reinterpret_cast<const float4*>(part + j * kGradCols + c);
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
      }
    float* dst = out + (size_t)j * a.K + col0 + c;
    if ((a.K & 3) == 0) {
      if (g.accumulate) {
        const float4 y = *reinterpret_cast<const float4*>(dst);
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
      }
      *reinterpret_cast<float4*>(dst) = x;
    } else {
      const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < width) dst[e] = g.accumulate ? dst[e] + v[e] : v[e];
    }
  }
  if (nsplit > 1) {
    cluster_arrive();
    cluster_wait();
  }
}

// Few rows: the gradient is mostly its own output. A thread sums eight ranks of four columns
// over the slot's rows, in plan order, in fp32; a slot without rows gets its zeros the same way.
constexpr int kFewGradThreads = 128, kFewGradRanks = 8, kFewGradCols = 4 * kFewGradThreads;

__global__ void __launch_bounds__(kFewGradThreads) k_grad_few(const __grid_constant__ GradArgs g) {
  const int which = (int)blockIdx.x < g.pass[0].blocks ? 0 : 1, slot = blockIdx.y, j0 = blockIdx.z * kFewGradRanks;
  const GradPass& a = g.pass[which];
  const int c = ((int)blockIdx.x - (which ? g.pass[0].blocks : 0)) * kFewGradCols + 4 * threadIdx.x;
  // what the call found is read before the wait on its first kernel (see the expansion)
  trigger_dependents();
  const int p0 = __ldcg(g.start + slot), r = __ldcg(g.rank + slot), p1 = r > j0 && __ldcg(g.planned) <= g.n_rows ? __ldcg(g.start + slot + 1) : p0;
  const bool vec = (a.K & 3) == 0;
  // eight rows at a time, their loads together: one row's took 0.6 us after the other's
  constexpr int kAhead = 8;
  uint2 x[kAhead];
  auto fetch = [&](int p) {
    int row[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) row[q] = __ldcg(g.perm + min(p + q, p1 - 1));
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const __half* h = a.in + (size_t)row[q] * a.K + c;
      x[q] = make_uint2(0, 0);
      if (p + q >= p1 || c >= a.K) continue;
      if (vec) {
        x[q] = __ldcg(reinterpret_cast<const uint2*>(h));
      } else {
        const unsigned short* u = reinterpret_cast<const unsigned short*>(h);
        const unsigned short e0 = __ldcg(u), e1 = c + 1 < a.K ? __ldcg(u + 1) : 0;
        const unsigned short e2 = c + 2 < a.K ? __ldcg(u + 2) : 0, e3 = c + 3 < a.K ? __ldcg(u + 3) : 0;
        x[q] = make_uint2((uint32_t)e0 | (uint32_t)e1 << 16, (uint32_t)e2 | (uint32_t)e3 << 16);
      }
    }
  };
  if (p0 < p1) fetch(p0);
  float acc[kFewGradRanks][4];
#pragma unroll
  for (int j = 0; j < kFewGradRanks; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
  grid_dependency_wait();
  for (int p = p0; p < p1; p += kAhead) {
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      // past the end x is 0 beside a repeated row's T
      const float4* t = reinterpret_cast<const float4*>(a.sums + (size_t)min(p + q, p1 - 1) * g.pp + j0);
      const float4 t0 = __ldcg(t), t1 = __ldcg(t + 1);
      const float tv[kFewGradRanks] = {t0.x, t0.y, t0.z, t0.w, t1.x, t1.y, t1.z, t1.w};
      const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&x[q].x)), hi = __half22float2(*reinterpret_cast<const __half2*>(&x[q].y));
#pragma unroll
      for (int j = 0; j < kFewGradRanks; ++j) {
        acc[j][0] = fmaf(tv[j], lo.x, acc[j][0]), acc[j][1] = fmaf(tv[j], lo.y, acc[j][1]);
        acc[j][2] = fmaf(tv[j], hi.x, acc[j][2]), acc[j][3] = fmaf(tv[j], hi.y, acc[j][3]);
      }
    }
    if (p + kAhead < p1) fetch(p + kAhead);
  }
  if (c >= a.K) return;
  float* out = a.g + (size_t)slot * g.max_rank * a.K + c;
#pragma unroll
  for (int j = 0; j < kFewGradRanks; ++j) {
    if (j0 + j >= g.max_rank) break;
    float* dst = out + (size_t)(j0 + j) * a.K;
    const bool add = g.accumulate && j0 + j < r && p0 < p1;
    if (g.accumulate && !add) continue;
    if (vec) {
      float4 x = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
      if (add) {
        const float4 y = *reinterpret_cast<const float4*>(dst);
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
      }
      *reinterpret_cast<float4*>(dst) = x;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < a.K) dst[e] = add ? dst[e] + acc[j][e] : acc[j][e];
    }
  }
}

// Zeros in the gradients of slots without rows or rank (of several): most slots of a large
// pool, which the gradient kernels' large CTAs would take waves for.
__global__ void __launch_bounds__(256) k_zero_unused(const __grid_constant__ GradArgs g) {
  grid_dependency_wait();
  trigger_dependents();
  const int slot = blockIdx.y;
  if (g.start[slot + 1] > g.start[slot] && g.rank[slot] > 0) return;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const size_t n = (size_t)g.max_rank * g.pass[i].K;
    float* out = g.pass[i].g + slot * n;
    const size_t first = (size_t)blockIdx.x * 256 + threadIdx.x, step = (size_t)gridDim.x * 256;
    if ((n & 3) == 0)
      for (size_t e = first; e < n / 4; e += step) reinterpret_cast<float4*>(out)[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    else
      for (size_t e = first; e < n; e += step) out[e] = 0.f;
  }
}

// ---- launches --------------------------------------------------------------------------
cudaError_t launch_pdl(const void* fn, dim3 grid, dim3 block, size_t smem, cudaStream_t stream, void** args,
                       dim3 cluster = dim3(1, 1, 1)) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster.x;
  attr[1].val.clusterDim.y = cluster.y;
  attr[1].val.clusterDim.z = cluster.z;
  cfg.attrs = attr;
  cfg.numAttrs = cluster.x * cluster.y * cluster.z > 1 ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

RowsArgs rows_args(const dictproj_adapters* a, const dictproj_rows* r, bool wide) {
  RowsArgs g = {};
  g.n_tiles = r->n_tiles + (wide ? 2 : 0);
  g.planned = r->n_tiles + 7;
  g.tiles = r->tiles[wide];
  g.perm = r->perm;
  g.rank = a->rank;
  g.scale = a->scale;
  g.rp = a->rp;
  g.pp = a->pp;
  g.n_slots = a->n_slots;
  g.rows = r->M;
  g.only = -1;
  g.cluster = kCluster;
  return g;
}
RowsPass rows_pass(const dictproj_adapters* a, bool forward, const __half* in, const __half* base, __half* out) {
  const __half* A = reinterpret_cast<const __half*>(a->A);
  const __half* B = reinterpret_cast<const __half*>(a->B);
  RowsPass p = {};
  p.in = in;
  p.base = base;
  p.out = out;
  p.P = forward ? A : B;
  p.Q = forward ? B : A;
  p.K = forward ? a->d_in : a->d_out;
  p.N = forward ? a->d_out : a->d_in;
  p.ld_p = forward ? a->d_in : a->ld_b;
  p.ld_q = forward ? a->ld_b : a->d_in;
  return p;
}
// The kernel of the smallest template rank that holds rp ranks.
#define DICTPROJ_BY_RANK(rp, call) \
  ((rp) <= 16 ? call(16) : (rp) <= 32 ? call(32) : (rp) <= 64 ? call(64) : call(128))

cudaError_t launch_few(const RowsArgs& g, int passes, const dictproj_rows* r, cudaStream_t stream) {
  void* args[] = {(void*)&g};
  const bool vec = ((g.pass[0].K | g.pass[0].N) & 7) == 0;
#define FEW(R) (vec ? (const void*)k_adapter_few<R, true> : (const void*)k_adapter_few<R, false>)
  return launch_pdl(DICTPROJ_BY_RANK(g.rp, FEW), dim3((unsigned)(adapter_tiles(r->M, r->n_slots, kFewRows) * kCluster), passes),
                    dim3(kRowThreads), 0, stream, args, dim3(kCluster, 1, 1));
#undef FEW
}
cudaError_t launch_contract(RowsArgs& g, int passes, bool exact_sums, const dictproj_adapters* pool, const dictproj_rows* r, cudaStream_t stream) {
  const int n_sm = pool->n_sm;
  if (tall_serves(pool, r)) return launch_contract_tall(g, passes, exact_sums, pool, r, stream);
  const int tiles = adapter_tiles(r->M, r->n_slots, kWideRows);
  const int full = r->M / kWideRows * passes;  // tiles that do exist, about
  g.cluster = 2;
  while (g.cluster < 8 && full * g.cluster < 2 * n_sm) g.cluster *= 2;
  void* args[] = {(void*)&g};
#define FN(R) (const void*)k_adapter_contract<R>
#define SMEM(R) ContractShape<R>::smem
  return launch_pdl(DICTPROJ_BY_RANK(g.rp, FN), dim3((unsigned)(tiles * g.cluster), passes), dim3(kRowThreads),
                    DICTPROJ_BY_RANK(g.rp, SMEM), stream, args, dim3(g.cluster, 1, 1));
#undef FN
#undef SMEM
}
cudaError_t launch_expand(const RowsArgs& g, const dictproj_adapters* pool, const dictproj_rows* r, cudaStream_t stream) {
  if (tall_serves(pool, r)) return launch_expand_tall(g, pool, r, stream);
  const int n_sm = pool->n_sm;
  const int tiles = adapter_tiles(r->M, r->n_slots, kWideRows), blocks = (g.pass[0].N + 127) / 128;
  const int full = std::max(1, r->M / kWideRows);  // tiles that do exist, about
  // as many CTAs as run at once (two an SM above rank 32): 2048 rows of rank 32 took 22.3 us
  // with three an SM, 24.1 with two, 26 with more than four
  const int parts = std::min(blocks, std::max(1, (g.rp <= 32 ? 3 : 2) * n_sm / full));
  void* args[] = {(void*)&g};
#define FN(R) (const void*)k_adapter_expand<R>
#define SMEM(R) ExpandShape<R>::smem
  return launch_pdl(DICTPROJ_BY_RANK(g.rp, FN), dim3(parts, tiles), dim3(kRowThreads),
                    DICTPROJ_BY_RANK(g.rp, SMEM), stream, args);
#undef FN
#undef SMEM
}

template <int R>
cudaError_t launch_grad(const GradArgs& args, dim3 grid, cudaStream_t stream) {
  void* a[] = {(void*)&args};
  return launch_pdl((const void*)k_adapter_grad<R>, grid, dim3(kGradThreads), GradShape<R>::smem, stream, a,
                    dim3(1, 1, grid.z));
}

template <int R>
cudaError_t allow_rank() {
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(k_adapter_contract<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, ContractShape<R>::smem)) ||
      (e = cudaFuncSetAttribute(k_adapter_expand<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, ExpandShape<R>::smem)))
    return e;
  return cudaFuncSetAttribute(k_adapter_grad<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, GradShape<R>::smem);
}

}  // namespace

cudaError_t prepare_adapter_kernels(int device) {
  (void)device;
  cudaError_t e;
  if ((e = allow_rank<16>()) || (e = allow_rank<32>()) || (e = allow_rank<64>()) || (e = allow_rank<128>())) return e;
  return cudaFuncSetAttribute(k_rows_plan, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (kPlanWarps + 4) * (DICTPROJ_MAX_SLOTS + 2) * (int)sizeof(int));
}

cudaError_t launch_adapter_set(const dictproj_adapters* a, int slot, int rank, float scale, const __half* A,
                               const __half* B, cudaStream_t stream) {
  uint16_t* sa = a->A + (size_t)slot * a->rp * a->d_in;
  uint16_t* sb = a->B + (size_t)slot * a->rp * a->ld_b;
  int* sr = a->rank + slot;
  float* ss = a->scale + slot;
  int rp = a->rp, d_in = a->d_in, d_out = a->d_out, ld_b = a->ld_b;
  void* args[] = {&A, &B, &rank, &scale, &rp, &d_in, &d_out, &ld_b, &sa, &sb, &sr, &ss};
  return launch_pdl((const void*)k_adapter_set, dim3(a->rp, (std::max(d_in, ld_b) + kSetCols - 1) / kSetCols), dim3(256), 0,
                    stream, args);
}

cudaError_t launch_rows_plan(const dictproj_rows* r, const int* ids, int M, cudaStream_t stream) {
  int ns = r->n_slots;
  void* args[] = {&ids, &M, &ns, (void*)&r->perm, (void*)&r->start, (void*)&r->n_tiles, (void*)&r->tiles[0],
                  (void*)&r->tiles[1], (void*)&r->tiles[2], (void*)&r->runs[0], (void*)&r->runs[1],
                  (void*)&r->first64, (void*)&r->used};
  return launch_pdl((const void*)k_rows_plan, dim3(1), dim3(kPlanWarps * 32),
                    ((size_t)kPlanWarps * (ns + 1) + 4 * (ns + 2)) * sizeof(int), stream, args);
}

// What a contraction leaves: pass 0 for an expansion, both passes for the weight gradients.
static void set_parts(const dictproj_adapters* a, RowsArgs& g, bool expand, bool grads) {
  if (expand) {
    g.pass[0].parts = reinterpret_cast<__half*>(a->parts);
    g.pass[0].unit = a->unit;
  }
  for (int i = 0; i < 2 && grads; ++i) {
    g.pass[i].gparts = reinterpret_cast<__half*>(a->gparts[i]);
    g.pass[i].gunit = a->gunit[i];
  }
}

cudaError_t launch_adapter_forward(const dictproj_adapters* a, const dictproj_rows* r, const __half* X,
                                   const __half* base, __half* Y, cudaStream_t stream) {
  // A slot's rows go to the kernels of few rows up to kCrowd of them, to those of many rows
  // above. The host knows how many rows there are, not how they fall on the slots. From
  // kCrowd rows a slot on average the second kind takes every slot (4096 -> 4096, one slot
  // of rank 64: 192 rows 22.4 us by the first kind, 12.3 by the second; 128 rows 12.5 and
  // 12.2; rank 16: 256 rows 10.0 and 9.1, 384 rows 16.4 and 9.3). With fewer on average,
  // both kinds run and each takes its slots, which their launches have to be worth: 16 slots
  // of rank 64 took 32 us by the first kind alone at 256 rows and 39 by both, at 512 rows 64
  // and 24.
  const int many_rows = a->rp <= 16 ? 256 : 192;
  const bool all = r->M >= many_rows && r->M >= kCrowd * a->n_slots, many = all || r->M >= 512;
  cudaError_t e = cudaSuccess;
  if (!all) {
    RowsArgs g = rows_args(a, r, false);
    g.pass[0] = rows_pass(a, true, X, base, Y);
    if (many) g.only = 0;
    e = launch_few(g, 1, r, stream);
  }
  if (e != cudaSuccess || !many) return e;
  RowsArgs g = rows_args(a, r, true);
  g.pass[0] = rows_pass(a, true, X, base, Y);
  if (!all) g.only = 1;
  set_parts(a, g, true, false);
  e = launch_contract(g, 1, false, a, r, stream);
  return e == cudaSuccess ? launch_expand(g, a, r, stream) : e;
}

static cudaError_t launch_grads(const GradArgs& w, const dictproj_adapters* a, const dictproj_rows* r, int slots,
                                cudaStream_t stream) {
  if (tall_serves(a, r)) return launch_grad_tall(w, a, r, stream);
  const int blocks = w.pass[0].blocks + w.pass[1].blocks;
  int split = 1;
  while (split < 8 && blocks * slots * split < 3 * a->n_sm && 64 * slots * split < r->M) split *= 2;
  const dim3 grid(blocks, slots, split);
  if (a->rp <= 16) return launch_grad<16>(w, grid, stream);
  if (a->rp <= 32) return launch_grad<32>(w, grid, stream);
  if (a->rp <= 64) return launch_grad<64>(w, grid, stream);
  return launch_grad<128>(w, grid, stream);
}

cudaError_t launch_adapter_backward(const dictproj_adapters* a, const dictproj_rows* r, const __half* X,
                                    const __half* dY, const __half* base, __half* dX, float* dA, float* dB,
                                    bool accumulate, cudaStream_t stream) {
  RowsArgs g = rows_args(a, r, true);
  g.pass[0] = rows_pass(a, false, dY, base, dX);
  g.pass[1] = rows_pass(a, true, X, nullptr, nullptr);
  set_parts(a, g, dX != nullptr, dA != nullptr);
  GradArgs w = {};
  for (int i = 0; i < 2; ++i) {
    w.pass[i].in = i ? dY : X;
    w.pass[i].parts = g.pass[i].gparts;
    w.pass[i].unit = g.pass[i].gunit;
    w.pass[i].g = i ? dB : dA;
    w.pass[i].K = i ? a->d_out : a->d_in;
    w.pass[i].blocks = (w.pass[i].K + kGradCols - 1) / kGradCols;
  }
  w.start = r->start;
  w.first64 = r->first64;
  w.runs = r->runs[0];
  w.perm = r->perm;
  w.rank = a->rank;
  w.rp = a->rp;
  w.pp = a->pp;
  w.max_rank = a->max_rank;
  w.accumulate = accumulate;
  w.n_rows = r->M;
  w.used = r->used;
  w.n_used = r->n_tiles + 6;
  w.planned = r->n_tiles + 7;
  w.zeroed = a->n_slots > 1;
  // The kernels of few rows, both contractions and dX in one launch, for some rows a slot
  // (4096 and 4096 wide, rank 16: 1 slot 8 rows 8.5 us against 10.5, 32 rows 15.6 against
  // 10.7; 16 slots 64 rows 16.7 against 23.3, 128 rows 23.1 and 23.8).
  if (r->M <= std::min(128, 12 + 4 * a->n_slots)) {
    RowsArgs f = rows_args(a, r, false);
    for (int i = 0; i < 2; ++i) {
      f.pass[i] = g.pass[i];
      w.pass[i].sums = f.pass[i].sums = dA ? reinterpret_cast<float*>(a->gparts[i]) : nullptr;
      w.pass[i].blocks = (w.pass[i].K + kFewGradCols - 1) / kFewGradCols;
    }
    const cudaError_t e = launch_few(f, dA ? 2 : 1, r, stream);
    if (e != cudaSuccess || !dA) return e;
    void* args[] = {(void*)&w};
    return launch_pdl((const void*)k_grad_few,
                      dim3(w.pass[0].blocks + w.pass[1].blocks, a->n_slots, (a->max_rank + kFewGradRanks - 1) / kFewGradRanks),
                      dim3(kFewGradThreads), 0, stream, args);
  }
  const int slots = std::min(a->n_slots, r->M);  // that can have rows
  if (dA && w.zeroed && !accumulate) {
    void* args[] = {(void*)&w};
    const size_t most = (size_t)a->max_rank * std::max(a->d_in, a->d_out) / 4;
    const int per = (int)std::min<size_t>(std::max(1, 8 * a->n_sm / a->n_slots), most / 1024 + 1);
    const cudaError_t z = launch_pdl((const void*)k_zero_unused, dim3(per, a->n_slots), dim3(256), 0, stream, args);
    if (z != cudaSuccess) return z;
  }
  // The gradients before the expansion, whose first loads (base and weights) then go out while
  // the gradients end (2048 rows, 4096 and 11008 wide: 41.6 us, the other way round 44.8). T is the
  // call's own, and whoever reads it waits for it himself: an expansion that read it as soon as the
  // gradients released it, on the strength of their wait, took 2 us of 112 less at 8192 rows and 4
  // of 26 at 5461 rows of 416 and 856 columns. What was there before the call is complete when a
  // launch behind the contraction starts; reading that, too, behind the wait alone costs 21.2 ->
  // 23.8 us (forward, 2048 rows) and 41.5 -> 45.5 us (backward).
  cudaError_t e = launch_contract(g, dA ? 2 : 1, dA != nullptr, a, r, stream);
  if (e == cudaSuccess && dA) e = launch_grads(w, a, r, slots, stream);
  if (e != cudaSuccess || !dX) return e;
  return launch_expand(g, a, r, stream);
}

}  // namespace dictproj
