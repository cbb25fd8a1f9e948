// Adapters of many rows on the 5th-generation tensor cores: the contraction T = X A^T, the
// expansion base + T B and the weight gradients T^T X, for row lengths that TMA can read
// (multiples of 8).
//
// All three stream the activations once for few operations, so the aim is to move them with
// as few instructions as can be: the rows of a tile arrive by TMA (128-byte swizzle) and
// are multiplied by one thread's tcgen05.mma; the mma.sync kernels of adapter.cu, which
// serve the other row lengths, spend 28 M warp instructions where these need 9 M (8192
// rows of 4096, rank 64, both contractions). Rows that follow one another in the batch
// (a sequence's) come as one box, others by gathers of four rows, which move about 6 bytes
// a clock and SM: both contractions of 2048 rows (4096 + 11008 wide) took 38 us by gathers
// alone. A slot's rows ascend in the plan, so they follow one another when the last is as
// far from the first as there are rows between.
//
// Every spin-wait is bounded; a wait that gives up sets the file's device error word and
// the kernel unwinds (frees its tensor memory) without hanging.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <utility>

#include "adapter.cuh"
#include "common.cuh"
#include "dictproj_internal.h"
#include "kernels.h"
#include "tcgen05.cuh"

namespace dictproj {
namespace {

constexpr int kTallThreads = 192;  // warp 0 TMA, warp 1 MMA + tensor memory, warps 2..5 epilogue
constexpr int kExpandThreads = 320;  // the expansion: eight epilogue warps, 2..9
constexpr int kCols = 64;          // columns of a stage (one 128-byte swizzle row)

// ---- contraction -------------------------------------------------------------------------
// A cluster splits the K columns of one tile of up to 128 rows of one slot. Per 64-column
// stage 128 gathered rows of In (16 KB) and r rows of P_s; D = In P^T, rows x r, in tensor
// memory. The CTAs' partial sums meet through distributed shared memory, in rank order;
// each CTA writes its share of the rows as two fp16 parts, with a unit for each row and, for
// the weight gradients, once more with one for each rank of 64 rows.
// A long accumulation on the tensor cores is less exact than fp32 sums: with all of K in one
// accumulator the weight gradients of 2048 rows came out more than 1e-6 off (relative norm).
// For them every `flush` stages get an accumulator of their own (two in turn), which the
// epilogue warps add in fp32 (3e-7, at no cost in time); the forward's fp16 result takes one
// for all.
struct TallContractArgs {
  CUtensorMap in[2], box[2], p[2];  // In by single rows and by 64, P by 16
  RowsArgs g;
  int stages, flush;
};

constexpr int kMaxStages = 12;

template <int R>
struct TallContract {
  static constexpr int kInBytes = kTallRows * 128, kStageBytes = kInBytes + R * 128;
  static constexpr int kPitch = R + 4;  // floats of a row of the partial sums, which lie over the drained ring
  static constexpr int kPart = kTallRows * kPitch * 4;
  // behind the ring, largest values (bits) of the share's rows [64] and of the ranks in it [R], of
  // the ranks by CTA [4][R] (those of 64 rows are half a cluster), and the ranks' units [R]
  static constexpr int kFixed = (kWideRows + 6 * R) * 4;
  static constexpr int kTmem = 2 * R;
};

template <int R>
__global__ void __launch_bounds__(kTallThreads) k_contract_tall(const __grid_constant__ TallContractArgs args) {
  using S = TallContract<R>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], dfull[2], dempty[2];
  __shared__ uint32_t tmem_slot;
  const RowsArgs& g = args.g;
  const RowsPass& a = g.pass[blockIdx.y];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, stages = args.stages;
  const int cluster = g.cluster, rankc = blockIdx.x % cluster, tile_no = blockIdx.x / cluster;
  uint32_t* rowmax = reinterpret_cast<uint32_t*>(smem + stages * S::kStageBytes);
  uint32_t *rankmax = rowmax + kWideRows, *allmax = rankmax + R;
  float* units = reinterpret_cast<float*>(allmax + 4 * R);
  for (int i = threadIdx.x; i < kWideRows + R; i += kTallThreads) rowmax[i] = 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 2);  // In's bytes and P's are announced apart
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&dfull[s], 1);
      mbar_init(&dempty[s], 4);
    }
    fence_mbar_init();
    tma_prefetch_map(&args.box[blockIdx.y]);
    tma_prefetch_map(&args.p[blockIdx.y]);
  }
  if (warp == 1) tmem_alloc(&tmem_slot, S::kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  grid_dependency_wait();
  trigger_dependents();  // not before the tensor memory is ours: a dependent may want all of it
  const int4 tile = g.tiles[tile_no];
  const int run_row = g.runs[tile_no];
  const bool live = takes_tile(g, tile_no, tile, true);
  const int count = tile.z & (kCrowdTile - 1), slot = tile.x;
  // the cluster's CTAs take the column blocks in turn, so that they read neighbouring parts
  // of the rows at the same time
  const int kc = (a.K + kCols - 1) / kCols, nk = (kc - rankc + cluster - 1) / cluster;
  // In's first stages are on their way before the rank is known
  const bool run = run_row >= 0;
  const int boxes = run ? (count + kWideRows - 1) / kWideRows : 0, first = min(stages, nk);
  int row[4] = {0, 0, 0, 0};
  auto load_in = [&](int s) {
    const uint32_t st = smem_u32(smem + s % stages * S::kStageBytes);
    const int x = (s * cluster + rankc) * kCols;
    uint64_t* bar = &full[s % stages];
    if (lane == 0) mbar_arrive_expect_tx(bar, run ? boxes * kWideRows * 128 : S::kInBytes);
    __syncwarp();
    if (!run) tma_gather4(st + 512 * lane, &args.in[blockIdx.y], x, row[0], row[1], row[2], row[3], bar);
    else if (lane < boxes) tma_load_2d(st + 8192 * lane, &args.box[blockIdx.y], x, run_row + kWideRows * lane, bar);
  };
  if (warp == 0 && live) {
    if (!run)  // lane l gathers rows 4 l .. 4 l + 3 of the tile; past its end any row will do
#pragma unroll
      for (int q = 0; q < 4; ++q) row[q] = g.perm[tile.y + min(4 * lane + q, count - 1)];
    for (int s = 0; s < first; ++s) load_in(s);
  }
  const int r = live ? g.rank[slot] : 0, r16 = (r + 15) & ~15;
  if (r == 0) {  // no tile, or an empty slot's (the whole cluster): what was asked for has to land
    if (warp == 0 && live && lane == 0)
      for (int s = 0; s < first; ++s) {
        mbar_arrive(&full[s]);
        mbar_wait_bounded(&full[s], 0);
      }
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, S::kTmem);
    return;
  }
  const float scale = g.scale[slot];

  if (warp == 0) {
    auto load_p = [&](int s) {
      uint64_t* bar = &full[s % stages];
      if (lane == 0) mbar_arrive_expect_tx(bar, r16 * 128);
      __syncwarp();
      if (lane < r16 / 16)
        tma_load_2d(smem_u32(smem + s % stages * S::kStageBytes) + S::kInBytes + 2048 * lane, &args.p[blockIdx.y],
                    (s * cluster + rankc) * kCols, slot * g.rp + 16 * lane, bar);
    };
    for (int s = 0; s < first; ++s) load_p(s);
    for (int s = first; s < nk; ++s) {
      bool ok = true;
      if (lane == 0) ok = mbar_wait_bounded(&empty[s % stages], (s / stages - 1) & 1);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) {
        drain(full, stages, s);
        break;
      }
      load_in(s);
      load_p(s);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // kind::f16, A and B fp16, D fp32, K-major, M = 128 rows, N = r16
      const uint32_t idesc = (1u << 4) | ((uint32_t)(r16 >> 3) << 17) | ((uint32_t)(kTallRows >> 4) << 24);
      const uint64_t in0 = smem_desc_sw128(smem_u32(smem)), p0 = smem_desc_sw128(smem_u32(smem) + S::kInBytes);
      RingPos at;
      int group = 0, in_group = 0;  // accumulators done, stages in the present one
      for (int s = 0; s < nk; ++s, at.next(stages)) {
        const int d = group & 1;
        if (in_group == 0 && group >= 2 && !mbar_wait_bounded(&dempty[d], (group / 2 - 1) & 1)) break;
        if (!mbar_wait_bounded(&full[at.slot], at.phase)) break;
        tc_fence_after();
        const uint32_t off = at.slot * S::kStageBytes;
        const uint64_t in = desc_at(in0, off), pd = desc_at(p0, off);
#pragma unroll
        for (int j = 0; j < kCols / 16; ++j)
          mma_f16_ss(tmem + d * R, desc_at(in, 32 * j), desc_at(pd, 32 * j), idesc, (in_group | j) != 0);
        mma_commit(&empty[at.slot]);
        if (++in_group == args.flush || s == nk - 1) {
          mma_commit(&dfull[d]);
          ++group, in_group = 0;
        }
      }
    }
  }
  __syncwarp();
  float* part = reinterpret_cast<float*>(smem);  // [128][kPitch], over the drained ring
  if (warp >= 2) {
    const int q = warp & 3, tr = 32 * q + lane, groups = (nk + args.flush - 1) / args.flush;
    float sum[R];
#pragma unroll
    for (int j = 0; j < R; ++j) sum[j] = 0.f;
    for (int k = 0; k < groups; ++k) {
      if (!mbar_wait_bounded(&dfull[k & 1], (k / 2) & 1)) break;
      tc_fence_after();
#pragma unroll
      for (int t = 0; t < R / 16; ++t) {
        if (16 * t >= r16) break;
        uint32_t v[16];
        tmem_ld16(tmem + ((uint32_t)(32 * q) << 16) + (k & 1) * R + 16 * t, v);
#pragma unroll
        for (int e = 0; e < 16; ++e) sum[16 * t + e] += __uint_as_float(v[e]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&dempty[k & 1]);
    }
    // the last accumulator was read: no operand of the ring is in use any more (all four warps
    // have to be here, since the sums of one lie where another's last operands may)
    asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
    for (int j = 0; j < R; j += 4)
      if (j < r16) *reinterpret_cast<float4*>(part + tr * S::kPitch + j) = make_float4(sum[j], sum[j + 1], sum[j + 2], sum[j + 3]);
  }
  tc_fence_before();
  cluster_arrive();
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmem);
  }
  // the cluster's sum of this CTA's share of the rows, CTAs in order: scale * T, zero past
  // the slot's rank and the tile's rows. A share lies in one 64-row tile, whose CTAs are half of
  // the cluster. A thread takes the same four ranks of every `step`-th row.
  const uint32_t pbase = smem_u32(part);
  const int share = kTallRows / cluster, row_lo = rankc * share, quads = r16 / 4, step = kTallThreads / quads;
  const int half = row_lo / kWideRows, near = cluster / 2, j = 4 * (threadIdx.x % quads), at_row = threadIdx.x / quads;
  const bool there = half == 0 || count > kWideRows;  // the 64-row tile exists
  constexpr int kLeast = kTallThreads / (R / 4), kMine = (kWideRows + kLeast - 1) / kLeast;  // rows of a thread, cluster >= 2
  float4 mine[kMine];
  uint4 most = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int q = 0; q < kMine; ++q) {
    const int in = at_row + q * step, row = row_lo + in;
    mine[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (at_row >= step || in >= share || row >= count) continue;
    const float4 x = sum_peers(pbase + 4 * (row * S::kPitch + j), cluster);
    mine[q] = make_float4(j < r ? x.x * scale : 0.f, j + 1 < r ? x.y * scale : 0.f, j + 2 < r ? x.z * scale : 0.f,
                          j + 3 < r ? x.w * scale : 0.f);
    const uint4 bits = finite_bits(mine[q]);
    if (a.parts) atomicMax(rowmax + in, largest(bits));
    most = larger(most, bits);
  }
  if (a.gparts && at_row < step) atomic_larger(rankmax + j, most);
  __syncthreads();
  if (a.gparts)
    for (int i = threadIdx.x; i < r16 * near; i += kTallThreads)
      st_peer_u32(peer_smem(smem_u32(allmax + (rankc - half * near) * R + i % r16), half * near + i / r16), rankmax[i % r16]);
  cluster_arrive();
  auto write = [&](__half* parts, int q, const float4& u) {
    const int in = at_row + q * step;
    if (there && at_row < step && in < share)
      write_parts(parts + ((size_t)tile.w * kWideRows + row_lo + in) * (2 * g.pp) + j, g.pp, mine[q], u);
  };
  if (a.parts) {
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      const float u = split_unit(__uint_as_float(rowmax[min(at_row + q * step, share - 1)]));
      write(a.parts, q, make_float4(u, u, u, u));
    }
    if (there && (int)threadIdx.x < share)
      a.unit[(size_t)tile.w * kWideRows + row_lo + threadIdx.x] = 1.f / split_unit(__uint_as_float(rowmax[threadIdx.x]));
  }
  cluster_wait();
  if (a.gparts) {
    if ((int)threadIdx.x < r16) {
      units[threadIdx.x] = rank_unit(allmax + threadIdx.x, R, near);
      if (there && rankc == half * near) a.gunit[(size_t)(tile.w + half) * g.pp + threadIdx.x] = 1.f / units[threadIdx.x];
    }
    __syncthreads();
    const float4 u = *reinterpret_cast<const float4*>(units + j);
#pragma unroll
    for (int q = 0; q < kMine; ++q) write(a.gparts, q, u);
  }
}

// ---- expansion -------------------------------------------------------------------------------
// A CTA takes some 64-column blocks of one tile of up to 128 rows. T's parts, side by side
// as one row of 2 R elements, are the MMA's A operand for all of them; per block r rows of
// Q (B, MN-major, used by both parts) and the base tile (16 KB) arrive by TMA, D = T Q gets
// one of two accumulators, and eight epilogue warps (thread = 32 columns of a row) add base,
// round once and write the rows out. (Four warps took 1 us a block and were what 2048 rows
// waited for.) Started as the mma.sync expansion is: what was
// there before the call is read before the wait on the contraction.
struct TallExpandArgs {
  CUtensorMap in, box, q, parts;  // base by single rows and by 64, Q by 16
  RowsArgs g;
  int stages;
};

template <int R>
struct TallExpand {
  static constexpr int kTChunks = R <= 32 ? 1 : R / 32, kTBytes = kTChunks * kTallRows * 128;
  static constexpr int kBaseBytes = kTallRows * 128, kStageBytes = kBaseBytes + R * 128;
  static constexpr int kPart = 0, kOutBytes = 8 * 2048;  // a warp's 32 rows of 32 columns on their way out
  static constexpr int kFixed = kTBytes + kOutBytes;
  static constexpr int kTmem = 2 * kCols;
};

template <int R>
__global__ void __launch_bounds__(kExpandThreads) k_expand_tall(const __grid_constant__ TallExpandArgs args) {
  using S = TallExpand<R>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* ring = smem + S::kTBytes + S::kOutBytes;
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], tfull, dfull[2], dempty[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int srow[kTallRows];
  const RowsArgs& g = args.g;
  const RowsPass& a = g.pass[0];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, stages = args.stages;
  const int tile_no = blockIdx.y, parts = gridDim.x, b0 = blockIdx.x;
  const bool in_place = a.base == a.out;
  const int4 tile = __ldcg(g.tiles + tile_no);
  const int run_row = __ldcg(g.runs + tile_no);
  const bool live = takes_tile(g, tile_no, tile, in_place);
  const int count = tile.z & (kCrowdTile - 1), slot = tile.x;
  const int r = live && slot < g.n_slots ? __ldcg(g.rank + slot) : 0, r16 = (r + 15) & ~15;
  const int blocks = (a.N + kCols - 1) / kCols, nb = (blocks - b0 + parts - 1) / parts;
  if (r == 0) {  // no tile, or base alone
    trigger_dependents();
    grid_dependency_wait();
    if (live && !in_place)
      for (int b = b0; b < blocks; b += parts)
        copy_rows(a, g.rows, g.perm + tile.y, count, b * (kCols / 8), min((b + 1) * (kCols / 8), a.N / 8));
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 9);  // the MMA and the eight epilogue warps
    }
    mbar_init(&tfull, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&dfull[s], 1);
      mbar_init(&dempty[s], 8);
    }
    fence_mbar_init();
    tma_prefetch_map(&args.box);
    tma_prefetch_map(&args.q);
    tma_prefetch_map(&args.parts);
  }
  if (warp == 1) tmem_alloc(&tmem_slot, S::kTmem);
  for (int i = threadIdx.x; i < kTallRows; i += kExpandThreads) srow[i] = __ldcg(g.perm + tile.y + min(i, count - 1));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  trigger_dependents();  // not before the tensor memory is ours
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    const bool run = run_row >= 0;
    const int boxes = run ? (count + kWideRows - 1) / kWideRows : 0;
    const uint32_t base_bytes = a.base == nullptr ? 0 : run ? boxes * kWideRows * 128 : S::kBaseBytes;
    auto load = [&](int i) {
      const uint32_t st = smem_u32(ring + i % stages * S::kStageBytes);
      const int x = (b0 + i * parts) * kCols;
      uint64_t* bar = &full[i % stages];
      if (lane == 0) mbar_arrive_expect_tx(bar, base_bytes + r16 * 128);
      __syncwarp();
      if (lane < r16 / 16) tma_load_2d(st + S::kBaseBytes + 2048 * lane, &args.q, x, slot * g.rp + 16 * lane, bar);
      if (a.base) {
        if (!run) tma_gather4(st + 512 * lane, &args.in, x, srow[4 * lane], srow[4 * lane + 1], srow[4 * lane + 2], srow[4 * lane + 3], bar);
        else if (lane < boxes) tma_load_2d(st + 8192 * lane, &args.box, x, run_row + kWideRows * lane, bar);
      }
    };
    const int first = min(stages, nb);
    for (int i = 0; i < first; ++i) load(i);
    grid_dependency_wait();
    {  // T: chunks of 64 of a row's 2 R elements, 64 rows a box; past the tile's rows whatever is there
      const int half = S::kTChunks / 2, used = R <= 64 ? S::kTChunks : r16 > 64 ? 4 : 2;
      if (lane == 0) mbar_arrive_expect_tx(&tfull, used * kTallRows * 128);
      __syncwarp();
      if (lane < 2 * used) {
        const int u = lane >> 1, c = R > 64 && used == 2 ? u * half : u;
        tma_load_2d(smem_u32(smem) + 16384 * c + 8192 * (lane & 1), &args.parts, 64 * c, (tile.w + (lane & 1)) * kWideRows, &tfull);
      }
    }
    for (int i = first; i < nb; ++i) {
      bool ok = true;
      if (lane == 0) ok = mbar_wait_bounded(&empty[i % stages], (i / stages - 1) & 1);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) {
        drain(full, stages, i);
        break;
      }
      load(i);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // kind::f16, A (K-major) and B (MN-major) fp16, D fp32, M = 128 rows, N = 64 columns
      const uint32_t idesc = (1u << 4) | (1u << 16) | ((uint32_t)(kCols >> 3) << 17) | ((uint32_t)(kTallRows >> 4) << 24);
      const uint64_t ta = smem_desc_sw128(smem_u32(smem)), q0 = smem_desc_mn_sw128(smem_u32(ring) + S::kBaseBytes);
      const bool there = mbar_wait_bounded(&tfull, 0);
      RingPos at;
      for (int i = 0; i < nb && there; ++i, at.next(stages)) {
        const int d = i & 1;
        if (i >= 2 && !mbar_wait_bounded(&dempty[d], (i / 2 - 1) & 1)) break;
        if (!mbar_wait_bounded(&full[at.slot], at.phase)) break;
        tc_fence_after();
        const uint64_t q = desc_at(q0, at.slot * S::kStageBytes);
#pragma unroll
        for (int pt = 1; pt >= 0; --pt)  // the low part first
#pragma unroll
          for (int j = 0; j < R / 16; ++j) {
            if (16 * j >= r16) break;
            const int e = pt * R + 16 * j;  // first of the 16 elements of T's row
            mma_f16_ss(tmem + d * kCols, desc_at(ta, e / 64 * 16384 + e % 64 * 2), desc_at(q, 2048 * j), idesc, pt == 0 || j != 0);
          }
        mma_commit(&empty[at.slot]);
        mma_commit(&dfull[d]);
      }
    }
  }
  __syncwarp();
  if (warp >= 2) {
    grid_dependency_wait();  // the units are the contraction's
    const int q = warp & 3, h = (warp - 2) >> 2, tr = 32 * q + lane;
    const uint32_t mine = smem_u32(smem + S::kTBytes) + (warp - 2) * 2048;
    const float back = tr < count ? __ldcg(a.unit + (size_t)tile.w * kWideRows + tr) : 0.f;
    RingPos at;
    for (int i = 0; i < nb; ++i, at.next(stages)) {
      const uint32_t st = smem_u32(ring + at.slot * S::kStageBytes);
      if (!mbar_wait_bounded(&full[at.slot], at.phase) || !mbar_wait_bounded(&dfull[i & 1], (i / 2) & 1)) break;
      tc_fence_after();
      uint32_t v[32];
      tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + (i & 1) * kCols + 32 * h, v);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&dempty[i & 1]);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t spot = st + tr * 128 + 16 * ((4 * h + c) ^ (tr & 7));
        const uint4 b = a.base ? lds_u32x4(spot) : make_uint4(0, 0, 0, 0);
        const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&bw[e]));
          const __half2 x = __floats2half2_rn(fmaf(__uint_as_float(v[8 * c + 2 * e]), back, f.x), fmaf(__uint_as_float(v[8 * c + 2 * e + 1]), back, f.y));
          o[e] = *reinterpret_cast<const uint32_t*>(&x);
        }
        sts_v4(mine + lane * 64 + 16 * (c ^ ((lane >> 1) & 3)), o[0], o[1], o[2], o[3]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[at.slot]);
      // the warp's own 32 rows of 32 columns, four lanes a row
      const int c = (b0 + i * parts) * kCols + 32 * h + 8 * (lane & 3);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int wr = 8 * k + (lane >> 2), row = 32 * q + wr;
        if (row < count && c < a.N)
          *reinterpret_cast<uint4*>(a.out + (size_t)srow[row] * a.N + c) = lds_u32x4(mine + wr * 64 + 16 * ((lane & 3) ^ ((wr >> 1) & 3)));
      }
      __syncwarp();
    }
  }
  grid_dependency_wait();  // who waits for this launch waits for those before it too
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmem);
  }
}

// ---- weight gradients ------------------------------------------------------------------------
// G_s[j][i] (+)= sum over the slot's 64-row tiles of unit_j * (T parts)^T In, as G^T: 128
// columns of In are the MMA's rows (A, gathered, MN-major), the ranks its columns (B, T's
// parts, MN-major), 64 rows its reduction. Each tile gets an accumulator of its own in
// tensor memory (two in turn), which the epilogue warps add, times the ranks' units, to
// fp32 sums in registers (thread = column): a long sum is rounded to nearest once a tile.
// A cluster splits the tiles and sums through distributed shared memory in rank order.
struct TallGradArgs {
  CUtensorMap in[2], box[2], parts[2];
  GradArgs g;
  int stages;
};

template <int R>
struct TallGrad {
  static constexpr int kInBytes = 2 * kWideRows * 128;  // two chunks of 64 columns
  // 64-element chunks of T's rows [high R | low R]: both parts in one, or one or two each
  static constexpr int kTChunks = R <= 32 ? 1 : R / 32, kTBytes = kTChunks * kWideRows * 128;
  static constexpr int kLow = R <= 32 ? 2 * R : kTBytes / 2;  // bytes from the high part to the low
  static constexpr int kStageBytes = kInBytes + kTBytes;
  static constexpr int kPart = R * kGradCols * 4, kFixed = 0;  // the partial sums lie over the drained ring
  // up to rank 32 both parts are one operand of 2 R columns, so that In is read once
  static constexpr bool kBoth = R <= 32;
  static constexpr int kD = kBoth ? 2 * R : R;  // columns of an accumulator
  static constexpr int kTmem = 2 * kD;
};

template <int R>
__global__ void __launch_bounds__(kTallThreads) k_grad_tall(const __grid_constant__ TallGradArgs args) {
  using S = TallGrad<R>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], dfull[2], dempty[2];
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(16) float units[4][2][R];  // each epilogue warp's own, of two tiles in turn
  const GradArgs& g = args.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, stages = args.stages;
  const int split = blockIdx.z, nsplit = gridDim.z, slot = grad_slot(g);
  if (slot < 0) {
    grid_dependency_wait();
    return;
  }
  const int which = (int)blockIdx.x < g.pass[0].blocks ? 0 : 1;
  const GradPass& a = g.pass[which];
  const int col0 = ((int)blockIdx.x - (which ? g.pass[0].blocks : 0)) * kGradCols;
  // The launch before is the contraction of the same call: what was there
  // before the call (plan, ranks, In) is complete and may be read before the wait.
  const int p0 = __ldcg(g.start + slot), rows = __ldcg(g.start + slot + 1) - p0, tile0 = __ldcg(g.first64 + slot);
  const int r = rows ? __ldcg(g.rank + slot) : 0, r16 = (r + 15) & ~15;
  float* out = a.g + (size_t)slot * g.max_rank * a.K;
  const int width = min(kGradCols, a.K - col0);
  if (r == 0) {
    grid_dependency_wait();
    if (!g.zeroed && !g.accumulate) zero_columns(out + col0, a.K, width, g.max_rank, split, nsplit);
    return;
  }
  const int nt_all = (rows + kWideRows - 1) / kWideRows, t_lo = (int)((long)nt_all * split / nsplit);
  const int nt = (int)((long)nt_all * (split + 1) / nsplit) - t_lo;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&dfull[s], 1);
      mbar_init(&dempty[s], 4);
    }
    fence_mbar_init();
    tma_prefetch_map(&args.box[which]);
    tma_prefetch_map(&args.parts[which]);
  }
  if (warp == 1) tmem_alloc(&tmem_slot, S::kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    const int half = S::kTChunks / 2, used = R <= 64 ? S::kTChunks : r16 > 64 ? 4 : 2;  // chunks with ranks in them
    const uint32_t bytes = S::kInBytes + used * kWideRows * 128;
    const int chunk = lane >> 4, r4 = 4 * (lane & 15);  // this lane's chunk and first row of a tile
    const int x = col0 + 64 * chunk < a.K ? col0 + 64 * chunk : col0;  // past the end any columns will do
    // In's part of stage s: a whole tile of rows in a run as two boxes. Rows past the slot's
    // end must not be others' (0 * inf): the ragged tile gathers, repeating its last row (T
    // is zero there). Whether a tile is a run is loaded one stage ahead.
    int next = nt > 0 ? __ldcg(g.runs + tile0 + t_lo) : -1;
    auto gather = [&](int s) {
      const uint32_t st = smem_u32(smem + s % stages * S::kStageBytes);
      const int row_a = next;
      if (row_a >= 0 && rows - (t_lo + s) * kWideRows >= kWideRows) {
        if (lane < 2) tma_load_2d(st + 8192 * lane, &args.box[which], col0 + 64 * lane < a.K ? col0 + 64 * lane : col0, row_a, &full[s % stages]);
      } else {
        int row[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) row[q] = __ldcg(g.perm + p0 + min((t_lo + s) * kWideRows + r4 + q, rows - 1));
        tma_gather4(st + 8192 * chunk + 128 * r4, &args.in[which], x, row[0], row[1], row[2], row[3], &full[s % stages]);
      }
      next = s + 1 < nt ? __ldcg(g.runs + tile0 + t_lo + s + 1) : -1;
    };
    auto parts = [&](int s) {
      if (lane < used) {
        const int c = R > 64 && used == 2 ? lane * half : lane;  // the first chunk of each part, or all
        tma_load_2d(smem_u32(smem + s % stages * S::kStageBytes) + S::kInBytes + 8192 * c, &args.parts[which], 64 * c,
                    (tile0 + t_lo + s) * kWideRows, &full[s % stages]);
      }
    };
    const int first = min(nt, stages);
    for (int s = 0; s < first; ++s) {
      if (lane == 0) mbar_arrive_expect_tx(&full[s], bytes);
      __syncwarp();
      gather(s);
    }
    grid_dependency_wait();
    trigger_dependents();  // all CTAs hold their tensor memory; the expansion's first loads may go out
    for (int s = 0; s < first; ++s) parts(s);
    for (int s = first; s < nt; ++s) {
      bool ok = true;
      if (lane == 0) {
        ok = mbar_wait_bounded(&empty[s % stages], (s / stages - 1) & 1);
        if (ok) mbar_arrive_expect_tx(&full[s % stages], bytes);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) {
        drain(full, stages, s);
        break;
      }
      gather(s);
      parts(s);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // kind::f16, A and B fp16 and MN-major, D fp32, M = 128 columns, N = r16
      const uint32_t idesc = (1u << 4) | (1u << 15) | (1u << 16) | ((uint32_t)((S::kBoth ? 2 * R : r16) >> 3) << 17) | ((uint32_t)(kGradCols >> 4) << 24);
      const uint64_t in0 = smem_desc_mn_sw128(smem_u32(smem)), t0 = smem_desc_mn_sw128(smem_u32(smem) + S::kInBytes);
      RingPos at;
      for (int s = 0; s < nt; ++s, at.next(stages)) {
        const int d = s & 1;
        if (s >= 2 && !mbar_wait_bounded(&dempty[d], (s / 2 - 1) & 1)) break;
        if (!mbar_wait_bounded(&full[at.slot], at.phase)) break;
        tc_fence_after();
        const uint32_t off = at.slot * S::kStageBytes;
        const uint64_t in = desc_at(in0, off), tp = desc_at(t0, off);
#pragma unroll
        for (int pt = S::kBoth ? 0 : 1; pt >= 0; --pt)  // the low part first
#pragma unroll
          for (int j = 0; j < kWideRows / 16; ++j)
            mma_f16_ss(tmem + d * S::kD, desc_at(in, 2048 * j), desc_at(tp, pt * S::kLow + 2048 * j), idesc,
                       (!S::kBoth && pt == 0) || j != 0);
        mma_commit(&empty[at.slot]);
        mma_commit(&dfull[d]);
      }
    }
  }
  __syncwarp();
  float* part = reinterpret_cast<float*>(smem);  // [R][128], over the drained ring
  if (warp >= 2) {
    grid_dependency_wait();  // the units are the contraction's
    trigger_dependents();
    const int q = warp & 3;
    float sum[R];
#pragma unroll
    for (int j = 0; j < R; ++j) sum[j] = 0.f;
    // the ranks' units, loaded a tile ahead
    constexpr int kUnits = (R + 31) / 32;
    const float* unit_at = a.unit + (size_t)(tile0 + t_lo) * g.pp + lane;
    float next[kUnits];
    auto fetch = [&](int s) {
#pragma unroll
      for (int u = 0; u < kUnits; ++u) next[u] = s < nt && lane + 32 * u < r16 ? __ldcg(unit_at + (size_t)s * g.pp + 32 * u) : 0.f;
    };
    fetch(0);
    for (int s = 0; s < nt; ++s) {
      float* own = units[warp - 2][s & 1];  // read two tiles ago
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
        if (lane + 32 * u < r16) own[lane + 32 * u] = next[u];
      __syncwarp();
      fetch(s + 1);
      const float4* unit = reinterpret_cast<const float4*>(own);
      if (!mbar_wait_bounded(&dfull[s & 1], (s / 2) & 1)) break;
      tc_fence_after();
#pragma unroll
      for (int t = 0; t < R / 16; ++t) {
        if (16 * t >= r16) break;
        uint32_t v[16];
        const uint32_t at = tmem + ((uint32_t)(32 * q) << 16) + (s & 1) * S::kD + 16 * t;
        tmem_ld16(at, v);
        if constexpr (S::kBoth) {
          uint32_t w[16];
          tmem_ld16(at + R, w);
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) + __uint_as_float(w[e]));
        }
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float4 u = unit[4 * t + e / 4];
          float* y = sum + 16 * t + e;
          y[0] = fmaf(__uint_as_float(v[e]), u.x, y[0]), y[1] = fmaf(__uint_as_float(v[e + 1]), u.y, y[1]);
          y[2] = fmaf(__uint_as_float(v[e + 2]), u.z, y[2]), y[3] = fmaf(__uint_as_float(v[e + 3]), u.w, y[3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&dempty[s & 1]);
    }
    // every MMA of the last tile has completed (its accumulator was read), so that no
    // operand of the ring is in use any more
#pragma unroll
    for (int j = 0; j < R; ++j) part[j * kGradCols + 32 * q + lane] = sum[j];
  } else if (warp == 1) {
    grid_dependency_wait();
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
    tmem_dealloc(tmem, S::kTmem);
  }
  // this CTA's share of the gradient's rows; rows past the rank are zero
  const uint32_t pbase = smem_u32(part);
  for (int i = split * kTallThreads + threadIdx.x; i < g.max_rank * (kGradCols / 4); i += nsplit * kTallThreads) {
    const int j = i / (kGradCols / 4), c = 4 * (i % (kGradCols / 4));
    if (c >= width) continue;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (j < r)
      for (int s = 0; s < nsplit; ++s) {
        const float4 y = nsplit > 1 ? ld_peer_v4f(peer_smem(pbase + 4 * (j * kGradCols + c), s))
                                    : *reinterpret_cast<const float4*>(part + j * kGradCols + c);
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
      }
    float* dst = out + (size_t)j * a.K + col0 + c;  // K % 8 == 0: 16-byte aligned, c + 4 <= width
    if (g.accumulate) {
      const float4 y = *reinterpret_cast<const float4*>(dst);
      x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
    }
    *reinterpret_cast<float4*>(dst) = x;
  }
  if (nsplit > 1) {
    cluster_arrive();
    cluster_wait();
  }
}

// Self-test of this file's bounded-wait error path (its own device error word): one warp
// waits on an mbarrier that expects two arrivals and receives one.
__global__ void k_wait_probe_tall(long long cycles) {
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

cudaError_t launch_pdl_cluster(const void* fn, dim3 grid, size_t smem, cudaStream_t stream, void** args, dim3 cluster,
                               int threads = kTallThreads) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
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
  cfg.numAttrs = cluster.x * cluster.z > 1 ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

// Rows of an activation array: boxes of 64 columns by one row (gathers) and by 64 rows.
cudaError_t encode_rows(CUtensorMap* single, CUtensorMap* box, const __half* x, int K, int M) {
  const cudaError_t e = encode_tiled_2d(single, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, x, (uint64_t)K, (uint64_t)M, (uint64_t)K * 2,
                                        kCols, 1, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  return encode_tiled_2d(box, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, x, (uint64_t)K, (uint64_t)M, (uint64_t)K * 2, kCols, kWideRows,
                         CU_TENSOR_MAP_SWIZZLE_128B);
}

// Stages of a ring, and the shared memory it takes: what an SM holds, shared by the CTAs
// that run on it, since a load takes some 2 us and every stage in flight counts; no more
// than there is work for, no less than the partial sums need.
constexpr int kSmPerSm = 216 * 1024, kTallSlack = 1024 + 1024;  // alignment, static shared memory
struct Ring {
  int stages, smem;
};
Ring plan_ring(int stage_bytes, int part_bytes, int fixed_bytes, int work, int share) {
  Ring r;
  const int room = (kSmPerSm / share - kTallSlack - fixed_bytes) / stage_bytes;
  r.stages = std::min({kMaxStages, std::max(1, work), std::max(2, room)});
  r.stages = std::max(r.stages, (part_bytes + stage_bytes - 1) / stage_bytes);
  r.smem = r.stages * stage_bytes + fixed_bytes + 1024;
  return r;
}
// CTAs of an SM: two (clusters of eight with one an SM leave SMs idle: 16 of them fit a
// GPU of 148), or three where there are more than that anyway (384 CTAs of the gradients: a
// whole pass took 101.8 us with two, 106.4 with three).
int sm_share(long ctas, int n_sm) { return ctas > 3l * n_sm ? 3 : 2; }

template <int R>
cudaError_t allow_tall() {
  const int most = kSmPerSm - 1024;
  cudaError_t e = cudaFuncSetAttribute(k_contract_tall<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(k_expand_tall<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, most))) return e;
  return cudaFuncSetAttribute(k_grad_tall<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

}  // namespace

cudaError_t prepare_tall_kernels(int device) {
  (void)device;
  cudaError_t e;
  if ((e = allow_tall<16>()) || (e = allow_tall<32>()) || (e = allow_tall<64>())) return e;
  return allow_tall<128>();
}

cudaError_t encode_adapter_maps(dictproj_adapters* a) {
  cudaError_t e;
  const uint64_t ranks = (uint64_t)a->n_slots * a->rp, rows = (uint64_t)adapter_tiles(a->max_tokens, a->n_slots, kWideRows) * kWideRows;
  if ((e = encode_tiled_2d(&a->a_map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a->A, (uint64_t)a->d_in, ranks, (uint64_t)a->d_in * 2,
                           kCols, 16, CU_TENSOR_MAP_SWIZZLE_128B)) ||
      (e = encode_tiled_2d(&a->b_map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a->B, (uint64_t)a->ld_b, ranks, (uint64_t)a->ld_b * 2,
                           kCols, 16, CU_TENSOR_MAP_SWIZZLE_128B)))
    return e;
  auto parts = [&](CUtensorMap* map, const uint16_t* p) {
    return encode_tiled_2d(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p, (uint64_t)2 * a->pp, rows, (uint64_t)4 * a->pp, 64, kWideRows,
                           CU_TENSOR_MAP_SWIZZLE_128B);
  };
  if ((e = parts(&a->part_map, a->parts)) || (e = parts(&a->gpart_map[0], a->gparts[0]))) return e;
  return parts(&a->gpart_map[1], a->gparts[1]);
}

// Rows that TMA can read, and enough of them to fill 128-row tiles: up to rank 32 the
// mma.sync kernels are as fast until there are about a hundred rows a slot (backward, 4096
// and 4096 wide, rank 16: 1 slot 384 rows 20.8 us there, 16.5 here; 16 slots 1024 rows 29
// and 39), above it their instructions cost more from 256 rows on (rank 64: 1 slot 256 rows
// 24.3 and 18.7, 16 slots 53 and 46).
bool tall_serves(const dictproj_adapters* a, const dictproj_rows* r) {
  return a->d_out % 8 == 0 && r->M >= (a->rp <= 32 ? std::max(384, 96 * a->n_slots) : 256);
}

struct TallKernel {
  const void* fn;
  int stage_bytes, part_bytes, fixed_bytes;
};
#define DICTPROJ_TALL_R(kernel, shape, R) TallKernel{(const void*)kernel<R>, shape<R>::kStageBytes, shape<R>::kPart, shape<R>::kFixed}
#define DICTPROJ_TALL(rp, kernel, shape)                  \
  ((rp) <= 16   ? DICTPROJ_TALL_R(kernel, shape, 16)      \
   : (rp) <= 32 ? DICTPROJ_TALL_R(kernel, shape, 32)      \
   : (rp) <= 64 ? DICTPROJ_TALL_R(kernel, shape, 64)      \
                : DICTPROJ_TALL_R(kernel, shape, 128))

cudaError_t launch_contract_tall(RowsArgs& g, int passes, bool exact_sums, const dictproj_adapters* a, const dictproj_rows* r,
                                 cudaStream_t stream) {
  TallContractArgs args;
  cudaError_t e;
  for (int i = 0; i < passes; ++i) {
    if ((e = encode_rows(&args.in[i], &args.box[i], g.pass[i].in, g.pass[i].K, r->M)) != cudaSuccess) return e;
    args.p[i] = reinterpret_cast<const uint16_t*>(g.pass[i].P) == a->A ? a->a_map : a->b_map;
  }
  args.g = g;
  args.g.tiles = r->tiles[2];
  args.g.n_tiles = r->n_tiles + 4;
  args.g.runs = r->runs[1];
  const int full = std::max(1, r->M / kTallRows) * passes;  // tiles that do exist, about
  args.g.cluster = 2;
  while (args.g.cluster < 8 && full * args.g.cluster < 3 * a->n_sm / 2) args.g.cluster *= 2;
  const TallKernel k = DICTPROJ_TALL(g.rp, k_contract_tall, TallContract);
  const int kc = (std::max(g.pass[0].K, g.pass[passes - 1].K) + kCols - 1) / kCols;
  const Ring ring = plan_ring(k.stage_bytes, k.part_bytes, k.fixed_bytes, (kc + args.g.cluster - 1) / args.g.cluster,
                              sm_share((long)full * args.g.cluster, a->n_sm));
  args.stages = ring.stages;
  args.flush = exact_sums ? 2 : 1 << 20;
  void* p[] = {(void*)&args};
  return launch_pdl_cluster(k.fn, dim3((unsigned)(adapter_tiles(r->M, r->n_slots, kTallRows) * args.g.cluster), passes), ring.smem,
                            stream, p, dim3(args.g.cluster, 1, 1));
}

cudaError_t launch_expand_tall(const RowsArgs& g, const dictproj_adapters* a, const dictproj_rows* r, cudaStream_t stream) {
  TallExpandArgs args;
  const RowsPass& p = g.pass[0];
  // without a base its maps are not used; out stands in for them
  cudaError_t e = encode_rows(&args.in, &args.box, p.base ? p.base : p.out, p.N, r->M);
  if (e != cudaSuccess) return e;
  args.q = reinterpret_cast<const uint16_t*>(p.Q) == a->A ? a->a_map : a->b_map;
  args.parts = a->part_map;
  args.g = g;
  args.g.tiles = r->tiles[2];
  args.g.n_tiles = r->n_tiles + 4;
  args.g.runs = r->runs[1];
  const TallKernel k = DICTPROJ_TALL(g.rp, k_expand_tall, TallExpand);
  const int blocks = (p.N + kCols - 1) / kCols;
  const int share = g.rp <= 64 ? 2 : 1, full = std::max(1, r->M / kTallRows);  // tiles that do exist, about
  const int ragged = std::min(a->n_slots, full) / 2;  // and those that end a slot's rows
  const int parts = std::min(blocks, std::max(1, share * a->n_sm / (full + ragged)));  // as many CTAs as run at once
  const Ring ring = plan_ring(k.stage_bytes, 0, k.fixed_bytes, (blocks + parts - 1) / parts, share);
  args.stages = ring.stages;
  void* pp[] = {(void*)&args};
  return launch_pdl_cluster(k.fn, dim3(parts, adapter_tiles(r->M, r->n_slots, kTallRows)), ring.smem, stream, pp, dim3(1, 1, 1),
                            kExpandThreads);
}

// CTAs that the tiles of a gradient are split over: with `at_once` CTAs running, each is as
// long as its tiles and a fixed part (set-up, first loads, cluster sum) worth about eight.
static int grad_split(int blocks, int tiles, int at_once) {
  int best = 1;
  double cost = 1e30;
  for (int s = 1; s <= 8 && (s == 1 || s <= tiles); s *= 2) {
    const double w = (double)blocks * s / at_once;  // between whole waves and none
    const double c = std::max(1.0, 0.5 * (w + std::ceil(w))) * ((tiles + s - 1) / s + 8);
    if (c < cost) cost = c, best = s;
  }
  return best;
}

cudaError_t launch_grad_tall(const GradArgs& w, const dictproj_adapters* a, const dictproj_rows* r, cudaStream_t stream) {
  TallGradArgs args;
  cudaError_t e;
  for (int i = 0; i < 2; ++i) {
    if ((e = encode_rows(&args.in[i], &args.box[i], w.pass[i].in, w.pass[i].K, r->M)) != cudaSuccess) return e;
    args.parts[i] = a->gpart_map[i];
  }
  args.g = w;
  const int blocks = w.pass[0].blocks + w.pass[1].blocks;
  const int slots = std::min(a->n_slots, r->M);  // that can have rows
  const int split = grad_split(blocks * slots, r->M / (kWideRows * slots), a->n_sm * (w.rp <= 32 ? 3 : w.rp <= 64 ? 2 : 1));
  const TallKernel k = DICTPROJ_TALL(w.rp, k_grad_tall, TallGrad);
  const int tiles = (r->M / (kWideRows * slots) + split) / split;
  // above rank 32 the sums' registers let two CTAs run on an SM (8192 rows, 4096 and 11008 wide,
  // rank 64: the whole pass 158 us with rings for two, 166 with rings for three)
  const int share = w.rp > 32 ? 2 : sm_share((long)blocks * slots * split, a->n_sm);
  const Ring ring = plan_ring(k.stage_bytes, k.part_bytes, 0, tiles, share);
  args.stages = ring.stages;
  void* p[] = {(void*)&args};
  return launch_pdl_cluster(k.fn, dim3(blocks, slots, split), ring.smem, stream, p, dim3(1, 1, split));
}

cudaError_t launch_wait_probe_tall(long long cycles, cudaStream_t stream) {
  k_wait_probe_tall<<<1, 32, 0, stream>>>(cycles);
  return cudaGetLastError();
}

cudaError_t take_tall_error(unsigned int* out) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_dictproj_error, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_dictproj_error, &zero, sizeof(unsigned int));
}

}  // namespace dictproj
