// C ABI of the adapters: pools, row plans, forward and backward calls, and the
// AdamW step (validation and handles; the kernels are in adapter.cu,
// adapter_tall.cu, backward.cu and adamw.cu).
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "dictproj.h"
#include "dictproj_internal.h"
#include "kernels.h"

namespace dictproj {
namespace {

// The handle's device has to be the current one.
int check_device(int device, const char* who) {
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, who);
  if (dev != device)
    return fail(DICTPROJ_ERR_MISMATCH, "%s: current device %d, handles on device %d", who, dev, device);
  return DICTPROJ_OK;
}

bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

struct Range {
  const void* p;
  size_t bytes;
  bool written = false;
};
bool overlap(Range a, Range b) {
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}

// Whether an array that the AdamW step writes overlaps another one of the list (gradients,
// which it only reads, may be shared).
bool written_twice(const dictproj_adamw_tensor* tensors, int n, int state_bytes) {
  std::vector<Range> all;
  all.reserve(7 * (size_t)n);
  for (int i = 0; i < n; ++i) {
    const dictproj_adamw_tensor& t = tensors[i];
    if (t.n == 0) continue;
    const size_t e = (size_t)t.n, blocks = (e + DICTPROJ_ADAMW_BLOCK - 1) / DICTPROJ_ADAMW_BLOCK;
    all.push_back({t.g, 4 * e, false});
    all.push_back({t.p, 4 * e, true});
    all.push_back({t.m, state_bytes * e, true});
    all.push_back({t.v, state_bytes * e, true});
    if (t.copy) all.push_back({t.copy, 2 * e, true});
    if (state_bytes == 1) {
      all.push_back({t.m_scale, 4 * blocks, true});
      all.push_back({t.v_scale, 4 * blocks, true});
    }
  }
  std::sort(all.begin(), all.end(), [](const Range& a, const Range& b) { return (uintptr_t)a.p < (uintptr_t)b.p; });
  uintptr_t end = 0, written_end = 0;  // of the arrays that start at or before this one
  for (const Range& r : all) {
    const uintptr_t first = (uintptr_t)r.p;
    if (first < (r.written ? end : written_end)) return true;
    end = std::max(end, first + r.bytes);
    if (r.written) written_end = std::max(written_end, first + r.bytes);
  }
  return false;
}

// What every call on a pool and a plan checks; *M gets the planned rows.
int check_call(const dictproj_adapters* a, const dictproj_rows* rows, const char* who, int* M) {
  if (!a || !rows) return fail(DICTPROJ_ERR_NULL, "%s: NULL handle", who);
  if (rows->M < 1) return fail(DICTPROJ_ERR_RANGE, "%s: no rows planned (dictproj_rows_set)", who);
  if (rows->M > a->max_tokens)
    return fail(DICTPROJ_ERR_RANGE, "%s: %d rows planned, the pool takes %d", who, rows->M, a->max_tokens);
  if (rows->n_slots != a->n_slots)
    return fail(DICTPROJ_ERR_RANGE, "%s: plan over %d slots, pool of %d", who, rows->n_slots, a->n_slots);
  if (rows->device != a->device)
    return fail(DICTPROJ_ERR_MISMATCH, "%s: plan on device %d, pool on device %d", who, rows->device, a->device);
  *M = rows->M;
  return DICTPROJ_OK;
}

int check_forward(const dictproj_adapters* a, const dictproj_rows* rows, const void* X, const void* base, void* Y,
                  const char* who) {
  int M = 0, st;
  if (!X || !Y) return fail(DICTPROJ_ERR_NULL, "%s: NULL pointer", who);
  if ((st = check_call(a, rows, who, &M))) return st;
  if (misaligned(X, 16) || misaligned(Y, 16) || misaligned(base, 16))
    return fail(DICTPROJ_ERR_ALIGN, "%s: X, base and Y must be 16-byte aligned", who);
  const Range x{X, (size_t)M * a->d_in * 2}, y{Y, (size_t)M * a->d_out * 2}, b{base, y.bytes};
  if (overlap(x, y)) return fail(DICTPROJ_ERR_RANGE, "%s: Y overlaps X", who);
  if (base != Y && overlap(b, y)) return fail(DICTPROJ_ERR_RANGE, "%s: Y overlaps base without being base", who);
  return DICTPROJ_OK;
}

}  // namespace
}  // namespace dictproj

using namespace dictproj;

extern "C" {

// ---- pools and plans -------------------------------------------------------------
int dictproj_adapters_create(int d_in, int d_out, int max_rank, int n_slots, int max_tokens, dictproj_adapters** out) {
  clear_error();
  if (!out) return fail(DICTPROJ_ERR_NULL, "adapters_create: NULL output");
  *out = nullptr;
  if (d_in <= 0 || d_in % 32 || d_out <= 0 || d_out > (1 << 24) || d_in > (1 << 24))
    return fail(DICTPROJ_ERR_SHAPE, "adapters_create: need d_in %% 32 == 0 and 0 < d_in, d_out <= 2^24 (got %d, %d)", d_in, d_out);
  if (max_rank < 1 || max_rank > DICTPROJ_MAX_RANK)
    return fail(DICTPROJ_ERR_RANGE, "adapters_create: max_rank=%d outside [1, %d]", max_rank, DICTPROJ_MAX_RANK);
  if (n_slots < 1 || n_slots > DICTPROJ_MAX_SLOTS)
    return fail(DICTPROJ_ERR_RANGE, "adapters_create: n_slots=%d outside [1, %d]", n_slots, DICTPROJ_MAX_SLOTS);
  if (max_tokens < 1 || max_tokens > DICTPROJ_MAX_ROWS)
    return fail(DICTPROJ_ERR_RANGE, "adapters_create: max_tokens=%d outside [1, %d]", max_tokens, DICTPROJ_MAX_ROWS);
  int dev, st;
  if ((st = ensure_device(&dev))) return st;
  dictproj_adapters* a = new (std::nothrow) dictproj_adapters();
  if (!a) return fail(DICTPROJ_ERR_OOM, "adapters_create: host allocation failed");
  a->device = dev;
  a->d_in = d_in;
  a->d_out = d_out;
  a->max_rank = max_rank;
  a->n_slots = n_slots;
  a->max_tokens = max_tokens;
  a->rp = (max_rank + 15) / 16 * 16;
  a->pp = a->rp <= 16 ? 16 : a->rp <= 32 ? 32 : a->rp <= 64 ? 64 : 128;
  a->ld_b = (d_out + 7) / 8 * 8;
  cudaError_t e = cudaDeviceGetAttribute(&a->n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) {
    delete a;
    return cuda_fail(e, "adapters_create: SM count");
  }
  const size_t ab = (size_t)n_slots * a->rp * d_in * 2, bb = (size_t)n_slots * a->rp * a->ld_b * 2;
  const size_t t64 = (size_t)adapter_tiles(max_tokens, n_slots, 64), pb = t64 * 64 * a->pp * 4, ub = t64 * sizeof(float);
  if ((e = dmalloc((void**)&a->A, ab)) || (e = dmalloc((void**)&a->B, bb)) ||
      (e = dmalloc((void**)&a->rank, (size_t)n_slots * 4)) || (e = dmalloc((void**)&a->scale, (size_t)n_slots * 4)) ||
      (e = dmalloc((void**)&a->parts, pb)) || (e = dmalloc((void**)&a->unit, ub * 64)) ||
      (e = dmalloc((void**)&a->gparts[0], pb)) || (e = dmalloc((void**)&a->gparts[1], pb)) ||
      (e = dmalloc((void**)&a->gunit[0], ub * a->pp)) || (e = dmalloc((void**)&a->gunit[1], ub * a->pp))) {
    dictproj_free_adapters(a);
    cudaGetLastError();
    return fail(DICTPROJ_ERR_OOM, "adapters_create: device allocation failed (%s)", cudaGetErrorName(e));
  }
  if ((e = cudaMemset(a->A, 0, ab)) || (e = cudaMemset(a->B, 0, bb)) ||
      (e = cudaMemset(a->rank, 0, (size_t)n_slots * 4)) || (e = cudaMemset(a->scale, 0, (size_t)n_slots * 4)) ||
      (e = cudaDeviceSynchronize())) {
    dictproj_free_adapters(a);
    cudaGetLastError();
    return cuda_fail(e, "adapters_create: empty slots");
  }
  if ((e = encode_adapter_maps(a)) != cudaSuccess) {
    dictproj_free_adapters(a);
    return cuda_fail(e, "adapters_create: tensor maps");
  }
  *out = a;
  return DICTPROJ_OK;
}

void dictproj_free_adapters(dictproj_adapters* a) {
  if (!a) return;
  cudaFree(a->A);
  cudaFree(a->B);
  cudaFree(a->rank);
  cudaFree(a->scale);
  cudaFree(a->parts);
  cudaFree(a->unit);
  for (int i = 0; i < 2; ++i) {
    cudaFree(a->gparts[i]);
    cudaFree(a->gunit[i]);
  }
  delete a;
}

int dictproj_adapters_set(dictproj_adapters* a, int slot, int rank, float scale, const void* A, const void* B,
                          void* stream) {
  clear_error();
  if (!a) return fail(DICTPROJ_ERR_NULL, "adapters_set: NULL handle");
  if (slot < 0 || slot >= a->n_slots)
    return fail(DICTPROJ_ERR_RANGE, "adapters_set: slot %d outside [0, %d)", slot, a->n_slots);
  if (rank < 0 || rank > a->max_rank)
    return fail(DICTPROJ_ERR_RANGE, "adapters_set: rank %d outside [0, %d]", rank, a->max_rank);
  if (rank > 0 && (!A || !B)) return fail(DICTPROJ_ERR_NULL, "adapters_set: NULL weights");
  if (!std::isfinite(scale)) return fail(DICTPROJ_ERR_VALUE, "adapters_set: scale is not finite");
  if (misaligned(A, 2) || misaligned(B, 2)) return fail(DICTPROJ_ERR_ALIGN, "adapters_set: A and B must be 2-byte aligned");
  int st;
  if ((st = check_device(a->device, "adapters_set"))) return st;
  const cudaError_t e = launch_adapter_set(a, slot, rank, scale, static_cast<const __half*>(A),
                                           static_cast<const __half*>(B), (cudaStream_t)stream);
  return e == cudaSuccess ? DICTPROJ_OK : cuda_fail(e, "adapters_set: launch");
}

int dictproj_adapters_slot(const dictproj_adapters* a, int slot, void** A, void** B, int* ld_B) {
  clear_error();
  if (!a) return fail(DICTPROJ_ERR_NULL, "adapters_slot: NULL handle");
  if (slot < 0 || slot >= a->n_slots)
    return fail(DICTPROJ_ERR_RANGE, "adapters_slot: slot %d outside [0, %d)", slot, a->n_slots);
  if (A) *A = a->A + (size_t)slot * a->rp * a->d_in;
  if (B) *B = a->B + (size_t)slot * a->rp * a->ld_b;
  if (ld_B) *ld_B = a->ld_b;
  return DICTPROJ_OK;
}

int dictproj_rows_create(int max_rows, int n_slots, dictproj_rows** out) {
  clear_error();
  if (!out) return fail(DICTPROJ_ERR_NULL, "rows_create: NULL output");
  *out = nullptr;
  if (max_rows < 1 || max_rows > DICTPROJ_MAX_ROWS)
    return fail(DICTPROJ_ERR_RANGE, "rows_create: max_rows=%d outside [1, %d]", max_rows, DICTPROJ_MAX_ROWS);
  if (n_slots < 1 || n_slots > DICTPROJ_MAX_SLOTS)
    return fail(DICTPROJ_ERR_RANGE, "rows_create: n_slots=%d outside [1, %d]", n_slots, DICTPROJ_MAX_SLOTS);
  int dev, st;
  if ((st = ensure_device(&dev))) return st;
  dictproj_rows* r = new (std::nothrow) dictproj_rows();
  if (!r) return fail(DICTPROJ_ERR_OOM, "rows_create: host allocation failed");
  r->device = dev;
  r->max_rows = max_rows;
  r->n_slots = n_slots;
  cudaError_t e;
  if ((e = dmalloc((void**)&r->perm, (size_t)max_rows * 4)) || (e = dmalloc((void**)&r->start, (size_t)(n_slots + 2) * 4)) ||
      (e = dmalloc((void**)&r->n_tiles, 8 * sizeof(int))) || (e = dmalloc((void**)&r->used, (size_t)n_slots * 4)) || (e = dmalloc((void**)&r->first64, (size_t)n_slots * 4)) ||
      (e = dmalloc((void**)&r->tiles[0], (size_t)adapter_tiles(max_rows, n_slots, 4) * sizeof(int4))) ||
      (e = dmalloc((void**)&r->tiles[1], (size_t)adapter_tiles(max_rows, n_slots, 64) * sizeof(int4))) ||
      (e = dmalloc((void**)&r->runs[0], (size_t)adapter_tiles(max_rows, n_slots, 64) * sizeof(int))) ||
      (e = dmalloc((void**)&r->runs[1], (size_t)adapter_tiles(max_rows, n_slots, 128) * sizeof(int))) ||
      (e = dmalloc((void**)&r->tiles[2], (size_t)adapter_tiles(max_rows, n_slots, 128) * sizeof(int4)))) {
    dictproj_free_rows(r);
    cudaGetLastError();
    return fail(DICTPROJ_ERR_OOM, "rows_create: device allocation failed (%s)", cudaGetErrorName(e));
  }
  // no rows until a plan has run: rows_set may have been captured and not replayed yet
  if ((e = cudaMemset(r->start, 0, (size_t)(n_slots + 2) * 4)) || (e = cudaMemset(r->n_tiles, 0, 8 * sizeof(int))) ||
      (e = cudaDeviceSynchronize())) {
    dictproj_free_rows(r);
    cudaGetLastError();
    return cuda_fail(e, "rows_create: empty plan");
  }
  *out = r;
  return DICTPROJ_OK;
}

void dictproj_free_rows(dictproj_rows* r) {
  if (!r) return;
  cudaFree(r->perm);
  cudaFree(r->start);
  cudaFree(r->n_tiles);
  cudaFree(r->used);
  cudaFree(r->first64);
  cudaFree(r->tiles[0]);
  cudaFree(r->tiles[1]);
  cudaFree(r->tiles[2]);
  cudaFree(r->runs[0]);
  cudaFree(r->runs[1]);
  delete r;
}

int dictproj_rows_set(dictproj_rows* rows, const int* ids, int M, void* stream) {
  clear_error();
  if (!rows || !ids) return fail(DICTPROJ_ERR_NULL, "rows_set: NULL pointer");
  if (M < 1 || M > rows->max_rows) return fail(DICTPROJ_ERR_RANGE, "rows_set: M=%d outside [1, %d]", M, rows->max_rows);
  if (misaligned(ids, 4)) return fail(DICTPROJ_ERR_ALIGN, "rows_set: ids must be 4-byte aligned");
  int st;
  if ((st = check_device(rows->device, "rows_set"))) return st;
  const cudaError_t e = launch_rows_plan(rows, ids, M, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "rows_set: launch");
  rows->M = M;
  return DICTPROJ_OK;
}

// ---- forward and backward ----------------------------------------------------------
int dictproj_adapter_forward(const dictproj_adapters* a, const dictproj_rows* rows, const void* X, const void* base,
                             void* Y, void* stream) {
  clear_error();
  int st;
  if ((st = check_forward(a, rows, X, base, Y, "adapter_forward"))) return st;
  if ((st = check_device(a->device, "adapter_forward"))) return st;
  const cudaError_t e = launch_adapter_forward(a, rows, static_cast<const __half*>(X), static_cast<const __half*>(base),
                                               static_cast<__half*>(Y), (cudaStream_t)stream);
  return e == cudaSuccess ? DICTPROJ_OK : cuda_fail(e, "adapter_forward: launch");
}

int dictproj_forward_adapters(const void* X, const dictproj_layer* layer, const dictproj_group* group,
                              const dictproj_adapters* a, const dictproj_rows* rows, void* Y, void* stream) {
  clear_error();
  int st;
  if (!layer || !group) return fail(DICTPROJ_ERR_NULL, "forward_adapters: NULL handle");
  if ((st = check_forward(a, rows, X, Y, Y, "forward_adapters"))) return st;
  if (group->d_in != a->d_in || layer->d_out != a->d_out)
    return fail(DICTPROJ_ERR_MISMATCH, "forward_adapters: projection %d -> %d, pool %d -> %d", group->d_in,
                layer->d_out, a->d_in, a->d_out);
  if (group->device != a->device)
    return fail(DICTPROJ_ERR_MISMATCH, "forward_adapters: projection on device %d, pool on device %d", group->device,
                a->device);
  if ((st = dictproj_forward(X, rows->M, layer, group, Y, stream))) return st;  // validates before it launches
  const cudaError_t e = launch_adapter_forward(a, rows, static_cast<const __half*>(X), static_cast<const __half*>(Y),
                                               static_cast<__half*>(Y), (cudaStream_t)stream);
  return e == cudaSuccess ? DICTPROJ_OK : cuda_fail(e, "forward_adapters: launch");
}

int dictproj_adapter_backward(const dictproj_adapters* a, const dictproj_rows* rows, const void* X, const void* dY,
                              const void* base, void* dX, float* dA, float* dB, int accumulate, void* stream) {
  clear_error();
  int M = 0, st;
  if (!X || !dY) return fail(DICTPROJ_ERR_NULL, "adapter_backward: NULL pointer");
  if (!dA != !dB) return fail(DICTPROJ_ERR_NULL, "adapter_backward: dA and dB go together");
  if (!dX && !dA) return fail(DICTPROJ_ERR_NULL, "adapter_backward: no output");
  if ((st = check_call(a, rows, "adapter_backward", &M))) return st;
  if (misaligned(X, 16) || misaligned(dY, 16) || misaligned(base, 16) || misaligned(dX, 16) || misaligned(dA, 16) ||
      misaligned(dB, 16))
    return fail(DICTPROJ_ERR_ALIGN, "adapter_backward: every array must be 16-byte aligned");
  const size_t wide = (size_t)a->n_slots * a->max_rank * sizeof(float);
  const Range in[] = {{X, (size_t)M * a->d_in * 2}, {dY, (size_t)M * a->d_out * 2}};
  const Range b{dX ? base : nullptr, in[0].bytes};
  const Range out[] = {{dX, in[0].bytes}, {dA, wide * a->d_in}, {dB, wide * a->d_out}};
  for (int i = 0; i < 3; ++i) {
    for (const Range& r : in)
      if (overlap(out[i], r)) return fail(DICTPROJ_ERR_RANGE, "adapter_backward: an output overlaps X or dY");
    if (!(i == 0 && base == dX) && overlap(out[i], b))
      return fail(DICTPROJ_ERR_RANGE, "adapter_backward: an output overlaps base (dX may be base itself)");
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return fail(DICTPROJ_ERR_RANGE, "adapter_backward: outputs overlap");
  }
  if ((st = check_device(a->device, "adapter_backward"))) return st;
  const cudaError_t e = launch_adapter_backward(
      a, rows, static_cast<const __half*>(X), static_cast<const __half*>(dY), static_cast<const __half*>(base),
      static_cast<__half*>(dX), dA, dB, accumulate != 0, (cudaStream_t)stream);
  return e == cudaSuccess ? DICTPROJ_OK : cuda_fail(e, "adapter_backward: launch");
}

int dictproj_group_reserve_backward(dictproj_group* g, int max_d_out) {
  clear_error();
  if (!g) return fail(DICTPROJ_ERR_NULL, "group_reserve_backward: NULL handle");
  int st = check_device(g->device, "group_reserve_backward");
  if (st || (st = dictproj_group_reserve_prefill(g, max_d_out)) || g->ddense) return st;
  uint16_t *p = nullptr, *more = nullptr;
  cudaError_t e = dmalloc((void**)&p, (size_t)g->k * g->d_in * sizeof(uint16_t));
  if (e == cudaSuccess) e = dmalloc((void**)&more, ((size_t)g->max_tokens + kFineRows) * g->k * sizeof(uint16_t));
  if (e != cudaSuccess) {
    cudaFree(p);
    cudaGetLastError();
    return fail(DICTPROJ_ERR_OOM, "group_reserve_backward: device allocation failed (%s)", cudaGetErrorName(e));
  }
  g->zmore = more;
  g->ddense = p;
  return DICTPROJ_OK;
}

int dictproj_backward_input(const void* dY, int M, const dictproj_layer* layer, const dictproj_group* group, void* dX,
                            void* stream) {
  clear_error();
  if (!dY || !dX || !layer || !group) return fail(DICTPROJ_ERR_NULL, "backward_input: NULL pointer");
  if (M < 1 || M > group->max_tokens)
    return fail(DICTPROJ_ERR_RANGE, "backward_input: M=%d outside [1, %d]", M, group->max_tokens);
  if (layer->k != group->k)
    return fail(DICTPROJ_ERR_MISMATCH, "backward_input: layer k=%d != group k=%d", layer->k, group->k);
  if (layer->device != group->device)
    return fail(DICTPROJ_ERR_MISMATCH, "backward_input: layer on device %d, group on device %d", layer->device,
                group->device);
  if (misaligned(dY, 16) || misaligned(dX, 16))
    return fail(DICTPROJ_ERR_ALIGN, "backward_input: dY and dX must be 16-byte aligned");
  if (layer->d_out % 8)
    return fail(DICTPROJ_ERR_SHAPE, "backward_input: needs d_out %% 8 == 0 (got %d)", layer->d_out);
  if (!group->ddense || layer->d_out > group->cdense_cols)
    return fail(DICTPROJ_ERR_RANGE, "backward_input: needs the group's scratch for d_out=%d; call "
                "dictproj_group_reserve_backward first", layer->d_out);
  const Range x{dX, (size_t)M * group->d_in * 2}, y{dY, (size_t)M * layer->d_out * 2};
  if (overlap(x, y)) return fail(DICTPROJ_ERR_RANGE, "backward_input: dX overlaps dY");
  int st;
  if ((st = check_device(group->device, "backward_input"))) return st;
  cudaStream_t s = (cudaStream_t)stream;
  __half* cd = reinterpret_cast<__half*>(group->cdense);
  cudaError_t e;
  if ((e = launch_densify_coeff(layer, cd, s)) != cudaSuccess)
    return cuda_fail(e, "backward_input: coefficient densify launch");
  if ((e = launch_backward_input(group, layer, static_cast<const __half*>(dY), M, cd, static_cast<__half*>(dX), s)) != cudaSuccess)
    return cuda_fail(e, "backward_input: launch");
  return DICTPROJ_OK;
}

// ---- AdamW ---------------------------------------------------------------------------
int dictproj_adamw_create(const dictproj_adamw_tensor* tensors, int n_tensors, int state_bits, dictproj_adamw** out) {
  clear_error();
  if (!tensors || !out) return fail(DICTPROJ_ERR_NULL, "adamw_create: NULL pointer");
  *out = nullptr;
  if (n_tensors < 1 || n_tensors > (1 << 20))
    return fail(DICTPROJ_ERR_RANGE, "adamw_create: n_tensors=%d outside [1, 2^20]", n_tensors);
  if (state_bits != 8 && state_bits != 32)
    return fail(DICTPROJ_ERR_RANGE, "adamw_create: state_bits=%d is neither 8 nor 32", state_bits);
  const int sb = state_bits / 8;  // bytes of a state's element
  long long chunks = 0;
  for (int i = 0; i < n_tensors; ++i) {
    const dictproj_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n >= (1ll << 32)) return fail(DICTPROJ_ERR_RANGE, "adamw_create: tensor %d: n=%lld", i, t.n);
    chunks += (t.n + kAdamwChunk - 1) / kAdamwChunk;
    if (t.n == 0) continue;
    if (!t.p || !t.g || !t.m || !t.v) return fail(DICTPROJ_ERR_NULL, "adamw_create: tensor %d: NULL array", i);
    if (state_bits == 8 && (!t.m_scale || !t.v_scale))
      return fail(DICTPROJ_ERR_NULL, "adamw_create: tensor %d: 8-bit states need their scales", i);
    if (misaligned(t.p, 4) || misaligned(t.g, 4) || misaligned(t.copy, 2) || misaligned(t.m, sb) || misaligned(t.v, sb) ||
        (state_bits == 8 && (misaligned(t.m_scale, 4) || misaligned(t.v_scale, 4))))
      return fail(DICTPROJ_ERR_ALIGN, "adamw_create: tensor %d: an array is not aligned to its elements", i);
  }
  if (chunks > 0x7fffffffll)
    return fail(DICTPROJ_ERR_RANGE, "adamw_create: more than 2^31 - 1 chunks of %d elements", kAdamwChunk);
  std::vector<AdamwChunk> table;
  bool twice;
  try {
    twice = written_twice(tensors, n_tensors, sb);
    table.resize((size_t)chunks);
  } catch (...) {
    return fail(DICTPROJ_ERR_OOM, "adamw_create: host allocation failed");
  }
  if (twice) return fail(DICTPROJ_ERR_RANGE, "adamw_create: an array that the step writes overlaps another array");
  int dev, st;
  if ((st = ensure_device(&dev))) return st;
  size_t at = 0;
  for (int i = 0; i < n_tensors; ++i) {
    const dictproj_adamw_tensor& t = tensors[i];
    const bool vec = !misaligned(t.p, 16) && !misaligned(t.g, 16) && !misaligned(t.m, 4 * sb) &&
                     !misaligned(t.v, 4 * sb) && !misaligned(t.copy, 8);
    for (long long e = 0; e < t.n; e += kAdamwChunk) {
      AdamwChunk& c = table[at++];
      c.p = t.p + e;
      c.g = t.g + e;
      c.m = static_cast<char*>(t.m) + e * sb;
      c.v = static_cast<char*>(t.v) + e * sb;
      c.m_scale = t.m_scale ? t.m_scale + e / DICTPROJ_ADAMW_BLOCK : nullptr;
      c.v_scale = t.v_scale ? t.v_scale + e / DICTPROJ_ADAMW_BLOCK : nullptr;
      c.copy = t.copy ? static_cast<char*>(t.copy) + 2 * e : nullptr;
      c.first = (uint32_t)e;
      c.count = (uint16_t)std::min<long long>(kAdamwChunk, t.n - e);
      c.vec = vec;
    }
  }
  dictproj_adamw* w = new (std::nothrow) dictproj_adamw();
  if (!w) return fail(DICTPROJ_ERR_OOM, "adamw_create: host allocation failed");
  w->device = dev;
  w->bits = state_bits;
  w->chunks = chunks;
  const size_t bytes = table.size() * sizeof(AdamwChunk);
  cudaError_t e = dmalloc((void**)&w->table, bytes);
  if (e != cudaSuccess) {
    dictproj_free_adamw(w);
    cudaGetLastError();
    return fail(DICTPROJ_ERR_OOM, "adamw_create: device allocation failed (%s)", cudaGetErrorName(e));
  }
  if ((e = h2d(w->table, table.data(), bytes))) {
    dictproj_free_adamw(w);
    cudaGetLastError();
    return cuda_fail(e, "adamw_create: copy to device");
  }
  *out = w;
  return DICTPROJ_OK;
}

void dictproj_free_adamw(dictproj_adamw* w) {
  if (!w) return;
  cudaFree(w->table);
  delete w;
}

int dictproj_adamw_step(const dictproj_adamw* w, long long step, double lr, double beta1, double beta2, double eps,
                        double weight_decay, double grad_scale, void* stream) {
  clear_error();
  if (!w) return fail(DICTPROJ_ERR_NULL, "adamw_step: NULL handle");
  if (step < 1) return fail(DICTPROJ_ERR_RANGE, "adamw_step: step=%lld < 1", step);
  if (!std::isfinite(lr) || !std::isfinite(eps) || !std::isfinite(weight_decay) || !std::isfinite(grad_scale) ||
      !std::isfinite(beta1) || !std::isfinite(beta2))
    return fail(DICTPROJ_ERR_VALUE, "adamw_step: a factor is not finite");
  if (beta1 < 0 || beta1 >= 1 || beta2 < 0 || beta2 >= 1 || eps < 0 || lr < 0 || weight_decay < 0)
    return fail(DICTPROJ_ERR_RANGE, "adamw_step: need 0 <= beta < 1 and lr, eps, weight_decay >= 0");
  int st;
  if ((st = check_device(w->device, "adamw_step"))) return st;
  AdamwFactors f;
  f.grad_scale = (float)grad_scale;
  f.b1 = (float)beta1;
  f.omb1 = (float)(1.0 - beta1);
  f.b2 = (float)beta2;
  f.omb2 = (float)(1.0 - beta2);
  f.rbc2 = (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, (double)step)));
  f.eps = (float)eps;
  f.decay = (float)(1.0 - lr * weight_decay);
  f.alpha = (float)(lr / (1.0 - std::pow(beta1, (double)step)));
  f.step = (uint32_t)step;
  const cudaError_t e = launch_adamw(w, f, (cudaStream_t)stream);
  return e == cudaSuccess ? DICTPROJ_OK : cuda_fail(e, "adamw_step: launch");
}

}  // extern "C"
