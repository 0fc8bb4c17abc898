// Lookup of scaled rows, and the gradient of the table by sorted row ids.
//
// out[t][j*D + c] = scale * table[ids[t][j]][c], ids of -1 giving zeros.
// G[r] = scale * sum over the entries i with ids[i] == r of dout[i].
//
// The gradient sorts the entries by (id, i) with a stable least-significant-
// digit radix sort, so the entries of a row are neighbours in their original
// order, and every sum is taken in a fixed order: the result does not change
// from run to run.
#include <cuda_runtime.h>
#include <stdint.h>

#include "engram_internal.h"
#include "train_device.cuh"

namespace engram {
namespace {

using train::round256;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <class E>
__global__ void __launch_bounds__(kThreads) lookup_kernel(const typename E::T* __restrict__ table, int64_t total_rows,
                                                          int32_t dim, const int32_t* __restrict__ ids, int64_t n,
                                                          int32_t n_cols, float scale,
                                                          typename E::T* __restrict__ out, int64_t out_stride,
                                                          int32_t* status) {
  const int lane = threadIdx.x & 31;
  const int64_t nw = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < n; i += nw) {
    const int32_t r = ids[i];
    const bool ok = r >= 0 && r < total_rows;
    if (!ok && r != ENGRAM_DEAD && lane == 0 && status != nullptr) atomicOr(status, ENGRAM_ST_BAD_ROW);
    const int64_t t = i / n_cols;
    typename E::T* o = out + t * out_stride + (i - t * n_cols) * dim;
    const typename E::T* src = table + static_cast<int64_t>(ok ? r : 0) * dim;
    for (int c = lane; c < dim; c += 32) E::store(o + c, ok ? scale * E::load(src + c) : 0.f);
  }
}

// ---------------------------------------------------------------- sort by id

constexpr int kItems = 16;                    // entries per thread
constexpr int kChunk = kThreads * kItems;     // entries per block
constexpr int kDigits = 256;

__device__ __forceinline__ uint32_t entry_key(int32_t id, int64_t total_rows) {
  return id >= 0 && id < total_rows ? static_cast<uint32_t>(id) : static_cast<uint32_t>(total_rows);
}

// counts[block][digit] of one pass; `first` reads the ids themselves.
__global__ void __launch_bounds__(kThreads) sort_count_kernel(const uint32_t* __restrict__ keys, bool first,
                                                              int64_t total_rows, int32_t n, int shift,
                                                              int32_t* __restrict__ counts, int32_t* status) {
  __shared__ int32_t hist[kDigits];
  hist[threadIdx.x] = 0;
  __syncthreads();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kChunk;
  bool bad = false;
  for (int k = 0; k < kItems; ++k) {
    const int64_t i = base + k * kThreads + threadIdx.x;
    if (i < n) {
      uint32_t key = keys[i];
      if (first) {
        const int32_t id = static_cast<int32_t>(key);
        bad |= id != ENGRAM_DEAD && (id < 0 || id >= total_rows);
        key = entry_key(id, total_rows);
      }
      atomicAdd(&hist[(key >> shift) & (kDigits - 1)], 1);
    }
  }
  if (bad && status != nullptr) atomicOr(status, ENGRAM_ST_BAD_ROW);
  __syncthreads();
  counts[static_cast<int64_t>(blockIdx.x) * kDigits + threadIdx.x] = hist[threadIdx.x];
}

// Moves each entry to its place: entries of smaller digits, entries of the
// same digit in earlier blocks, earlier warps, earlier rounds and lower lanes
// come before it, which keeps the pass stable.
__global__ void __launch_bounds__(kThreads) sort_move_kernel(const uint32_t* __restrict__ keys,
                                                             const int32_t* __restrict__ idx, bool first,
                                                             int64_t total_rows, int32_t n, int shift,
                                                             const int32_t* __restrict__ counts,
                                                             uint32_t* __restrict__ keys_out,
                                                             int32_t* __restrict__ idx_out) {
  __shared__ int32_t hist[kWarps][kDigits];
  __shared__ int32_t totals[kDigits];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = threadIdx.x;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) hist[w][d] = 0;
  __syncthreads();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kChunk + warp * (32 * kItems);
  uint32_t key[kItems];
  int32_t rank[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int64_t i = base + k * 32 + lane;
    key[k] = i < n ? keys[i] : 0u;
    if (first) key[k] = entry_key(static_cast<int32_t>(key[k]), total_rows);
    const uint32_t digit = i < n ? (key[k] >> shift) & (kDigits - 1) : kDigits;
    const uint32_t peers = __match_any_sync(0xffffffffu, digit);
    int32_t before = 0;
    if (i < n) before = hist[warp][digit];
    rank[k] = before + __popc(peers & ((1u << lane) - 1u));
    __syncwarp();
    if (i < n && (peers >> lane) == 1u) hist[warp][digit] = before + __popc(peers);  // the highest lane of each digit
    __syncwarp();
  }
  __syncthreads();
  int32_t total = 0, prior = 0;
  for (int b = 0; b < static_cast<int>(gridDim.x); ++b) {
    if (b == static_cast<int>(blockIdx.x)) prior = total;
    total += counts[static_cast<int64_t>(b) * kDigits + d];
  }
  totals[d] = total;
  __syncthreads();
  for (int o = 1; o < kDigits; o <<= 1) {
    const int32_t add = d >= o ? totals[d - o] : 0;
    __syncthreads();
    totals[d] += add;
    __syncthreads();
  }
  int32_t at = totals[d] - total + prior;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int32_t c = hist[w][d];
    hist[w][d] = at;
    at += c;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int64_t i = base + k * 32 + lane;
    if (i < n) {
      const int32_t to = hist[warp][(key[k] >> shift) & (kDigits - 1)] + rank[k];
      keys_out[to] = key[k];
      idx_out[to] = first ? static_cast<int32_t>(i) : idx[i];
    }
  }
}

// ------------------------------------------------------- segments of equal id

constexpr int kSegItems = 4;
constexpr int kSegChunk = kThreads * kSegItems;

__device__ __forceinline__ bool is_head(const uint32_t* keys, int64_t i, int32_t n, uint32_t none) {
  return i < n && keys[i] != none && (i == 0 || keys[i] != keys[i - 1]);
}

__global__ void __launch_bounds__(kThreads) seg_count_kernel(const uint32_t* __restrict__ keys, int32_t n,
                                                             uint32_t none, int32_t* __restrict__ counts) {
  int32_t c = 0;
  for (int k = 0; k < kSegItems; ++k)
    c += is_head(keys, static_cast<int64_t>(blockIdx.x) * kSegChunk + threadIdx.x * kSegItems + k, n, none);
  __shared__ int32_t sum;
  if (threadIdx.x == 0) sum = 0;
  __syncthreads();
  atomicAdd(&sum, c);
  __syncthreads();
  if (threadIdx.x == 0) counts[blockIdx.x] = sum;
}

// start[s] = first entry of segment s, row[s] its id; start[count] = entries
// with a row; rows past the count get -1.
__global__ void __launch_bounds__(kThreads) seg_write_kernel(const uint32_t* __restrict__ keys, int32_t n,
                                                             uint32_t none, const int32_t* __restrict__ counts,
                                                             int32_t* __restrict__ start, int32_t* __restrict__ row,
                                                             int32_t* __restrict__ count) {
  __shared__ int32_t scan[kThreads];
  __shared__ int32_t base, all;
  const int t = threadIdx.x;
  if (t == 0) base = all = 0;
  __syncthreads();
  int32_t before = 0, whole = 0;
  for (int b = t; b < static_cast<int>(gridDim.x); b += kThreads) {
    const int32_t c = counts[b];
    whole += c;
    if (b < static_cast<int>(blockIdx.x)) before += c;
  }
  atomicAdd(&base, before);
  atomicAdd(&all, whole);
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kSegChunk + t * kSegItems;
  int32_t c = 0;
  for (int k = 0; k < kSegItems; ++k) c += is_head(keys, i0 + k, n, none);
  scan[t] = c;
  __syncthreads();
  for (int o = 1; o < kThreads; o <<= 1) {
    const int32_t add = t >= o ? scan[t - o] : 0;
    __syncthreads();
    scan[t] += add;
    __syncthreads();
  }
  int32_t s = base + scan[t] - c;
  for (int k = 0; k < kSegItems; ++k) {
    const int64_t i = i0 + k;
    if (is_head(keys, i, n, none)) {
      start[s] = static_cast<int32_t>(i);
      row[s] = static_cast<int32_t>(keys[i]);
      ++s;
    }
    if (i < n && i >= all) row[i] = -1;
    // the first entry without a row ends the last segment
    if (i < n && keys[i] == none && (i == 0 || keys[i - 1] != none)) start[all] = static_cast<int32_t>(i);
    if (i == n - 1 && keys[i] != none) start[all] = n;
  }
  if (blockIdx.x == 0 && t == 0) *count = all;
}

// One warp per segment and 32-column step: the sum over the segment's entries.
template <class E>
__global__ void __launch_bounds__(kThreads) seg_sum_kernel(const typename E::T* __restrict__ dout, int64_t dout_stride,
                                                           int32_t dim, int32_t n_cols, int32_t n, float scale,
                                                           const int32_t* __restrict__ idx,
                                                           const int32_t* __restrict__ start,
                                                           const int32_t* __restrict__ row,
                                                           const int32_t* __restrict__ count, bool dense,
                                                           float* __restrict__ grad) {
  const int lane = threadIdx.x & 31;
  const int64_t nw = static_cast<int64_t>(gridDim.x) * kWarps;
  const int32_t segs = *count;
  for (int64_t s = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); s < n; s += nw) {
    if (s >= segs && dense) break;
    const int32_t a = s < segs ? start[s] : 0, b = s < segs ? start[s + 1] : 0;
    float* o = grad + (dense ? static_cast<int64_t>(row[s]) : s) * dim;
    for (int c = lane; c < dim; c += 32) {
      float sum = 0.f;
      for (int32_t k = a; k < b; ++k) {
        const int32_t i = idx[k];
        const int32_t t = i / n_cols;
        sum += E::load(dout + t * dout_stride + static_cast<int64_t>(i - t * n_cols) * dim + c);
      }
      o[c] = scale * sum;
    }
  }
}

int check_lookup(int32_t type, int64_t total_rows, int32_t row_dim, int64_t n_tokens, int32_t n_cols, int64_t stride) {
  if (!train::known_type(type)) return fail(ENGRAM_E_INVALID, "type %d is not ENGRAM_T_BF16 or ENGRAM_T_F32", type);
  if (total_rows < 0 || n_tokens < 0) return fail(ENGRAM_E_INVALID, "negative size");
  if (total_rows >= (int64_t(1) << 31) - 1) return fail(ENGRAM_E_RANGE, "total_rows must be below 2^31 - 1");
  if (row_dim < 1 || row_dim > (1 << 20)) return fail(ENGRAM_E_SHAPE, "row_dim %d not in [1, 2^20]", row_dim);
  if (n_cols < 1 || n_cols > (1 << 20)) return fail(ENGRAM_E_SHAPE, "n_cols %d not in [1, 2^20]", n_cols);
  if (n_tokens > (int64_t(1) << 31) / n_cols - 1) return fail(ENGRAM_E_RANGE, "n_tokens * n_cols must be below 2^31");
  if (stride < static_cast<int64_t>(n_cols) * row_dim)
    return fail(ENGRAM_E_SHAPE, "row stride %lld below n_cols * row_dim", static_cast<long long>(stride));
  return ENGRAM_OK;
}

// The parts of the gradient's workspace.
struct GradSpace {
  uint32_t* key[2];
  int32_t* idx[2];
  int32_t* start;
  int32_t* row;
  int32_t* counts;
  int32_t* count;
  size_t bytes;
};

GradSpace grad_space(void* base, int64_t n) {
  GradSpace s;
  char* p = static_cast<char*>(base);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* q = p + at;
    at += round256(bytes);
    return q;
  };
  const size_t words = static_cast<size_t>(n + 1) * 4;
  for (int k = 0; k < 2; ++k) s.key[k] = reinterpret_cast<uint32_t*>(take(words));
  for (int k = 0; k < 2; ++k) s.idx[k] = reinterpret_cast<int32_t*>(take(words));
  s.start = reinterpret_cast<int32_t*>(take(words));
  s.row = reinterpret_cast<int32_t*>(take(words));
  const size_t blocks = static_cast<size_t>((n + kChunk - 1) / kChunk);
  s.counts = reinterpret_cast<int32_t*>(take(blocks * kDigits * 4));
  s.count = reinterpret_cast<int32_t*>(take(4));
  s.bytes = at;
  return s;
}

int lookup_grad(const void* dout_d, int32_t type, int64_t dout_stride, const int32_t* ids_d, int64_t n_tokens,
                int32_t n_cols, int32_t row_dim, int64_t total_rows, float scale, bool dense, int32_t* rows_d,
                float* grad_d, int32_t* count_d, void* workspace_d, size_t workspace_bytes, int32_t* status_d,
                void* stream) {
  int rc = check_lookup(type, total_rows, row_dim, n_tokens, n_cols, dout_stride);
  if (rc) return rc;
  const int64_t n64 = n_tokens * n_cols;
  const int32_t n = static_cast<int32_t>(n64);
  cudaStream_t st = as_stream(stream);
  if (dense && total_rows == 0) return ENGRAM_OK;
  if (!grad_d && (dense || n > 0)) return fail(ENGRAM_E_INVALID, "null device pointer");
  if (!dense && (!count_d || (n > 0 && !rows_d))) return fail(ENGRAM_E_INVALID, "null device pointer");
  if (n > 0 && (!dout_d || !ids_d || !workspace_d)) return fail(ENGRAM_E_INVALID, "null device pointer");
  if (!aligned(grad_d, 4) || !aligned(dout_d, train::type_bytes(type)))
    return fail(ENGRAM_E_ALIGN, "dout and grad must be aligned to their elements");
  if (n > 0 && !aligned(workspace_d, 256)) return fail(ENGRAM_E_ALIGN, "workspace must be 256-byte aligned");
  if (n > 0 && workspace_bytes < engram_lookup_grad_workspace_bytes(n_tokens, n_cols, row_dim))
    return fail(ENGRAM_E_RANGE, "workspace too small");
  int sms = 0;
  if ((rc = check_device(&sms))) return rc;
  if (dense) cudaMemsetAsync(grad_d, 0, static_cast<size_t>(total_rows) * row_dim * 4, st);
  if (n == 0) {
    if (!dense) cudaMemsetAsync(count_d, 0, 4, st);
    return check_launch("lookup gradient");
  }
  GradSpace w = grad_space(workspace_d, n);
  if (dense) {
    rows_d = w.row;
    count_d = w.count;
  }
  int bits = 0;
  while ((total_rows >> bits) != 0) ++bits;
  const int passes = bits == 0 ? 1 : (bits + 7) / 8;
  const int blocks = (n + kChunk - 1) / kChunk;
  const uint32_t* kin = reinterpret_cast<const uint32_t*>(ids_d);
  const int32_t* iin = nullptr;
  for (int p = 0; p < passes; ++p) {
    const bool first = p == 0;
    sort_count_kernel<<<blocks, kThreads, 0, st>>>(kin, first, total_rows, n, 8 * p, w.counts, status_d);
    sort_move_kernel<<<blocks, kThreads, 0, st>>>(kin, iin, first, total_rows, n, 8 * p, w.counts, w.key[p & 1],
                                                  w.idx[p & 1]);
    kin = w.key[p & 1];
    iin = w.idx[p & 1];
  }
  const int sblocks = (n + kSegChunk - 1) / kSegChunk;
  const uint32_t none = static_cast<uint32_t>(total_rows);
  seg_count_kernel<<<sblocks, kThreads, 0, st>>>(kin, n, none, w.counts);
  seg_write_kernel<<<sblocks, kThreads, 0, st>>>(kin, n, none, w.counts, w.start, rows_d, count_d);
  const int64_t want = (n64 + kWarps - 1) / kWarps, cap = static_cast<int64_t>(sms) * 8;
  const int gblocks = static_cast<int>(want < cap ? want : cap);
  if (type == ENGRAM_T_BF16)
    seg_sum_kernel<train::Bf16><<<gblocks, kThreads, 0, st>>>(static_cast<const uint16_t*>(dout_d), dout_stride,
                                                              row_dim, n_cols, n, scale, iin, w.start, rows_d, count_d,
                                                              dense, grad_d);
  else
    seg_sum_kernel<train::F32><<<gblocks, kThreads, 0, st>>>(static_cast<const float*>(dout_d), dout_stride, row_dim,
                                                             n_cols, n, scale, iin, w.start, rows_d, count_d, dense,
                                                             grad_d);
  return check_launch("lookup gradient");
}

}  // namespace
}  // namespace engram

using namespace engram;

extern "C" int engram_lookup(const void* table_d, int32_t type, int64_t total_rows, int32_t row_dim,
                             const int32_t* row_ids_d, int64_t n_tokens, int32_t n_cols, float scale, void* out_d,
                             int64_t out_stride, int32_t* status_d, void* stream) {
  int rc = check_lookup(type, total_rows, row_dim, n_tokens, n_cols, out_stride);
  if (rc) return rc;
  if (n_tokens == 0) return ENGRAM_OK;
  if ((!table_d && total_rows > 0) || !row_ids_d || !out_d) return fail(ENGRAM_E_INVALID, "null device pointer");
  if (!aligned(table_d, train::type_bytes(type)) || !aligned(out_d, train::type_bytes(type)))
    return fail(ENGRAM_E_ALIGN, "table and out must be aligned to their elements");
  int sms = 0;
  if ((rc = check_device(&sms))) return rc;
  const int64_t n = n_tokens * n_cols;
  const int64_t want = (n + kWarps - 1) / kWarps, cap = static_cast<int64_t>(sms) * 8;
  const int blocks = static_cast<int>(want < cap ? want : cap);
  if (type == ENGRAM_T_BF16)
    lookup_kernel<train::Bf16><<<blocks, kThreads, 0, as_stream(stream)>>>(
        static_cast<const uint16_t*>(table_d), total_rows, row_dim, row_ids_d, n, n_cols, scale,
        static_cast<uint16_t*>(out_d), out_stride, status_d);
  else
    lookup_kernel<train::F32><<<blocks, kThreads, 0, as_stream(stream)>>>(
        static_cast<const float*>(table_d), total_rows, row_dim, row_ids_d, n, n_cols, scale,
        static_cast<float*>(out_d), out_stride, status_d);
  return check_launch("lookup_kernel");
}

extern "C" size_t engram_lookup_grad_workspace_bytes(int64_t n_tokens, int32_t n_cols, int32_t row_dim) {
  if (n_tokens < 0 || n_cols < 1 || row_dim < 1) return 0;
  return grad_space(nullptr, n_tokens * n_cols).bytes;
}

extern "C" int engram_lookup_grad(const void* dout_d, int32_t type, int64_t dout_stride, const int32_t* row_ids_d,
                                  int64_t n_tokens, int32_t n_cols, int32_t row_dim, int64_t total_rows, float scale,
                                  float* grad_d, void* workspace_d, size_t workspace_bytes, int32_t* status_d,
                                  void* stream) {
  return lookup_grad(dout_d, type, dout_stride, row_ids_d, n_tokens, n_cols, row_dim, total_rows, scale, true, nullptr,
                     grad_d, nullptr, workspace_d, workspace_bytes, status_d, stream);
}

extern "C" int engram_lookup_grad_rows(const void* dout_d, int32_t type, int64_t dout_stride,
                                       const int32_t* row_ids_d, int64_t n_tokens, int32_t n_cols, int32_t row_dim,
                                       int64_t total_rows, float scale, int32_t* rows_d, float* grad_d,
                                       int32_t* count_d, void* workspace_d, size_t workspace_bytes,
                                       int32_t* status_d, void* stream) {
  return lookup_grad(dout_d, type, dout_stride, row_ids_d, n_tokens, n_cols, row_dim, total_rows, scale, false, rows_d,
                     grad_d, count_d, workspace_d, workspace_bytes, status_d, stream);
}
