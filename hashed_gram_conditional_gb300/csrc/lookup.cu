// Lookup of scaled rows, and the gradient of the table by sorted row ids.
//
// out[t][j*D + c] = scale * table[ids[t][j]][c], ids of -1 giving zeros.
// G[r] = scale * sum over the entries i with ids[i] == r of dout[i].
//
// The gradient sorts the entries by (id, i) with a stable least-significant-
// digit radix sort (Knuth, The Art of Computer Programming, vol. 3, 5.2.5), so
// the entries of a row are neighbours in their original order, and every sum is
// taken in a fixed order: the result does not change from run to run.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "engram_internal.h"
#include "train_device.cuh"

namespace engram {
namespace {

using train::round256;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// ---------------------------------------------------------------- the lookup

// x / d for 0 <= x < 2^31 by a multiplication (Granlund and Montgomery 1994).
struct Divider {
  uint32_t d, m, shift;
};
inline Divider make_divider(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  return Divider{d, static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1), s};
}
__device__ __forceinline__ uint32_t divide(uint32_t x, const Divider& v) { return (__umulhi(x, v.m) + x) >> v.shift; }

template <int kBytes>
struct Piece;
template <>
struct Piece<16> {
  using T = uint4;
};
template <>
struct Piece<8> {
  using T = uint2;
};
template <>
struct Piece<4> {
  using T = uint32_t;
};
template <>
struct Piece<2> {
  using T = uint16_t;
};

template <class E, int kBytes>
__device__ __forceinline__ typename Piece<kBytes>::T scaled(const typename Piece<kBytes>::T& x, float scale) {
  if constexpr (kBytes == 2) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(scale * __uint_as_float(static_cast<uint32_t>(x) << 16)));
  } else {
    typename Piece<kBytes>::T r;
    const uint32_t* in = reinterpret_cast<const uint32_t*>(&x);
    uint32_t* out = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
    for (int k = 0; k < kBytes / 4; ++k) {
      if constexpr (E::kBytes == 4) {
        out[k] = __float_as_uint(scale * __uint_as_float(in[k]));
      } else {
        const __nv_bfloat162 b = __floats2bfloat162_rn(scale * __uint_as_float(in[k] << 16),
                                                       scale * __uint_as_float(in[k] & 0xffff0000u));
        out[k] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    return r;
  }
}

// The output as one sequence of pieces of kBytes, the widest that rows and
// pointers are aligned to: a block takes kAtOnce pieces a thread, its threads
// neighbouring ones, all loads before the stores.  The rows' ids come from the
// first-level cache, which their neighbours share.  Bound by memory: rows of
// 512 bytes are read at random and written in order (16,384 x 24 rows of 256
// bf16, 201 MB out: 52 us, the frequent rows coming from the L2 cache).
constexpr int kAtOnce = 2;  // 55 us for 16,384 x 24 rows of 256 bf16; 4: 61 us, 8: 72 us

template <class E, int kBytes>
__global__ void __launch_bounds__(kThreads) lookup_kernel(const typename Piece<kBytes>::T* __restrict__ table,
                                                          int64_t total_rows, Divider per_row, const int32_t* __restrict__ ids,
                                                          int64_t pieces, int32_t n_cols, float scale,
                                                          typename Piece<kBytes>::T* __restrict__ out, int64_t out_pieces,
                                                          int32_t* status) {
  using T = typename Piece<kBytes>::T;
  const bool contiguous = out_pieces == static_cast<int64_t>(n_cols) * per_row.d;
  for (int64_t p0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kAtOnce); p0 < pieces;
       p0 += static_cast<int64_t>(gridDim.x) * (kThreads * kAtOnce)) {
    const int64_t e0 = p0 / per_row.d;  // the block's first entry
    const uint32_t in_row = static_cast<uint32_t>(p0 - e0 * per_row.d);
    T x[kAtOnce];
    int64_t to[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const uint32_t at = in_row + threadIdx.x + k * kThreads;
      const int64_t p = p0 + threadIdx.x + k * kThreads;
      x[k] = T{};
      to[k] = -1;
      if (p < pieces) {
        const uint32_t e = divide(at, per_row), c = at - e * per_row.d;
        const int64_t i = e0 + e;
        const int32_t r = __ldg(ids + i);
        if (r >= 0 && r < total_rows) x[k] = __ldg(table + static_cast<int64_t>(r) * per_row.d + c);
        else if (r != ENGRAM_DEAD && c == 0 && status != nullptr) atomicOr(status, ENGRAM_ST_BAD_ROW);
        to[k] = p;
        if (!contiguous) {
          const int64_t t = i / n_cols;
          to[k] = t * out_pieces + (i - t * n_cols) * per_row.d + c;
        }
        // (a row that is not there gives +0 whatever the scale)
        if (!(r >= 0 && r < total_rows)) to[k] = ~to[k];
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (p0 + threadIdx.x + k * kThreads >= pieces) break;
      if (to[k] >= 0) out[to[k]] = scaled<E, kBytes>(x[k], scale);
      else out[~to[k]] = T{};
    }
  }
}

template <class E, int kBytes>
int launch_lookup(const void* table, int64_t total_rows, int32_t row_dim, const int32_t* ids, int64_t n, int32_t n_cols,
                  float scale, void* out, int64_t out_stride, int32_t* status, int sms, cudaStream_t st) {
  using T = typename Piece<kBytes>::T;
  const Divider per_row = make_divider(static_cast<uint32_t>(static_cast<int64_t>(row_dim) * E::kBytes / kBytes));
  const int64_t pieces = n * per_row.d;
  const int64_t want = (pieces + kThreads * kAtOnce - 1) / (kThreads * kAtOnce), cap = static_cast<int64_t>(sms) * 64;
  lookup_kernel<E, kBytes><<<static_cast<int>(want < cap ? want : cap), kThreads, 0, st>>>(
      static_cast<const T*>(table), total_rows, per_row, ids, pieces, n_cols, scale, static_cast<T*>(out),
      out_stride * E::kBytes / kBytes, status);
  return check_launch("lookup_kernel");
}

template <class E>
int lookup_rows(const void* table, int64_t total_rows, int32_t row_dim, const int32_t* ids, int64_t n, int32_t n_cols,
                float scale, void* out, int64_t out_stride, int32_t* status, int sms, cudaStream_t st) {
  auto fits = [&](int bytes) {
    return static_cast<int64_t>(row_dim) * E::kBytes % bytes == 0 && out_stride * E::kBytes % bytes == 0 &&
           aligned(table, bytes) && aligned(out, bytes);
  };
  if (fits(16)) return launch_lookup<E, 16>(table, total_rows, row_dim, ids, n, n_cols, scale, out, out_stride, status, sms, st);
  if (fits(8)) return launch_lookup<E, 8>(table, total_rows, row_dim, ids, n, n_cols, scale, out, out_stride, status, sms, st);
  if (E::kBytes == 4 || fits(4))
    return launch_lookup<E, 4>(table, total_rows, row_dim, ids, n, n_cols, scale, out, out_stride, status, sms, st);
  return launch_lookup<E, E::kBytes>(table, total_rows, row_dim, ids, n, n_cols, scale, out, out_stride, status, sms, st);
}

// ---------------------------------------------------------------- sort by id

// One kernel sorts: its blocks (all resident, a cooperative launch) share out
// the entries in order and meet at a barrier between counting and moving.  Ids
// of 26 bits take three passes of 9 bits.  A few thousand entries are one
// block's work, without barriers.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kItems = 4;                         // entries per thread and round
constexpr int kRound = kSortThreads * kItems;     // entries per block and round
constexpr int kDigitBits = 9;
constexpr int kMaxDigits = 1 << kDigitBits;
constexpr int kMarked = kSortWarps * kMaxDigits * 16;  // rows that clear_meanwhile can mark
constexpr int kGroup = 13;  // blocks whose digits are summed up for the others: 12 groups of 152 blocks

__device__ __forceinline__ uint32_t entry_key(int32_t id, int64_t total_rows) {
  return id >= 0 && id < total_rows ? static_cast<uint32_t>(id) : static_cast<uint32_t>(total_rows);
}

// A sorted entry: its id and its place i (one 8-byte store where it is moved to).
struct __align__(8) Entry {
  uint32_t key;
  int32_t idx;
};
__device__ __forceinline__ Entry load_entry(const Entry* p) {
  const uint2 v = __ldcg(reinterpret_cast<const uint2*>(p));
  return Entry{v.x, static_cast<int32_t>(v.y)};
}

__device__ __forceinline__ bool is_head(const Entry* e, int64_t i, int32_t n, uint32_t none) {
  if (i >= n) return false;
  const uint32_t k = load_entry(e + i).key;
  return k != none && (i == 0 || k != load_entry(e + i - 1).key);
}

constexpr int kMaxRange = 256;  // rows that a block clears at a time, at most

// count floats from row on, by a warp: 16 bytes a lane from the first 16-byte
// boundary to the last
__device__ __forceinline__ void zero_rows(float* row, int64_t count, int lane) {
  const int64_t head = (4 - (reinterpret_cast<uintptr_t>(row) / 4 & 3)) & 3;
  const int64_t c0 = head < count ? head : count, c1 = c0 + (count - c0) / 4 * 4;
  if (lane < c0) row[lane] = 0.f;
#pragma unroll 4
  for (int64_t c = c0 + lane * 4; c < c1; c += 128)
    __stcs(reinterpret_cast<float4*>(row + c), make_float4(0.f, 0.f, 0.f, 0.f));
  if (c1 + lane < count) row[c1 + lane] = 0.f;
}

struct SortArgs {
  const int32_t* ids;
  int64_t total_rows;
  int32_t n, per;  // entries, and how many each block handles
  int32_t passes, bits;
  Entry* list[2];
  int32_t blocks;   // that sort; further ones clear rows
  int32_t* counts;  // [block][digit]
  int32_t* groups;  // [pass][group of kGroup blocks][digit], zeroed by the caller
  int32_t* barrier;  // [0] arrivals, [1] whether the list is sorted
  int32_t absent;    // arrivals that every wait expects beyond the blocks' (0; see engram_selftest_grad_wait)
  int32_t chunk, chunks;  // sorted entries that are summed together (see seg_sum_kernel), and how many such
  int32_t* base;   // segments that begin in the block's chunks before each chunk, or null
  int32_t chunks_per;  // chunks whose segments each block counts
  int32_t* heads;      // [block]: segments that begin in its chunks
  int32_t* next;   // the summing kernel's two counters, zeroed here where a block sorts alone
  int32_t dim, range;  // the result's columns, and rows that a block clears at a time (dense form)
  float* grad;
  int32_t* status;
};

constexpr int32_t kGaveUp = 1 << 30;  // more than any call's tasks (2^25 for 2^37 elements, which fill the memory)

// All blocks meet; false when the wait ran out (the blocks are co-resident, so
// that means a broken launch).  The list may hold anything then, so the counter
// of the tasks that follow it is set behind the last of them.  What a block's
// threads wrote before is released by its first thread, which they meet first.
__device__ __forceinline__ bool meet(const SortArgs& a, int32_t& met) {
  __syncthreads();
  if (a.blocks == 1) return true;
  const int32_t want = ++met * a.blocks + a.absent;
  bool ok = true;
  if (threadIdx.x == 0) {
    __threadfence();
    asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(a.barrier) : "memory");
    const long long begun = clock64();
    while (true) {
      int32_t v;
      asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(a.barrier) : "memory");
      if (v >= want) break;
      if (clock64() - begun > kWaitBudgetCycles) {
        ok = false;
        atomicMax(a.next, kGaveUp);
        if (a.status != nullptr) atomicOr(a.status, ENGRAM_ST_TIMEOUT);
        break;
      }
    }
    __threadfence();
  }
  return __syncthreads_and(ok);
}

// What the blocks that do not sort do meanwhile: they clear rows that no entry
// names, which a bit per row in shared memory tells them, range by range from the
// summing kernel's counter, until the list is sorted.  They wait for nothing.
__device__ __forceinline__ void clear_meanwhile(const SortArgs& a, uint32_t* bits, int32_t& taken) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int w = threadIdx.x; w < (a.total_rows + 31) / 32; w += kSortThreads) bits[w] = 0u;
  __syncthreads();
#pragma unroll 4
  for (int32_t i = threadIdx.x; i < a.n; i += kSortThreads) {
    const int32_t id = __ldg(a.ids + i);
    if (id >= 0 && id < a.total_rows && !(bits[id >> 5] >> (id & 31) & 1u)) atomicOr(bits + (id >> 5), 1u << (id & 31));
  }
  while (true) {
    __syncthreads();
    if (threadIdx.x == 0) taken = *reinterpret_cast<volatile int32_t*>(a.barrier + 1) != 0 ? -1 : atomicAdd(a.next + 1, 1);
    __syncthreads();
    const int64_t r0 = static_cast<int64_t>(taken) * a.range;
    if (r0 < 0 || r0 >= a.total_rows) return;
    for (int r = warp; r < a.range && r0 + r < a.total_rows; r += kSortWarps)
      if (!(bits[(r0 + r) >> 5] >> ((r0 + r) & 31) & 1u)) zero_rows(a.grad + (r0 + r) * a.dim, a.dim, lane);
  }
}

// Moves each entry to its place: entries of smaller digits, entries of the
// same digit in earlier blocks, rounds, warps and lanes come before it, which
// keeps the passes stable.  Where a block's entries are one round (up to
// 622,592 entries on 152 SMs) they are ranked while they are counted and stay in
// registers over the barrier; otherwise they are counted first.
//
// Bound by waits, not by bytes: a pass is two barriers, one scattered 8-byte
// store an entry and the counts in between.  393,216 ids of 26 bits in three
// passes: 44 us; 16,384 of 17 bits in two, by 16 blocks: 25 us, in which the other
// blocks clear rows (dense gradient of 16,384 rows of 5120 into 99,092: 348 us
// without that, 336 with it).
__global__ void __launch_bounds__(kSortThreads) sort_kernel(SortArgs a) {
  __shared__ __align__(16) uint16_t hist[kSortWarps][kMaxDigits];
  __shared__ int32_t place[kMaxDigits], half[kMaxDigits], warp_sum[kSortWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int digits = 1 << a.bits, blocks = a.blocks, me = static_cast<int>(blockIdx.x);
  if (me >= blocks) {
    static_assert(sizeof(hist) * 8 == kMarked, "a bit for every row");
    allow_dependent_launch();
    clear_meanwhile(a, reinterpret_cast<uint32_t*>(hist), place[0]);
    return;
  }
  const int32_t e0 = a.n < static_cast<int64_t>(me) * a.per ? a.n : me * a.per;
  const int32_t e1 = a.n - e0 < a.per ? a.n : e0 + a.per;
  const bool one_round = a.per <= kRound;
  int32_t met = 0;
  allow_dependent_launch();
  if (gridDim.x == 1 && tid < 2) a.next[tid] = 0;

  for (int pass = 0; pass < a.passes; ++pass) {
    const bool first = pass == 0;
    const int shift = pass * a.bits;
    const Entry* in_list = a.list[(pass + 1) & 1];
    Entry* out_list = a.list[pass & 1];
    auto digit_of = [&](uint32_t key) { return (key >> shift) & (digits - 1); };
    auto entry_at = [&](int32_t i) {
      return first ? Entry{entry_key(__ldg(a.ids + i), a.total_rows), i} : load_entry(in_list + i);
    };
    bool bad = false;

    // a round's entries, each with its rank among those of its warp and digit;
    // then hist: its digit's entries in earlier warps, half: in the round
    Entry entry[kItems];
    int rank[kItems];
    auto in_round = [&](int32_t r0, int k) {
      return static_cast<int64_t>(r0) + warp * (32 * kItems) + lane + 32 * k < e1;
    };
    auto take = [&](int32_t r0) {
      const int32_t at = r0 + warp * (32 * kItems) + lane;  // (below 2^31 where it is used)
      for (int d = lane; d < digits; d += 32) hist[warp][d] = 0;
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        entry[k] = in_round(r0, k) ? entry_at(at + 32 * k) : Entry{0u, 0};
        if (first && in_round(r0, k) && entry[k].key == static_cast<uint32_t>(a.total_rows))
          bad |= __ldg(a.ids + at + 32 * k) != ENGRAM_DEAD;
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        const bool in = in_round(r0, k);
        const uint32_t d = digit_of(entry[k].key);
        uint32_t peers = __ballot_sync(0xffffffffu, in);  // the lanes with the same digit, bit by bit
#pragma unroll
        for (int bit = 0; bit < kDigitBits; ++bit) {
          const bool one = d >> bit & 1u;
          const uint32_t ones = __ballot_sync(0xffffffffu, one);
          peers &= one ? ones : ~ones;
        }
        const int before = in ? hist[warp][d] : 0;
        rank[k] = before + __popc(peers & ((1u << lane) - 1u));
        __syncwarp();
        if (in && (peers >> lane) == 1u) hist[warp][d] = static_cast<uint16_t>(before + __popc(peers));  // the highest lane
        __syncwarp();
      }
      __syncthreads();
      if (tid < digits) {
        int c[kSortWarps], run = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) c[w] = hist[w][tid];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
          hist[w][tid] = static_cast<uint16_t>(run);
          run += c[w];
        }
        half[tid] = run;
      }
      __syncthreads();
    };
    auto put = [&](int32_t r0) {
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        if (in_round(r0, k)) {
          const uint32_t d = digit_of(entry[k].key);
          const int32_t to = place[d] + hist[warp][d] + rank[k];
          __stcg(reinterpret_cast<uint2*>(out_list + to), make_uint2(entry[k].key, static_cast<uint32_t>(entry[k].idx)));
        }
      }
    };

    // this block's digits
    if (one_round) {
      take(e0);
      if (tid < digits) place[tid] = half[tid];
    } else {
      if (tid < digits) place[tid] = 0;
      __syncthreads();
      for (int32_t i = e0 + tid; i < e1; i += kSortThreads) {
        const Entry e = entry_at(i);
        atomicAdd(&place[digit_of(e.key)], 1);
      }
      __syncthreads();
    }
    int32_t* groups = nullptr;
    if (blocks > 1) {
      const int n_groups = (blocks + kGroup - 1) / kGroup;
      groups = a.groups + static_cast<int64_t>(pass) * n_groups * digits;
      if (tid < digits) {
        __stcg(a.counts + static_cast<int64_t>(me) * digits + tid, place[tid]);
        if (place[tid] != 0) atomicAdd(groups + (me / kGroup) * digits + tid, place[tid]);
      }
      if (!meet(a, met)) return;
    }

    // per digit: its entries in all blocks, and in the blocks before this one:
    // whole groups, then the blocks of this one's group.  Eight neighbouring
    // lanes sum four digits, an eighth of the groups and blocks each.
    int32_t total = 0, prior = 0;
    if (blocks > 1) {
      constexpr int kParts = 8;
      static_assert(kSortThreads / kParts * 4 >= kMaxDigits, "every digit is summed");
      const int quad = tid / kParts, part = tid % kParts;
      const int my_group = me / kGroup, n_groups = (blocks + kGroup - 1) / kGroup;
      int all[4] = {}, early[4] = {};
      auto add = [](int (&to)[4], const int4& c, bool on) {
        to[0] += on ? c.x : 0;
        to[1] += on ? c.y : 0;
        to[2] += on ? c.z : 0;
        to[3] += on ? c.w : 0;
      };
      if (4 * quad < digits) {
#pragma unroll 4
        for (int g = part; g < n_groups; g += kParts) {
          const int4 c = __ldcg(reinterpret_cast<const int4*>(groups + static_cast<int64_t>(g) * digits + 4 * quad));
          add(all, c, true);
          add(early, c, g < my_group);
        }
#pragma unroll 2
        for (int b = my_group * kGroup + part; b < me; b += kParts)
          add(early, __ldcg(reinterpret_cast<const int4*>(a.counts + static_cast<int64_t>(b) * digits + 4 * quad)), true);
      }
#pragma unroll
      for (int o = 1; o < kParts; o <<= 1)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          all[j] += __shfl_xor_sync(0xffffffffu, all[j], o);
          early[j] += __shfl_xor_sync(0xffffffffu, early[j], o);
        }
      __syncthreads();  // (half may still be read as this round's counts)
      if (part == 0 && 4 * quad < digits) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          half[4 * quad + j] = all[j];
          place[4 * quad + j] = early[j];
        }
      }
      __syncthreads();
      if (tid < digits) {
        total = half[tid];
        prior = place[tid];
      }
    } else if (tid < digits) {
      total = place[tid];
    }
    // exclusive sums over the digits (the first warps' threads hold one each)
    int32_t x = tid < digits ? total : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    if (tid < digits) {
      for (int w = 0; w < warp; ++w) x += warp_sum[w];
      place[tid] = x - total + prior;
    }
    __syncthreads();

    if (one_round) {
      put(e0);
    } else {
      for (int32_t r0 = e0; r0 < e1; r0 += kRound) {
        take(r0);
        put(r0);
        __syncthreads();
        if (tid < digits) place[tid] += half[tid];
        __syncthreads();
      }
    }
    if (bad && a.status != nullptr) atomicOr(a.status, ENGRAM_ST_BAD_ROW);
    if (!meet(a, met)) return;
  }
  if (a.base == nullptr) {
    if (me == 0 && tid == 0) *reinterpret_cast<volatile int32_t*>(a.barrier + 1) = 1;
    return;
  }

  // segments that begin in each chunk, summed up over the chunks before it of
  // this block's; the blocks' own sums are left to those who read them
  const uint32_t none = static_cast<uint32_t>(a.total_rows);
  const Entry* list = a.list[(a.passes - 1) & 1];
  const int32_t c0 = a.chunks < static_cast<int64_t>(me) * a.chunks_per ? a.chunks : me * a.chunks_per;
  const int32_t c1 = a.chunks - c0 < a.chunks_per ? a.chunks : c0 + a.chunks_per;
  int32_t before = 0;
  for (int32_t r0 = c0; r0 < c1; r0 += kSortThreads) {  // (uniform over the block)
    __syncthreads();
    place[tid & (kMaxDigits - 1)] = half[tid & (kMaxDigits - 1)] = 0;  // heads of the round's chunks
    __syncthreads();
    int32_t* heads_of = tid < kMaxDigits ? place : half;  // the thread's own
    for (int32_t c = r0 + warp; c < c1 && c < r0 + kSortThreads; c += kSortWarps) {
      int32_t heads = 0;
      for (int k = 0; k < a.chunk; k += 32)
        heads += __popc(__ballot_sync(0xffffffffu, k + lane < a.chunk &&
                                                       is_head(list, static_cast<int64_t>(c) * a.chunk + k + lane, a.n, none)));
      if (lane == 0) (c - r0 < kMaxDigits ? place : half)[(c - r0) & (kMaxDigits - 1)] = heads;
    }
    __syncthreads();
    const int32_t c = r0 + tid, own = heads_of[tid & (kMaxDigits - 1)];
    int32_t x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int32_t whole = 0;
    for (int w = 0; w < kSortWarps; ++w) {
      if (w < warp) x += warp_sum[w];
      whole += warp_sum[w];
    }
    if (c < c1) a.base[c] = before + x - own;
    before += whole;
  }
  if (tid == 0) a.heads[me] = before;
}

// ------------------------------------------------------- segments of equal id

// The sorted entries are summed in chunks: equal work however long or short the
// segments are.  A segment inside its chunk goes straight to the result; one
// that crosses a border leaves a part in each chunk it touches, and the parts
// are joined in order afterwards.

// 8 bf16 or 4 fp32 columns of a row per lane.  Aligned rows are read 16 bytes
// a lane; others column by column, the lanes next to one another.
template <class E>
constexpr int kCols = 16 / E::kBytes;

template <class E, bool kAligned>
__device__ __forceinline__ int col_of(int j, int lane, int lanes) {
  return kAligned ? lane * kCols<E> + j : j * lanes + lane;
}

template <class E, bool kAligned>
__device__ __forceinline__ uint4 load_cols(const typename E::T* row, int c0, int lane, int lanes, int dim) {
  uint4 r = make_uint4(0u, 0u, 0u, 0u);
  if constexpr (kAligned) {
    const int c = c0 + lane * kCols<E>;
    if (c < dim) r = __ldg(reinterpret_cast<const uint4*>(row + c));
  } else {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < kCols<E>; ++j) {
      const int c = c0 + j * lanes + lane;
      if (c < dim) {
        if constexpr (E::kBytes == 2) w[j / 2] |= static_cast<uint32_t>(row[c]) << (16 * (j & 1));
        else w[j] = __float_as_uint(row[c]);
      }
    }
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return r;
}

template <class E>
__device__ __forceinline__ void add_cols(const uint4& x, float (&acc)[kCols<E>]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int j = 0; j < kCols<E>; ++j) {
    if constexpr (E::kBytes == 2) acc[j] += __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
    else acc[j] += __uint_as_float(w[j]);
  }
}

// fp32 rows of results and parts.
template <class E, bool kAligned>
__device__ __forceinline__ void store_cols(float* row, int c0, int lane, int lanes, int dim, float scale,
                                           const float (&v)[kCols<E>]) {
  if constexpr (kAligned) {
    const int c = c0 + lane * kCols<E>;
    if (c < dim) {
      if constexpr (kCols<E> == 8) {
        // one 32-byte store a lane: whole sectors, rows of 8 n floats on 32-byte boundaries
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(row + c), "f"(scale * v[0]),
                     "f"(scale * v[1]), "f"(scale * v[2]), "f"(scale * v[3]), "f"(scale * v[4]), "f"(scale * v[5]),
                     "f"(scale * v[6]), "f"(scale * v[7])
                     : "memory");
      } else {
        *reinterpret_cast<float4*>(row + c) = make_float4(scale * v[0], scale * v[1], scale * v[2], scale * v[3]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < kCols<E>; ++j) {
      const int c = c0 + j * lanes + lane;
      if (c < dim) row[c] = scale * v[j];
    }
  }
}

template <class E>
struct SumArgs {
  const typename E::T* dout;
  int64_t dout_stride;
  int32_t dim, n_cols, n, chunk, chunks, tiles;  // tiles of a row's columns
  float scale;
  const Entry* list;
  uint32_t none;
  bool dense, contiguous;
  const int32_t* base;   // rows form: see SortArgs
  const int32_t* heads;
  int32_t chunks_per, heads_count;
  int32_t* count;        // rows form: all segments
  int64_t total_rows;    // dense form
  int32_t range;         // dense form: rows that a block clears at a time
  float* grad;
  int32_t* rows;
  float *head, *tail;    // [chunk][dim]: the parts of a segment from before, of one that goes on
  int32_t* next;         // [0] next task (from kGaveUp on: there is no list), [1] next rows to clear (zeroed by the sort)
};

// before[b]: segments that begin in the chunks of the sort's blocks before b, and
// last all of them; filled by the block's first warp.
constexpr int kMaxSortBlocks = 256;  // one per SM
template <class E>
__device__ __forceinline__ void sum_heads(const SumArgs<E>& a, int32_t (&before)[kMaxSortBlocks + 1]) {
  const int lane = threadIdx.x & 31;
  if (threadIdx.x >= 32) return;
  int32_t run = 0;
  for (int b0 = 0; b0 < a.heads_count; b0 += 32) {
    const int32_t c = b0 + lane < a.heads_count ? a.heads[b0 + lane] : 0;
    int32_t x = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (b0 + lane < a.heads_count) before[b0 + lane] = run + x - c;
    run += __shfl_sync(0xffffffffu, x, 31);
  }
  if (lane == 0) before[a.heads_count] = run;
}

template <class E>
__device__ __forceinline__ const typename E::T* entry_row(const SumArgs<E>& a, int32_t i) {
  if (a.contiguous) return a.dout + static_cast<int64_t>(i) * a.dim;
  const int32_t t = i / a.n_cols;
  return a.dout + t * a.dout_stride + static_cast<int64_t>(i - t * a.n_cols) * a.dim;
}

// A sort that gave up leaves a list of anything, which must not be followed: there
// is no gradient then, but zeros and no rows.
template <class E>
__device__ __forceinline__ void no_gradient(const SumArgs<E>& a) {
  if (!a.dense && blockIdx.x == 0 && threadIdx.x == 0) *a.count = 0;
  const int64_t rows = a.dense ? a.total_rows : a.n;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32; r < rows;
       r += static_cast<int64_t>(gridDim.x) * kWarps) {
    if (!a.dense && threadIdx.x % 32 == 0) a.rows[r] = -1;
    zero_rows(a.grad + r * a.dim, a.dim, threadIdx.x % 32);
  }
}

// kLanes lanes handle one (chunk, tile of kLanes * kCols columns) at a time,
// taken from a counter; the rows that no entry names are cleared in the same
// way, when the chunks are given out.  Which warp takes what changes nothing in
// the results.
//
// Bound by memory: every entry's row is read once, with the rows of kAhead
// entries under way, and every row of the result is written once, in whole
// 32-byte sectors, the zeros of the rows form behind its count among them.  393,216 bf16 rows of 256 (201 MB in, 403 MB out): 103 us,
// 5.9 TB/s; 16,384 rows of 5120 into 99,092 (168 MB in, 2.03 GB out): 299 us,
// 7.3 TB/s.  Four blocks an SM, which 64 registers allow; three are slower.
template <class E, int kLanes, bool kAligned>
__global__ void __launch_bounds__(kThreads, 4) seg_sum_kernel(SumArgs<E> a) {
  constexpr int N = kCols<E>, kGroups = 32 / kLanes, kAhead = 8;
  const int wl = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lane = threadIdx.x % kLanes;
  const int64_t tasks = static_cast<int64_t>(a.chunks) * a.tiles;
  __shared__ int32_t before[kMaxSortBlocks + 1];
  wait_prior_grids();  // the sort; after it, the joins may be launched and read what it wrote
  allow_dependent_launch();
  if (!a.dense) {
    sum_heads(a, before);
    __syncthreads();
  }
  while (true) {
    int32_t got = 0;
    if (wl == 0) got = atomicAdd(a.next, 1);
    got = __shfl_sync(0xffffffffu, got, 0);
    const int64_t task = static_cast<int64_t>(got) * kGroups + wl / kLanes;
    if (task - wl / kLanes >= tasks) {
      if (got < kGaveUp) break;
      no_gradient(a);
      return;
    }
    if (task >= tasks) continue;
    const int32_t chunk = static_cast<int32_t>(task / a.tiles);
    const int32_t tile = static_cast<int32_t>(task - static_cast<int64_t>(chunk) * a.tiles);
    const int c0 = tile * kLanes * N;
    const int32_t e0 = chunk * a.chunk, e1 = a.n - e0 < a.chunk ? a.n : e0 + a.chunk;
    uint32_t key = a.list[e0].key;
    if (key == a.none) continue;  // sorted: none of the chunk's entries has a row
    bool from_before = e0 > 0 && a.list[e0 - 1].key == key;
    int32_t seg = a.dense ? 0 : a.base[chunk] + before[chunk / a.chunks_per];
    if (from_before) --seg;
    float acc[N];
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = 0.f;
    for (int32_t e = e0; e < e1; e += kAhead) {
      uint4 x[kAhead];
      uint32_t after[kAhead];  // the next entry's key
      // two entries a load; the list's end is padded to whole 256 bytes
#pragma unroll
      for (int k = 0; k < kAhead; k += 2) {
        const uint4 two = __ldg(reinterpret_cast<const uint4*>(a.list + e + k));
        x[k] = x[k + 1] = make_uint4(0u, 0u, 0u, 0u);
        if (e + k < e1) x[k] = load_cols<E, kAligned>(entry_row(a, static_cast<int32_t>(two.y)), c0, lane, kLanes, a.dim);
        if (e + k + 1 < e1)
          x[k + 1] = load_cols<E, kAligned>(entry_row(a, static_cast<int32_t>(two.w)), c0, lane, kLanes, a.dim);
        if (k > 0) after[k - 1] = e + k < a.n ? two.x : a.none;
        after[k] = e + k + 1 < a.n ? two.z : a.none;
      }
      after[kAhead - 1] = e + kAhead < a.n ? __ldg(&a.list[e + kAhead].key) : a.none;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (e + k >= e1 || key == a.none) break;
        add_cols<E>(x[k], acc);
        const bool ends = after[k] != key, border = e + k + 1 == e1;
        if (ends || border) {
          if (from_before) {
            store_cols<E, kAligned>(a.head + static_cast<int64_t>(chunk) * a.dim, c0, lane, kLanes, a.dim, 1.f, acc);
          } else if (!ends) {
            store_cols<E, kAligned>(a.tail + static_cast<int64_t>(chunk) * a.dim, c0, lane, kLanes, a.dim, 1.f, acc);
            if (!a.dense && tile == 0 && lane == 0) a.rows[seg] = static_cast<int32_t>(key);
          } else {
            store_cols<E, kAligned>(a.grad + (a.dense ? static_cast<int64_t>(key) : seg) * a.dim, c0, lane, kLanes, a.dim,
                                    a.scale, acc);
            if (!a.dense && tile == 0 && lane == 0) a.rows[seg] = static_cast<int32_t>(key);
          }
#pragma unroll
          for (int j = 0; j < N; ++j) acc[j] = 0.f;
          if (ends) ++seg;
          from_before = false;
          key = after[k];
        }
      }
    }
  }

  if (!a.dense) {
    const int32_t segs = before[a.heads_count];
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.count = segs;
    constexpr int kRows = 16;  // a warp's share at a time
    while (true) {
      int32_t got = 0;
      if (wl == 0) got = atomicAdd(a.next + 1, 1);
      const int64_t s0 = segs + static_cast<int64_t>(__shfl_sync(0xffffffffu, got, 0)) * kRows;
      if (s0 >= a.n) break;
      const int64_t s1 = s0 + kRows < a.n ? s0 + kRows : a.n;
      if (s0 + wl < s1) a.rows[s0 + wl] = -1;
      zero_rows(a.grad + s0 * a.dim, (s1 - s0) * a.dim, wl);
    }
    return;
  }
  // ranges of rows: the entries of a range are neighbours in the sorted order,
  // their rows are marked, the others are cleared
  const int kRange = a.range;
  __shared__ uint32_t named[kMaxRange / 32];
  __shared__ int32_t start;
  __shared__ int32_t taken;
  while (true) {
    __syncthreads();
    if (threadIdx.x == 0) taken = atomicAdd(a.next + 1, 1);
    __syncthreads();
    const int64_t r0 = static_cast<int64_t>(taken) * kRange;
    if (r0 >= a.total_rows) break;
    if (threadIdx.x < kMaxRange / 32) named[threadIdx.x] = 0u;
    if (warp == 0) {  // the first entry of row r0 or a later one, 32 probes at a time
      int32_t lo = 0, hi = a.n;
      while (hi > lo) {
        const int32_t step = (hi - lo + 31) / 32, q = lo + step * wl;
        const int k = __popc(__ballot_sync(0xffffffffu, q < hi && q >= lo && a.list[q].key < r0));
        if (k == 0) break;
        hi = step * k < hi - lo ? lo + step * k : hi;
        lo = lo + step * (k - 1) + 1;
      }
      if (wl == 0) start = lo;
    }
    __syncthreads();
    for (int32_t e = start + threadIdx.x;; e += kThreads) {
      const uint32_t key = e < a.n && e >= 0 ? a.list[e].key : a.none;
      const bool in = key < r0 + kRange && key != a.none;
      if (in) atomicOr(&named[(key - r0) >> 5], 1u << ((key - r0) & 31));
      if (!__syncthreads_or(in)) break;
    }
    for (int r = warp; r < kRange && r0 + r < a.total_rows; r += kWarps)
      if (!(named[r >> 5] >> (r & 31) & 1u)) zero_rows(a.grad + (r0 + r) * a.dim, a.dim, wl);
  }
}

// Joins the parts of the segments that cross chunks.  Every warp looks at one
// chunk; where a segment begins in it and goes on, the warp adds the parts, or,
// if there are many, all warps of the block do: warp w the parts w, w + 16, ...
// of the segment, then the warps' sums in order.  Bound by the longest segment's
// chain of loads (12 to 16 us at the sizes above), hence kBatch parts at a time.
constexpr int kOwnParts = 12;  // parts that one warp adds alone (whole calls with 4, 12 and 32: 393,216 rows of 256
                               // 167, 168 and 171 us, 16,384 of 5120 into 99,092 336, 336 and 342)
constexpr int kJoinWarps = 16;  // with 8, 16 and 32: 170, 168 and 170 us, 335, 336 and 344; where every entry has one
                                // id, 393,216 of 256 233, 202 and 198, 5000 of 64 47, 45 and 47

template <class E, bool kAligned>
__global__ void __launch_bounds__(kJoinWarps * 32) seg_join_kernel(SumArgs<E> a) {
  constexpr int N = kCols<E>, kWarps = kJoinWarps;
  __shared__ float sums[kWarps][32 * N];
  __shared__ int32_t parts[kWarps], segment[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t chunk = blockIdx.x * kWarps + warp, e0 = chunk * a.chunk, e1 = e0 + a.chunk;
  // the parts begin + step * i below count of the segment that begins in chunk c,
  // kBatch of them in flight
  constexpr int kBatch = 8;
  auto add = [&](int32_t c, int32_t begin, int32_t step, int32_t count, int c0, float (&acc)[N]) {
    for (int32_t k0 = begin; k0 < count; k0 += kBatch * step) {
      float q[kBatch][N];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int32_t k = k0 + b * step;
        const float* part = (k == 0 ? a.tail : a.head) + static_cast<int64_t>(c + k) * a.dim + c0;
#pragma unroll
        for (int j = 0; j < N; j += kAligned ? 4 : 1) {
          const int col = kAligned ? lane * N + j : j * 32 + lane;
          const bool in = k < count && c0 + col < a.dim;
          if constexpr (kAligned) {
            const float4 v = in ? *reinterpret_cast<const float4*>(part + col) : make_float4(0.f, 0.f, 0.f, 0.f);
            q[b][j] = v.x;
            q[b][j + 1] = v.y;
            q[b][j + 2] = v.z;
            q[b][j + 3] = v.w;
          } else {
            q[b][j] = in ? part[col] : 0.f;
          }
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] += q[b][j];
    }
  };
  __shared__ int32_t before[kMaxSortBlocks + 1];
  const bool no_list = __ldcg(a.next) >= kGaveUp;
  if (!a.dense) {
    sum_heads(a, before);
    __syncthreads();
  }
  int32_t mine = 0, seg = 0;
  if (chunk < a.chunks - 1) {
    const uint32_t key = a.list[e1 - 1].key;
    if (key != a.none && a.list[e1].key == key && (e0 == 0 || a.list[e0 - 1].key != key)) {
      // the segment's end, 32 probes at a time: the entry lo - 1 has the key, the entry hi a larger one
      int32_t lo = e1 + 1, hi = a.n;
      while (hi > lo) {
        const int32_t step = (hi - lo + 31) / 32;
        const int64_t q = static_cast<int64_t>(lo) + static_cast<int64_t>(step) * lane;
        const int k = __popc(__ballot_sync(0xffffffffu, q < hi && a.list[q].key == key));
        if (k == 0) break;
        hi = static_cast<int64_t>(step) * k < hi - lo ? lo + step * k : hi;
        lo = lo + step * (k - 1) + 1;
      }
      mine = (lo - 1) / a.chunk - chunk + 1;
      seg = static_cast<int32_t>(key);
      if (!a.dense) {  // the last segment that begins in this chunk
        int32_t heads = 0;
        for (int k = 0; k < a.chunk; k += 32)
          heads += __popc(__ballot_sync(0xffffffffu, k + lane < a.chunk && is_head(a.list, static_cast<int64_t>(e0) + k + lane,
                                                                                   a.n, a.none)));
        seg = a.base[chunk] + before[chunk / a.chunks_per] + heads - 1;
      }
    }
  }
  if (no_list) mine = 0;  // (no place of the list was followed so far)
  if (lane == 0) {
    parts[warp] = mine;
    segment[warp] = seg;
  }
  wait_prior_grids();  // the parts
  for (int c0 = blockIdx.y * 32 * N; c0 < a.dim; c0 += gridDim.y * 32 * N) {
    if (mine > 0 && mine <= kOwnParts) {
      float acc[N];
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] = 0.f;
      add(chunk, 0, 1, mine, c0, acc);
      store_cols<E, kAligned>(a.grad + static_cast<int64_t>(seg) * a.dim, c0, lane, 32, a.dim, a.scale, acc);
    }
    for (int s = 0; s < kWarps; ++s) {
      __syncthreads();
      if (parts[s] <= kOwnParts) continue;  // the same for all warps
      float acc[N];
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] = 0.f;
      add(blockIdx.x * kWarps + s, warp, kWarps, parts[s], c0, acc);
#pragma unroll
      for (int j = 0; j < N; ++j) sums[warp][kAligned ? lane * N + j : j * 32 + lane] = acc[j];
      __syncthreads();
      float* out = a.grad + static_cast<int64_t>(segment[s]) * a.dim;
      for (int c = threadIdx.x; c < 32 * N; c += kWarps * 32) {
        float total = sums[0][c];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) total += sums[w][c];
        if (c0 + c < a.dim) out[c0 + c] = a.scale * total;
      }
    }
  }
}

// ------------------------------------------------------------------ few entries

// Up to kFew entries need no sort: every block holds all ids and finds by
// comparing them which entry is the first of its row and which others share
// it.  A warp adds up one row's entries, in order, for one tile of columns, a
// whole block those of a row with many; the blocks then clear the other rows in
// shares.  One launch where the sort, the sums and the joins take three.  Bound by
// latency: the comparisons, then the loads of a row's entries, eight at a time.
// Calls with random ids (with one id): 300 entries of 64 bf16 columns 21 (25) against
// 34 (32) us by the sort, of 418 bf16 columns 25 (35) against 37 (36); 512 of 1280
// bf16 columns 42 (43) against 28 (32).
constexpr int kFew = 320;

template <class E, bool kAligned>
__global__ void __launch_bounds__(kThreads) few_kernel(SumArgs<E> a, const int32_t* __restrict__ ids, int32_t* status) {
  constexpr int N = kCols<E>, kBatch = 8, kOwn = 2 * kBatch;  // entries that one warp adds alone
  __shared__ __align__(16) uint32_t key[kFew];
  __shared__ uint32_t heads[kFew / 32];  // a bit per entry that is the first of its row
  __shared__ uint32_t longs[kFew / 32];  // of those, the ones whose rows the whole block adds up
  __shared__ float sums[kWarps][32 * N];
  __shared__ uint32_t named[kMaxRange / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  for (int i = tid; i < kFew; i += kThreads) {
    key[i] = a.none;
    if (i < a.n) {
      const int32_t id = ids[i];
      key[i] = entry_key(id, a.total_rows);
      bad |= id != ENGRAM_DEAD && (id < 0 || id >= a.total_rows);
    }
  }
  if (bad && blockIdx.x == 0 && status != nullptr) atomicOr(status, ENGRAM_ST_BAD_ROW);
  __syncthreads();
  const int words = (a.n + 31) / 32;
  for (int w = warp; w < words; w += kWarps) {  // the lane's entry against all, four a load
    const int i = w * 32 + lane;
    const uint32_t mine = key[i];
    bool first = mine != a.none;
    int count = 0;
    for (int j = 0; j < words * 32; j += 4) {
      const uint4 q = *reinterpret_cast<const uint4*>(key + j);
      const bool e0 = q.x == mine, e1 = q.y == mine, e2 = q.z == mine, e3 = q.w == mine;
      first = first && !((e0 && j < i) || (e1 && j + 1 < i) || (e2 && j + 2 < i) || (e3 && j + 3 < i));
      count += e0 + e1 + e2 + e3;
    }
    const uint32_t bits = __ballot_sync(0xffffffffu, first);
    const uint32_t many = __ballot_sync(0xffffffffu, first && count > kOwn);
    if (lane == 0) longs[w] = many;
    if (lane == 0) heads[w] = bits;
  }
  __syncthreads();

  // the row of the result
  auto row_of = [&](uint32_t mine) {
    if (a.dense) return static_cast<int64_t>(mine);
    int smaller = 0;  // rows with smaller ids
    for (int w = 0; w < words; ++w) smaller += (heads[w] >> lane & 1u) && key[w * 32 + lane] < mine;
    return static_cast<int64_t>(__reduce_add_sync(0xffffffffu, smaller));
  };
  // acc: every shares-th entry of the row from the entry i on, in order
  auto add_row = [&](int i, uint32_t mine, int c0, int share, int shares, float (&acc)[N]) {
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = 0.f;
    int at[kBatch], held = 0, before = 0;  // entries found and not added yet
    auto flush = [&]() {
      uint4 x[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        x[b] = make_uint4(0u, 0u, 0u, 0u);
        if (b < held) x[b] = load_cols<E, kAligned>(entry_row(a, at[b]), c0, lane, 32, a.dim);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (b < held) add_cols<E>(x[b], acc);
      held = 0;
    };
    for (int w = i / 32; w < words; ++w) {
      uint32_t same = __ballot_sync(0xffffffffu, key[w * 32 + lane] == mine);
      if (shares > 1) {
        const int place = before + __popc(same & ((1u << lane) - 1u));
        before += __popc(same);
        same &= __ballot_sync(0xffffffffu, place % shares == share);
      }
      while (same != 0) {
        const int e = w * 32 + __ffs(same) - 1;
        same &= same - 1;
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
          if (b == held) at[b] = e;
        if (++held == kBatch) flush();
      }
    }
    if (held > 0) flush();
  };

  const int64_t tasks = static_cast<int64_t>(a.n) * a.tiles, step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t task = static_cast<int64_t>(blockIdx.x) * kWarps + warp; task < tasks; task += step) {
    const int i = static_cast<int>(task / a.tiles), c0 = static_cast<int>(task - static_cast<int64_t>(i) * a.tiles) * 32 * N;
    if (!((heads[i / 32] & ~longs[i / 32]) >> (i & 31) & 1u)) continue;
    const uint32_t mine = key[i];
    const int64_t row = row_of(mine);
    if (!a.dense && c0 == 0 && lane == 0) a.rows[row] = static_cast<int32_t>(mine);
    float acc[N];
    add_row(i, mine, c0, 0, 1, acc);
    store_cols<E, kAligned>(a.grad + row * a.dim, c0, lane, 32, a.dim, a.scale, acc);
  }

  int turn = 0;  // (row, tile) pairs of the long rows, one block each
  for (int w = 0; w < words; ++w) {
    for (uint32_t left = longs[w]; left != 0; left &= left - 1) {
      const int i = w * 32 + __ffs(left) - 1;
      const uint32_t mine = key[i];
      for (int tile = 0; tile < a.tiles; ++tile, ++turn) {
        if (turn % static_cast<int>(gridDim.x) != static_cast<int>(blockIdx.x)) continue;
        const int c0 = tile * 32 * N;
        float acc[N];
        add_row(i, mine, c0, warp, kWarps, acc);
#pragma unroll
        for (int j = 0; j < N; ++j) sums[warp][kAligned ? lane * N + j : j * 32 + lane] = acc[j];
        const int64_t row = row_of(mine);
        if (!a.dense && tile == 0 && tid == 0) a.rows[row] = static_cast<int32_t>(mine);
        __syncthreads();
        for (int c = tid; c < 32 * N && c0 + c < a.dim; c += kThreads) {
          float total = sums[0][c];
#pragma unroll
          for (int v = 1; v < kWarps; ++v) total += sums[v][c];
          a.grad[row * a.dim + c0 + c] = a.scale * total;
        }
        __syncthreads();
      }
    }
  }

  if (!a.dense) {
    int found = 0;
    for (int w = 0; w < words; ++w) found += __popc(heads[w]);
    if (blockIdx.x == 0 && tid == 0) *a.count = found;
    for (int64_t s = found + static_cast<int64_t>(blockIdx.x) * kWarps + warp; s < a.n; s += step) {
      if (lane == 0) a.rows[s] = -1;
      zero_rows(a.grad + s * a.dim, a.dim, lane);
    }
    return;
  }
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * a.range; r0 < a.total_rows;
       r0 += static_cast<int64_t>(gridDim.x) * a.range) {
    __syncthreads();
    if (tid < kMaxRange / 32) named[tid] = 0u;
    __syncthreads();
    for (int i = tid; i < a.n; i += kThreads) {
      const int64_t r = static_cast<int64_t>(key[i]) - r0;
      if (key[i] != a.none && r >= 0 && r < a.range) atomicOr(&named[r >> 5], 1u << (r & 31));
    }
    __syncthreads();
    for (int r = warp; r < a.range && r0 + r < a.total_rows; r += kWarps)
      if (!(named[r >> 5] >> (r & 31) & 1u)) zero_rows(a.grad + (r0 + r) * a.dim, a.dim, lane);
  }
}

template <class E, bool kAligned>
int launch_few(const SumArgs<E>& a0, const int32_t* ids, int sms, int32_t* status, cudaStream_t st) {
  SumArgs<E> a = a0;
  a.tiles = (a.dim + 32 * kCols<E> - 1) / (32 * kCols<E>);
  const int64_t want = (static_cast<int64_t>(a.n) * a.tiles + kWarps - 1) / kWarps, full = static_cast<int64_t>(sms) * 4;
  const int64_t ranges = a.dense ? (a.total_rows + a.range - 1) / a.range : 0;
  const int64_t blocks = want > ranges ? want : ranges;
  few_kernel<E, kAligned><<<static_cast<int>(blocks < full ? blocks : full), kThreads, 0, st>>>(a, ids, status);
  return check_launch("lookup gradient");
}

int check_lookup(int32_t type, int64_t total_rows, int32_t row_dim, int64_t n_tokens, int32_t n_cols, int64_t stride) {
  if (!train::known_type(type)) return fail(ENGRAM_E_INVALID, "type %d is not ENGRAM_T_BF16 or ENGRAM_T_F32", type);
  if (total_rows < 0 || n_tokens < 0) return fail(ENGRAM_E_INVALID, "negative size");
  if (total_rows >= (int64_t(1) << 31) - 1) return fail(ENGRAM_E_RANGE, "total_rows must be below 2^31 - 1");
  if (row_dim < 1 || row_dim > (1 << 20)) return fail(ENGRAM_E_SHAPE, "row_dim %d not in [1, 2^20]", row_dim);
  if (n_cols < 1 || n_cols > (1 << 20)) return fail(ENGRAM_E_SHAPE, "n_cols %d not in [1, 2^20]", n_cols);
  if (n_tokens > ((int64_t(1) << 31) - 8192) / n_cols)
    return fail(ENGRAM_E_RANGE, "n_tokens * n_cols must be at most 2^31 - 8192");
  if (stride < static_cast<int64_t>(n_cols) * row_dim)
    return fail(ENGRAM_E_SHAPE, "row stride %lld below n_cols * row_dim", static_cast<long long>(stride));
  return ENGRAM_OK;
}

// The parts of the gradient's workspace.
struct GradSpace {
  Entry* list[2];
  int32_t* base;
  int32_t* counts;
  int32_t* barrier;  // two words, the summing kernel's counters, then the group sums
  int32_t* heads;
  float *head, *tail;
  size_t bytes;
};

constexpr int64_t kMeanwhile = 1 << 22;  // elements of a result that more SMs clear during the sort
constexpr int kMaxGroups = (kMaxSortBlocks + kGroup - 1) / kGroup, kMaxPasses = 4;

// Lanes per task: the smallest power of two that covers a narrow row.
int lanes_for(int32_t dim, int cols) {
  int lanes = 32;
  while (lanes > 4 && lanes / 2 * cols >= dim) lanes /= 2;
  return lanes;
}

// Entries per chunk: the fewest of 16, 32, 64 and 128 that give no more tasks
// than five quarters of the lane groups that 152 SMs hold (4 blocks of 8 warps:
// 4864, a number here because the workspace's size, which follows from it, is asked
// for without a device).  Fewer entries shorten a small call, whose tasks all run at once;
// more entries leave fewer parts to join (393,216 entries of 256 columns with 32,
// 64 and 128: 193, 182 and 171 us; 16,384 of 5120: 341, 333 and 333).
int32_t chunk_for(int64_t n, int32_t dim, int cols) {
  const int lanes = lanes_for(dim, cols);
  const int64_t tiles = (dim + lanes * cols - 1) / (lanes * cols), groups = 4864 * (32 / lanes);
  int32_t chunk = 16;
  while (chunk < 128 && (n + chunk - 1) / chunk * tiles > groups * 5 / 4) chunk *= 2;
  return chunk;
}

GradSpace grad_space(void* at, int64_t n, int32_t dim) {
  GradSpace s;
  char* p = static_cast<char*>(at);
  size_t used = 0;
  auto take = [&](size_t bytes) {
    char* q = p + used;
    used += round256(bytes);
    return q;
  };
  const int32_t fewest = std::min(chunk_for(n, dim, kCols<train::Bf16>), chunk_for(n, dim, kCols<train::F32>));
  const size_t chunks = static_cast<size_t>((n + fewest - 1) / fewest);
  s.barrier = reinterpret_cast<int32_t*>(take((4 + static_cast<size_t>(kMaxPasses) * kMaxGroups * kMaxDigits) * 4));
  s.heads = reinterpret_cast<int32_t*>(take(kMaxSortBlocks * 4));
  for (int k = 0; k < 2; ++k) s.list[k] = reinterpret_cast<Entry*>(take(static_cast<size_t>(n) * sizeof(Entry)));
  s.base = reinterpret_cast<int32_t*>(take(chunks * 4));
  s.counts = reinterpret_cast<int32_t*>(take(static_cast<size_t>(kMaxSortBlocks) * kMaxDigits * 4));
  s.head = reinterpret_cast<float*>(take(chunks * dim * 4));
  s.tail = reinterpret_cast<float*>(take(chunks * dim * 4));
  s.bytes = used;
  return s;
}

template <class E, bool kAligned>
int launch_sums(const SumArgs<E>& a0, int sms, cudaStream_t st) {
  SumArgs<E> a = a0;
  const int lanes = lanes_for(a.dim, kCols<E>);
  a.tiles = (a.dim + lanes * kCols<E> - 1) / (lanes * kCols<E>);
  const int64_t groups = kThreads / lanes;
  const int64_t want = (static_cast<int64_t>(a.chunks) * a.tiles + groups - 1) / groups, full = static_cast<int64_t>(sms) * 4;
  // the resident blocks at most; all of them where there may be rows to clear
  const int g = static_cast<int>(a.dense || want > full ? full : want);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(g));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;  // launched while the kernel before it runs
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto kernel = lanes == 32   ? seg_sum_kernel<E, 32, kAligned>
                : lanes == 16 ? seg_sum_kernel<E, 16, kAligned>
                : lanes == 8  ? seg_sum_kernel<E, 8, kAligned>
                              : seg_sum_kernel<E, 4, kAligned>;
  cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, a);
  if (err == cudaSuccess && a.chunks > 1) {
    const int ty = (a.dim + 32 * kCols<E> - 1) / (32 * kCols<E>);
    cfg.gridDim = dim3((a.chunks + kJoinWarps - 1) / kJoinWarps, ty < 65535 ? ty : 65535);
    cfg.blockDim = dim3(kJoinWarps * 32);
    err = cudaLaunchKernelEx(&cfg, seg_join_kernel<E, kAligned>, a);
  }
  if (err != cudaSuccess) return fail(ENGRAM_E_CUDA, "lookup gradient launch: %s", cudaGetErrorString(err));
  return check_launch("lookup gradient");
}

int lookup_grad(const void* dout_d, int32_t type, int64_t dout_stride, const int32_t* ids_d, int64_t n_tokens,
                int32_t n_cols, int32_t row_dim, int64_t total_rows, float scale, bool dense, int32_t* rows_d,
                float* grad_d, int32_t* count_d, void* workspace_d, size_t workspace_bytes, int32_t* status_d,
                void* stream, int32_t absent = 0) {
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
  if (n == 0) {
    if (dense) cudaMemsetAsync(grad_d, 0, static_cast<size_t>(total_rows) * row_dim * 4, st);
    else cudaMemsetAsync(count_d, 0, 4, st);
    return check_launch("lookup gradient");
  }
  const GradSpace w = grad_space(workspace_d, n, row_dim);
  const bool few = n <= kFew;
  const int32_t chunk = chunk_for(n, row_dim, type == ENGRAM_T_BF16 ? kCols<train::Bf16> : kCols<train::F32>);
  const int32_t chunks = static_cast<int32_t>((n64 + chunk - 1) / chunk);
  const uint32_t none = static_cast<uint32_t>(total_rows);
  // 64 KB at least, to hide the search, and no more ranges than needed to spread over the SMs; but kMaxRange rows at
  // most, which are less than 64 KB where a row has fewer than 64 columns
  const int64_t spread = total_rows / (static_cast<int64_t>(sms) * 32), least = std::max((1 << 14) / row_dim, 1);
  const int32_t range = static_cast<int32_t>(std::min<int64_t>(std::max(spread, least), kMaxRange));
  SortArgs sa{};
  int blocks = 1;
  if (!few) {
    int width = 1;  // bits of the keys, total_rows standing for "no row"
    while ((total_rows >> width) != 0) ++width;
    sa.ids = ids_d;
    sa.total_rows = total_rows;
    sa.n = n;
    sa.passes = (width + kDigitBits - 1) / kDigitBits;
    sa.bits = (width + sa.passes - 1) / sa.passes;
    if (sa.bits < 2) sa.bits = 2;  // counts are read four at a time
    for (int k = 0; k < 2; ++k) sa.list[k] = w.list[k];
    sa.counts = w.counts;
    sa.barrier = w.barrier;
    sa.absent = absent;
    sa.groups = w.barrier + 4;
    sa.chunk = chunk;
    sa.chunks = chunks;
    sa.base = dense ? nullptr : w.base;
    sa.heads = w.heads;
    sa.next = w.barrier + 2;
    sa.status = status_d;
    // one block up to a round of entries; more blocks (at least 1024 entries
    // each) shorten the passes but cost two barriers a pass
    if (n > kRound) {
      blocks = sms < kMaxSortBlocks ? sms : kMaxSortBlocks;
      if (n / 1024 < blocks) blocks = n / 1024;
    }
    sa.per = (n + blocks - 1) / blocks;
    sa.chunks_per = (chunks + blocks - 1) / blocks;
    sa.blocks = blocks;
    sa.dim = row_dim;
    sa.range = range;
    sa.grad = grad_d;
    // the other SMs clear rows meanwhile
    int all = blocks;
    if (dense && total_rows <= kMarked && total_rows * row_dim >= kMeanwhile) all = sms;
    if (all > 1) {
      const size_t groups = blocks > 1 ? static_cast<size_t>(sa.passes) * ((blocks + kGroup - 1) / kGroup) * (1 << sa.bits) : 0;
      const size_t zeroed = 4 + groups;
      cudaError_t err = cudaMemsetAsync(w.barrier, 0, zeroed * 4, st);
      if (err != cudaSuccess) return fail(ENGRAM_E_CUDA, "cudaMemsetAsync: %s", cudaGetErrorString(err));
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(all));
    cfg.blockDim = dim3(kSortThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeCooperative;
    attr.val.cooperative = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = blocks > 1 ? 1 : 0;
    cudaError_t err = cudaLaunchKernelEx(&cfg, sort_kernel, sa);
    if (err != cudaSuccess) return fail(ENGRAM_E_CUDA, "sort_kernel launch: %s", cudaGetErrorString(err));
    if ((rc = check_launch("sort_kernel"))) return rc;
  }
  auto go = [&](auto e) {
    using E = decltype(e);
    SumArgs<E> a{};
    a.dout = static_cast<const typename E::T*>(dout_d);
    a.dout_stride = dout_stride;
    a.dim = row_dim;
    a.n_cols = n_cols;
    a.n = n;
    a.chunk = chunk;
    a.chunks = chunks;
    a.scale = scale;
    a.list = w.list[(sa.passes - 1) & 1];
    a.none = none;
    a.dense = dense;
    a.contiguous = dout_stride == static_cast<int64_t>(n_cols) * row_dim;
    a.base = w.base;
    a.heads = w.heads;
    a.heads_count = blocks;
    a.chunks_per = sa.chunks_per;
    a.count = count_d;
    a.total_rows = total_rows;
    a.range = range;
    a.grad = grad_d;
    a.rows = rows_d;
    a.head = w.head;
    a.tail = w.tail;
    a.next = w.barrier + 2;
    const bool vec = row_dim % kCols<E> == 0 && dout_stride % kCols<E> == 0 && aligned(dout_d, 16) &&
                     aligned(grad_d, E::kBytes == 2 ? 32 : 16);
    if (few) return vec ? launch_few<E, true>(a, ids_d, sms, status_d, st) : launch_few<E, false>(a, ids_d, sms, status_d, st);
    return vec ? launch_sums<E, true>(a, sms, st) : launch_sums<E, false>(a, sms, st);
  };
  return type == ENGRAM_T_BF16 ? go(train::Bf16{}) : go(train::F32{});
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
  return type == ENGRAM_T_BF16
             ? lookup_rows<train::Bf16>(table_d, total_rows, row_dim, row_ids_d, n, n_cols, scale, out_d, out_stride, status_d,
                                        sms, as_stream(stream))
             : lookup_rows<train::F32>(table_d, total_rows, row_dim, row_ids_d, n, n_cols, scale, out_d, out_stride, status_d,
                                       sms, as_stream(stream));
}

extern "C" size_t engram_lookup_grad_workspace_bytes(int64_t n_tokens, int32_t n_cols, int32_t row_dim) {
  if (n_tokens < 0 || n_cols < 1 || row_dim < 1) return 0;
  return grad_space(nullptr, n_tokens * n_cols, row_dim).bytes;
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

extern "C" int engram_selftest_grad_wait(const void* dout_d, int32_t type, int64_t dout_stride,
                                         const int32_t* row_ids_d, int64_t n_tokens, int32_t n_cols, int32_t row_dim,
                                         int64_t total_rows, int32_t* rows_d, float* grad_d, int32_t* count_d,
                                         void* workspace_d, size_t workspace_bytes, int32_t* status_d, void* stream) {
  if (n_tokens < 0 || n_cols < 1 || n_tokens > 0x7fffffff / n_cols || n_tokens * n_cols <= kRound)
    return fail(ENGRAM_E_RANGE, "only the sort of more than %d entries waits", kRound);
  return lookup_grad(dout_d, type, dout_stride, row_ids_d, n_tokens, n_cols, row_dim, total_rows, 1.f, rows_d == nullptr,
                     rows_d, grad_d, count_d, workspace_d, workspace_bytes, status_d, stream, 1);
}
