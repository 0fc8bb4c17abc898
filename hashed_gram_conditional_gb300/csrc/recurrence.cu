// Gated linear recurrence over packed sequences, its backward pass and its
// one-position step.
//
// Per channel, with f_t = sigmoid(g_t):
//   s_t = f_t s_{t-1} + (1 - f_t) x_t,   y_t = s_t
// A masked position holds the state, gives y = 0 and takes no gradient.
// Backward, with l the gradient of the state:
//   l_t = dy_t + f_{t+1} l_{t+1},  dx_t = l_t (1 - f_t),
//   dg_t = l_t (s_{t-1} - x_t) f_t (1 - f_t)
// 1 - f_t is computed as sigmoid(-g_t), which keeps its relative precision
// where f_t rounds to one.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "engram_internal.h"
#include "train_device.cuh"

namespace engram {
namespace {

using train::round256;

constexpr uint32_t kFull = 0xffffffffu;

// Every lane handles 8 bytes of a row: four bf16 channels or two fp32 ones; a
// warp reads 256 bytes of a row.
template <class E>
constexpr int kLaneCh = 8 / E::kBytes;
template <class E>
constexpr int kGroup = 32 * kLaneCh<E>;  // channels of a block
constexpr int kRowBytes = 256;

// f = sigmoid(g) and u = sigmoid(-g) of two channels.
//
// bf16 data: with e = exp(-g), f = 1 / (1 + e) and u = e / (1 + e), neither of
// which cancels.  g is taken as at least -40 (gate_row), so that e stays finite:
// f is 4e-18 where it would be smaller.  The hardware's base-2 exponential and
// reciprocal (2^-22 and 2^-23 relative, plus |g| 2^-24 from rounding the
// exponent) are far below the data's own rounding.  Every channel has its own
// reciprocal, so that a NaN stays in it: one of (1 + e0)(1 + e1) for both would
// carry it over, and is no faster (16,384 x 5120, a scan 113 us either way, with
// its backward pass 311 against 309).
// fp32 data: expf and the rounded reciprocal, on exp(-|g|).
template <class E>
__device__ __forceinline__ void gates2(float g0, float g1, float (&f)[2], float (&u)[2]) {
  if constexpr (E::kBytes == 2) {
    float t0, t1, e0, e1, d0, d1;
    f2_split(f2_mul(f2(g0, g1), f2(-1.4426950408889634f, -1.4426950408889634f)), t0, t1);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(t0));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(t1));
    f2_split(f2_add(f2(e0, e1), f2(1.f, 1.f)), d0, d1);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(f[0]) : "f"(d0));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(f[1]) : "f"(d1));
    f2_split(f2_mul(f2(f[0], f[1]), f2(e0, e1)), u[0], u[1]);
  } else {
    const float g[2] = {g0, g1};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float e = expf(-fabsf(g[j])), big = __frcp_rn(1.f + e), small = e * big;
      f[j] = g[j] >= 0.f ? big : small;
      u[j] = g[j] >= 0.f ? small : big;
    }
  }
}

template <class E>
__device__ __forceinline__ void gates(const float (&g)[kLaneCh<E>], float (&f)[kLaneCh<E>], float (&u)[kLaneCh<E>]) {
#pragma unroll
  for (int j = 0; j < kLaneCh<E>; j += 2) {
    float f2v[2], u2v[2];
    gates2<E>(g[j], g[j + 1], f2v, u2v);
    f[j] = f2v[0];
    f[j + 1] = f2v[1];
    u[j] = u2v[0];
    u[j + 1] = u2v[1];
  }
}

// a b + c and a b of a lane's channels, two at a time.
template <int V>
__device__ __forceinline__ void fma_v(const float (&a)[V], const float (&b)[V], const float (&c)[V], float (&r)[V]) {
#pragma unroll
  for (int j = 0; j < V; j += 2)
    f2_split(f2_fma(f2(a[j], a[j + 1]), f2(b[j], b[j + 1]), f2(c[j], c[j + 1])), r[j], r[j + 1]);
}
template <int V>
__device__ __forceinline__ void mul_v(const float (&a)[V], const float (&b)[V], float (&r)[V]) {
#pragma unroll
  for (int j = 0; j < V; j += 2)
    f2_split(f2_mul(f2(a[j], a[j + 1]), f2(b[j], b[j + 1])), r[j], r[j + 1]);
}

template <class E>
struct Args {
  const typename E::T *x, *g, *dy;
  typename E::T *y, *dx, *dg;
  int64_t x_stride, g_stride, dy_stride, y_stride, dx_stride, dg_stride;
  const int64_t* cu;
  int64_t n_seqs;
  const int32_t* slots;
  const uint8_t* mask;
  const float* state;
  float* state_out;
  float* dstate;
  int64_t n_slots;
  float* carry;
  int32_t n_tokens, dim, n_tiles, n_groups;
  bool move_empty;  // the states of empty sequences go from state to state_out
  uint8_t* flags;   // [n_tokens], see mark_kernel
  int32_t* slot;    // [n_tokens]: the state slot of a first or last position
  int32_t* ticket;  // [0] next block number, [1] a wait ran out
  int32_t n_runs;
  float2* map;      // [group][place][kGroup]: a tile as v -> A v + B
  float2* run_map;  // [group][run][kGroup]: kRun tiles as one map
  float* run_value; // [group][run][kGroup]: the value behind a run
  int32_t* status;
};

// The state slot of sequence q, or -1 for a padding sequence.
template <class E>
__device__ __forceinline__ int32_t slot_of(const Args<E>& a, int64_t q) {
  const int32_t s = a.slots != nullptr ? a.slots[q] : static_cast<int32_t>(q);
  if (s < 0) return -1;
  if (a.n_slots > 0 && s >= a.n_slots) {
    if (a.status != nullptr) atomicOr(a.status, ENGRAM_ST_BAD_SLOT);
    return -1;
  }
  return s;
}

// ------------------------------------------------ 8 bytes of a row per lane

// A warp's kSteps rows of 256 bytes into shared memory, without waiting.
// Channels past the width and rows past the end read as zeros.
template <class E, bool kVec, int kSteps>
__device__ __forceinline__ void fetch_rows(unsigned char* dst, const typename E::T* src, int64_t stride, int t, int n_tokens,
                                           int c0, int dim, int lane) {
  if constexpr (kVec) {
    constexpr int N = 16 / E::kBytes;
    const int c = c0 + (lane & 15) * N, r0 = lane >> 4;
    const typename E::T* p = src + (t + r0) * stride + c;
    const uint32_t d = smem_u32(dst + r0 * kRowBytes + (lane & 15) * 16);
    if (t + kSteps <= n_tokens) {
      const int bytes = c < dim ? 16 : 0;
      if (c >= dim) p = src;
      const int64_t two = c < dim ? 2 * stride : 0;
#pragma unroll
      for (int k = 0; k < kSteps; k += 2) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d + k * kRowBytes), "l"(p), "r"(bytes) : "memory");
        p += two;
      }
    } else {
#pragma unroll 1
      for (int k = 0; k < kSteps; k += 2) {
        const bool ok = t + r0 + k < n_tokens && c < dim;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d + k * kRowBytes),
                     "l"(ok ? p + k * stride : src), "r"(ok ? 16 : 0)
                     : "memory");
      }
    }
  } else {
    typename E::T* d = reinterpret_cast<typename E::T*>(dst);
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
      for (int j = 0; j < kLaneCh<E>; ++j) {
        const int c = j * 32 + lane;
        const bool ok = t + k < n_tokens && c0 + c < dim;
        d[k * kGroup<E> + c] = ok ? src[(t + k) * stride + c0 + c] : typename E::T(0);
      }
  }
}

__device__ __forceinline__ void wait_rows() {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
}

template <class E>
__device__ __forceinline__ void spread(const uint2& w, float (&v)[kLaneCh<E>]) {
  if constexpr (E::kBytes == 2) {
    v[0] = __uint_as_float(w.x << 16);
    v[1] = __uint_as_float(w.x & 0xffff0000u);
    v[2] = __uint_as_float(w.y << 16);
    v[3] = __uint_as_float(w.y & 0xffff0000u);
  } else {
    v[0] = __uint_as_float(w.x);
    v[1] = __uint_as_float(w.y);
  }
}

template <class E>
__device__ __forceinline__ void lane_row(const unsigned char* row, int lane, float (&v)[kLaneCh<E>]) {
  spread<E>(*reinterpret_cast<const uint2*>(row + lane * 8), v);
}
// A row of g, with gates2's lower bound for bf16.
template <class E>
__device__ __forceinline__ uint2 bounded(uint2 w) {
  if constexpr (E::kBytes == 2) {
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w.x) : "r"(0xc220c220u));  // -40
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w.y) : "r"(0xc220c220u));
  }
  return w;
}
template <class E>
__device__ __forceinline__ void gate_row(const unsigned char* row, int lane, float (&v)[kLaneCh<E>]) {
  spread<E>(bounded<E>(*reinterpret_cast<const uint2*>(row + lane * 8)), v);
}

template <class E, bool kVec>
__device__ __forceinline__ void store_row(typename E::T* row, int c, int dim, const float (&v)[kLaneCh<E>]) {
  if constexpr (kVec) {
    if (c >= dim) return;
    if constexpr (E::kBytes == 2) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
      *reinterpret_cast<uint2*>(row + c) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    } else {
      *reinterpret_cast<float2*>(row + c) = make_float2(v[0], v[1]);
    }
  } else {
    // (whole words where they can be: 4096 x 4902 49 us forward, 57 without)
    if constexpr (E::kBytes == 2) {
      if (c + 3 < dim && (reinterpret_cast<uintptr_t>(row) & 3) == 0) {
        *reinterpret_cast<__nv_bfloat162*>(row + c) = __floats2bfloat162_rn(v[0], v[1]);
        *reinterpret_cast<__nv_bfloat162*>(row + c + 2) = __floats2bfloat162_rn(v[2], v[3]);
        return;
      }
    }
#pragma unroll
    for (int j = 0; j < kLaneCh<E>; ++j)
      if (c + j < dim) E::store(row + c + j, v[j]);
  }
}

// fp32 [.][dim] rows of the states and saved states.
template <class E>
__device__ __forceinline__ void load_state(const float* row, int c, int dim, float (&v)[kLaneCh<E>]) {
#pragma unroll
  for (int j = 0; j < kLaneCh<E>; ++j) v[j] = c + j < dim ? row[c + j] : 0.f;
}
template <class E>
__device__ __forceinline__ void store_state(float* row, int c, int dim, const float (&v)[kLaneCh<E>]) {
#pragma unroll
  for (int j = 0; j < kLaneCh<E>; ++j)
    if (c + j < dim) row[c + j] = v[j];
}
// a lane's channels of an fp32 row in shared memory
template <class E>
__device__ __forceinline__ void get_lane(const float* row, int lane, float (&v)[kLaneCh<E>]) {
  if constexpr (kLaneCh<E> == 4) {
    const float4 q = *reinterpret_cast<const float4*>(row + 4 * lane);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  } else {
    const float2 q = *reinterpret_cast<const float2*>(row + 2 * lane);
    v[0] = q.x; v[1] = q.y;
  }
}
template <class E>
__device__ __forceinline__ void put_lane(float* row, int lane, const float (&v)[kLaneCh<E>]) {
  if constexpr (kLaneCh<E> == 4) *reinterpret_cast<float4*>(row + 4 * lane) = make_float4(v[0], v[1], v[2], v[3]);
  else *reinterpret_cast<float2*>(row + 2 * lane) = make_float2(v[0], v[1]);
}

// What a tile publishes needs no flag and no fence: the words are kNotYet until
// they are written (a NaN that no result is: those are stored as the plain
// NaN), each is valid by itself, and a reader polls the words it needs.
constexpr uint32_t kNotYet = 0xffffffffu;

// ------------------------------------------------------ what the positions are

constexpr int kLive = 1, kFirst = 2, kLast = 4;

// kLive where position t counts (not masked, not in a padding sequence), kFirst /
// kLast where a sequence begins / ends; `slot`: the sequence's (-1: padding).
template <class E>
__device__ __forceinline__ int mark_position(const Args<E>& a, int64_t t, int32_t& slot) {
  int64_t lo = 0, hi = a.n_seqs;  // the last sequence with cu <= t
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (a.cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  slot = slot_of(a, lo);
  const bool live = slot >= 0 && (a.mask == nullptr || a.mask[t] == 0);
  return (live ? kLive : 0) | (a.cu[lo] == t ? kFirst : 0) | (a.cu[lo + 1] == t + 1 ? kLast : 0);
}

// The states of empty sequences move on unchanged: channels d0, d0 + 256, ...
// below d1, sequences q0, q0 + step, ...
template <class E>
__device__ __forceinline__ void move_states(const Args<E>& a, int64_t q0, int64_t step, int d0, int d1, int threads) {
  for (int64_t q = q0; q < a.n_seqs; q += step) {
    if (a.cu[q] != a.cu[q + 1]) continue;
    const int32_t slot = slot_of(a, q);
    for (int d = d0 + threadIdx.x; slot >= 0 && d < d1; d += threads)
      a.state_out[static_cast<int64_t>(slot) * a.dim + d] =
          a.state != nullptr ? a.state[static_cast<int64_t>(slot) * a.dim + d] : 0.f;
  }
}

// Marks every position for the scan (flags[t], and slot[t] where a sequence
// begins or ends), readies the counters and the tiles' words (`cleared` 16-byte
// vectors) and moves the states of empty sequences.  A scan of one tile does
// without it: its blocks mark the positions themselves.
template <class E>
__global__ void __launch_bounds__(256) mark_kernel(Args<E> a, uint4* words, int64_t cleared) {
  allow_dependent_launch();
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, step = static_cast<int64_t>(gridDim.x) * 256;
  if (i0 < 2 && cleared > 0) a.ticket[i0] = 0;
#pragma unroll 4
  for (int64_t i = i0; i < cleared; i += step) words[i] = make_uint4(kNotYet, kNotYet, kNotYet, kNotYet);
  for (int64_t t = i0; t < a.n_tokens; t += step) {
    int32_t slot;
    const int f = mark_position(a, t, slot);
    a.flags[t] = static_cast<uint8_t>(f);
    if (f & (kFirst | kLast)) a.slot[t] = slot;
  }
  if (a.move_empty) move_states(a, blockIdx.x, gridDim.x, 0, a.dim, 256);
}

// What a block needs before its tile: its number in walking order, and the
// positions' marks, from memory or, where the scan is one tile (kAlone), made
// here.
template <int kLen>
struct Start {
  uint32_t cuts;  // a bit per warp in which a sequence begins
  int32_t number;
  uint8_t flags[kLen > 0 ? kLen : 1];
  int32_t slot[kLen > 0 ? kLen : 1];
};
template <bool kAlone, class E, int kLen>
__device__ __forceinline__ int begin_tile(const Args<E>& a, Start<kLen>& s, int threads) {
  if (threadIdx.x == 0) s.cuts = 0u;
  if constexpr (!kAlone) {
    wait_prior_grids();
    if (threadIdx.x == 0) s.number = atomicAdd(a.ticket, 1);
    __syncthreads();
    return s.number;
  } else {
    for (int t = threadIdx.x; t < a.n_tokens; t += threads) {
      int32_t slot;
      s.flags[t] = static_cast<uint8_t>(mark_position(a, t, slot));
      s.slot[t] = slot;
    }
    const int d0 = static_cast<int>(blockIdx.x) * kGroup<E>;
    if (a.move_empty) move_states(a, 0, 1, d0, d0 + kGroup<E> < a.dim ? d0 + kGroup<E> : a.dim, threads);
    __syncthreads();
    return static_cast<int>(blockIdx.x);
  }
}

// A position that does not count is given g = +inf, x = 0 (and dy = 0) in shared
// memory: f = 1 and u x = 0 hold the state, whatever the row holds.
template <class E>
__device__ __forceinline__ void put_neutral(unsigned char* g, unsigned char* x, int lane) {
  const uint32_t inf = E::kBytes == 2 ? 0x7f807f80u : 0x7f800000u;
  *reinterpret_cast<uint2*>(g + lane * 8) = make_uint2(inf, inf);
  *reinterpret_cast<uint2*>(x + lane * 8) = make_uint2(0u, 0u);
}

// The flags of a warp's positions as one bit per position.
struct Marks {
  uint32_t live, first, last;
};
template <int kSteps>
__device__ __forceinline__ Marks marks_of(const uint8_t* flags, int n_tokens, int t, int lane) {
  const int f = lane < kSteps && t + lane < n_tokens ? flags[t + lane] : 0;
  Marks m;
  m.live = __ballot_sync(kFull, f & kLive);
  m.first = __ballot_sync(kFull, f & kFirst);
  m.last = __ballot_sync(kFull, f & kLast);
  return m;
}

// ------------------------------------------------------------ across the tiles

__device__ __forceinline__ uint32_t load_word(const void* p) {
  uint32_t v;
  asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint2 load_pair(const void* p) {
  uint2 v;
  asm volatile("ld.relaxed.gpu.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t plain(float v) {
  const uint32_t w = __float_as_uint(v);
  return w == kNotYet ? 0x7fffffffu : w;
}
__device__ __forceinline__ void store_word(void* p, float v) {
  asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(plain(v)) : "memory");
}
__device__ __forceinline__ void store_pair(void* p, float x, float y) {
  asm volatile("st.relaxed.gpu.global.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(plain(x)), "r"(plain(y)) : "memory");
}

// Maps v -> A v + B with A >= 0.  Where a sequence begins nothing before it
// counts, which A = -0 stands for, so that a product of gates that underflows
// to +0 still carries a NaN on, as the recurrence itself does.
constexpr float kCut = -0.f;

__device__ __forceinline__ float apply_map(float A, float B, float v) { return fmaf(A, signbit(A) ? 0.f : v, B); }
__device__ __forceinline__ float apply_map(const uint2& m, float v) {
  return apply_map(__uint_as_float(m.x), __uint_as_float(m.y), v);
}
__device__ __forceinline__ float join_factor(float p, float A) { return signbit(p) || signbit(A) ? kCut : p * A; }

// What comes into the tile at place `pos` of the walk, for one channel: the
// tiles' maps applied one by one to the value in front of them.  Runs of kRun
// tiles are joined to one map by their last tile, so that a look back passes
// over at most kRun - 1 tiles of its own run and then over whole runs (a scan in
// one pass by looking back: Merrill and Garland 2016).  Every value is built by
// the same steps in the same order whatever has been published when, so results
// do not change from run to run.
//
// Tiles take their numbers from a counter in walking order, so every tile that
// is waited for is already running.  (A, B) is the tile's own map; a warp's
// lanes are neighbouring channels.  `meanwhile` runs between the publishing of
// the map and the first look at the others.  A look costs about 1000 cycles
// whatever it finds, so the maps of the tile's own run and what is usually
// there of the two runs before it are read together.
constexpr int kRun = 8;

template <class E, class F>
__device__ __forceinline__ float come_in(const Args<E>& a, int group, int pos, int ch, float A, float B, F meanwhile) {
  constexpr int G = kGroup<E>;
  const int lane = threadIdx.x & 31;
  const long long begun = clock64();
  auto give_up = [&]() {
    const bool out = clock64() - begun > kWaitBudgetCycles || load_word(a.ticket + 1) != 0;
    if (!__any_sync(kFull, out)) return false;
    if (lane == 0) {
      atomicExch(a.ticket + 1, 1);
      if (a.status != nullptr) atomicOr(a.status, ENGRAM_ST_TIMEOUT);
    }
    return true;
  };
  const int run = pos / kRun, behind = pos % kRun;  // tiles of this run before this one
  const int64_t base = static_cast<int64_t>(group) * a.n_tiles;
  const float2* maps = a.map + (base + pos) * G + ch;
  const bool last_of_all = pos + 1 == a.n_tiles;
  if (!last_of_all) store_pair(a.map + (base + pos) * G + ch, A, B);
  meanwhile();

  const int64_t rbase = static_cast<int64_t>(group) * a.n_runs;
  uint32_t near = 0u, far = 0u;  // the values behind the last run and the one before it
  uint2 step = make_uint2(0u, 0u);  // the last run's map
  if (run > 0) near = load_word(a.run_value + (rbase + run - 1) * G + ch);
  if (run > 1) {
    far = load_word(a.run_value + (rbase + run - 2) * G + ch);
    step = load_pair(a.run_map + (rbase + run - 1) * G + ch);
  }
  uint2 m[kRun - 1];  // m[i]: the map of the tile i + 1 places before
#pragma unroll
  for (int i = 0; i < kRun - 1; ++i) m[i] = i < behind ? load_pair(maps - (i + 1) * G) : make_uint2(0u, 0u);
  while (true) {
    bool all = true;
#pragma unroll
    for (int i = 0; i < kRun - 1; ++i) all = all && m[i].x != kNotYet && m[i].y != kNotYet;
    if (__all_sync(kFull, all)) break;
    if (give_up()) return 0.f;
#pragma unroll
    for (int i = 0; i < kRun - 1; ++i)
      if (m[i].x == kNotYet || m[i].y == kNotYet) m[i] = load_pair(maps - (i + 1) * G);
  }

  float RA = A, RB = B;  // the run's map, where this tile ends it
  const bool ends_run = behind == kRun - 1 && !last_of_all;
  if (ends_run) {
    RA = 1.f;
    RB = 0.f;
#pragma unroll
    for (int i = kRun - 2; i >= 0; --i) {
      const float p = __uint_as_float(m[i].x);
      RB = i == kRun - 2 ? __uint_as_float(m[i].y) : apply_map(m[i], RB);
      RA = i == kRun - 2 ? p : join_factor(p, RA);
    }
    RB = apply_map(A, B, RB);
    RA = join_factor(A, RA);
    store_pair(a.run_map + (rbase + run) * G + ch, RA, RB);
  }

  // the value in front of the run
  float v = 0.f;
  if (run == 0) {
    // nothing is in front of it
  } else if (__all_sync(kFull, near != kNotYet)) {
    v = __uint_as_float(near);
  } else if (run > 1 && __all_sync(kFull, far != kNotYet && step.x != kNotYet && step.y != kNotYet)) {
    v = apply_map(step, __uint_as_float(far));
  } else {
    int depth = 0;  // run maps to apply
    const int ch0 = ch - lane;
    while (true) {
      const int mine = run - 1 - depth - lane;
      const bool has_value = mine < 0 || load_word(a.run_value + (rbase + mine) * G + ch0) != kNotYet;
      const bool has_map = mine < 0 || load_word(a.run_map + (rbase + mine) * G + ch0) != kNotYet;
      const uint32_t done = __ballot_sync(kFull, has_value), some = __ballot_sync(kFull, has_value || has_map);
      const uint32_t before = done != 0 ? (done & -done) - 1u : kFull;  // the lanes nearer than the first value
      if ((some & before) == before) {
        if (done != 0) {
          depth += __ffs(done) - 1;
          break;
        }
        depth += 32;
        continue;
      }
      depth = 0;
      if (give_up()) return 0.f;
    }
    const int from = run - 1 - depth;
    if (from >= 0) {
      const float* p = a.run_value + (rbase + from) * G + ch;
      uint32_t w = load_word(p);
      while (!__all_sync(kFull, w != kNotYet)) {
        if (give_up()) return 0.f;
        w = load_word(p);
      }
      v = __uint_as_float(w);
    }
    constexpr int kBatch = 8;
    for (int r0 = from + 1; r0 < run; r0 += kBatch) {
      uint2 w[kBatch];
      const float2* p = a.run_map + (rbase + r0) * G + ch;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) w[b] = r0 + b < run ? load_pair(p + b * G) : make_uint2(0u, 0u);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (r0 + b >= run) break;
        while (!__all_sync(kFull, w[b].x != kNotYet && w[b].y != kNotYet)) {
          if (give_up()) return 0.f;
          w[b] = load_pair(p + b * G);
        }
        v = apply_map(w[b], v);
      }
    }
  }
  if (ends_run) store_word(a.run_value + (rbase + run) * G + ch, apply_map(RA, RB, v));
#pragma unroll
  for (int i = kRun - 2; i >= 0; --i)
    if (i < behind) v = apply_map(m[i], v);
  return v;
}

// --------------------------------------------------------------------- forward

// A block handles kFwdTile positions of one group of channels, in one
// pass over memory: every warp fetches its rows into shared memory and reduces
// them to a map s -> A s + B per channel; one warp joins the maps, publishes
// the block's, and looks back over the blocks before it for the state that
// comes in; then the warps walk their positions again, from shared memory, and
// write y.  The gates are computed twice rather than kept: that frees the
// registers, so that three blocks fit an SM and their loads cover one another's
// waits.
//
// 16,384 x 5120 bf16 (503 MB): 107 us, 4.7 TB/s, 69 % of a copy's rate.  Neither
// memory nor issue is full (46 % of DRAM, 0.48 instructions a cycle and scheduler
// at half the length); what is left are waits, for the copies and for the tiles
// before: a block has no loads under way while it looks back and writes.  Tiles of 64 positions, blocks of 4 warps and runs of 4, 12 or 16
// tiles are slower.
constexpr int kFwdTile = 128, kBwdTile = ENGRAM_RECURRENCE_TILE;  // a state is saved in front of every backward tile
static_assert(kFwdTile % kBwdTile == 0, "saved states fall between a forward tile's warps");

constexpr int kFwdWarps = 8;

template <class E, bool kVec, bool kAlone>
__global__ void __launch_bounds__(kFwdWarps * 32, 3) forward_kernel(const Args<E> a) {
  constexpr int kWarps = kFwdWarps, kTile = kFwdTile, kSteps = kTile / kWarps;
  constexpr int V = kLaneCh<E>, G = kGroup<E>;
  extern __shared__ __align__(16) unsigned char smem[];
  unsigned char* xs = smem;
  unsigned char* gs = xs + kTile * kRowBytes;
  float(*mapA)[G] = reinterpret_cast<float(*)[G]>(gs + kTile * kRowBytes);
  float(*mapB)[G] = mapA + kWarps;
  __shared__ Start<kAlone ? kTile : 0> start;
  uint32_t& cuts = start.cuts;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = begin_tile<kAlone>(a, start, kWarps * 32);
  const uint8_t* flags = kAlone ? start.flags : a.flags;
  const int32_t* slots = kAlone ? start.slot : a.slot;
  const int tile = n / a.n_groups, group = n - tile * a.n_groups;
  const int c0 = group * G, c = c0 + lane * V;
  const int t0 = tile * kTile, tw = t0 + warp * kSteps;
  unsigned char* xw = xs + warp * kSteps * kRowBytes;
  unsigned char* gw = gs + warp * kSteps * kRowBytes;
  fetch_rows<E, kVec, kSteps>(gw, a.g, a.g_stride, tw, a.n_tokens, c0, a.dim, lane);
  fetch_rows<E, kVec, kSteps>(xw, a.x, a.x_stride, tw, a.n_tokens, c0, a.dim, lane);
  const Marks mk = marks_of<kSteps>(flags, a.n_tokens, tw, lane);
  wait_rows();

  constexpr uint32_t kAll = (1u << kSteps) - 1u;
  for (uint32_t dead = ~mk.live & kAll; dead != 0; dead &= dead - 1u) {
    const int k = __ffs(dead) - 1;
    put_neutral<E>(gw + k * kRowBytes, xw + k * kRowBytes, lane);
  }

  // s <- f s + u x; a sequence's first position starts from its own state
  float s[V], A[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    A[j] = 1.f;
    s[j] = 0.f;
  }
  auto begin = [&](int k) {
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = 0.f;
    const int32_t slot = slots[tw + k];
    if (slot >= 0 && a.state != nullptr) load_state<E>(a.state + static_cast<int64_t>(slot) * a.dim, c, a.dim, s);
  };
  // Where the states are updated in place, the warp that holds a sequence's
  // end may overwrite the first state before this warp's second walk: the state
  // of the one sequence that begins here and ends behind this warp is kept, in
  // the place of the warp's A (which nothing uses where a sequence begins).
  auto goes_on = [&](int k) { return (mk.last >> k) == 0u; };
  auto advance = [&](int k, float (&f)[V]) {
    float gv[V], xv[V], u[V];
    gate_row<E>(gw + k * kRowBytes, lane, gv);
    lane_row<E>(xw + k * kRowBytes, lane, xv);
    gates<E>(gv, f, u);
    mul_v<V>(u, xv, xv);
    fma_v<V>(f, s, xv, s);
  };
  if (mk.first == 0) {  // the usual case, without branches
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      float f[V];
      advance(k, f);
      mul_v<V>(A, f, A);
    }
  } else {
#pragma unroll 1
    for (int k = 0; k < kSteps; ++k) {
      if (mk.first >> k & 1u) {
        begin(k);
        if (goes_on(k)) put_lane<E>(mapA[warp], lane, s);
      }
      float f[V];
      advance(k, f);
    }
  }
  if (mk.first == 0) put_lane<E>(mapA[warp], lane, A);
  put_lane<E>(mapB[warp], lane, s);
  if (lane == 0 && mk.first != 0) atomicOr(&cuts, 1u << warp);
  __syncthreads();

  if (warp * 32 < G) {  // a lane per channel: the tile's map, and what comes into it and into every warp
    const int ch = warp * 32 + lane;
    const uint32_t cut = cuts;
    float TA = 1.f, TB = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float p = cut >> w & 1u ? kCut : mapA[w][ch];
      TB = apply_map(p, mapB[w][ch], TB);
      TA = join_factor(p, TA);
    }
    float v = come_in<E>(a, group, tile, ch, TA, TB, [] {});
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w * kSteps % kBwdTile == 0 && a.carry != nullptr && c0 + ch < a.dim && t0 + w * kSteps < a.n_tokens)
        a.carry[static_cast<int64_t>((t0 + w * kSteps) / kBwdTile) * a.dim + c0 + ch] = v;
      const float q = mapB[w][ch];
      mapB[w][ch] = v;
      v = apply_map(cut >> w & 1u ? kCut : mapA[w][ch], q, v);
    }
  }
  __syncthreads();

  get_lane<E>(mapB[warp], lane, s);
  typename E::T* y = a.y + tw * a.y_stride;
  const bool plain = (mk.first | mk.last) == 0 && tw + kSteps <= a.n_tokens;
  if (plain) {
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      float f[V];
      advance(k, f);
      store_row<E, kVec>(y, c, a.dim, s);
      y += a.y_stride;
    }
    const float zeros[V] = {};
    for (uint32_t dead = ~mk.live & kAll; dead != 0; dead &= dead - 1u)  // over what was just written
      store_row<E, kVec>(a.y + (tw + __ffs(dead) - 1) * a.y_stride, c, a.dim, zeros);
  } else {
#pragma unroll 1
    for (int k = 0; k < kSteps && tw + k < a.n_tokens; ++k) {
      if (mk.first >> k & 1u) {
        if (goes_on(k)) get_lane<E>(mapA[warp], lane, s);
        else begin(k);
      }
      float f[V], out[V];
      advance(k, f);
#pragma unroll
      for (int j = 0; j < V; ++j) out[j] = mk.live >> k & 1u ? s[j] : 0.f;
      store_row<E, kVec>(y + k * a.y_stride, c, a.dim, out);
      if (mk.last >> k & 1u) {
        const int32_t slot = slots[tw + k];
        if (slot >= 0 && a.state_out != nullptr)
          store_state<E>(a.state_out + static_cast<int64_t>(slot) * a.dim, c, a.dim, s);
      }
    }
  }
}

template <class E>
constexpr int kFwdSmem = 2 * kFwdTile * kRowBytes + 2 * kFwdWarps * kGroup<E> * 4;

// -------------------------------------------------------------------- backward

// The same scheme walked from the last tile to the first.  With m_t = f_t l_t,
// what position t passes back, m_t = f_t (dy_t + m_{t+1}): a tile maps the m
// that comes in to A m + C, A being the product of its gates.  The states
// before its positions come from the state saved in front of the tile.
//
// A position's gradients need its state, known in ascending order, and l,
// known in descending order: the ascending walk leaves s_{t-1} - x in registers.
// The gates are computed in each of the three walks: their smaller one would
// have to stand for both where one is kept, and telling them apart costs more
// instructions than a pair's two exponentials and two reciprocals.
//
// 16,384 x 5120 bf16 (844 MB with the saved states): 191 us, 4.4 TB/s, 65 % of a
// copy's rate, at 0.55 instructions a cycle and scheduler and half of DRAM's
// cycles.  Tiles of 128 positions (one block less an SM) and blocks of 4 warps
// gain nothing.
constexpr int kBwdWarps = 8;

template <class E, bool kVec, bool kAlone>
__global__ void __launch_bounds__(kBwdWarps * 32, 3) backward_kernel(const Args<E> a) {
  constexpr int kWarps = kBwdWarps, kTile = kBwdTile, kSteps = kTile / kWarps;
  constexpr int V = kLaneCh<E>, G = kGroup<E>;
  extern __shared__ __align__(16) unsigned char smem[];
  unsigned char* xs = smem;
  unsigned char* gs = xs + kTile * kRowBytes;
  unsigned char* ds = gs + kTile * kRowBytes;
  float(*mapA)[G] = reinterpret_cast<float(*)[G]>(ds + kTile * kRowBytes);
  float(*mapB)[G] = mapA + kWarps;
  float(*mapC)[G] = mapB + kWarps;
  // the gradient of the last state of the sequence that ends here and began
  // before this warp, whose first state's gradient may be written in its place
  float(*held)[G] = mapC + kWarps;
  __shared__ Start<kAlone ? kTile : 0> start;
  uint32_t& cuts = start.cuts;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = begin_tile<kAlone>(a, start, kWarps * 32);
  const uint8_t* flags = kAlone ? start.flags : a.flags;
  const int32_t* slots = kAlone ? start.slot : a.slot;
  const int back = n / a.n_groups, group = n - back * a.n_groups;
  const int tile = a.n_tiles - 1 - back;
  const int c0 = group * G, c = c0 + lane * V;
  const int t0 = tile * kTile, tw = t0 + warp * kSteps;
  unsigned char* xw = xs + warp * kSteps * kRowBytes;
  unsigned char* gw = gs + warp * kSteps * kRowBytes;
  unsigned char* dw = ds + warp * kSteps * kRowBytes;
  fetch_rows<E, kVec, kSteps>(gw, a.g, a.g_stride, tw, a.n_tokens, c0, a.dim, lane);
  fetch_rows<E, kVec, kSteps>(xw, a.x, a.x_stride, tw, a.n_tokens, c0, a.dim, lane);
  fetch_rows<E, kVec, kSteps>(dw, a.dy, a.dy_stride, tw, a.n_tokens, c0, a.dim, lane);
  const Marks mk = marks_of<kSteps>(flags, a.n_tokens, tw, lane);
  float carry[V];
  load_state<E>(a.carry + static_cast<int64_t>(tile) * a.dim, c, a.dim, carry);
  wait_rows();

  for (uint32_t dead = ~mk.live & ((1u << kSteps) - 1u); dead != 0; dead &= dead - 1u) {
    const int k = __ffs(dead) - 1;
    put_neutral<E>(gw + k * kRowBytes, xw + k * kRowBytes, lane);
    *reinterpret_cast<uint2*>(dw + k * kRowBytes + lane * 8) = make_uint2(0u, 0u);
  }

  float s[V], A[V], C[V];
  auto begin = [&](int k) {
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = 0.f;
    const int32_t slot = slots[tw + k];
    if (slot >= 0 && a.state != nullptr) load_state<E>(a.state + static_cast<int64_t>(slot) * a.dim, c, a.dim, s);
  };
  auto advance = [&](int k, float (&xv)[V], float (&f)[V], float (&u)[V]) {
    float gv[V], b[V];
    gate_row<E>(gw + k * kRowBytes, lane, gv);
    lane_row<E>(xw + k * kRowBytes, lane, xv);
    gates<E>(gv, f, u);
    mul_v<V>(u, xv, b);
    fma_v<V>(f, s, b, s);
  };
  auto pass_back = [&](int k, const float (&f)[V]) {
    float dv[V];
    lane_row<E>(dw + k * kRowBytes, lane, dv);
    mul_v<V>(A, f, A);
    fma_v<V>(A, dv, C, C);
  };
  auto from_before = [&](int k) { return (mk.first & ((2u << k) - 1u)) == 0u; };
#pragma unroll
  for (int j = 0; j < V; ++j) {
    A[j] = 1.f;
    s[j] = C[j] = 0.f;
  }
  const bool straight = (mk.first | mk.last) == 0 && tw + kSteps <= a.n_tokens;  // the usual case, without branches
  if (straight) {
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      float xv[V], f[V], u[V];
      advance(k, xv, f, u);
      pass_back(k, f);
    }
  } else {
#pragma unroll 1
    for (int k = 0; k < kSteps; ++k) {
      if (mk.first >> k & 1u) begin(k);
      float xv[V], f[V], u[V];
      advance(k, xv, f, u);
      if (from_before(k)) pass_back(k, f);  // nothing is passed back over a sequence's beginning
      if ((mk.last >> k & 1u) && from_before(k)) {
        float l[V] = {};
        const int32_t slot = slots[tw + k];
        if (slot >= 0 && a.dstate != nullptr) load_state<E>(a.dstate + static_cast<int64_t>(slot) * a.dim, c, a.dim, l);
        put_lane<E>(held[warp], lane, l);
        fma_v<V>(A, l, C, C);
      }
    }
  }
  put_lane<E>(mapA[warp], lane, A);
  put_lane<E>(mapB[warp], lane, s);
  put_lane<E>(mapC[warp], lane, C);
  if (lane == 0 && mk.first != 0) atomicOr(&cuts, 1u << warp);
  __syncthreads();

  // the walk in ascending order, from the state in front of the tile
  float gap[kSteps][V];
  auto ascend = [&]() {
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = carry[j];
    const uint32_t cut = cuts;
    for (int p = 0; p < warp; ++p) {
      float f[V], q[V];
      get_lane<E>(mapA[p], lane, f);
      get_lane<E>(mapB[p], lane, q);
      if (cut >> p & 1u) {
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = q[j];
      } else {
        fma_v<V>(f, s, q, s);
      }
    }
    auto walk = [&](int k) {
      float xv[V], f[V], u[V], before[V];
#pragma unroll
      for (int j = 0; j < V; ++j) before[j] = s[j];
      advance(k, xv, f, u);
#pragma unroll
      for (int j = 0; j < V; ++j) gap[k][j] = before[j] - xv[j];
    };
    if (straight) {
#pragma unroll
      for (int k = 0; k < kSteps; ++k) walk(k);
    } else {
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        if (mk.first >> k & 1u) begin(k);
        walk(k);
      }
    }
  };
  if (warp * 32 < G) {  // a lane per channel, from behind: the tile's map, and what comes into it and into every warp
    const int ch = warp * 32 + lane;
    const uint32_t cut = cuts;
    float TA = 1.f, TC = 0.f;
#pragma unroll
    for (int w = kWarps - 1; w >= 0; --w) {
      const float p = cut >> w & 1u ? kCut : mapA[w][ch];
      TC = apply_map(p, mapC[w][ch], TC);
      TA = join_factor(p, TA);
    }
    float v = come_in<E>(a, group, back, ch, TA, TC, ascend);
#pragma unroll
    for (int w = kWarps - 1; w >= 0; --w) {
      const float q = mapC[w][ch];
      mapC[w][ch] = v;
      v = apply_map(cut >> w & 1u ? kCut : mapA[w][ch], q, v);
    }
  } else {
    ascend();
  }
  __syncthreads();

  float m[V];
  get_lane<E>(mapC[warp], lane, m);
  typename E::T* dx = a.dx + tw * a.dx_stride;
  typename E::T* dg = a.dg + tw * a.dg_stride;
  auto descend = [&](int k) {
    float gv[V], dv[V], f[V], u[V], ox[V], og[V];
    lane_row<E>(dw + k * kRowBytes, lane, dv);
    gate_row<E>(gw + k * kRowBytes, lane, gv);
    gates<E>(gv, f, u);
#pragma unroll
    for (int j = 0; j < V; ++j) dv[j] += m[j];
    mul_v<V>(dv, f, m);
    mul_v<V>(dv, u, ox);
    mul_v<V>(m, u, og);
    mul_v<V>(og, gap[k], og);
    store_row<E, kVec>(dx + k * a.dx_stride, c, a.dim, ox);
    store_row<E, kVec>(dg + k * a.dg_stride, c, a.dim, og);
  };
  if (straight) {
#pragma unroll
    for (int k = kSteps - 1; k >= 0; --k) descend(k);
  } else {
#pragma unroll
    for (int k = kSteps - 1; k >= 0; --k) {
      if (tw + k >= a.n_tokens) continue;
      if (mk.last >> k & 1u) {
        if (from_before(k)) {
          get_lane<E>(held[warp], lane, m);
        } else {
          const int32_t slot = slots[tw + k];
#pragma unroll
          for (int j = 0; j < V; ++j) m[j] = 0.f;
          if (slot >= 0 && a.dstate != nullptr) load_state<E>(a.dstate + static_cast<int64_t>(slot) * a.dim, c, a.dim, m);
        }
      }
      descend(k);
      if (mk.first >> k & 1u) {
        const int32_t slot = slots[tw + k];
        if (slot >= 0 && a.dstate != nullptr) store_state<E>(a.dstate + static_cast<int64_t>(slot) * a.dim, c, a.dim, m);
#pragma unroll
        for (int j = 0; j < V; ++j) m[j] = 0.f;
      }
    }
  }
  // positions that do not count, over what was just written
  const float zeros[V] = {};
  for (uint32_t dead = ~mk.live & ((1u << kSteps) - 1u); dead != 0; dead &= dead - 1u) {
    const int64_t t = tw + __ffs(dead) - 1;
    if (t >= a.n_tokens) break;
    store_row<E, kVec>(a.dx + t * a.dx_stride, c, a.dim, zeros);
    store_row<E, kVec>(a.dg + t * a.dg_stride, c, a.dim, zeros);
  }
}

template <class E>
constexpr int kBwdSmem = 3 * kBwdTile * kRowBytes + 4 * kBwdWarps * kGroup<E> * 4;

// ------------------------------------------------------------------ other parts

constexpr int kThreads = 128;

// One position: a read of x, g and the state, one multiply-add, a write of y and
// the state.  A block takes a row's stretch of channels, so that a few sequences
// are as fast as the launch; 256 x 5120 bf16 (18 MB): 6.5 us, 4 x 1280: 3.8 us.
template <class E, bool kVec>
__global__ void __launch_bounds__(kThreads) step_kernel(Args<E> a) {
  constexpr int V = kLaneCh<E>;
  const int64_t b = blockIdx.x;
  const int c = (blockIdx.y * kThreads + threadIdx.x) * V;
  if (c >= a.dim) return;
  float xv[V], gv[V], s[V] = {};
  const typename E::T* xr = a.x + b * a.x_stride;
  const typename E::T* gr = a.g + b * a.g_stride;
  if constexpr (kVec) {
    lane_row<E>(reinterpret_cast<const unsigned char*>(xr + c), 0, xv);
    gate_row<E>(reinterpret_cast<const unsigned char*>(gr + c), 0, gv);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      xv[j] = c + j < a.dim ? E::load(xr + c + j) : 0.f;
      gv[j] = c + j < a.dim ? E::load(gr + c + j) : 0.f;
      if (E::kBytes == 2 && gv[j] < -40.f) gv[j] = -40.f;  // as in gate_row
    }
  }
  const int32_t slot = slot_of(a, b);
  if (slot >= 0) {
    float f[V], u[V];
    load_state<E>(a.state + static_cast<int64_t>(slot) * a.dim, c, a.dim, s);
    gates<E>(gv, f, u);
    mul_v<V>(u, xv, xv);
    fma_v<V>(f, s, xv, s);
    store_state<E>(a.state_out + static_cast<int64_t>(slot) * a.dim, c, a.dim, s);
  }
  store_row<E, kVec>(a.y + b * a.y_stride, c, a.dim, s);
}

// The parts of the scans' workspace: the counters, the positions' marks, then
// the tiles' maps and values.
struct ScanSpace {
  int32_t* ticket;
  uint8_t* flags;
  int32_t* slot;
  float* words;
  size_t bytes;
};

// Sized for the narrower group, which serves both types.
ScanSpace scan_space(void* base, int64_t n_tokens, int32_t dim) {
  constexpr int kNarrow = kGroup<train::F32>;
  const size_t tiles = static_cast<size_t>((n_tokens + kBwdTile - 1) / kBwdTile);  // the smaller of the two
  const size_t groups = static_cast<size_t>((dim + kNarrow - 1) / kNarrow) + 1;  // + 1: a bf16 group may be half empty
  ScanSpace s;
  char* p = static_cast<char*>(base);
  s.ticket = reinterpret_cast<int32_t*>(p);
  size_t at = 256;
  s.flags = reinterpret_cast<uint8_t*>(p + at);
  at += round256(static_cast<size_t>(n_tokens));
  s.slot = reinterpret_cast<int32_t*>(p + at);
  at += round256(static_cast<size_t>(n_tokens) * 4);
  s.words = reinterpret_cast<float*>(p + at);
  const size_t runs = (tiles + kRun - 1) / kRun;
  s.bytes = at + round256((tiles * 8 + runs * 12) * groups * kNarrow);
  return s;
}

int check_common(int32_t type, int64_t n_tokens, int32_t dim, int64_t n_seqs, int64_t n_slots, bool has_state) {
  if (!train::known_type(type)) return fail(ENGRAM_E_INVALID, "type %d is not ENGRAM_T_BF16 or ENGRAM_T_F32", type);
  if (n_tokens < 0 || n_seqs < 0 || n_slots < 0) return fail(ENGRAM_E_INVALID, "negative size");
  if (dim < 1 || dim > (1 << 20)) return fail(ENGRAM_E_SHAPE, "dim %d not in [1, 2^20]", dim);
  if (n_tokens > 0x7fffff00 || n_seqs > 0x7fffff00) return fail(ENGRAM_E_RANGE, "too many positions or sequences");
  if (has_state && n_slots < 1) return fail(ENGRAM_E_INVALID, "a state needs n_slots >= 1");
  return ENGRAM_OK;
}

int check_rows(const void* p, int32_t type, int64_t stride, int32_t dim, const char* name) {
  if (p == nullptr) return fail(ENGRAM_E_INVALID, "null device pointer: %s", name);
  if (stride < dim) return fail(ENGRAM_E_SHAPE, "row stride of %s below dim", name);
  if (!aligned(p, train::type_bytes(type))) return fail(ENGRAM_E_ALIGN, "%s must be aligned to its elements", name);
  return ENGRAM_OK;
}

// Whether rows of `stride` elements from p lie on 16-byte boundaries.
template <class E>
bool rows16(const void* p, int64_t stride) {
  return aligned(p, 16) && stride * E::kBytes % 16 == 0;
}

template <class E, bool kVec, bool kAlone>
int launch_pass(const Args<E>& a, bool backward, int grid, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3((backward ? kBwdWarps : kFwdWarps) * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;  // launched while the marks are made
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = kAlone ? 0 : 1;
  const int smem = backward ? kBwdSmem<E> : kFwdSmem<E>;
  static std::atomic<uint64_t> attr_set[2] = {{0}, {0}};  // one bit per device: the shared-memory opt-in was made
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
  cudaError_t e;
  if (bit == 0 || !(attr_set[backward].load(std::memory_order_relaxed) & bit)) {
    e = backward ? cudaFuncSetAttribute(backward_kernel<E, kVec, kAlone>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)
                 : cudaFuncSetAttribute(forward_kernel<E, kVec, kAlone>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return fail(ENGRAM_E_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    attr_set[backward].fetch_or(bit, std::memory_order_relaxed);
  }
  cfg.dynamicSmemBytes = smem;
  e = backward ? cudaLaunchKernelEx(&cfg, backward_kernel<E, kVec, kAlone>, a) : cudaLaunchKernelEx(&cfg, forward_kernel<E, kVec, kAlone>, a);
  if (e != cudaSuccess) return fail(ENGRAM_E_CUDA, "recurrence launch: %s", cudaGetErrorString(e));
  return check_launch("recurrence");
}

template <class E>
int launch_scan(Args<E>& a, bool backward, void* workspace, int sms, cudaStream_t st) {
  const ScanSpace w = scan_space(workspace, a.n_tokens, a.dim);
  const int tile = backward ? kBwdTile : kFwdTile;
  a.n_tiles = (a.n_tokens + tile - 1) / tile;
  a.n_groups = (a.dim + kGroup<E> - 1) / kGroup<E>;
  a.ticket = w.ticket;
  a.flags = w.flags;
  a.slot = w.slot;
  const int64_t blocks = static_cast<int64_t>(a.n_tiles) * a.n_groups;
  if (blocks > 0x7fffff00) return fail(ENGRAM_E_RANGE, "too many positions times channels");
  a.move_empty = !backward && a.state_out != nullptr && a.state_out != a.state;
  a.n_runs = (a.n_tiles + kRun - 1) / kRun;
  const int64_t tile_words = blocks * kGroup<E>, run_words = static_cast<int64_t>(a.n_runs) * a.n_groups * kGroup<E>;
  a.map = reinterpret_cast<float2*>(w.words);
  a.run_map = a.map + tile_words;
  a.run_value = reinterpret_cast<float*>(a.run_map + run_words);
  const int64_t cleared = (2 * tile_words + 3 * run_words) / 4;  // kGroup is a multiple of 4
  if (a.n_tiles > 1) {
    const int64_t want = ((a.n_tokens > cleared ? a.n_tokens : cleared) + 255) / 256, cap = static_cast<int64_t>(sms) * 8;
    mark_kernel<E><<<static_cast<int>(want < cap ? want : cap), 256, 0, st>>>(a, reinterpret_cast<uint4*>(w.words), cleared);
    int rc = check_launch("mark_kernel");
    if (rc) return rc;
  }
  bool vec = a.dim * E::kBytes % 16 == 0 && rows16<E>(a.x, a.x_stride) && rows16<E>(a.g, a.g_stride);
  if (!backward) vec = vec && rows16<E>(a.y, a.y_stride);
  else vec = vec && rows16<E>(a.dy, a.dy_stride) && rows16<E>(a.dx, a.dx_stride) && rows16<E>(a.dg, a.dg_stride);
  const int grid = static_cast<int>(blocks);
  if (a.n_tiles == 1)
    return vec ? launch_pass<E, true, true>(a, backward, grid, st) : launch_pass<E, false, true>(a, backward, grid, st);
  return vec ? launch_pass<E, true, false>(a, backward, grid, st) : launch_pass<E, false, false>(a, backward, grid, st);
}

template <class E>
int launch_step(const Args<E>& a, int64_t batch, cudaStream_t st) {
  const int per = kThreads * kLaneCh<E>;
  const dim3 grid(static_cast<unsigned>(batch), (a.dim + per - 1) / per);
  const bool vec = a.dim % kLaneCh<E> == 0 && rows16<E>(a.x, a.x_stride) && rows16<E>(a.g, a.g_stride) &&
                   rows16<E>(a.y, a.y_stride);
  if (vec) step_kernel<E, true><<<grid, kThreads, 0, st>>>(a);
  else step_kernel<E, false><<<grid, kThreads, 0, st>>>(a);
  return check_launch("step_kernel");
}

}  // namespace
}  // namespace engram

using namespace engram;

extern "C" size_t engram_recurrence_carry_bytes(int64_t n_tokens, int32_t dim) {
  if (n_tokens < 0 || dim < 1) return 0;
  return static_cast<size_t>((n_tokens + ENGRAM_RECURRENCE_TILE - 1) / ENGRAM_RECURRENCE_TILE) * dim * sizeof(float);
}

extern "C" size_t engram_recurrence_workspace_bytes(int64_t n_tokens, int32_t dim) {
  if (n_tokens < 0 || dim < 1) return 0;
  return scan_space(nullptr, n_tokens, dim).bytes;
}

extern "C" int engram_recurrence(const void* x_d, int64_t x_stride, const void* g_d, int64_t g_stride, int32_t type,
                                 int64_t n_tokens, int32_t dim, const int64_t* cu_seqlens_d, int64_t n_seqs,
                                 const int32_t* slots_d, const uint8_t* mask_d, const float* state_d,
                                 float* state_out_d, int64_t n_slots, void* y_d, int64_t y_stride, float* carry_d,
                                 void* workspace_d, size_t workspace_bytes, int32_t* status_d, void* stream) {
  const bool has_state = state_d != nullptr || state_out_d != nullptr;
  int rc = check_common(type, n_tokens, dim, n_seqs, n_slots, has_state);
  if (rc) return rc;
  if (n_seqs == 0) return n_tokens == 0 ? ENGRAM_OK : fail(ENGRAM_E_SHAPE, "positions without a sequence");
  if (!cu_seqlens_d) return fail(ENGRAM_E_INVALID, "null device pointer: cu_seqlens");
  if (n_tokens > 0) {
    if ((rc = check_rows(x_d, type, x_stride, dim, "x"))) return rc;
    if ((rc = check_rows(g_d, type, g_stride, dim, "g"))) return rc;
    if ((rc = check_rows(y_d, type, y_stride, dim, "y"))) return rc;
    if (!workspace_d) return fail(ENGRAM_E_INVALID, "null device pointer: workspace");
    if (!aligned(workspace_d, 256)) return fail(ENGRAM_E_ALIGN, "workspace must be 256-byte aligned");
    if (workspace_bytes < engram_recurrence_workspace_bytes(n_tokens, dim))
      return fail(ENGRAM_E_RANGE, "workspace too small");
  }
  int sms = 0;
  if ((rc = check_device(&sms))) return rc;
  auto go = [&](auto e) {
    using E = decltype(e);
    Args<E> a{};
    a.x = static_cast<const typename E::T*>(x_d);
    a.g = static_cast<const typename E::T*>(g_d);
    a.y = static_cast<typename E::T*>(y_d);
    a.x_stride = x_stride;
    a.g_stride = g_stride;
    a.y_stride = y_stride;
    a.cu = cu_seqlens_d;
    a.n_seqs = n_seqs;
    a.slots = slots_d;
    a.mask = mask_d;
    a.state = state_d;
    a.state_out = state_out_d;
    a.n_slots = has_state ? n_slots : 0;
    a.carry = carry_d;
    a.n_tokens = static_cast<int32_t>(n_tokens);
    a.dim = dim;
    a.status = status_d;
    if (n_tokens > 0) return launch_scan<E>(a, false, workspace_d, sms, as_stream(stream));
    if (state_out_d == nullptr || state_out_d == state_d) return static_cast<int>(ENGRAM_OK);
    const int64_t cap = static_cast<int64_t>(sms) * 4;
    a.move_empty = true;
    mark_kernel<E><<<static_cast<int>(n_seqs < cap ? n_seqs : cap), 256, 0, as_stream(stream)>>>(a, nullptr, 0);
    return check_launch("mark_kernel");
  };
  return type == ENGRAM_T_BF16 ? go(train::Bf16{}) : go(train::F32{});
}

extern "C" int engram_recurrence_grad(const void* dy_d, int64_t dy_stride, const void* x_d, int64_t x_stride,
                                      const void* g_d, int64_t g_stride, int32_t type, int64_t n_tokens, int32_t dim,
                                      const int64_t* cu_seqlens_d, int64_t n_seqs, const int32_t* slots_d,
                                      const uint8_t* mask_d, const float* state_d, const float* carry_d,
                                      float* dstate_d, int64_t n_slots, void* dx_d, int64_t dx_stride, void* dg_d,
                                      int64_t dg_stride, void* workspace_d, size_t workspace_bytes,
                                      int32_t* status_d, void* stream) {
  const bool has_state = state_d != nullptr || dstate_d != nullptr;
  int rc = check_common(type, n_tokens, dim, n_seqs, n_slots, has_state);
  if (rc) return rc;
  if (n_seqs == 0) return n_tokens == 0 ? ENGRAM_OK : fail(ENGRAM_E_SHAPE, "positions without a sequence");
  if (n_tokens == 0) return ENGRAM_OK;  // the state's gradient passes through empty sequences
  if (!cu_seqlens_d || !carry_d) return fail(ENGRAM_E_INVALID, "null device pointer: cu_seqlens or carry");
  if ((rc = check_rows(dy_d, type, dy_stride, dim, "dy"))) return rc;
  if ((rc = check_rows(x_d, type, x_stride, dim, "x"))) return rc;
  if ((rc = check_rows(g_d, type, g_stride, dim, "g"))) return rc;
  if ((rc = check_rows(dx_d, type, dx_stride, dim, "dx"))) return rc;
  if ((rc = check_rows(dg_d, type, dg_stride, dim, "dg"))) return rc;
  if (!workspace_d) return fail(ENGRAM_E_INVALID, "null device pointer: workspace");
  if (!aligned(workspace_d, 256)) return fail(ENGRAM_E_ALIGN, "workspace must be 256-byte aligned");
  if (workspace_bytes < engram_recurrence_workspace_bytes(n_tokens, dim))
    return fail(ENGRAM_E_RANGE, "workspace too small");
  int sms = 0;
  if ((rc = check_device(&sms))) return rc;
  auto go = [&](auto e) {
    using E = decltype(e);
    Args<E> a{};
    a.dy = static_cast<const typename E::T*>(dy_d);
    a.x = static_cast<const typename E::T*>(x_d);
    a.g = static_cast<const typename E::T*>(g_d);
    a.dx = static_cast<typename E::T*>(dx_d);
    a.dg = static_cast<typename E::T*>(dg_d);
    a.dy_stride = dy_stride;
    a.x_stride = x_stride;
    a.g_stride = g_stride;
    a.dx_stride = dx_stride;
    a.dg_stride = dg_stride;
    a.cu = cu_seqlens_d;
    a.n_seqs = n_seqs;
    a.slots = slots_d;
    a.mask = mask_d;
    a.state = state_d;
    a.dstate = dstate_d;
    a.n_slots = has_state ? n_slots : 0;
    a.carry = const_cast<float*>(carry_d);
    a.n_tokens = static_cast<int32_t>(n_tokens);
    a.dim = dim;
    a.status = status_d;
    return launch_scan<E>(a, true, workspace_d, sms, as_stream(stream));
  };
  return type == ENGRAM_T_BF16 ? go(train::Bf16{}) : go(train::F32{});
}

extern "C" int engram_recurrence_step(const void* x_d, int64_t x_stride, const void* g_d, int64_t g_stride,
                                      int32_t type, int64_t batch, int32_t dim, const int32_t* slots_d,
                                      const float* state_d, float* state_out_d, int64_t n_slots, void* y_d,
                                      int64_t y_stride, int32_t* status_d, void* stream) {
  int rc = check_common(type, batch, dim, batch, n_slots, true);
  if (rc) return rc;
  if (batch == 0) return ENGRAM_OK;
  if (!slots_d || !state_d || !state_out_d) return fail(ENGRAM_E_INVALID, "null device pointer: slots or state");
  if ((rc = check_rows(x_d, type, x_stride, dim, "x"))) return rc;
  if ((rc = check_rows(g_d, type, g_stride, dim, "g"))) return rc;
  if ((rc = check_rows(y_d, type, y_stride, dim, "y"))) return rc;
  if ((rc = check_device(nullptr))) return rc;
  auto go = [&](auto e) {
    using E = decltype(e);
    Args<E> a{};
    a.x = static_cast<const typename E::T*>(x_d);
    a.g = static_cast<const typename E::T*>(g_d);
    a.y = static_cast<typename E::T*>(y_d);
    a.x_stride = x_stride;
    a.g_stride = g_stride;
    a.y_stride = y_stride;
    a.slots = slots_d;
    a.state = state_d;
    a.state_out = state_out_d;
    a.n_slots = n_slots;
    a.dim = dim;
    a.status = status_d;
    return launch_step<E>(a, batch, as_stream(stream));
  };
  return type == ENGRAM_T_BF16 ? go(train::Bf16{}) : go(train::F32{});
}
