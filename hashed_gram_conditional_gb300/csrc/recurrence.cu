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

#include "engram_internal.h"
#include "train_device.cuh"

namespace engram {
namespace {

using train::round256;

constexpr int kTile = ENGRAM_RECURRENCE_TILE;  // positions between saved states; the tile of the backward pass
constexpr int kSteps = 8;                      // positions per warp
constexpr uint32_t kFull = 0xffffffffu;

// Every lane handles 4 bytes of a row: two bf16 channels or one fp32 channel,
// so a warp reads a row in one 128-byte request.
template <class E>
constexpr int kLaneCh = 4 / E::kBytes;
template <class E>
constexpr int kGroup = 32 * kLaneCh<E>;  // channels of a block

struct Gate {
  float f, u;  // sigmoid(g), sigmoid(-g)
};

// With e = exp(-|g|) the larger of the two is 1 / (1 + e) and the smaller
// e / (1 + e): neither cancels nor overflows, and the smaller one with the
// sign of g (gate_code) stands for both.  bf16 data takes the hardware's
// base-2 exponential and reciprocal (2^-22 and 2^-23 relative, plus |g| 2^-24
// from rounding the exponent), far below its own rounding; fp32 data takes
// expf and the rounded reciprocal.
template <class E>
__device__ __forceinline__ float gate_code(float g) {
  float small;
  if (E::kBytes == 2) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * fabsf(g)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    small = e * r;
  } else {
    const float e = expf(-fabsf(g));
    small = e * __frcp_rn(1.f + e);
  }
  return copysignf(small, g);  // +: sigmoid(-g), -: sigmoid(g)
}

__device__ __forceinline__ Gate gate_of(float code) {
  const float small = fabsf(code), big = 1.f - small;
  const bool neg = signbit(code);
  return Gate{neg ? small : big, neg ? big : small};
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
  int32_t* ticket;  // [0] next block number, [1] a wait ran out
  int32_t* flag;    // [group][tile]: 0 nothing, 1 the tile's map, 2 the value after it
  float2* map;      // [group][tile][kGroup]: the tile as v -> A v + B
  float* value;     // [group][tile][kGroup]
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

// ------------------------------------------------ 4 bytes of a row per lane

template <class E, bool kVec>
__device__ __forceinline__ uint32_t load4(const typename E::T* row, int c, int dim) {
  if constexpr (E::kBytes == 4) return c < dim ? __float_as_uint(__ldg(row + c)) : 0u;
  else if constexpr (kVec) return c < dim ? __ldg(reinterpret_cast<const uint32_t*>(row + c)) : 0u;
  else {
    const uint32_t lo = c < dim ? row[c] : 0u, hi = c + 1 < dim ? row[c + 1] : 0u;
    return lo | hi << 16;
  }
}

template <class E, bool kVec>
__device__ __forceinline__ void store4(typename E::T* row, int c, int dim, const float (&v)[kLaneCh<E>]) {
  if constexpr (E::kBytes == 4) {
    if (c < dim) row[c] = v[0];
  } else if constexpr (kVec) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[0], v[1]);
    if (c < dim) *reinterpret_cast<__nv_bfloat162*>(row + c) = b;
  } else {
    if (c < dim) E::store(row + c, v[0]);
    if (c + 1 < dim) E::store(row + c + 1, v[1]);
  }
}

template <class E>
__device__ __forceinline__ void widen(uint32_t raw, float (&v)[kLaneCh<E>]) {
  if constexpr (E::kBytes == 4) v[0] = __uint_as_float(raw);
  else {
    v[0] = __uint_as_float(raw << 16);
    v[1] = __uint_as_float(raw & 0xffff0000u);
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

// ------------------------------------------------- what a tile's positions are

// Position p of the tile: first[p] / last[p] = the slot (or -1: without a
// state) of the sequence that begins / ends there, kNone where none does;
// dead[p] = masked, in a padding sequence, or past the end.
constexpr int32_t kNone = -2;
template <int kLen>
struct Marks {
  int32_t first[kLen], last[kLen];
  uint8_t dead[kLen];
  bool any_first;
};

// Filled by one warp.  Empty sequences have no positions; `copy_empty` moves
// their states for the channels of this block.
template <class E, int kLen>
__device__ __forceinline__ void mark_tile(const Args<E>& a, int t0, Marks<kLen>& m, int lane, int c, bool copy_empty,
                                          bool has_state) {
  for (int p = lane; p < kLen; p += 32) {
    m.first[p] = m.last[p] = kNone;
    const int t = t0 + p;
    m.dead[p] = t >= a.n_tokens || (a.mask != nullptr && a.mask[t] != 0);
  }
  if (lane == 0) m.any_first = false;
  __syncwarp();
  // the first sequence that begins at t0 or later: the lanes probe 32 equal
  // parts of the range at a time
  int64_t lo = 0, hi = a.n_seqs;  // cu[q] < t0 below lo, >= t0 from hi on
  while (hi > lo) {
    const int64_t step = (hi - lo + 31) / 32;
    const int64_t q = lo + step * lane;
    const uint32_t below = __ballot_sync(kFull, q < hi && a.cu[q] < t0);
    const int n = __popc(below);  // the probes below t0 are a prefix
    if (n == 0) break;
    const int64_t l2 = lo + step * (n - 1) + 1, h2 = lo + step * n;
    lo = l2;
    hi = h2 < hi ? h2 : hi;
  }
  const bool ends = t0 + kLen >= a.n_tokens;  // empty sequences after the last position belong to the last tile
  const int t1 = ends ? a.n_tokens : t0 + kLen;
  for (int64_t q0 = lo > 0 ? lo - 1 : 0;; q0 += 32) {
    const int64_t q = q0 + lane;
    int64_t b = INT64_MAX, e = INT64_MAX;
    if (q < a.n_seqs) {
      b = a.cu[q];
      e = a.cu[q + 1];
    }
    const bool some = e > b && q < a.n_seqs;
    const bool here = b < t1 || (ends && b == t1);
    if (some && here) {
      const int32_t slot = slot_of(a, q);
      const int32_t mark = has_state ? slot : -1;
      if (b >= t0) {
        m.first[b - t0] = mark;
        m.any_first = true;
      }
      if (e > t0 && e <= t1) m.last[e - 1 - t0] = mark;
      if (slot < 0) {
        const int64_t from = b > t0 ? b - t0 : 0, to = (e < t1 ? e : t1) - t0;
        for (int64_t p = from; p < to; ++p) m.dead[p] = 1;
      }
    }
    uint32_t empty = __ballot_sync(kFull, copy_empty && q < a.n_seqs && e == b && b >= t0 && here);
    while (empty != 0) {  // rare: every lane copies its channels
      const int src = __ffs(empty) - 1;
      empty &= empty - 1;
      const int32_t slot = slot_of(a, q0 + src);
      if (slot >= 0) {
        float v[kLaneCh<E>] = {};
        if (a.state != nullptr) load_state<E>(a.state + static_cast<int64_t>(slot) * a.dim, c, a.dim, v);
        store_state<E>(a.state_out + static_cast<int64_t>(slot) * a.dim, c, a.dim, v);
      }
    }
    if (!__any_sync(kFull, q < a.n_seqs && lane == 31 && here)) break;
  }
  __syncwarp();
}

// ------------------------------------------------------------ across the tiles

__device__ __forceinline__ int32_t load_flag(const int32_t* p) {
  int32_t v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void store_flag(int32_t* p, int32_t v) {
  asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Maps v -> A v + B with A >= 0.  A sequence's first position cuts: nothing
// before it counts, which A = -0 stands for, so that a product of gates that
// underflows to +0 still carries a NaN on as the recurrence itself does.
constexpr float kCut = -0.f;

__device__ __forceinline__ float apply_map(float A, float B, float v) {
  return signbit(A) ? B : fmaf(A, v, B);
}
// The factor of the map p after the map A.
__device__ __forceinline__ float join_factor(float p, float A) {
  return signbit(p) || signbit(A) ? kCut : p * A;
}

// The value that comes into a tile: from the nearest tile behind it (in
// walking order) that has published its value, through the maps of those
// between.  Tiles take their numbers from a counter in walking order, so every
// tile that is waited for is already running.  The maps are applied one by one
// from the farthest on, which is how the published values themselves arise:
// the result does not depend on how far the look had to go.
template <class E>
__device__ __forceinline__ void look_back(const Args<E>& a, int group, int tile, int step, int lane,
                                          float (&v)[kLaneCh<E>]) {
  constexpr int V = kLaneCh<E>;
  const int64_t base = static_cast<int64_t>(group) * a.n_tiles;
  const long long begun = clock64();
  int depth = 0;  // maps to apply
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = 0.f;
  while (true) {
    const int mine = tile - step * (depth + 1 + lane);
    const bool in = mine >= 0 && mine < a.n_tiles;
    const int32_t f = in ? load_flag(a.flag + base + mine) : 2;
    const uint32_t done = __ballot_sync(kFull, f == 2), some = __ballot_sync(kFull, f >= 1);
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
    const bool out = clock64() - begun > kWaitBudgetCycles || load_flag(a.ticket + 1) != 0;
    if (__any_sync(kFull, out)) {
      if (lane == 0) {
        store_flag(a.ticket + 1, 1);
        if (a.status != nullptr) atomicOr(a.status, ENGRAM_ST_TIMEOUT);
      }
      return;
    }
  }
  __syncwarp();
  const int from = tile - step * (depth + 1);
  if (from >= 0 && from < a.n_tiles) {
    const float* p = a.value + (base + from) * kGroup<E> + lane * V;
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = __ldcg(p + j);
  }
#pragma unroll 4
  for (int i = depth; i > 0; --i) {
    const float2* m = a.map + (base + tile - step * i) * kGroup<E> + lane * V;
    if constexpr (V == 2) {
      const float4 q = __ldcg(reinterpret_cast<const float4*>(m));
      v[0] = apply_map(q.x, q.y, v[0]);
      v[1] = apply_map(q.z, q.w, v[1]);
    } else {
      const float2 q = __ldcg(m);
      v[0] = apply_map(q.x, q.y, v[0]);
    }
  }
}

template <class E>
__device__ __forceinline__ void publish_map(const Args<E>& a, int group, int tile, int lane, const float (&A)[kLaneCh<E>],
                                            const float (&B)[kLaneCh<E>]) {
  const int64_t at = static_cast<int64_t>(group) * a.n_tiles + tile;
  float2* m = a.map + at * kGroup<E> + lane * kLaneCh<E>;
#pragma unroll
  for (int j = 0; j < kLaneCh<E>; ++j) __stcg(m + j, make_float2(A[j], B[j]));
  __threadfence();
  __syncwarp();
  if (lane == 0) store_flag(a.flag + at, 1);
}

template <class E>
__device__ __forceinline__ void publish_value(const Args<E>& a, int group, int tile, int lane,
                                              const float (&v)[kLaneCh<E>]) {
  const int64_t at = static_cast<int64_t>(group) * a.n_tiles + tile;
  float* p = a.value + at * kGroup<E> + lane * kLaneCh<E>;
#pragma unroll
  for (int j = 0; j < kLaneCh<E>; ++j) __stcg(p + j, v[j]);
  __threadfence();
  __syncwarp();
  if (lane == 0) store_flag(a.flag + at, 2);
}

// The block's number in walking order.
__device__ __forceinline__ int take_ticket(int32_t* ticket, int32_t* shared) {
  if (threadIdx.x == 0) *shared = atomicAdd(ticket, 1);
  __syncthreads();
  return *shared;
}

// --------------------------------------------------------------------- forward

// A block handles kWarps * kSteps positions of 32 * kLaneCh channels, in one
// pass over memory: every warp loads its positions, reduces them to a map s ->
// A s + B per channel, one warp joins the maps, publishes the block's and
// looks back over the blocks before it for the state that comes in; then the
// warps walk their positions again, from registers, and write y.
constexpr int kFwdWarps = 8;
constexpr int kFwdTile = kFwdWarps * kSteps;
static_assert(kTile % kFwdTile == 0, "saved states fall on forward tiles");

template <class E, bool kVec>
__global__ void __launch_bounds__(kFwdWarps * 32, 4) forward_kernel(Args<E> a) {
  constexpr int V = kLaneCh<E>, G = kGroup<E>;
  __shared__ Marks<kFwdTile> marks;
  __shared__ float mapA[kFwdWarps][G], mapB[kFwdWarps][G], in[G];
  __shared__ int32_t number;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = take_ticket(a.ticket, &number);
  const int tile = n / a.n_groups, group = n - tile * a.n_groups;
  const int c = group * G + lane * V;
  const int t0 = tile * kFwdTile, tw = t0 + warp * kSteps;

  uint32_t xr[kSteps], gr[kSteps];
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int64_t t = tw + k;
    const bool ok = t < a.n_tokens;
    xr[k] = ok ? load4<E, kVec>(a.x + t * a.x_stride, c, a.dim) : 0u;
    gr[k] = ok ? load4<E, kVec>(a.g + t * a.g_stride, c, a.dim) : 0u;
  }
  const bool has_state = a.state != nullptr || a.state_out != nullptr;
  if (warp == 0)
    mark_tile<E, kFwdTile>(a, t0, marks, lane, c, a.state_out != nullptr && a.state_out != a.state, has_state);
  __syncthreads();
  const int at = warp * kSteps + (lane < kSteps ? lane : 0);
  const uint32_t live = __ballot_sync(kFull, lane < kSteps && marks.dead[at] == 0);
  const uint32_t first = __ballot_sync(kFull, lane < kSteps && marks.first[at] != kNone);
  const uint32_t last = __ballot_sync(kFull, lane < kSteps && marks.last[at] != kNone);

  // s_k = f s_{k-1} + b; a sequence's first position has f = 0
  float f[kSteps][V], b[kSteps][V], A[V], B[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    A[j] = 1.f;
    B[j] = 0.f;
  }
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    if (live >> k & 1u) {
      float gv[V], xv[V];
      widen<E>(gr[k], gv);
      widen<E>(xr[k], xv);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const Gate q = gate_of(gate_code<E>(gv[j]));
        f[k][j] = q.f;
        b[k][j] = q.u * xv[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        f[k][j] = 1.f;
        b[k][j] = 0.f;
      }
    }
    if (first >> k & 1u) {
      const int32_t slot = marks.first[warp * kSteps + k];
      float s0[V] = {};
      if (slot >= 0 && a.state != nullptr) load_state<E>(a.state + static_cast<int64_t>(slot) * a.dim, c, a.dim, s0);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        b[k][j] = fmaf(f[k][j], s0[j], b[k][j]);
        f[k][j] = 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      B[j] = fmaf(f[k][j], first >> k & 1u ? 0.f : B[j], b[k][j]);
      A[j] = first >> k & 1u ? kCut : A[j] * f[k][j];
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    mapA[warp][lane * V + j] = A[j];
    mapB[warp][lane * V + j] = B[j];
  }
  __syncthreads();

  if (warp == 0) {
    float v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      A[j] = 1.f;
      B[j] = 0.f;
    }
#pragma unroll
    for (int w = 0; w < kFwdWarps; ++w)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float p = mapA[w][lane * V + j], q = mapB[w][lane * V + j];
        B[j] = apply_map(p, q, B[j]);
        A[j] = join_factor(p, A[j]);
      }
    const bool cut = marks.any_first, more = tile + 1 < a.n_tiles;
    if (more) {
      if (cut) publish_value<E>(a, group, tile, lane, B);  // a sequence begins here: its state owes nothing to before
      else if (tile > 0) publish_map<E>(a, group, tile, lane, A, B);
    }
    if (tile == 0 || marks.first[0] != kNone) {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = 0.f;
    } else {
      look_back<E>(a, group, tile, 1, lane, v);
    }
    if (more && !cut) {
      float w[V];
#pragma unroll
      for (int j = 0; j < V; ++j) w[j] = apply_map(A[j], B[j], v[j]);
      publish_value<E>(a, group, tile, lane, w);
    }
    if (a.carry != nullptr && t0 % kTile == 0) store_state<E>(a.carry + static_cast<int64_t>(t0 / kTile) * a.dim, c, a.dim, v);
#pragma unroll
    for (int j = 0; j < V; ++j) in[lane * V + j] = v[j];
  }
  __syncthreads();

  float s[V];
#pragma unroll
  for (int j = 0; j < V; ++j) s[j] = in[lane * V + j];
  for (int w = 0; w < warp; ++w)
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = apply_map(mapA[w][lane * V + j], mapB[w][lane * V + j], s[j]);
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int64_t t = tw + k;
    if (t >= a.n_tokens) break;
    const bool start = first >> k & 1u, on = live >> k & 1u;
    float y[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      s[j] = fmaf(f[k][j], start ? 0.f : s[j], b[k][j]);
      y[j] = on ? s[j] : 0.f;
    }
    store4<E, kVec>(a.y + t * a.y_stride, c, a.dim, y);
    if (last >> k & 1u) {
      const int32_t slot = marks.last[warp * kSteps + k];
      if (slot >= 0 && a.state_out != nullptr)
        store_state<E>(a.state_out + static_cast<int64_t>(slot) * a.dim, c, a.dim, s);
    }
  }
}

// -------------------------------------------------------------------- backward

// The same scheme walked from the last tile to the first.  With m_t = f_t l_t,
// what position t passes back, m_t = f_t (dy_t + m_{t+1}): a tile maps the m
// that comes in to A m + C, A being the product of its gates.  The states
// before its positions come from the state saved in front of the tile.  Of a
// position only its gate code, w = f u (s_{t-1} - x) and dy stay in registers.
constexpr int kBwdWarps = kTile / kSteps;

template <class E, bool kVec>
__global__ void __launch_bounds__(kBwdWarps * 32, 2) backward_kernel(Args<E> a) {
  constexpr int V = kLaneCh<E>, G = kGroup<E>;
  __shared__ Marks<kTile> marks;
  __shared__ float mapA[kBwdWarps][G], mapB[kBwdWarps][G], mapC[kBwdWarps][G], in[G];
  // the last states' gradients, read before the tile publishes: a block that
  // waits for this one may then write the first states' in their place
  __shared__ float held[kTile][G];
  __shared__ int32_t number;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = take_ticket(a.ticket, &number);
  const int back = n / a.n_groups, group = n - back * a.n_groups;
  const int tile = a.n_tiles - 1 - back;
  const int c = group * G + lane * V;
  const int t0 = tile * kTile, tw = t0 + warp * kSteps;

  uint32_t xr[kSteps], gr[kSteps], dr[kSteps];
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int64_t t = tw + k;
    const bool ok = t < a.n_tokens;
    xr[k] = ok ? load4<E, kVec>(a.x + t * a.x_stride, c, a.dim) : 0u;
    gr[k] = ok ? load4<E, kVec>(a.g + t * a.g_stride, c, a.dim) : 0u;
    dr[k] = ok ? load4<E, kVec>(a.dy + t * a.dy_stride, c, a.dim) : 0u;
  }
  if (warp == 0) mark_tile<E, kTile>(a, t0, marks, lane, c, false, a.state != nullptr || a.dstate != nullptr);
  __syncthreads();
  const int at = warp * kSteps + (lane < kSteps ? lane : 0);
  const uint32_t live = __ballot_sync(kFull, lane < kSteps && marks.dead[at] == 0);
  const uint32_t first = __ballot_sync(kFull, lane < kSteps && marks.first[at] != kNone);
  const uint32_t last = __ballot_sync(kFull, lane < kSteps && marks.last[at] != kNone);

  float code[kSteps][V], A[V], B[V], C[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    A[j] = 1.f;
    B[j] = 0.f;
    C[j] = 0.f;
  }
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    if (live >> k & 1u) {
      float gv[V];
      widen<E>(gr[k], gv);
#pragma unroll
      for (int j = 0; j < V; ++j) code[k][j] = gate_code<E>(gv[j]);
    } else {  // f = 1, u = 0
      xr[k] = dr[k] = 0u;
#pragma unroll
      for (int j = 0; j < V; ++j) code[k][j] = 0.f;
    }
    float xv[V], s0[V] = {};
    widen<E>(xr[k], xv);
    const bool start = first >> k & 1u;
    if (start) {
      const int32_t slot = marks.first[warp * kSteps + k];
      if (slot >= 0 && a.state != nullptr) load_state<E>(a.state + static_cast<int64_t>(slot) * a.dim, c, a.dim, s0);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const Gate q = gate_of(code[k][j]);
      B[j] = fmaf(q.f, start ? s0[j] : B[j], q.u * xv[j]);
      A[j] = start ? kCut : A[j] * q.f;
    }
  }
#pragma unroll
  for (int k = kSteps - 1; k >= 0; --k) {
    float dv[V];
    widen<E>(dr[k], dv);
    if (last >> k & 1u) {
      const int32_t slot = marks.last[warp * kSteps + k];
      float ds[V] = {};
      if (slot >= 0 && a.dstate != nullptr) load_state<E>(a.dstate + static_cast<int64_t>(slot) * a.dim, c, a.dim, ds);
#pragma unroll
      for (int j = 0; j < V; ++j) {  // nothing comes from the positions behind
        C[j] = ds[j];
        held[warp * kSteps + k][lane * V + j] = ds[j];
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const Gate q = gate_of(code[k][j]);
      C[j] = first >> k & 1u ? 0.f : q.f * (dv[j] + C[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    mapA[warp][lane * V + j] = A[j];
    mapB[warp][lane * V + j] = B[j];
    mapC[warp][lane * V + j] = C[j];
  }
  __syncthreads();

  if (warp == 0) {
    float v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      A[j] = 1.f;
      C[j] = 0.f;
    }
#pragma unroll
    for (int w = kBwdWarps - 1; w >= 0; --w)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float p = mapA[w][lane * V + j], q = mapC[w][lane * V + j];
        C[j] = apply_map(p, q, C[j]);
        A[j] = join_factor(p, A[j]);
      }
    const bool cut = marks.any_first, ends = tile + 1 == a.n_tiles, more = tile > 0;
    if (more) {
      if (cut) publish_value<E>(a, group, tile, lane, C);
      else if (!ends) publish_map<E>(a, group, tile, lane, A, C);
    }
    if (ends) {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = 0.f;
    } else {
      look_back<E>(a, group, tile, -1, lane, v);
    }
    if (more && !cut) {
      float w[V];
#pragma unroll
      for (int j = 0; j < V; ++j) w[j] = apply_map(A[j], C[j], v[j]);
      publish_value<E>(a, group, tile, lane, w);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) in[lane * V + j] = v[j];
  }
  // meanwhile the other warps: the states before their positions
  float s[V], w[kSteps][V];
  load_state<E>(a.carry + static_cast<int64_t>(tile) * a.dim, c, a.dim, s);
  for (int p = 0; p < warp; ++p)
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = apply_map(mapA[p][lane * V + j], mapB[p][lane * V + j], s[j]);
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    float xv[V];
    widen<E>(xr[k], xv);
    if (first >> k & 1u) {
      const int32_t slot = marks.first[warp * kSteps + k];
#pragma unroll
      for (int j = 0; j < V; ++j) s[j] = 0.f;
      if (slot >= 0 && a.state != nullptr) load_state<E>(a.state + static_cast<int64_t>(slot) * a.dim, c, a.dim, s);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const Gate q = gate_of(code[k][j]);
      w[k][j] = q.f * (s[j] - xv[j]) * q.u;
      s[j] = fmaf(q.f, s[j], q.u * xv[j]);
    }
  }
  __syncthreads();

  float m[V];
#pragma unroll
  for (int j = 0; j < V; ++j) m[j] = in[lane * V + j];
  for (int p = kBwdWarps - 1; p > warp; --p)
#pragma unroll
    for (int j = 0; j < V; ++j) m[j] = apply_map(mapA[p][lane * V + j], mapC[p][lane * V + j], m[j]);
#pragma unroll
  for (int k = kSteps - 1; k >= 0; --k) {
    const int64_t t = tw + k;
    if (t >= a.n_tokens) continue;
    if (last >> k & 1u) {
#pragma unroll
      for (int j = 0; j < V; ++j) m[j] = held[warp * kSteps + k][lane * V + j];
    }
    const bool on = live >> k & 1u;
    float dv[V], dx[V], dg[V];
    widen<E>(dr[k], dv);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const Gate q = gate_of(code[k][j]);
      const float l = dv[j] + m[j];
      dx[j] = on ? l * q.u : 0.f;
      dg[j] = on ? l * w[k][j] : 0.f;
      m[j] = q.f * l;
    }
    store4<E, kVec>(a.dx + t * a.dx_stride, c, a.dim, dx);
    store4<E, kVec>(a.dg + t * a.dg_stride, c, a.dim, dg);
    if (first >> k & 1u) {
      const int32_t slot = marks.first[warp * kSteps + k];
      if (slot >= 0 && a.dstate != nullptr) store_state<E>(a.dstate + static_cast<int64_t>(slot) * a.dim, c, a.dim, m);
#pragma unroll
      for (int j = 0; j < V; ++j) m[j] = 0.f;
    }
  }
}

// ------------------------------------------------------------------ other parts

// The states of empty sequences when there are no positions at all.
template <class E>
__global__ void __launch_bounds__(128) copy_states_kernel(Args<E> a) {
  const int32_t slot = slot_of(a, blockIdx.x);
  if (slot < 0) return;
  for (int d = threadIdx.x; d < a.dim; d += blockDim.x)
    a.state_out[static_cast<int64_t>(slot) * a.dim + d] =
        a.state != nullptr ? a.state[static_cast<int64_t>(slot) * a.dim + d] : 0.f;
}

constexpr int kThreads = 128;

template <class E, bool kVec>
__global__ void __launch_bounds__(kThreads) step_kernel(Args<E> a) {
  constexpr int V = kLaneCh<E>;
  const int64_t b = blockIdx.x;
  const int c = (blockIdx.y * kThreads + threadIdx.x) * V;
  if (c >= a.dim) return;
  const uint32_t xr = load4<E, kVec>(a.x + b * a.x_stride, c, a.dim);
  const uint32_t gr = load4<E, kVec>(a.g + b * a.g_stride, c, a.dim);
  const int32_t slot = slot_of(a, b);
  float s[V] = {};
  if (slot >= 0) {
    float xv[V], gv[V];
    load_state<E>(a.state + static_cast<int64_t>(slot) * a.dim, c, a.dim, s);
    widen<E>(xr, xv);
    widen<E>(gr, gv);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const Gate q = gate_of(gate_code<E>(gv[j]));
      s[j] = fmaf(q.f, s[j], q.u * xv[j]);
    }
    store_state<E>(a.state_out + static_cast<int64_t>(slot) * a.dim, c, a.dim, s);
  }
  store4<E, kVec>(a.y + b * a.y_stride, c, a.dim, s);
}

// The parts of the scans' workspace: counters and flags (zeroed before each
// scan), then the tiles' maps and values.
struct ScanSpace {
  int32_t* ticket;
  int32_t* flag;
  float2* map;
  float* value;
  size_t zeroed, bytes;
};

// Sized for the smaller of the two tiles and the narrower group, which serves
// both passes and both types.
ScanSpace scan_space(void* base, int64_t n_tokens, int32_t dim) {
  constexpr int kNarrow = kGroup<train::F32>;
  const size_t tiles = static_cast<size_t>((n_tokens + kFwdTile - 1) / kFwdTile);
  const size_t groups = static_cast<size_t>((dim + kNarrow - 1) / kNarrow) + 1;  // + 1: a bf16 group may be half empty
  ScanSpace s;
  char* p = static_cast<char*>(base);
  s.ticket = reinterpret_cast<int32_t*>(p);
  s.flag = s.ticket + 2;
  s.zeroed = (2 + tiles * groups) * 4;
  size_t at = round256(s.zeroed);
  s.map = reinterpret_cast<float2*>(p + at);
  at += round256(tiles * groups * kNarrow * 8);
  s.value = reinterpret_cast<float*>(p + at);
  s.bytes = at + round256(tiles * groups * kNarrow * 4);
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

// Whether rows of `stride` elements from p can be read 4 bytes at a time.
template <class E>
bool pairs(const void* p, int64_t stride) {
  return E::kBytes == 4 || (aligned(p, 4) && stride % 2 == 0);
}

template <class E>
int launch_scan(Args<E>& a, bool backward, void* workspace, cudaStream_t st) {
  const ScanSpace w = scan_space(workspace, a.n_tokens, a.dim);
  const int tile = backward ? kTile : kFwdTile;
  a.n_tiles = (a.n_tokens + tile - 1) / tile;
  a.n_groups = (a.dim + kGroup<E> - 1) / kGroup<E>;
  a.ticket = w.ticket;
  a.flag = w.flag;
  a.map = w.map;
  a.value = w.value;
  const int64_t blocks = static_cast<int64_t>(a.n_tiles) * a.n_groups;
  if (blocks > 0x7fffffff) return fail(ENGRAM_E_RANGE, "too many positions times channels");
  cudaError_t err = cudaMemsetAsync(w.ticket, 0, (2 + static_cast<size_t>(blocks)) * 4, st);
  if (err != cudaSuccess) return fail(ENGRAM_E_CUDA, "cudaMemsetAsync: %s", cudaGetErrorString(err));
  const int grid = static_cast<int>(blocks);
  bool vec = a.dim % kLaneCh<E> == 0 && pairs<E>(a.x, a.x_stride) && pairs<E>(a.g, a.g_stride);
  if (!backward) {
    vec = vec && pairs<E>(a.y, a.y_stride);
    if (vec) forward_kernel<E, true><<<grid, kFwdWarps * 32, 0, st>>>(a);
    else forward_kernel<E, false><<<grid, kFwdWarps * 32, 0, st>>>(a);
  } else {
    vec = vec && pairs<E>(a.dy, a.dy_stride) && pairs<E>(a.dx, a.dx_stride) && pairs<E>(a.dg, a.dg_stride);
    if (vec) backward_kernel<E, true><<<grid, kBwdWarps * 32, 0, st>>>(a);
    else backward_kernel<E, false><<<grid, kBwdWarps * 32, 0, st>>>(a);
  }
  return check_launch("recurrence");
}

template <class E>
int launch_step(const Args<E>& a, int64_t batch, cudaStream_t st) {
  const int per = kThreads * kLaneCh<E>;
  const dim3 grid(static_cast<unsigned>(batch), (a.dim + per - 1) / per);
  const bool vec = a.dim % kLaneCh<E> == 0 && pairs<E>(a.x, a.x_stride) && pairs<E>(a.g, a.g_stride) &&
                   pairs<E>(a.y, a.y_stride);
  if (vec) step_kernel<E, true><<<grid, kThreads, 0, st>>>(a);
  else step_kernel<E, false><<<grid, kThreads, 0, st>>>(a);
  return check_launch("step_kernel");
}

}  // namespace
}  // namespace engram

using namespace engram;

extern "C" size_t engram_recurrence_carry_bytes(int64_t n_tokens, int32_t dim) {
  if (n_tokens < 0 || dim < 1) return 0;
  return static_cast<size_t>((n_tokens + kTile - 1) / kTile) * dim * sizeof(float);
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
    if (n_tokens > 0) return launch_scan<E>(a, false, workspace_d, as_stream(stream));
    if (state_out_d == nullptr || state_out_d == state_d) return static_cast<int>(ENGRAM_OK);
    copy_states_kernel<E><<<static_cast<int>(n_seqs), 128, 0, as_stream(stream)>>>(a);
    return check_launch("copy_states_kernel");
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
  if ((rc = check_device(nullptr))) return rc;
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
    return launch_scan<E>(a, true, workspace_d, as_stream(stream));
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
