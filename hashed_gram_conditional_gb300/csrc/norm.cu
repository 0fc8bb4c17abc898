// The norm behind a block with its gate, the residual add with its scale, and
// the norm in front of the next block; and the gradient of the three together.
//
// With r(u) = (mean(u^2) + eps)^-1/2, over each group of y's row and over h'
// whole row:
//   n  = y r(y) w silu(gate)
//   h' = h + s n                      (rounded to the type)
//   x  = h' r(h') w_next
// and, with l the gradient of h' in all, c = (dx w_next . h') r(h')^3 / dim:
//   l  = dh + dx w_next r(h') - h' c
//   dn = l s,  dgate = dn y r w silu'(gate),  p = dn silu(gate) w
//   dy = p r - y r^3 (p . y) / group
//   dw_next = sum dx h' r(h'),  dscale = sum l n,  dw = sum dn silu(gate) y r
//
// Every array is read or written once.  A block holds a row in registers, in 16-byte
// vectors, from the first sum to the last store; with many rows of one group the blocks
// stay and go from row to row with the next rows on their way; the gradient's always do, and
// keep the weights' sums of their columns.
// 16,384 x 5120 bf16 with gate, residual and next norm: 130 us (6.5 TB/s, 97 % of a copy's
// rate), bound by memory, as is the gradient: 237 us, of which 227 (5.9 TB/s) for the rows and
// 9 for the weights' sums.  Rows that are not 16-byte aligned go a value a thread
// (8192 x 5119: 381 and 950 us), and rows longer than a block's threads hold are walked
// several times.  The gradient of aligned rows of more than 7504 bf16 or 3752 fp32 values, of
// which no three fit a block's shared memory, goes without rows on their way: 16,384 x 8192
// bf16 701 us (3.1 TB/s), 16,384 x 5120 fp32 721 (3.7), where sums of columns take registers
// that are not there.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "engram_internal.h"
#include "train_device.cuh"

namespace engram {
namespace {

constexpr int kMaxGroups = ENGRAM_NORM_MAX_GROUPS;
constexpr int kAnyThreads = 256;
// Blocks that a gradient's sums of the weights are spread over.
constexpr int kParts = 304;

struct Args {
  const void *y, *gate, *h, *dh, *dx;
  void *h_out, *x_out, *dy, *dgate, *dres;
  int64_t y_stride, gate_stride, h_stride, h_out_stride, x_stride, dh_stride, dx_stride, dy_stride, dgate_stride, dres_stride;
  const float *w, *scale, *w_next;
  float* parts;  // [2][blocks][dim]: the sums of l silu(gate) y r, for w and scale, and of dx h' r, for w_next
  int64_t rows;
  int32_t dim, groups, width;  // width: of a group
  int32_t vecs, vecs_log2;     // 16-byte vectors of a row; log2 of a group's if they are 1, 2, 4 .. 32, else -1
  float eps;
};

constexpr int kThreads = 512;  // at most, where registers for more than one vector a thread are wanted

// What a thread reads and writes at once: 16 bytes, or where rows are not aligned to
// them one value.
template <class E_>
struct Wide {
  using E = E_;
  using Raw = uint4;
  static constexpr int N = 16 / E::kBytes, kMost = kThreads;
  static __device__ __forceinline__ Raw none() { return make_uint4(0u, 0u, 0u, 0u); }
  static __device__ __forceinline__ void widen(const Raw& x, float (&f)[N]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (E::kBytes == 2) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      } else {
        f[j] = __uint_as_float(w[j]);
      }
    }
  }
  static __device__ __forceinline__ Raw narrow(const float (&f)[N]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (E::kBytes == 2) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&b);
      } else {
        w[j] = __float_as_uint(f[j]);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ void weights(const float* p, float (&f)[N]) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(p + j));
      f[j] = x.x;
      f[j + 1] = x.y;
      f[j + 2] = x.z;
      f[j + 3] = x.w;
    }
  }
};
// The same in pairs, for the instructions that take two values at once.
template <class E>
struct Pairs {
  static constexpr int N = 8 / E::kBytes;
  static __device__ __forceinline__ void widen(const uint4& x, uint64_t (&f)[N]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if constexpr (E::kBytes == 2) f[j] = f2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
      else f[j] = f2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
    }
  }
  static __device__ __forceinline__ uint4 narrow(const uint64_t (&f)[N]) {
    float x[2 * N];
#pragma unroll
    for (int j = 0; j < N; ++j) f2_split(f[j], x[2 * j], x[2 * j + 1]);
    return Wide<E>::narrow(x);
  }
  static __device__ __forceinline__ void weights(const float* p, uint64_t (&f)[N]) {
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      const float4 x = p != nullptr ? __ldg(reinterpret_cast<const float4*>(p + 2 * j)) : make_float4(1.f, 1.f, 1.f, 1.f);
      f[j] = f2(x.x, x.y);
      f[j + 1] = f2(x.z, x.w);
    }
  }
};
__device__ __forceinline__ uint64_t f2_both(float x) { return f2(x, x); }
__device__ __forceinline__ float f2_sum(uint64_t x) {
  float a, b;
  f2_split(x, a, b);
  return a + b;
}

template <class E_>
struct Single {
  using E = E_;
  using Raw = typename E::T;
  static constexpr int N = 1, kMost = 1024;
  static __device__ __forceinline__ Raw none() { return Raw(0); }
  static __device__ __forceinline__ void widen(const Raw& x, float (&f)[1]) { f[0] = E::load(&x); }
  static __device__ __forceinline__ Raw narrow(const float (&f)[1]) {
    Raw x;
    E::store(&x, f[0]);
    return x;
  }
  static __device__ __forceinline__ void weights(const float* p, float (&f)[1]) { f[0] = __ldg(p); }
};

template <class P>
__device__ __forceinline__ void load_weights(const float* p, float (&f)[P::N]) {
  if (p != nullptr) {
    P::weights(p, f);
  } else {
#pragma unroll
    for (int j = 0; j < P::N; ++j) f[j] = 1.f;
  }
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float inverse_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// sigmoid(z): bf16's from the hardware's exponential and division (2^-21, and 2^-24 |z| from
// the exponent's rounding: 2^-17 at |z| = 80, far below a bf16 rounding), fp32's from the
// rounded ones.
template <class E>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (E::kBytes == 2) return __fdividef(1.f, 1.f + __expf(-z));
  return 1.f / (1.f + expf(-z));
}

template <class E>
__device__ __forceinline__ uint64_t sigmoid_pair(uint64_t z) {
  float a, b;
  if constexpr (E::kBytes == 2) {
    f2_split(f2_mul(z, f2(-1.4426950408889634f, -1.4426950408889634f)), a, b);
    f2_split(f2_add(f2(exp2_fast(a), exp2_fast(b)), f2(1.f, 1.f)), a, b);
    return f2(inverse_fast(a), inverse_fast(b));
  }
  f2_split(z, a, b);
  return f2(sigmoid<E>(a), sigmoid<E>(b));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The block's sum, the same in every thread.  `slot` has a place for each warp
// and is free again at the block's next barrier but one.
__device__ __forceinline__ float block_sum(float v, float* slot) {
  v = warp_sum(v);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < warps ? slot[lane] : 0.f);
}

// The sum over each group of the values that the vectors give, for the groups of
// this thread's vectors.  Groups of 1, 2, .. 32 vectors are joined among lanes, a
// row that is one group by the block, and others by way of `part`, which has a
// place for every vector and is free again at the block's next barrier.
template <int kPer>
__device__ __forceinline__ void group_sums(const Args& a, float (&v)[kPer], float* part, float* slot) {
  if (a.groups == 1) {
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) all += v[i];
    all = block_sum(all, slot);
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = all;
    return;
  }
  const int per = a.vecs / a.groups;
  if (a.vecs_log2 >= 0) {  // lanes of a group lie together: vector t + i * blockDim, and 32 divides blockDim
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      for (int o = per >> 1; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    return;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int at = threadIdx.x + i * blockDim.x;
    if (at < a.vecs) part[at] = v[i];
  }
  __syncthreads();
  float* sums = part + a.vecs;
  for (int g = threadIdx.x >> 5; g < a.groups; g += blockDim.x >> 5) {
    float s = 0.f;
    for (int k = threadIdx.x & 31; k < per; k += 32) s += part[g * per + k];
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0) sums[g] = s;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int at = threadIdx.x + i * blockDim.x;
    v[i] = at < a.vecs ? sums[at / per] : 0.f;
  }
  __syncthreads();
}

template <class E, class As = typename E::T>
__device__ __forceinline__ const As* row_of(const void* p, int64_t row, int64_t stride) {
  return reinterpret_cast<const As*>(static_cast<const typename E::T*>(p) + row * stride);
}
template <class E, class As = typename E::T>
__device__ __forceinline__ As* row_of(void* p, int64_t row, int64_t stride) {
  return reinterpret_cast<As*>(static_cast<typename E::T*>(p) + row * stride);
}
// (cached no longer than the row's own use)
template <class P>
__device__ __forceinline__ typename P::Raw vector_at(const void* p, int64_t row, int64_t stride, int v) {
  return __ldcs(row_of<typename P::E, typename P::Raw>(p, row, stride) + v);
}

__device__ __forceinline__ const float* weights_at(const Args& a, int e) {
  return a.w == nullptr ? nullptr : a.w + (a.groups == 1 ? e : e % a.width);
}

__device__ __forceinline__ void copy_vec(uint32_t to, const uint4* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ uint4 own_vec(uint32_t at) {
  uint4 x;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at) : "memory");
  return x;
}
constexpr int kRingThreads = 640, kRingSmem = 220 * 1024;

// ------------------------------------------------------------------- forward

template <class P, int kPer>
__global__ void __launch_bounds__(P::kMost) norm_kernel(Args a) {
  using E = typename P::E;
  using Raw = typename P::Raw;
  constexpr int N = P::N;
  extern __shared__ float part[];
  __shared__ float slot[2][32];
  const int64_t row = blockIdx.x;
  const Raw none = P::none();
  Raw ry[kPer], rz[kPer], rh[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    ry[i] = v < a.vecs ? vector_at<P>(a.y, row, a.y_stride, v) : none;
    rz[i] = v < a.vecs && a.gate ? vector_at<P>(a.gate, row, a.gate_stride, v) : none;
    rh[i] = v < a.vecs && a.h ? vector_at<P>(a.h, row, a.h_stride, v) : none;
  }
  float sq[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    float y[N];
    P::widen(ry[i], y);
    sq[i] = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) sq[i] = fmaf(y[j], y[j], sq[i]);
  }
  group_sums(a, sq, part, slot[0]);
  const float inv_width = 1.f / a.width, r_all = rsqrtf(sq[0] * inv_width + a.eps);  // (of a row that is one group)
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= a.vecs) continue;
    const float r = a.groups == 1 ? r_all : rsqrtf(sq[i] * inv_width + a.eps);
    float y[N], h[N], w[N];
    P::widen(ry[i], y);
    P::widen(rh[i], h);
    load_weights<P>(weights_at(a, v * N), w);
#pragma unroll
    for (int j = 0; j < N; ++j) y[j] *= r * w[j];
    if (a.gate) {
      float z[N];
      P::widen(rz[i], z);
#pragma unroll
      for (int j = 0; j < N; ++j) y[j] *= z[j] * sigmoid<E>(z[j]);
    }
    load_weights<P>(a.scale ? a.scale + v * N : nullptr, w);
#pragma unroll
    for (int j = 0; j < N; ++j) h[j] = fmaf(y[j], w[j], h[j]);
    rh[i] = P::narrow(h);
    row_of<E, Raw>(a.h_out, row, a.h_out_stride)[v] = rh[i];
    P::widen(rh[i], h);
#pragma unroll
    for (int j = 0; j < N; ++j) sum = fmaf(h[j], h[j], sum);
  }
  if (a.x_out == nullptr) return;
  sum = block_sum(sum, slot[1]);
  const float r = rsqrtf(sum / a.dim + a.eps);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= a.vecs) continue;
    float h[N], w[N];
    P::widen(rh[i], h);
    load_weights<P>(a.w_next ? a.w_next + v * N : nullptr, w);
#pragma unroll
    for (int j = 0; j < N; ++j) h[j] *= r * w[j];
    row_of<E, Raw>(a.x_out, row, a.x_stride)[v] = P::narrow(h);
  }
}

// The same for many rows of one group: the blocks stay and go from row to row, with the next
// rows on their way through shared memory (a thread copies and reads its own vectors, one of
// each array) and the weights of their columns in registers.  A row's sum of h'^2 and the
// next one's of y^2 are joined at one barrier.  (us, this form and a block for each row,
// bf16: 16,384 x 5120 130 and 147; 32,768 x 1280 74 and 80; 2048 x 5120 26 and 27; 700 x 5120
// 17 and 16; in 40 groups, which the lanes join, 16,384 x 5120 156 and 152.)
constexpr int kAheadRows = 4;  // rows in use and on their way
template <class E>
__global__ void __launch_bounds__(kRingThreads, 1) norm_ring_kernel(Args a) {
  using V = Pairs<E>;
  constexpr int N = V::N;
  extern __shared__ __align__(16) float part[];
  __shared__ float2 slot[2][32];
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5, v = threadIdx.x;
  const bool in = v < a.vecs;
  const uint32_t ring = smem_u32(part) + v * 16;
  auto place = [&](int stage, int array) { return ring + (stage * 3 + array) * a.vecs * 16; };
  const float inv_dim = 1.f / a.dim;
  uint64_t ws[N], wn[N];  // w times scale, and w_next
  if (in) {
    uint64_t s[N];
    V::weights(a.w ? a.w + v * 2 * N : nullptr, ws);
    V::weights(a.scale ? a.scale + v * 2 * N : nullptr, s);
    V::weights(a.w_next ? a.w_next + v * 2 * N : nullptr, wn);
#pragma unroll
    for (int j = 0; j < N; ++j) ws[j] = f2_mul(ws[j], s[j]);
  }
  auto fetch = [&](int64_t row, int stage) {
    if (row < a.rows && in) {
      copy_vec(place(stage, 0), row_of<E, uint4>(a.y, row, a.y_stride) + v);
      if (a.gate) copy_vec(place(stage, 1), row_of<E, uint4>(a.gate, row, a.gate_stride) + v);
      if (a.h) copy_vec(place(stage, 2), row_of<E, uint4>(a.h, row, a.h_stride) + v);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto square = [&](int stage) {
    if (!in) return 0.f;
    uint64_t y[N], yy = f2_both(0.f);
    V::widen(own_vec(place(stage, 0)), y);
#pragma unroll
    for (int j = 0; j < N; ++j) yy = f2_fma(y[j], y[j], yy);
    return f2_sum(yy);
  };
  // The block's two sums at one barrier, in places that the next but one takes again.
  int parity = 0;
  auto join = [&](float& s0, float& s1) {
    s0 = warp_sum(s0);
    s1 = warp_sum(s1);
    if (warps == 1) return;
    float2* to = slot[parity];
    parity ^= 1;
    if (lane == 0) to[threadIdx.x >> 5] = make_float2(s0, s1);
    __syncthreads();
    const float2 x = lane < warps ? to[lane] : make_float2(0.f, 0.f);
    s0 = warp_sum(x.x);
    s1 = warp_sum(x.y);
  };
  for (int k = 0; k < kAheadRows - 1; ++k) fetch(blockIdx.x + static_cast<int64_t>(k) * gridDim.x, k);
  asm volatile("cp.async.wait_group %0;" ::"n"(kAheadRows - 2) : "memory");
  float sum = 0.f, sq = square(0);
  join(sum, sq);
  int stage = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int next = stage + 1 == kAheadRows ? 0 : stage + 1;
    fetch(row + static_cast<int64_t>(kAheadRows - 1) * gridDim.x, stage == 0 ? kAheadRows - 1 : stage - 1);
    uint64_t h[N], hh = f2_both(0.f);
    if (in) {
      const float r = rsqrtf(sq * inv_dim + a.eps);
      uint64_t y[N];
      V::widen(own_vec(place(stage, 0)), y);
#pragma unroll
      for (int j = 0; j < N; ++j) y[j] = f2_mul(f2_mul(y[j], f2_both(r)), ws[j]);
      if (a.gate) {
        uint64_t z[N];
        V::widen(own_vec(place(stage, 1)), z);
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] = f2_mul(y[j], f2_mul(z[j], sigmoid_pair<E>(z[j])));
      }
      if (a.h) {
        V::widen(own_vec(place(stage, 2)), h);
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] = f2_add(y[j], h[j]);
      }
      const uint4 kept = V::narrow(y);
      row_of<E, uint4>(a.h_out, row, a.h_out_stride)[v] = kept;
      V::widen(kept, h);
#pragma unroll
      for (int j = 0; j < N; ++j) hh = f2_fma(h[j], h[j], hh);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kAheadRows - 2) : "memory");
    sq = square(next);  // (of a row behind the last: not used)
    sum = f2_sum(hh);
    join(sum, sq);
    if (in && a.x_out != nullptr) {
      const float r = rsqrtf(sum * inv_dim + a.eps);
#pragma unroll
      for (int j = 0; j < N; ++j) h[j] = f2_mul(f2_mul(h[j], f2_both(r)), wn[j]);
      row_of<E, uint4>(a.x_out, row, a.x_stride)[v] = V::narrow(h);
    }
    stage = next;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// out[g] = last(sum over the group's values of f(g, place in it)), by a warp for each group
// or, where there are few, by the block; a barrier follows.
template <class F, class L>
__device__ __forceinline__ void any_groups(const Args& a, float* out, float* slot, F f, L last) {
  if (a.groups < kAnyThreads / 32) {
    for (int g = 0; g < a.groups; ++g) {
      float s = 0.f;
      for (int k = threadIdx.x; k < a.width; k += kAnyThreads) s += f(g, k);
      s = block_sum(s, slot);
      if (threadIdx.x == 0) out[g] = last(s);
      __syncthreads();
    }
    return;
  }
  for (int g = threadIdx.x >> 5; g < a.groups; g += kAnyThreads / 32) {
    float s = 0.f;
    for (int k = threadIdx.x & 31; k < a.width; k += 32) s += f(g, k);
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0) out[g] = last(s);
  }
  __syncthreads();
}

template <class E>
__global__ void __launch_bounds__(kAnyThreads) norm_any_kernel(Args a) {
  __shared__ float sums[kMaxGroups], slot[32];
  const int64_t row = blockIdx.x;
  const auto* y = row_of<E>(a.y, row, a.y_stride);
  auto* out = row_of<E>(a.h_out, row, a.h_out_stride);
  any_groups(a, sums, slot,
             [&](int g, int k) {
               const float v = E::load(y + g * a.width + k);
               return v * v;
             },
             [&](float s) { return rsqrtf(s / a.width + a.eps); });
  float sum = 0.f;
  for (int e = threadIdx.x; e < a.dim; e += kAnyThreads) {
    const int g = e / a.width;
    float n = E::load(y + e) * (sums[g] * (a.w ? a.w[e - g * a.width] : 1.f));
    if (a.gate) {
      const float z = E::load(row_of<E>(a.gate, row, a.gate_stride) + e);
      n *= z * sigmoid<E>(z);
    }
    const float h = a.h ? E::load(row_of<E>(a.h, row, a.h_stride) + e) : 0.f;
    E::store(out + e, fmaf(n, a.scale ? a.scale[e] : 1.f, h));
    const float kept = E::load(out + e);
    sum = fmaf(kept, kept, sum);
  }
  if (a.x_out == nullptr) return;
  const float r = rsqrtf(block_sum(sum, slot) / a.dim + a.eps);
  auto* x = row_of<E>(a.x_out, row, a.x_stride);
  for (int e = threadIdx.x; e < a.dim; e += kAnyThreads)
    E::store(x + e, E::load(out + e) * (r * (a.w_next ? a.w_next[e] : 1.f)));
}

// ------------------------------------------------------------------ gradient

template <class P, int kPer, int kMost>
__global__ void __launch_bounds__(kMost) norm_grad_kernel(Args a) {
  using E = typename P::E;
  using Raw = typename P::Raw;
  constexpr int N = P::N;
  extern __shared__ float part[];
  __shared__ float slot[4][32];
  const Raw none = P::none();
  // the columns' sums: single values' threads have them in shared memory, each its own
  constexpr bool kKept = N > 1;
  float q[kKept ? kPer : 1][N] = {}, dn[kKept ? kPer : 1][N] = {};
  float* sums = part + (a.groups > 1 && a.vecs_log2 < 0 ? a.vecs + a.groups : 0);
  for (int v = threadIdx.x; !kKept && v < a.vecs; v += blockDim.x) sums[v] = sums[a.vecs + v] = 0.f;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    Raw ry[kPer], rz[kPer], rl[kPer], rh[kPer], rx[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      const bool in = v < a.vecs;
      ry[i] = in ? vector_at<P>(a.y, row, a.y_stride, v) : none;
      rh[i] = in && a.dx ? vector_at<P>(a.h, row, a.h_stride, v) : none;
      rx[i] = in && a.dx ? vector_at<P>(a.dx, row, a.dx_stride, v) : none;
      rl[i] = in && a.dh ? vector_at<P>(a.dh, row, a.dh_stride, v) : none;
      rz[i] = in && a.gate ? vector_at<P>(a.gate, row, a.gate_stride, v) : none;
    }
    float sq[kPer], l[kPer][N];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      float y[N];
      P::widen(ry[i], y);
      P::widen(rl[i], l[i]);
      sq[i] = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) sq[i] = fmaf(y[j], y[j], sq[i]);
    }
    if (a.dx) {
      float hh = 0.f, xh = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= a.vecs) continue;
        float h[N], x[N], w[N];
        P::widen(rh[i], h);
        P::widen(rx[i], x);
        load_weights<P>(a.w_next ? a.w_next + v * N : nullptr, w);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          hh = fmaf(h[j], h[j], hh);
          xh = fmaf(x[j] * w[j], h[j], xh);
        }
      }
      hh = block_sum(hh, slot[0]);
      xh = block_sum(xh, slot[1]);
      const float r = rsqrtf(hh / a.dim + a.eps), c = xh * r * r * r / a.dim;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= a.vecs) continue;
        float h[N], x[N], w[N];
        P::widen(rh[i], h);
        P::widen(rx[i], x);
        load_weights<P>(a.w_next ? a.w_next + v * N : nullptr, w);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          x[j] *= r;
          l[i][j] += x[j] * w[j] - h[j] * c;
          if constexpr (kKept) dn[i][j] = fmaf(x[j], h[j], dn[i][j]);
          else sums[a.vecs + v] = fmaf(x[j], h[j], sums[a.vecs + v]);
        }
      }
    }
    group_sums(a, sq, part, slot[2]);
    const float inv_width = 1.f / a.width, r_all = rsqrtf(sq[0] * inv_width + a.eps);
    float along[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      along[i] = 0.f;
      if (v >= a.vecs) continue;
      if (a.dres) row_of<E, Raw>(a.dres, row, a.dres_stride)[v] = P::narrow(l[i]);
      const float r = a.groups == 1 ? r_all : rsqrtf(sq[i] * inv_width + a.eps);
      sq[i] = r;
      float y[N], z[N], w[N], s[N], dz[N];
      P::widen(ry[i], y);
      P::widen(rz[i], z);
      load_weights<P>(weights_at(a, v * N), w);
      load_weights<P>(a.scale ? a.scale + v * N : nullptr, s);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float sig = a.gate ? sigmoid<E>(z[j]) : 1.f, act = a.gate ? z[j] * sig : 1.f;
        const float hat = y[j] * r, g = l[i][j] * s[j] * w[j];  // g: the gradient of y r silu(gate)
        if constexpr (kKept) q[i][j] = fmaf(l[i][j] * act, hat, q[i][j]);
        else sums[v] = fmaf(l[i][j] * act, hat, sums[v]);
        dz[j] = g * hat * sig * fmaf(z[j], 1.f - sig, 1.f);
        l[i][j] = g * act;
        along[i] = fmaf(l[i][j], y[j], along[i]);
      }
      if (a.dgate) row_of<E, Raw>(a.dgate, row, a.dgate_stride)[v] = P::narrow(dz);
    }
    group_sums(a, along, part, slot[3]);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= a.vecs) continue;
      const float r = sq[i], c = along[i] * r * r * r * inv_width;
      float y[N];
      P::widen(ry[i], y);
#pragma unroll
      for (int j = 0; j < N; ++j) l[i][j] = l[i][j] * r - y[j] * c;
      row_of<E, Raw>(a.dy, row, a.dy_stride)[v] = P::narrow(l[i]);
    }
  }
  if (a.parts == nullptr) return;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= a.vecs) continue;
    float* to = a.parts + static_cast<int64_t>(blockIdx.x) * a.dim + v * N;
    const int64_t next = static_cast<int64_t>(gridDim.x) * a.dim;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      to[j] = kKept ? q[kKept ? i : 0][j] : sums[v];
      to[next + j] = kKept ? dn[kKept ? i : 0][j] : sums[a.vecs + v];
    }
  }
}

// The same with the rows on their way through shared memory: a thread copies its own
// vectors of the block's next rows ahead, and reads them when it wants them, so that
// registers hold little more than the weights and their sums and no barrier is for the
// copies.  (16,384 x 5120 bf16, us: 319 with single values and the weights read again for
// every row, 300 in pairs of values, 280 with w and scale in registers, 227 with w_next too.)
constexpr int kRing = 3;  // rows of a block in use, next, and on their way
constexpr int kArrays = 5;   // y, gate, dh, h', dx

template <class E, int kPer>
__global__ void __launch_bounds__(kPer == 1 ? kRingThreads : kThreads, 1) norm_grad_ring_kernel(Args a) {
  using V = Pairs<E>;
  using Raw = uint4;
  constexpr int N = V::N;  // pairs of a vector
  extern __shared__ __align__(16) float part[];
  __shared__ float slot[2][4][32], slot_along[32];
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const uint32_t ring = smem_u32(part) + (a.groups > 1 && a.vecs_log2 < 0 ? (a.vecs + a.groups + 3) / 4 * 16 : 0);
  const uint32_t array_bytes = static_cast<uint32_t>(a.vecs) * 16;
  auto place = [&](int stage, int array, int v) { return ring + (stage * kArrays + array) * array_bytes + v * 16; };
  const float inv_dim = 1.f / a.dim, inv_width = 1.f / a.width;
  // w times scale and w_next, of the thread's columns; where it has two vectors, whose sums
  // take the registers, read again for every row
  auto scaled_weights = [&](int v, uint64_t (&ws)[N]) {
    uint64_t s[N];
    V::weights(weights_at(a, v * 2 * N), ws);
    V::weights(a.scale ? a.scale + v * 2 * N : nullptr, s);
#pragma unroll
    for (int j = 0; j < N; ++j) ws[j] = f2_mul(ws[j], s[j]);
  };
  auto next_weights = [&](int v, uint64_t (&wn)[N]) { V::weights(a.w_next ? a.w_next + v * 2 * N : nullptr, wn); };
  uint64_t own_ws[N], own_wn[N];
  if (kPer == 1 && static_cast<int>(threadIdx.x) < a.vecs) {
    scaled_weights(threadIdx.x, own_ws);
    next_weights(threadIdx.x, own_wn);
  }
  auto fetch = [&](int64_t row, int stage) {
    if (row < a.rows) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= a.vecs) continue;
        copy_vec(place(stage, 0, v), row_of<E, Raw>(a.y, row, a.y_stride) + v);
        if (a.gate) copy_vec(place(stage, 1, v), row_of<E, Raw>(a.gate, row, a.gate_stride) + v);
        if (a.dh) copy_vec(place(stage, 2, v), row_of<E, Raw>(a.dh, row, a.dh_stride) + v);
        if (a.dx) {
          copy_vec(place(stage, 3, v), row_of<E, Raw>(a.h, row, a.h_stride) + v);
          copy_vec(place(stage, 4, v), row_of<E, Raw>(a.dx, row, a.dx_stride) + v);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // of a row: its sums of h'^2 and dx w_next h', and y^2 of the thread's vectors
  auto first = [&](int stage, float (&sum)[4], float (&sq)[kPer]) {
    uint64_t hh = f2_both(0.f), xh = hh;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      sq[i] = 0.f;
      if (v >= a.vecs) continue;
      uint64_t y[N], yy = f2_both(0.f);
      V::widen(own_vec(place(stage, 0, v)), y);
#pragma unroll
      for (int j = 0; j < N; ++j) yy = f2_fma(y[j], y[j], yy);
      sq[i] = f2_sum(yy);
      sum[2] += sq[i];
      if (a.dx) {
        uint64_t h[N], x[N], w[N];
        V::widen(own_vec(place(stage, 3, v)), h);
        V::widen(own_vec(place(stage, 4, v)), x);
        if (kPer > 1) next_weights(v, w);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          hh = f2_fma(h[j], h[j], hh);
          xh = f2_fma(f2_mul(x[j], kPer > 1 ? w[j] : own_wn[j]), h[j], xh);
        }
      }
    }
    sum[0] += f2_sum(hh);
    sum[1] += f2_sum(xh);
  };
  // The block's four sums at one barrier.  A lane keeps half of what it has at each of
  // the first two exchanges: eight lanes have one sum each, 6 exchanges and not 20.
  int parity = 0;
  const int mine = lane >> 3;
  auto join = [&](float (&sum)[4]) {
    const bool up = lane & 16, odd = lane & 8;
    const float a0 = up ? sum[0] : sum[2], a1 = up ? sum[1] : sum[3];
    float k0 = (up ? sum[2] : sum[0]) + __shfl_xor_sync(0xffffffffu, a0, 16);
    float k1 = (up ? sum[3] : sum[1]) + __shfl_xor_sync(0xffffffffu, a1, 16);
    float s = (odd ? k1 : k0) + __shfl_xor_sync(0xffffffffu, odd ? k0 : k1, 8);
    s += __shfl_xor_sync(0xffffffffu, s, 4);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    if (warps > 1) {
      float(&to)[4][32] = slot[parity];
      parity ^= 1;
      if ((lane & 7) == 0) to[mine][threadIdx.x >> 5] = s;
      __syncthreads();
      s = 0.f;
#pragma unroll
      for (int w = 0; w < 32; w += 8)
        if (w + (lane & 7) < warps) s += to[mine][w + (lane & 7)];
      s += __shfl_xor_sync(0xffffffffu, s, 4);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      s += __shfl_xor_sync(0xffffffffu, s, 1);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[k] = __shfl_sync(0xffffffffu, s, k * 8);
  };
  // sums over the rows: l silu(gate) y r, of which dw and dscale are multiples by column, and dx h' r
  uint64_t q[kPer][N], dn[kPer][N];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) q[i][j] = dn[i][j] = f2_both(0.f);
  for (int k = 0; k < kRing - 1; ++k) fetch(blockIdx.x + static_cast<int64_t>(k) * gridDim.x, k);
  asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
  float sum[4] = {0.f, 0.f, 0.f, 0.f}, sq[kPer];
  first(0, sum, sq);
  join(sum);
  int stage = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int next = stage + 1 == kRing ? 0 : stage + 1;
    fetch(row + static_cast<int64_t>(kRing - 1) * gridDim.x, stage == 0 ? kRing - 1 : stage - 1);
    if (a.groups == 1) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) sq[i] = sum[2];
    } else {
      group_sums(a, sq, part, slot_along);
    }
    const float r2 = rsqrtf(sum[0] * inv_dim + a.eps), c2 = sum[1] * r2 * r2 * r2 * inv_dim;
    float along[kPer], r1[kPer];
    uint64_t l[kPer][N];
    float coming[4] = {0.f, 0.f, 0.f, 0.f};  // the next row's sums, and this one's of p y
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      along[i] = 0.f;
      if (v >= a.vecs) continue;
      if (a.dh) {
        V::widen(own_vec(place(stage, 2, v)), l[i]);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) l[i][j] = f2_both(0.f);
      }
      if (a.dx) {
        uint64_t h[N], x[N], w[N];
        V::widen(own_vec(place(stage, 3, v)), h);
        V::widen(own_vec(place(stage, 4, v)), x);
        if (kPer > 1) next_weights(v, w);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          x[j] = f2_mul(x[j], f2_both(r2));
          l[i][j] = f2_fma(h[j], f2_both(-c2), f2_fma(x[j], kPer > 1 ? w[j] : own_wn[j], l[i][j]));
          dn[i][j] = f2_fma(x[j], h[j], dn[i][j]);
        }
      }
      if (a.dres) row_of<E, Raw>(a.dres, row, a.dres_stride)[v] = V::narrow(l[i]);
      r1[i] = rsqrtf(sq[i] * inv_width + a.eps);
      uint64_t y[N], z[N], ws[N], dz[N], py = f2_both(0.f);
      V::widen(own_vec(place(stage, 0, v)), y);
      if (a.gate) V::widen(own_vec(place(stage, 1, v)), z);
      if (kPer > 1) scaled_weights(v, ws);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint64_t hat = f2_mul(y[j], f2_both(r1[i]));
        uint64_t g = f2_mul(l[i][j], kPer > 1 ? ws[j] : own_ws[j]), la = l[i][j];  // g: the gradient of y r silu(gate)
        if (a.gate) {
          const uint64_t sig = sigmoid_pair<E>(z[j]), act = f2_mul(z[j], sig), one = f2_both(1.f);
          const uint64_t slope = f2_mul(sig, f2_fma(z[j], f2_fma(sig, f2_both(-1.f), one), one));
          dz[j] = f2_mul(f2_mul(g, hat), slope);
          la = f2_mul(la, act);
          g = f2_mul(g, act);
        }
        q[i][j] = f2_fma(la, hat, q[i][j]);
        l[i][j] = g;
        py = f2_fma(g, y[j], py);
      }
      along[i] = f2_sum(py);
      coming[3] += along[i];
      if (a.dgate) row_of<E, Raw>(a.dgate, row, a.dgate_stride)[v] = V::narrow(dz);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
    if (row + gridDim.x < a.rows) first(next, coming, sq);
    join(coming);
    if (a.groups == 1) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) along[i] = coming[3];
    } else {
      group_sums(a, along, part, slot_along);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= a.vecs) continue;
      const float r = r1[i], c = along[i] * r * r * r * inv_width;
      uint64_t y[N];
      V::widen(own_vec(place(stage, 0, v)), y);
#pragma unroll
      for (int j = 0; j < N; ++j) l[i][j] = f2_fma(y[j], f2_both(-c), f2_mul(l[i][j], f2_both(r)));
      row_of<E, Raw>(a.dy, row, a.dy_stride)[v] = V::narrow(l[i]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[k] = coming[k];
    stage = next;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (a.parts == nullptr) return;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= a.vecs) continue;
    float* to = a.parts + static_cast<int64_t>(blockIdx.x) * a.dim + v * 2 * N;
    const int64_t next = static_cast<int64_t>(gridDim.x) * a.dim;
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      *reinterpret_cast<ulonglong2*>(to + 2 * j) = make_ulonglong2(q[i][j], q[i][j + 1]);
      *reinterpret_cast<ulonglong2*>(to + next + 2 * j) = make_ulonglong2(dn[i][j], dn[i][j + 1]);
    }
  }
}

template <class E>
__global__ void __launch_bounds__(kAnyThreads) norm_grad_any_kernel(Args a) {
  __shared__ float sums[kMaxGroups], along[kMaxGroups], slot[2][32];
  const int64_t next = static_cast<int64_t>(gridDim.x) * a.dim;
  float* to = a.parts ? a.parts + static_cast<int64_t>(blockIdx.x) * a.dim : nullptr;
  for (int e = threadIdx.x; to && e < a.dim; e += kAnyThreads) to[e] = to[next + e] = 0.f;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const auto* y = row_of<E>(a.y, row, a.y_stride);
    __syncthreads();  // the last row's sums are no longer read
    any_groups(a, sums, slot[0],
               [&](int g, int k) {
                 const float v = E::load(y + g * a.width + k);
                 return v * v;
               },
               [&](float s) { return rsqrtf(s / a.width + a.eps); });
    float r2 = 0.f, c2 = 0.f;
    if (a.dx) {
      float hh = 0.f, xh = 0.f;
      for (int e = threadIdx.x; e < a.dim; e += kAnyThreads) {
        const float h = E::load(row_of<E>(a.h, row, a.h_stride) + e);
        hh = fmaf(h, h, hh);
        xh = fmaf(E::load(row_of<E>(a.dx, row, a.dx_stride) + e) * (a.w_next ? a.w_next[e] : 1.f), h, xh);
      }
      hh = block_sum(hh, slot[0]);
      xh = block_sum(xh, slot[1]);
      __syncthreads();
      r2 = rsqrtf(hh / a.dim + a.eps);
      c2 = xh * r2 * r2 * r2 / a.dim;
    }
    // the gradient of h', and from it that of y r w
    auto at = [&](int e, float& l, float& p, float& sig, float& act, float& z) {
      l = a.dh ? E::load(row_of<E>(a.dh, row, a.dh_stride) + e) : 0.f;
      if (a.dx)
        l += E::load(row_of<E>(a.dx, row, a.dx_stride) + e) * (a.w_next ? a.w_next[e] : 1.f) * r2 -
             E::load(row_of<E>(a.h, row, a.h_stride) + e) * c2;
      z = a.gate ? E::load(row_of<E>(a.gate, row, a.gate_stride) + e) : 0.f;
      sig = a.gate ? sigmoid<E>(z) : 1.f;
      act = a.gate ? z * sig : 1.f;
      p = l * (a.scale ? a.scale[e] : 1.f);
    };
    any_groups(a, along, slot[0],
               [&](int g, int k) {
                 const int e = g * a.width + k;
                 float l, p, sig, act, z;
                 at(e, l, p, sig, act, z);
                 return p * act * (a.w ? a.w[k] : 1.f) * E::load(y + e);
               },
               [](float s) { return s; });
    for (int e = threadIdx.x; e < a.dim; e += kAnyThreads) {
      const int g = e / a.width;
      float l, p, sig, act, z;
      at(e, l, p, sig, act, z);
      const float r = sums[g], v = E::load(y + e), hat = v * r, w = a.w ? a.w[e - g * a.width] : 1.f;
      if (to) {
        to[e] = fmaf(l * act, hat, to[e]);
        if (a.dx)
          to[next + e] = fmaf(E::load(row_of<E>(a.dx, row, a.dx_stride) + e) * r2,
                              E::load(row_of<E>(a.h, row, a.h_stride) + e), to[next + e]);
      }
      if (a.dres) E::store(row_of<E>(a.dres, row, a.dres_stride) + e, l);
      if (a.dgate) E::store(row_of<E>(a.dgate, row, a.dgate_stride) + e, p * hat * w * sig * fmaf(z, 1.f - sig, 1.f));
      E::store(row_of<E>(a.dy, row, a.dy_stride) + e, p * act * w * r - v * (along[g] * r * r * r / a.width));
    }
  }
}

// The blocks' sums joined in order by a block's 1024 threads: kCols columns by 1024 / kCols
// threads each, four values on their way at a time, whose sums are then added.  32 columns,
// or for w of several groups, where the groups are added too, 8 (a sector of memory).  (304
// blocks' sums, dim 1280 in 10 groups: 6.2 us, with 32 columns everywhere 15.3; dim 5120 in
// one: 9.2, with 8 columns 25.7.)
constexpr int kJoinThreads = 1024;
template <int kCols>
__device__ __forceinline__ void join_columns(const Args& a, int blocks, int which, float* out, float* sum) {
  constexpr int kRows = kJoinThreads / kCols;
  const int cols = which == 0 ? a.width : a.dim, x = threadIdx.x % kCols, y = threadIdx.x / kCols, c = blockIdx.x * kCols + x;
  if (static_cast<int>(blockIdx.x) * kCols >= cols) return;
  // (a block's groups follow one another: place k is `cols` further than place k - 1)
  const float* from = a.parts + static_cast<int64_t>(which == 2 ? 1 : 0) * blocks * a.dim + c;
  const int per = a.dim / cols, n = blocks * per;
  const float* scale = which == 0 ? a.scale : nullptr;
  float s = 0.f;
  if (c < cols) {
    int k = y;
    for (; k + 3 * kRows < n; k += 4 * kRows) {
      float v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = from[static_cast<int64_t>(k + u * kRows) * cols];
      if (scale != nullptr) {
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] *= scale[(k + u * kRows) % per * cols + c];
      }
      s += (v[0] + v[1]) + (v[2] + v[3]);
    }
    for (; k < n; k += kRows) s += from[static_cast<int64_t>(k) * cols] * (scale != nullptr ? scale[k % per * cols + c] : 1.f);
  }
  sum[y * (kCols + 1) + x] = s;
  __syncthreads();
  if (y != 0 || c >= cols) return;
  s = 0.f;
#pragma unroll 32
  for (int k = 0; k < kRows; ++k) s += sum[k * (kCols + 1) + x];
  out[c] = which == 1 && a.w != nullptr ? s * a.w[c % a.width] : s;
}
__global__ void __launch_bounds__(kJoinThreads) norm_join_kernel(Args a, int blocks, float* dw, float* ds, float* dn) {
  __shared__ float sum[kJoinThreads / 8 * 9];
  float* out = blockIdx.y == 0 ? dw : blockIdx.y == 1 ? ds : dn;
  if (out == nullptr) return;
  if (blockIdx.y == 0 && a.groups > 1) join_columns<8>(a, blocks, 0, out, sum);
  else join_columns<32>(a, blocks, blockIdx.y, out, sum);
}

// -------------------------------------------------------------------- launch

// Pieces that a thread of a block of at most kThreads holds; 0: the row is too long.
int per_thread(int pieces, int most) {
  for (int per = 1; per <= most; per *= 2)
    if (pieces <= per * kThreads) return per;
  return 0;
}
constexpr int kSingles = 8;  // values a thread, where rows are not aligned: of 8192 at most

int opt_in(const void* kernel, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
  if (bit != 0 && (done.load(std::memory_order_relaxed) & bit)) return ENGRAM_OK;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmem);
  if (e != cudaSuccess) return fail(ENGRAM_E_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  done.fetch_or(bit, std::memory_order_relaxed);
  return ENGRAM_OK;
}

template <class E>
bool by_vectors(const Args& a) {
  auto ok = [](const void* p, int64_t stride) { return p == nullptr || (aligned(p, 16) && stride * E::kBytes % 16 == 0); };
  return a.width % Wide<E>::N == 0 && ok(a.y, a.y_stride) && ok(a.gate, a.gate_stride) && ok(a.h, a.h_stride) &&
         ok(a.dh, a.dh_stride) && ok(a.dx, a.dx_stride) && ok(a.h_out, a.h_out_stride) && ok(a.x_out, a.x_stride) &&
         ok(a.dy, a.dy_stride) && ok(a.dgate, a.dgate_stride) && ok(a.dres, a.dres_stride) && aligned(a.w, 16) &&
         aligned(a.scale, 16) && aligned(a.w_next, 16) && per_thread(a.dim / Wide<E>::N, 4) != 0;
}

template <class P>
void set_vecs(Args& a) {
  a.vecs = a.dim / P::N;
  const int per = a.vecs / a.groups;
  a.vecs_log2 = -1;
  for (int k = 0; k <= 5; ++k)
    if (per == 1 << k) a.vecs_log2 = k;
}

// Rows for each block from which on the blocks stay (see norm_ring_kernel).
constexpr int kManyRows = 8;
template <class E>
int launch_norm(Args a, int sms, cudaStream_t st) {
  const unsigned rows = static_cast<unsigned>(a.rows);
  const bool wide = by_vectors<E>(a);
  if (!wide && a.dim > kSingles * Single<E>::kMost) {
    norm_any_kernel<E><<<rows, kAnyThreads, 0, st>>>(a);
    return check_launch("norm_any_kernel");
  }
  if (wide) set_vecs<Wide<E>>(a);
  else set_vecs<Single<E>>(a);
  if (wide && a.groups == 1 && a.vecs <= kRingThreads) {
    const size_t ring = static_cast<size_t>(kAheadRows) * 3 * a.vecs * 16;
    const int threads = (a.vecs + 31) / 32 * 32, at_once = std::min(kRingThreads / threads, static_cast<int>(kRingSmem / ring));
    const int64_t blocks = static_cast<int64_t>(std::min(at_once, 8)) * sms;
    if (a.rows >= kManyRows * blocks) {
      static std::atomic<uint64_t> done{0};
      const int r = opt_in(reinterpret_cast<const void*>(norm_ring_kernel<E>), done);
      if (r) return r;
      norm_ring_kernel<E><<<static_cast<unsigned>(blocks), threads, ring, st>>>(a);
      return check_launch("norm_ring_kernel");
    }
  }
  const int per = wide ? per_thread(a.vecs, 4) : a.vecs <= 4 * kThreads ? 4 : kSingles;
  const int threads = ((a.vecs + per - 1) / per + 31) / 32 * 32;
  const size_t smem = a.groups > 1 && a.vecs_log2 < 0 ? sizeof(float) * (a.vecs + a.groups) : 0;
  if (!wide && per == 4) norm_kernel<Single<E>, 4><<<rows, threads, smem, st>>>(a);
  else if (!wide) norm_kernel<Single<E>, kSingles><<<rows, threads, smem, st>>>(a);
  else if (per == 1) norm_kernel<Wide<E>, 1><<<rows, threads, smem, st>>>(a);
  else if (per == 2) norm_kernel<Wide<E>, 2><<<rows, threads, smem, st>>>(a);
  else norm_kernel<Wide<E>, 4><<<rows, threads, smem, st>>>(a);
  return check_launch("norm_kernel");
}

// Blocks of a gradient's kernel that stay on an SM together: two where registers and shared
// memory leave room, else one.
int staying(const void* kernel, std::atomic<int>& registers, int threads, size_t smem, int* out) {
  int regs = registers.load(std::memory_order_relaxed);
  if (regs == 0) {
    cudaFuncAttributes at;
    cudaError_t e = cudaFuncGetAttributes(&at, kernel);
    if (e != cudaSuccess) return fail(ENGRAM_E_CUDA, "cudaFuncGetAttributes: %s", cudaGetErrorString(e));
    registers.store(regs = (at.numRegs + 7) / 8 * 8, std::memory_order_relaxed);
  }
  // (each of the SM's four parts has 16,384 registers for its warps)
  *out = (2 * (threads / 32) + 3) / 4 * 32 * regs <= 16384 && 2 * (smem + 10 * 1024) <= 228 * 1024 ? 2 : 1;
  return ENGRAM_OK;
}

template <class E>
int launch_grad(Args a, float* dw, float* ds, float* dn, int sms, cudaStream_t st) {
  int blocks = 0;
  // (16,384 rows, bf16: of 3600 in blocks of 480 threads and 96 registers 212 us with two for each SM,
  // one after the other, 207 with one; of 2560 in blocks of 320 threads 173 with one, 129 with two; of
  // 8192 without a ring, 512 threads and 64 registers, 1113 with one, 701 with two)
  auto go = [&](auto kernel, std::atomic<uint64_t>& done, std::atomic<int>& registers, int threads, size_t smem) {
    const void* fn = reinterpret_cast<const void*>(kernel);
    int at_once = 0, r = smem > 0 ? opt_in(fn, done) : ENGRAM_OK;
    if (r || (r = staying(fn, registers, threads, smem, &at_once))) return r;
    blocks = static_cast<int>(std::min<int64_t>(a.rows, std::min(kParts, at_once * sms)));
    kernel<<<blocks, threads, smem, st>>>(a);
    return check_launch("norm_grad_kernel");
  };
  const bool wide = by_vectors<E>(a);
  int rc;
  if (!wide && a.dim > kSingles * Single<E>::kMost) {
    static std::atomic<uint64_t> done{0};
    static std::atomic<int> registers{0};
    rc = go(norm_grad_any_kernel<E>, done, registers, kAnyThreads, 0);
  } else if (!wide) {
    static std::atomic<uint64_t> done[2] = {{0}, {0}};
    static std::atomic<int> registers[2] = {{0}, {0}};
    set_vecs<Single<E>>(a);
    const int per = a.vecs <= 4 * kThreads ? 4 : kSingles, threads = ((a.vecs + per - 1) / per + 31) / 32 * 32;
    const size_t smem = sizeof(float) * (2 * a.vecs + (a.groups > 1 && a.vecs_log2 < 0 ? a.vecs + a.groups : 0));
    rc = per == 4 ? go(norm_grad_kernel<Single<E>, 4, kThreads>, done[0], registers[0], threads, smem)
                  : go(norm_grad_kernel<Single<E>, kSingles, 1024>, done[1], registers[1], threads, smem);
  } else {
    static std::atomic<uint64_t> done[3] = {{0}, {0}, {0}};
    static std::atomic<int> registers[3] = {{0}, {0}, {0}};
    set_vecs<Wide<E>>(a);
    // two vectors a thread at most: the sums of four's columns would not fit the registers
    const int per = a.vecs <= kRingThreads ? 1 : 2, threads = ((a.vecs + per - 1) / per + 31) / 32 * 32;
    const size_t smem = a.groups > 1 && a.vecs_log2 < 0 ? static_cast<size_t>(a.vecs + a.groups + 3) / 4 * 16 : 0;
    const size_t ring = smem + static_cast<size_t>(kRing) * kArrays * a.vecs * 16;
    rc = ring > kRingSmem ? go(norm_grad_kernel<Wide<E>, 2, 2 * kThreads>, done[0], registers[0], threads, smem)
         : per == 1       ? go(norm_grad_ring_kernel<E, 1>, done[1], registers[1], threads, ring)
                          : go(norm_grad_ring_kernel<E, 2>, done[2], registers[2], threads, ring);
  }
  if (rc || a.parts == nullptr) return rc;
  const int across = std::max((a.dim + 31) / 32, a.groups > 1 ? (a.width + 7) / 8 : 0);
  norm_join_kernel<<<dim3(across, 3), kJoinThreads, 0, st>>>(a, blocks, dw, ds, dn);
  return check_launch("norm_join_kernel");
}

int check_sizes(int32_t type, int64_t n_rows, int32_t dim, int32_t groups, float eps) {
  if (!train::known_type(type)) return fail(ENGRAM_E_INVALID, "type %d is not ENGRAM_T_BF16 or ENGRAM_T_F32", type);
  if (n_rows < 0) return fail(ENGRAM_E_INVALID, "n_rows < 0");
  if (n_rows > 0x7fffffff) return fail(ENGRAM_E_RANGE, "n_rows must be below 2^31");
  if (dim < 1 || dim > 0x1000000) return fail(ENGRAM_E_SHAPE, "dim must be in [1, 2^24]");
  if (groups < 1 || groups > kMaxGroups || dim % groups != 0)
    return fail(ENGRAM_E_SHAPE, "groups must divide dim and be in [1, %d]", kMaxGroups);
  if (!(eps >= 0.f) || eps > 3.0e38f) return fail(ENGRAM_E_INVALID, "eps must be finite and not negative");
  return ENGRAM_OK;
}

int check_rows(const void* p, int32_t type, int64_t stride, int32_t dim, const char* name, bool needed) {
  if (p == nullptr) return needed ? fail(ENGRAM_E_INVALID, "null device pointer: %s", name) : ENGRAM_OK;
  if (stride < dim) return fail(ENGRAM_E_SHAPE, "%s: row stride below dim", name);
  if (!aligned(p, train::type_bytes(type))) return fail(ENGRAM_E_ALIGN, "%s must be aligned to its elements", name);
  return ENGRAM_OK;
}

int check_weights(const float* w, const float* scale, const float* w_next) {
  if (!aligned(w, 4) || !aligned(scale, 4) || !aligned(w_next, 4))
    return fail(ENGRAM_E_ALIGN, "w, scale and w_next must be aligned to their elements");
  return ENGRAM_OK;
}

}  // namespace
}  // namespace engram

using namespace engram;

extern "C" int engram_norm_add(const void* y_d, int64_t y_stride, const void* gate_d, int64_t gate_stride,
                               const void* h_d, int64_t h_stride, int32_t type, int64_t n_rows, int32_t dim,
                               int32_t groups, float eps, const float* w_d, const float* scale_d,
                               const float* w_next_d, void* h_out_d, int64_t h_out_stride, void* x_d,
                               int64_t x_stride, void* stream) {
  int rc = check_sizes(type, n_rows, dim, groups, eps);
  if (rc) return rc;
  if (n_rows == 0) return ENGRAM_OK;
  if ((rc = check_rows(y_d, type, y_stride, dim, "y", true))) return rc;
  if ((rc = check_rows(gate_d, type, gate_stride, dim, "gate", false))) return rc;
  if ((rc = check_rows(h_d, type, h_stride, dim, "h", false))) return rc;
  if ((rc = check_rows(h_out_d, type, h_out_stride, dim, "h_out", true))) return rc;
  if ((rc = check_rows(x_d, type, x_stride, dim, "x", false))) return rc;
  if ((rc = check_weights(w_d, scale_d, w_next_d))) return rc;
  if (h_out_d == h_d && h_out_stride != h_stride) return fail(ENGRAM_E_SHAPE, "in place, h_out has the stride of h");
  int sms = 0;
  if ((rc = check_device(&sms))) return rc;
  Args a{};
  a.y = y_d;
  a.gate = gate_d;
  a.h = h_d;
  a.h_out = h_out_d;
  a.x_out = x_d;
  a.y_stride = y_stride;
  a.gate_stride = gate_stride;
  a.h_stride = h_stride;
  a.h_out_stride = h_out_stride;
  a.x_stride = x_stride;
  a.w = w_d;
  a.scale = scale_d;
  a.w_next = w_next_d;
  a.rows = n_rows;
  a.dim = dim;
  a.groups = groups;
  a.width = dim / groups;
  a.eps = eps;
  return type == ENGRAM_T_BF16 ? launch_norm<train::Bf16>(a, sms, as_stream(stream))
                               : launch_norm<train::F32>(a, sms, as_stream(stream));
}

extern "C" size_t engram_norm_add_workspace_bytes(int64_t n_rows, int32_t dim) {
  if (n_rows < 0 || dim < 1) return 0;
  return sizeof(float) * 2 * static_cast<size_t>(std::min<int64_t>(n_rows, kParts)) * dim;
}

extern "C" int engram_norm_add_grad(const void* dh_d, int64_t dh_stride, const void* dx_d, int64_t dx_stride,
                                    const void* y_d, int64_t y_stride, const void* gate_d, int64_t gate_stride,
                                    const void* h_out_d, int64_t h_out_stride, int32_t type, int64_t n_rows,
                                    int32_t dim, int32_t groups, float eps, const float* w_d, const float* scale_d,
                                    const float* w_next_d, void* dy_d, int64_t dy_stride, void* dgate_d,
                                    int64_t dgate_stride, void* dres_d, int64_t dres_stride, float* dw_d,
                                    float* dscale_d, float* dw_next_d, void* workspace_d, size_t workspace_bytes,
                                    void* stream) {
  int rc = check_sizes(type, n_rows, dim, groups, eps);
  if (rc) return rc;
  const bool sums = dw_d || dscale_d || dw_next_d;
  if (n_rows > 0) {
    if (!dh_d && !dx_d) return fail(ENGRAM_E_INVALID, "neither dh nor dx");
    if ((rc = check_rows(dh_d, type, dh_stride, dim, "dh", false))) return rc;
    if ((rc = check_rows(dx_d, type, dx_stride, dim, "dx", false))) return rc;
    if ((rc = check_rows(y_d, type, y_stride, dim, "y", true))) return rc;
    if ((rc = check_rows(gate_d, type, gate_stride, dim, "gate", dgate_d != nullptr))) return rc;
    if ((rc = check_rows(h_out_d, type, h_out_stride, dim, "h_out", dx_d != nullptr))) return rc;
    if ((rc = check_rows(dy_d, type, dy_stride, dim, "dy", true))) return rc;
    if ((rc = check_rows(dgate_d, type, dgate_stride, dim, "dgate", false))) return rc;
    if ((rc = check_rows(dres_d, type, dres_stride, dim, "dres", false))) return rc;
    if (dres_d == dh_d && dres_d && dres_stride != dh_stride)
      return fail(ENGRAM_E_SHAPE, "in place, dres has the stride of dh");
    if (sums) {
      if (!workspace_d) return fail(ENGRAM_E_INVALID, "null device pointer: workspace");
      if (!aligned(workspace_d, 256)) return fail(ENGRAM_E_ALIGN, "workspace must be 256-byte aligned");
      if (workspace_bytes < engram_norm_add_workspace_bytes(n_rows, dim))
        return fail(ENGRAM_E_RANGE, "workspace too small");
    }
  }
  if ((rc = check_weights(w_d, scale_d, w_next_d))) return rc;
  if ((rc = check_weights(dw_d, dscale_d, dw_next_d))) return rc;
  if (n_rows == 0 && !sums) return ENGRAM_OK;
  int sms = 0;
  if ((rc = check_device(&sms))) return rc;
  Args a{};
  a.y = y_d;
  a.gate = gate_d;
  a.h = dx_d ? h_out_d : nullptr;
  a.dh = dh_d;
  a.dx = dx_d;
  a.dy = dy_d;
  a.dgate = dgate_d;
  a.dres = dres_d;
  a.y_stride = y_stride;
  a.gate_stride = gate_stride;
  a.h_stride = h_out_stride;
  a.dh_stride = dh_stride;
  a.dx_stride = dx_stride;
  a.dy_stride = dy_stride;
  a.dgate_stride = dgate_stride;
  a.dres_stride = dres_stride;
  a.w = w_d;
  a.scale = scale_d;
  a.w_next = w_next_d;
  a.parts = sums ? static_cast<float*>(workspace_d) : nullptr;
  a.rows = n_rows;
  a.dim = dim;
  a.groups = groups;
  a.width = dim / groups;
  a.eps = eps;
  if (n_rows == 0) {  // sums of nothing
    float* const out[3] = {dw_d, dscale_d, dw_next_d};
    for (int k = 0; k < 3; ++k)
      if (out[k] && cudaMemsetAsync(out[k], 0, sizeof(float) * (k == 0 ? a.width : dim), as_stream(stream)) != cudaSuccess)
        return check_launch("cudaMemsetAsync");
    return ENGRAM_OK;
  }
  return type == ENGRAM_T_BF16 ? launch_grad<train::Bf16>(a, dw_d, dscale_d, dw_next_d, sms, as_stream(stream))
                               : launch_grad<train::F32>(a, dw_d, dscale_d, dw_next_d, sms, as_stream(stream));
}
