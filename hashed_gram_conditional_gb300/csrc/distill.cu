// Distillation from a teacher's top logits: the loss of every position and
// the gradient of the student's logits.
//
// With q = softmax(z / tau) over the vocabulary, p the teacher's
// probabilities at its K entries and P their sum:
//   loss = w tau^2 sum_k p_k (ln p_k - ln q_k)
//   dz_v = w tau (P q_v - p_v)
//
// A position's gradient needs its whole row's maximum and sum, so a row is
// read once and kept: a cluster of 1 to 8 blocks holds it in shared memory
// (bulk copies), exchanges its blocks' (maximum, sum) pairs through
// distributed shared memory, and writes the gradient from the copy.  Memory
// traffic is then the logits once and the gradient once.  Rows are split so
// that a block's part is at most 72 KB where that is possible: three blocks
// share an SM, so that one loads while another exchanges or writes.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "engram_internal.h"
#include "train_device.cuh"

namespace engram {
namespace {

constexpr int kWarps = 8;               // that go over the row
constexpr int kData = kWarps * 32;
constexpr int kThreads = kData + 32;    // and one that prepares the teacher's probabilities meanwhile
constexpr int kMaxTop = ENGRAM_DISTILL_MAX_TOP;
constexpr int kMaxCluster = 8;
constexpr int kChunks = 4;                 // pieces of a part that are awaited one by one
constexpr int kPartBytes = 72 * 1024;      // a part's size where the cluster can be made large enough
constexpr int kPartLimit = 200 * 1024;     // beyond this in a cluster of 8 the row is read twice instead

struct Args {
  int64_t vocab, z_stride, dz_stride;
  const int32_t* ids;
  const float* t;
  int32_t top, cluster;
  float tau;
  const float* lse;
  const float* weight;
  float* loss;
  int32_t* status;
};

struct Head {  // in front of the dynamic shared memory
  uint64_t bar[kChunks];
  uint64_t met;              // completes when every block's pair is here
  float2 part[kMaxCluster];  // the blocks' (maximum, sum of exponentials relative to it)
  float2 warp[kWarps];
  float norm, mass;          // of the teacher's entries
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <bool kMax>
__device__ __forceinline__ float warp_reduce(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? fmaxf(v, w) : v + w;
  }
  return v;
}

// 16 bytes of a row: 8 bf16 or 4 fp32 values.
template <class E>
constexpr int kVec = 16 / E::kBytes;

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <class E>
__device__ __forceinline__ void widen(const uint4& x, float (&f)[kVec<E>]) {
  if constexpr (E::kBytes == 2) {
    f[0] = lo16(x.x); f[1] = hi16(x.x); f[2] = lo16(x.y); f[3] = hi16(x.y);
    f[4] = lo16(x.z); f[5] = hi16(x.z); f[6] = lo16(x.w); f[7] = hi16(x.w);
  } else {
    f[0] = __uint_as_float(x.x); f[1] = __uint_as_float(x.y);
    f[2] = __uint_as_float(x.z); f[3] = __uint_as_float(x.w);
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

template <class E>
__device__ __forceinline__ uint4 narrow(const float (&f)[kVec<E>]) {
  if constexpr (E::kBytes == 2)
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
  else
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// The largest of a vector's values, NaN passed over.
template <class E>
__device__ __forceinline__ float largest(const uint4& x) {
  if constexpr (E::kBytes == 2) {
    auto as = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    const __nv_bfloat162 b = __hmax2(__hmax2(as(x.x), as(x.y)), __hmax2(as(x.z), as(x.w)));
    return fmaxf(__low2float(b), __high2float(b));
  } else {
    return fmaxf(fmaxf(__uint_as_float(x.x), __uint_as_float(x.y)), fmaxf(__uint_as_float(x.z), __uint_as_float(x.w)));
  }
}

// (m, s) <- the pair of both: sums of 2^((z - m) c), -inf maxima count nothing.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2, float c) {
  const float top = fmaxf(m, m2), at = top == -INFINITY ? 0.f : top;
  s = s * ex2((m - at) * c) + s2 * ex2((m2 - at) * c);
  m = top;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// One cluster of a.cluster blocks per position.  The row is handled in 16-byte
// vectors counted from the aligned address at or before its first element
// (`off` elements before it); vectors that reach over the row's ends are
// filled up with -inf, which adds nothing to the sums.
template <class E, bool kResident>
__global__ void __launch_bounds__(kThreads, 3) distill_kernel(const typename E::T* z,
                                                                              typename E::T* dz, Args a) {
  constexpr int N = kVec<E>;
  extern __shared__ __align__(128) unsigned char smem[];
  Head& h = *reinterpret_cast<Head*>(smem);
  float* p = reinterpret_cast<float*>(smem + sizeof(Head));
  int32_t* id = reinterpret_cast<int32_t*>(p + a.top);
  float* zk = reinterpret_cast<float*>(id + a.top);
  uint4* row_s = reinterpret_cast<uint4*>(smem + ((sizeof(Head) + 12 * static_cast<size_t>(a.top) + 127) & ~size_t(127)));

  const int tid = threadIdx.x;
  const uint32_t rank = a.cluster > 1 ? cluster_rank() : 0u;
  const int64_t row = blockIdx.x / a.cluster;
  const typename E::T* zr = z + row * a.z_stride;
  typename E::T* dr = dz + row * a.dz_stride;
  const int V = static_cast<int>(a.vocab);
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(zr) & 15) / E::kBytes);
  const int doff = static_cast<int>((reinterpret_cast<uintptr_t>(dr) & 15) / E::kBytes);
  const int vecs = (V + off + N - 1) / N, per = (vecs + a.cluster - 1) / a.cluster;
  const int v0 = static_cast<int>(rank) * per < vecs ? static_cast<int>(rank) * per : vecs;
  const int v1 = v0 + per < vecs ? v0 + per : vecs;
  const uint4* zv = reinterpret_cast<const uint4*>(zr - off);
  // vectors wholly inside the row
  const int in0 = off > 0 ? 1 : 0, in1 = (V + off) / N;
  // the vector that reaches over the row's end is in this block's part
  const bool tail = in1 < vecs && v0 <= in1 && in1 < v1 && !(in1 == 0 && in0 > 0);

  const float w = a.weight != nullptr ? a.weight[row] : 1.f;
  auto zeros = [&]() {  // this block's part of a gradient of zeros
    if (dz == nullptr) return;
    const int e0 = v0 * N - off > 0 ? v0 * N - off : 0, e1 = v1 * N - off < V ? v1 * N - off : V;
    if (off == doff) {
      for (int v = (v0 > in0 ? v0 : in0) + tid; v < v1 && v < in1; v += kThreads)
        reinterpret_cast<uint4*>(dr - off)[v] = make_uint4(0u, 0u, 0u, 0u);
      if (in0 > 0 && v0 == 0 && tid < N - off && tid < V) E::store(dr + tid, 0.f);
      if (tail && in1 * N - off + tid < V) E::store(dr + in1 * N - off + tid, 0.f);
    } else {
      for (int e = e0 + tid; e < e1; e += kThreads) E::store(dr + e, 0.f);
    }
  };
  if (w == 0.f) {  // nothing to learn here
    if (rank == 0 && tid == 0) a.loss[row] = 0.f;
    zeros();
    return;
  }

  // the row's values of a vector, -inf outside
  auto edge = [&](int v) {
    float f[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = v * N + j - off;
      f[j] = e >= 0 && e < V ? E::load(zr + e) : -INFINITY;
    }
    return narrow<E>(f);
  };
  // whole rounds of the threads
  const int chunk = ((v1 - v0 + kChunks - 1) / kChunks + kData - 1) / kData * kData;
  if (tid == 0) {
#pragma unroll
    for (int k = 0; k < kChunks; ++k) mbar_init(smem_u32(&h.bar[k]), 1);
    mbar_init(smem_u32(&h.met), 1);
    fence_mbar_init();
    if (a.cluster > 1) mbar_arrive_expect_tx(smem_u32(&h.met), static_cast<uint32_t>(a.cluster) * sizeof(float2));
    if (kResident) {
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        int b0 = v0 + k * chunk, b1 = b0 + chunk < v1 ? b0 + chunk : v1;
        b0 = b0 > in0 ? b0 : in0;
        b1 = b1 < in1 ? b1 : in1;
        const uint32_t bytes = b1 > b0 ? static_cast<uint32_t>(b1 - b0) * 16u : 0u;
        mbar_arrive_expect_tx(smem_u32(&h.bar[k]), bytes);
        if (bytes > 0) bulk_g2s(smem_u32(row_s + (b0 - v0)), zv + b0, bytes, smem_u32(&h.bar[k]));
      }
    }
  }
  if (kResident) {
    if (tid == 32 && in0 > 0 && v0 == 0 && v1 > 0) row_s[0] = edge(0);
    if (tid == 64 && tail) row_s[in1 - v0] = edge(in1);
  }
  __syncthreads();
  if (a.cluster > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

  constexpr int kAhead = 4;
  const float inv_tau = 1.f / a.tau, c = 1.4426950408889634f * inv_tau;
  const int lane = tid & 31, warp = tid >> 5;
  bool late = false;
  if (warp == kWarps) {
    // the teacher's entries: id, logit / tau and the student's logit
    float top = -INFINITY;
    for (int k = lane; k < a.top; k += 32) {
      int32_t v = a.ids[row * a.top + k];
      if (v >= a.vocab) {
        if (a.status != nullptr) atomicOr(a.status, ENGRAM_ST_BAD_TOKEN);
        v = -1;
      }
      id[k] = v < 0 ? -1 : v;
      p[k] = v >= 0 ? a.t[row * a.top + k] * inv_tau : -INFINITY;
      zk[k] = v >= 0 ? E::load(zr + v) : 0.f;
      top = fmaxf(top, p[k]);
    }
    top = warp_reduce<true>(top);
    float norm = 0.f;
    if (a.lse != nullptr) {
      norm = a.lse[row];
    } else if (top != -INFINITY) {
      float sum = 0.f;
      for (int k = lane; k < a.top; k += 32) sum += expf(p[k] - top);
      norm = top + logf(warp_reduce<false>(sum));
    }
    float mass = 0.f;
    for (int k = lane; k < a.top; k += 32) mass += expf(p[k] - norm);
    mass = warp_reduce<false>(mass);
    if (lane == 0) {
      h.norm = norm;
      h.mass = mass;
    }
  } else {
    // the maximum and the sum of this block's part, kAhead vectors a step: their
    // maximum first, so that the exponentials do not wait for one another
    float m = -INFINITY, s = 0.f;
    auto add = [&](const uint4 (&x)[kAhead]) {
      const float big = fmaxf(fmaxf(largest<E>(x[0]), largest<E>(x[1])), fmaxf(largest<E>(x[2]), largest<E>(x[3])));
      const float top = fmaxf(m, big), at = top == -INFINITY ? 0.f : -top;
      s *= ex2((m + at) * c);
      m = top;
      uint64_t sum = f2(0.f, 0.f);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        float f[N];
        widen<E>(x[u], f);
#pragma unroll
        for (int j = 0; j < N; j += 2) {
          float x0, x1;
          f2_split(f2_mul(f2_add(f2(f[j], f[j + 1]), f2(at, at)), f2(c, c)), x0, x1);
          sum = f2_add(sum, f2(ex2(x0), ex2(x1)));
        }
      }
      float s0, s1;
      f2_split(sum, s0, s1);
      s += s0 + s1;
    };
    const uint32_t low = E::kBytes == 2 ? 0xff80ff80u : 0xff800000u;  // -inf
    const uint4 nothing = make_uint4(low, low, low, low);
    if (kResident) {
#pragma unroll 1
      for (int k = 0; k < kChunks; ++k) {
        if (!mbar_wait_bounded(smem_u32(&h.bar[k]), 0, nullptr)) {
          late = true;  // give the copy one more chance to land before the block goes on
          mbar_wait_bounded(smem_u32(&h.bar[k]), 0, nullptr);
        }
        const int b0 = k * chunk, b1 = b0 + chunk < v1 - v0 ? b0 + chunk : v1 - v0;
        for (int v = b0 + tid; v < b1; v += kAhead * kData) {
          uint4 x[kAhead];
#pragma unroll
          for (int u = 0; u < kAhead; ++u) x[u] = v + u * kData < b1 ? row_s[v + u * kData] : nothing;
          add(x);
        }
      }
    } else {
      for (int v = v0 + tid; v < v1; v += kAhead * kData) {
        uint4 x[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int vu = v + u * kData;
          x[u] = vu >= v1 ? nothing : vu >= in0 && vu < in1 ? zv[vu] : edge(vu);
        }
        add(x);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      // both lanes of a pair join in the same order, so that they agree
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
      const bool first = (tid & o) == 0;
      float ma = first ? m : m2, sa = first ? s : s2;
      join(ma, sa, first ? m2 : m, first ? s2 : s, c);
      m = ma;
      s = sa;
    }
    if (lane == 0) h.warp[warp] = make_float2(m, s);
  }
  if (late && a.status != nullptr) atomicOr(a.status, ENGRAM_ST_TIMEOUT);
  __syncthreads();
  float m = h.warp[0].x, s = h.warp[0].y;
#pragma unroll
  for (int k = 1; k < kWarps; ++k) join(m, s, h.warp[k].x, h.warp[k].y, c);
  if (a.cluster > 1) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every block's barriers are set up
    if (tid < a.cluster) {
      uint32_t to, bar;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(&h.part[rank])), "r"(tid));
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(smem_u32(&h.met)), "r"(tid));
      asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(to), "f"(m),
                   "f"(s), "r"(bar)
                   : "memory");
    }
    __syncwarp();
    // (bounded; the pairs are read by this block alone once all are here, so
    // that no block needs another one after this)
    if (!mbar_wait_bounded(smem_u32(&h.met), 0, nullptr) && tid == 0 && a.status != nullptr)
      atomicOr(a.status, ENGRAM_ST_TIMEOUT);
    m = h.part[0].x;
    s = h.part[0].y;
    for (int k = 1; k < a.cluster; ++k) join(m, s, h.part[k].x, h.part[k].y, c);
  }

  const float mass = h.mass;
  const bool none = mass == 0.f;
  if (rank == 0 && warp == kWarps) {
    const float norm = h.norm, log_sum = logf(s);
    float loss = 0.f;
    for (int k = lane; k < a.top; k += 32) {
      const float pk = expf(p[k] - norm);
      if (pk > 0.f || pk != pk) loss += pk * ((p[k] - norm) - ((zk[k] - m) * inv_tau - log_sum));
    }
    loss = warp_reduce<false>(loss);
    if (lane == 0) a.loss[row] = none ? 0.f : w * a.tau * a.tau * loss;
  }
  if (dz == nullptr) return;
  if (none) {
    zeros();
    return;
  }

  const float scale = w * a.tau, coef = scale * mass / s;
  auto grad = [&](const uint4& x, float (&f)[N]) {
    widen<E>(x, f);
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      float x0, x1;
      f2_split(f2_mul(f2_add(f2(f[j], f[j + 1]), f2(-m, -m)), f2(c, c)), x0, x1);
      f2_split(f2_mul(f2(ex2(x0), ex2(x1)), f2(coef, coef)), f[j], f[j + 1]);
    }
  };
  auto grad_edge = [&](int v) {
    float f[N];
    grad(kResident ? row_s[v - v0] : edge(v), f);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = v * N + j - off;
      if (e >= 0 && e < V) E::store(dr + e, f[j]);
    }
  };
  if (warp == kWarps) {
    // (the row is the other warps')
  } else if (off == doff) {
    const uint4* src = kResident ? row_s - v0 : zv;
    uint4* dv = reinterpret_cast<uint4*>(dr - off);
    const int end = v1 < in1 ? v1 : in1;
    int v = (v0 > in0 ? v0 : in0) + tid;
    for (; v + (kAhead - 1) * kData < end; v += kAhead * kData) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        float f[N];
        grad(src[v + u * kData], f);
        __stcs(dv + v + u * kData, narrow<E>(f));
      }
    }
    for (; v < end; v += kData) {
      float f[N];
      grad(src[v], f);
      __stcs(dv + v, narrow<E>(f));
    }
    if (tid == 32 && in0 > 0 && v0 == 0 && v1 > 0) grad_edge(0);
    if (tid == 64 && tail) grad_edge(in1);
  } else {  // the gradient's rows lie differently: value by value
    const int e0 = v0 * N - off > 0 ? v0 * N - off : 0, e1 = v1 * N - off < V ? v1 * N - off : V;
    const typename E::T* part = kResident ? reinterpret_cast<const typename E::T*>(row_s) + off - v0 * N : zr;
    for (int e = e0 + tid; e < e1; e += kData) E::store(dr + e, ex2((E::load(part + e) - m) * c) * coef);
  }
  // the entries' own gradients, over what was just written
  __syncthreads();
  const float norm = h.norm;
  for (int k = tid; k < a.top; k += kThreads) {
    const int mine = id[k], v = mine < 0 ? -1 : (mine + off) / N;
    if (v < v0 || v >= v1) continue;
    float pk = 0.f;
#pragma unroll 4
    for (int i = 0; i < a.top; ++i)
      if (id[i] == mine) pk += expf(p[i] - norm);  // an id given twice adds up
    E::store(dr + mine, ex2((zk[k] - m) * c) * coef - scale * pk);
  }
}

template <class E, bool kResident>
int launch(const void* z, void* dz, const Args& a, int64_t rows, size_t smem, cudaStream_t st) {
  static std::atomic<uint64_t> attr_set{0};  // one bit per device: the shared-memory opt-in was made
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
  if (bit == 0 || !(attr_set.load(std::memory_order_relaxed) & bit)) {
    cudaError_t e = cudaFuncSetAttribute(distill_kernel<E, kResident>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kPartLimit + 16 * 1024);
    if (e != cudaSuccess) return fail(ENGRAM_E_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    attr_set.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * a.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(a.cluster);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, distill_kernel<E, kResident>, static_cast<const typename E::T*>(z),
                                     static_cast<typename E::T*>(dz), a);
  if (e != cudaSuccess) return fail(ENGRAM_E_CUDA, "distill_kernel launch: %s", cudaGetErrorString(e));
  return check_launch("distill_kernel");
}

template <class E>
int launch_distill(const void* z, void* dz, Args a, int64_t rows, cudaStream_t st) {
  const int64_t bytes = a.vocab * E::kBytes + 16;  // with a misaligned row's first vector
  a.cluster = 1;
  while (a.cluster < kMaxCluster && bytes / a.cluster > kPartBytes) a.cluster *= 2;
  const int64_t vecs = (bytes + 15) / 16, per = (vecs + a.cluster - 1) / a.cluster;
  const size_t head = (sizeof(Head) + 12 * static_cast<size_t>(a.top) + 127) & ~size_t(127);
  if (per * 16 <= kPartLimit) return launch<E, true>(z, dz, a, rows, head + static_cast<size_t>(per) * 16, st);
  return launch<E, false>(z, dz, a, rows, head, st);
}

}  // namespace
}  // namespace engram

using namespace engram;

extern "C" int engram_distill(const void* logits_d, int32_t type, int64_t n_tokens, int64_t vocab,
                              int64_t logits_stride, const int32_t* teacher_ids_d, const float* teacher_logits_d,
                              int32_t top, float temperature, const float* teacher_lse_d, const float* weight_d,
                              float* loss_d, void* dlogits_d, int64_t dlogits_stride, int32_t* status_d,
                              void* stream) {
  if (!train::known_type(type)) return fail(ENGRAM_E_INVALID, "type %d is not ENGRAM_T_BF16 or ENGRAM_T_F32", type);
  if (n_tokens < 0) return fail(ENGRAM_E_INVALID, "n_tokens < 0");
  if (n_tokens > 0x7fffffff / kMaxCluster) return fail(ENGRAM_E_RANGE, "n_tokens must be below 2^28");
  if (vocab < 1 || vocab > 0x7fffff00) return fail(ENGRAM_E_SHAPE, "vocab must be in [1, 2^31 - 256]");
  if (top < 0 || top > kMaxTop) return fail(ENGRAM_E_SHAPE, "top %d not in [0, %d]", top, kMaxTop);
  if (!(temperature > 0.f) || temperature > 3.0e38f) return fail(ENGRAM_E_INVALID, "temperature must be positive and finite");
  if (logits_stride < vocab || (dlogits_d && dlogits_stride < vocab))
    return fail(ENGRAM_E_SHAPE, "row stride below vocab");
  if (n_tokens == 0) return ENGRAM_OK;
  if (!logits_d || !loss_d || (top > 0 && (!teacher_ids_d || !teacher_logits_d)))
    return fail(ENGRAM_E_INVALID, "null device pointer");
  if (!aligned(logits_d, train::type_bytes(type)) || !aligned(dlogits_d, train::type_bytes(type)))
    return fail(ENGRAM_E_ALIGN, "logits and dlogits must be aligned to their elements");
  if (dlogits_d == logits_d && dlogits_stride != logits_stride)
    return fail(ENGRAM_E_SHAPE, "in place, dlogits has the stride of logits");
  int rc = check_device(nullptr);
  if (rc) return rc;
  Args a{vocab, logits_stride, dlogits_stride, teacher_ids_d, teacher_logits_d, top, 1, temperature, teacher_lse_d,
         weight_d, loss_d, status_d};
  return type == ENGRAM_T_BF16 ? launch_distill<train::Bf16>(logits_d, dlogits_d, a, n_tokens, as_stream(stream))
                               : launch_distill<train::F32>(logits_d, dlogits_d, a, n_tokens, as_stream(stream));
}
