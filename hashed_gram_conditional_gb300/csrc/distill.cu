// Distillation from a teacher's top logits: the loss of every position and
// the gradient of the student's logits.
//
// With q = softmax(z / tau) over the vocabulary, p the teacher's
// probabilities at its K entries and P their sum:
//   loss = w tau^2 sum_k p_k (ln p_k - ln q_k)
//   dz_v = w tau (P q_v - p_v)
//
// A position's gradient needs its whole row's maximum and sum, so a row is
// read once and kept: the blocks of a cluster hold its parts in shared memory,
// exchange their (maximum, sum) pairs through distributed shared memory, and
// write the gradient from there.  Memory traffic is then the logits once and
// the gradient once.  The blocks stay and go from row to row, with the copies
// of the next rows under way (rows_kernel); rows too long for a cluster's
// shared memory are read twice (long_rows_kernel), and short ones are a warp's
// work (short_rows_kernel).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "engram_internal.h"
#include "train_device.cuh"

namespace engram {
namespace {

constexpr int kMaxTop = ENGRAM_DISTILL_MAX_TOP;
constexpr int kMaxCluster = 8;

struct Args {
  int64_t vocab, z_stride, dz_stride;
  int32_t rows;
  const int32_t* ids;
  const float* t;
  int32_t top, cluster, depth, keep, slot_bytes;
  int32_t cluster_log2, table_log2;
  bool aligned;  // the rows' strides are multiples of 16 bytes
  uint32_t absent;  // bytes that every row's pairs are expected to have beyond theirs (0; see engram_selftest_distill_wait)
  float tau;
  const float* lse;
  const float* weight;
  float* loss;
  int32_t* status;
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 2^x of two values, by the hardware's exponential for either type: results below
// 2^-126 are zero.  (In an earlier form of the walks a quarter of the pairs through
// the FMA units, by a sixth-order series, took 498 us against 418 at 4096 x 129,280
// bf16: they are bound by instructions issued, not by the exponentials.)
__device__ __forceinline__ uint64_t ex2_pair(uint64_t x) {
  float x0, x1;
  f2_split(x, x0, x1);
  return f2(ex2(x0), ex2(x1));
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

// A row in 16-byte vectors counted from the aligned address at or before its
// first element (`off` elements before it).  Vectors that reach over the row's
// ends are filled up with -inf, which adds nothing to the sums.
template <class E>
struct Row {
  static constexpr int N = kVec<E>;
  const typename E::T* z;
  typename E::T* dz;
  int V, off, doff;  // doff: the same of the gradient's row
  int in0, in1;      // vectors wholly inside the row
  int v0, v1;        // this block's part
  bool head, tail;   // it has the vector over the row's beginning, over its end

  // The row's place; its geometry is the same for every row if their strides
  // are multiples of 16 bytes (`aligned`), and is then worked out once.
  __device__ __forceinline__ void at(const typename E::T* z_all, typename E::T* dz_all, const Args& a, int64_t row, int rank,
                                     bool again) {
    z = z_all + row * a.z_stride;
    dz = dz_all + row * a.dz_stride;
    if (again && a.aligned) return;
    V = static_cast<int>(a.vocab);
    off = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15) / E::kBytes);
    doff = static_cast<int>((reinterpret_cast<uintptr_t>(dz) & 15) / E::kBytes);
    const int vecs = (V + off + N - 1) / N, per = (vecs + a.cluster - 1) >> a.cluster_log2;
    v0 = rank * per < vecs ? rank * per : vecs;
    v1 = v0 + per < vecs ? v0 + per : vecs;
    in0 = off > 0 ? 1 : 0;
    in1 = (V + off) / N;
    head = in0 > 0 && v0 == 0 && v1 > 0;
    tail = in1 < vecs && v0 <= in1 && in1 < v1 && !(in1 == 0 && in0 > 0);
  }
  __device__ __forceinline__ const uint4* vectors() const { return reinterpret_cast<const uint4*>(z - off); }
  __device__ __forceinline__ int first() const { return v0 > in0 ? v0 : in0; }  // of the part's whole vectors
  __device__ __forceinline__ int end() const { return v1 < in1 ? v1 : in1; }
  __device__ __forceinline__ uint4 edge(int v) const {
    float f[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = v * N + j - off;
      f[j] = e >= 0 && e < V ? E::load(z + e) : -INFINITY;
    }
    return narrow<E>(f);
  }
  // The element of the part's edge vectors that a lane stands for, or -1: lanes
  // 0 .. N - 1 the head's, N .. 2 N - 1 the tail's.
  __device__ __forceinline__ int edge_element(int lane) const {
    const bool mine = lane < N ? head : lane < 2 * N && tail;
    const int e = (lane < N ? 0 : in1) * N + lane % N - off;
    return mine && e >= 0 && e < V ? e : -1;
  }
  __device__ __forceinline__ void store_edge(int v, const float (&f)[N]) const {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = v * N + j - off;
      if (e >= 0 && e < V) E::store(dz + e, f[j]);
    }
  }
  // this block's part of a gradient of zeros, by `threads` threads
  __device__ __forceinline__ void zeros(int tid, int threads) const {
    if (off == doff) {
      for (int v = first() + tid; v < end(); v += threads)
        reinterpret_cast<uint4*>(dz - off)[v] = make_uint4(0u, 0u, 0u, 0u);
      const float none[N] = {};
      if (head && tid == 0) store_edge(0, none);
      if (tail && tid == 0) store_edge(in1, none);
    } else {
      const int e1 = v1 * N - off < V ? v1 * N - off : V;
      for (int e = (v0 * N - off > 0 ? v0 * N - off : 0) + tid; e < e1; e += threads) E::store(dz + e, 0.f);
    }
  }
};

// Adds kAhead vectors to (m, s): their maximum first, so that the exponentials
// do not wait for one another.
constexpr int kAhead = 4;
template <class E>
__device__ __forceinline__ void add_vectors(const uint4 (&x)[kAhead], float c, float& m, float& s) {
  constexpr int N = kVec<E>;
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
      const uint64_t x = f2_mul(f2_add(f2(f[j], f[j + 1]), f2(at, at)), f2(c, c));
      sum = f2_add(sum, ex2_pair(x));
    }
  }
  float s0, s1;
  f2_split(sum, s0, s1);
  s += s0 + s1;
}

template <class E>
__device__ __forceinline__ uint4 no_vector() {
  const uint32_t low = E::kBytes == 2 ? 0xff80ff80u : 0xff800000u;  // -inf
  return make_uint4(low, low, low, low);
}

// The warp's pairs joined: the largest maximum, then one rescaled sum a lane,
// added up in the same order in every lane's view.
__device__ __forceinline__ void join_warp(float& m, float& s, float c) {
  float top;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(top) : "f"(m));
  const float at = top == -INFINITY ? 0.f : top;
  s *= ex2((m - at) * c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  m = top;
}

// coef 2^((z - m) c) of a vector
template <class E>
__device__ __forceinline__ void grad_vector(const uint4& x, float m, float c, float coef, float (&f)[kVec<E>]) {
  widen<E>(x, f);
#pragma unroll
  for (int j = 0; j < kVec<E>; j += 2) {
    const uint64_t e = f2_mul(f2_add(f2(f[j], f[j + 1]), f2(-m, -m)), f2(c, c));
    f2_split(f2_mul(ex2_pair(e), f2(coef, coef)), f[j], f[j + 1]);
  }
}

// A position's teacher's entries in shared memory, four arrays of `top`.
struct Entries {
  int32_t* id;  // -1 where unused
  float* p;     // logits / tau, up to a constant that the normaliser has too
  float* zk;    // the student's logits
  float* sum;   // probabilities, an id's entries added up (the id's first entry; the others' id is then -1)

  __device__ __forceinline__ Entries(void* base, int top) {
    id = static_cast<int32_t*>(base);
    p = reinterpret_cast<float*>(id + top);
    zk = p + top;
    sum = zk + top;
  }
};
constexpr int kEntryBytes = 16;

// Entries with the same id are told by a table in shared memory, open
// addressing with at least two places an entry: an id's place holds the id and
// the number of its first entry, with kAgain where it has more.  That entry gets
// the sum of all of them, which the warp takes together and in a fixed order, and
// stands for the others.
constexpr int kAgain = 1 << 30;
inline int table_log2(int top) {
  int log2 = 6;
  while ((1 << log2) < 2 * top) ++log2;
  return log2;
}
__host__ __device__ constexpr size_t table_bytes(int log2) { return size_t(8) << log2; }

// The entries, their normaliser and their mass, by one warp.
template <class E>
__device__ __forceinline__ void read_teacher(const Args& a, const typename E::T* z, int64_t row, float inv_tau, int lane,
                                             const Entries& e, void* table, float& norm, float& mass) {
  const int places = 1 << a.table_log2;
  int32_t *held = static_cast<int32_t*>(table), *first = held + places;
  for (int i = lane * 4; i < places; i += 128) {
    *reinterpret_cast<int4*>(held + i) = make_int4(-1, -1, -1, -1);
    *reinterpret_cast<int4*>(first + i) = make_int4(kAgain - 1, kAgain - 1, kAgain - 1, kAgain - 1);
  }
  float top = -INFINITY;
  bool bad = false;
#pragma unroll 4
  for (int k = lane; k < a.top; k += 32) {
    int32_t v = __ldg(a.ids + row * a.top + k);
    bad |= v >= a.vocab;
    v = v < 0 || v >= a.vocab ? -1 : v;
    const float t = v >= 0 ? __ldg(a.t + row * a.top + k) : -INFINITY;
    e.id[k] = v;
    e.p[k] = t;
    e.zk[k] = v >= 0 ? E::load(z + v) : 0.f;
    top = fmaxf(top, t);
  }
  if (bad && a.status != nullptr) atomicOr(a.status, ENGRAM_ST_BAD_TOKEN);
  top = warp_reduce<true>(top);
  // without a normaliser of the teacher's own the logits are taken relative to the
  // largest, so that norm is the logarithm of their sum alone and rounds like it
  const float base = a.lse != nullptr || top == -INFINITY ? 0.f : top;
  float sum = 0.f;
  for (int k = lane; k < a.top; k += 32) {
    const float t = (e.p[k] - base) * inv_tau;
    e.p[k] = t;
    if (a.lse == nullptr) sum += expf(t);
  }
  // (a position without an entry to learn from has no mass, whatever comes as its normaliser)
  norm = top == -INFINITY ? 0.f : a.lse != nullptr ? __ldg(a.lse + row) : logf(warp_reduce<false>(sum));
  __syncwarp();
  mass = 0.f;
  for (int k = lane; k < a.top; k += 32) {
    mass += expf(e.p[k] - norm);
    const int32_t v = e.id[k];
    if (v < 0) continue;
    int at = static_cast<int>(static_cast<uint32_t>(v) * 2654435769u >> (32 - a.table_log2));
    while (true) {  // half of the places at least are never taken
      const int32_t old = atomicCAS(held + at, -1, v);
      if (old == -1 || old == v) break;
      at = (at + 1) & (places - 1);
    }
    atomicMin(first + at, k);
    e.sum[k] = __int_as_float(at);
  }
  mass = warp_reduce<false>(mass);
  __syncwarp();
  for (int k = lane; k < a.top; k += 32) {
    if (e.id[k] < 0) continue;
    int32_t* f = first + __float_as_int(e.sum[k]);
    if ((*f & (kAgain - 1)) != k) atomicOr(f, kAgain);
  }
  __syncwarp();
  for (int k0 = 0; k0 < a.top; k0 += 32) {
    const int k = k0 + lane;
    const int32_t v = k < a.top ? e.id[k] : -1;
    const int32_t f = v >= 0 ? first[__float_as_int(e.sum[k])] : 0;
    const bool stands = v >= 0 && (f & (kAgain - 1)) == k;
    float pk = stands ? expf(e.p[k] - norm) : -1.f;  // -1: another entry stands for it
    for (uint32_t left = __ballot_sync(0xffffffffu, stands && (f & kAgain)); left != 0; left &= left - 1) {
      const int32_t of = __shfl_sync(0xffffffffu, v, __ffs(left) - 1);
      float sum = 0.f;
      for (int i = lane; i < a.top; i += 32)
        if (e.id[i] == of) sum += expf(e.p[i] - norm);
      sum = warp_reduce<false>(sum);
      if (of == v && stands) pk = sum;
    }
    if (v >= 0) e.sum[k] = pk;
  }
  __syncwarp();
  for (int k = lane; k < a.top; k += 32)
    if (e.sum[k] < 0.f) e.id[k] = -1;
  __syncwarp();
}

// sum_k p_k (ln p_k - ln q_k), by one warp
__device__ __forceinline__ float sum_loss(const Args& a, const Entries& e, float norm, float m, float s, float inv_tau,
                                          int lane) {
  const float log_sum = logf(s);
  float loss = 0.f;
  for (int k = lane; k < a.top; k += 32) {
    const float pk = expf(e.p[k] - norm);
    if (pk > 0.f || pk != pk) loss += pk * ((e.p[k] - norm) - ((e.zk[k] - m) * inv_tau - log_sum));
  }
  return warp_reduce<false>(loss);
}

// The gradients of the entries in the block's part, over what the row's walk
// wrote there, by `threads` threads.
template <class E>
__device__ __forceinline__ void fix_entries(const Args& a, const Row<E>& r, const Entries& e, float m, float c, float coef,
                                            float scale, int tid, int threads) {
  for (int k = tid; k < a.top; k += threads) {
    const int v = e.id[k] < 0 ? -1 : (e.id[k] + r.off) / Row<E>::N;
    if (v >= r.v0 && v < r.v1) E::store(r.dz + e.id[k], ex2((e.zk[k] - m) * c) * coef - scale * e.sum[k]);
  }
}

// a table, and the entries
__host__ __device__ constexpr size_t short_bytes(int top, int log2) {
  return table_bytes(log2) + static_cast<size_t>(kEntryBytes) * top;
}

// --------------------------------------------------------- rows that stay on chip

// The blocks of a cluster share a row and go from row to row.  In a block
//   - the copying warp keeps the copies of the next `depth` rows under way, and
//     finishes a row when its walk is done: the entries' gradients, the loss;
//   - kPrep warps prepare the teacher's entries of the next rows, in turn (nearly
//     all of their time are waits for memory);
//   - kW warps walk the rows: of row i + 1 the maximum and the sum, which they
//     send to every block of the cluster, then of row i, whose pairs have
//     arrived meanwhile, the gradient.
// Waits are for copies, for the other blocks' pairs and for the block's own
// warps; all are bounded.  Where one runs out, the block's warps leave at their
// next wait: what they waited for may still be in use.
//
// 4096 rows of 129,280 bf16 (2.12 GB): 370 us, 5.7 TB/s, 84 % of a copy's rate.
// Bound by instructions issued in the two walks, each with an exponential a
// value.  The loss alone, one walk without stores, takes 254 us (4.2 TB/s) through
// the same slots and pairs, which it could do without.
constexpr int kPairs = 4;    // rows whose pairs may be under way: see `send`
// (4096 x 129,280 bf16 with 16 walking warps: 371 us with 4, 366 with 6, 369 with
// 8; 4096 x 8000 with 4: 50, 53 and 52)
template <int kW>
constexpr int kPrep = kW == 16 ? 6 : 4;
constexpr int kTeacher = 8;  // rows whose teacher's entries are kept, at most
constexpr int kMaxDepth = 4;  // rows whose copies may be under way

template <int kW>
struct Head {  // in front of the dynamic shared memory
  uint64_t full[kMaxDepth];    // a row's copy is here
  uint64_t walked[kMaxDepth];  // its gradient is written: kW arrivals
  uint64_t met[kPairs];        // all pairs of a row are here
  uint64_t known[kTeacher], used[kTeacher];  // the teacher's entries are ready / no longer needed
  float2 pair[kPairs][kMaxCluster * kW];
  float2 stats[kMaxDepth];     // a row's (maximum, sum), for the copying warp
  float weight[kMaxDepth];
  float2 teacher[kTeacher];    // (normaliser, mass)
  int abort;
};

// Warps that prepare, at most one for each row that is kept: a warp that waits for
// row i - keep to be used has waited for row i - keep - preparing before, which
// must be row i - 2 keep or a later one, as the barriers tell two uses apart and
// not three.
template <int kW>
__host__ __device__ constexpr int preparing(int keep) {
  return keep < kPrep<kW> ? keep : kPrep<kW>;
}

template <int kW>
__host__ __device__ constexpr size_t tables_at(int top, int keep) {  // after the teacher's entries
  return (sizeof(Head<kW>) + static_cast<size_t>(keep) * kEntryBytes * top + 127) & ~size_t(127);
}
template <int kW>
__host__ __device__ constexpr size_t head_bytes(int top, int keep, int log2) {
  return tables_at<kW>(top, keep) + preparing<kW>(keep) * table_bytes(log2);
}

template <class E, int kW>
__global__ void __launch_bounds__((kW + 1 + kPrep<kW>) * 32) rows_kernel(const typename E::T* z, typename E::T* dz, Args a) {
  constexpr int N = kVec<E>, kData = kW * 32;
  extern __shared__ __align__(128) unsigned char smem[];
  Head<kW>& h = *reinterpret_cast<Head<kW>*>(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_rank());
  const int first_row = static_cast<int>(blockIdx.x) / a.cluster, step = static_cast<int>(gridDim.x) / a.cluster;
  const int n = first_row < a.rows ? (a.rows - 1 - first_row) / step + 1 : 0;  // this cluster's rows
  const float inv_tau = 1.f / a.tau, c = 1.4426950408889634f * inv_tau;
  auto row_at = [&](int i) { return static_cast<int64_t>(first_row) + static_cast<int64_t>(i) * step; };
  auto slot = [&](int i) { return reinterpret_cast<uint4*>(smem + head_bytes<kW>(a.top, a.keep, a.table_log2) + (i % a.depth) * static_cast<size_t>(a.slot_bytes)); };
  auto entries = [&](int i) { return Entries(smem + sizeof(Head<kW>) + (i % a.keep) * kEntryBytes * a.top, a.top); };
  auto wait = [&](uint64_t& bar, int use) {
    if (__all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&bar), use & 1, &h.abort))) return true;
    if (a.status != nullptr) atomicOr(a.status, ENGRAM_ST_TIMEOUT);
    *reinterpret_cast<volatile int*>(&h.abort) = 1;  // the other waits give up too, and the block ends
    return false;
  };

  if (tid == 0) {
    for (int k = 0; k < kMaxDepth; ++k) {
      mbar_init(smem_u32(&h.full[k]), 2);
      mbar_init(smem_u32(&h.walked[k]), kW);
    }
    for (int k = 0; k < kPairs; ++k) mbar_init(smem_u32(&h.met[k]), 1);
    for (int k = 0; k < kTeacher; ++k) {
      mbar_init(smem_u32(&h.known[k]), 1);
      mbar_init(smem_u32(&h.used[k]), 1);
    }
    h.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (a.cluster > 1) {  // every block's barriers are set up before pairs are sent to them
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }

  if (warp == kW) {
    // ---- copies, and what is left of a row when it has been walked
    auto weight_at = [&](int i) { return i < n && a.weight != nullptr ? __ldg(a.weight + row_at(i)) : 1.f; };
    Row<E> r;
    auto copy = [&](int i, float w) {
      r.at(z, dz, a, row_at(i), rank, i > 0);
      uint4* s = slot(i);
      const bool on = w != 0.f;  // a row without weight is not read
      const uint32_t bar = smem_u32(&h.full[i % a.depth]);
      if (lane == 0) {
        h.weight[i % a.depth] = w;
        // the pairs of the row: expected before any of this block's own
        mbar_arrive_expect_tx(smem_u32(&h.met[i % kPairs]), static_cast<uint32_t>(a.cluster) * kW * sizeof(float2) + a.absent);
        const uint32_t bytes = on && r.end() > r.first() ? static_cast<uint32_t>(r.end() - r.first()) * 16u : 0u;
        mbar_arrive_expect_tx(bar, bytes);
        if (bytes > 0) bulk_g2s(smem_u32(s + (r.first() - r.v0)), r.vectors() + r.first(), bytes, bar);
      }
      __syncwarp();
      if (on && (r.head || r.tail)) {
        if (lane < 2 * N && (lane < N ? r.head : r.tail)) {
          const int e = r.edge_element(lane);
          const int at = ((lane < N ? 0 : r.in1) - r.v0) * N + lane % N;
          E::store(reinterpret_cast<typename E::T*>(s) + at, e >= 0 ? E::load(r.z + e) : -INFINITY);
          // (a later row that lies otherwise has its whole vectors copied over this place)
          fence_proxy_async_smem();
        }
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(bar);
    };
    int begun = 0;  // copies
    for (; begun < a.depth && begun < n; ++begun) copy(begun, weight_at(begun));
    float next = weight_at(a.depth);
    for (int i = 0; i < n; ++i) {
      const float ahead = weight_at(i + a.depth + 1);
      if (!wait(h.walked[i % a.depth], i / a.depth)) break;
      const float w = h.weight[i % a.depth];
      const float2 teacher = h.teacher[i % a.keep], st = h.stats[i % a.depth];
      const bool none = w == 0.f || teacher.y == 0.f;
      const Entries e = entries(i);
      int edge = -1;  // a value of the row's first or last vector that this lane finishes
      float edge_z = 0.f;
      if (dz != nullptr && !none) {
        r.at(z, dz, a, row_at(i), rank, true);
        edge = r.off == r.doff ? r.edge_element(lane) : -1;
        if (edge >= 0) edge_z = E::load(reinterpret_cast<const typename E::T*>(slot(i)) + (edge + r.off - r.v0 * N));
      }
      __syncwarp();
      if (i + a.depth < n) copy(begun++, next);
      next = ahead;
      if (dz != nullptr && !none) {
        r.at(z, dz, a, row_at(i), rank, true);
        const float scale = w * a.tau, coef = scale * teacher.y / st.y;
        if (edge >= 0) E::store(r.dz + edge, ex2((edge_z - st.x) * c) * coef);
        __syncwarp();
        fix_entries<E>(a, r, e, st.x, c, coef, scale, lane, 32);
      }
      if (rank == 0) {
        const float loss = none ? 0.f : sum_loss(a, e, teacher.x, st.x, st.y, inv_tau, lane);
        if (lane == 0) a.loss[row_at(i)] = none ? 0.f : w * a.tau * a.tau * loss;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&h.used[i % a.keep]));
    }
    if (h.abort) {  // copies still under way land before the shared memory is released
      for (int i = begun > a.depth ? begun - a.depth : 0; i < begun; ++i)
        mbar_wait_bounded(smem_u32(&h.full[i % a.depth]), i / a.depth & 1, nullptr);
    }
  } else if (warp > kW) {
    // ---- the teacher's entries, rows in turn
    const int prep = preparing<kW>(a.keep);
    for (int i = warp - kW - 1; warp - kW - 1 < prep && i < n; i += prep) {
      if (i >= a.keep && !wait(h.used[i % a.keep], i / a.keep - 1)) break;
      const int64_t row = row_at(i);
      float norm = 0.f, mass = 0.f;
      if (a.weight == nullptr || __ldg(a.weight + row) != 0.f) {
        read_teacher<E>(a, z + row * a.z_stride, row, inv_tau, lane, entries(i),
                        smem + tables_at<kW>(a.top, a.keep) + (warp - kW - 1) * table_bytes(a.table_log2), norm, mass);
      }
      if (lane == 0) h.teacher[i % a.keep] = make_float2(norm, mass);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&h.known[i % a.keep]));
    }
  } else {
    // ---- the walks
    // A block sends the pairs of row i when it has all those of row i - 2, so
    // every block has sent those, and had used up those of row i - kPairs before.
    auto send = [&](int i, float m, float s) {
      const float2* from = &h.pair[i % kPairs][rank * kW + warp];
      if (lane < a.cluster) {
        uint32_t to, bar;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(from)), "r"(lane));
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(smem_u32(&h.met[i % kPairs])), "r"(lane));
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(to), "f"(m),
                     "f"(s), "r"(bar)
                     : "memory");
      }
      __syncwarp();
    };
    Row<E> r;
    auto walk = [&](int i) {
      if (!wait(h.met[i % kPairs], i / kPairs)) return false;
      float m = -INFINITY, s = 0.f;
      for (int k = lane; k < a.cluster * kW; k += 32) {
        const float2 q = h.pair[i % kPairs][k];
        join(m, s, q.x, q.y, c);
      }
      join_warp(m, s, c);
      const float w = h.weight[i % a.depth], mass = h.teacher[i % a.keep].y;
      if (tid == 0) h.stats[i % a.depth] = make_float2(m, s);
      if (dz != nullptr) {
        r.at(z, dz, a, row_at(i), rank, true);
        if (w == 0.f || mass == 0.f) {  // nothing to learn here
          r.zeros(tid, kData);
        } else {
          const float coef = w * a.tau * mass / s;
          const uint4* src = slot(i) - r.v0;
          if (r.off == r.doff) {
            uint4* dv = reinterpret_cast<uint4*>(r.dz - r.off);
            const int end = r.end();
            int v = r.first() + tid;
            for (; v + (kAhead - 1) * kData < end; v += kAhead * kData) {
              uint4 x[kAhead];
#pragma unroll
              for (int u = 0; u < kAhead; ++u) x[u] = src[v + u * kData];
#pragma unroll
              for (int u = 0; u < kAhead; ++u) {
                float f[N];
                grad_vector<E>(x[u], m, c, coef, f);
                __stcs(dv + v + u * kData, narrow<E>(f));
              }
            }
            for (; v < end; v += kData) {
              float f[N];
              grad_vector<E>(src[v], m, c, coef, f);
              __stcs(dv + v, narrow<E>(f));
            }
          } else {  // the gradient's rows lie differently: value by value
            const typename E::T* part = reinterpret_cast<const typename E::T*>(src) + r.off;
            const int e1 = r.v1 * N - r.off < r.V ? r.v1 * N - r.off : r.V;
            for (int e = (r.v0 * N - r.off > 0 ? r.v0 * N - r.off : 0) + tid; e < e1; e += kData)
              E::store(r.dz + e, ex2((E::load(part + e) - m) * c) * coef);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&h.walked[i % a.depth]));
      return true;
    };
    bool on = n > 0;
    for (int i = 0; i < n; ++i) {
      if (!(on = wait(h.full[i % a.depth], i / a.depth))) break;
      float m = -INFINITY, s = 0.f;
      r.at(z, dz, a, row_at(i), rank, i > 0);
      if (h.weight[i % a.depth] != 0.f) {
        const uint4* part = slot(i);
        const int count = r.v1 - r.v0;
        for (int v = tid; v < count; v += kAhead * kData) {
          uint4 x[kAhead];
#pragma unroll
          for (int u = 0; u < kAhead; ++u) x[u] = v + u * kData < count ? part[v + u * kData] : no_vector<E>();
          add_vectors<E>(x, c, m, s);
        }
        join_warp(m, s, c);
      }
      // the student's logits of the entries have been read before any block
      // may write this row's gradient over them
      if (!(on = wait(h.known[i % a.keep], i / a.keep))) break;
      send(i, m, s);
      if (i > 0 && !(on = walk(i - 1))) break;
    }
    if (on) walk(n - 1);
  }
  // no block leaves while another one may still send to it
  __syncthreads();
  if (a.cluster > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  if (h.abort) {  // pairs that it has not waited for may be on their way: they take some microseconds
    const long long begun = clock64();
    while (clock64() - begun < (1 << 20)) {
    }
  }
}

// --------------------------------------------------------------------- long rows

// One cluster of 8 blocks per row, which is read twice: a row that does not fit
// 8 blocks' shared memory would have to be.  Bound by memory: 512 rows of 600,001
// fp32 (2.46 GB in, 1.23 GB out): 716 us, 5.1 TB/s.
constexpr int kLongWarps = 8, kLongThreads = kLongWarps * 32;

template <class E>
__global__ void __launch_bounds__(kLongThreads, 3) long_rows_kernel(const typename E::T* z, typename E::T* dz, Args a) {
  constexpr int N = kVec<E>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float2 pair[kMaxCluster], warp_pair[kLongWarps], teacher;
  const Entries e(smem + table_bytes(a.table_log2), a.top);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_rank());
  const int64_t row = blockIdx.x / a.cluster;
  Row<E> r;
  r.at(z, dz, a, row, rank, false);
  const float inv_tau = 1.f / a.tau, c = 1.4426950408889634f * inv_tau;
  const float w = a.weight != nullptr ? a.weight[row] : 1.f;
  if (w == 0.f) {  // nothing to learn here (the same for the whole cluster)
    if (rank == 0 && tid == 0) a.loss[row] = 0.f;
    if (dz != nullptr) r.zeros(tid, kLongThreads);
    return;
  }
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if (warp == 0) {
    float norm, mass;
    read_teacher<E>(a, r.z, row, inv_tau, lane, e, smem, norm, mass);
    if (lane == 0) teacher = make_float2(norm, mass);
  }
  const uint4* zv = r.vectors();
  float m = -INFINITY, s = 0.f;
  for (int v = r.v0 + tid; v < r.v1; v += kAhead * kLongThreads) {
    uint4 x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int vu = v + u * kLongThreads;
      x[u] = vu >= r.v1 ? no_vector<E>() : vu >= r.in0 && vu < r.in1 ? zv[vu] : r.edge(vu);
    }
    add_vectors<E>(x, c, m, s);
  }
  join_warp(m, s, c);
  if (lane == 0) warp_pair[warp] = make_float2(m, s);
  __syncthreads();
  m = warp_pair[0].x;
  s = warp_pair[0].y;
#pragma unroll
  for (int k = 1; k < kLongWarps; ++k) join(m, s, warp_pair[k].x, warp_pair[k].y, c);
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every block of the cluster runs
  if (tid < a.cluster) {
    uint32_t to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(&pair[rank])), "r"(tid));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(m), "f"(s) : "memory");
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  m = pair[0].x;
  s = pair[0].y;
  for (int k = 1; k < a.cluster; ++k) join(m, s, pair[k].x, pair[k].y, c);

  const float norm = teacher.x, mass = teacher.y;
  if (rank == 0 && warp == 0) {
    const float loss = mass == 0.f ? 0.f : sum_loss(a, e, norm, m, s, inv_tau, lane);
    if (lane == 0) a.loss[row] = mass == 0.f ? 0.f : w * a.tau * a.tau * loss;
  }
  if (dz == nullptr) return;
  if (mass == 0.f) {
    r.zeros(tid, kLongThreads);
    return;
  }
  const float scale = w * a.tau, coef = scale * mass / s;
  if (r.off == r.doff) {
    uint4* dv = reinterpret_cast<uint4*>(r.dz - r.off);
#pragma unroll 4
    for (int v = r.first() + tid; v < r.end(); v += kLongThreads) {
      float f[N];
      grad_vector<E>(zv[v], m, c, coef, f);
      dv[v] = narrow<E>(f);
    }
    float f[N];
    if (r.head && tid == 0) {
      grad_vector<E>(r.edge(0), m, c, coef, f);
      r.store_edge(0, f);
    }
    if (r.tail && tid == 32) {
      grad_vector<E>(r.edge(r.in1), m, c, coef, f);
      r.store_edge(r.in1, f);
    }
  } else {
    const int e1 = r.v1 * N - r.off < r.V ? r.v1 * N - r.off : r.V;
    for (int e = (r.v0 * N - r.off > 0 ? r.v0 * N - r.off : 0) + tid; e < e1; e += kLongThreads)
      E::store(r.dz + e, ex2((E::load(r.z + e) - m) * c) * coef);
  }
  __syncthreads();
  fix_entries<E>(a, r, e, m, c, coef, scale, tid, kLongThreads);
}

// -------------------------------------------------------------------- short rows

// A warp per row: nothing is handed between warps, and the second walk finds the
// row in the caches.  Bound by latency, which 32 warps an SM hide from one
// another.  16,384 rows of 20 entries, this kernel against rows_kernel: of 1000
// bf16 32 against 76 us, of 4000 (8 KB) 66 against 95, of 8000 150 against 130.
constexpr int kShortWarps = 4;
constexpr int kShortBytes = 8192;

template <class E>
__global__ void __launch_bounds__(kShortWarps * 32, 8) short_rows_kernel(const typename E::T* z, typename E::T* dz, Args a) {
  constexpr int N = kVec<E>;
  extern __shared__ __align__(128) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned char* table = smem + warp * short_bytes(a.top, a.table_log2);
  const Entries e(table + table_bytes(a.table_log2), a.top);
  const float inv_tau = 1.f / a.tau, c = 1.4426950408889634f * inv_tau;
  Row<E> r;
  bool again = false;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kShortWarps + warp; row < a.rows;
       row += static_cast<int64_t>(gridDim.x) * kShortWarps, again = true) {
    __syncwarp();  // the last row's entries are no longer read
    r.at(z, dz, a, row, 0, again);
    const float w = a.weight != nullptr ? __ldg(a.weight + row) : 1.f;
    if (w == 0.f) {  // nothing to learn here
      if (lane == 0) a.loss[row] = 0.f;
      if (dz != nullptr) r.zeros(lane, 32);
      continue;
    }
    const uint4* zv = r.vectors();
    auto vector = [&](int v) { return v >= r.v1 ? no_vector<E>() : v >= r.in0 && v < r.in1 ? zv[v] : r.edge(v); };
    uint4 x[kAhead];  // on their way while the teacher's entries are read
#pragma unroll
    for (int u = 0; u < kAhead; ++u) x[u] = vector(lane + u * 32);
    float norm, mass, m = -INFINITY, s = 0.f;
    read_teacher<E>(a, r.z, row, inv_tau, lane, e, table, norm, mass);
    for (int v = lane;;) {
      add_vectors<E>(x, c, m, s);
      v += kAhead * 32;
      if (v - lane >= r.v1) break;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) x[u] = vector(v + u * 32);
    }
    join_warp(m, s, c);
    const float loss = mass == 0.f ? 0.f : sum_loss(a, e, norm, m, s, inv_tau, lane);
    if (lane == 0) a.loss[row] = mass == 0.f ? 0.f : w * a.tau * a.tau * loss;
    if (dz == nullptr) continue;
    if (mass == 0.f) {
      r.zeros(lane, 32);
      continue;
    }
    const float scale = w * a.tau, coef = scale * mass / s;
    if (r.off == r.doff) {
      uint4* dv = reinterpret_cast<uint4*>(r.dz - r.off);
#pragma unroll 4
      for (int v = r.first() + lane; v < r.end(); v += 32) {
        float f[N];
        grad_vector<E>(zv[v], m, c, coef, f);
        __stcs(dv + v, narrow<E>(f));
      }
      const int edge = r.edge_element(lane);
      if (edge >= 0) E::store(r.dz + edge, ex2((E::load(r.z + edge) - m) * c) * coef);
    } else {
      for (int i = lane; i < r.V; i += 32) E::store(r.dz + i, ex2((E::load(r.z + i) - m) * c) * coef);
    }
    __syncwarp();
    fix_entries<E>(a, r, e, m, c, coef, scale, lane, 32);
  }
}

// ------------------------------------------------------------------------ launch

constexpr int kSmem = 224 * 1024;  // dynamic shared memory of a block, at most

// Sets the kernel's shared-memory limit once per device.
int opt_in(const void* kernel, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
  if (bit != 0 && (done.load(std::memory_order_relaxed) & bit)) return ENGRAM_OK;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return fail(ENGRAM_E_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  done.fetch_or(bit, std::memory_order_relaxed);
  return ENGRAM_OK;
}

// Clusters that are on the GPU at once.  Blocks wait for one another within
// their cluster alone, so the number matters for speed and nothing else.  The
// runtime's answer for a kernel and its sizes is kept.
int clusters_at_once(const void* kernel, int cluster, int threads, size_t smem, int* out) {
  struct Known {
    const void* kernel;
    int dev, cluster;
    size_t smem;
    int clusters;
  };
  static std::mutex mu;
  static Known known[64];
  static int n_known = 0;
  int dev = 0;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lock(mu);
  for (int k = 0; k < n_known; ++k)
    if (known[k].kernel == kernel && known[k].dev == dev && known[k].cluster == cluster && known[k].smem == smem) {
      *out = known[k].clusters;
      return ENGRAM_OK;
    }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cluster));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(cluster);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaOccupancyMaxActiveClusters(out, kernel, &cfg);
  if (e != cudaSuccess) return fail(ENGRAM_E_CUDA, "cudaOccupancyMaxActiveClusters: %s", cudaGetErrorString(e));
  if (*out < 1) return fail(ENGRAM_E_CUDA, "no cluster of %d blocks fits the device", cluster);
  known[n_known < 64 ? n_known++ : 0] = Known{kernel, dev, cluster, smem, *out};
  return ENGRAM_OK;
}

template <class K, class T>
int launch(K kernel, int64_t blocks, int threads, size_t smem, const T* z, T* dz, const Args& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(a.cluster);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, z, dz, a);
  if (e != cudaSuccess) return fail(ENGRAM_E_CUDA, "distill launch: %s", cudaGetErrorString(e));
  return check_launch("distill");
}

template <class E, int kW>
int launch_rows(const void* z, void* dz, const Args& a, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  int rc = opt_in(reinterpret_cast<const void*>(rows_kernel<E, kW>), done);
  if (rc) return rc;
  constexpr int kThreads = (kW + 1 + kPrep<kW>) * 32;
  const size_t smem = head_bytes<kW>(a.top, a.keep, a.table_log2) + static_cast<size_t>(a.depth) * a.slot_bytes;
  int clusters = 0;
  if ((rc = clusters_at_once(reinterpret_cast<const void*>(rows_kernel<E, kW>), a.cluster, kThreads, smem, &clusters)))
    return rc;
  return launch(rows_kernel<E, kW>, std::min<int64_t>(a.rows, clusters) * a.cluster, kThreads, smem,
                static_cast<const typename E::T*>(z), static_cast<typename E::T*>(dz), a, st);
}

template <class E>
int launch_distill(const void* z, void* dz, Args a, int sms, cudaStream_t st) {
  a.aligned = a.z_stride * E::kBytes % 16 == 0 && (dz == nullptr || a.dz_stride * E::kBytes % 16 == 0);
  const int64_t vecs = (a.vocab * E::kBytes + 16 + 15) / 16;  // with a misaligned row's first vector
  a.table_log2 = table_log2(a.top);
  if (vecs * 16 <= kShortBytes) {
    static std::atomic<uint64_t> done{0};
    int rc = opt_in(reinterpret_cast<const void*>(short_rows_kernel<E>), done);
    if (rc) return rc;
    a.cluster = 1;
    const int64_t want = (static_cast<int64_t>(a.rows) + kShortWarps - 1) / kShortWarps;
    return launch(short_rows_kernel<E>, std::min<int64_t>(want, static_cast<int64_t>(sms) * 8), kShortWarps * 32,
                  kShortWarps * short_bytes(a.top, a.table_log2), static_cast<const typename E::T*>(z), static_cast<typename E::T*>(dz), a, st);
  }
  // fewer where the entries would take the rows' place: 4096 rows of 50,000 bf16 with
  // 1024 entries take 1950 us with 4 and 2790 with 8 (with 200 entries, where there
  // still is room, 318 and 222)
  a.keep = a.top <= 128 ? kTeacher : 4;
  const int64_t room = kSmem - static_cast<int64_t>(head_bytes<16>(a.top, a.keep, a.table_log2));
  // the smallest cluster that holds three rows (four where they fit); of 4 or 8
  // blocks two will do
  for (a.cluster = 1, a.cluster_log2 = 0; a.cluster <= kMaxCluster; a.cluster *= 2, ++a.cluster_log2) {
    const int64_t part = ((vecs + a.cluster - 1) / a.cluster * 16 + 127) / 128 * 128;
    for (a.depth = kMaxDepth; a.depth >= (a.cluster >= 4 ? 2 : 3); --a.depth) {
      if (part * a.depth > room) continue;
      a.slot_bytes = static_cast<int32_t>(part);
      // warps for the length of their walk, us with 4, 8 and 16 of them: 16,384 rows of
      // 5000 bf16 (10 KB) 106, 164 and -, of 8000 131, 177 and -, of 10,000 (20 KB) -,
      // 189 and 311, of 16,000 -, 344 and 333, of 20,000 (40 KB) -, 359 and 357, 4096 of
      // 129,280 (64 KB parts) -, 400 and 379 (20 and 64 entries, gradients elsewhere)
      return part <= 16 * 1024   ? launch_rows<E, 4>(z, dz, a, st)
             : part <= 40 * 1024 ? launch_rows<E, 8>(z, dz, a, st)
                                 : launch_rows<E, 16>(z, dz, a, st);
    }
  }
  a.cluster = kMaxCluster;
  a.cluster_log2 = 3;
  return launch(long_rows_kernel<E>, static_cast<int64_t>(a.rows) * a.cluster, kLongThreads, short_bytes(a.top, a.table_log2),
                static_cast<const typename E::T*>(z), static_cast<typename E::T*>(dz), a, st);
}

}  // namespace
}  // namespace engram

using namespace engram;

namespace {
int distill(const void* logits_d, int32_t type, int64_t n_tokens, int64_t vocab, int64_t logits_stride,
            const int32_t* teacher_ids_d, const float* teacher_logits_d, int32_t top, float temperature,
            const float* teacher_lse_d, const float* weight_d, float* loss_d, void* dlogits_d, int64_t dlogits_stride,
            int32_t* status_d, void* stream, uint32_t absent) {
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
  int sms = 0;
  int rc = check_device(&sms);
  if (rc) return rc;
  Args a{};
  a.vocab = vocab;
  a.z_stride = logits_stride;
  a.dz_stride = dlogits_stride;
  a.rows = static_cast<int32_t>(n_tokens);
  a.ids = teacher_ids_d;
  a.t = teacher_logits_d;
  a.top = top;
  a.tau = temperature;
  a.lse = teacher_lse_d;
  a.weight = weight_d;
  a.loss = loss_d;
  a.status = status_d;
  a.absent = absent;
  return type == ENGRAM_T_BF16 ? launch_distill<train::Bf16>(logits_d, dlogits_d, a, sms, as_stream(stream))
                               : launch_distill<train::F32>(logits_d, dlogits_d, a, sms, as_stream(stream));
}
}  // namespace

extern "C" int engram_distill(const void* logits_d, int32_t type, int64_t n_tokens, int64_t vocab,
                              int64_t logits_stride, const int32_t* teacher_ids_d, const float* teacher_logits_d,
                              int32_t top, float temperature, const float* teacher_lse_d, const float* weight_d,
                              float* loss_d, void* dlogits_d, int64_t dlogits_stride, int32_t* status_d,
                              void* stream) {
  return distill(logits_d, type, n_tokens, vocab, logits_stride, teacher_ids_d, teacher_logits_d, top, temperature,
                 teacher_lse_d, weight_d, loss_d, dlogits_d, dlogits_stride, status_d, stream, 0);
}

extern "C" int engram_selftest_distill_wait(const void* logits_d, int32_t type, int64_t n_tokens, int64_t vocab,
                                            int64_t logits_stride, const int32_t* teacher_ids_d,
                                            const float* teacher_logits_d, int32_t top, float* loss_d,
                                            void* dlogits_d, int64_t dlogits_stride, int32_t* status_d,
                                            void* stream) {
  return distill(logits_d, type, n_tokens, vocab, logits_stride, teacher_ids_d, teacher_logits_d, top, 1.f, nullptr,
                 nullptr, loss_d, dlogits_d, dlogits_stride, status_d, stream, sizeof(float2));
}
