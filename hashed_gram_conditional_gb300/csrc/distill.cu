// Distillation from a teacher's top logits: the loss of every position and
// the gradient of the student's logits.
//
// With q = softmax(z / tau) over the vocabulary, p the teacher's
// probabilities at its K entries and P their sum:
//   loss = w tau^2 sum_k p_k (ln p_k - ln q_k)
//   dz_v = w tau (P q_v - p_v)
// The rows are walked by the kernels of logit_rows.cuh.
#include "logit_rows.cuh"

namespace engram {
namespace {

using namespace rows;
constexpr int kMaxTop = ENGRAM_DISTILL_MAX_TOP;

struct Args : RowArgs {
  const int32_t* ids;
  const float* t;
  const float* lse;
};

// A position's teacher's entries in shared memory, four arrays of `top`.
struct Held {
  int32_t* id;  // -1 where unused
  float* p;     // logits / tau, up to a constant that the normaliser has too
  float* zk;    // the student's logits
  float* sum;   // probabilities, an id's entries added up (the id's first entry; the others' id is then -1)

  __device__ __forceinline__ Held(void* base, int top) {
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
                                             const Held& e, void* table, float& norm, float& mass) {
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
__device__ __forceinline__ float sum_loss(const Args& a, const Held& e, float norm, float m, float s, float inv_tau,
                                          int lane) {
  const float log_sum = logf(s);
  float loss = 0.f;
  for (int k = lane; k < a.top; k += 32) {
    const float pk = expf(e.p[k] - norm);
    if (pk > 0.f || pk != pk) loss += pk * ((e.p[k] - norm) - ((e.zk[k] - m) * inv_tau - log_sum));
  }
  return warp_reduce<false>(loss);
}

struct Teacher {
  using Args = engram::Args;
  using Entries = Held;
  static constexpr int kEntryBytes = engram::kEntryBytes;
  static constexpr bool kKnown = true;
  static int table_log2(int top) { return engram::table_log2(top); }
  static __host__ __device__ constexpr size_t table_bytes(int log2) { return engram::table_bytes(log2); }
  static __device__ __forceinline__ float weight(const Args& a, int64_t row) {
    return a.weight != nullptr ? __ldg(a.weight + row) : 1.f;
  }
  static __device__ __forceinline__ float factor(const Args& a, float w) { return w * a.tau; }
  // the normaliser and the mass
  template <class E>
  static __device__ __forceinline__ void read(const Args& a, const typename E::T* z, int64_t row, float inv_tau, int lane,
                                              const Entries& e, void* table, float& norm, float& mass) {
    read_teacher<E>(a, z, row, inv_tau, lane, e, table, norm, mass);
  }
  static __device__ __forceinline__ void skip(const Args&, int64_t, int) {}
  static __device__ __forceinline__ float mass(const Args&, const Entries&, float2 known, float, float, float) {
    return known.y;
  }
  template <class E>
  static __device__ __forceinline__ void fix(const Args& a, const Row<E>& r, const Entries& e, float, float m, float c,
                                             float coef, float scale, int tid, int threads) {
    fix_entries<E>(a, r, [&](int k) { return e.id[k]; }, [&](int k) { return e.zk[k]; }, [&](int k) { return e.sum[k]; }, m,
                   c, coef, scale, tid, threads);
  }
  static __device__ __forceinline__ void finish(const Args& a, const Entries& e, int64_t row, float w, float2 known, float m,
                                                float s, float inv_tau, int lane) {
    const bool none = w == 0.f || known.y == 0.f;
    const float loss = none ? 0.f : sum_loss(a, e, known.x, m, s, inv_tau, lane);
    if (lane == 0) a.loss[row] = none ? 0.f : w * a.tau * a.tau * loss;
  }
};

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
  return type == ENGRAM_T_BF16 ? launch_loss<Teacher, train::Bf16>(logits_d, dlogits_d, a, sms, as_stream(stream))
                               : launch_loss<Teacher, train::F32>(logits_d, dlogits_d, a, sms, as_stream(stream));
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
