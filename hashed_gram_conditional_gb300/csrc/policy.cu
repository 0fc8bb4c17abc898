// The clipped policy loss of sampled tokens with a KL term towards a reference,
// and the gradient of the logits.
//
// With q = softmax(z / tau), l = ln q_a of the sampled token a, r = exp(l - l_old),
// and d = l_ref - l:
//   loss = w (-min(r A, clip(r, 1 - low, 1 + high) A) + kl (e^d - 1 - d))
//   dloss/dl = w (-[not clipped] r A - kl (e^d - 1))
//   dz_v = dloss/dl ([v = a] - q_v) / tau
// which is a softmax row with one entry: W = w, P = p_a = -(dloss/dl) / (w tau).  (W = w tau, as
// the distillation has it, would take tau^-2, which an fp32 number need not hold.)  The rows
// are walked by the kernels of logit_rows.cuh.
#include "logit_rows.cuh"

namespace engram {
namespace {

struct Args : rows::RowArgs {
  const int32_t* ids;
  const float *adv, *old, *ref;
  float* logp;
  float low, high, kl;
};

// A position's numbers in shared memory.
struct Numbers {
  int32_t id;
  float logit, adv, old, ref;
  int32_t unused[3];
};

struct Sampled {
  using Args = engram::Args;
  static constexpr int kEntryBytes = sizeof(Numbers);
  static constexpr bool kKnown = false;
  struct Entries {
    Numbers* at;
    __device__ __forceinline__ Entries(void* base, int) : at(static_cast<Numbers*>(base)) {}
  };
  static int table_log2(int) { return 0; }
  static __host__ __device__ constexpr size_t table_bytes(int) { return 0; }

  static __device__ __forceinline__ float weight(const Args& a, int64_t row) {
    const int32_t id = __ldg(a.ids + row);
    if (id < 0 || id >= a.vocab) return 0.f;
    return a.weight != nullptr ? __ldg(a.weight + row) : 1.f;
  }
  static __device__ __forceinline__ float factor(const Args&, float w) { return w; }
  static __device__ __forceinline__ void skip(const Args& a, int64_t row, int lane) {
    if (lane == 0 && __ldg(a.ids + row) >= a.vocab && a.status != nullptr) atomicOr(a.status, ENGRAM_ST_BAD_TOKEN);
  }
  template <class E>
  static __device__ __forceinline__ void read(const Args& a, const typename E::T* z, int64_t row, float, int lane,
                                              const Entries& e, void*, float& x0, float& x1) {
    x0 = x1 = 0.f;
    if (lane == 0) {
      const int32_t id = __ldg(a.ids + row);
      e.at->id = id;
      e.at->logit = E::load(z + id);
      e.at->adv = __ldg(a.adv + row);
      e.at->old = a.old != nullptr ? __ldg(a.old + row) : 0.f;
      e.at->ref = a.ref != nullptr ? __ldg(a.ref + row) : 0.f;
    }
    __syncwarp();
  }

  static __device__ __forceinline__ float logp(const Entries& e, float m, float s, float inv_tau) {
    return (e.at->logit - m) * inv_tau - logf(s);
  }
  static __device__ __forceinline__ float ratio(const Args& a, const Entries& e, float l) {
    return a.old != nullptr ? expf(l - e.at->old) : 1.f;
  }
  static __device__ __forceinline__ float clipped(const Args& a, float r) {
    return r < 1.f - a.low ? 1.f - a.low : r > 1.f + a.high ? 1.f + a.high : r;  // (a NaN stays)
  }
  // Every warp that walks a row computes this, with the hardware's exponential (2^-22) as
  // for the row's own; the loss, one warp's work, has expf and expm1f.
  static __device__ __forceinline__ float mass(const Args& a, const Entries& e, float2, float m, float s, float inv_tau) {
    constexpr float kLog2e = 1.4426950408889634f;
    const float l = logp(e, m, s, inv_tau), r = a.old != nullptr ? rows::ex2((l - e.at->old) * kLog2e) : 1.f;
    const float plain = r * e.at->adv;
    float d = plain > clipped(a, r) * e.at->adv ? 0.f : plain;  // -dloss/dl / w
    if (a.ref != nullptr) {
      const float x = e.at->ref - l;
      // e^x - 1; for small x, where the difference would cancel, from its series
      d = fmaf(a.kl, fabsf(x) < 0.125f ? fmaf(gap_series(x) * x, x, x) : rows::ex2(x * kLog2e) - 1.f, d);
    }
    return d * inv_tau;
  }
  template <class E>
  static __device__ __forceinline__ void fix(const Args& a, const rows::Row<E>& r, const Entries& e, float mass, float m,
                                             float c, float coef, float scale, int tid, int threads) {
    rows::fix_entries<E>(a, r, [&](int) { return e.at->id; }, [&](int) { return e.at->logit; }, [&](int) { return mass; },
                         m, c, coef, scale, tid, threads);
  }
  static __device__ __forceinline__ void finish(const Args& a, const Entries& e, int64_t row, float w, float2, float m,
                                                float s, float inv_tau, int lane) {
    if (lane != 0) return;
    float loss = 0.f, l = 0.f;
    if (w != 0.f) {
      l = logp(e, m, s, inv_tau);
      const float r = ratio(a, e, l), plain = r * e.at->adv, cut = clipped(a, r) * e.at->adv;
      loss = -(plain > cut ? cut : plain);
      if (a.ref != nullptr) {
        const float d = e.at->ref - l;
        loss = fmaf(a.kl, gap(d), loss);
      }
      loss *= w;
    }
    a.loss[row] = loss;
    if (a.logp != nullptr) a.logp[row] = l;
  }
  // e^d - 1 - d; for small d, where the difference would cancel, its series, whose
  // next term is below 2^-24 of the first for |d| < 1/8; infinite with e^d
  static __device__ __forceinline__ float gap(float d) {
    const float x = expm1f(d);
    return x == INFINITY ? x : fabsf(d) >= 0.125f ? x - d : gap_series(d) * d * d;
  }
  static __device__ __forceinline__ float gap_series(float d) {
    float p = 1.f / 362880.f;
    p = fmaf(p, d, 1.f / 40320.f);
    p = fmaf(p, d, 1.f / 5040.f);
    p = fmaf(p, d, 1.f / 720.f);
    p = fmaf(p, d, 1.f / 120.f);
    p = fmaf(p, d, 1.f / 24.f);
    p = fmaf(p, d, 1.f / 6.f);
    return fmaf(p, d, 0.5f);
  }
};

}  // namespace
}  // namespace engram

using namespace engram;

extern "C" int engram_policy(const void* logits_d, int32_t type, int64_t n_tokens, int64_t vocab, int64_t logits_stride,
                             const int32_t* ids_d, const float* advantage_d, const float* old_logp_d,
                             const float* ref_logp_d, float clip_low, float clip_high, float kl, float temperature,
                             const float* weight_d, float* loss_d, float* logp_d, void* dlogits_d,
                             int64_t dlogits_stride, int32_t* status_d, void* stream) {
  if (!train::known_type(type)) return fail(ENGRAM_E_INVALID, "type %d is not ENGRAM_T_BF16 or ENGRAM_T_F32", type);
  if (n_tokens < 0) return fail(ENGRAM_E_INVALID, "n_tokens < 0");
  if (n_tokens > 0x7fffffff / rows::kMaxCluster) return fail(ENGRAM_E_RANGE, "n_tokens must be below 2^28");
  if (vocab < 1 || vocab > 0x7fffff00) return fail(ENGRAM_E_SHAPE, "vocab must be in [1, 2^31 - 256]");
  if (!(temperature > 0.f) || temperature > 3.0e38f) return fail(ENGRAM_E_INVALID, "temperature must be positive and finite");
  if (!(clip_low >= 0.f) || !(clip_high >= 0.f) || clip_low > 3.0e38f || clip_high > 3.0e38f)
    return fail(ENGRAM_E_INVALID, "clip bounds must be finite and not negative");
  if (!(kl >= 0.f) || kl > 3.0e38f) return fail(ENGRAM_E_INVALID, "kl must be finite and not negative");
  if (logits_stride < vocab || (dlogits_d && dlogits_stride < vocab))
    return fail(ENGRAM_E_SHAPE, "row stride below vocab");
  if (n_tokens == 0) return ENGRAM_OK;
  if (!logits_d || !loss_d || !ids_d || !advantage_d) return fail(ENGRAM_E_INVALID, "null device pointer");
  if (kl > 0.f && !ref_logp_d) return fail(ENGRAM_E_INVALID, "a KL term needs ref_logp");
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
  a.top = 1;
  a.tau = temperature;
  a.weight = weight_d;
  a.loss = loss_d;
  a.status = status_d;
  a.ids = ids_d;
  a.adv = advantage_d;
  a.old = old_logp_d;
  a.ref = kl > 0.f ? ref_logp_d : nullptr;
  a.logp = logp_d;
  a.low = clip_low;
  a.high = clip_high;
  a.kl = kl;
  return type == ENGRAM_T_BF16 ? rows::launch_loss<Sampled, train::Bf16>(logits_d, dlogits_d, a, sms, as_stream(stream))
                               : rows::launch_loss<Sampled, train::F32>(logits_d, dlogits_d, a, sms, as_stream(stream));
}
