// Distillation from a teacher's top logits: the loss of every position and
// the gradient of the student's logits.
//
// With q = softmax(z / tau) over the vocabulary, p the teacher's
// probabilities at its K entries and P their sum:
//   loss = w tau^2 sum_k p_k (ln p_k - ln q_k)
//   dz_v = w tau (P q_v - p_v)
#include <cuda_runtime.h>
#include <stdint.h>

#include "engram_internal.h"
#include "train_device.cuh"

namespace engram {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTop = ENGRAM_DISTILL_MAX_TOP;

struct Args {
  int64_t vocab, z_stride, dz_stride;
  const int32_t* ids;
  const float* t;
  int32_t top;
  float tau;
  const float* lse;
  const float* weight;
  float* loss;
  int32_t* status;
};

// Sum or maximum over the block, the same in every thread and run.
template <bool kMax>
__device__ float block_reduce(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? fmaxf(v, w) : v + w;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) v = kMax ? fmaxf(v, red[w]) : v + red[w];
  return v;
}

// One block per position.
template <class E>
__global__ void __launch_bounds__(kThreads) distill_kernel(const typename E::T* __restrict__ z,
                                                           typename E::T* dz, Args a) {
  __shared__ float red[kThreads / 32];
  __shared__ float p[kMaxTop];
  __shared__ int32_t id[kMaxTop];
  const int64_t row = blockIdx.x;
  const typename E::T* zr = z + row * a.z_stride;
  typename E::T* dr = dz + row * a.dz_stride;
  const float w = a.weight != nullptr ? a.weight[row] : 1.f;
  const float inv_tau = 1.f / a.tau;

  // the teacher's probabilities
  float top = -INFINITY;
  for (int k = threadIdx.x; k < a.top; k += kThreads) {
    int32_t v = a.ids[row * a.top + k];
    if (v >= a.vocab) {
      if (a.status != nullptr) atomicOr(a.status, ENGRAM_ST_BAD_TOKEN);
      v = -1;
    }
    id[k] = v;
    p[k] = v >= 0 ? a.t[row * a.top + k] * inv_tau : -INFINITY;
    top = fmaxf(top, p[k]);
  }
  top = block_reduce<true>(top, red);
  float norm = 0.f;
  if (a.lse != nullptr) {
    norm = a.lse[row];
  } else {
    float sum = 0.f;
    for (int k = threadIdx.x; k < a.top; k += kThreads) sum += top == -INFINITY ? 0.f : expf(p[k] - top);
    sum = block_reduce<false>(sum, red);
    norm = top == -INFINITY ? 0.f : top + logf(sum);
  }
  float mass = 0.f;
  for (int k = threadIdx.x; k < a.top; k += kThreads) mass += expf(p[k] - norm);
  mass = block_reduce<false>(mass, red);
  if (w == 0.f || mass == 0.f) {  // nothing to learn here
    if (threadIdx.x == 0) a.loss[row] = 0.f;
    if (dz != nullptr)
      for (int64_t v = threadIdx.x; v < a.vocab; v += kThreads) E::store(dr + v, 0.f);
    return;
  }

  float m = -INFINITY;
  for (int64_t v = threadIdx.x; v < a.vocab; v += kThreads) m = fmaxf(m, E::load(zr + v));
  m = block_reduce<true>(m, red);
  float sum = 0.f;
  for (int64_t v = threadIdx.x; v < a.vocab; v += kThreads) sum += expf((E::load(zr + v) - m) * inv_tau);
  sum = block_reduce<false>(sum, red);
  const float log_sum = logf(sum);

  float loss = 0.f;
  for (int k = threadIdx.x; k < a.top; k += kThreads) {
    const float pk = expf(p[k] - norm);
    if (pk > 0.f) loss += pk * ((p[k] - norm) - ((E::load(zr + id[k]) - m) * inv_tau - log_sum));
  }
  loss = block_reduce<false>(loss, red);
  if (threadIdx.x == 0) a.loss[row] = w * a.tau * a.tau * loss;
  if (dz == nullptr) return;

  const float scale = w * a.tau;
  const float c = scale * mass / sum;
  // the entries' gradients first: dz may be z itself
  float mine[(kMaxTop + kThreads - 1) / kThreads];
#pragma unroll
  for (int j = 0; j < (kMaxTop + kThreads - 1) / kThreads; ++j) {
    const int k = threadIdx.x + j * kThreads;
    mine[j] = 0.f;
    if (k < a.top && id[k] >= 0) {
      float pk = 0.f;
      for (int i = 0; i < a.top; ++i) pk += id[i] == id[k] ? expf(p[i] - norm) : 0.f;  // an id given twice adds up
      mine[j] = c * expf((E::load(zr + id[k]) - m) * inv_tau) - scale * pk;
    }
  }
  __syncthreads();
  for (int64_t v = threadIdx.x; v < a.vocab; v += kThreads) E::store(dr + v, c * expf((E::load(zr + v) - m) * inv_tau));
  __syncthreads();
#pragma unroll
  for (int j = 0; j < (kMaxTop + kThreads - 1) / kThreads; ++j) {
    const int k = threadIdx.x + j * kThreads;
    if (k < a.top && id[k] >= 0) E::store(dr + id[k], mine[j]);
  }
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
  if (n_tokens > 0x7fffffff) return fail(ENGRAM_E_RANGE, "n_tokens must be below 2^31");
  if (vocab < 1 || vocab > 0x7fffffff) return fail(ENGRAM_E_SHAPE, "vocab must be in [1, 2^31)");
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
  Args a{vocab, logits_stride, dlogits_stride, teacher_ids_d, teacher_logits_d, top, temperature, teacher_lse_d, weight_d,
         loss_d, status_d};
  if (type == ENGRAM_T_BF16)
    distill_kernel<train::Bf16><<<static_cast<int>(n_tokens), kThreads, 0, as_stream(stream)>>>(
        static_cast<const uint16_t*>(logits_d), static_cast<uint16_t*>(dlogits_d), a);
  else
    distill_kernel<train::F32><<<static_cast<int>(n_tokens), kThreads, 0, as_stream(stream)>>>(
        static_cast<const float*>(logits_d), static_cast<float*>(dlogits_d), a);
  return check_launch("distill_kernel");
}
