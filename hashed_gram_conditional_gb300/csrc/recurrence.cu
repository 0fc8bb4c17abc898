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

constexpr int kThreads = 128;
constexpr int kTile = ENGRAM_RECURRENCE_TILE;

struct Gate {
  float f, u;  // sigmoid(g), sigmoid(-g)
};

// With e = exp(-|g|): the larger of the two is 1 / (1 + e), the smaller
// e / (1 + e); neither cancels nor overflows.
__device__ __forceinline__ Gate gate_of(float g) {
  const float e = expf(-fabsf(g));
  const float big = 1.f / (1.f + e), small = e * big;
  Gate r;
  r.f = g >= 0.f ? big : small;
  r.u = g >= 0.f ? small : big;
  return g != g ? Gate{g, g} : r;
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
  int32_t dim;
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

// One thread per (sequence, channel).
template <class E>
__global__ void __launch_bounds__(kThreads) forward_kernel(Args<E> a) {
  const int64_t q = blockIdx.x;
  const int d = blockIdx.y * kThreads + threadIdx.x;
  if (d >= a.dim) return;
  const int32_t slot = slot_of(a, q);
  float s = slot >= 0 && a.state != nullptr ? a.state[static_cast<int64_t>(slot) * a.dim + d] : 0.f;
  for (int64_t t = a.cu[q]; t < a.cu[q + 1]; ++t) {
    if (a.carry != nullptr && t % kTile == 0) a.carry[t / kTile * a.dim + d] = s;
    const bool live = slot >= 0 && (a.mask == nullptr || a.mask[t] == 0);
    if (live) {
      const Gate k = gate_of(E::load(a.g + t * a.g_stride + d));
      s = fmaf(k.f, s, k.u * E::load(a.x + t * a.x_stride + d));
    }
    E::store(a.y + t * a.y_stride + d, live ? s : 0.f);
  }
  if (slot >= 0 && a.state_out != nullptr) a.state_out[static_cast<int64_t>(slot) * a.dim + d] = s;
}

// One thread per (sequence, channel), tiles from the last to the first; each
// tile's states are computed again from the state saved before it.
template <class E>
__global__ void __launch_bounds__(kThreads) backward_kernel(Args<E> a) {
  const int64_t q = blockIdx.x;
  const int d = blockIdx.y * kThreads + threadIdx.x;
  if (d >= a.dim) return;
  const int32_t slot = slot_of(a, q);
  const int64_t t0 = a.cu[q], t1 = a.cu[q + 1];
  float l = slot >= 0 && a.dstate != nullptr ? a.dstate[static_cast<int64_t>(slot) * a.dim + d] : 0.f;
  for (int64_t hi = t1; hi > t0;) {
    const int64_t tile = (hi - 1) / kTile;
    const int64_t lo = tile * kTile > t0 ? tile * kTile : t0;
    float s = tile * kTile >= t0 ? a.carry[tile * a.dim + d]
              : slot >= 0 && a.state != nullptr ? a.state[static_cast<int64_t>(slot) * a.dim + d] : 0.f;
    float before[kTile];
    for (int64_t t = lo; t < hi; ++t) {
      before[t - lo] = s;
      if (slot >= 0 && (a.mask == nullptr || a.mask[t] == 0)) {
        const Gate k = gate_of(E::load(a.g + t * a.g_stride + d));
        s = fmaf(k.f, s, k.u * E::load(a.x + t * a.x_stride + d));
      }
    }
    for (int64_t t = hi - 1; t >= lo; --t) {
      float dx = 0.f, dg = 0.f;
      if (slot >= 0 && (a.mask == nullptr || a.mask[t] == 0)) {
        const Gate k = gate_of(E::load(a.g + t * a.g_stride + d));
        l += E::load(a.dy + t * a.dy_stride + d);
        dx = l * k.u;
        dg = dx * k.f * (before[t - lo] - E::load(a.x + t * a.x_stride + d));
        l *= k.f;
      }
      E::store(a.dx + t * a.dx_stride + d, dx);
      E::store(a.dg + t * a.dg_stride + d, dg);
    }
    hi = lo;
  }
  if (slot >= 0 && a.dstate != nullptr) a.dstate[static_cast<int64_t>(slot) * a.dim + d] = l;
}

template <class E>
__global__ void __launch_bounds__(kThreads) step_kernel(Args<E> a) {
  const int64_t b = blockIdx.x;
  const int d = blockIdx.y * kThreads + threadIdx.x;
  if (d >= a.dim) return;
  const int32_t slot = slot_of(a, b);
  float s = 0.f;
  if (slot >= 0) {
    const Gate k = gate_of(E::load(a.g + b * a.g_stride + d));
    s = fmaf(k.f, a.state[static_cast<int64_t>(slot) * a.dim + d], k.u * E::load(a.x + b * a.x_stride + d));
    a.state_out[static_cast<int64_t>(slot) * a.dim + d] = s;
  }
  E::store(a.y + b * a.y_stride + d, s);
}

int check_common(int32_t type, int64_t n_tokens, int32_t dim, int64_t n_seqs, int64_t n_slots, bool has_state) {
  if (!train::known_type(type)) return fail(ENGRAM_E_INVALID, "type %d is not ENGRAM_T_BF16 or ENGRAM_T_F32", type);
  if (n_tokens < 0 || n_seqs < 0 || n_slots < 0) return fail(ENGRAM_E_INVALID, "negative size");
  if (dim < 1 || dim > (1 << 20)) return fail(ENGRAM_E_SHAPE, "dim %d not in [1, 2^20]", dim);
  if (n_tokens > 0x7fffffff || n_seqs > 0x7fffffff) return fail(ENGRAM_E_RANGE, "too many positions or sequences");
  if (has_state && n_slots < 1) return fail(ENGRAM_E_INVALID, "a state needs n_slots >= 1");
  return ENGRAM_OK;
}

int check_rows(const void* p, int32_t type, int64_t stride, int32_t dim, const char* name) {
  if (p == nullptr) return fail(ENGRAM_E_INVALID, "null device pointer: %s", name);
  if (stride < dim) return fail(ENGRAM_E_SHAPE, "row stride of %s below dim", name);
  if (!aligned(p, train::type_bytes(type))) return fail(ENGRAM_E_ALIGN, "%s must be aligned to its elements", name);
  return ENGRAM_OK;
}

template <class E>
int launch(const Args<E>& a, int what, int64_t rows, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(rows), (a.dim + kThreads - 1) / kThreads);
  if (what == 0)
    forward_kernel<E><<<grid, kThreads, 0, st>>>(a);
  else if (what == 1)
    backward_kernel<E><<<grid, kThreads, 0, st>>>(a);
  else
    step_kernel<E><<<grid, kThreads, 0, st>>>(a);
  return check_launch("recurrence");
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
  return 256;
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
    a.dim = dim;
    a.status = status_d;
    return launch<E>(a, 0, n_seqs, as_stream(stream));
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
    a.dim = dim;
    a.status = status_d;
    return launch<E>(a, 1, n_seqs, as_stream(stream));
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
    return launch<E>(a, 2, batch, as_stream(stream));
  };
  return type == ENGRAM_T_BF16 ? go(train::Bf16{}) : go(train::F32{});
}
