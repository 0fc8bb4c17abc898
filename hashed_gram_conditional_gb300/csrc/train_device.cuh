// Element access shared by the training operators: bf16 and fp32 arrays read
// and written as fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "engram_internal.h"

namespace engram {
namespace train {

struct Bf16 {
  using T = uint16_t;
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ float load(const T* p) {
    return __uint_as_float(static_cast<uint32_t>(*p) << 16);
  }
  static __device__ __forceinline__ void store(T* p, float v) {
    *p = __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
};

struct F32 {
  using T = float;
  static constexpr int kBytes = 4;
  static __device__ __forceinline__ float load(const T* p) { return *p; }
  static __device__ __forceinline__ void store(T* p, float v) { *p = v; }
};

inline bool known_type(int32_t type) { return type == ENGRAM_T_BF16 || type == ENGRAM_T_F32; }
inline int type_bytes(int32_t type) { return type == ENGRAM_T_BF16 ? 2 : 4; }

inline size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace train
}  // namespace engram
