// Four consecutive values as one load or store (8 bytes of bf16, 16 of fp32), widened to fp32
// registers.
#pragma once

#include "gdn_device.h"

namespace gdn {

template <typename E>
struct Vec4 {
  typedef E raw __attribute__((ext_vector_type(4)));
  static __device__ __forceinline__ raw load_raw(const E* p) {
    return *reinterpret_cast<const raw*>(p);
  }
  static __device__ __forceinline__ void wide(const raw& r, float* out) {
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = (float)r[i];
  }
  static __device__ __forceinline__ void load(const E* p, float* out) { wide(load_raw(p), out); }
  static __device__ __forceinline__ void store(E* p, const float* in) {
    raw v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (E)in[i];
    *reinterpret_cast<raw*>(p) = v;
  }
};

}  // namespace gdn
