// Eight consecutive values of bf16 or fp32 as one 16-byte load or store (two for fp32), widened to
// fp32 registers.
#pragma once

#include "gdn_device.h"

namespace gdn {

template <typename E> struct Vec8;

template <> struct Vec8<bf16> {
  typedef bf16x8 raw;
  static __device__ __forceinline__ raw load_raw(const bf16* p) {
    return *reinterpret_cast<const bf16x8*>(p);
  }
  static __device__ __forceinline__ void wide(const raw& r, float* out) {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = (float)r[i];
  }
  static __device__ __forceinline__ void load(const bf16* p, float* out) { wide(load_raw(p), out); }
  static __device__ __forceinline__ void store(bf16* p, const float* in) {
    bf16x8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (bf16)in[i];
    *reinterpret_cast<bf16x8*>(p) = v;
  }
};

template <> struct Vec8<float> {
  struct raw {
    f32x4 a, b;
  };
  static __device__ __forceinline__ raw load_raw(const float* p) {
    return raw{reinterpret_cast<const f32x4*>(p)[0], reinterpret_cast<const f32x4*>(p)[1]};
  }
  static __device__ __forceinline__ void wide(const raw& r, float* out) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      out[i] = r.a[i];
      out[i + 4] = r.b[i];
    }
  }
  static __device__ __forceinline__ void load(const float* p, float* out) { wide(load_raw(p), out); }
  static __device__ __forceinline__ void store(float* p, const float* in) {
    reinterpret_cast<f32x4*>(p)[0] = f32x4{in[0], in[1], in[2], in[3]};
    reinterpret_cast<f32x4*>(p)[1] = f32x4{in[4], in[5], in[6], in[7]};
  }
};

// Four consecutive values: 8 bytes of bf16, 16 of fp32.
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
