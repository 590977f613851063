// Device pieces of the 16-bit dense product: the matrix instruction of either type
// and the epilogue.
#pragma once

#include "device_common.h"

namespace chord {

typedef __attribute__((ext_vector_type(8))) _Float16 f16x8_t;

// Eight neighbouring values along K.
union Operand {
  uint16_t h[8];
  u32x4_t u;
};

template <bool F16>
__device__ __forceinline__ f32x4_t mfma(const Operand& a, const Operand& b, f32x4_t c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a.u), __builtin_bit_cast(f16x8_t, b.u),
                                                  c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a.u),
                                                   __builtin_bit_cast(bf16x8_t, b.u), c, 0, 0, 0);
}

// Activation in fp32.  The results are rounded to 16 bits, or stand beside sums of
// products whose own error in fp32 is larger.
__device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    case CHORD_ACT_RELU: return z > 0.f ? z : z < 0.f ? 0.f : z;  // (NaN stays)
    case CHORD_ACT_SILU: return z / (1.f + expf(-z));
    case CHORD_ACT_GELU:  // (erfc has no cancellation where the result is small)
      return 0.5f * z * erfcf(z * -0.70710678118654752f);
    case CHORD_ACT_GELU_TANH:  // (1 + tanh y) / 2 = 1 / (1 + e^-2y)
      return z / (1.f + expf(-1.5957691216057308f * (z + 0.044715f * z * z * z)));
    default: return z;
  }
}

__device__ __forceinline__ float value16(uint16_t h, bool f16) {
  return f16 ? (float)__builtin_bit_cast(_Float16, h) : bf16_to_f32(h);
}
__device__ __forceinline__ uint16_t round16(float v, bool f16) {
  return f16 ? __builtin_bit_cast(uint16_t, (_Float16)v) : to_bf16(v);
}
__device__ __forceinline__ float bias_at(const LinearArgs& a, int64_t n) {
  if (a.bias == nullptr) return 0.f;
  return a.bias_f32 ? static_cast<const float*>(a.bias)[n] : value16(static_cast<const uint16_t*>(a.bias)[n], a.f16);
}

// One output from its sums over K (up: the up row's, where gated).
__device__ __forceinline__ void store_out(const LinearArgs& a, int64_t m, int n, float z, float up) {
  float h = activate(a.act, z + bias_at(a, n));
  if (a.gated) h *= up + bias_at(a, (int64_t)a.N + n);
  h *= a.scale;
  if (a.out_f32) {
    if (a.residual != nullptr) h += static_cast<const float*>(a.residual)[m * a.ldr + n];
    static_cast<float*>(a.out)[m * a.ldo + n] = h;
  } else {
    if (a.residual != nullptr) h += value16(static_cast<const uint16_t*>(a.residual)[m * a.ldr + n], a.f16);
    static_cast<uint16_t*>(a.out)[m * a.ldo + n] = round16(h, a.f16);
  }
}

}  // namespace chord
