// Device pieces of the 16-bit dense product: loads, the matrix instruction of either
// type, and the epilogue.
#pragma once

#include "device_common.h"

namespace chord {

typedef __attribute__((ext_vector_type(8))) _Float16 f16x8_t;

constexpr int kLinRsrcWord3 = 0x00020000;
constexpr uint32_t kLinNothing = 0xC0000000u;  // byte offset past any buffer: reads as zeros

template <bool F16>
__device__ __forceinline__ f32x4_t mfma16(u32x4_t a, u32x4_t b, f32x4_t c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c,
                                                  0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// Buffer over `rows` rows of K values, `ld` apart.  Without rows, whose lanes all ask for
// kLinNothing, it is as long as one: a load's range check takes the offset of its chunk
// off the length, which has to stay positive.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const uint16_t* p, int64_t rows, int64_t ld, int K) {
  const int64_t bytes = ((rows > 0 ? rows - 1 : 0) * ld + K) * 2;
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)bytes, kLinRsrcWord3);
}

// All waves' LDS accesses before it are done; loads and stores of memory go on.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// z / (1 + e^-y) with the hardware's exponential and reciprocal (about a unit of 2^-24
// each, and of the exponent's argument y one for each unit of y).  Of h = e^(-|y| / 2),
// below 0 as z h h / (1 + h h): e^-y leaves fp32 below -88, and its reciprocal the normal
// numbers before that, where the result is still there.
__device__ __forceinline__ float gate_of(float z, float y) {
  const float h = __expf(-0.5f * fabsf(y)), r = __builtin_amdgcn_rcpf(__builtin_fmaf(h, h, 1.f));
  return (y < 0.f ? z * h * h : z) * r;
}
// The activations of a few instructions (all but GELU).
__device__ __forceinline__ float activate_short(int act, float z) {
  if (act == CHORD_ACT_SILU) return gate_of(z, z);
  if (act == CHORD_ACT_GELU_TANH)  // (1 + tanh y) / 2 = 1 / (1 + e^-2y)
    return gate_of(z, 1.5957691216057308f * (z + 0.044715f * z * z * z));
  return z > 0.f ? z : z < 0.f ? 0.f : z;  // RELU (NaN stays)
}
// Activation in fp32.  The results are rounded to 16 bits, or stand beside sums of
// products whose own error in fp32 is larger.
__device__ __forceinline__ float activate(int act, float z) {
  if (act == CHORD_ACT_NONE) return z;
  if (act == CHORD_ACT_GELU)  // (erfc has no cancellation where the result is small)
    return 0.5f * z * erfcf(z * -0.70710678118654752f);
  return activate_short(act, z);
}

__device__ __forceinline__ float value16(uint32_t h, bool f16) {
  return f16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)h) : bf16_to_f32(h);
}
__device__ __forceinline__ uint16_t round16(float v, bool f16) {
  return f16 ? __builtin_bit_cast(uint16_t, (_Float16)v) : to_bf16(v);
}
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (F16) {
    half2_t r;
    r[0] = (_Float16)a;
    r[1] = (_Float16)b;
    return __builtin_bit_cast(uint32_t, r);
  } else {
    return pk_bf16(a, b);
  }
}
__device__ __forceinline__ uint32_t round16x2(float a, float b, bool f16) {
  return (uint32_t)round16(a, f16) | (uint32_t)round16(b, f16) << 16;
}

// n (of four) neighbouring values of 16 bits or fp32 at p[i], by words where `wide`.
__device__ __forceinline__ f32x4_t load4(const void* p, int64_t i, bool f32, bool f16, bool wide, int n) {
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  if (f32) {
    const float* q = static_cast<const float*>(p) + i;
    if (wide) return *reinterpret_cast<const f32x4_t*>(q);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) v[j] = q[j];
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
    if (wide) {
      const uint2 u = *reinterpret_cast<const uint2*>(q);
      return f32x4_t{value16(u.x & 0xFFFF, f16), value16(u.x >> 16, f16), value16(u.y & 0xFFFF, f16),
                     value16(u.y >> 16, f16)};
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) v[j] = value16(q[j], f16);
  }
  return v;
}

// The outputs n .. n + 3 (those below N) of any row: what does not depend on the row.
struct OutQuad {
  int n, left;
  bool whole, wide_res, wide_out;
  f32x4_t bias, bias_up;
};
__device__ __forceinline__ OutQuad out_quad(const LinearArgs& a, int n) {
  OutQuad o;
  o.n = n;
  o.left = a.N - n;
  o.whole = o.left >= 4;
  o.wide_res = o.whole && (a.wide & kLinWideResidual);
  o.wide_out = o.whole && (a.wide & kLinWideOut);
  o.bias = o.bias_up = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (a.bias != nullptr && o.left > 0) {
    const bool wide = o.whole && (a.wide & kLinWideBias);
    o.bias = load4(a.bias, n, a.bias_f32, a.f16, wide, o.left);
    if (a.gated) o.bias_up = load4(a.bias, (int64_t)a.N + n, a.bias_f32, a.f16, wide && a.N % 4 == 0, o.left);
  }
  return o;
}
__device__ __forceinline__ f32x4_t out_residual(const LinearArgs& a, const OutQuad& o, int64_t m) {
  if (a.residual == nullptr) return f32x4_t{0.f, 0.f, 0.f, 0.f};
  return load4(a.residual, m * a.ldr + o.n, a.out_f32, a.f16, o.wide_res, o.left);
}
// The residual as it lies in memory (wide_res; 16-bit values in the first two words), so
// that many loads can be on their way before the first is looked at.
template <bool F32>
__device__ __forceinline__ u32x4_t raw_residual(const LinearArgs& a, const OutQuad& o, int64_t m) {
  if (F32) return *reinterpret_cast<const u32x4_t*>(static_cast<const float*>(a.residual) + m * a.ldr + o.n);
  const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.residual) + m * a.ldr + o.n);
  return u32x4_t{u.x, u.y, 0u, 0u};
}
__device__ __forceinline__ f32x4_t residual_value(const LinearArgs& a, u32x4_t r) {
  if (a.out_f32) return __builtin_bit_cast(f32x4_t, r);
  return f32x4_t{value16(r[0] & 0xFFFF, a.f16), value16(r[0] >> 16, a.f16), value16(r[1] & 0xFFFF, a.f16),
                 value16(r[1] >> 16, a.f16)};
}
// From the sums over K; `up` holds the up rows' where gated.
__device__ __forceinline__ void out_store(const LinearArgs& a, const OutQuad& o, int64_t m, f32x4_t z, f32x4_t up,
                                          f32x4_t residual) {
  z += o.bias;
  if (a.act != CHORD_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = activate(a.act, z[i]);
  }
  if (a.gated) z *= up + o.bias_up;
  z = z * a.scale + residual;
  if (a.out_f32) {
    float* p = static_cast<float*>(a.out) + m * a.ldo + o.n;
    if (o.wide_out) {
      *reinterpret_cast<f32x4_t*>(p) = z;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < o.left) p[i] = z[i];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(a.out) + m * a.ldo + o.n;
    if (o.wide_out) {
      *reinterpret_cast<uint2*>(p) = make_uint2(round16x2(z[0], z[1], a.f16), round16x2(z[2], z[3], a.f16));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < o.left) p[i] = round16(z[i], a.f16);
    }
  }
}
__device__ __forceinline__ void store_out4(const LinearArgs& a, int64_t m, int n, f32x4_t z, f32x4_t up) {
  const OutQuad o = out_quad(a, n);
  if (o.left > 0) out_store(a, o, m, z, up, out_residual(a, o, m));
}

}  // namespace chord
