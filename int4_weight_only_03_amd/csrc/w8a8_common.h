// Device code shared by the 8-bit operators: loads of 8 activations, a group of 128's
// largest magnitude, its scale and codes, codes to fp16.
#pragma once

#include "moe_common.h"
#include "w8a8_internal.h"

namespace w4a16 {
namespace {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kLanes8 = 16;  // lanes of a group of 128 values, 8 each

// 8 codes to fp16, exactly
__device__ __forceinline__ half8v widen8(uint32_t lo, uint32_t hi) {
  const half2v a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false),
               b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true),
               c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false),
               d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
  return half8v{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}
__device__ __forceinline__ void load8(const _Float16 *p, float (&v)[8]) {
  const half8v a = *reinterpret_cast<const half8v *>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = float(a[i]);
}
__device__ __forceinline__ void load8(const Bf16 *p, float (&v)[8]) {
  const u32x4m a = *reinterpret_cast<const u32x4m *>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(a[i] << 16);
    v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
  }
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8]) {
  struct alignas(16) Eight {
    T v[8];
  } e;
#pragma unroll
  for (int i = 0; i < 8; ++i) e.v[i] = from_f32<T>(v[i]);
  *reinterpret_cast<Eight *>(p) = e;
}

// The largest of `m` over the 16 lanes of a DPP row, in all of them.
__device__ __forceinline__ uint32_t row_max(uint32_t m) {
  m = max(m, uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0x128, 0xf, 0xf, true)));  // row_ror:8
  m = max(m, uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0x124, 0xf, 0xf, true)));
  m = max(m, uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0x122, 0xf, 0xf, true)));
  m = max(m, uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0x121, 0xf, 0xf, true)));
  return m;
}

// Codes of a group's values, 8 to a lane, and the group's scale.  Every one of the
// group's 16 lanes has to call it (those behind the row's end with zeros).
// Magnitudes are compared as integers, so that a NaN is the largest of all.
// v / scale: v times the reciprocal, mended by its remainder, which is the quotient rounded to
// fp32 but once in 10^8 (v * f alone is 2^-22 off at most and, near a tie of e4m3, on the
// other side of it four times as often).  The largest value's is at most 448 (1 + 2^-23), which rounds
// to 448.
__device__ __forceinline__ uint2 quantize8(const float (&v)[8], float &scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  m = row_max(m);
  float s = fmaxf(__uint_as_float(m) / 448.0f, 0x1p-126f);
  if (m >= 0x7f800000u) s = __builtin_nanf("");
  if (m == 0) s = 0.0f;
  scale = s;
  const float f = m == 0 ? 0.0f : __builtin_amdgcn_rcpf(s);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[i] = v[i] * f;
    q[i] = fmaf(fmaf(-q[i], s, v[i]), f, q[i]);
  }
  int a = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  a = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], a, true);
  int b = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], b, true);
  return make_uint2(uint32_t(a), uint32_t(b));
}

}  // namespace
}  // namespace w4a16
