// Activations held in 8 bits, and the vector accesses of the training operators.
//
// A row of channels is held as one signed 8-bit code per channel and one scale byte for every 32
// channels (the last group of a row may be shorter).  The scale is the least power of two 2^e with
// max |x| <= 127 * 2^e over the group, stored as the fp32 exponent field of 2^e (e + 127, at least 1);
// the code is x / 2^e rounded to the nearest integer, ties to even.  A power of two makes the
// scaling exact, so the only error is that one rounding (at most 2^(e-1), under 1/126 of the group's
// largest value), there is no division, and a code times its scale is exact in fp32 and in bf16.
// Finite values above 127 * 2^121, which would round up to infinity, are held as that.  A group that
// holds an infinity or a NaN has the scale byte 255 and zero codes, and reads back as NaN.
#pragma once

#include "common.cuh"

namespace gdn2 {

constexpr int ACT_GROUP = 32;  // channels that share a scale

// The scale byte of a group from the largest |x| bit pattern in it (NaN > inf > finite, as integers).
__device__ __forceinline__ uint32_t act8_scale(uint32_t amax_bits) {
  const int p = (int)(amax_bits >> 23);  // 127 * 2^e = 1.984375 * 2^(e+6): mantissas above .984375 need e + 1
  const int e = p - 6 + ((amax_bits & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return p == 255 ? 255u : (uint32_t)max(e, 1);
}
// 1 / scale (a power of two, exact); 0 for the NaN scale.
__device__ __forceinline__ float act8_inverse(uint32_t s) { return s == 255u ? 0.f : __uint_as_float((254u - s) << 23); }
// The scale itself; +inf for the NaN scale, which the zero codes turn into NaN.
__device__ __forceinline__ float act8_unit(uint32_t s) { return __uint_as_float(s << 23); }

// x / scale rounded to an integer in the low byte: adding 1.5 * 2^23 leaves the integer part in the
// last mantissa bits, rounded once by the fused multiply-add, ties to even.
__device__ __forceinline__ uint32_t act8_round(float x, float inv) {
  return __float_as_uint(fmaf(x, inv, 12582912.f));
}
__device__ __forceinline__ uint32_t act8_code4(const float *x, float inv) {
  const uint32_t lo = __byte_perm(act8_round(x[0], inv), act8_round(x[1], inv), 0x0040);
  const uint32_t hi = __byte_perm(act8_round(x[2], inv), act8_round(x[3], inv), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}
// Four codes of a word times their unit: each byte (offset by 128) becomes the low mantissa byte of
// 2^23 + 128 + code; the difference and the product are exact.
__device__ __forceinline__ void act8_value4(uint32_t w, float unit, float *x) {
  const uint32_t o = w ^ 0x80808080u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = (__uint_as_float(__byte_perm(o, 0x4b000000u, 0x7440 + i)) - 8388736.f) * unit;
}

// VEC consecutive values of one lane, in memory.
template <typename T, int VEC> struct alignas(sizeof(T) * VEC) LaneVec { T e[VEC]; };

template <int VEC>
__device__ __forceinline__ void widen(const LaneVec<float, VEC> &r, float (&f)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) f[i] = r.e[i];
}
template <int VEC>
__device__ __forceinline__ void widen(const LaneVec<__nv_bfloat16, VEC> &r, float (&f)[VEC]) {
  if constexpr (VEC % 2 == 0) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&r);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {  // a bf16 is the top half of the fp32 of the same value
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = __bfloat162float(r.e[i]);
  }
}
template <int VEC>
__device__ __forceinline__ void widen(const LaneVec<int8_t, VEC> &r, float unit, float (&f)[VEC]) {
  if constexpr (VEC % 4 == 0) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&r);
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) act8_value4(w[i], unit, f + 4 * i);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = (float)r.e[i] * unit;
  }
}
template <int VEC>
__device__ __forceinline__ void narrow(const float (&f)[VEC], LaneVec<float, VEC> &r) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) r.e[i] = f[i];
}
template <int VEC>
__device__ __forceinline__ void narrow(const float (&f)[VEC], LaneVec<__nv_bfloat16, VEC> &r) {
  if constexpr (VEC % 2 == 0) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i)
      reinterpret_cast<__nv_bfloat162 *>(&r)[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) r.e[i] = __float2bfloat16_rn(f[i]);
  }
}

// VEC consecutive fp32 values, 16 bytes at a time where VEC allows (p then on a 16-byte boundary).
template <int VEC>
__device__ __forceinline__ void load_f32(const float *p, float (&f)[VEC]) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const float4 q = *reinterpret_cast<const float4 *>(p + i);
      f[i] = q.x;
      f[i + 1] = q.y;
      f[i + 2] = q.z;
      f[i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = p[i];
  }
}
template <int VEC>
__device__ __forceinline__ void store_f32(const float (&f)[VEC], float *p) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) *reinterpret_cast<float4 *>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p[i] = f[i];
  }
}

// The codes of a lane's VEC values and their group's scale byte; the 32 / VEC lanes that hold a
// group are consecutive and aligned, and the whole warp calls this together (values past a row's
// end are passed as 0).
template <int VEC>
__device__ __forceinline__ LaneVec<int8_t, VEC> act8_encode(const float (&x)[VEC], uint32_t &scale) {
  constexpr uint32_t TOP = 0x7f7e0000u;  // 127 * 2^121
  uint32_t amax = 0;
  float f[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    f[i] = x[i];
    amax = max(amax, __float_as_uint(f[i]) & 0x7fffffffu);
  }
#pragma unroll
  for (int m = 1; m < ACT_GROUP / VEC; m <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  if (amax > TOP && amax < 0x7f800000u) {
    amax = TOP;
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = fminf(fmaxf(f[i], -__uint_as_float(TOP)), __uint_as_float(TOP));
  }
  scale = act8_scale(amax);
  const float inv = act8_inverse(scale);
  LaneVec<int8_t, VEC> c;
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i)
      reinterpret_cast<uint32_t *>(&c)[i] = scale == 255u ? 0u : act8_code4(f + 4 * i, inv);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) c.e[i] = scale == 255u ? 0 : (int8_t)act8_round(f[i], inv);
  }
  return c;
}

// Sums of `parts` rows of `ncols` fp32 partial results, column by column in a fixed order, into up to
// three outputs that follow one another along the columns (defined in act8.cu).  It is launched as
// the programmatic dependent of the kernel that writes the rows.
struct ColSumArgs {
  const float *parts;
  int nparts, ncols;
  float *out[3];  // a null output's columns are skipped
  int end[3];     // first column past each output
};
cudaError_t launch_colsum(const ColSumArgs &a, cudaStream_t stream);

}  // namespace gdn2
