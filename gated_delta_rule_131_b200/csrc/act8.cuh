// Activations held in 8 bits, and the vector accesses of the training operators.
//
// A row of channels is held as one signed 8-bit code per channel and one scale byte for every 32
// channels (the last group of a row may be shorter).  The scale is the least power of two 2^e with
// max |x| <= 127 * 2^e over the group, stored as the fp32 exponent field of 2^e (e + 127, at least 1);
// the code is x / 2^e rounded to the nearest integer, ties to even.  A power of two makes the
// scaling exact, so the only error is that one rounding, there is no division, and a code times its scale
// is exact in fp32 and in bf16.  Finite values above 127 * 2^121, which would round up to infinity, are
// held as that.  The error is at most 2^(e-1), or 2^121 for a value above 127 * 2^121; either is under 1/127
// of the group's largest value, as long as that is above 127 * 2^-127.  In a group below it e stays at -126:
// the error is at most 2^-127, which may be all of a value.  A group that
// holds an infinity or a NaN has the scale byte 255 and zero codes, and reads back as NaN.
#pragma once

#include <cooperative_groups.h>

#include <atomic>

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

// N values as fp32 pairs: sums, products and fused multiply-adds run two to an instruction.
template <int N> struct Pairs {
  static_assert(N % 2 == 0, "whole pairs");
  float2 p[N / 2];
  __device__ __forceinline__ float get(int i) const { return i & 1 ? p[i >> 1].y : p[i >> 1].x; }
  __device__ __forceinline__ void set(int i, float v) { (i & 1 ? p[i >> 1].y : p[i >> 1].x) = v; }
};
__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }
template <int N> __device__ __forceinline__ void fill(Pairs<N> &a, float x) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) a.p[i] = splat(x);
}
template <int N> __device__ __forceinline__ float total(const Pairs<N> &a) {
  float2 s = a.p[0];
#pragma unroll
  for (int i = 1; i < N / 2; ++i) s = __fadd2_rn(s, a.p[i]);
  return s.x + s.y;
}
template <int N> __device__ __forceinline__ float dot(const Pairs<N> &a, const Pairs<N> &b) {
  float2 s = __fmul2_rn(a.p[0], b.p[0]);
#pragma unroll
  for (int i = 1; i < N / 2; ++i) s = __ffma2_rn(a.p[i], b.p[i], s);
  return s.x + s.y;
}

// 32 bytes at once (on a 32-byte boundary), marked first to leave the L2 where STREAM.
struct alignas(32) Words8 { uint32_t w[8]; };
template <bool STREAM> __device__ __forceinline__ Words8 load32(const void *p) {
  Words8 v;
  if constexpr (STREAM)
    asm volatile("ld.global.cs.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7])
                 : "l"(p) : "memory");
  else
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7])
                 : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void store32(void *p, const Words8 &v) {
  asm volatile("st.global.cs.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v.w[0]), "r"(v.w[1]), "r"(v.w[2]),
               "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]), "r"(v.w[7])
               : "memory");
}

// VEC consecutive values of one lane, in memory.  Streams are read and written once: `load` and
// `store` mark their lines first to leave the L2.
template <typename T, int VEC> struct alignas(sizeof(T) * VEC) LaneVec {
  T e[VEC];
  static constexpr int BYTES = sizeof(T) * VEC;
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (BYTES == 32) *reinterpret_cast<Words8 *>(this) = load32<true>(p);
    else if constexpr (BYTES == 16) *reinterpret_cast<uint4 *>(this) = __ldcs(reinterpret_cast<const uint4 *>(p));
    else if constexpr (BYTES == 8) *reinterpret_cast<uint2 *>(this) = __ldcs(reinterpret_cast<const uint2 *>(p));
    else if constexpr (BYTES == 4) *reinterpret_cast<uint32_t *>(this) = __ldcs(reinterpret_cast<const uint32_t *>(p));
    else if constexpr (BYTES == 2) *reinterpret_cast<uint16_t *>(this) = __ldcs(reinterpret_cast<const uint16_t *>(p));
    else *reinterpret_cast<uint8_t *>(this) = __ldcs(reinterpret_cast<const uint8_t *>(p));
  }
  // The same through the L1 as usual.
  __device__ __forceinline__ void load_cached(const T *p) {
    if constexpr (BYTES == 32) *reinterpret_cast<Words8 *>(this) = load32<false>(p);
    else *this = *reinterpret_cast<const LaneVec *>(p);
  }
  __device__ __forceinline__ void store(T *p) const {
    if constexpr (BYTES == 32) store32(p, *reinterpret_cast<const Words8 *>(this));
    else if constexpr (BYTES == 16) __stcs(reinterpret_cast<uint4 *>(p), *reinterpret_cast<const uint4 *>(this));
    else if constexpr (BYTES == 8) __stcs(reinterpret_cast<uint2 *>(p), *reinterpret_cast<const uint2 *>(this));
    else if constexpr (BYTES == 4) __stcs(reinterpret_cast<uint32_t *>(p), *reinterpret_cast<const uint32_t *>(this));
    else if constexpr (BYTES == 2) __stcs(reinterpret_cast<uint16_t *>(p), *reinterpret_cast<const uint16_t *>(this));
    else __stcs(reinterpret_cast<uint8_t *>(p), *reinterpret_cast<const uint8_t *>(this));
  }
};
// Whether every one of the given pointers lies on a 32-byte boundary.
template <typename... P> inline bool on32(const P *...p) { return ((reinterpret_cast<uintptr_t>(p) | ...) & 31u) == 0; }

// Values AT .. AT + VEC - 1 of `f` from a lane's vector; codes are multiplied by their group's unit.
template <int AT, int VEC, int N>
__device__ __forceinline__ void widen(const LaneVec<float, VEC> &r, Pairs<N> &f) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) f.set(AT + i, r.e[i]);
}
template <int AT, int VEC, int N>
__device__ __forceinline__ void widen(const LaneVec<__nv_bfloat16, VEC> &r, Pairs<N> &f) {
  if constexpr (VEC % 2 == 0) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&r);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i)  // a bf16 is the top half of the fp32 of the same value
      f.p[AT / 2 + i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  } else {
    f.set(AT, __bfloat162float(r.e[0]));
  }
}
// Each byte of the codes, offset by 128, becomes the low mantissa byte of 2^23 + 128 + code; the
// difference and the product are exact.
template <int AT, int VEC, int N>
__device__ __forceinline__ void widen(const LaneVec<int8_t, VEC> &r, float unit, Pairs<N> &f) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int k = 0; k < VEC / 4; ++k) {
      const uint32_t o = reinterpret_cast<const uint32_t *>(&r)[k] ^ 0x80808080u;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 v = make_float2(__uint_as_float(__byte_perm(o, 0x4b000000u, 0x7440 + 2 * i)),
                                     __uint_as_float(__byte_perm(o, 0x4b000000u, 0x7441 + 2 * i)));
        f.p[AT / 2 + 2 * k + i] = __fmul2_rn(__fadd2_rn(v, splat(-8388736.f)), splat(unit));
      }
    }
  } else {
    f.set(AT, (float)r.e[0] * unit);
  }
}
template <int AT, int VEC, int N>
__device__ __forceinline__ void narrow(const Pairs<N> &f, LaneVec<float, VEC> &r) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) r.e[i] = f.get(AT + i);
}
template <int AT, int VEC, int N>
__device__ __forceinline__ void narrow(const Pairs<N> &f, LaneVec<__nv_bfloat16, VEC> &r) {
  if constexpr (VEC % 2 == 0) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) reinterpret_cast<__nv_bfloat162 *>(&r)[i] = __float22bfloat162_rn(f.p[AT / 2 + i]);
  } else {
    r.e[0] = __float2bfloat16_rn(f.get(AT));
  }
}

// The largest |x| bit pattern of a lane's vector.
template <int VEC>
__device__ __forceinline__ uint32_t amax_bits(const LaneVec<float, VEC> &r) {
  uint32_t m = __float_as_uint(r.e[0]) & 0x7fffffffu;
#pragma unroll
  for (int i = 1; i < VEC; ++i) m = max(m, __float_as_uint(r.e[i]) & 0x7fffffffu);
  return m;
}
template <int VEC>
__device__ __forceinline__ uint32_t amax_bits(const LaneVec<__nv_bfloat16, VEC> &r) {
  if constexpr (VEC % 2 == 0) {  // two 15-bit patterns to a word
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&r);
    uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < VEC / 2; i += 2)
      m = __vimax3_s16x2(m, w[i] & 0x7fff7fffu, w[i + 1 < VEC / 2 ? i + 1 : i] & 0x7fff7fffu);
    return max(m & 0xffff0000u, m << 16);
  } else {
    return (uint32_t)(__bfloat16_as_ushort(r.e[0]) & 0x7fffu) << 16;
  }
}

// The codes of a lane's vector r (`x` holds its values at AT onwards) and their group's scale byte;
// the 32 / VEC lanes that hold a group are consecutive and aligned, and the whole warp calls this
// together, a lane past its row's end with inside == false.  Adding 1.5 * 2^23 to x / scale leaves its
// integer part in the last mantissa bits, rounded once by the fused multiply-add, ties to even.
template <int AT, typename T, int VEC, int N>
__device__ __forceinline__ LaneVec<int8_t, VEC> act8_encode(const LaneVec<T, VEC> &r, const Pairs<N> &x, bool inside,
                                                            uint32_t &scale) {
  constexpr uint32_t TOP = 0x7f7e0000u;  // 127 * 2^121
  uint32_t amax = inside ? amax_bits(r) : 0;
#pragma unroll
  for (int m = 1; m < ACT_GROUP / VEC; m <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  float2 v[(VEC + 1) / 2];
#pragma unroll
  for (int i = 0; i < (VEC + 1) / 2; ++i) v[i] = VEC == 1 ? make_float2(x.get(AT), 0.f) : x.p[AT / 2 + i];
  if (amax > TOP && amax < 0x7f800000u) {  // hardly ever
    const float t = __uint_as_float(TOP);
#pragma unroll
    for (int i = 0; i < (VEC + 1) / 2; ++i)
      v[i] = make_float2(fminf(fmaxf(v[i].x, -t), t), fminf(fmaxf(v[i].y, -t), t));
    amax = TOP;
  }
  scale = act8_scale(amax);
  const float2 inv = splat(act8_inverse(scale));
  uint32_t q[VEC + 1];
#pragma unroll
  for (int i = 0; i < (VEC + 1) / 2; ++i) {
    const float2 c = __ffma2_rn(v[i], inv, splat(12582912.f));
    q[2 * i] = __float_as_uint(c.x);
    q[2 * i + 1] = __float_as_uint(c.y);
  }
  LaneVec<int8_t, VEC> c;
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const uint32_t lo = __byte_perm(q[4 * i], q[4 * i + 1], 0x0040), hi = __byte_perm(q[4 * i + 2], q[4 * i + 3], 0x0040);
      reinterpret_cast<uint32_t *>(&c)[i] = scale == 255u ? 0u : __byte_perm(lo, hi, 0x5410);
    }
  } else {
    c.e[0] = scale == 255u ? 0 : (int8_t)q[0];
  }
  return c;
}

// N fp32 values that every row reads (weights), VEC at a time.
template <int AT, int VEC, int N>
__device__ __forceinline__ void load_f32(const float *p, Pairs<N> &f) {
  if constexpr (VEC % 4 == 0) {  // p on a 16-byte boundary
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const float4 q = *reinterpret_cast<const float4 *>(p + i);
      f.p[(AT + i) / 2] = make_float2(q.x, q.y);
      f.p[(AT + i) / 2 + 1] = make_float2(q.z, q.w);
    }
  } else {
    f.set(AT, p[0]);
  }
}
template <int AT, int VEC, int N>
__device__ __forceinline__ void store_f32(const Pairs<N> &f, float *p) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4)
      *reinterpret_cast<float4 *>(p + i) = make_float4(f.p[(AT + i) / 2].x, f.p[(AT + i) / 2].y, f.p[(AT + i) / 2 + 1].x,
                                                       f.p[(AT + i) / 2 + 1].y);
  } else {
    p[0] = f.get(AT);
  }
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

// A short call needs no rows of partial sums: its blocks, launched as one cluster of CLUSTER_BLOCKS (some
// perhaps without rows), add their sums, each block's `n` floats at the same place of its shared memory,
// through it, in the order of their ranks, column by column into at most two outputs.  That saves the
// second launch and the workspace, 4 of 17 us of the host's time.
constexpr int CLUSTER_BLOCKS = 8;  // what every GPU of this kind can launch
__device__ __forceinline__ void cluster_sum(float *sums, int n, float *out0, int end0, float *out1) {
  const auto cluster = cooperative_groups::this_cluster();
  cluster.sync();
  for (int c = cluster.block_rank() * blockDim.x + threadIdx.x; c < n; c += CLUSTER_BLOCKS * blockDim.x) {
    float v[CLUSTER_BLOCKS], s = 0.f;
#pragma unroll
    for (int r = 0; r < CLUSTER_BLOCKS; ++r) v[r] = cluster.map_shared_rank(sums, r)[c];
#pragma unroll
    for (int r = 0; r < CLUSTER_BLOCKS; ++r) s += v[r];
    if (c < end0) out0[c] = s;
    else if (out1) out1[c - end0] = s;
  }
  cluster.sync();  // no block leaves while another reads its memory
}
template <typename... P, typename... A>
cudaError_t launch_cluster(void (*kernel)(P...), int threads, int smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {CLUSTER_BLOCKS, 1, 1};
  cfg.gridDim = dim3(CLUSTER_BLOCKS);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Raises a kernel's limit of dynamic shared memory to `bytes`, always the same for a kernel, on the
// current device; `devices` remembers where that is done (one bit per device).
cudaError_t allow_smem(const void *kernel, int bytes, std::atomic<uint64_t> &devices);

}  // namespace gdn2
