// q8.cuh -- activations in 8 bits: groups of 128 columns of a row, each with
// one power-of-two scale (fp32), values e4m3 or int8.
//
// The scale of a group is the smallest power of two s >= 2^-100 with
// amax <= s * (448 for e4m3, 127 for int8).  A power of two costs no extra
// rounding: v / s is exact, the one rounding is to the 8-bit format (nearest
// even), and q * s has at most 8 significant bits, so a stored value read
// back as bf16 is exact and the tensor-core products take it as it is.  A
// group that holds a NaN or an infinity gets the scale NaN and reads back as
// NaN: nothing non-finite turns into a number.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace pkm {

constexpr int kQ8Group = PKM_Q8_GROUP;
constexpr int kUnit = 8;                          // columns one thread handles at a time
constexpr int kGroupLanes = kQ8Group / kUnit;     // 16 consecutive lanes hold a group
constexpr int kQ8MinExp = -100;

__host__ __device__ inline int q8_groups(int d) { return (d + kQ8Group - 1) / kQ8Group; }

// 8 consecutive elements as fp32 (one 16-byte load for bf16, two for fp32).
// Plain loads, not the read-only path: several callers write in place.
template <pkm_dtype DT>
__device__ __forceinline__ void load8(const typename Elem<DT>::T* p, float* f) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  unpack16<DT>(a, f);
  if constexpr (DT == PKM_F32) {
    const uint4 b = *reinterpret_cast<const uint4*>(p + 4);
    unpack16<DT>(b, f + 4);
  }
}

// 8 consecutive elements as they are held: loads are issued for several
// units before the first is unpacked, and wait in half the registers.
template <pkm_dtype DT>
struct Raw8 {
  uint4 v[DT == PKM_F32 ? 2 : 1];
  __device__ __forceinline__ void zero() {
    v[0] = make_uint4(0, 0, 0, 0);
    if constexpr (DT == PKM_F32) v[1] = v[0];
  }
  __device__ __forceinline__ void load(const typename Elem<DT>::T* p) {
    v[0] = *reinterpret_cast<const uint4*>(p);
    if constexpr (DT == PKM_F32) v[1] = *reinterpret_cast<const uint4*>(p + 4);
  }
  __device__ __forceinline__ void unpack(float* f) const {
    unpack16<DT>(v[0], f);
    if constexpr (DT == PKM_F32) unpack16<DT>(v[1], f + 4);
  }
};

// fp32 -> 8 consecutive elements (one rounding)
template <pkm_dtype DT>
__device__ __forceinline__ void store8(typename Elem<DT>::T* p, const float* f) {
  *reinterpret_cast<uint4*>(p) = pack16<DT>(f);
  if constexpr (DT == PKM_F32) *reinterpret_cast<uint4*>(p + 4) = pack16<DT>(f + 4);
}

// The storage dtype's value of each element
template <pkm_dtype DT>
__device__ __forceinline__ void round8(float* f) {
  if constexpr (DT == PKM_BF16) {
    float r[8];
    unpack16<DT>(pack16<DT>(f), r);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = r[e];
  }
}

// Largest |v| over the lane's 8 values and its group's 16 lanes, as bits (a
// NaN or infinity compares above every finite value).  All 32 lanes call it;
// lanes past the row's end pass zeros.
__device__ __forceinline__ uint32_t group_amax_bits(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
#pragma unroll
  for (int o = kGroupLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// Exponent bits only: scale = 2^k; 448 = 1.75 * 2^8 and 127 = 1.984375 * 2^6.
__device__ __forceinline__ float q8_scale(uint32_t amax, pkm_q8 fmt) {
  if (amax >= 0x7f800000u) return __uint_as_float(0x7fffffffu);  // NaN
  const int e = (int)(amax >> 23) - 127;
  const uint32_t mant = amax & 0x7fffffu;
  int k = fmt == PKM_Q8_E4M3 ? e - 8 + (mant > 0x600000u) : e - 6 + (mant > 0x7e0000u);
  k = max(k, kQ8MinExp);
  return __uint_as_float((uint32_t)(k + 127) << 23);
}
// 1 / scale (exact: -100 <= k <= 122, the largest for int8 near the top of fp32)
__device__ __forceinline__ float q8_inverse(float scale) {
  const uint32_t b = __float_as_uint(scale);
  return b >= 0x7f800000u ? scale : __uint_as_float((254u << 23) - b);
}

__device__ __forceinline__ uint2 q8_encode(const float* v, float inv, pkm_q8 fmt) {
  uint32_t w[2];
  if (fmt == PKM_Q8_E4M3) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(
          make_float2(v[4 * h] * inv, v[4 * h + 1] * inv), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(
          make_float2(v[4 * h + 2] * inv, v[4 * h + 3] * inv), __NV_SATFINITE, __NV_E4M3);
      w[h] = lo | (hi << 16);
    }
  } else {
    // 1.5 * 2^23 + v / s rounds to an integer whose low byte is two's complement
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = __float_as_uint(fmaf(v[4 * h + e], inv, 12582912.0f));
      w[h] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    }
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void q8_decode(const uint2& q, float scale, pkm_q8 fmt, float* v) {
  const uint32_t w[2] = {q.x, q.y};
  if (fmt == PKM_Q8_E4M3) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(
          (__nv_fp8x2_storage_t)(w[h >> 1] >> (16 * (h & 1))), __NV_E4M3);
      const float2 f = __half22float2(__half2(r));
      v[2 * h] = f.x * scale;
      v[2 * h + 1] = f.y * scale;
    }
  } else {
    // a byte u = q + 128 put under the exponent of 2^23 is the fp32 number
    // 2^23 + u, from which 2^23 + 128 goes off exactly
    const float2 off = make_float2(-8388736.0f, -8388736.0f), s2 = make_float2(scale, scale);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const uint32_t u = w[e >> 2] ^ 0x80808080u;
      const float2 f = make_float2(
          __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440u | (e & 3))),
          __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440u | ((e + 1) & 3))));
      const float2 r = __fmul2_rn(__fadd2_rn(f, off), s2);
      v[e] = r.x;
      v[e + 1] = r.y;
    }
  }
}

}  // namespace pkm
