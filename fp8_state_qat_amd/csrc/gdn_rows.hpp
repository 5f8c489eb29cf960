// gdn_rows.hpp -- pieces of the row-wise kernels (activation codes, block
// norms): octets of eight consecutive columns, E4M3 codes of an octet, and
// sums over the threads that share a row.
#pragma once

#include "gdn_device.hpp"
#include "gdn_launch.hpp"

namespace gdn {

constexpr int kGroupCols = 64;  // columns that share one scale: the octets of 8 lanes

// Workgroups of one launch at most: a launch takes fewer than 2^32 threads in
// a dimension.  Larger calls go in several launches, rows after rows.
constexpr int64_t max_blocks(int threads) { return (((int64_t)1 << 32) - 1) / threads; }

// Eight consecutive columns of a row as fp32, n of them valid (the rest 0).
// kVec: every row starts at a multiple of 16 bytes and cols % 8 == 0, so an
// octet is whole or empty and moves in 16-byte accesses; else column by column.
template <typename T, bool kVec>
__device__ __forceinline__ void ld_oct(const T* p, int n, float (&x)[8]) {
  if constexpr (kVec) {
    if (n <= 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.0f;
    } else if constexpr (sizeof(T) == 2) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] = bf16_lo(w[j]);
        x[2 * j + 1] = bf16_hi(w[j]);
      }
    } else {
      const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
      x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = j < n ? io<T>::ld(p + j) : 0.0f;
  }
}

template <typename T, bool kVec>
__device__ __forceinline__ void st_oct(T* p, int n, const float (&x)[8]) {
  if constexpr (kVec) {
    if (n <= 0) return;
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    } else {
      reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) {
        if constexpr (sizeof(T) == 2) p[j] = (T)(pack_bf16x2(x[j], x[j]) & 0xffffu);
        else p[j] = x[j];
      }
  }
}

// Scale of a 64-column group from one octet of each of its 8 lanes: RN(amax /
// 448), 1 where that is not positive.
__device__ __forceinline__ float group_scale(const float (&x)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(x[j]));
  return qdq_scale_f64(lane8_max_dpp(m));
}

// E4M3 codes of an octet at scale s: RN(x / s) in fp32 (through the fp64
// quotient), then the nearest E4M3 value, ties to even.  Where s is
// subnormal x / s can exceed 448 by s's rounding, and the conversion would
// make that NaN: it is held at 448 (a normal s leaves at most 448 (1 + 2^-23),
// which converts to 448).  A NaN stays a NaN.
__device__ __forceinline__ uint2 e4m3_oct(const float (&x)[8], float s) {
  const double r = rcp_f64(s);
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = div_rn_f64(x[j], r);
  if (__ballot(s < 0x1p-126f) != 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = y[j] > 448.0f ? 448.0f : (y[j] < -448.0f ? -448.0f : y[j]);
  }
  int a = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  a = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], a, true);
  int b = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], b, true);
  return make_uint2((uint32_t)a, (uint32_t)b);
}

// The fp32 values code * s of an octet of codes.
__device__ __forceinline__ void e4m3_values(uint2 c, float s, float (&x)[8]) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, true);
  const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, false), e = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, true);
  x[0] = a[0] * s; x[1] = a[1] * s; x[2] = b[0] * s; x[3] = b[1] * s;
  x[4] = d[0] * s; x[5] = d[1] * s; x[6] = e[0] * s; x[7] = e[1] * s;
}

template <bool kVec>
__device__ __forceinline__ uint2 ld_codes(const uint8_t* p, int n) {
  if constexpr (kVec) {
    return n > 0 ? *reinterpret_cast<const uint2*>(p) : make_uint2(0, 0);
  } else {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
    return make_uint2(w[0], w[1]);
  }
}

template <bool kVec>
__device__ __forceinline__ void st_codes(uint8_t* p, int n, uint2 c) {
  if constexpr (kVec) {
    if (n > 0) *reinterpret_cast<uint2*>(p) = c;
  } else {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
  }
}

// Sums of K values over the TPR threads of a row, in a fixed order; every
// thread of the row receives them.  TPR <= 64: lanes of one wave.  Larger: a
// whole workgroup of TPR threads, through `red` (K * TPR / 64 floats, one
// buffer for each call of a row, so that one barrier is enough).
template <int TPR, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float* red) {
#pragma unroll
  for (int i = 0; i < K; ++i)
#pragma unroll
    for (int off = 1; off < (TPR < 64 ? TPR : 64); off <<= 1) v[i] += __shfl_xor(v[i], off, 64);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < K; ++i) red[i * W + w] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < K; ++i) {
      float s = red[i * W];
#pragma unroll
      for (int j = 1; j < W; ++j) s += red[i * W + j];
      v[i] = s;
    }
  }
}

}  // namespace gdn
