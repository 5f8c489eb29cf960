// gdn_act8.hip -- activations as 8-bit codes: every 64 consecutive columns of
// a row share a scale s = RN(amax / 448) (1 where that is not positive), code
// = E4M3(RN(x / s)), ties to even; and back, x = RN(code * s).
//
// Memory bound: 2 or 4 bytes read and 1 + 4/64 written a value (the reverse
// for the way back).  A lane takes eight consecutive columns, the eight lanes
// of a group find its amax by DPP moves, and a workgroup takes kUnroll
// neighbouring runs of 32 groups, all its loads in flight at once (16384 x
// 4096 bf16 there and back: 73 us, 5.6 TB/s; 75 with one run, 76 with four).
#include "gdn_rows.hpp"

namespace gdn {

constexpr int kUnroll = 2;

template <typename T, bool kVec>
__global__ __launch_bounds__(kThreads) void act_pack_kernel(const T* __restrict__ x, uint8_t* __restrict__ codes,
                                                            float* __restrict__ scales, uint32_t n_groups,
                                                            uint32_t groups, int cols) {
  const int l8 = threadIdx.x & 7;
  constexpr uint32_t stride = kThreads / 8;
  const uint32_t g0 = blockIdx.x * (kUnroll * stride) + (threadIdx.x >> 3);
  float v[kUnroll][8];
  int64_t at[kUnroll];
  int n[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const uint32_t gi = g0 + u * stride;
    const uint32_t row = gi / groups;
    const int col = (int)(gi - row * groups) * kGroupCols + 8 * l8;
    n[u] = gi < n_groups ? cols - col : 0;
    at[u] = (int64_t)row * cols + col;
    ld_oct<T, kVec>(x + (n[u] > 0 ? at[u] : 0), n[u], v[u]);
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const float s = group_scale(v[u]);
    const uint32_t gi = g0 + u * stride;
    if (n[u] > 0) st_codes<kVec>(codes + at[u], n[u], e4m3_oct(v[u], s));
    if (l8 == 0 && gi < n_groups) scales[gi] = s;
  }
}

template <typename T, bool kVec>
__global__ __launch_bounds__(kThreads) void act_unpack_kernel(const uint8_t* __restrict__ codes,
                                                              const float* __restrict__ scales, T* __restrict__ x,
                                                              uint32_t n_groups, uint32_t groups, int cols) {
  const int l8 = threadIdx.x & 7;
  constexpr uint32_t stride = kThreads / 8;
  const uint32_t g0 = blockIdx.x * (kUnroll * stride) + (threadIdx.x >> 3);
  uint2 c[kUnroll];
  float s[kUnroll];
  int64_t at[kUnroll];
  int n[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const uint32_t gi = g0 + u * stride;
    const uint32_t row = gi / groups;
    const int col = (int)(gi - row * groups) * kGroupCols + 8 * l8;
    n[u] = gi < n_groups ? cols - col : 0;
    at[u] = (int64_t)row * cols + col;
    c[u] = ld_codes<kVec>(codes + (n[u] > 0 ? at[u] : 0), n[u]);
    s[u] = gi < n_groups ? scales[gi] : 0.0f;
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    float v[8];
    e4m3_values(c[u], s[u], v);
    if (n[u] > 0) st_oct<T, kVec>(x + at[u], n[u], v);
  }
}

// Runs go(first row, groups, blocks) for as many launches as the rows need:
// kUnroll groups of 8 lanes for each 8 threads.  The host has checked that the
// groups fit 31 bits.
template <class F>
static void act_launches(int64_t rows, int64_t groups, F go) {
  constexpr int64_t kPer = kUnroll * (kThreads / 8);
  const int64_t most = max_blocks(kThreads) * kPer / groups;
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t n = (rows - r < most ? rows - r : most) * groups;
    go(r, (uint32_t)n, (unsigned)((n + kPer - 1) / kPer));
  }
}

static bool act_vec(const void* p, const void* codes, int cols) {
  return cols % 8 == 0 && (uintptr_t)p % 16 == 0 && (uintptr_t)codes % 8 == 0;
}

hipError_t launch_act_pack(const void* x, int dtype, uint8_t* codes, float* scales, int64_t rows, int cols,
                           hipStream_t stream) {
  const int64_t groups = ((int64_t)cols + kGroupCols - 1) / kGroupCols;
  auto go = [&](auto kern, auto* p) {
    act_launches(rows, groups, [&](int64_t r, uint32_t n, unsigned blocks) {
      hipLaunchKernelGGL(kern, dim3(blocks), dim3(kThreads), 0, stream, p + r * cols, codes + r * cols,
                         scales + r * groups, n, (uint32_t)groups, cols);
    });
  };
  const bool vec = act_vec(x, codes, cols);
  if (dtype == GDN_BF16) {
    if (vec) go(act_pack_kernel<uint16_t, true>, (const uint16_t*)x);
    else go(act_pack_kernel<uint16_t, false>, (const uint16_t*)x);
  } else {
    if (vec) go(act_pack_kernel<float, true>, (const float*)x);
    else go(act_pack_kernel<float, false>, (const float*)x);
  }
  return hipGetLastError();
}

hipError_t launch_act_unpack(const uint8_t* codes, const float* scales, void* x, int dtype, int64_t rows, int cols,
                             hipStream_t stream) {
  const int64_t groups = ((int64_t)cols + kGroupCols - 1) / kGroupCols;
  auto go = [&](auto kern, auto* p) {
    act_launches(rows, groups, [&](int64_t r, uint32_t n, unsigned blocks) {
      hipLaunchKernelGGL(kern, dim3(blocks), dim3(kThreads), 0, stream, codes + r * cols, scales + r * groups,
                         p + r * cols, n, (uint32_t)groups, cols);
    });
  };
  const bool vec = act_vec(x, codes, cols);
  if (dtype == GDN_BF16) {
    if (vec) go(act_unpack_kernel<uint16_t, true>, (uint16_t*)x);
    else go(act_unpack_kernel<uint16_t, false>, (uint16_t*)x);
  } else {
    if (vec) go(act_unpack_kernel<float, true>, (float*)x);
    else go(act_unpack_kernel<float, false>, (float*)x);
  }
  return hipGetLastError();
}

}  // namespace gdn
