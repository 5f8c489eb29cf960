// gdn_lin_step.hip -- linear attention, one token for each sequence against a
// stored state:  S <- e^g S + v k^T,  o = S q  (S [dv, dk] fp32 in place).
//
// Memory bound: the state is read once and written once, 8 dv dk bytes a
// head; the rest is a few hundred bytes.  A workgroup takes kRows value rows
// of one (sequence, head); thread t holds the float4 column group t % (dk/4)
// of rows t / (dk/4) + p 1024/dk, so every access of the workgroup covers
// 4 KiB of contiguous state.  The rows' products with q are summed over their
// dk/4 lanes by DPP moves in a fixed order.
#include "gdn_device.hpp"
#include "gdn_launch.hpp"

namespace gdn {

template <int DK, typename T, int kRows>
__global__ __launch_bounds__(kThreads) void lin_step_kernel(const T* __restrict__ q, const T* __restrict__ k,
                                                            const T* __restrict__ v, const float* __restrict__ g,
                                                            float* __restrict__ state, T* __restrict__ o, int H,
                                                            int share, int dv, int64_t g_row) {
  constexpr int F = DK / 4;
  constexpr int RPP = kThreads / F;
  constexpr int NP = kRows / RPP;
  __shared__ float s_o[kRows];
  const int tiles = dv / kRows;
  const int vt = blockIdx.x % tiles;
  const int64_t nh = blockIdx.x / tiles;   // n * H + h
  const int64_t n = nh / H;
  const int h = (int)(nh - n * H);
  const int64_t qk = (n * (H / share) + h / share) * DK;
  const int t = threadIdx.x, c4 = t % F, rr = t / F;
  float4* S = reinterpret_cast<float4*>(state + (nh * dv + (int64_t)kRows * vt) * DK);
  float4 x[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) x[p] = ld_stream(S + t + kThreads * p);
  float kc[4], qc[4], vr[NP];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    kc[j] = io<T>::ld(k + qk + 4 * c4 + j);
    qc[j] = io<T>::ld(q + qk + 4 * c4 + j);
  }
#pragma unroll
  for (int p = 0; p < NP; ++p) vr[p] = io<T>::ld(v + nh * dv + kRows * vt + rr + RPP * p);
  const float a = exp_full(g[n * g_row + h]);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    x[p].x = fmaf(x[p].x, a, vr[p] * kc[0]);
    x[p].y = fmaf(x[p].y, a, vr[p] * kc[1]);
    x[p].z = fmaf(x[p].z, a, vr[p] * kc[2]);
    x[p].w = fmaf(x[p].w, a, vr[p] * kc[3]);
    st_stream(S + t + kThreads * p, x[p]);
    const float z = group_sum<F>(x[p].x * qc[0] + x[p].y * qc[1] + x[p].z * qc[2] + x[p].w * qc[3]);
    if (c4 == 0) s_o[rr + RPP * p] = z;
  }
  __syncthreads();
  if (t < kRows) io<T>::st(o + nh * dv + kRows * vt + t, s_o[t]);
}

// Rows of a workgroup: 64 (32 KiB of state at dk = 128, eight 16-byte loads a
// thread in flight) when that still gives the card a workgroup for every
// compute unit, else 16, which spreads a small batch over four times as many.
static bool lin_step_wide(const gdn_lin_t& s) { return (int64_t)s.n_seqs * s.n_heads * (s.dv / 64) >= 512; }

bool lin_step_fits(const gdn_lin_t& s) {
  return (int64_t)s.n_seqs * s.n_heads * (s.dv / (lin_step_wide(s) ? 64 : 16)) * kThreads < (int64_t)1 << 32;
}

hipError_t launch_lin_step(const gdn_lin_t& s, const void* q, const void* k, const void* v, const float* g,
                           float* state, void* o, hipStream_t stream) {
  const int64_t nh = (int64_t)s.n_seqs * s.n_heads;
  const int share = s.n_heads / s.qk_heads;
  const bool wide = lin_step_wide(s);
  const int rows = wide ? 64 : 16;
  auto go = [&](auto kern, auto tag) {
    using T = decltype(tag);
    hipLaunchKernelGGL(kern, dim3((unsigned)(nh * (s.dv / rows))), dim3(kThreads), 0, stream, (const T*)q,
                       (const T*)k, (const T*)v, g, state, (T*)o, s.n_heads, share, s.dv,
                       (int64_t)(s.gate_per_token ? s.n_heads : 0));
  };
  auto typed = [&](auto tag) {
    using T = decltype(tag);
    if (s.dk == 64) {
      if (wide) go(lin_step_kernel<64, T, 64>, tag);
      else go(lin_step_kernel<64, T, 16>, tag);
    } else {
      if (wide) go(lin_step_kernel<128, T, 64>, tag);
      else go(lin_step_kernel<128, T, 16>, tag);
    }
  };
  if (s.io_dtype == GDN_BF16) typed(uint16_t());
  else typed(float());
  return hipGetLastError();
}

}  // namespace gdn
