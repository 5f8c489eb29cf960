// gdn_block_norm.hip -- the norm after a block, its gate, the scaled residual
// and the norm before the next block, in one pass over the rows; its backward;
// the block's output and gate optionally kept as E4M3 codes between the two.
//
//   r = 1 / sqrt(mean f^2 + eps)      y = f r w_post a(z)      (a = 1 without a gate)
//   x = res_scale y + residual        h = x w_pre / sqrt(mean x^2 + eps)
// and with t = d_h w_pre, xh = x / sqrt(mean x^2 + eps), n = f r:
//   dx' = d_x + r_x (t - xh mean(t xh))        d_w_pre = sum_rows d_h xh
//   d_residual = dx'                           d_w_post = sum_rows dy a n
//   d_z = dy n w_post a'(z)                    dy = res_scale dx'
//   d_f = r (u - n mean(u n)),  u = dy a w_post
//
// Memory bound: every array is read or written once, a few tens of operations
// a value.  A row belongs to TPR threads (a power of two: 8 lanes for 64
// columns up to a workgroup of 1024), thread i of it to the octets
// (i + TPR j) of eight consecutive columns, j < V, held in registers between
// the row sums; the sums of a wave go by lane moves, those of a workgroup
// through LDS behind one barrier each.  All arithmetic is fp32; h is formed
// from x before x is rounded for its store.
//
// The weights' gradients are sums over the rows: in the backward a workgroup
// walks rows kSweep apart with its threads on fixed columns, keeps their partial sums in fp32 registers and writes one partial row; a
// second kernel adds the partial rows in fp64, in a fixed order.  A thread adds
// kSumRows rows at most, which leaves 2^-19 of the sum of their magnitudes
// whatever the number of rows; larger calls take more workgroups, kSweep of
// them after kSweep over neighbouring rows (a million rows of 512: 1.63 ms, as
// with 1024 workgroups over all rows; 1.82 with every workgroup's rows spread
// over the whole call).
#include <type_traits>

#include "gdn_rows.hpp"

namespace gdn {

struct NormArgs {
  const void* f;             // io values, or E4M3 codes in the backward (f_scales given)
  const void* z;             // the gate, the same way; null: none
  float* f_scales;
  float* z_scales;
  uint8_t* f_codes;          // forward: checkpoint outputs (null: none)
  uint8_t* z_codes;
  const float* w_post;
  const float* w_pre;        // null: no norm before the next block
  const void* res;           // forward: the residual (null: none); backward: x
  const void* d_x;
  const void* d_h;
  void* x;                   // forward: x; backward: d_residual (null: not wanted)
  void* h;                   // forward: h; backward: d_f
  void* d_z;
  float* part_post;          // backward: [gridDim.x, cols] partial sums
  float* part_pre;
  int64_t rows;
  int cols;
  int act;
  float res_scale, eps;
};

// The gate's value a(z) and, for the backward, its derivative, from e = e^-|z|,
// which does not overflow: with r = 1 / (1 + e) the sigmoid p and 1 - p are r
// and e r, in the order of z's sign.  fp32 rows take exp_full and the correctly
// rounded quotient.  bf16 rows take the hardware's 2^x of |z| log2(e) and its
// reciprocal, which leave 2^-20 + |z| 2^-24 of a value, far below the output's
// 2^-9 (fp32's way takes half of the kernel's instructions); both flush
// subnormal numbers, so they are kept 2^24 away from them.  The forward does
// without the sign there, p = 1 / (1 + e^-z): heads of 262144 x 128 take 37.6
// us so, 38.9 with it.
template <typename T, bool kDer>
__device__ __forceinline__ void gate_act(float z, int act, float& a, float& da) {
  constexpr float kLog2e = 1.4426950408889634f;
  if constexpr (sizeof(T) == 2 && !kDer) {
    const float e = __builtin_amdgcn_exp2f(fmaf(z, -kLog2e, -24.0f));
    const float p = __builtin_amdgcn_rcpf(e + 0x1p-24f) * 0x1p-24f;
    a = act == GDN_ACT_SIGMOID ? p : z * p;
    return;
  }
  float r, er;
  if constexpr (sizeof(T) == 4) {
    const float e = exp_full(-fabsf(z));
    r = 1.0f / (1.0f + e);
    er = e * r;
  } else {
    const float e = __builtin_amdgcn_exp2f(fmaf(fabsf(z), -kLog2e, 24.0f));
    r = __builtin_amdgcn_rcpf(fmaf(e, 0x1p-24f, 1.0f));
    er = e * r * 0x1p-24f;
  }
  const float p = z < 0.0f ? er : r, q = z < 0.0f ? r : er;
  if (act == GDN_ACT_SIGMOID) {
    a = p;
    da = p * q;
  } else {
    a = z * p;
    da = p * (1.0f + z * q);
  }
}

// The backward: workgroups that walk together, and rows each of them adds in fp32.
constexpr int kSweep = 1024, kSumRows = 32;

template <int TPR>
constexpr int norm_block() { return TPR > kThreads ? TPR : kThreads; }

template <typename TIO, typename TX, int TPR, int V, bool kVec, bool kCkpt>
__global__ __launch_bounds__(norm_block<TPR>()) void block_norm_fwd_kernel(NormArgs A) {
  constexpr int kRows = norm_block<TPR>() / TPR;   // rows of a workgroup
  __shared__ float red[TPR > 64 ? 2 * (TPR / 64) : 1];
  const int i = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  const bool live = row < A.rows;                  // rows past the end run with no columns
  const int64_t base = row * A.cols;
  const float inv = 1.0f / (float)A.cols;
  float f[V][8], y[V][8];
  int n[V], col[V];
  float ss[1] = {0.0f};
#pragma unroll
  for (int j = 0; j < V; ++j) {
    col[j] = 8 * (i + TPR * j);
    n[j] = live ? A.cols - col[j] : 0;
    const int64_t at = n[j] > 0 ? base + col[j] : 0;
    ld_oct<TIO, kVec>((const TIO*)A.f + at, n[j], f[j]);
    if (A.z) ld_oct<TIO, kVec>((const TIO*)A.z + at, n[j], y[j]);
  }
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int c = 0; c < 8; ++c) ss[0] = fmaf(f[j][c], f[j][c], ss[0]);
  if constexpr (kCkpt) {
    const int groups = (A.cols + kGroupCols - 1) / kGroupCols;
#pragma unroll
    for (int j = 0; j < V; ++j) {   // the 8 lanes of a group hold its octets
      const float s = group_scale(f[j]);
      const bool first = n[j] > 0 && (i & 7) == 0;
      if (n[j] > 0) st_codes<kVec>(A.f_codes + base + col[j], n[j], e4m3_oct(f[j], s));
      if (first) A.f_scales[row * groups + col[j] / kGroupCols] = s;
      if (A.z) {
        const float sz = group_scale(y[j]);
        if (n[j] > 0) st_codes<kVec>(A.z_codes + base + col[j], n[j], e4m3_oct(y[j], sz));
        if (first) A.z_scales[row * groups + col[j] / kGroupCols] = sz;
      }
    }
  }
  row_sum<TPR, 1>(ss, red);
  const float r = 1.0f / sqrtf(ss[0] * inv + A.eps);
  float sx[1] = {0.0f};
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float w[8], x[8];
    ld_oct<float, kVec>(A.w_post + (n[j] > 0 ? col[j] : 0), n[j], w);
    if (A.res) ld_oct<TX, kVec>((const TX*)A.res + (n[j] > 0 ? base + col[j] : 0), n[j], x);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      float t = f[j][c] * r * w[c];
      if (A.z) {
        float a, da;
        gate_act<TIO, false>(y[j][c], A.act, a, da);
        t *= a;
      }
      t *= A.res_scale;
      if (A.res) t += x[c];
      y[j][c] = t;
      sx[0] = fmaf(t, t, sx[0]);
    }
    if (n[j] > 0) st_oct<TX, kVec>((TX*)A.x + base + col[j], n[j], y[j]);
  }
  if (A.w_pre == nullptr) return;
  row_sum<TPR, 1>(sx, red + TPR / 64);
  const float rx = 1.0f / sqrtf(sx[0] * inv + A.eps);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float w[8];
    ld_oct<float, kVec>(A.w_pre + (n[j] > 0 ? col[j] : 0), n[j], w);
#pragma unroll
    for (int c = 0; c < 8; ++c) y[j][c] = y[j][c] * rx * w[c];
    if (n[j] > 0) st_oct<TIO, kVec>((TIO*)A.h + base + col[j], n[j], y[j]);
  }
}

template <typename TIO, typename TX, int TPR, int V, bool kVec, bool kCkpt>
__global__ __launch_bounds__(norm_block<TPR>()) void block_norm_bwd_kernel(NormArgs A) {
  constexpr int kBlock = norm_block<TPR>();
  constexpr int kRows = kBlock / TPR;
  constexpr int W = TPR > 64 ? TPR / 64 : 1;
  __shared__ float red[8 * W];                     // two rows' buffers: one barrier each suffices
  __shared__ float s_part[kRows > 1 ? kBlock * 8 * V : 1];
  const int i = threadIdx.x % TPR, rr = threadIdx.x / TPR;
  const float inv = 1.0f / (float)A.cols;
  const int groups = (A.cols + kGroupCols - 1) / kGroupCols;
  int col[V];
  float wp[V][8], we[V][8], acc_p[V][8], acc_e[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    col[j] = 8 * (i + TPR * j);
    const int n = A.cols - col[j];
    ld_oct<float, kVec>(A.w_post + (n > 0 ? col[j] : 0), n, wp[j]);
    if (A.w_pre) ld_oct<float, kVec>(A.w_pre + (n > 0 ? col[j] : 0), n, we[j]);
#pragma unroll
    for (int c = 0; c < 8; ++c) acc_p[j][c] = acc_e[j][c] = 0.0f;
  }
  int flip = 0;
  const int64_t sweep = min((int)gridDim.x, kSweep), from = blockIdx.x / kSweep * (sweep * kRows * kSumRows);
  const int64_t end = min(A.rows, from + sweep * kRows * kSumRows);
  for (int64_t row0 = from + blockIdx.x % kSweep * kRows; row0 < end; row0 += sweep * kRows) {
    const int64_t row = row0 + rr;
    const bool live = row < A.rows;
    const int64_t base = row * A.cols;
    float f[V][8], z[V][8], d[V][8], x[V][8], t[V][8];
    int n[V];
    float s[3] = {0.0f, 0.0f, 0.0f};               // f f, x x, t x
#pragma unroll
    for (int j = 0; j < V; ++j) {
      n[j] = live ? A.cols - col[j] : 0;
      const int64_t at = n[j] > 0 ? base + col[j] : 0;
      if constexpr (kCkpt) {
        const int64_t gi = n[j] > 0 ? row * groups + col[j] / kGroupCols : 0;
        e4m3_values(ld_codes<kVec>((const uint8_t*)A.f + at, n[j]), A.f_scales[gi], f[j]);
        if (A.z) e4m3_values(ld_codes<kVec>((const uint8_t*)A.z + at, n[j]), A.z_scales[gi], z[j]);
        if (n[j] <= 0) {
#pragma unroll
          for (int c = 0; c < 8; ++c) f[j][c] = z[j][c] = 0.0f;
        }
      } else {
        ld_oct<TIO, kVec>((const TIO*)A.f + at, n[j], f[j]);
        if (A.z) ld_oct<TIO, kVec>((const TIO*)A.z + at, n[j], z[j]);
      }
      ld_oct<TX, kVec>((const TX*)A.d_x + at, n[j], d[j]);
      if (A.w_pre) {
        ld_oct<TX, kVec>((const TX*)A.res + at, n[j], x[j]);
        ld_oct<TIO, kVec>((const TIO*)A.d_h + at, n[j], t[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        s[0] = fmaf(f[j][c], f[j][c], s[0]);
        if (A.w_pre) {
          s[1] = fmaf(x[j][c], x[j][c], s[1]);
          s[2] = fmaf(t[j][c] * we[j][c], x[j][c], s[2]);
        }
      }
    float* rb = red + 4 * W * flip;
    flip ^= 1;
    row_sum<TPR, 3>(s, rb);
    const float r = 1.0f / sqrtf(s[0] * inv + A.eps);
    if (A.w_pre) {
      const float rx = 1.0f / sqrtf(s[1] * inv + A.eps);
      const float m = s[2] * rx * inv;             // mean(t xh)
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float xh = x[j][c] * rx;
          acc_e[j][c] = fmaf(t[j][c], xh, acc_e[j][c]);
          d[j][c] += rx * (t[j][c] * we[j][c] - xh * m);
        }
    }
    float q[1] = {0.0f};                           // u n
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (A.x != nullptr && n[j] > 0) st_oct<TX, kVec>((TX*)A.x + base + col[j], n[j], d[j]);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float dy = A.res_scale * d[j][c], nn = f[j][c] * r;
        float a = 1.0f, da = 0.0f;
        if (A.z) gate_act<TIO, true>(z[j][c], A.act, a, da);
        z[j][c] = dy * nn * wp[j][c] * da;
        const float u = dy * a;
        acc_p[j][c] = fmaf(u, nn, acc_p[j][c]);
        d[j][c] = u * wp[j][c];
        f[j][c] = nn;
        q[0] = fmaf(d[j][c], nn, q[0]);
      }
      if (A.z && n[j] > 0) st_oct<TIO, kVec>((TIO*)A.d_z + base + col[j], n[j], z[j]);
    }
    row_sum<TPR, 1>(q, rb + 3 * W);
    const float m = q[0] * inv;
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
      for (int c = 0; c < 8; ++c) d[j][c] = r * (d[j][c] - f[j][c] * m);
      if (n[j] > 0) st_oct<TIO, kVec>((TIO*)A.h + base + col[j], n[j], d[j]);
    }
  }
  // this workgroup's partial sums over its rows
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    float* out = pass ? A.part_pre : A.part_post;
    if (pass && A.w_pre == nullptr) break;
    if constexpr (kRows > 1) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int c = 0; c < 8; ++c) s_part[rr * TPR * 8 * V + col[j] + c] = pass ? acc_e[j][c] : acc_p[j][c];
      __syncthreads();
      for (int c = threadIdx.x; c < A.cols; c += kBlock) {
        double sum = 0.0;
        for (int k = 0; k < kRows; ++k) sum += (double)s_part[k * TPR * 8 * V + c];
        out[(int64_t)blockIdx.x * A.cols + c] = (float)sum;
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int n = A.cols - col[j];
        if (n > 0) st_oct<float, kVec>(out + (int64_t)blockIdx.x * A.cols + col[j], n, pass ? acc_e[j] : acc_p[j]);
      }
    }
  }
}

// Column sums of the partial rows: 32 columns a workgroup, its kSlices row
// slices added in fp64 in a fixed order (with 8 slices the sums of 2048
// columns' 1024 rows took 8.4 us instead of 4.9).
constexpr int kSlices = 32;
__global__ __launch_bounds__(32 * kSlices) void norm_reduce_kernel(const float* __restrict__ part_post,
                                                                   const float* __restrict__ part_pre,
                                                                   float* __restrict__ dw_post,
                                                                   float* __restrict__ dw_pre, int parts, int cols) {
  __shared__ double s[kSlices][32];
  const float* part = blockIdx.y ? part_pre : part_post;
  const int c = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  double a = 0.0;
  if (col < cols) {
#pragma unroll 8
    for (int p = sl; p < parts; p += kSlices) a += (double)part[(int64_t)p * cols + col];
  }
  s[sl][c] = a;
  __syncthreads();
  if (sl == 0 && col < cols) {
    double t = s[0][c];
    for (int k = 1; k < kSlices; ++k) t += s[k][c];
    (blockIdx.y ? dw_pre : dw_post)[col] = (float)t;
  }
}

// Rows layout by the column count: one octet a thread while a row fits 64
// lanes (no barrier), then a wave with two, then workgroups.  Rows that do not
// allow 16-byte accesses take the two general layouts.
struct NormPlan { int tpr, v; };
static NormPlan norm_plan(int cols, bool vec) {
  if (!vec) return cols <= 512 ? NormPlan{64, 1} : NormPlan{512, 4};
  if (cols <= 64) return {8, 1};
  if (cols <= 128) return {16, 1};
  if (cols <= 256) return {32, 1};
  if (cols <= 512) return {64, 1};
  if (cols <= 1024) return {64, 2};
  if (cols <= 2048) return {256, 1};
  if (cols <= 4096) return {256, 2};
  if (cols <= 8192) return {512, 2};
  return {512, 4};
}

static int norm_rows_of(const NormPlan& p) { return p.tpr >= kThreads ? 1 : kThreads / p.tpr; }

// Workgroups of the backward: enough to fill the card four times over, so
// that the partial rows stay a few percent of the traffic, and as many again
// for every kSumRows rows of theirs.  (Rows that pass 2^32 threads this way do
// not fit the memory.)
static int64_t norm_bwd_blocks(const gdn_norm_t& s, const NormPlan& p) {
  const int64_t need = (s.rows + norm_rows_of(p) - 1) / norm_rows_of(p);
  if (need < kSweep) return need < 1 ? 1 : need;
  return (need + kSweep * kSumRows - 1) / (kSweep * kSumRows) * kSweep;
}

size_t block_norm_bwd_workspace_bytes(const gdn_norm_t& s) {
  // the larger of the two layouts' partial rows (which one runs depends on the pointers' alignment)
  const int64_t a = norm_bwd_blocks(s, norm_plan(s.cols, true)), b = norm_bwd_blocks(s, norm_plan(s.cols, false));
  return (size_t)((a > b ? a : b) * s.cols * 2 * 4);
}

template <typename TIO, typename TX, bool kVec, bool kCkpt, bool kBwd>
static void norm_go(const NormArgs& A, const NormPlan& p, int64_t blocks, hipStream_t stream) {
  auto go = [&](auto kern) {
    const int threads = p.tpr > kThreads ? p.tpr : kThreads;
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(threads), 0, stream, A);
  };
#define GDN_NORM_KERNEL(TPR, V)                                               \
  do {                                                                        \
    if constexpr (kBwd) go(block_norm_bwd_kernel<TIO, TX, TPR, V, kVec, kCkpt>); \
    else go(block_norm_fwd_kernel<TIO, TX, TPR, V, kVec, kCkpt>);             \
  } while (0)
  if constexpr (!kVec) {
    if (p.tpr == 64) GDN_NORM_KERNEL(64, 1);
    else GDN_NORM_KERNEL(512, 4);
  } else {
    switch (p.tpr * 16 + p.v) {
      case 8 * 16 + 1: GDN_NORM_KERNEL(8, 1); break;
      case 16 * 16 + 1: GDN_NORM_KERNEL(16, 1); break;
      case 32 * 16 + 1: GDN_NORM_KERNEL(32, 1); break;
      case 64 * 16 + 1: GDN_NORM_KERNEL(64, 1); break;
      case 64 * 16 + 2: GDN_NORM_KERNEL(64, 2); break;
      case 256 * 16 + 1: GDN_NORM_KERNEL(256, 1); break;
      case 256 * 16 + 2: GDN_NORM_KERNEL(256, 2); break;
      case 512 * 16 + 2: GDN_NORM_KERNEL(512, 2); break;
      default: GDN_NORM_KERNEL(512, 4); break;
    }
  }
#undef GDN_NORM_KERNEL
}

// The forward's arguments from row r on.
static NormArgs norm_from(NormArgs A, const gdn_norm_t& s, int64_t r) {
  const int64_t n = r * s.cols, g = r * ((s.cols + kGroupCols - 1) / kGroupCols);
  const int64_t io = s.io_dtype == GDN_F32 ? 4 : 2, xt = s.x_dtype == GDN_F32 ? 4 : 2;
  auto at = [](auto*& p, int64_t bytes) {
    if (p != nullptr) p = (std::remove_reference_t<decltype(p)>)((uintptr_t)p + bytes);
  };
  at(A.f, n * io);
  at(A.z, n * io);
  at(A.res, n * xt);
  at(A.x, n * xt);
  at(A.h, n * io);
  at(A.f_codes, n);
  at(A.z_codes, n);
  at(A.f_scales, g * 4);
  at(A.z_scales, g * 4);
  A.rows = s.rows - r;
  return A;
}

template <bool kBwd>
static hipError_t norm_launch(const gdn_norm_t& s, const NormArgs& all, bool vec, bool ckpt, hipStream_t stream) {
  const NormPlan p = norm_plan(s.cols, vec);
  const int64_t rows_of = norm_rows_of(p);
  const int64_t most = max_blocks(p.tpr > kThreads ? p.tpr : kThreads);
  NormArgs A = all;
  int64_t blocks = kBwd ? norm_bwd_blocks(s, p) : (s.rows + rows_of - 1) / rows_of;
  auto typed = [&](auto tio, auto tx) {
    using TIO = decltype(tio);
    using TX = decltype(tx);
    if (vec) {
      if (ckpt) norm_go<TIO, TX, true, true, kBwd>(A, p, blocks, stream);
      else norm_go<TIO, TX, true, false, kBwd>(A, p, blocks, stream);
    } else {
      if (ckpt) norm_go<TIO, TX, false, true, kBwd>(A, p, blocks, stream);
      else norm_go<TIO, TX, false, false, kBwd>(A, p, blocks, stream);
    }
  };
  auto launch = [&] {
    if (s.io_dtype == GDN_F32) typed(float(), float());
    else if (s.x_dtype == GDN_F32) typed(uint16_t(), float());
    else typed(uint16_t(), uint16_t());
  };
  if (kBwd || blocks <= most) {
    launch();
    return hipGetLastError();
  }
  for (int64_t b = 0, all_blocks = blocks; b < all_blocks; b += most) {
    blocks = all_blocks - b < most ? all_blocks - b : most;
    A = norm_from(all, s, b * rows_of);
    A.rows = A.rows < blocks * rows_of ? A.rows : blocks * rows_of;
    launch();
  }
  return hipGetLastError();
}

static bool all16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if ((uintptr_t)p % 16 != 0) return false;
  return true;
}

hipError_t launch_block_norm_fwd(const gdn_norm_t& s, const void* f, const void* gate, const void* residual,
                                 const float* w_post, const float* w_pre, void* x, void* h, uint8_t* f_codes,
                                 float* f_scales, uint8_t* z_codes, float* z_scales, hipStream_t stream) {
  NormArgs A{};
  A.f = f; A.z = gate; A.res = residual; A.w_post = w_post; A.w_pre = w_pre; A.x = x; A.h = h;
  A.f_codes = f_codes; A.f_scales = f_scales; A.z_codes = z_codes; A.z_scales = z_scales;
  A.rows = s.rows; A.cols = s.cols; A.act = s.act; A.res_scale = s.res_scale; A.eps = s.eps;
  const bool vec = s.cols % 8 == 0 && all16({f, gate, residual, w_post, w_pre, x, h, f_codes, z_codes});
  return norm_launch<false>(s, A, vec, f_codes != nullptr, stream);
}

hipError_t launch_block_norm_bwd(const gdn_norm_t& s, const void* f, const float* f_scales, const void* gate,
                                 const float* gate_scales, const float* w_post, const float* w_pre, const void* x,
                                 const void* d_x, const void* d_h, void* d_f, void* d_z, void* d_residual,
                                 float* dw_post, float* dw_pre, void* workspace, hipStream_t stream) {
  NormArgs A{};
  A.f = f; A.z = gate; A.f_scales = const_cast<float*>(f_scales); A.z_scales = const_cast<float*>(gate_scales);
  A.w_post = w_post; A.w_pre = w_pre; A.res = x; A.d_x = d_x; A.d_h = d_h; A.h = d_f; A.d_z = d_z;
  A.x = d_residual;
  A.rows = s.rows; A.cols = s.cols; A.act = s.act; A.res_scale = s.res_scale; A.eps = s.eps;
  const bool vec = s.cols % 8 == 0 && all16({f, gate, x, d_x, d_h, w_post, w_pre, d_f, d_z, d_residual, workspace});
  const int parts = (int)norm_bwd_blocks(s, norm_plan(s.cols, vec));
  A.part_post = (float*)workspace;
  A.part_pre = A.part_post + (int64_t)parts * s.cols;
  const hipError_t e = norm_launch<true>(s, A, vec, f_scales != nullptr, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(norm_reduce_kernel, dim3((s.cols + 31) / 32, w_pre ? 2 : 1), dim3(32 * kSlices), 0, stream,
                     A.part_post, A.part_pre, dw_post, dw_pre, parts, s.cols);
  return hipGetLastError();
}

}  // namespace gdn
