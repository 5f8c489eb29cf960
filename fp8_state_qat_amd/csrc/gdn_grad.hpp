// gdn_grad.hpp -- all gradients of the chunked gated delta rule: what its
// kernels share.
//
// Mathematics.  Chunk of C = 64 tokens, G_r the sum of the log-gates up to
// token r, D_rs = e^(G_r - G_s) (s <= r), S the state (dv x dk) entering it,
//   B_rs = D_rs k_r.k_s (s < r),  P_rs = D_rs q_r.k_s (s <= r),  b = beta
//   M = (I + B diag(b))^-1                     (unit lower triangular)
//   E = M (V - e^G K S^T)                      (errors v - S k of the tokens)
//   S' = e^(G_C) S + (b E)^T (e^(G_C - G) K),  O = e^G Q S^T + P (b E)
// Backwards, R the gradient of S':
//   F = P^T dO + e^(G_C - G) K R^T             (gradient of b E)
//   Y = M^T (b F)                              (gradient of V)
//   dS = e^(G_C) R + dO^T (e^G Q) - Y^T (e^G K)
//   W_rs = D_rs b_s dO_r.E_s (s <= r),  N_rs = -D_rs b_s Y_r.E_s (s < r)
//   dq = e^G dO S + W K
//   dk = -e^G Y S + b e^(G_C - G) E R + W^T Q + N K + N^T K
//   db_s = sum_r P_rs dO_r.E_s - sum_r B_rs Y_r.E_s + k_s.(e^(G_C - G) E R)_s
// and the gradient of log-gate t is the sum of every product that lies across
// token t: the pairs r >= t > s of b_s (P_rs dO_r.E_s - B_rs Y_r.E_s), the
// parts q_r.dq_r + k_r.dk_r of the entering state for r >= t, the parts
// k_s.dk_s of the leaving state for s < t, and e^(G_C) <R, S>.
// The state's quantization is the identity in all of this (straight-through);
// it shows in the S that the chunks start from.
//
// Three launches (gdn_grad.hip): records of every (chunk, head) in parallel
// (M, P, gates); the chains, forwards (S; it leaves S and E of every chunk) and
// backwards (R; R and Y), which need nothing of each other and run side by side;
// the gradients of every (chunk, head) in parallel, from S, R, E and Y.
#pragma once

#include "gdn_lin_scan.hpp"
#include "gdn_prep_item.hpp"

namespace gdn {

struct GradArgs {
  const void *q, *k, *v, *d_o;
  const float *beta, *g;
  const int32_t *cu, *seq_lens, *offs;
  int32_t* status;
  const float* init;   // initial state or null
  const float* kept;   // fp32 states after every chunk [chunk][H][dv][dk], or null
  int64_t n_kept;      // its entries
  const float* d_fin;  // gradient of the last states, or null
  char* rec;           // records (GradRec), one for each (chunk, head)
  float* S;            // states entering every (chunk, head), as kept (null with kept)
  float* R;            // gradients of the states after every (chunk, head)
  float *E, *Y;        // [chunk][H][dv][64]: the tokens' errors, and their gradients (V's), transposed
  void *dq, *dk, *d_v;
  float *d_beta, *dg, *d_init;
  int N, H, dv;
};

// Products of two operands split into bf16 planes keep the pairs of planes
// down to the last plane's size.
__host__ __device__ constexpr bool plane_pair(int i, int j, int planes) { return i + j < planes; }

// Record of a (chunk, head): the lower-triangular M and P as their ten 16 x 16
// blocks (row tile, column tile), each row-major, so that one copy gives rows
// and, by transpose reads, columns; then the gates.  bf16 inputs: three bf16
// planes (with two of P beta's and the gates' gradients were off by 4e-6, with
// three by 5e-7); fp32 inputs: fp32.
template <class Eng>
struct GradRec {
  static constexpr bool kBF = Eng::kSplit;
  static constexpr int kMPlanes = kBF ? 3 : 1, kPPlanes = kMPlanes;
  static constexpr int kBlock = 256 * (int)sizeof(typename Eng::E);
  static constexpr int kPlane = 10 * kBlock;
  static constexpr int oP = kMPlanes * kPlane;
  static constexpr int oG = oP + kPPlanes * kPlane;
  static constexpr int kGates = 2048;
  static constexpr int kBytes = oG + kGates;
};
__host__ __device__ constexpr int tri_block(int ti, int tj) { return ti * (ti + 1) / 2 + tj; }

// Gates of a chunk.  Rows past its end: eg, el and beta 0.  The first KiB is
// what the chains need.
struct GradGates {
  float eg[kChunk];    // e^G
  float el[kChunk];    // e^(G_C - G)
  float beta[kChunk];
  float ec[kChunk];    // e^(G_C), all alike
  int n[kChunk];       // G log2(e) = n + f
  float f[kChunk];
  float g[kChunk];     // the log-gates
  float zero[kChunk];  // 1 where beta is 0, whose place 2^-60 takes in beta
};
static_assert(sizeof(GradGates) == 2048, "the record's gates");

// True where the call computes nothing: index arrays out of contract, or
// fewer states than chunks.
__device__ __forceinline__ bool grad_refused(const GradArgs& a) {
  return index_check_failed(a.status) || (a.kept != nullptr && (int64_t)uniform(a.offs[a.N]) > a.n_kept);
}

// Place of a chunk in the batch.
struct GradPlace {
  int n, c, t0, nv, L;
};
__device__ __forceinline__ GradPlace grad_place(const GradArgs& a, int j) {
  int lo = 0, hi = a.N - 1;   // last sequence with offs[n] <= j
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.offs[mid] <= j) lo = mid; else hi = mid - 1;
  }
  GradPlace p;
  p.n = uniform(lo);
  p.c = j - uniform(a.offs[p.n]);
  const int seg0 = uniform(a.cu[p.n]);
  p.L = a.seq_lens ? uniform(a.seq_lens[p.n]) : uniform(a.cu[p.n + 1]) - seg0;
  p.t0 = seg0 + p.c * kChunk;
  p.nv = min(kChunk, p.L - p.c * kChunk);
  return p;
}

// Element (row, col) of a record's block, in units of four elements swizzled so
// that reads of rows (16 of them, one unit a lane) and of columns meet no bank
// twice.
template <class Eng>
__device__ __forceinline__ int tri_at(int row, int col) {
  const int u = (col >> 2) ^ (Eng::kSplit ? (row >> 3) << 1 : row >> 2);
  return 16 * row + 4 * u + (col & 3);
}
// Rows of a record's blocks as a fragment: row 16 ti + ln, columns kperm of
// k-block kb; blocks above the diagonal are zero.
template <class Eng>
__device__ __forceinline__ typename Eng::Fr tri_rows(const char* plane, int ti, int kb, int ln, int gq) {
  using E = typename Eng::E;
  constexpr int kBlock = GradRec<Eng>::kBlock;
  const char* p = plane + tri_at<Eng>(ln, 4 * gq) * sizeof(E);
  const E* a = (const E*)(p + tri_block(ti, 2 * kb) * kBlock);
  if (2 * kb + 1 <= ti) return Eng::ld2(a, (const E*)(p + tri_block(ti, 2 * kb + 1) * kBlock));
  if constexpr (Eng::kSplit) {
    const uint2 u = *reinterpret_cast<const uint2*>(a);
    return __builtin_bit_cast(bf16x8, make_uint4(u.x, u.y, 0, 0));
  } else {
    const float4 u = *reinterpret_cast<const float4*>(a);
    return Frag8{{u.x, u.y, u.z, u.w, 0.0f, 0.0f, 0.0f, 0.0f}};
  }
}
// The transposed matrix's: column 16 si + ln, rows kperm of k-block kb.
template <class Eng>
__device__ __forceinline__ typename Eng::Fr tri_cols(const char* plane, int si, int kb, int ln, int gq) {
  using E = typename Eng::E;
  constexpr int kBlock = GradRec<Eng>::kBlock;
  const bool first = 2 * kb >= si;
  if constexpr (Eng::kSplit) {
    const char* p = plane + tri_at<Eng>(4 * gq + (ln >> 2), 4 * (ln & 3)) * 2;
    uint2 u = make_uint2(0, 0);
    if (first) u = lds_read_tr16(p + tri_block(2 * kb, si) * kBlock);
    const uint2 v = lds_read_tr16(p + tri_block(2 * kb + 1, si) * kBlock);
    return __builtin_bit_cast(bf16x8, make_uint4(u.x, u.y, v.x, v.y));
  } else {
    Frag8 r;
    const E* p = (const E*)plane + tri_at<Eng>(4 * gq, ln);   // rows 4 gq + j share a swizzle
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r.v[j] = first ? p[tri_block(2 * kb, si) * 256 + 16 * j] : 0.0f;
      r.v[4 + j] = p[tri_block(2 * kb + 1, si) * 256 + 16 * j];
    }
    return r;
  }
}

// x in P planes (P = 1: fp32 inputs).
template <class Eng, int P>
__device__ __forceinline__ void split_planes(const float (&x)[8], typename Eng::Fr (&f)[P]) {
  if constexpr (P == 3) Eng::split3(x, f[0], f[1], f[2]);
  else if constexpr (P == 2) Eng::split(x, f[0], f[1]);
  else f[0] = Eng::round(x);
}

// Bytes (a multiple of 1 KiB) from memory into LDS as they are, by NW waves.
template <int NW>
__device__ __forceinline__ void ask_bytes(uint32_t lds, const void* p, int bytes) {
  const int w = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  for (int i = w; i < bytes / 1024; i += NW) lds_load16(p, (uint32_t)((i * 64 + lane) * 16), lds + i * 1024);
}

// Value j of a column fragment (or an fp32 one).
__device__ __forceinline__ void frag_values(const bf16x8& f, float (&x)[8]) {
  const uint4 u = __builtin_bit_cast(uint4, f);
  x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
  x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z); x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
}
__device__ __forceinline__ void frag_values(const Frag8& f, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = f.v[j];
}

hipError_t launch_grad_bf16(const gdn_shape_t& s, const GradArgs& a, int64_t items, hipStream_t stream);
hipError_t launch_grad_f32(const gdn_shape_t& s, const GradArgs& a, int64_t items, hipStream_t stream);

}  // namespace gdn
