// gdn_grad_kernels.hpp -- the three kernels of the gated delta rule's
// gradients (mathematics in gdn_grad.hpp), instantiated for bf16 inputs
// (gdn_grad_bf16.hip) and fp32 inputs (gdn_grad_f32.hip).
#pragma once

#include "gdn_grad.hpp"

namespace gdn {

// Eight columns of a tile row in the order kperm of k-block p.
template <class Eng, class Tile>
__device__ __forceinline__ typename Eng::Fr row_kperm(const char* t, int row, int p, int gq) {
  using E = typename Eng::E;
  constexpr int D = Tile::kUnits * 16 / (int)sizeof(E), kPer = 16 / (int)sizeof(E);
  const char* base = t + row * D * sizeof(E);
  const int c0 = 32 * p + 4 * gq, c1 = c0 + 16;
  return Eng::ld2((const E*)(base + 16 * lin_unit<Tile::kUnits>(row, c0 / kPer) + (c0 % kPer) * sizeof(E)),
                  (const E*)(base + 16 * lin_unit<Tile::kUnits>(row, c1 / kPer) + (c1 % kPer) * sizeof(E)));
}

// ---------------------------------------------------------------------------
// Records.  One workgroup of four waves for each (chunk, head).
// ---------------------------------------------------------------------------
template <class Eng, int DK>
struct GradPrepLds {
  static constexpr int kTile = kChunk * DK * (int)sizeof(typename Eng::E);
  static constexpr int kKQ = 2 * kTile > kChunk * kL64 * 4 ? 2 * kTile : kChunk * kL64 * 4;   // X overlays K and Q
  static constexpr int oA = kKQ;
  static constexpr int oG = oA + kChunk * kL64 * 4;
  static constexpr int bytes = oG + (int)sizeof(GradGates);
};

// One wave: the gates of a chunk.  The sums run in fp64 and base 2 (far tokens
// of a strongly decaying chunk differ by large G); a log-gate below -1e4 has
// the weight 0 and is held there.
__device__ __forceinline__ void grad_gates(GradGates& s, float g, float beta, int nv) {
  const int ln = threadIdx.x & 63;
  const double G = wave_prefix_f64((double)(g < -1e4f ? -1e4f : g) * 1.4426950408889634);
  const double C = last_lane(G);
  const LinLog x = lin_log(G);
  const float eg = lin_pow(x.n, x.f), ec = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(eg), 63));
  s.eg[ln] = ln < nv ? eg : 0.0f;
  s.el[ln] = ln < nv ? lin_pow(C - G) : 0.0f;
  // beta's gradient is a quotient by it: 0 goes as 2^-60 (rows past the end stay 0)
  s.beta[ln] = ln < nv && fabsf(beta) < 0x1p-60f ? copysignf(0x1p-60f, beta) : beta;
  s.ec[ln] = ec;
  s.n[ln] = x.n;
  s.f[ln] = x.f;
  s.g[ln] = g;
  s.zero[ln] = beta == 0.0f ? 1.0f : 0.0f;
}

// Four values into bf16 planes (or fp32), plane i at p + i * stride.
template <class Eng, int P>
__device__ __forceinline__ void put4(char* p, int stride, const float (&x)[4]) {
  if constexpr (!Eng::kSplit) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
    uint32_t a[3], b[3];
    if constexpr (P == 3) {
      split3_bf16x2(x[0], x[1], a[0], a[1], a[2]);
      split3_bf16x2(x[2], x[3], b[0], b[1], b[2]);
    } else {
      split_bf16x2(x[0], x[1], a[0], a[1]);
      split_bf16x2(x[2], x[3], b[0], b[1]);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) *reinterpret_cast<uint2*>(p + i * stride) = make_uint2(a[i], b[i]);
  }
}

template <class Eng, int DK>
__global__ __launch_bounds__(kThreads) void grad_prep_kernel(GradArgs a) {
  using E = typename Eng::E;
  using TK = LinTile<E, DK>;
  using Rows = LinRows<E, DK, kThreads>;
  using Rec = GradRec<Eng>;
  using Ls = GradPrepLds<Eng, DK>;
  extern __shared__ __align__(16) char smem[];
  if (grad_refused(a)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = kStatusBadIndex;
    return;
  }
  const int j = blockIdx.x / a.H, h = blockIdx.x % a.H;
  if (j >= a.offs[a.N]) return;   // the grid is sized for the worst case
  const GradPlace pl = grad_place(a, j);
  const int nv = pl.nv;
  const uint32_t lds0 = lds_base_u32(smem);
  const int tid = threadIdx.x, w = uniform(tid >> 6), l64 = tid & 63, ln = l64 & 15, gq = l64 >> 4;
  const char* sK = smem;
  const char* sQ = smem + Ls::kTile;
  float* sX = reinterpret_cast<float*>(smem);
  float* sA = reinterpret_cast<float*>(smem + Ls::oA);
  GradGates& sg = *reinterpret_cast<GradGates*>(smem + Ls::oG);
  char* rec = a.rec + ((int64_t)j * a.H + h) * Rec::kBytes;

  const int64_t row0 = (int64_t)pl.t0 * a.H + h;
  Rows::ask(lds0, (const E*)a.k + row0 * DK, a.H * DK, nv);
  Rows::ask(lds0 + Ls::kTile, (const E*)a.q + row0 * DK, a.H * DK, nv);
  if (w == 0) {
    const bool live = l64 < nv;
    const float g = live ? a.g[row0 + (int64_t)l64 * a.H] : 0.0f, b = live ? a.beta[row0 + (int64_t)l64 * a.H] : 0.0f;
    grad_gates(sg, g, b, nv);
  }
  wait_vmem();
  __syncthreads();
  if (tid < (int)sizeof(GradGates) / 16)
    reinterpret_cast<uint4*>(rec + Rec::oG)[tid] = reinterpret_cast<const uint4*>(&sg)[tid];

  // the ten tiles (R, S): lane holds row r = 16 R + ln, columns s = 16 S + 4 gq + i
  for (int job = w; job < 10; job += 4) {
    const int R = job < 1 ? 0 : job < 3 ? 1 : job < 6 ? 2 : 3, S = job - R * (R + 1) / 2;
    f32x4 ck = {0.0f, 0.0f, 0.0f, 0.0f}, cq = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 0; p < DK / 32; ++p) {
      const auto af = TK::template row8<Eng>(sK, 16 * S + ln, 32 * p + 8 * gq);
      Eng::mma(ck, af, TK::template row8<Eng>(sK, 16 * R + ln, 32 * p + 8 * gq));
      Eng::mma(cq, af, TK::template row8<Eng>(sQ, 16 * R + ln, 32 * p + 8 * gq));
    }
    const int r = 16 * R + ln;
    const int rn = sg.n[r];
    const float rf = sg.f[r];
    float va[4], vp[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = 16 * S + 4 * gq + i;
      const float d = s <= r ? lin_pow(rn - sg.n[s], rf - sg.f[s]) : 0.0f;
      va[i] = s < r ? sg.beta[s] * d * ck[i] : 0.0f;
      vp[i] = s <= r && r < nv ? d * cq[i] : 0.0f;   // rows past the chunk's end are zero
    }
    *reinterpret_cast<float4*>(sA + r * kL64 + 16 * S + 4 * gq) = make_float4(va[0], va[1], va[2], va[3]);
    put4<Eng, Rec::kPPlanes>(rec + Rec::oP + tri_block(R, S) * Rec::kBlock + tri_at<Eng>(ln, 4 * gq) * (int)sizeof(E),
                             Rec::kPlane, vp);
  }
  __syncthreads();
  solve_unit_lower(sA, sX, tid);
  for (int i = tid; i < 640; i += kThreads) {   // (block, row, four columns)
    const int blk = i >> 6, r = (i >> 2) & 15, c = 4 * (i & 3);
    const int R = blk < 1 ? 0 : blk < 3 ? 1 : blk < 6 ? 2 : 3, S = blk - R * (R + 1) / 2;
    const float4 x = *reinterpret_cast<const float4*>(sX + (16 * R + r) * kL64 + 16 * S + c);
    const float x4[4] = {x.x, x.y, x.z, x.w};
    put4<Eng, Rec::kMPlanes>(rec + blk * Rec::kBlock + tri_at<Eng>(r, c) * (int)sizeof(E), Rec::kPlane, x4);
  }
}

// ---------------------------------------------------------------------------
// The chains.  A workgroup of four waves walks one sequence and head for 64
// value columns, forwards (S) or backwards (R); wave w holds columns 16 w ..
// 16 w + 15 of the transposed state in accumulators (rows: key channels as
// dkmap orders them), which are the B operand of K S^T as they stand; X, E,
// U follow the same way, from registers to registers.
// ---------------------------------------------------------------------------
template <class Eng, int DK>
struct GradScanLds {
  using E = typename Eng::E;
  static constexpr int kTile = kChunk * DK * (int)sizeof(E);
  static constexpr int kVTile = kChunk * 64 * (int)sizeof(E);
  static constexpr int oQ = kTile;                                 // backwards only
  static constexpr int oV = 2 * kTile;                             // V, or dO
  static constexpr int oM = oV + kVTile;
  static constexpr int oP = oM + GradRec<Eng>::oP;
  static constexpr int oG = oM + GradRec<Eng>::oG;
  static constexpr int buf = oG + 1024;
  static constexpr int kBufs = 2 * buf <= 160 * 1024 ? 2 : 1;
  static constexpr int bytes = kBufs * buf;
};

template <class Eng, int DK, bool kRev>
struct GradWalk {
  using E = typename Eng::E;
  using Fr = typename Eng::Fr;
  using TK = LinTile<E, DK>;
  using TV = LinTile<E, 64>;
  using Ls = GradScanLds<Eng, DK>;
  using Rec = GradRec<Eng>;
  static constexpr int NT = DK / 16, NKB = DK / 32;
  static constexpr int P = Eng::kSplit ? 3 : 1;   // planes of what the states are formed from

  const GradArgs& a;
  const int n, h, vt, w, ln, gq;
  f32x4 X[NT];

  __device__ __forceinline__ GradWalk(const GradArgs& args, int seq, int head, int tile)
      : a(args), n(seq), h(head), vt(tile), w(uniform(threadIdx.x >> 6)), ln(threadIdx.x & 15),
        gq((threadIdx.x >> 4) & 3) {}

  // element of a [dv][dk] state that X[tr][0] of this lane is
  __device__ __forceinline__ int at(int tr) const {
    return (64 * vt + 16 * w + ln) * DK + 32 * (tr / 2) + 8 * gq + 4 * (tr & 1);
  }
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int tr = 0; tr < NT; ++tr) {
      X[tr] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (p != nullptr) X[tr] = *reinterpret_cast<const f32x4*>(p + ((int64_t)n * a.H + h) * a.dv * DK + at(tr));
    }
  }
  __device__ __forceinline__ void store(float* p) const {
#pragma unroll
    for (int tr = 0; tr < NT; ++tr)
      *reinterpret_cast<f32x4*>(p + ((int64_t)n * a.H + h) * a.dv * DK + at(tr)) = X[tr];
  }

  __device__ __forceinline__ void ask(uint32_t buf, int j, int t0, int nv) const {
    using RK = LinRows<E, DK, kThreads>;
    using RV = LinRows<E, 64, kThreads>;
    const int64_t row0 = (int64_t)t0 * a.H + h;
    RK::ask(buf, (const E*)a.k + row0 * DK, a.H * DK, nv);
    if constexpr (kRev) RK::ask(buf + Ls::oQ, (const E*)a.q + row0 * DK, a.H * DK, nv);
    RV::ask(buf + Ls::oV, (const E*)(kRev ? a.d_o : a.v) + row0 * a.dv + 64 * vt, a.H * a.dv, nv);
    const char* rec = a.rec + ((int64_t)j * a.H + h) * Rec::kBytes;
    ask_bytes<4>(buf + Ls::oM, rec, kRev ? Rec::oG : Rec::oP);
    if (w == 3) lds_load16(rec + Rec::oG, (uint32_t)(threadIdx.x & 63) * 16, buf + Ls::oG);
  }

  // the state's planes of k-block p: 32 channels
  __device__ __forceinline__ void planes(int p, Fr (&f)[P]) const {
    const float x[8] = {X[2 * p][0], X[2 * p][1], X[2 * p][2], X[2 * p][3],
                        X[2 * p + 1][0], X[2 * p + 1][1], X[2 * p + 1][2], X[2 * p + 1][3]};
    split_planes<Eng, P>(x, f);
  }
  // the state for the gradients' kernel (past the caches, the half lines of each store would go to memory by
  // themselves: 835 MB for 530 in the training batch)
  __device__ __forceinline__ void dump(float* slot, int p) const {
#pragma unroll
    for (int tr = 2 * p; tr < 2 * p + 2; ++tr)
      *reinterpret_cast<f32x4*>(slot + at(tr)) = X[tr];
  }
  // acc = K X
  __device__ __forceinline__ void against_k(const char* sK, float* slot, f32x4 (&acc)[4]) const {
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) acc[rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 0; p < NKB; ++p) {
      Fr xf[P], kf[4];
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) kf[rt] = TK::template row8<Eng>(sK, 16 * rt + ln, 32 * p + 8 * gq);
      planes(p, xf);
      dump(slot, p);
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) Eng::mma(acc[rt], kf[rt], xf[i]);
    }
  }
  // X += A^T B for a tile A of 64 rows, B in planes
  __device__ __forceinline__ void update(const char* sA, const Fr (&b)[2][P]) {
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      constexpr int kStep = Eng::kSplit ? 4 : 2;   // row tiles whose products alternate
#pragma unroll
      for (int tr0 = 0; tr0 < NT; tr0 += kStep) {
        Fr af[kStep];
#pragma unroll
        for (int i = 0; i < kStep; ++i)
          af[i] = TK::template cols8<Eng, 8>(sA, kb, 32 * ((tr0 + i) / 2) + 4 * (i & 1), ln, gq);
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
          for (int t = 0; t < kStep; ++t) Eng::mma(X[tr0 + t], af[t], b[kb][i]);
      }
    }
  }
  __device__ __forceinline__ void weights(const float* v, int kb, float (&x)[8]) const {
    const f32x4 u = *reinterpret_cast<const f32x4*>(v + 32 * kb + 4 * gq);
    const f32x4 y = *reinterpret_cast<const f32x4*>(v + 32 * kb + 16 + 4 * gq);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = u[j];
      x[4 + j] = y[j];
    }
  }

  __device__ __forceinline__ void forward(const char* buf, float* slot) {
    const char* sM = buf + Ls::oM;
    const GradGates& g = *reinterpret_cast<const GradGates*>(buf + Ls::oG);
    f32x4 acc[4];
    against_k(buf, slot, acc);
    Fr xf[2][P];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      float v[8], e[8];
      frag_values(TV::template cols8<Eng, 4>(buf + Ls::oV, kb, 16 * w, ln, gq), v);
      weights(g.eg, kb, e);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = fmaf(-e[j], acc[2 * kb + (j >> 2)][j & 3], v[j]);
      split_planes<Eng, P>(v, xf[kb]);
    }
    f32x4 er[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) er[rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int rt = 2 * kb; rt < 4; ++rt) {
          const Fr mf = tri_rows<Eng>(sM + i * Rec::kPlane, rt, kb, ln, gq);
#pragma unroll
          for (int k = 0; plane_pair(i, k, P); ++k) Eng::mma(er[rt], mf, xf[kb][k]);
        }
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      float u[8], e[8];
      weights(g.el, kb, u);
      weights(g.beta, kb, e);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = u[j] * e[j] * er[2 * kb + (j >> 2)][j & 3];
      split_planes<Eng, P>(u, xf[kb]);
    }
    const float ec = g.ec[0];
#pragma unroll
    for (int tr = 0; tr < NT; ++tr)
#pragma unroll
      for (int r = 0; r < 4; ++r) X[tr][r] *= ec;
    update(buf, xf);
  }

  __device__ __forceinline__ void backward(const char* buf, float* slot) {
    const char* sM = buf + Ls::oM;
    const char* sP = buf + Ls::oP;
    const GradGates& g = *reinterpret_cast<const GradGates*>(buf + Ls::oG);
    Fr of[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) of[kb] = TV::template cols8<Eng, 4>(buf + Ls::oV, kb, 16 * w, ln, gq);
    f32x4 acc[4], fr[4];
    against_k(buf, slot, acc);
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) fr[rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < Rec::kPPlanes; ++i)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int rt = 0; rt < 2 * kb + 2; ++rt)
          Eng::mma(fr[rt], tri_cols<Eng>(sP + i * Rec::kPlane, rt, kb, ln, gq), of[kb]);
    Fr zf[2][P];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      float e[8], b[8];
      weights(g.el, kb, e);
      weights(g.beta, kb, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = b[j] * fmaf(e[j], acc[2 * kb + (j >> 2)][j & 3], fr[2 * kb + (j >> 2)][j & 3]);
      split_planes<Eng, P>(e, zf[kb]);
    }
    f32x4 y[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) y[rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int rt = 0; rt < 2 * kb + 2; ++rt) {
          const Fr mf = tri_cols<Eng>(sM + i * Rec::kPlane, rt, kb, ln, gq);
#pragma unroll
          for (int k = 0; plane_pair(i, k, P); ++k) Eng::mma(y[rt], mf, zf[kb][k]);
        }
    const float ec = g.ec[0];
#pragma unroll
    for (int tr = 0; tr < NT; ++tr)
#pragma unroll
      for (int r = 0; r < 4; ++r) X[tr][r] *= ec;
    Fr qf[2][P];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      float o[8], e[8], u[8];
      frag_values(of[kb], o);
      weights(g.eg, kb, e);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o[j] *= e[j];
        u[j] = -e[j] * y[2 * kb + (j >> 2)][j & 3];
      }
      split_planes<Eng, P>(o, qf[kb]);
      split_planes<Eng, P>(u, zf[kb]);
    }
    update(buf + Ls::oQ, qf);
    update(buf, zf);
  }

  // Rows of a segment behind its sequence: zero gradients.
  __device__ __forceinline__ void clear_padding(int t0, int t1) const {
    const int64_t from = (int64_t)t0 * a.H + h;
    for (int i = threadIdx.x; i < (t1 - t0) * 64; i += kThreads)
      ((E*)a.d_v)[(from + (int64_t)(i >> 6) * a.H) * a.dv + 64 * vt + (i & 63)] = 0;
    if (vt != 0) return;
    for (int i = threadIdx.x; i < (t1 - t0) * DK; i += kThreads) {
      const int64_t e = (from + (int64_t)(i / DK) * a.H) * DK + i % DK;
      ((E*)a.dq)[e] = 0;
      ((E*)a.dk)[e] = 0;
    }
    for (int i = threadIdx.x; i < t1 - t0; i += kThreads) {
      a.d_beta[from + (int64_t)i * a.H] = 0.0f;
      a.dg[from + (int64_t)i * a.H] = 0.0f;
    }
  }

  __device__ __forceinline__ void run(char* smem) {
    const uint32_t lds0 = lds_base_u32(smem);
    const int seg0 = uniform(a.cu[n]), end = uniform(a.cu[n + 1]);
    const int L = a.seq_lens ? uniform(a.seq_lens[n]) : end - seg0;
    const int nch = (L + kChunk - 1) / kChunk, chunk0 = uniform(a.offs[n]);
    if (kRev && seg0 + L < end) clear_padding(seg0 + L, end);
    load(kRev ? a.d_fin : a.init);
    auto chunk = [&](int it) { return kRev ? nch - 1 - it : it; };
    auto ask_chunk = [&](int it) {
      const int c = chunk(it);
      ask(lds0 + (uint32_t)((it % Ls::kBufs) * Ls::buf), chunk0 + c, seg0 + c * kChunk, min(kChunk, L - c * kChunk));
    };
    if (nch > 0) ask_chunk(0);
    for (int it = 0; it < nch; ++it) {
      const char* buf = smem + (it % Ls::kBufs) * Ls::buf;
      wait_vmem();
      __syncthreads();   // the chunk's rows are there; the other buffer is free
      if (Ls::kBufs == 2 && it + 1 < nch) ask_chunk(it + 1);
      float* slot = (kRev ? a.R : a.S) + ((int64_t)(chunk0 + chunk(it)) * a.H + h) * a.dv * DK;
      if constexpr (kRev) backward(buf, slot);
      else forward(buf, slot);
      if (Ls::kBufs == 1 && it + 1 < nch) {
        __syncthreads();
        ask_chunk(it + 1);
      }
    }
    if constexpr (kRev) store(a.d_init);
  }
};

// Workgroups 0 .. n_rev - 1 walk backwards, the rest (none with kept states)
// forwards.  Each direction's workgroups of an XCD (workgroup b runs on XCD b %
// 8) take neighbouring value tiles, which share K, Q and the records.
template <class Eng, int DK>
__global__ __launch_bounds__(kThreads, 1) void grad_scan_kernel(GradArgs a, int n_rev) {
  extern __shared__ __align__(16) char smem[];
  if (grad_refused(a)) return;
  const bool rev = (int)blockIdx.x < n_rev;
  const int nb = rev ? n_rev : (int)gridDim.x - n_rev, b = rev ? (int)blockIdx.x : (int)blockIdx.x - n_rev;
  const int xq = nb / 8, xr = nb % 8, xc = b % 8;
  const int item = xc * xq + min(xc, xr) + b / 8;
  const int tiles = a.dv / 64, vt = item % tiles, nh = item / tiles;
  if (rev) {
    GradWalk<Eng, DK, true> walk(a, nh / a.H, nh % a.H, vt);
    walk.run(smem);
  } else {
    GradWalk<Eng, DK, false> walk(a, nh / a.H, nh % a.H, vt);
    walk.run(smem);
  }
}

// ---------------------------------------------------------------------------
// The gradients of a (chunk, head), the value columns in tiles of TV = 16 G, by
// 2 G waves.  First wave c < G does a forward chain's step for 16 columns, from S
// as it is stored (fp32) and with the chains' precision: E, and o, the forward's
// output; wave G + c the backward one's: Y.  What beta's and the gates' gradients
// are made of falls off here, as sums over the columns: with p_r = dO_r.o_r -
// Y_r.V_r,
//     db_r = Y_r.E_r / b_r           dg_t = <dS, S> - sum_(r<t) p_r
// (S_t = a_t S_(t-1) + b_t e_t k_t^T leaves <dS_t, S_t> = <dS_(t+1), S_(t+1)> +
// p_t; dS is the gradient of S itself, the chunk before's R), so that errors of dg
// are relative to the sums of its own chunk.  (beta = 0 goes as 2^-60: Y is a
// multiple of it.)
//
// Then E and Y, and HV columns at a time S and R, go into LDS as two bf16 planes,
// and all waves contract over them: S and R against dO, Y, E (a wave: 32 channels and
// its share of the tokens), and the triangle's pairs dO E^T, Y E^T; last the
// pairs become W and N, and W, N and their transposes meet K and Q.
//
// The split over the directions leaves a wave half of the registers that both
// would take: sixteen waves a compute unit at 128 columns.
// ---------------------------------------------------------------------------
template <class Eng, int DK, int G>
struct GradChunkLds {
  using E = typename Eng::E;
  using Rec = GradRec<Eng>;
  static constexpr int NW = 2 * G;
  static constexpr int SP = Eng::kSplit ? 2 : 1;                    // planes of S, R, E, Y, W, N
  static constexpr int TV = 16 * G, HV = Eng::kSplit && G == 4 ? 64 : 32;   // columns of a tile and of a step's
  static constexpr int kTile = kChunk * DK * (int)sizeof(E);
  static constexpr int kVTile = kChunk * TV * (int)sizeof(E);
  static constexpr int kSTile = HV * DK * (int)sizeof(E);
  static constexpr int kTri = Rec::kPlane;
  static constexpr int oQ = kTile;
  static constexpr int oO = 2 * kTile;
  static constexpr int oG = oO + kVTile;
  static constexpr int oSum = oG + (int)sizeof(GradGates);          // [3][G][64] floats, [G] doubles
  static constexpr int base = oSum + 3 * G * kChunk * 4 + (G * 8 + 15) / 16 * 16;
  // first: V, M, P, and E in fp32 from the forward waves to the backward ones
  static constexpr int oV = base;
  static constexpr int oM = oV + kVTile;
  static constexpr int oP = oM + Rec::oP;
  static constexpr int oX = oM + Rec::oG;
  static constexpr int end1 = oX + G * 16 * 64 * 4;
  // then: E and Y, S and R of a step's columns
  static constexpr int oE = base;
  static constexpr int oY = oE + SP * kVTile;
  static constexpr int oS = oY + SP * kVTile;
  static constexpr int oR = oS + SP * kSTile;
  static constexpr int end2 = oR + SP * kSTile;
  // last: W, N
  static constexpr int oW = base;
  static constexpr int oN = oW + SP * kTri;
  static constexpr int end3 = oN + SP * kTri;
  static constexpr int bytes = end1 > end2 ? (end1 > end3 ? end1 : end3) : (end2 > end3 ? end2 : end3);
  static_assert(bytes <= 160 * 1024, "LDS budget exceeded");
  static_assert(base % 16 == 0 && TV % HV == 0, "16-byte aligned, whole steps");
};

// The lane, as a value that the compiler does not know from before: addresses
// formed from it are not those of an earlier part kept in registers.
__device__ __forceinline__ int fresh_lane() {
  int l = threadIdx.x;
  asm volatile("" : "+v"(l));
  return l & 63;
}

// The first part of a wave: its columns' state, E or Y, and sums.
template <class Eng, int DK, int G>
struct GradStep {
  using E = typename Eng::E;
  using Fr = typename Eng::Fr;
  using Ls = GradChunkLds<Eng, DK, G>;
  using Rec = GradRec<Eng>;
  using TK = LinTile<E, DK>;
  using TO = LinTile<E, Ls::TV>;
  static constexpr int P = Rec::kMPlanes, NKB = DK / 32, NT = DK / 16;

  char* smem;
  int c, ln, gq;        // columns 16 c .. of the tile
  f32x4 st[NT];         // S or R: tile tr holds channels dkmap(16 tr + 4 gq ..) of column 16 c + ln
  f32x4 x[4];           // E or Y: tokens 16 rt + 4 gq + i of it

  __device__ __forceinline__ const GradGates& gates() const {
    return *reinterpret_cast<const GradGates*>(smem + Ls::oG);
  }
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int tr = 0; tr < NT; ++tr) {
      st[tr] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (p != nullptr)
        st[tr] = *reinterpret_cast<const f32x4*>(p + (int64_t)(16 * c + ln) * DK + 8 * gq + 32 * (tr / 2) + 4 * (tr & 1));
    }
  }
  // this lane's part of <state at p, st>
  __device__ __forceinline__ float dot(const float* p) const {
    float z = 0.0f;
#pragma unroll
    for (int tr = 0; tr < NT; ++tr) {
      const f32x4 y = *reinterpret_cast<const f32x4*>(p + (int64_t)(16 * c + ln) * DK + 8 * gq + 32 * (tr / 2) + 4 * (tr & 1));
#pragma unroll
      for (int i = 0; i < 4; ++i) z = fmaf(st[tr][i], y[i], z);
    }
    return z;
  }
  // K (and Q) against the planes of the state
  template <bool kQ>
  __device__ __forceinline__ void against(f32x4 (&ck)[4], f32x4 (&cq)[4]) const {
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      ck[rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if constexpr (kQ) cq[rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int p = 0; p < NKB; ++p) {
      const float x8[8] = {st[2 * p][0], st[2 * p][1], st[2 * p][2], st[2 * p][3],
                           st[2 * p + 1][0], st[2 * p + 1][1], st[2 * p + 1][2], st[2 * p + 1][3]};
      Fr sf[P], f[4];
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) f[rt] = TK::template row8<Eng>(smem, 16 * rt + ln, 32 * p + 8 * gq);
      split_planes<Eng, P>(x8, sf);
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) Eng::mma(ck[rt], f[rt], sf[i]);
      if constexpr (kQ) {
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) f[rt] = TK::template row8<Eng>(smem + Ls::oQ, 16 * rt + ln, 32 * p + 8 * gq);
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
          for (int rt = 0; rt < 4; ++rt) Eng::mma(cq[rt], f[rt], sf[i]);
      }
      __builtin_amdgcn_sched_barrier(0);   // reads in flight stay within the registers
    }
  }
  __device__ __forceinline__ Fr column(int o, int kb) const {
    return TO::template cols8<Eng, 4>(smem + o, kb, 16 * c, ln, gq);
  }
  // acc += A b for the record's lower-triangular A at o, or its transpose
  template <bool kT, int PA>
  __device__ __forceinline__ void tri(f32x4 (&acc)[4], int o, const Fr (&b)[2][P]) const {
#pragma unroll
    for (int i = 0; i < PA; ++i)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int rt = kT ? 0 : 2 * kb; rt < (kT ? 2 * kb + 2 : 4); ++rt) {
          const char* p = smem + o + i * Rec::kPlane;
          const Fr a = kT ? tri_cols<Eng>(p, rt, kb, ln, gq) : tri_rows<Eng>(p, rt, kb, ln, gq);
#pragma unroll
          for (int k = 0; plane_pair(i, k, P); ++k) Eng::mma(acc[rt], a, b[kb][k]);
        }
  }
  static __device__ __forceinline__ void zero(f32x4 (&a)[4]) {
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) a[rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  // sums over the columns of v (this lane's tokens) into LDS, [G][64]
  __device__ __forceinline__ void sums(float* to, int rt, int i, float v) const {
    v = group_sum<16>(v);
    if (ln == 0) to[kChunk * c + 16 * rt + 4 * gq + i] = v;
  }

  // E = M (V - e^G K S^T) into x and, in fp32, for the backward wave; sums of dO.o
  __device__ __forceinline__ void forward(float* sum_o) {
    const GradGates& g = gates();
    f32x4 ks[4], o[4];
    against<true>(ks, o);
    Fr f[2][P];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      float v[8];
      frag_values(column(Ls::oV, kb), v);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int rt = 2 * kb + (k >> 2), i = k & 3;
        const float eg = g.eg[16 * rt + 4 * gq + i];
        v[k] = fmaf(-eg, ks[rt][i], v[k]);
        o[rt][i] *= eg;
      }
      split_planes<Eng, P>(v, f[kb]);
    }
    zero(x);
    tri<false, P>(x, Ls::oM, f);
    __builtin_amdgcn_sched_barrier(0);
    float* ex = reinterpret_cast<float*>(smem + Ls::oX) + c * 1024;
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) reinterpret_cast<f32x4*>(ex)[64 * rt + 16 * gq + ln] = x[rt];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      float u[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int rt = 2 * kb + (k >> 2), i = k & 3;
        u[k] = g.beta[16 * rt + 4 * gq + i] * x[rt][i];
      }
      split_planes<Eng, P>(u, f[kb]);
    }
    tri<false, Rec::kPPlanes>(o, Ls::oP, f);
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      float d[8];
      frag_values(column(Ls::oO, kb), d);
#pragma unroll
      for (int k = 0; k < 8; ++k) sums(sum_o, 2 * kb + (k >> 2), k & 3, d[k] * o[2 * kb + (k >> 2)][k & 3]);
    }
  }
  // Y = M^T b (P^T dO + e^(G_C - G) K R^T) into x; sums of Y.V
  __device__ __forceinline__ void backward(float* sum_v) {
    const GradGates& g = gates();
    f32x4 kr[4], f1[4];
    against<false>(kr, kr);
    zero(f1);
    Fr f[2][P];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const Fr of = column(Ls::oO, kb);
#pragma unroll
      for (int i = 0; i < Rec::kPPlanes; ++i)
#pragma unroll
        for (int rt = 0; rt < 2 * kb + 2; ++rt)
          Eng::mma(f1[rt], tri_cols<Eng>(smem + Ls::oP + i * Rec::kPlane, rt, kb, ln, gq), of);
    }
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      float z[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int rt = 2 * kb + (k >> 2), i = k & 3, t = 16 * rt + 4 * gq + i;
        z[k] = g.beta[t] * fmaf(g.el[t], kr[rt][i], f1[rt][i]);
      }
      split_planes<Eng, P>(z, f[kb]);
    }
    zero(x);
    tri<true, P>(x, Ls::oM, f);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      float v[8];
      frag_values(column(Ls::oV, kb), v);
#pragma unroll
      for (int k = 0; k < 8; ++k) sums(sum_v, 2 * kb + (k >> 2), k & 3, v[k] * x[2 * kb + (k >> 2)][k & 3]);
    }
  }
  // sums of Y.E, E from the forward wave
  __device__ __forceinline__ void meet(float* sum_b) const {
    const float* ex = reinterpret_cast<const float*>(smem + Ls::oX) + c * 1024;
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      const f32x4 e = reinterpret_cast<const f32x4*>(ex)[64 * rt + 16 * gq + ln];
#pragma unroll
      for (int i = 0; i < 4; ++i) sums(sum_b, rt, i, e[i] * x[rt][i]);
    }
  }
  // the state's planes, row `row` of a step's tile
  __device__ __forceinline__ void put_state(char* to, int row) const {
#pragma unroll
    for (int p = 0; p < NKB; ++p) {
      const int col = 32 * p + 8 * gq;
      const float x8[8] = {st[2 * p][0], st[2 * p][1], st[2 * p][2], st[2 * p][3],
                           st[2 * p + 1][0], st[2 * p + 1][1], st[2 * p + 1][2], st[2 * p + 1][3]};
      if constexpr (Eng::kSplit) {
        Fr f[2];
        Eng::split(x8, f[0], f[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          Eng::st((E*)(to + i * Ls::kSTile + row * DK * 2 + 16 * lin_unit<TK::kUnits>(row, col / 8)), f[i]);
      } else {
        *(float4*)(to + row * DK * 4 + 16 * lin_unit<TK::kUnits>(row, col / 4)) = make_float4(x8[0], x8[1], x8[2], x8[3]);
        *(float4*)(to + row * DK * 4 + 16 * lin_unit<TK::kUnits>(row, col / 4 + 1)) = make_float4(x8[4], x8[5], x8[6], x8[7]);
      }
    }
  }
  // x's planes, this lane's column of the token rows
  __device__ __forceinline__ void put_x(char* to) const {
    constexpr int kPer = 16 / (int)sizeof(E);
    const int col = 16 * c + ln, in = (col % kPer) * (int)sizeof(E);
#pragma unroll
    for (int rt = 0; rt < 4; ++rt)
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const int ra = 16 * rt + 4 * gq + i, rb = ra + 1;
        char* a = to + ra * Ls::TV * (int)sizeof(E) + 16 * lin_unit<TO::kUnits>(ra, col / kPer) + in;
        char* b = to + rb * Ls::TV * (int)sizeof(E) + 16 * lin_unit<TO::kUnits>(rb, col / kPer) + in;
        if constexpr (Eng::kSplit) {
          uint32_t hi, lo;
          split_bf16x2(x[rt][i], x[rt][i + 1], hi, lo);
          *(uint16_t*)a = (uint16_t)hi;
          *(uint16_t*)b = (uint16_t)(hi >> 16);
          *(uint16_t*)(a + Ls::kVTile) = (uint16_t)lo;
          *(uint16_t*)(b + Ls::kVTile) = (uint16_t)(lo >> 16);
        } else {
          *(float*)a = x[rt][i];
          *(float*)b = x[rt][i + 1];
        }
      }
  }
};

template <class Eng, int DK, int G, bool kOne>
__global__ __launch_bounds__(128 * G, G / 2) void grad_chunk_kernel(GradArgs a) {
  using E = typename Eng::E;
  using Fr = typename Eng::Fr;
  using Ls = GradChunkLds<Eng, DK, G>;
  using Rec = GradRec<Eng>;
  constexpr int NW = Ls::NW, SP = Ls::SP, TV = Ls::TV, HV = Ls::HV, T = 64 * NW;
  using TK = LinTile<E, DK>;
  using TO = LinTile<E, TV>;
  extern __shared__ __align__(16) char smem[];
  if (grad_refused(a)) return;
  const int j = blockIdx.x / a.H, h = blockIdx.x % a.H;
  if (j >= a.offs[a.N]) return;   // the grid is sized for the worst case
  const GradPlace pl = grad_place(a, j);
  const int nv = pl.nv, H = a.H, dv = a.dv;
  const uint32_t lds0 = lds_base_u32(smem);
  const int tid = threadIdx.x, w = uniform(tid >> 6);
  const bool rev = w >= G;
  const char* sK = smem;
  const char* sQ = smem + Ls::oQ;
  const char* sO = smem + Ls::oO;
  const GradGates& g = *reinterpret_cast<const GradGates*>(smem + Ls::oG);
  float* sum_o = reinterpret_cast<float*>(smem + Ls::oSum);         // [G][64] dO.o
  float* sum_v = sum_o + G * kChunk;                                // Y.V
  float* sum_b = sum_v + G * kChunk;                                // Y.E
  double* sum_z = reinterpret_cast<double*>(sum_b + G * kChunk);    // [G] <dS, S>

  const int64_t row0 = (int64_t)pl.t0 * H + h;
  const int64_t ch = (int64_t)j * H + h, state = (int64_t)dv * DK;
  const char* rec = a.rec + ch * Rec::kBytes;
  {
    using RK = LinRows<E, DK, T>;
    RK::ask(lds0, (const E*)a.k + row0 * DK, H * DK, nv);
    RK::ask(lds0 + Ls::oQ, (const E*)a.q + row0 * DK, H * DK, nv);
    ask_bytes<NW>(lds0 + Ls::oG, rec + Rec::oG, Rec::kGates);
  }
  // the entering state (kept, the initial one, or the chain's), its gradient, and the leaving one's
  const int64_t seq = ((int64_t)pl.n * H + h) * state;
  const float* ps = a.kept == nullptr ? a.S + ch * state
                    : pl.c > 0 ? a.kept + (ch - H) * state : a.init == nullptr ? nullptr : a.init + seq;
  const float* pd = pl.c > 0 ? a.R + (ch - H) * state : a.d_init + seq;
  const float* pr = a.R + ch * state;

  // this wave's share of the contractions: channels 32 wc .. 32 wc + 31, token tiles TPW tg ..
  constexpr int CP = DK / 32, TG = NW / CP < 4 ? NW / CP : 4, TPW = 4 / TG;
  constexpr bool kIdle = TG * CP < NW;   // more waves than shares (dk = 64 and 128 columns)
  const int wc = w % CP, tg = w / CP;
  const bool share = !kIdle || tg < TG;
  f32x4 aq[TPW][2], ax[TPW][2], as[TPW][2];
  // and of the triangle's ten tiles: w, w + NW, ..
  constexpr int NTri = (10 + NW - 1) / NW;
  f32x4 pe[NTri], ye[NTri];
  auto clear = [&] {
#pragma unroll
    for (int t = 0; t < TPW; ++t)
#pragma unroll
      for (int m = 0; m < 2; ++m) aq[t][m] = ax[t][m] = as[t][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NTri; ++i) pe[i] = ye[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  };
  if constexpr (!kOne) clear();
  auto tri_of = [](int job, int& Tt, int& St) {
    Tt = job < 1 ? 0 : job < 3 ? 1 : job < 6 ? 2 : 3;
    St = job - Tt * (Tt + 1) / 2;
  };
  double z = 0.0;
  float keep_p = 0.0f, keep_b = 0.0f;   // sums of the earlier tiles (wave c: its columns'; lane: token)

  for (int v0 = 0; kOne ? v0 == 0 : v0 < dv; v0 += TV) {
    f32x4 st[DK / 16];
    const int c = rev ? w - G : w;
    char* sE = smem + Ls::oE;
    char* sY = smem + Ls::oY;
    {
      const int l64 = fresh_lane();
      GradStep<Eng, DK, G> step;
      step.smem = smem;
      step.c = c;
      step.ln = l64 & 15;
      step.gq = l64 >> 4;
      step.load(rev ? pr + (int64_t)v0 * DK : ps == nullptr ? nullptr : ps + (int64_t)v0 * DK);
      if (v0 > 0) __syncthreads();   // the last tile is consumed
      {
        using RV = LinRows<E, TV, T>;
        RV::ask(lds0 + Ls::oO, (const E*)a.d_o + row0 * dv + v0, H * dv, nv);
        RV::ask(lds0 + Ls::oV, (const E*)a.v + row0 * dv + v0, H * dv, nv);
        ask_bytes<NW>(lds0 + Ls::oM, rec, Rec::oG);
      }
      if (!rev && ps != nullptr) z += (double)step.dot(pd + (int64_t)v0 * DK);
      wait_vmem();
      __syncthreads();
      if (rev) step.backward(sum_v);
      else step.forward(sum_o);
      __syncthreads();   // E has come
      if (rev) step.meet(sum_b);
      __syncthreads();
      if constexpr (!kOne) {
        if (!rev && v0 + TV < dv) {   // the next tile's sums take the place
          keep_p += sum_o[kChunk * w + l64] - sum_v[kChunk * w + l64];
          keep_b += sum_b[kChunk * w + l64];
        }
      }
      step.put_x(rev ? sY : sE);
#pragma unroll
      for (int tr = 0; tr < DK / 16; ++tr) st[tr] = step.st[tr];
    }
    if constexpr (kOne) clear();   // not kept through the first part

#pragma unroll
    for (int h0 = 0; h0 < TV; h0 += HV) {
      const int l64 = fresh_lane(), ln = l64 & 15, gq = l64 >> 4;
      char* sS = smem + Ls::oS;
      char* sR = smem + Ls::oR;
      if (h0 > 0) __syncthreads();   // the last columns are consumed
      if (16 * c >= h0 && 16 * c < h0 + HV) {
        GradStep<Eng, DK, G> step;
        step.c = c;
        step.ln = ln;
        step.gq = gq;
#pragma unroll
        for (int tr = 0; tr < DK / 16; ++tr) step.st[tr] = st[tr];
        step.put_state(rev ? sR : sS, 16 * c - h0 + ln);
      }
      __syncthreads();

      if (h0 == 0) {   // d_v: Y's first plane is Y rounded to bf16
        for (int i = tid; i < kChunk * TO::kUnits; i += T) {
          const int row = i / TO::kUnits, u = i % TO::kUnits;
          if (row < nv) {
            uint4 x = *reinterpret_cast<const uint4*>(sY + row * TV * (int)sizeof(E) + 16 * lin_unit<TO::kUnits>(row, u));
            if (g.zero[row] != 0.0f) x = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>((E*)a.d_v + (row0 + (int64_t)row * H) * dv + v0 + u * (16 / (int)sizeof(E))) = x;
          }
        }
      }
      // S against dO and Y, R against E (the barriers for the scheduler keep reads in flight within the registers)
      if (share) {
#pragma unroll
        for (int kb = 0; kb < HV / 32; ++kb) {
          auto column = [&](const char* p, Fr (&f)[2][SP]) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int i = 0; i < SP; ++i)
                f[m][i] = TK::template cols8<Eng, 8>(p + i * Ls::kSTile, kb, 32 * wc + 4 * m, ln, gq);
          };
          const int hb = h0 / 32 + kb;
          Fr sf[2][SP];
          column(sS, sf);
#pragma unroll
          for (int t = 0; t < TPW; ++t) {
            const int row = 16 * (TPW * tg + t) + ln;
            const Fr of = row_kperm<Eng, TO>(sO, row, hb, gq);
            Fr yf[SP];
#pragma unroll
            for (int i = 0; i < SP; ++i) yf[i] = row_kperm<Eng, TO>(sY + i * Ls::kVTile, row, hb, gq);
#pragma unroll
            for (int i = 0; i < SP; ++i)
#pragma unroll
              for (int m = 0; m < 2; ++m) Eng::mma(aq[t][m], sf[m][i], of);
#pragma unroll
            for (int i = 0; i < SP; ++i)
#pragma unroll
              for (int k = 0; plane_pair(i, k, SP); ++k)
#pragma unroll
                for (int m = 0; m < 2; ++m) Eng::mma(ax[t][m], sf[m][i], yf[k]);
          }
          __builtin_amdgcn_sched_barrier(0);
          column(sR, sf);
#pragma unroll
          for (int t = 0; t < TPW; ++t) {
            const int row = 16 * (TPW * tg + t) + ln;
            Fr ef[SP];
#pragma unroll
            for (int i = 0; i < SP; ++i) ef[i] = row_kperm<Eng, TO>(sE + i * Ls::kVTile, row, hb, gq);
#pragma unroll
            for (int i = 0; i < SP; ++i)
#pragma unroll
              for (int k = 0; plane_pair(i, k, SP); ++k)
#pragma unroll
                for (int m = 0; m < 2; ++m) Eng::mma(as[t][m], sf[m][i], ef[k]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      // the triangle: lane holds token t = 16 T + ln, s = 16 S + 4 gq + i
#pragma unroll
      for (int i = 0; i < NTri; ++i) {
        if (w + NW * i >= 10) break;
        int Tt, St;
        tri_of(w + NW * i, Tt, St);
#pragma unroll
        for (int p = 0; p < HV / 32; ++p) {
          const int col = h0 + 32 * p + 8 * gq;
          const Fr of = TO::template row8<Eng>(sO, 16 * Tt + ln, col);
          Fr ef[SP], yf[SP];
#pragma unroll
          for (int k = 0; k < SP; ++k) {
            ef[k] = TO::template row8<Eng>(sE + k * Ls::kVTile, 16 * St + ln, col);
            yf[k] = TO::template row8<Eng>(sY + k * Ls::kVTile, 16 * Tt + ln, col);
          }
#pragma unroll
          for (int k = 0; k < SP; ++k) {
            Eng::mma(pe[i], ef[k], of);
#pragma unroll
            for (int l = 0; plane_pair(k, l, SP); ++l) Eng::mma(ye[i], ef[k], yf[l]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  __syncthreads();   // the last columns are consumed

  {
    const int l64 = fresh_lane(), ln = l64 & 15, gq = l64 >> 4;
    if (!rev) {
      if constexpr (!kOne) {
        sum_o[kChunk * w + l64] += keep_p;
        sum_b[kChunk * w + l64] += keep_b;
      }
      z = last_lane(wave_prefix_f64(z));
      if (l64 == 0) sum_z[w] = z;
    }
    // pairs
#pragma unroll
    for (int i = 0; i < NTri; ++i) {
      if (w + NW * i >= 10) break;
      int Tt, St;
      tri_of(w + NW * i, Tt, St);
      const int t = 16 * Tt + ln, tn = g.n[t];
      const float tf = g.f[t];
      float wv[4], nn[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int s = 16 * St + 4 * gq + k;
        const float d = s <= t && t < nv ? g.beta[s] * lin_pow(tn - g.n[s], tf - g.f[s]) : 0.0f;
        wv[k] = d * pe[i][k];
        nn[k] = s < t ? -d * ye[i][k] : 0.0f;
      }
      const int at = tri_block(Tt, St) * Rec::kBlock + tri_at<Eng>(ln, 4 * gq) * (int)sizeof(E);
      put4<Eng, SP>(smem + Ls::oW + at, Ls::kTri, wv);
      put4<Eng, SP>(smem + Ls::oN + at, Ls::kTri, nn);
    }
    if (share) {
#pragma unroll
      for (int t = 0; t < TPW; ++t) {
        const int tok = 16 * (TPW * tg + t) + ln;
        const float eg = g.eg[tok], bl = g.beta[tok] * g.el[tok];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            aq[t][m][r] *= eg;
            ax[t][m][r] = fmaf(bl, as[t][m][r], -eg * ax[t][m][r]);
          }
      }
    }
    __syncthreads();

    if (w == NW - 1) {
      const int t = l64;
      double p = 0.0, b = 0.0, zz = 0.0;
#pragma unroll
      for (int i = 0; i < G; ++i) {
        p += (double)sum_o[kChunk * i + t] - (double)sum_v[kChunk * i + t];
        b += (double)sum_b[kChunk * i + t];
        zz += sum_z[i];
      }
      double d = zz - (wave_prefix_f64(p) - p);
      if (g.g[t] < -104.0f) d = 0.0;   // e^-104 rounds to 0: nothing lies across the token
      if (t < nv) {
        a.d_beta[row0 + (int64_t)t * H] = (float)(b / (double)g.beta[t]);
        a.dg[row0 + (int64_t)t * H] = (float)d;
      }
    }
    if (!share) return;
  }
  // dq += W K, dk += W^T Q + N K + N^T K; a lane: token 16 tile + ln, channels 32 wc + 8 gq ..
  const int lz = fresh_lane(), lnz = lz & 15, gz = lz >> 4;
#pragma unroll
  for (int kb = 0; kb < 2; ++kb) {
    Fr kf[2], qf[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      kf[m] = TK::template cols8<Eng, 8>(sK, kb, 32 * wc + 4 * m, lnz, gz);
      qf[m] = TK::template cols8<Eng, 8>(sQ, kb, 32 * wc + 4 * m, lnz, gz);
    }
#pragma unroll
    for (int t = 0; t < TPW; ++t) {
      const int tile = TPW * tg + t;
#pragma unroll
      for (int i = 0; i < SP; ++i) {
        const char* sW = smem + Ls::oW + i * Ls::kTri;
        const char* sN = smem + Ls::oN + i * Ls::kTri;
        if (2 * kb <= tile) {
          const Fr wf = tri_rows<Eng>(sW, tile, kb, lnz, gz), nf = tri_rows<Eng>(sN, tile, kb, lnz, gz);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            Eng::mma(aq[t][m], kf[m], wf);
            Eng::mma(ax[t][m], kf[m], nf);
          }
        }
        if (2 * kb + 1 >= tile) {
          const Fr wf = tri_cols<Eng>(sW, tile, kb, lnz, gz), nf = tri_cols<Eng>(sN, tile, kb, lnz, gz);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            Eng::mma(ax[t][m], qf[m], wf);
            Eng::mma(ax[t][m], kf[m], nf);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int t = 0; t < TPW; ++t) {
    const int tok = 16 * (TPW * tg + t) + lnz;
    if (tok >= nv) continue;
    const int64_t at = (row0 + (int64_t)tok * H) * DK + 32 * wc + 8 * gz;
    const float q8[8] = {aq[t][0][0], aq[t][0][1], aq[t][0][2], aq[t][0][3],
                         aq[t][1][0], aq[t][1][1], aq[t][1][2], aq[t][1][3]};
    const float k8[8] = {ax[t][0][0], ax[t][0][1], ax[t][0][2], ax[t][0][3],
                         ax[t][1][0], ax[t][1][1], ax[t][1][2], ax[t][1][3]};
    Eng::st((E*)a.dq + at, Eng::round(q8));
    Eng::st((E*)a.dk + at, Eng::round(k8));
  }
}

template <class Eng, int DK, int G, bool kOne>
hipError_t launch_grad_chunk(const GradArgs& a, int64_t items, hipStream_t stream) {
  auto kern = grad_chunk_kernel<Eng, DK, G, kOne>;
  constexpr size_t lds = GradChunkLds<Eng, DK, G>::bytes;
  static PerDeviceOnce once;
  hipError_t e = set_dyn_lds_once(once, (const void*)kern, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)items), dim3(128 * G), lds, stream, a);
  return hipGetLastError();
}

template <class Eng, int DK>
hipError_t launch_grad(const gdn_shape_t& s, const GradArgs& a, int64_t items, hipStream_t stream) {
  hipError_t e;
  if (items > 0) {
    auto kern = grad_prep_kernel<Eng, DK>;
    constexpr size_t lds = GradPrepLds<Eng, DK>::bytes;
    static PerDeviceOnce once;
    if ((e = set_dyn_lds_once(once, (const void*)kern, lds)) != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)items), dim3(kThreads), lds, stream, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  {
    auto kern = grad_scan_kernel<Eng, DK>;
    constexpr size_t lds = GradScanLds<Eng, DK>::bytes;
    static PerDeviceOnce once;
    if ((e = set_dyn_lds_once(once, (const void*)kern, lds)) != hipSuccess) return e;
    const int chains = s.n_seqs * s.n_heads * (s.dv / 64);
    hipLaunchKernelGGL(kern, dim3((unsigned)(a.kept ? chains : 2 * chains)), dim3(kThreads), lds, stream, a, chains);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (items > 0) {
    // 128 value columns at once, where that is all of them; else (and fp32, whose tiles would not fit) 64 at a time
    constexpr int kWide = Eng::kSplit ? 8 : 4;
    if (s.dv == 16 * kWide) e = launch_grad_chunk<Eng, DK, kWide, true>(a, items, stream);
    else e = launch_grad_chunk<Eng, DK, 4, false>(a, items, stream);
  } else {
    e = hipSuccess;
  }
  return e;
}

}  // namespace gdn
