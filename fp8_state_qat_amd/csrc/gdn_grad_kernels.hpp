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
  s.beta[ln] = beta;
  s.ec[ln] = ec;
  s.n[ln] = x.n;
  s.f[ln] = x.f;
  s.g[ln] = g;
  s.pad[ln] = 0.0f;
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
    put4<Eng, Rec::kPPlanes>(rec + Rec::oP + tri_block(R, S) * Rec::kBlock + (16 * ln + 4 * gq) * (int)sizeof(E),
                             Rec::kPlane, vp);
  }
  __syncthreads();
  solve_unit_lower(sA, sX, tid);
  for (int i = tid; i < 640; i += kThreads) {   // (block, row, four columns)
    const int blk = i >> 6, r = (i >> 2) & 15, c = 4 * (i & 3);
    const int R = blk < 1 ? 0 : blk < 3 ? 1 : blk < 6 ? 2 : 3, S = blk - R * (R + 1) / 2;
    const float4 x = *reinterpret_cast<const float4*>(sX + (16 * R + r) * kL64 + 16 * S + c);
    const float x4[4] = {x.x, x.y, x.z, x.w};
    put4<Eng, Rec::kMPlanes>(rec + blk * Rec::kBlock + (16 * r + c) * (int)sizeof(E), Rec::kPlane, x4);
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

  // the state's planes of k-block p, its columns against 32 channels; the
  // first two are what the gradients' kernel reads
  __device__ __forceinline__ void planes(int p, Fr (&f)[P]) const {
    const float x[8] = {X[2 * p][0], X[2 * p][1], X[2 * p][2], X[2 * p][3],
                        X[2 * p + 1][0], X[2 * p + 1][1], X[2 * p + 1][2], X[2 * p + 1][3]};
    split_planes<Eng, P>(x, f);
  }
  __device__ __forceinline__ void dump(char* slot, int p, const Fr (&f)[P]) const {
    const int el = (64 * vt + 16 * w + ln) * DK + 32 * p + 8 * gq;
    if constexpr (Eng::kSplit) {
      const int64_t plane = (int64_t)a.dv * DK * 2;
      *reinterpret_cast<uint4*>(slot + 2 * el) = __builtin_bit_cast(uint4, f[0]);
      *reinterpret_cast<uint4*>(slot + plane + 2 * el) = __builtin_bit_cast(uint4, f[1]);
    } else {
      Eng::st((E*)slot + el, f[0]);
    }
  }
  // acc = K X
  __device__ __forceinline__ void against_k(const char* sK, char* slot, f32x4 (&acc)[4]) const {
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) acc[rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 0; p < NKB; ++p) {
      Fr xf[P], kf[4];
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) kf[rt] = TK::template row8<Eng>(sK, 16 * rt + ln, 32 * p + 8 * gq);
      planes(p, xf);
      dump(slot, p, xf);
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

  __device__ __forceinline__ void forward(const char* buf, char* slot) {
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

  __device__ __forceinline__ void backward(const char* buf, char* slot) {
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
      char* slot = (kRev ? a.R : a.S) + ((int64_t)(chunk0 + chunk(it)) * a.H + h) * grad_state_bytes(a.dv, DK);
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
// The gradients of a (chunk, head): eight waves, the value columns in tiles of
// TV.  For a tile, waves 0 .. TV / 16 - 1 form E and the next TV / 16 form Y, 16
// columns each, as the chains do; then all waves contract over the tile's
// columns: rows of S and R against dO, Y, E (a wave: 32 channels, 64 / (8 /
// (DK / 32)) tokens) and the triangle's pairs dO E^T, Y E^T (a wave: one or two
// 16 x 16 tiles).  After the last tile the pairs become W, N and the sums that
// beta's and the gates' gradients take.
// ---------------------------------------------------------------------------
constexpr int kGradThreads = 512;

template <class Eng, int DK>
struct GradChunkLds {
  using E = typename Eng::E;
  static constexpr int SP = Eng::kSplit ? 2 : 1;                    // planes of S, R, E, Y, W, N
  static constexpr int TV = Eng::kSplit || DK == 64 ? 64 : 32;      // value columns of a tile
  static constexpr int kTile = kChunk * DK * (int)sizeof(E);
  static constexpr int kVTile = kChunk * TV * (int)sizeof(E);
  static constexpr int kSTile = TV * DK * (int)sizeof(E);
  static constexpr int kTri = GradRec<Eng>::kPlane;
  static constexpr int oQ = kTile;
  static constexpr int oO = 2 * kTile;
  static constexpr int oE = oO + kVTile;                            // its first plane takes V's place
  static constexpr int oY = oE + SP * kVTile;
  static constexpr int oS = oY + SP * kVTile;
  static constexpr int oR = oS + SP * kSTile;
  static constexpr int oM = oR + SP * kSTile;
  static constexpr int oP = oM + SP * kTri;
  static constexpr int oG = oP + GradRec<Eng>::kPPlanes * kTri;
  static constexpr int bytes = oG + (int)sizeof(GradGates);
  // after the last tile: W and N in place of S and R, sums in place of dO
  static constexpr int oW = oS;
  static constexpr int oN = oW + SP * kTri;
  static_assert(oN + SP * kTri <= oM, "W and N fit over S and R");
  static constexpr int oSum = oO;
  static_assert((3 * 4 + 3 * 4) * kChunk * 4 + 64 <= kVTile, "the sums fit over dO");
  static_assert(bytes <= 160 * 1024, "LDS budget exceeded");
};

template <class Eng, int DK>
__global__ __launch_bounds__(kGradThreads, 2) void grad_chunk_kernel(GradArgs a) {
  using E = typename Eng::E;
  using Fr = typename Eng::Fr;
  using Ls = GradChunkLds<Eng, DK>;
  using Rec = GradRec<Eng>;
  constexpr int SP = Ls::SP, TV = Ls::TV, NKB = DK / 32;
  using TK = LinTile<E, DK>;
  using TT = LinTile<E, TV>;
  extern __shared__ __align__(16) char smem[];
  if (grad_refused(a)) return;
  const int j = blockIdx.x / a.H, h = blockIdx.x % a.H;
  if (j >= a.offs[a.N]) return;   // the grid is sized for the worst case
  const GradPlace pl = grad_place(a, j);
  const int nv = pl.nv, H = a.H, dv = a.dv;
  const uint32_t lds0 = lds_base_u32(smem);
  const int tid = threadIdx.x, w = uniform(tid >> 6), l64 = tid & 63, ln = l64 & 15, gq = l64 >> 4;
  const char* sK = smem;
  const char* sQ = smem + Ls::oQ;
  char* sO = smem + Ls::oO;
  char* sE = smem + Ls::oE;
  char* sY = smem + Ls::oY;
  char* sS = smem + Ls::oS;
  char* sR = smem + Ls::oR;
  const char* sM = smem + Ls::oM;
  const char* sP = smem + Ls::oP;
  const GradGates& g = *reinterpret_cast<const GradGates*>(smem + Ls::oG);

  const int64_t row0 = (int64_t)pl.t0 * H + h;
  const int64_t ch = (int64_t)j * H + h;
  {
    using RK = LinRows<E, DK, kGradThreads>;
    RK::ask(lds0, (const E*)a.k + row0 * DK, H * DK, nv);
    RK::ask(lds0 + Ls::oQ, (const E*)a.q + row0 * DK, H * DK, nv);
    const char* rec = a.rec + ch * Rec::kBytes;
    ask_bytes<8>(lds0 + Ls::oM, rec, SP * Ls::kTri);
    ask_bytes<8>(lds0 + Ls::oP, rec + Rec::oP, Rec::kBytes - Rec::oP);   // P and the gates
  }
  // the entering state: stored planes, or fp32 (kept, or the initial state)
  const float* s32 = nullptr;
  if (a.kept != nullptr) {
    if (pl.c > 0) s32 = a.kept + (ch - H) * dv * DK;
    else if (a.init != nullptr) s32 = a.init + ((int64_t)pl.n * H + h) * dv * DK;
  }
  const char* slotS = a.kept == nullptr ? a.S + ch * grad_state_bytes(dv, DK) : nullptr;
  const char* slotR = a.R + ch * grad_state_bytes(dv, DK);

  // this wave's share of the contractions: channels 32 wc .. 32 wc + 31, token tiles TPW tg ..
  constexpr int CP = DK / 32, TG = 8 / CP, TPW = 4 / TG;
  const int wc = w % CP, tg = w / CP;
  f32x4 aq[TPW][2], ax[TPW][2], as[TPW][2];
#pragma unroll
  for (int t = 0; t < TPW; ++t)
#pragma unroll
    for (int m = 0; m < 2; ++m) aq[t][m] = ax[t][m] = as[t][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // and of the triangle's tiles: w, and 8 + w where there is one
  const int n_tri = w < 2 ? 2 : 1;
  f32x4 pe[2], ye[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) pe[i] = ye[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto tri_at = [](int job, int& T, int& S) {
    T = job < 1 ? 0 : job < 3 ? 1 : job < 6 ? 2 : 3;
    S = job - T * (T + 1) / 2;
  };
  double z = 0.0;

  for (int v0 = 0; v0 < dv; v0 += TV) {
    if (v0 > 0) __syncthreads();   // the last tile is consumed
    {
      using RV = LinRows<E, TV, kGradThreads>;
      static_assert(TV == 64 || TV == 32, "tile rows");
      RV::ask(lds0 + Ls::oE, (const E*)a.v + row0 * dv + v0, H * dv, nv);
      RV::ask(lds0 + Ls::oO, (const E*)a.d_o + row0 * dv + v0, H * dv, nv);
      // TV rows of a state plane
      auto ask_state = [&](uint32_t to, const char* from) {
        constexpr int kUnits = DK * (int)sizeof(E) / 16, kAll = TV * kUnits;
        static_assert(kAll % kGradThreads == 0, "whole steps");
#pragma unroll
        for (int i = 0; i < kAll / kGradThreads; ++i) {
          const int idx = tid + kGradThreads * i, row = idx / kUnits, u = lin_unit<kUnits>(row, idx % kUnits);
          lds_load16(from, (uint32_t)(row * DK * (int)sizeof(E) + 16 * u), to + 16 * 64 * w + 16 * kGradThreads * i);
        }
      };
      const int64_t plane = (int64_t)dv * DK * 2;
#pragma unroll
      for (int i = 0; i < SP; ++i) {
        ask_state(lds0 + Ls::oR + i * Ls::kSTile, slotR + i * plane + (int64_t)v0 * DK * sizeof(E));
        if (slotS != nullptr)
          ask_state(lds0 + Ls::oS + i * Ls::kSTile, slotS + i * plane + (int64_t)v0 * DK * sizeof(E));
      }
      if (slotS == nullptr) {
        for (int i = tid; i < TV * DK / 8; i += kGradThreads) {
          const int row = i / (DK / 8), c = 8 * (i % (DK / 8));
          float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
          if (s32 != nullptr) {
            const float4* p = reinterpret_cast<const float4*>(s32 + (int64_t)(v0 + row) * DK + c);
            const float4 u = p[0], y = p[1];
            x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w; x[4] = y.x; x[5] = y.y; x[6] = y.z; x[7] = y.w;
          }
          if constexpr (Eng::kSplit) {
            Fr f[2];
            split_planes<Eng, 2>(x, f);
#pragma unroll
            for (int k = 0; k < 2; ++k)
              Eng::st((E*)(sS + k * Ls::kSTile + row * DK * 2 + 16 * lin_unit<TK::kUnits>(row, c / 8)), f[k]);
          } else {
            float4* p0 = (float4*)(sS + row * DK * 4 + 16 * lin_unit<TK::kUnits>(row, c / 4));
            float4* p1 = (float4*)(sS + row * DK * 4 + 16 * lin_unit<TK::kUnits>(row, c / 4 + 1));
            *p0 = make_float4(x[0], x[1], x[2], x[3]);
            *p1 = make_float4(x[4], x[5], x[6], x[7]);
          }
        }
      }
    }
    wait_vmem();
    __syncthreads();

    if (w < 2 * (TV / 16)) {
      const bool rev = w >= TV / 16;
      const int cw = rev ? w - TV / 16 : w;         // columns 16 cw ..
      const char* st = rev ? sR : sS;
      f32x4 acc[4], r4[4];
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) acc[rt] = r4[rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int p = 0; p < NKB; ++p) {
        Fr kf[4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) kf[rt] = TK::template row8<Eng>(sK, 16 * rt + ln, 32 * p + 8 * gq);
#pragma unroll
        for (int i = 0; i < SP; ++i) {
          const Fr sf = TK::template row8<Eng>(st + i * Ls::kSTile, 16 * cw + ln, 32 * p + 8 * gq);
#pragma unroll
          for (int rt = 0; rt < 4; ++rt) Eng::mma(acc[rt], kf[rt], sf);
        }
      }
      Fr xf[2][SP];
      const float* wt = rev ? g.el : g.eg;
      Fr vf[2];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) vf[kb] = TT::template cols8<Eng, 4>(rev ? sO : sE, kb, 16 * cw, ln, gq);
      if (rev) {
#pragma unroll
        for (int i = 0; i < Rec::kPPlanes; ++i)
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int rt = 0; rt < 2 * kb + 2; ++rt)
              Eng::mma(r4[rt], tri_cols<Eng>(sP + i * Rec::kPlane, rt, kb, ln, gq), vf[kb]);
      }
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        float x[8];
        frag_values(vf[kb], x);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int t = 32 * kb + 4 * gq + (k & 3) + 16 * (k >> 2);
          const float s = acc[2 * kb + (k >> 2)][k & 3];
          x[k] = rev ? g.beta[t] * fmaf(wt[t], s, r4[2 * kb + (k >> 2)][k & 3]) : fmaf(-wt[t], s, x[k]);
        }
        split_planes<Eng, SP>(x, xf[kb]);
      }
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) r4[rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (rev) {
#pragma unroll
        for (int i = 0; i < SP; ++i)
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int rt = 0; rt < 2 * kb + 2; ++rt) {
              const Fr mf = tri_cols<Eng>(sM + i * Ls::kTri, rt, kb, ln, gq);
#pragma unroll
              for (int k = 0; plane_pair(i, k, SP); ++k) Eng::mma(r4[rt], mf, xf[kb][k]);
            }
      } else {
#pragma unroll
        for (int i = 0; i < SP; ++i)
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int rt = 2 * kb; rt < 4; ++rt) {
              const Fr mf = tri_rows<Eng>(sM + i * Ls::kTri, rt, kb, ln, gq);
#pragma unroll
              for (int k = 0; plane_pair(i, k, SP); ++k) Eng::mma(r4[rt], mf, xf[kb][k]);
            }
      }
      // into the tile of E (over V, whose columns are this wave's too) or Y, row-major
      char* to = rev ? sY : sE;
      const int col = 16 * cw + ln;
#pragma unroll
      for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const int ra = 16 * rt + 4 * gq + i, rb = ra + 1;
          constexpr int kPer = 16 / (int)sizeof(E);
          const int oa = ra * TV * (int)sizeof(E) + 16 * lin_unit<TT::kUnits>(ra, col / kPer) + (col % kPer) * (int)sizeof(E);
          const int ob = rb * TV * (int)sizeof(E) + 16 * lin_unit<TT::kUnits>(rb, col / kPer) + (col % kPer) * (int)sizeof(E);
          if constexpr (Eng::kSplit) {
            uint32_t hi, lo;
            split_bf16x2(r4[rt][i], r4[rt][i + 1], hi, lo);
            *(uint16_t*)(to + oa) = (uint16_t)hi;
            *(uint16_t*)(to + ob) = (uint16_t)(hi >> 16);
            *(uint16_t*)(to + Ls::kVTile + oa) = (uint16_t)lo;
            *(uint16_t*)(to + Ls::kVTile + ob) = (uint16_t)(lo >> 16);
          } else {
            *(float*)(to + oa) = r4[rt][i];
            *(float*)(to + ob) = r4[rt][i + 1];
          }
        }
    }
    __syncthreads();

    // d_v: Y's first plane is Y rounded to bf16
    {
      constexpr int kUnits = TT::kUnits;
      for (int i = tid; i < kChunk * kUnits; i += kGradThreads) {
        const int row = i / kUnits, u = i % kUnits;
        if (row < nv)
          *reinterpret_cast<uint4*>((E*)a.d_v + (row0 + (int64_t)row * H) * dv + v0 + u * (16 / (int)sizeof(E))) =
              *reinterpret_cast<const uint4*>(sY + row * TV * (int)sizeof(E) + 16 * lin_unit<kUnits>(row, u));
      }
    }
    // S and R against dO, Y and E
#pragma unroll
    for (int kb = 0; kb < TV / 32; ++kb) {
      Fr sf[2][SP], rf[2][SP];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < SP; ++i) {
          sf[m][i] = TK::template cols8<Eng, 8>(sS + i * Ls::kSTile, kb, 32 * wc + 4 * m, ln, gq);
          rf[m][i] = TK::template cols8<Eng, 8>(sR + i * Ls::kSTile, kb, 32 * wc + 4 * m, ln, gq);
        }
#pragma unroll
      for (int t = 0; t < TPW; ++t) {
        const int row = 16 * (TPW * tg + t) + ln;
        const Fr of = row_kperm<Eng, TT>(sO, row, kb, gq);
        Fr yf[SP], ef[SP];
#pragma unroll
        for (int i = 0; i < SP; ++i) {
          yf[i] = row_kperm<Eng, TT>(sY + i * Ls::kVTile, row, kb, gq);
          ef[i] = row_kperm<Eng, TT>(sE + i * Ls::kVTile, row, kb, gq);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
#pragma unroll
          for (int i = 0; i < SP; ++i) Eng::mma(aq[t][m], sf[m][i], of);
#pragma unroll
          for (int i = 0; i < SP; ++i)
#pragma unroll
            for (int k = 0; plane_pair(i, k, SP); ++k) {
              Eng::mma(ax[t][m], sf[m][i], yf[k]);
              Eng::mma(as[t][m], rf[m][i], ef[k]);
            }
        }
      }
    }
    // the triangle: lane holds token t = 16 T + ln, s = 16 S + 4 gq + i
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i >= n_tri) break;
      int T, S;
      tri_at(i == 0 ? w : 8 + w, T, S);
#pragma unroll
      for (int p = 0; p < TV / 32; ++p) {
        const Fr of = TT::template row8<Eng>(sO, 16 * T + ln, 32 * p + 8 * gq);
        Fr ef[SP], yf[SP];
#pragma unroll
        for (int k = 0; k < SP; ++k) {
          ef[k] = TT::template row8<Eng>(sE + k * Ls::kVTile, 16 * S + ln, 32 * p + 8 * gq);
          yf[k] = TT::template row8<Eng>(sY + k * Ls::kVTile, 16 * T + ln, 32 * p + 8 * gq);
        }
#pragma unroll
        for (int k = 0; k < SP; ++k) {
          Eng::mma(pe[i], ef[k], of);
#pragma unroll
          for (int l = 0; plane_pair(k, l, SP); ++l) Eng::mma(ye[i], ef[k], yf[l]);
        }
      }
    }
    // <R, S>
    for (int i = tid; i < TV * DK / 8; i += kGradThreads) {
      float x[8], y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = y[k] = 0.0f;
#pragma unroll
      for (int k = 0; k < SP; ++k) {
        const int row = i / (DK / 8), c = 8 * (i % (DK / 8));
        float p[8];
        frag_values(TK::template row8<Eng>(sS + k * Ls::kSTile, row, c), p);
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] += p[q];
        frag_values(TK::template row8<Eng>(sR + k * Ls::kSTile, row, c), p);
#pragma unroll
        for (int q = 0; q < 8; ++q) y[q] += p[q];
      }
      float d = 0.0f;
#pragma unroll
      for (int q = 0; q < 8; ++q) d = fmaf(x[q], y[q], d);
      z += (double)d;
    }
  }
  __syncthreads();   // S, R, dO, E, Y are consumed

  float* sum_q = reinterpret_cast<float*>(smem + Ls::oSum);   // [CP][64] q.dq, k.dk (entering), k.dk (leaving, without beta)
  float* sum_x = sum_q + 4 * kChunk;
  float* sum_s = sum_x + 4 * kChunk;
  float* col_b = sum_s + 4 * kChunk;    // [4][64] by token tile: sums over t of P dO.E - B Y.E, t >= s
  float* col_s = col_b + 4 * kChunk;    // the same for t > s
  float* row_t = col_s + 4 * kChunk;    // [4][64] by s tile: sums over s of beta_s (..), s < t
  double* sum_z = reinterpret_cast<double*>(row_t + 4 * kChunk);
  z = last_lane(wave_prefix_f64(z));
  if (l64 == 0) sum_z[w] = z;

  // pairs
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (i >= n_tri) break;
    int T, S;
    tri_at(i == 0 ? w : 8 + w, T, S);
    f32x4 ck = {0.0f, 0.0f, 0.0f, 0.0f}, cq = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 0; p < NKB; ++p) {
      const Fr kf = TK::template row8<Eng>(sK, 16 * S + ln, 32 * p + 8 * gq);
      Eng::mma(ck, kf, TK::template row8<Eng>(sK, 16 * T + ln, 32 * p + 8 * gq));
      Eng::mma(cq, kf, TK::template row8<Eng>(sQ, 16 * T + ln, 32 * p + 8 * gq));
    }
    const int t = 16 * T + ln, tn = g.n[t];
    const float tf = g.f[t];
    float wv[4], nvv[4], row = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int s = 16 * S + 4 * gq + k;
      const bool low = s <= t && t < nv, strict = s < t && t < nv;
      const float b = g.beta[s];
      const float d = low ? lin_pow(tn - g.n[s], tf - g.f[s]) : 0.0f;
      const float de = d * pe[i][k], dy = strict ? d * ye[i][k] : 0.0f;
      wv[k] = b * de;
      nvv[k] = -b * dy;
      const float m1 = de * cq[k], m2 = dy * ck[k];
      const float cs = strict ? m1 - m2 : 0.0f;
      row = fmaf(b, cs, row);
      const float all = group_sum<16>(m1 - m2), off = group_sum<16>(cs);
      if (ln == 0) {
        col_b[kChunk * T + s] = all;
        col_s[kChunk * T + s] = off;
      }
    }
    row += __shfl_xor(row, 16, 64);
    row += __shfl_xor(row, 32, 64);
    if (gq == 0) row_t[kChunk * S + t] = row;
    const int at = tri_block(T, S) * Rec::kBlock + (16 * ln + 4 * gq) * (int)sizeof(E);
    put4<Eng, SP>(smem + Ls::oW + at, Ls::kTri, wv);
    put4<Eng, SP>(smem + Ls::oN + at, Ls::kTri, nvv);
  }
  // state parts, their weights, and their products with q and k
#pragma unroll
  for (int t = 0; t < TPW; ++t) {
    const int tok = 16 * (TPW * tg + t) + ln;
    const float eg = g.eg[tok], el = g.el[tok], b = g.beta[tok];
    float q[8], k[8];
    frag_values(TK::template row8<Eng>(sQ, tok, 32 * wc + 8 * gq), q);
    frag_values(TK::template row8<Eng>(sK, tok, 32 * wc + 8 * gq), k);
    float dq = 0.0f, dx = 0.0f, ds = 0.0f;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float q1 = eg * aq[t][m][r], x1 = -eg * ax[t][m][r], s1 = el * as[t][m][r];
        dq = fmaf(q[4 * m + r], q1, dq);
        dx = fmaf(k[4 * m + r], x1, dx);
        ds = fmaf(k[4 * m + r], s1, ds);
        aq[t][m][r] = q1;
        ax[t][m][r] = fmaf(b, s1, x1);
      }
    dq += __shfl_xor(dq, 16, 64);
    dq += __shfl_xor(dq, 32, 64);
    dx += __shfl_xor(dx, 16, 64);
    dx += __shfl_xor(dx, 32, 64);
    ds += __shfl_xor(ds, 16, 64);
    ds += __shfl_xor(ds, 32, 64);
    if (gq == 0) {
      sum_q[kChunk * wc + tok] = dq;
      sum_x[kChunk * wc + tok] = dx;
      sum_s[kChunk * wc + tok] = ds;
    }
  }
  __syncthreads();

  if (w == 0) {
    const int t = l64;
    double own = 0.0, out = 0.0, zz = 0.0;
    float col = 0.0f, off = 0.0f;
#pragma unroll
    for (int i = 0; i < CP; ++i) {
      own += (double)sum_q[kChunk * i + t] + (double)sum_x[kChunk * i + t];
      out += (double)sum_s[kChunk * i + t];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i <= t >> 4) own += (double)row_t[kChunk * i + t];
      if (i >= t >> 4) {
        col += col_b[kChunk * i + t];
        off += col_s[kChunk * i + t];
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) zz += sum_z[i];
    const double b = (double)g.beta[t];
    own -= b * (double)off;
    if (t >= nv) own = 0.0;
    const double head = wave_prefix_f64(own);
    double before = __shfl_up(wave_prefix_f64(b * out), 1, 64);   // without the token's own
    if (t == 0) before = 0.0;
    double d = (last_lane(head) - head + own) + before + zz * (double)g.ec[0];
    if (g.g[t] < -104.0f) d = 0.0;   // e^-104 rounds to 0: nothing lies across the token
    if (t < nv) {
      a.d_beta[row0 + (int64_t)t * H] = col + (float)out;
      a.dg[row0 + (int64_t)t * H] = (float)d;
    }
  }

  // dq += W K, dk += W^T Q + N K + N^T K; a lane: token 16 tile + ln, channels 32 wc + 8 gq ..
#pragma unroll
  for (int kb = 0; kb < 2; ++kb) {
    Fr kf[2], qf[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      kf[m] = TK::template cols8<Eng, 8>(sK, kb, 32 * wc + 4 * m, ln, gq);
      qf[m] = TK::template cols8<Eng, 8>(sQ, kb, 32 * wc + 4 * m, ln, gq);
    }
#pragma unroll
    for (int t = 0; t < TPW; ++t) {
      const int tile = TPW * tg + t;
#pragma unroll
      for (int i = 0; i < SP; ++i) {
        if (2 * kb <= tile) {
          const Fr wf = tri_rows<Eng>(smem + Ls::oW + i * Ls::kTri, tile, kb, ln, gq);
          const Fr nf = tri_rows<Eng>(smem + Ls::oN + i * Ls::kTri, tile, kb, ln, gq);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            Eng::mma(aq[t][m], kf[m], wf);
            Eng::mma(ax[t][m], kf[m], nf);
          }
        }
        if (2 * kb + 1 >= tile) {
          const Fr wf = tri_cols<Eng>(smem + Ls::oW + i * Ls::kTri, tile, kb, ln, gq);
          const Fr nf = tri_cols<Eng>(smem + Ls::oN + i * Ls::kTri, tile, kb, ln, gq);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            Eng::mma(ax[t][m], qf[m], wf);
            Eng::mma(ax[t][m], kf[m], nf);
          }
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TPW; ++t) {
    const int tok = 16 * (TPW * tg + t) + ln;
    if (tok >= nv) continue;
    const int64_t at = (row0 + (int64_t)tok * H) * DK + 32 * wc + 8 * gq;
    const float q8[8] = {aq[t][0][0], aq[t][0][1], aq[t][0][2], aq[t][0][3],
                         aq[t][1][0], aq[t][1][1], aq[t][1][2], aq[t][1][3]};
    const float k8[8] = {ax[t][0][0], ax[t][0][1], ax[t][0][2], ax[t][0][3],
                         ax[t][1][0], ax[t][1][1], ax[t][1][2], ax[t][1][3]};
    Eng::st((E*)a.dq + at, Eng::round(q8));
    Eng::st((E*)a.dk + at, Eng::round(k8));
  }
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
    auto kern = grad_chunk_kernel<Eng, DK>;
    constexpr size_t lds = GradChunkLds<Eng, DK>::bytes;
    static PerDeviceOnce once;
    if ((e = set_dyn_lds_once(once, (const void*)kern, lds)) != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)items), dim3(kGradThreads), lds, stream, a);
    e = hipGetLastError();
  } else {
    e = hipSuccess;
  }
  return e;
}

}  // namespace gdn
