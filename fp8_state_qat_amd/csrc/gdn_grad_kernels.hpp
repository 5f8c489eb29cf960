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
// Records.  One workgroup of four waves for each (chunk, head).  Bounded by
// memory: 16384 tokens, 16 heads of 128 read 0.14 GB and write 0.13 in 66 us.
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
// The chains.  A workgroup of 2 CG waves walks one sequence and head for 16 CG
// value columns, forwards (S) or backwards (R).  A pair of waves holds 16 columns
// of the transposed state in accumulators, wave HS of it half HS of the key
// channels (rows, as dkmap orders them), which are the B operand of K S^T as they
// stand.  A chunk's chain of products is long and each depends on the one before:
// two waves on a SIMD run beside each other where one waits, and each does half of
// every product.  K S^T is a sum over the channels: the waves swap halves of their
// sums, and wave HS goes on with tokens 32 HS .. 32 HS + 31, whose half of the
// triangular product it also forms (half kb of the operand is known to the wave
// kb; the other needs it where the triangle does); the halves of its result are
// swapped again for the state's update.  (One wave with all channels: a chunk in
// 9.4 thousand cycles, 7.4 thousand so.)
//
// States, E and Y have 24 bits in every product: operands formed on the way are
// three bf16 planes, K, Q, V and dO enter as they are.  With two planes beta's and
// the gates' gradients were off by 3e-6 to 5e-6.
//
// Memory and the chain bound it: 4 x 4096 tokens, 16 heads, 128 x 128 in bf16 take
// 358 us for 0.53 GB read and 0.81 written (3.7 TB/s of the copy's 5.0), matrix
// units busy 24% of the time, backwards alone 324 us, forwards 278; one sequence
// of 8192 tokens 378 us, 7.1 thousand cycles a chunk.  What did not help: loads of
// the next chunk through registers (417 us for 385), at the start or the end of a
// chunk alone (423, 413), 32 columns a wave (409).
// ---------------------------------------------------------------------------
template <class Eng, int DK, int CG>
struct GradScanLds {
  using E = typename Eng::E;
  static constexpr int kTile = kChunk * DK * (int)sizeof(E);
  static constexpr int kVTile = kChunk * 16 * CG * (int)sizeof(E);
  static constexpr int oQ = kTile;                                 // backwards only
  static constexpr int oV = 2 * kTile;                             // V, or dO
  static constexpr int oM = oV + kVTile;
  static constexpr int oP = oM + GradRec<Eng>::oP;
  static constexpr int oG = oM + GradRec<Eng>::oG;
  static constexpr int buf = oG + 1024;
  // what the waves of a pair swap: 2 KiB of sums for either, later planes in
  // their place; the other planes in the place of P, which is consumed by then
  // (forwards it is not there at all)
  static constexpr int kSwap = 4096, kPlanes = (Eng::kSplit ? 3 : 1) * 64 * 8 * (int)sizeof(E);
  static_assert(kPlanes <= kSwap && CG * kPlanes <= GradRec<Eng>::oG - GradRec<Eng>::oP, "the swaps' places");
  static constexpr int kBufs = 2 * buf + CG * kSwap <= 160 * 1024 ? 2 : 1;
  static constexpr int oSwap = kBufs * buf;
  static constexpr int bytes = oSwap + CG * kSwap;
  static_assert(bytes <= 160 * 1024, "LDS budget exceeded");
};

template <class Eng, int DK, int CG, int HS, bool kRev, bool kKept = false>
struct GradWalk {
  using E = typename Eng::E;
  using Fr = typename Eng::Fr;
  using TK = LinTile<E, DK>;
  using TV = LinTile<E, 16 * CG>;
  using Ls = GradScanLds<Eng, DK, CG>;
  using Rec = GradRec<Eng>;
  static constexpr int kT = 128 * CG, kW = 2 * CG;      // threads, waves
  static constexpr int NT = DK / 32, NKB = DK / 64;     // of this wave's channels
  static constexpr int P = Eng::kSplit ? 3 : 1;   // planes of what the states are formed from

  const GradArgs& a;
  const int n, h, vt, w, ln, gq;
  char* const smem;
  f32x4 X[NT];

  __device__ __forceinline__ GradWalk(const GradArgs& args, int seq, int head, int tile, char* lds)
      : a(args), n(seq), h(head), vt(tile), w(uniform(threadIdx.x >> 6)), ln(threadIdx.x & 15),
        gq((threadIdx.x >> 4) & 3), smem(lds) {}

  __device__ __forceinline__ int col0() const { return 16 * (w % CG); }   // of the tile
  // element of a [dv][dk] state that X[tr][0] of this lane is
  __device__ __forceinline__ int at(int tr) const {
    return (16 * CG * vt + col0() + ln) * DK + DK / 2 * HS + 32 * (tr / 2) + 8 * gq + 4 * (tr & 1);
  }
  // the state of entry i of p's
  __device__ __forceinline__ void load(const float* p, int64_t i) {
#pragma unroll
    for (int tr = 0; tr < NT; ++tr) {
      X[tr] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (p != nullptr) X[tr] = *reinterpret_cast<const f32x4*>(p + (i * a.H + h) * a.dv * DK + at(tr));
    }
  }

  // What the next chunk needs, in kAsks steps: a step's load for each wave
  // (records: wave w the KiB w, w + kW, ..; the gates beside the last).
  using RK = LinRows<E, DK, kT>;
  using RV = LinRows<E, 16 * CG, kT>;
  static_assert(RK::kAll % kT == 0 && RV::kAll % kT == 0, "every thread has its share of the rows");
  static constexpr int kRecKiB = (kRev ? Rec::oG : Rec::oP) / 1024;
  static constexpr int kAsks = RK::kPer * (kRev ? 2 : 1) + RV::kPer + (kRecKiB + kW) / kW;
  struct Next {
    uint32_t buf;   // of this wave: + 1024 w
    const E *k, *q, *v;
    const char* rec;
  };
  uint32_t ko[RK::kPer], vo[RV::kPer];   // this lane's bytes from them, for chunks of `rows` rows
  int rows = -1;
  __device__ __forceinline__ Next next(uint32_t buf, int j, int t0, int nv) {
    if (nv != rows) {   // rows from nv on are copies of the last valid one, which no result takes in
      rows = nv;
#pragma unroll
      for (int i = 0; i < RK::kPer; ++i) ko[i] = RK::offset(i, a.H * DK, nv);
#pragma unroll
      for (int i = 0; i < RV::kPer; ++i) vo[i] = RV::offset(i, a.H * a.dv, nv);
    }
    const int64_t row0 = (int64_t)t0 * a.H + h;
    return Next{buf + 1024 * w, (const E*)a.k + row0 * DK, (const E*)a.q + row0 * DK,
                (const E*)(kRev ? a.d_o : a.v) + row0 * a.dv + 16 * CG * vt,
                a.rec + ((int64_t)j * a.H + h) * Rec::kBytes + 1024 * w};
  }
  __device__ __forceinline__ void ask(const Next& x, int i) const {
    if (i < RK::kPer) return lds_load16(x.k, ko[i], x.buf + 16 * kT * i);
    i -= RK::kPer;
    if (kRev) {
      if (i < RK::kPer) return lds_load16(x.q, ko[i], x.buf + Ls::oQ + 16 * kT * i);
      i -= RK::kPer;
    }
    if (i < RV::kPer) return lds_load16(x.v, vo[i], x.buf + Ls::oV + 16 * kT * i);
    i -= RV::kPer;
    const uint32_t lane16 = (uint32_t)(16 * (16 * gq + ln));
    if (kW * (i + 1) <= kRecKiB || kW * i + w < kRecKiB) {
      lds_load16(x.rec + 1024 * kW * i, lane16, x.buf + Ls::oM + 1024 * kW * i);
    } else if (kW * i + w == kRecKiB) {
      lds_load16(x.rec - 1024 * w + Rec::oG, lane16, x.buf - 1024 * w + Ls::oG);
    }
  }
  // job i of n asks for its share
  template <int N>
  __device__ __forceinline__ void ask_share(const Next& x, int i) const {
    if (Ls::kBufs == 1) return;
#pragma unroll
    for (int k = 0; k < kAsks; ++k)
      if (k * N / kAsks == i) ask(x, k);
  }

  // the state's planes of k-block p: 32 channels
  __device__ __forceinline__ void planes(int p, Fr (&f)[P]) const {
    const float x[8] = {X[2 * p][0], X[2 * p][1], X[2 * p][2], X[2 * p][3],
                        X[2 * p + 1][0], X[2 * p + 1][1], X[2 * p + 1][2], X[2 * p + 1][3]};
    split_planes<Eng, P>(x, f);
  }
  // the state for the gradients' kernel (past the caches, the half lines of each store would go to memory by
  // themselves: 835 MB for 530 in the training batch)
  __device__ __forceinline__ void dump(float* slot) const {
#pragma unroll
    for (int tr = 0; tr < NT; ++tr)
      *reinterpret_cast<f32x4*>(slot + at(tr)) = X[tr];
  }
  // this wave's tokens of E or Y for the gradients' kernel, transposed: a token row for each value column
  __device__ __forceinline__ void keep(float* to, const f32x4 (&x)[2]) const {
#pragma unroll
    for (int r = 0; r < 2; ++r)
      *reinterpret_cast<f32x4*>(to + (16 * CG * vt + col0() + ln) * kChunk + 32 * HS + 16 * r + 4 * gq) = x[r];
  }
  static constexpr int PP = Rec::kPPlanes;
  static constexpr int kMax = Eng::kSplit ? 4 : 2, kStep = NT < kMax ? NT : kMax;   // row tiles of a group of the update
  static constexpr int NU = 2 * NT / kStep;
  using Frags = Fr[6];

  // N groups of products, each group's operands read while the one before runs
  // (the barriers hold the order against the compiler, which moves each read next
  // to its use).
  template <int N, class Load, class Work>
  static __device__ __forceinline__ void pipeline(Load load, Work work) {
    Frags f[2];
    load(0, f[0]);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i + 1 < N) load(i + 1, f[(i + 1) & 1]);
      __builtin_amdgcn_sched_barrier(0);
      work(i, f[i & 1]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // K's rows, channels of this wave's k-block p
  __device__ __forceinline__ void rows_k(const char* sK, int p, Frags& f) const {
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) f[rt] = TK::template row8<Eng>(sK, 16 * rt + ln, DK / 2 * HS + 32 * p + 8 * gq);
  }
  // P^T's blocks (a plane): row tile rt, k-blocks from rt / 2 on
  __device__ __forceinline__ void blocks_p(const char* p, Frags& f) const {
    int n = 0;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int rt = 0; rt < 2 * kb + 2; ++rt) f[n++] = tri_cols<Eng>(p, rt, kb, ln, gq);
  }
  __device__ __forceinline__ void by_p(f32x4 (&acc)[4], const Frags& f, const Fr (&b)[2]) const {
    int n = 0;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int rt = 0; rt < 2 * kb + 2; ++rt) Eng::mma(acc[rt], f[n++], b[kb]);
  }
  // M's blocks (or M^T's) of this wave's tokens: k-blocks up to HS (from HS on)
  static constexpr int kb0 = kRev ? HS : 0, kb1 = kRev ? 2 : HS + 1;
  __device__ __forceinline__ void blocks_m(const char* p, Frags& f) const {
#pragma unroll
    for (int kb = kb0; kb < kb1; ++kb)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        f[2 * (kb - kb0) + r] = kRev ? tri_cols<Eng>(p, 2 * HS + r, kb, ln, gq) : tri_rows<Eng>(p, 2 * HS + r, kb, ln, gq);
  }
  // acc += (plane i) b
  __device__ __forceinline__ void by_m(f32x4 (&acc)[2], const Frags& f, const Fr (&b)[2][P], int i) const {
#pragma unroll
    for (int k = 0; plane_pair(i, k, P); ++k)
#pragma unroll
      for (int kb = kb0; kb < kb1; ++kb)
#pragma unroll
        for (int r = 0; r < 2; ++r) Eng::mma(acc[r], f[2 * (kb - kb0) + r], b[kb][k]);
  }
  // group u of X += A^T b for a tile A of 64 rows
  __device__ __forceinline__ void columns(const char* sA, int u, Frags& f) const {
    const int kb = u / (NT / kStep), tr0 = u % (NT / kStep) * kStep;
#pragma unroll
    for (int i = 0; i < kStep; ++i)
      f[i] = TK::template cols8<Eng, 8>(sA, kb, DK / 2 * HS + 32 * ((tr0 + i) / 2) + 4 * (i & 1), ln, gq);
  }
  __device__ __forceinline__ void update(int u, const Frags& f, const Fr (&b)[2][P]) {
    const int kb = u / (NT / kStep), tr0 = u % (NT / kStep) * kStep;
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int t = 0; t < kStep; ++t) Eng::mma(X[tr0 + t], f[t], b[kb][i]);
  }
  __device__ __forceinline__ void decay(float ec) {
#pragma unroll
    for (int tr = 0; tr < NT; ++tr)
#pragma unroll
      for (int r = 0; r < 4; ++r) X[tr][r] *= ec;
  }
  template <int N>
  static __device__ __forceinline__ void zero(f32x4 (&x)[N]) {
#pragma unroll
    for (int rt = 0; rt < N; ++rt) x[rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  // of tokens 16 rt + 4 gq + j, rt from r0 on
  template <int N>
  __device__ __forceinline__ void weights(const float* v, int r0, float (&x)[N]) const {
#pragma unroll
    for (int r = 0; r < N / 4; ++r) {
      const f32x4 u = *reinterpret_cast<const f32x4*>(v + 16 * (r0 + r) + 4 * gq);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[4 * r + j] = u[j];
    }
  }

  // The pair's swaps.  The receiver is the wave whose half of the triangular
  // product needs the other's (the sender's) half of the operand.
  static constexpr bool kReceiver = kRev == (HS == 0);
  __device__ __forceinline__ char* swap() const { return smem + Ls::oSwap + (w % CG) * Ls::kSwap; }
  __device__ __forceinline__ int lane() const { return 16 * gq + ln; }
  __device__ __forceinline__ void give_sums(const f32x4 (&x)[4]) const {   // the other's tokens
#pragma unroll
    for (int r = 0; r < 2; ++r)
      reinterpret_cast<f32x4*>(swap() + 2048 * (1 - HS))[64 * r + lane()] = x[2 * (1 - HS) + r];
  }
  __device__ __forceinline__ f32x4 other_sums(int r) const {
    return reinterpret_cast<const f32x4*>(swap() + 2048 * HS)[64 * r + lane()];
  }
  static __device__ __forceinline__ void put_planes(char* p, int lane, const Fr (&f)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) Eng::st((E*)p + 8 * (64 * i + lane), f[i]);
  }
  static __device__ __forceinline__ void get_planes(const char* p, int lane, Fr (&f)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) f[i] = Eng::ld((const E*)p + 8 * (64 * i + lane));
  }
  __device__ __forceinline__ char* swap_p(const char* buf) const {
    return const_cast<char*>(buf) + Ls::oP + (w % CG) * Ls::kPlanes;
  }
  __device__ __forceinline__ void give_half(const char* buf, const Fr (&f)[P]) const {
    if constexpr (!kReceiver) put_planes(swap_p(buf), lane(), f);
  }
  __device__ __forceinline__ void other_half(const char* buf, Fr (&f)[P]) const {
    if constexpr (kReceiver) get_planes(swap_p(buf), lane(), f);
  }
  __device__ __forceinline__ void give_update(const char* buf, const Fr (&f)[P]) const {
    put_planes(kReceiver ? swap_p(buf) : swap(), lane(), f);
  }
  __device__ __forceinline__ void other_update(const char* buf, Fr (&f)[P]) const {
    get_planes(kReceiver ? swap() : swap_p(buf), lane(), f);
  }

  // kKept: X is the state of this chunk alone, the next one's entry j (none: -1)
  __device__ __forceinline__ void forward(const char* buf, float* err, const Next& then, int64_t j) {
    const char* sM = buf + Ls::oM;
    const GradGates& g = *reinterpret_cast<const GradGates*>(buf + Ls::oG);
    constexpr int iM = NKB, iK = iM + P, N = kKept ? iK : iK + NU;
    f32x4 acc[4], er[2];
    zero(acc);
    zero(er);
    float eg[8], el[8], beta[8], ec = 0.0f;
    Fr vf, xf[2][P], pl[2][P];
    planes(0, pl[0]);
    pipeline<N>(
        [&](int i, Frags& f) {
          if (i < iM) rows_k(buf, i, f);
          if (i == iM - 1) {
            weights(g.eg, 2 * HS, eg);
            vf = TV::template cols8<Eng, 4>(buf + Ls::oV, HS, col0(), ln, gq);
            ec = g.ec[0];
          }
          if (i >= iM && i < iK) blocks_m(sM + (i - iM) * Rec::kPlane, f);
          if (i == iK - 1) {
            weights(g.el, 2 * HS, el);
            weights(g.beta, 2 * HS, beta);
          }
          if (i >= iK) columns(buf, i - iK, f);
        },
        [&](int i, const Frags& f) {
          ask_share<iK>(then, i);
          if (i < iM) {
            if (i + 1 < NKB) planes(i + 1, pl[(i + 1) & 1]);
#pragma unroll
            for (int k = 0; k < P; ++k)
#pragma unroll
              for (int rt = 0; rt < 4; ++rt) Eng::mma(acc[rt], f[rt], pl[i & 1][k]);
          } else if (i < iK) {
            if (i == iM) {
              give_sums(acc);
              if constexpr (!kKept) decay(ec);
              else if (j >= 0) load(a.kept, j);
              barrier_lds();
              float v[8];
              frag_values(vf, v);
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const f32x4 y = other_sums(r);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[4 * r + j] = fmaf(-eg[4 * r + j], acc[2 * HS + r][j] + y[j], v[4 * r + j]);
              }
              split_planes<Eng, P>(v, xf[HS]);
              give_half(buf, xf[HS]);
              barrier_lds();
              other_half(buf, xf[1 - HS]);
            }
            by_m(er, f, xf, i - iM);
          } else {
            if (i == iK) {
              keep(err, er);
              float u[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) u[j] = el[j] * beta[j] * er[j >> 2][j & 3];
              split_planes<Eng, P>(u, xf[HS]);
              give_update(buf, xf[HS]);
              barrier_lds();
              other_update(buf, xf[1 - HS]);
            }
            update(i - iK, f, xf);
          }
        });
    if constexpr (kKept) keep(err, er);
  }

  // The products with K (state) and P (the first wave one plane, the second the
  // others: it has less of M), the update by dO, which needs nothing of the chain,
  // in two parts beside the swaps, Y, the update by Y.
  __device__ __forceinline__ void backward(const char* buf, float* dvs, const Next& then) {
    const GradGates& g = *reinterpret_cast<const GradGates*>(buf + Ls::oG);
    constexpr int p0 = HS == 0 ? PP - 1 : 0, NP = PP == 1 ? (HS == 0 ? 0 : 1) : HS == 0 ? 1 : PP - 1;
    constexpr int iP = NKB, iQ = iP + NP, iR = iQ + NU / 2, iM = iR + NU / 2, iK = iM + P, N = iK + NU;
    f32x4 acc[4], fr[4], y[2];
    zero(acc);
    zero(fr);
    zero(y);
    float eg[16], el[16], beta[8], ec = 0.0f;
    Fr of[2], qf[2][P], zf[2][P], pl[2][P];
    planes(0, pl[0]);
    auto o = [&](int kb) {
      float x[8];
      frag_values(of[kb], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= eg[8 * kb + j];
      split_planes<Eng, P>(x, qf[kb]);
    };
    pipeline<N>(
        [&](int i, Frags& f) {
          if (i < iP) rows_k(buf, i, f);
          if (i == iP - 1) {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) of[kb] = TV::template cols8<Eng, 4>(buf + Ls::oV, kb, col0(), ln, gq);
            weights(g.eg, 0, eg);
            ec = g.ec[0];
          }
          if (i >= iP && i < iQ) blocks_p(buf + Ls::oP + (p0 + i - iP) * Rec::kPlane, f);
          if (i == iQ - 1) {
            weights(g.el, 0, el);
            weights(g.beta, 2 * HS, beta);
          }
          if (i >= iQ && i < iM) columns(buf + Ls::oQ, i - iQ, f);
          if (i >= iM && i < iK) blocks_m(buf + Ls::oM + (i - iM) * Rec::kPlane, f);
          if (i >= iK) columns(buf, i - iK, f);
        },
        [&](int i, const Frags& f) {
          ask_share<iK>(then, i);
          if (i < iP) {
            if (i + 1 < NKB) planes(i + 1, pl[(i + 1) & 1]);
#pragma unroll
            for (int k = 0; k < P; ++k)
#pragma unroll
              for (int rt = 0; rt < 4; ++rt) Eng::mma(acc[rt], f[rt], pl[i & 1][k]);
          } else if (i < iQ) {
            by_p(fr, f, of);
          } else if (i < iM) {
            if (i == iQ) {
#pragma unroll
              for (int rt = 0; rt < 4; ++rt)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[rt][j] = fmaf(el[4 * rt + j], acc[rt][j], fr[rt][j]);
              give_sums(acc);
              decay(ec);
              o(0);
              o(1);
            }
            if (i == iR) {
              barrier_lds();
              float x[8];
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const f32x4 t = other_sums(r);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[4 * r + j] = beta[4 * r + j] * (acc[2 * HS + r][j] + t[j]);
              }
              split_planes<Eng, P>(x, zf[HS]);
              give_half(buf, zf[HS]);
            }
            update(i - iQ, f, qf);
          } else if (i < iK) {
            if (i == iM) {
              barrier_lds();
              other_half(buf, zf[1 - HS]);
            }
            by_m(y, f, zf, i - iM);
          } else {
            if (i == iK) {
              keep(dvs, y);
              float x[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) x[j] = -eg[8 * HS + j] * y[j >> 2][j & 3];
              split_planes<Eng, P>(x, zf[HS]);
              give_update(buf, zf[HS]);
              barrier_lds();
              other_update(buf, zf[1 - HS]);
            }
            update(i - iK, f, zf);
          }
        });
  }

  // Rows of a segment behind its sequence: zero gradients.  Counted in 64 bits: a
  // segment may have 2^31 rows.
  __device__ __forceinline__ void clear_padding(int t0, int t1) const {
    constexpr int kC = 16 * CG, kPer = 16 / (int)sizeof(E);   // columns, of 16 bytes
    const int64_t rows = t1 - t0, from = (int64_t)t0 * a.H + h;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int64_t i = threadIdx.x; i < rows * (kC / kPer); i += kT)
      *reinterpret_cast<uint4*>((E*)a.d_v + (from + i / (kC / kPer) * a.H) * a.dv + kC * vt + i % (kC / kPer) * kPer) = zero;
    if (vt != 0) return;
    for (int64_t i = threadIdx.x; i < rows * (DK / kPer); i += kT) {
      const int64_t e = (from + i / (DK / kPer) * a.H) * DK + i % (DK / kPer) * kPer;
      *reinterpret_cast<uint4*>((E*)a.dq + e) = zero;
      *reinterpret_cast<uint4*>((E*)a.dk + e) = zero;
    }
    for (int64_t i = threadIdx.x; i < rows; i += kT) {
      a.d_beta[from + i * a.H] = 0.0f;
      a.dg[from + i * a.H] = 0.0f;
    }
  }

  __device__ __forceinline__ void run() {
    const uint32_t lds0 = lds_base_u32(smem);
    const int seg0 = uniform(a.cu[n]), end = uniform(a.cu[n + 1]);
    const int L = a.seq_lens ? uniform(a.seq_lens[n]) : end - seg0;
    const int nch = (L + kChunk - 1) / kChunk, chunk0 = uniform(a.offs[n]);
    if (kRev && seg0 + L < end) clear_padding(seg0 + L, end);
    load(kRev ? a.d_fin : a.init, n);
    auto chunk = [&](int it) { return kRev ? nch - 1 - it : it; };
    auto at = [&](int it) {
      const int c = chunk(it);
      return next(lds0 + (uint32_t)((it % Ls::kBufs) * Ls::buf), chunk0 + c, seg0 + c * kChunk, min(kChunk, L - c * kChunk));
    };
    auto ask_all = [&](int it) {
      const Next x = at(it);
#pragma unroll
      for (int k = 0; k < kAsks; ++k) ask(x, k);
    };
    auto slot = [&](int it) { return (int64_t)(chunk0 + chunk(it)) * a.H + h; };
    if (nch > 0) ask_all(0);
    if (!kKept && nch > 0) dump((kRev ? a.R : a.S) + slot(0) * a.dv * DK);
    for (int it = 0; it < nch; ++it) {
      const char* buf = smem + (it % Ls::kBufs) * Ls::buf;
      // the chunk's rows are there (asked for before the last chunk's stores, which have this one's time: 359 us for
      // 385 with them first, in the training batch); the other buffer and the swaps' places are free
      if (Ls::kBufs == 2 && it > 0 && !kKept) wait_vmem_but<NT + 2>();
      else wait_vmem();
      barrier_lds();
      // the last chunk asks for its own rows again, into the other buffer
      Next then = at(min(it + 1, nch - 1));
      then.buf = lds0 + (uint32_t)(((it + 1) % Ls::kBufs) * Ls::buf + 1024 * w);
      if constexpr (kRev) backward(buf, a.Y + slot(it) * a.dv * kChunk, then);
      else forward(buf, a.E + slot(it) * a.dv * kChunk, then, it + 1 < nch ? chunk0 + it : -1);
      if (!kKept && it + 1 < nch) dump((kRev ? a.R : a.S) + slot(it + 1) * a.dv * DK);
      if (Ls::kBufs == 1 && it + 1 < nch) {
        barrier_lds();
        ask_all(it + 1);
      }
    }
    wait_vmem();   // nothing is on the way into LDS when the wave ends
    if constexpr (kRev) dump(a.d_init + ((int64_t)n * a.H + h) * a.dv * DK);
  }
};

// Workgroups 0 .. n_rev - 1 walk backwards, the rest forwards (with kept states
// for E alone).  Each direction's workgroups of an XCD (workgroup b runs on XCD b %
// 8) take neighbouring value tiles, which share K, Q and the records.  Waves w and
// w + CG are a pair, on one SIMD.
template <class Eng, int DK, int CG>
__global__ __launch_bounds__(128 * CG, CG / 2) void grad_scan_kernel(GradArgs a, int n_rev) {
  extern __shared__ __align__(16) char smem[];
  if (grad_refused(a)) return;
  const bool rev = (int)blockIdx.x < n_rev;
  const int nb = rev ? n_rev : (int)gridDim.x - n_rev, b = rev ? (int)blockIdx.x : (int)blockIdx.x - n_rev;
  const int xq = nb / 8, xr = nb % 8, xc = b % 8;
  const int item = xc * xq + min(xc, xr) + b / 8;
  const int tiles = a.dv / (16 * CG), vt = item % tiles, nh = item / tiles, n = nh / a.H, h = nh % a.H;
  const bool second = uniform(threadIdx.x >> 6) >= CG;
  if (rev) {
    if (!second) GradWalk<Eng, DK, CG, 0, true>(a, n, h, vt, smem).run();
    else GradWalk<Eng, DK, CG, 1, true>(a, n, h, vt, smem).run();
  } else if (a.kept != nullptr) {
    if (!second) GradWalk<Eng, DK, CG, 0, false, true>(a, n, h, vt, smem).run();
    else GradWalk<Eng, DK, CG, 1, false, true>(a, n, h, vt, smem).run();
  } else {
    if (!second) GradWalk<Eng, DK, CG, 0, false>(a, n, h, vt, smem).run();
    else GradWalk<Eng, DK, CG, 1, false>(a, n, h, vt, smem).run();
  }
}

// ---------------------------------------------------------------------------
// The gradients of a (chunk, head) by four waves, 32 value columns at a time:
// S and R against dO, Y and E, and the triangle's pairs dO E^T, Y E^T; last the
// pairs become W and N, which meet K and Q with their transposes.  A wave has 32
// channels of S and R, which come from memory as the A operands of its products
// (a lane: two channels of eight columns), so that nothing but the tokens' rows
// passes through LDS, and 2 workgroups a compute unit cover each other's waits.
//
// beta's and the gates' gradients are sums of the same products: with the pairs
// B_rs = W_rs q_r.k_s + N_rs k_r.k_s (s < r),
//     db_r = Y_r.E_r / b_r
//     dg_t = e^(G_C) <R, S> + sum_(r>=t) (own_r + sum_s B_rs - sum_u B_ur)
//                           + sum_(s<t) b_s e^(G_C - G_s) k_s.(E R)_s
//     own_r = e^G (q_r.(dO S)_r - k_r.(Y S)_r)
// The sums over tokens and pairs are fp64, a pair the same fp32 number in its row
// and in its column: what does not lie across token t cancels to 2^-53, and dg keeps
// 20 bits and more also where a token forgets nearly all.  (By <dS, S> less the sum
// of dO_r.o_r - Y_r.V_r over the earlier tokens, which needs no k.(E R), errors were
// those of the whole chunk's sums, two to three times as large.)  beta = 0 goes as
// 2^-60: Y is a multiple of it.  All operands have the planes of the chains'
// products: with two planes, sixteen bits, of what dq and dk alone are made of (R,
// W, N) these differed from sums in fp32 by 1e-4 in norm, in values next to a border
// of bf16, for 1.7% of the time.
//
// Memory bounds it: 4 x 4096 tokens, 16 heads, 128 x 128 in bf16 take 305 us for
// 1.05 GB read and 0.24 written (4.2 TB/s of the copy's 5.0), at 1.85 GHz, matrix
// units busy a third of the time.  (Before, each chunk's E and Y were formed again
// here by sixteen waves and all of S, R, E, Y went through LDS: 555 us, most of it
// in one workgroup a compute unit's waits.)
// ---------------------------------------------------------------------------
template <class Eng, int DK>
struct GradChunkLds {
  using E = typename Eng::E;
  static constexpr int HV = 32;                          // columns of a step
  static constexpr int P = Eng::kSplit ? 3 : 1;          // planes of S, R, Y, E, W, N
  static constexpr int kTile = kChunk * DK * (int)sizeof(E);
  static constexpr int kStep = kChunk * HV * (int)sizeof(E);
  static constexpr int oQ = kTile;
  static constexpr int oG = 2 * kTile;
  static constexpr int oYE = oG + (int)sizeof(GradGates);   // [4][64] Y.E
  static constexpr int oQS = oYE + 4 * kChunk * 4;          // [4][64] q.(dO S)
  static constexpr int oKS = oQS + 4 * kChunk * 4;          // [4][64] k.(Y S)
  static constexpr int oKR = oKS + 4 * kChunk * 4;          // [4][64] k.(E R)
  static constexpr int oT = oKR + 4 * kChunk * 4;           // [64] the pairs' rows less their columns, fp64
  static constexpr int oZ = oT + kChunk * 8;                // [4] <R, S>
  static constexpr int oO = oZ + 4 * 8;                     // dO, twice, then planes of Y and of E, [column][token]
  static constexpr int oY = oO + 2 * kStep;
  static constexpr int oE = oY + P * kStep;
  static constexpr int oW = oO;                             // last W and N
  static constexpr int oN = oW + P * GradRec<Eng>::kPlane;
  static constexpr int oB = oN + P * GradRec<Eng>::kPlane;  // and the pairs' parts of the log-gates' gradients
  static constexpr int end1 = oE + P * kStep, end2 = oB + 10 * 256 * 4;
  static constexpr int bytes = end1 > end2 ? end1 : end2;
  static_assert(bytes <= 160 * 1024 && oO % 16 == 0, "LDS budget, 16-byte aligned");
};

// Eight values of a row fragment in the order kperm (or zeros) to memory.
template <class Eng>
__device__ __forceinline__ void put_dv(typename Eng::E* p, const typename Eng::Fr& f, bool zero) {
  if constexpr (Eng::kSplit) {
    uint4 u = __builtin_bit_cast(uint4, f);
    if (zero) u = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint2*>(p) = make_uint2(u.x, u.y);
    *reinterpret_cast<uint2*>(p + 16) = make_uint2(u.z, u.w);
  } else {
    *reinterpret_cast<float4*>(p) = zero ? float4{} : make_float4(f.v[0], f.v[1], f.v[2], f.v[3]);
    *reinterpret_cast<float4*>(p + 16) = zero ? float4{} : make_float4(f.v[4], f.v[5], f.v[6], f.v[7]);
  }
}

// The lane, as a value that the compiler does not know from before: addresses
// formed from it are not those of an earlier part kept in registers.
__device__ __forceinline__ int fresh_lane() {
  int l = threadIdx.x;
  asm volatile("" : "+v"(l));
  return l & 63;
}

template <class Eng, int DK>
__global__ __launch_bounds__(kThreads, Eng::kSplit ? 2 : 1) void grad_chunk_kernel(GradArgs a) {
  using E = typename Eng::E;
  using Fr = typename Eng::Fr;
  using Ls = GradChunkLds<Eng, DK>;
  using Rec = GradRec<Eng>;
  constexpr int P = Ls::P, HV = Ls::HV;
  using TK = LinTile<E, DK>;
  using TO = LinTile<E, HV>;
  using TY = LinTile<E, kChunk>;
  using RO = LinRows<E, HV, kThreads>;
  extern __shared__ __align__(16) char smem[];
  if (grad_refused(a)) return;
  const int j = blockIdx.x / a.H, h = blockIdx.x % a.H;
  if (j >= a.offs[a.N]) return;   // the grid is sized for the worst case
  const GradPlace pl = grad_place(a, j);
  const int nv = pl.nv, H = a.H, dv = a.dv;
  const uint32_t lds0 = lds_base_u32(smem);
  const int tid = threadIdx.x, w = uniform(tid >> 6);
  const char* sK = smem;
  const char* sQ = smem + Ls::oQ;
  const GradGates& g = *reinterpret_cast<const GradGates*>(smem + Ls::oG);

  const int64_t row0 = (int64_t)pl.t0 * H + h, ch = (int64_t)j * H + h;
  {
    using RK = LinRows<E, DK, kThreads>;
    RK::ask(lds0, (const E*)a.k + row0 * DK, H * DK, nv);
    RK::ask(lds0 + Ls::oQ, (const E*)a.q + row0 * DK, H * DK, nv);
    ask_bytes<4>(lds0 + Ls::oG, a.rec + ch * Rec::kBytes + Rec::oG, Rec::kGates);
  }
  // this wave's share: channels 32 wc .. 32 wc + 31, token tiles TPW tg ..
  constexpr int CP = DK / 32, TG = 4 / CP, TPW = 4 / TG;
  const int wc = w % CP, tg = TG == 1 ? 0 : w / CP;
  // the entering state (kept, the initial one, or the chain's) and the leaving one's gradient
  const int64_t state = (int64_t)dv * DK;
  const float* ps = a.kept == nullptr ? a.S + ch * state
                    : pl.c > 0 ? a.kept + (ch - H) * state
                    : a.init == nullptr ? nullptr : a.init + ((int64_t)pl.n * H + h) * state;
  const bool none = ps == nullptr;   // zeros
  if (none) ps = a.R + ch * state;
  const float* pr = a.R + ch * state;
  const float* pe_ = a.E + ch * dv * kChunk;
  const float* py_ = a.Y + ch * dv * kChunk;
  const E* po = (const E*)a.d_o + row0 * dv;

  // what the next step needs, on the way
  f32x2 sx[8], rx[8];        // columns kperm, channels 32 wc + 2 ln ..
  f32x4 ex[2], yx[2];        // column tid / 16 (+ 16), tokens 4 (tid % 16) ..
  auto fetch_state = [&](f32x2 (&x)[8], const float* p, int h0, int lanes) {
    const int l = fresh_lane(), at = (4 * (l >> 4) * DK + 2 * (l & 15)) & lanes;
    const float* c = p + (h0 * DK + 32 * wc);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = *reinterpret_cast<const f32x2*>(c + at + ((i & 3) + 16 * (i >> 2)) * DK);
  };
  auto fetch_rows = [&](int h0, int lanes) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ex[i] = *reinterpret_cast<const f32x4*>(pe_ + (h0 * kChunk + 1024 * i) + (4 * tid & lanes));
      yx[i] = *reinterpret_cast<const f32x4*>(py_ + (h0 * kChunk + 1024 * i) + (4 * tid & lanes));
    }
  };
  auto put_rows = [&](char* to, const f32x4 (&x)[2]) {   // planes, [column][token]
    const int l = w * 64 + fresh_lane();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int col = (l >> 4) + 16 * i, t0 = 4 * (l & 15);
      constexpr int kPer = 16 / (int)sizeof(E);
      const float x4[4] = {x[i][0], x[i][1], x[i][2], x[i][3]};
      put4<Eng, P>(to + col * kChunk * (int)sizeof(E) + 16 * lin_unit<TY::kUnits>(col, t0 / kPer) +
                       (t0 % kPer) * (int)sizeof(E),
                   Ls::kStep, x4);
    }
  };

  f32x4 aq[TPW][2], ax[TPW][2], as[TPW][2];
#pragma unroll
  for (int t = 0; t < TPW; ++t)
#pragma unroll
    for (int m = 0; m < 2; ++m) aq[t][m] = ax[t][m] = as[t][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // and of the triangle's ten tiles: w, w + 4, ..
  f32x4 pe[3], ye[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) pe[i] = ye[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto tri_of = [](int job, int& Tt, int& St) {
    Tt = job < 1 ? 0 : job < 3 ? 1 : job < 6 ? 2 : 3;
    St = job - Tt * (Tt + 1) / 2;
  };
  double z = 0.0;
  f32x4 dots = {0.0f, 0.0f, 0.0f, 0.0f};   // Y.E of tokens 4 (tid % 16) ..

  RO::ask(lds0 + Ls::oO, po, H * dv, nv);
  fetch_rows(0, ~0);
  fetch_state(sx, ps, 0, ~0);
  fetch_state(rx, pr, 0, ~0);
  __builtin_amdgcn_sched_barrier(0);
  for (int h0 = 0; h0 < dv; h0 += HV) {
    // the last step has no next one: each of its loads is of one place (a branch cost 48 registers' spills)
    const int hn = min(h0 + HV, dv - HV), lanes = h0 + HV < dv ? ~0 : 0;
    if (h0 > 0) barrier_lds();              // the last columns are consumed
    put_rows(smem + Ls::oY, yx);
    put_rows(smem + Ls::oE, ex);
    if (none) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sx[i] = f32x2{0.0f, 0.0f};
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) dots[k] = fmaf(ex[i][k], yx[i][k], dots[k]);
    Fr sf[2][P];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const float x8[8] = {sx[0][m], sx[1][m], sx[2][m], sx[3][m], sx[4][m], sx[5][m], sx[6][m], sx[7][m]};
      split_planes<Eng, P>(x8, sf[m]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) z += (double)fmaf(sx[i][1], rx[i][1], sx[i][0] * rx[i][0]);
    // dO, and first K, Q and the gates; R's eight loads came last
    wait_vmem_but<8>();
    barrier_lds();
    fetch_state(sx, ps, hn, lanes);
    __builtin_amdgcn_sched_barrier(0);

    // S against dO and Y
    const char* sO = smem + Ls::oO + (h0 / HV & 1) * Ls::kStep;
    const int l = fresh_lane(), ln = l & 15, gq = l >> 4;
#pragma unroll
    for (int t = 0; t < TPW; ++t) {
      const int tile = TPW * tg + t;
      const Fr of = row_kperm<Eng, TO>(sO, 16 * tile + ln, 0, gq);
      Fr yf[P];
#pragma unroll
      for (int i = 0; i < P; ++i)
        yf[i] = TY::template cols8<Eng, 4>(smem + Ls::oY + i * Ls::kStep, 0, 16 * tile, ln, gq);
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          Eng::mma(aq[t][m], sf[m][i], of);
          Eng::mma(ax[t][m], sf[m][0], yf[i]);
        }
#pragma unroll
      for (int i = 1; i < P; ++i)
#pragma unroll
        for (int k = 0; plane_pair(i, k, P); ++k)
#pragma unroll
          for (int m = 0; m < 2; ++m) Eng::mma(ax[t][m], sf[m][i], yf[k]);
      __builtin_amdgcn_sched_barrier(0);   // reads in flight stay within the registers
    }
    if (lanes) RO::ask(lds0 + Ls::oO + (h0 / HV + 1 & 1) * Ls::kStep, po + hn, H * dv, nv);
    fetch_rows(hn, lanes);
    // d_v, 16 tokens a wave: the first plane is Y rounded to bf16
    const Fr yw = TY::template cols8<Eng, 4>(smem + Ls::oY, 0, 16 * w, ln, gq);
    if (16 * w + ln < nv)
      put_dv<Eng>((E*)a.d_v + row0 * dv + h0 + (uint32_t)((16 * w + ln) * H * dv + 4 * gq), yw,
                  g.zero[16 * w + ln] != 0.0f);
    // R against E
    Fr rf[2][P];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const float x8[8] = {rx[0][m], rx[1][m], rx[2][m], rx[3][m], rx[4][m], rx[5][m], rx[6][m], rx[7][m]};
      split_planes<Eng, P>(x8, rf[m]);
    }
    fetch_state(rx, pr, hn, lanes);
#pragma unroll
    for (int t = 0; t < TPW; ++t) {
      Fr ef[P];
#pragma unroll
      for (int i = 0; i < P; ++i)
        ef[i] = TY::template cols8<Eng, 4>(smem + Ls::oE + i * Ls::kStep, 0, 16 * (TPW * tg + t), ln, gq);
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int k = 0; plane_pair(i, k, P); ++k)
#pragma unroll
          for (int m = 0; m < 2; ++m) Eng::mma(as[t][m], rf[m][i], ef[k]);
      __builtin_amdgcn_sched_barrier(0);
    }
    // the triangle: lane holds token t = 16 T + ln, s = 16 S + 4 gq + i
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      if (w + 4 * i >= 10) break;
      int Tt, St;
      tri_of(w + 4 * i, Tt, St);
      const Fr of = row_kperm<Eng, TO>(sO, 16 * Tt + ln, 0, gq);
      Fr ef[P], yf[P];
#pragma unroll
      for (int k = 0; k < P; ++k) {
        ef[k] = TY::template cols8<Eng, 4>(smem + Ls::oE + k * Ls::kStep, 0, 16 * St, ln, gq);
        yf[k] = TY::template cols8<Eng, 4>(smem + Ls::oY + k * Ls::kStep, 0, 16 * Tt, ln, gq);
      }
#pragma unroll
      for (int k = 0; k < P; ++k) {
        Eng::mma(pe[i], ef[k], of);
#pragma unroll
        for (int l = 0; plane_pair(k, l, P); ++l) Eng::mma(ye[i], ef[k], yf[l]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  barrier_lds();   // the last columns are consumed

  const int l64 = fresh_lane(), ln = l64 & 15, gq = l64 >> 4;
  auto over_quads = [](float v) {   // lanes ln, 16 + ln, 32 + ln, 48 + ln
    const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(x[0]) + __uint_as_float(x[1]);
    const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(y[0]) + __uint_as_float(y[1]);
  };
  float* sYE = reinterpret_cast<float*>(smem + Ls::oYE);
  float* sQS = reinterpret_cast<float*>(smem + Ls::oQS);
  float* sKS = reinterpret_cast<float*>(smem + Ls::oKS);
  float* sKR = reinterpret_cast<float*>(smem + Ls::oKR);
  double* sT = reinterpret_cast<double*>(smem + Ls::oT);
  float* sB = reinterpret_cast<float*>(smem + Ls::oB);
  double* sZ = reinterpret_cast<double*>(smem + Ls::oZ);
#pragma unroll
  for (int k = 0; k < 4; ++k) dots[k] = over_quads(dots[k]);
  if (gq == 0) *reinterpret_cast<f32x4*>(sYE + kChunk * w + 4 * ln) = dots;
  z = last_lane(wave_prefix_f64(z));
  if (l64 == 0) sZ[w] = tg == 0 ? z : 0.0;
#pragma unroll
  for (int t = 0; t < TPW; ++t) {
    const int tok = 16 * (TPW * tg + t) + ln;
    float q8[8], k8[8], dq = 0.0f, dk = 0.0f, dr = 0.0f;
    frag_values(TK::template row8<Eng>(sQ, tok, 32 * wc + 8 * gq), q8);
    frag_values(TK::template row8<Eng>(sK, tok, 32 * wc + 8 * gq), k8);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        dq = fmaf(q8[2 * i + m], aq[t][m][i], dq);
        dk = fmaf(k8[2 * i + m], ax[t][m][i], dk);
        dr = fmaf(k8[2 * i + m], as[t][m][i], dr);
      }
    dq = over_quads(dq);
    dk = over_quads(dk);
    dr = over_quads(dr);
    if (gq == 0) {
      sQS[kChunk * wc + tok] = dq;
      sKS[kChunk * wc + tok] = dk;
      sKR[kChunk * wc + tok] = dr;
    }
    // channels in the order of the products with K and Q
    const float eg = g.eg[tok], bl = g.beta[tok] * g.el[tok];
    f32x4 nq[2], nk[2];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      nq[c >> 2][c & 3] = eg * aq[t][c & 1][c >> 1];
      nk[c >> 2][c & 3] = fmaf(bl, as[t][c & 1][c >> 1], -eg * ax[t][c & 1][c >> 1]);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      aq[t][m] = nq[m];
      ax[t][m] = nk[m];
    }
  }
  // pairs
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (w + 4 * i >= 10) break;
    int Tt, St;
    tri_of(w + 4 * i, Tt, St);
    f32x4 cq = {0.0f, 0.0f, 0.0f, 0.0f}, ck = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 0; p < DK / 32; ++p) {
      const Fr kf = TK::template row8<Eng>(sK, 16 * St + ln, 32 * p + 8 * gq);
      Eng::mma(ck, kf, TK::template row8<Eng>(sK, 16 * Tt + ln, 32 * p + 8 * gq));
      Eng::mma(cq, kf, TK::template row8<Eng>(sQ, 16 * Tt + ln, 32 * p + 8 * gq));
    }
    const int t = 16 * Tt + ln, tn = g.n[t];
    const float tf = g.f[t];
    float wv[4], nn[4], b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int s = 16 * St + 4 * gq + k;
      const float d = s <= t && t < nv ? g.beta[s] * lin_pow(tn - g.n[s], tf - g.f[s]) : 0.0f;
      wv[k] = d * pe[i][k];
      nn[k] = s < t ? -d * ye[i][k] : 0.0f;
      b[k] = s < t ? fmaf(wv[k], cq[k], nn[k] * ck[k]) : 0.0f;
    }
    *reinterpret_cast<float4*>(sB + 256 * (w + 4 * i) + 16 * ln + 4 * gq) = make_float4(b[0], b[1], b[2], b[3]);
    const int at = tri_block(Tt, St) * Rec::kBlock + tri_at<Eng>(ln, 4 * gq) * (int)sizeof(E);
    put4<Eng, P>(smem + Ls::oW + at, Rec::kPlane, wv);
    put4<Eng, P>(smem + Ls::oN + at, Rec::kPlane, nn);
  }
  barrier_lds();
  {   // rows less columns of the pairs' parts, four lanes a token of this wave's sixteen
    const int tk = l64 >> 2, part = l64 & 3;
    double own = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i <= w) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(sB + 256 * tri_block(w, i) + 16 * tk + 4 * part);
        own += ((double)x[0] + (double)x[1]) + ((double)x[2] + (double)x[3]);
      }
      if (i >= w) {
        const float* x = sB + 256 * tri_block(i, w) + 64 * part + tk;
        own -= ((double)x[0] + (double)x[16]) + ((double)x[32] + (double)x[48]);
      }
    }
    own = dpp_add_f64<0xB1, 0xF>(own);   // lanes 1 0 3 2
    own = dpp_add_f64<0x4E, 0xF>(own);   // lanes 2 3 0 1
    if (part == 0) sT[16 * w + tk] = own;
  }
  barrier_lds();

  if (w == 3) {
    const int t = l64;
    double ye_ = 0.0, own = 0.0, out = 0.0, zz = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ye_ += (double)sYE[kChunk * i + t];
      zz += sZ[i];
      if (i < CP) {
        own += (double)sQS[kChunk * i + t] - (double)sKS[kChunk * i + t];
        out += (double)sKR[kChunk * i + t];
      }
    }
    own = fma(own, (double)g.eg[t], sT[t]);
    out *= (double)g.beta[t] * (double)g.el[t];
    const double later = wave_prefix_f64(own);
    double d = (double)g.ec[0] * zz + (last_lane(later) - later + own) + (wave_prefix_f64(out) - out);
    if (g.g[t] < -103.97208f) d = 0.0;   // e^g rounds to 0 (below 2^-150): nothing lies across the token
    if (t < nv) {
      a.d_beta[row0 + (int64_t)t * H] = (float)(ye_ / (double)g.beta[t]);
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
      for (int i = 0; i < P; ++i) {
        const char* sW = smem + Ls::oW + i * Rec::kPlane;
        const char* sN = smem + Ls::oN + i * Rec::kPlane;
        if (2 * kb <= tile) {
          const Fr wf = tri_rows<Eng>(sW, tile, kb, ln, gq), nf = tri_rows<Eng>(sN, tile, kb, ln, gq);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            Eng::mma(aq[t][m], kf[m], wf);
            Eng::mma(ax[t][m], kf[m], nf);
          }
        }
        if (2 * kb + 1 >= tile) {
          const Fr wf = tri_cols<Eng>(sW, tile, kb, ln, gq), nf = tri_cols<Eng>(sN, tile, kb, ln, gq);
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

template <class Eng, int DK, int CG>
hipError_t launch_grad_scan(const gdn_shape_t& s, const GradArgs& a, hipStream_t stream) {
  auto kern = grad_scan_kernel<Eng, DK, CG>;
  constexpr size_t lds = GradScanLds<Eng, DK, CG>::bytes;
  static PerDeviceOnce once;
  hipError_t e = set_dyn_lds_once(once, (const void*)kern, lds);
  if (e != hipSuccess) return e;
  const int chains = s.n_seqs * s.n_heads * (s.dv / (16 * CG));
  hipLaunchKernelGGL(kern, dim3((unsigned)(2 * chains)), dim3(128 * CG), lds, stream, a, chains);
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
  // 32 value columns a workgroup where a compute unit each is there for all of them, both ways: a chunk's step is
  // shorter (one sequence of 8192 tokens, 16 heads, 128 x 128: 378 us for 531), but two on a compute unit do not
  // fit (the training batch, twice as many as compute units: 429 us for 358)
  const bool few = (int64_t)s.n_seqs * s.n_heads * (s.dv / 32) * 2 <= device_cu_count();
  if ((e = few ? launch_grad_scan<Eng, DK, 2>(s, a, stream) : launch_grad_scan<Eng, DK, 4>(s, a, stream)) != hipSuccess)
    return e;
  if (items > 0) {
    auto kern = grad_chunk_kernel<Eng, DK>;
    constexpr size_t lds = GradChunkLds<Eng, DK>::bytes;
    static PerDeviceOnce once;
    if ((e = set_dyn_lds_once(once, (const void*)kern, lds)) != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)items), dim3(kThreads), lds, stream, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace gdn
