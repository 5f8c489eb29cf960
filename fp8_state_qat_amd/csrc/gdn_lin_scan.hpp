// gdn_lin_scan.hpp -- the scan kernel of linear attention with a decay for
// each head, forward and backward.
//
// Mathematics.  With G_i the sum of the log decays of a 64-token chunk up to
// token i, D_ij = e^(G_i - G_j) and S the state entering the chunk,
//     o_i  = sum_{j<=i} D_ij (q_i.k_j) v_j      + e^(G_i) S q_i
//     S   <- e^(G_C) S + sum_j e^(G_C - G_j) v_j k_j^T
// The gradients are three more sums of the same form (dS: gradient of the
// state at the chunk's end, which runs backwards in time):
//     dq_i = sum_{j<=i} D_ij (do_i.v_j) k_j     + e^(G_i) S^T do_i
//     dk_j = sum_{i>=j} D_ij (v_j.do_i) q_i     + e^(G_C - G_j) dS^T v_j
//     dv_j = sum_{i>=j} D_ij (k_j.q_i) do_i     + e^(G_C - G_j) dS k_j
//     dS  <- e^(G_C) dS + sum_i e^(G_i) do_i q_i^T
// so one kernel serves all of them: out_a = sum_b w_ab (Q_a.K_b) V_b + in_a X^T Q_a,
// X <- e^(G_C) X + sum_b out_b K_b V_b^T, with the operands' roles and the
// direction set by the mode.
//
// Gradient of the log decays.  g_t scales every product that lies across it:
// in a chunk, with M_ij = D_ij (q_i.k_j)(do_i.v_j) for i > j, r_i = q_i.(state
// part of dq_i), c_j = k_j.(state part of dk_j) and X = e^(G_C) <S, dS>,
//     dg_t = sum_{i>=t} (sum_j M_ij + r_i) - sum_{j>=t} sum_i M_ij + sum_{j<t} c_j + X.
// X is formed from the two states in every chunk, the forward one stored by
// the dq pass.  (X = <S', dS> - sum_j c_j with the state S' at the chunk's end
// would let X be carried from chunk to chunk with few stored states, but what
// is large or not finite in a chunk's k and v would reach the earlier chunks
// through that difference: a row of v 1e5 times the others left errors of 2e-3
// there instead of 2e-7.)  So errors of dg are relative to the largest sums of
// its own chunk.
//
// Work split.  A workgroup owns one segment (a run of whole chunks of one
// sequence) of one virtual head (a value head, or a 64- or 128-row tile of
// one) and walks its chunks with X in fp32 accumulators: wave w holds the
// columns 16 w .. 16 w + 15 of X for all CK rows (eight waves at 128 columns;
// four with 32 columns each left the same time at 128 x 128 bf16 and 13 to
// 30% more on smaller tiles and fp32).  Segments of a sequence run
// at once: state passes first form every segment's own sum and decay, a small
// kernel turns them into the state at each segment's start.  The segment
// length is set by the host so that the card is full; with enough (sequence,
// head) pairs there is one segment a sequence and the state passes vanish.
//
// Products (bf16 inputs: v_mfma_f32_16x16x32_bf16; fp32 inputs: fp32 MFMA).
// Inputs enter as they are.  fp32 operands are split into bf16 planes: the
// pair weights (24 bits of them would not show in a bf16 output) into two, X
// into two where it only reaches a bf16 output and three where its product
// enters dg, the weighted V rows of the state update into three, so that the
// states and dg keep fp32 accuracy.  (Two planes leave 2e-6 of a value.)
// The row relabelling dkmap makes the accumulators of X, in place, the A
// operand of X^T Q;
// P^T = K Q^T comes out as the B operand of the product with V.
//
// LDS: Q, K, V tiles of the chunk (64 rows, 16-byte units XOR-swizzled so
// that row fragments, transpose reads and stores spread over the banks), the
// fragments of P, gate vectors of this and the next chunk.  bf16 rows go from
// memory straight into LDS: Q and V are free after the state part, K has a
// second tile, so the next chunk's rows are asked for in the middle of this
// one and a chunk needs two barriers (a state pass one).  At 128 x 128 the
// tiles take 80 KB: two workgroups a compute unit.  fp32 rows, which would not
// fit twice, are fetched into registers a chunk ahead.
//
// A wave's waits decide as much as its work: the compiler's own waits count
// only its own loads and so drain the asked rows too.  Inside the walk there
// are none between asking and using: the state is waited for before it, gates,
// DQ's rows of E and DK's stored states before the rows are asked for, and a
// chunk's stores stay in flight over its end (28 us of a training batch's 399).
//
// Measured (MI355X, bf16, 16 heads of 128 x 128, cold to warm): 32768 tokens in
// one sequence, state pass 62 to 68 us (268 MB; 62 with its products taken out),
// output pass 133 to 150 (537 MB; 105 to 116 without products, 131 with every
// load a cache hit; vector, matrix and LDS units are each busy 40 to 50% of the
// time).  Backward of 4 x 4096 tokens: state passes 66 to 80, dq 123 to 141,
// dk and dv 189 to 236, of which about 20 and 15 the state of every chunk
// takes, stored (235 MB) and read.
#pragma once

#include <type_traits>

#include "gdn_chunk_common.hpp"
#include "gdn_lin.hpp"

namespace gdn {

// ---------------------------------------------------------------------------
// Segments.  Sequence n has max(1, ceil(L_n / seglen)) of them, numbered
// through the batch; every wave finds its own by scanning cu_seqlens.
// ---------------------------------------------------------------------------
struct LinSeg {
  int n;        // sequence, -1: the slot is unused
  int s, nseg;  // this segment of the sequence, their number
  int t0, len;  // first row and rows
  int slot0;    // slot of the sequence's first segment
  bool bad;     // cu_seqlens out of contract
};

// want_seq: `at` is a sequence instead of a slot.
__device__ __forceinline__ LinSeg lin_find(const int32_t* __restrict__ cu, int N, int64_t T, int seglen, int at,
                                           bool want_seq) {
  LinSeg r;
  r.n = -1;
  r.s = r.nseg = r.t0 = r.len = r.slot0 = 0;
  r.bad = false;
  const int ln = threadIdx.x & 63;
  int base = 0;
  for (int n0 = 0; n0 < N; n0 += 64) {
    const int n = n0 + ln;
    const bool in = n < N;
    const int a = in ? cu[n] : 0, b = in ? cu[n + 1] : 0;
    const bool wrong = in && (a < 0 || b < a || b > T);
    if (__ballot(wrong) != 0) {
      r.bad = true;
      return r;
    }
    const int L = b - a;
    const int cnt = in ? (L > 0 ? (L - 1) / seglen + 1 : 1) : 0;
    int sum = cnt;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int v = __shfl_up(sum, off, 64);
      if (ln >= off) sum += v;
    }
    const int lo = base + sum - cnt;
    const bool mine = in && (want_seq ? n == at : (at >= lo && at < lo + cnt));
    const unsigned long long m = __ballot(mine);
    if (m != 0) {
      const int src = __ffsll((unsigned long long)m) - 1;
      r.n = n0 + src;
      r.nseg = uniform(__shfl(cnt, src, 64));
      r.slot0 = uniform(__shfl(lo, src, 64));
      r.s = want_seq ? 0 : at - r.slot0;
      const int rows = uniform(__shfl(L, src, 64)) - r.s * seglen;
      r.t0 = uniform(__shfl(a, src, 64)) + r.s * seglen;
      r.len = want_seq ? rows : (rows < seglen ? rows : seglen);
    }
    base += __shfl(sum, 63, 64);
  }
  return r;
}

// Swizzled 16-byte unit u of a tile row of U units: the rows of a fragment
// (16 of them, one unit) and of a transpose read (4 rows, 4 units) both land
// in distinct banks.
template <int U>
__device__ __forceinline__ int lin_unit(int row, int u) {
  if constexpr (U >= 16) return u ^ (((row & 3) << 2) | ((row >> 2) & 3));
  else if constexpr (U >= 8) return u ^ ((((row >> 1) & 1) << 2) | ((row >> 2) & 3));
  else return u ^ ((row >> 2) & 3);
}

__device__ __forceinline__ f32x4 ld4(const uint16_t* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return f32x4{bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y)};
}
__device__ __forceinline__ f32x4 ld4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }

template <typename E, int D>
struct LinTile {
  static constexpr int kUnits = D * (int)sizeof(E) / 16;
  static constexpr int kBytes = kChunk * D * (int)sizeof(E);
  // eight consecutive columns from c0 of a row, as a fragment
  template <class Eng>
  static __device__ __forceinline__ typename Eng::Fr row8(const char* t, int row, int c0) {
    if constexpr (sizeof(E) == 2) {
      return Eng::ld((const E*)(t + row * D * 2 + 16 * lin_unit<kUnits>(row, c0 / 8)));
    } else {
      return Eng::ld2((const E*)(t + row * D * 4 + 16 * lin_unit<kUnits>(row, c0 / 4)),
                      (const E*)(t + row * D * 4 + 16 * lin_unit<kUnits>(row, c0 / 4 + 1)));
    }
  }
  // four consecutive columns from c0 of a row, as fp32
  static __device__ __forceinline__ f32x4 row4(const char* t, int row, int c0) {
    constexpr int kPer = 16 / (int)sizeof(E);
    return ld4((const E*)(t + row * D * sizeof(E) + 16 * lin_unit<kUnits>(row, c0 / kPer) +
                          (c0 % kPer) * sizeof(E)));
  }
  // column c0 + kStep (ln / 4) + ln % 4 of the rows kperm of k-block kb: a
  // transposed fragment of 16 columns, in order (kStep 4) or as dkmap
  // relabels them (kStep 8)
  template <class Eng, int kStep>
  static __device__ __forceinline__ typename Eng::Fr cols8(const char* t, int kb, int c0, int ln, int gq) {
    if constexpr (sizeof(E) == 2) {
      const int r0 = 32 * kb + 4 * gq + (ln >> 2), r1 = r0 + 16, c = c0 + kStep * (ln & 3);
      const uint2 a = lds_read_tr16(t + r0 * D * 2 + 16 * lin_unit<kUnits>(r0, c / 8) + (c & 4) * 2);
      const uint2 b = lds_read_tr16(t + r1 * D * 2 + 16 * lin_unit<kUnits>(r1, c / 8) + (c & 4) * 2);
      return __builtin_bit_cast(typename Eng::Fr, make_uint4(a.x, a.y, b.x, b.y));
    } else {
      typename Eng::Fr f;
      const int c = c0 + kStep * (ln >> 2) + (ln & 3);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = 32 * kb + 4 * gq + (j & 3) + 16 * (j >> 2);
        f.v[j] = *(const float*)(t + r * D * 4 + 16 * lin_unit<kUnits>(r, c / 4) + (c & 3) * 4);
      }
      return f;
    }
  }
};

// Rows of a chunk into a tile; NT threads (whole waves drop out of the last
// step where the units do not divide).
template <typename E, int D, int NT>
struct LinRows {
  static constexpr int kUnits = D * (int)sizeof(E) / 16;
  static constexpr int kAll = kChunk * kUnits;
  static constexpr int kPer = (kAll + NT - 1) / NT;
  static_assert(kAll % 64 == 0, "whole waves");
  // Asked for and on the way (wait_vmem, then a barrier): rows from n on are
  // copies of the last valid one, which no result takes in.
  static __device__ __forceinline__ void ask(uint32_t lds, const E* p, int stride, int n) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) ask_step(i, lds, p, stride, n);
  }
  static __device__ __forceinline__ void ask_step(int i, uint32_t lds, const E* p, int stride, int n) {
    if (kAll % NT != 0 && uniform((int)threadIdx.x + NT * i) >= kAll) return;
    lds_load16(p, offset(i, stride, n), lds + 16 * 64 * (threadIdx.x >> 6) + 16 * NT * i);
  }
  static __device__ __forceinline__ uint32_t offset(int i, int stride, int n) {   // bytes
    const int idx = (int)threadIdx.x + NT * i, row = idx / kUnits, u = lin_unit<kUnits>(row, idx % kUnits);
    const int r = row < n ? row : n - 1;
    return (uint32_t)(r * stride + u * (16 / (int)sizeof(E))) * (uint32_t)sizeof(E);
  }
  // Through registers, in two halves; rows from n on are 0.
  static __device__ __forceinline__ void fetch(uint4 (&x)[kPer], const E* p, int stride, int n) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int idx = (int)threadIdx.x + NT * i, row = idx / kUnits, u = idx % kUnits;
      x[i] = row < n ? *reinterpret_cast<const uint4*>(p + (uint32_t)(row * stride + u * (16 / (int)sizeof(E))))
                     : make_uint4(0, 0, 0, 0);
    }
  }
  static __device__ __forceinline__ void put(char* t, const uint4 (&x)[kPer]) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int idx = (int)threadIdx.x + NT * i, row = idx / kUnits, u = idx % kUnits;
      if (kAll % NT != 0 && idx >= kAll) break;
      *reinterpret_cast<uint4*>(t + row * D * sizeof(E) + 16 * lin_unit<kUnits>(row, u)) = x[i];
    }
  }
};

// A sum of log decays in base 2 as its nearest whole number and the rest, and
// 2^(n + f): decays are off by a few 2^-24 however strong they are.  (e^x as
// 2^x of a rounded x log2(e), or by expf compiled with contraction, is off by
// |x| 2^-24.)
struct LinLog {
  int n;
  float f;
};
__device__ __forceinline__ LinLog lin_log(double x) {
  const double n = x > -1e9 ? (x < 1e9 ? __builtin_rint(x) : 1e9) : -1e9;   // a NaN stays in the rest
  return {(int)n, (float)(x - n)};
}
__device__ __forceinline__ float lin_pow(int n, float f) { return ldexpf(__builtin_amdgcn_exp2f(f), n); }
__device__ __forceinline__ float lin_pow(double x) {
  const LinLog s = lin_log(x);
  return lin_pow(s.n, s.f);
}

struct LinGates {
  int n[kChunk];                 // G_i log2(e) = n + f
  float f[kChunk];
  float in[kChunk];              // weight of X^T Q_a
  float out[kChunk];             // weight of K_b V_b^T in the state
};
// of the reverse passes: in[63] is not e^(G_C) there
struct LinGatesRev : LinGates {
  float decay;                   // e^(G_C)
  float pad[3];
};
template <bool kRev>
using LinGatesOf = std::conditional_t<kRev, LinGatesRev, LinGates>;
__device__ __forceinline__ float lin_decay(const LinGates& g) { return g.in[kChunk - 1]; }
__device__ __forceinline__ float lin_decay(const LinGatesRev& g) { return g.decay; }

// One wave: the chunk's gate vectors; rows from n on have no weight in the
// state.  The sums run in fp64 (far tokens of a strongly decaying chunk differ
// by large G) and base 2; a log decay below -1e4 has the weight 0 and is held
// there, so that -inf leaves no NaN.  later: log decays between the chunk and
// the end that its state weights refer to.  Returns the chunk's sum.
template <bool kRev>
__device__ __forceinline__ double lin_gates(LinGatesOf<kRev>& s, float g, int n, double later = 0.0) {
  const int ln = threadIdx.x & 63;
  const double G = wave_prefix_f64((double)(g < -1e4f ? -1e4f : g) * 1.4426950408889634);
  const double C = last_lane(G);
  const LinLog own = lin_log(G);
  s.n[ln] = own.n;
  s.f[ln] = own.f;
  const float a = lin_pow(own.n, own.f), b = lin_pow(C - G + later);
  s.in[ln] = kRev ? b : a;
  s.out[ln] = ln < n ? (kRev ? a : b) : 0.0f;
  if constexpr (kRev) {
    if (ln == kChunk - 1) s.decay = a;
  }
  return C;
}


// The six 16 x 32 blocks of P (row tile rt, k-block kb) inside the triangle.
template <bool kRev>
__host__ __device__ constexpr bool lin_has(int rt, int kb) { return kRev ? 2 * kb + 1 >= rt : 2 * kb <= rt; }
template <bool kRev>
__host__ __device__ constexpr int lin_block(int rt, int kb) {
  return kRev ? (rt < 2 ? 2 * rt + kb : 2 + rt) : (rt < 2 ? rt : 2 * rt - 2 + kb);
}
template <bool kRev>
__device__ __forceinline__ void lin_block_at(int blk, int& rt, int& kb) {   // its inverse
  rt = kRev ? (blk < 4 ? blk >> 1 : blk - 2) : (blk < 2 ? blk : 1 + (blk >> 1));
  kb = kRev ? (blk < 4 ? blk & 1 : 1) : (blk < 2 ? 0 : blk & 1);
}

// wait_vmem for the rows asked for, but not for the kStores stores that every
// wave issued after them (four of a whole chunk's outputs, and DQ's of the
// state): vector memory operations of a wave retire in order, so at most
// kStores outstanding ones are those stores.
template <int kStores>
__device__ __forceinline__ void wait_rows() {
  static_assert(kStores == 4 || kStores == 8 || kStores == 12, "the builtin's operand below holds up to 15");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kStores) : "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70 + kStores);
}

// One workgroup's place in the batch, the same for all its waves.
struct LinPlace {
  LinSeg sg;
  int slot, vh, nch;
  int64_t sv, dump0;
  const float* pg;
  // false: nothing to do (unused slot, bad index arrays)
  __device__ __forceinline__ bool find(const LinScan& A) {
    slot = blockIdx.x / A.VH;
    vh = blockIdx.x % A.VH;
    sg = lin_find(A.cu, A.N, A.T, A.seglen, slot, false);
    if (A.status != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *A.status = sg.bad ? kStatusBadIndex : 0;
    if (sg.bad) return false;
    sv = (int64_t)slot * A.VH + vh;
    if (sg.n < 0) return false;
    // stored states: one after each chunk but a segment's last, from t0 / kChunk on, so that no two
    // segments share one and all lie below T / kChunk
    dump0 = (int64_t)sg.t0 / kChunk * A.VH + vh;
    nch = (sg.len + kChunk - 1) / kChunk;
    pg = A.g + sg.t0 * A.g_row + vh / A.tiles;
    return true;
  }
  template <bool kRev>
  __device__ __forceinline__ int chunk(int it) const { return kRev ? nch - 1 - it : it; }
  __device__ __forceinline__ int rows(int c) const {
    const int n = sg.len - kChunk * c;
    return n < kChunk ? n : kChunk;
  }
  // this lane's log decay of walk step it
  template <bool kRev>
  __device__ __forceinline__ float gate(int it, int64_t g_row) const {
    const int c = chunk<kRev>(it), l = threadIdx.x & 63;
    return it < nch && l < rows(c) ? pg[((int64_t)kChunk * c + l) * g_row] : 0.0f;
  }
};

// The walk of one role (mode) by its CV / 16 waves: X and the pieces of a
// chunk's work.  w: the wave's index in the role.
template <class Eng, int CK, int CV, int MODE>
struct LinWalk {
  using E = typename Eng::E;
  using Fr = typename Eng::Fr;
  using TK = LinTile<E, CK>;
  using TV = LinTile<E, CV>;
  static constexpr bool kOut = MODE != kLinStF && MODE != kLinStR;
  static constexpr bool kDots = MODE == kLinDQ || MODE == kLinDK;
  static constexpr bool kRev = MODE == kLinStR || MODE == kLinDV || MODE == kLinDK;
  // The forward state pass also walks from the last chunk to the first: its
  // weights hold the decays up to the segment's end, X needs none of its own,
  // and the chunks it read last are those that the output pass reads first.
  static constexpr bool kBack = kRev || MODE == kLinStF;
  using Gates = LinGatesOf<kRev>;
  static constexpr bool kXT = !kDots;      // X rows are key channels (else value rows)
  static constexpr int kXPlanes = Eng::kSplit ? (kDots ? 3 : 2) : 1;   // three where X's product enters dg
  static constexpr int kVPlanes = Eng::kSplit ? 3 : 1;
  static constexpr int NW = CV / 16, NT = 64 * NW;
  static constexpr int RT = CK / 16;       // row tiles of X
  static constexpr int kFrag = 64 * (sizeof(E) == 2 ? 16 : 32);
  static constexpr int kPBytes = 6 * Eng::kPlanes * kFrag;
  // the wave with the fewest pair blocks: it forms the next gates, and dg
  static constexpr int kLight = NW - 1;

  const LinScan& A;
  const LinPlace& L;
  const int w, l64, ln, gq;
  // X: tile tr holds rows dkmap(16 tr + 4 gq + r), column 16 w + ln; O: row
  // tile rt the row 16 rt + ln, columns 16 w + 4 gq + r
  f32x4 X[RT], O[4];
  Fr vf[2];                                // V^T fragments of this wave's columns
  float rdot, gate;                        // DK, light wave: this lane's r_i and log decay
  double dg_sum;

  __device__ __forceinline__ LinWalk(const LinScan& a, const LinPlace& l, int wave)
      : A(a), L(l), w(wave), l64(threadIdx.x & 63), ln(threadIdx.x & 15), gq((threadIdx.x >> 4) & 3), rdot(0.0f),
        gate(0.0f), dg_sum(0.0) {}

  __device__ __forceinline__ int64_t st_at(int tr, int r) const {
    const int row = 32 * (tr / 2) + 8 * gq + 4 * (tr & 1) + r, colx = 16 * w + ln;
    return kXT ? (int64_t)colx * CK + row : (int64_t)row * CV + colx;
  }
  __device__ __forceinline__ void load_state() {
    const int64_t size = (int64_t)A.tw * A.dk;
    const float* p = nullptr;
    if (kOut) {
      if (A.seg != nullptr) p = A.seg + L.sv * size;
      else if (A.first != nullptr) p = A.first + ((int64_t)L.sg.n * A.VH + L.vh) * size;
    }
#pragma unroll
    for (int tr = 0; tr < RT; ++tr) {
      f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
      if (p != nullptr) {
        if constexpr (kXT) x = *reinterpret_cast<const f32x4*>(p + st_at(tr, 0));
        else {
#pragma unroll
          for (int r = 0; r < 4; ++r) x[r] = p[st_at(tr, r)];
        }
      }
      X[tr] = x;
    }
  }
  // the state after the walk: a segment's sum, or the sequence's last state
  __device__ __forceinline__ void store_state() const {
    const int64_t size = (int64_t)A.tw * A.dk;
    float* p = nullptr;
    if (!kOut) p = A.seg + L.sv * size;
    else if (A.last != nullptr && L.sg.s == (kRev ? 0 : L.sg.nseg - 1))
      p = A.last + ((int64_t)L.sg.n * A.VH + L.vh) * size;
    if (p == nullptr) return;
#pragma unroll
    for (int tr = 0; tr < RT; ++tr) {
      if constexpr (kXT) *reinterpret_cast<f32x4*>(p + st_at(tr, 0)) = X[tr];
      else {
#pragma unroll
        for (int r = 0; r < 4; ++r) p[st_at(tr, r)] = X[tr][r];
      }
    }
  }
  // DQ: the state after chunk c, which is not the segment's last, for DK.  Past
  // the caches both ways, which the rows fill (415 us for 424 at 128 x 192).
  __device__ __forceinline__ f32x4* dumped(int c) const {
    return reinterpret_cast<f32x4*>(A.dump) + (L.dump0 + c * (int64_t)A.VH) * (CK * CV / 4) + 64 * w + l64;
  }
  __device__ __forceinline__ void store_dump(int c) const {
    f32x4* d = dumped(c);
#pragma unroll
    for (int tr = 0; tr < RT; ++tr) __builtin_nontemporal_store(X[tr], d + tr * NT);
  }
  // A value for each token and head: a chunk's first, and this lane's from there
  // (formed where it is used, not kept through the walk).
  __device__ __forceinline__ int64_t row0(int c) const { return ((int64_t)L.sg.t0 + kChunk * c) * A.VH + L.vh; }
  __device__ __forceinline__ uint32_t lane_row() const {
    uint32_t i = (uint32_t)(l64 * A.VH);
    asm volatile("" : "+v"(i));
    return i;
  }
  // DK: this wave's part of <S, dS>, S the state entering the chunk: from the
  // dq pass, or what that pass started the segment from; and the light wave's
  // r_i and log decays
  __device__ __forceinline__ void begin_dg(int c, int n, double* sY) {
    if (w == kLight) {
      rdot = l64 < n ? (A.rdot + row0(c))[lane_row()] : 0.0f;
      gate = l64 < n ? L.pg[((int64_t)kChunk * c + l64) * A.g_row] : 0.0f;
    }
    double y = 0.0;
    if (c > 0) {
      const f32x4* d = dumped(c - 1);
      f32x4 s[RT];
#pragma unroll
      for (int tr = 0; tr < RT; ++tr) s[tr] = __builtin_nontemporal_load(d + tr * NT);
      __builtin_amdgcn_sched_barrier(0);     // all on the way before the first is waited for
#pragma unroll
      for (int tr = 0; tr < RT; ++tr)
#pragma unroll
        for (int r = 0; r < 4; ++r) y = fma((double)s[tr][r], (double)X[tr][r], y);
    } else if (A.seg_in != nullptr || A.first_in != nullptr) {
      const int64_t size = (int64_t)A.tw * A.dk;
      const char* p = (const char*)(A.seg_in != nullptr ? A.seg_in + L.sv * size
                                                        : A.first_in + ((int64_t)L.sg.n * A.VH + L.vh) * size);
      uint32_t at = (uint32_t)st_at(0, 0) * 4;
      asm volatile("" : "+v"(at));           // one register, not one for each row
#pragma unroll
      for (int t0 = 0; t0 < RT; t0 += 4) {
        f32x4 s[4];
#pragma unroll
        for (int tr = 0; tr < 4; ++tr)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            s[tr][r] = *(const float*)(p + (32 * ((t0 + tr) / 2) + 4 * (tr & 1) + r) * CV * 4 + at);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int tr = 0; tr < 4; ++tr)
#pragma unroll
          for (int r = 0; r < 4; ++r) y = fma((double)s[tr][r], (double)X[t0 + tr][r], y);
      }
    }
    y = last_lane(wave_prefix_f64(y));
    if (l64 == 0) sY[w] = y;
  }

  // Pair products of the 16 x 32 blocks first, first + step, .., weighted, into
  // sP.  sE: DK's tile of k; sM: its sums of M over the rows of a tile (16 at
  // 64 a + 16 b) and over the columns of a block (16 at 256 + 64 kb + 16 a).
  static __device__ __forceinline__ void pairs(int first, int step, const char* sQ, const char* sK, const char* sV,
                                               const char* sE, const Gates& g, int n, char* sP, float* sM) {
    const int l64 = threadIdx.x & 63, ln = l64 & 15, gq = l64 >> 4;
#pragma unroll 1
    for (int blk = first; blk < 6; blk += step) {
      int a, kb;
      lin_block_at<kRev>(blk, a, kb);
      const int an = g.n[16 * a + ln];
      const float af = g.f[16 * a + ln];
      // both tiles of the block, also where the triangle leaves one out (2 of 6)
      f32x4 acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
      f32x4 acc2[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
      float cm = 0.0f;                     // DK: column sums of M
#pragma unroll
      for (int p = 0; p < CK / 32; ++p) {
        const Fr qf = TK::template row8<Eng>(sQ, 16 * a + ln, 32 * p + 8 * gq);
#pragma unroll
        for (int bb = 0; bb < 2; ++bb)
          Eng::mma(acc[bb], TK::template row8<Eng>(sK, 32 * kb + 16 * bb + ln, 32 * p + 8 * gq), qf);
      }
      if constexpr (MODE == kLinDK) {
#pragma unroll
        for (int p = 0; p < CV / 32; ++p) {
          const Fr ef = TV::template row8<Eng>(sE, 16 * a + ln, 32 * p + 8 * gq);
#pragma unroll
          for (int bb = 0; bb < 2; ++bb)
            Eng::mma(acc2[bb], TV::template row8<Eng>(sV, 32 * kb + 16 * bb + ln, 32 * p + 8 * gq), ef);
        }
      }
      float pw[8];
#pragma unroll
      for (int bb = 0; bb < 2; ++bb) {
        const int b = 2 * kb + bb;
        const int4 b4 = *reinterpret_cast<const int4*>(&g.n[16 * b + 4 * gq]);
        const int bn[4] = {b4.x, b4.y, b4.z, b4.w};
        const f32x4 bf = *reinterpret_cast<const f32x4*>(&g.f[16 * b + 4 * gq]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int ia = 16 * a + ln, ib = 16 * b + 4 * gq + r;
          const float d = kRev ? lin_pow(bn[r] - an, bf[r] - af) : lin_pow(an - bn[r], af - bf[r]);
          pw[4 * bb + r] = (kRev ? ib >= ia && ib < n : ib <= ia) ? acc[bb][r] * d : 0.0f;
          if constexpr (MODE == kLinDK) {
            const float m = ib > ia ? acc2[bb][r] * pw[4 * bb + r] : 0.0f;
            cm += m;
            const float rm = group_sum<16>(m);
            if (ln == 0) sM[64 * a + 16 * b + 4 * gq + r] = rm;
          }
        }
      }
      Fr pl[2];
      Eng::split(pw, pl[0], pl[1]);
      char* dst = sP + blk * Eng::kPlanes * kFrag + l64 * (kFrag / 64);
#pragma unroll
      for (int k = 0; k < Eng::kPlanes; ++k) Eng::st((E*)(dst + k * kFrag), pl[k]);
      if constexpr (MODE == kLinDK) {
        cm += __shfl_xor(cm, 16, 64);
        cm += __shfl_xor(cm, 32, 64);
        if (gq == 0) sM[256 + 64 * kb + 16 * a + ln] = cm;
      }
    }
  }

  __device__ __forceinline__ void take_v(const char* sV) {
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) vf[kb] = TV::template cols8<Eng, 4>(sV, kb, 16 * w, ln, gq);
  }

  // O: a weight of 0 times an infinity or a NaN of V would reach the tokens
  // before it.  Such values are taken out of the fragments; bad_from is the
  // first token of this lane's column with one (kChunk: none).  True where
  // the wave has any (rare: O and X are then put right by taint).
  __device__ __forceinline__ bool clear_v(int& bad_from) {
    constexpr int kWords = sizeof(Fr) / 4;
    struct Words {
      uint32_t u[kWords];
    };
    bool any;
    if constexpr (Eng::kSplit) {           // 0 times the columns on the matrix unit: NaN where one holds any
      f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
      const Fr zero = __builtin_bit_cast(Fr, make_uint4(0, 0, 0, 0));
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) Eng::mma(z, vf[kb], zero);
      any = !((z[0] + z[1]) + (z[2] + z[3]) == 0.0f);
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const Words x = __builtin_bit_cast(Words, vf[kb]);
#pragma unroll
        for (int j = 0; j < kWords; ++j) m = max(m, x.u[j] & 0x7fffffffu);
      }
      any = m >= 0x7f800000u;
    }
    if (__ballot(any) == 0) return false;
    int first = kChunk;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      Words x = __builtin_bit_cast(Words, vf[kb]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t& u = x.u[j * kWords / 8];
        const uint32_t inf = !Eng::kSplit ? 0x7f800000u : (j & 1) ? 0x7f800000u : 0x7f80u;
        const uint32_t all = !Eng::kSplit ? 0xffffffffu : (j & 1) ? 0xffff0000u : 0xffffu;
        if ((u & inf) != inf) continue;
        u &= ~all;
        first = min(first, 32 * kb + 4 * gq + (j & 3) + 16 * (j >> 2));
      }
      vf[kb] = __builtin_bit_cast(Fr, x);
    }
    first = min(first, __shfl_xor(first, 16, 64));
    bad_from = min(first, __shfl_xor(first, 32, 64));
    return true;
  }
  __device__ __forceinline__ void taint_out(int bad_from) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int from = __shfl(bad_from, 4 * gq + r, 64);
#pragma unroll
      for (int rt = 0; rt < 4; ++rt)
        if (16 * rt + ln >= from) O[rt][r] = __builtin_nanf("");
    }
  }
  __device__ __forceinline__ void taint_state(int bad_from) {
#pragma unroll
    for (int tr = 0; tr < RT; ++tr)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (bad_from < kChunk) X[tr][r] = __builtin_nanf("");
  }

  // State part: O^T = X^T Q^T, scaled by the rows' weights.
  __device__ __forceinline__ void state_part(const char* sQ, const Gates& g) {
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) O[rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 0; p < CK / 32; ++p) {
      Fr xf[3], qf[4];
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) qf[rt] = TK::template row8<Eng>(sQ, 16 * rt + ln, 32 * p + 8 * gq);
      const float x8[8] = {X[2 * p][0], X[2 * p][1], X[2 * p][2], X[2 * p][3],
                           X[2 * p + 1][0], X[2 * p + 1][1], X[2 * p + 1][2], X[2 * p + 1][3]};
      if constexpr (kXPlanes == 3) Eng::split3(x8, xf[0], xf[1], xf[2]);
      else Eng::split(x8, xf[0], xf[1]);
#pragma unroll
      for (int k = 0; k < kXPlanes; ++k)
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) Eng::mma(O[rt], xf[k], qf[rt]);
    }
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      const float s = g.in[16 * rt + ln];
#pragma unroll
      for (int r = 0; r < 4; ++r) O[rt][r] *= s;
    }
  }
  // DQ, DK: the wave's columns of r_i, c_j; e(rt): this lane's four columns of
  // E in row tile rt.
  template <class F>
  __device__ __forceinline__ void dots(int n, float* sR, F e) const {
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      const int row = 16 * rt + ln;
      const f32x4 ev = e(rt);
      float d = 0.0f;
#pragma unroll
      for (int r = 0; r < 4; ++r) d = fmaf(O[rt][r], ev[r], d);
      d += __shfl_xor(d, 16, 64);
      d += __shfl_xor(d, 32, 64);
      if (gq == 0) sR[kChunk * w + row] = row < n ? d : 0.0f;
    }
  }

  // Pair part: O^T += V^T P^T.
  __device__ __forceinline__ void pair_part(const char* sP) {
#pragma unroll
    for (int k = 0; k < Eng::kPlanes; ++k)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
          if (!lin_has<kRev>(rt, kb)) continue;
          const Fr pf = Eng::ld((const E*)(sP + (lin_block<kRev>(rt, kb) * Eng::kPlanes + k) * kFrag +
                                           l64 * (kFrag / 64)));
          Eng::mma(O[rt], vf[kb], pf);
        }
  }
  __device__ __forceinline__ void store_out(int c, int n) const {
    const bool wide = sizeof(E) == 4 || (kDots && A.out_f32);
    const int size = wide ? 4 : 2;
    // a chunk's rows lie within 2^31 bytes of its first: 32-bit offsets from there
    char* base = (char*)A.out + (((int64_t)L.sg.t0 + kChunk * c) * A.os + (int64_t)L.vh * CV) * size;
    uint32_t off = (uint32_t)((ln * A.os + 16 * w + 4 * gq) * size);
    asm volatile("" : "+v"(off));            // one register, not eight kept through the walk
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      if (16 * rt + ln >= n) continue;
      char* to = base + (int64_t)(16 * rt * A.os * size);
      if (wide)
        *reinterpret_cast<f32x4*>(to + off) = O[rt];
      else
        *reinterpret_cast<uint2*>(to + off) =
            make_uint2(pack_bf16x2(O[rt][0], O[rt][1]), pack_bf16x2(O[rt][2], O[rt][3]));
    }
  }
  // DQ's light wave: r_i; DK's: dg of the chunk's tokens.
  __device__ __forceinline__ void end_dots(int c, int n, const Gates& g, const float* sR, const float* sM,
                                           const double* sY) {
    float d = 0.0f;
#pragma unroll
    for (int k = 0; k < NW; ++k) d += sR[kChunk * k + l64];
    if constexpr (MODE == kLinDQ) {
      if (l64 < n) (A.rdot + row0(c))[lane_row()] = d;
    } else if constexpr (MODE == kLinDK) {
      double Xc = sY[0];
#pragma unroll
      for (int k = 1; k < NW; ++k) Xc += sY[k];
      Xc *= (double)lin_decay(g);
      // row sum of M, over the column blocks, and column sum, over the row
      // blocks; what no block writes is 0
      double rm = 0.0;
#pragma unroll
      for (int a = 0; a < 4; ++a) rm += (double)sM[64 * a + l64];
      const double cm = (double)sM[256 + l64] + (double)sM[320 + l64];
      const double own = rm + (double)rdot - cm;
      const double head = wave_prefix_f64(own);
      double pre = __shfl_up(wave_prefix_f64((double)d), 1, 64);   // without the token's own c
      if (l64 == 0) pre = 0.0;
      double dg = (last_lane(head) - head + own) + pre + Xc;
      // a decay of 0 (-inf, a reset) leaves no product across its token: 0, not what the sums' rounding leaves
      if (gate < -104.0f) dg *= 0.0;         // e^-104 rounds to 0
      if (l64 < n) {
        if (A.dg_tok != nullptr) (A.dg_tok + row0(c))[lane_row()] = (float)dg;
        dg_sum += dg;
      }
    }
  }

  // X <- e^(G_C) X + sum_b out_b K_b V_b^T
  __device__ __forceinline__ void update(const char* sK, const Gates& g) {
    if constexpr (MODE != kLinStF) {
      const float dec = lin_decay(g);
#pragma unroll
      for (int tr = 0; tr < RT; ++tr)
#pragma unroll
        for (int r = 0; r < 4; ++r) X[tr][r] *= dec;
    }
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const f32x4 w0 = *reinterpret_cast<const f32x4*>(&g.out[32 * kb + 4 * gq]);
      const f32x4 w1 = *reinterpret_cast<const f32x4*>(&g.out[32 * kb + 16 + 4 * gq]);
      Fr wv[3];
      float x8[8];
      if constexpr (Eng::kSplit) {
        const uint4 u = __builtin_bit_cast(uint4, vf[kb]);
        x8[0] = bf16_lo(u.x) * w0[0]; x8[1] = bf16_hi(u.x) * w0[1];
        x8[2] = bf16_lo(u.y) * w0[2]; x8[3] = bf16_hi(u.y) * w0[3];
        x8[4] = bf16_lo(u.z) * w1[0]; x8[5] = bf16_hi(u.z) * w1[1];
        x8[6] = bf16_lo(u.w) * w1[2]; x8[7] = bf16_hi(u.w) * w1[3];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x8[j] = vf[kb].v[j] * (j < 4 ? w0[j] : w1[j & 3]);
      }
      Eng::split3(x8, wv[0], wv[1], wv[2]);
      constexpr int kStep = Eng::kSplit ? 4 : 2;   // row tiles whose products alternate
#pragma unroll
      for (int tr0 = 0; tr0 < RT; tr0 += kStep) {
        Fr kf[kStep];
#pragma unroll
        for (int i = 0; i < kStep; ++i)
          kf[i] = TK::template cols8<Eng, 8>(sK, kb, 32 * ((tr0 + i) / 2) + 4 * (i & 1), ln, gq);
#pragma unroll
        for (int k = 0; k < kVPlanes; ++k)
#pragma unroll
          for (int i = 0; i < kStep; ++i) Eng::mma(X[tr0 + i], kf[i], wv[k]);
      }
    }
  }
};

// Forward passes and state passes: one role, CV / 16 waves.
template <class Eng, int CK, int CV, int MODE>
struct LinLds {
  using E = typename Eng::E;
  using W = LinWalk<Eng, CK, CV, MODE>;
  static constexpr bool kDirect = sizeof(E) == 2;
  static constexpr int kVTiles = kDirect && !W::kOut ? 2 : 1;
  static constexpr int K = 0;
  static constexpr int V = K + (kDirect ? 2 : 1) * W::TK::kBytes;
  static constexpr int Q = V + kVTiles * W::TV::kBytes;
  static constexpr int P = Q + (W::kOut ? W::TK::kBytes : 0);
  static constexpr int G = P + (W::kOut ? W::kPBytes : 0);
  static constexpr int R = G + 2 * (int)sizeof(typename W::Gates);
  static constexpr int kBytes = R + (W::kDots ? W::NW * kChunk * 4 : 0);
};

template <class Eng, int CK, int CV, int MODE>
__device__ __forceinline__ void lin_scan_walk(const LinScan& A) {
  using E = typename Eng::E;
  using Lds = LinLds<Eng, CK, CV, MODE>;
  using W = LinWalk<Eng, CK, CV, MODE>;
  using RowsK = LinRows<E, CK, W::NT>;
  using RowsV = LinRows<E, CV, W::NT>;
  constexpr bool kOut = W::kOut, kDots = W::kDots, kDirect = Lds::kDirect, kRev = W::kRev, kBack = W::kBack;

  extern __shared__ char smem[];
  auto* sG = reinterpret_cast<typename W::Gates*>(smem + Lds::G);
  float* sR = reinterpret_cast<float*>(smem + Lds::R);
  const uint32_t lds0 = lds_base_u32(smem);

  LinPlace L;
  if (!L.find(A)) return;
  // the state pass leaves out the segment whose sum nothing reads
  if (MODE == kLinStF && L.sg.s == L.sg.nseg - 1) return;
  if (MODE == kLinStR && L.sg.s == 0) return;
  const int w = uniform(threadIdx.x >> 6);
  W S(A, L, w);

  const int64_t t0 = L.sg.t0;
  const E* pK = (const E*)A.K + t0 * A.ks + (int64_t)(L.vh / A.kd) * CK;
  const E* pV = (const E*)A.V + t0 * A.vs + (int64_t)(L.vh / A.vd) * CV;
  const E* pQ = kOut ? (const E*)A.Q + t0 * A.qs + (int64_t)(L.vh / A.qd) * CK : nullptr;
  const E* pE = kDots ? (const E*)A.E + t0 * A.es + (int64_t)(L.vh / A.ed) * CV : nullptr;
  // the rows of walk step it: K into its tile, V and Q into theirs.  K's other
  // tile is free a whole chunk ahead, and O asks for it once the gates are
  // formed (DQ waits for its rows of E after that)
  constexpr bool kEarly = MODE == kLinO;
  auto ask_k = [&](int it) {
    const int c = L.chunk<kBack>(it), n = L.rows(c);
    RowsK::ask(lds0 + Lds::K + (it & 1) * W::TK::kBytes, pK + (int64_t)kChunk * c * A.ks, A.ks, n);
  };
  auto ask = [&](int it) {
    const int c = L.chunk<kBack>(it), n = L.rows(c);
    const int64_t r0 = (int64_t)kChunk * c;
    RowsV::ask(lds0 + Lds::V + (kOut ? 0 : (it & 1) * W::TV::kBytes), pV + r0 * A.vs, A.vs, n);
    if constexpr (kOut) RowsK::ask(lds0 + Lds::Q, pQ + r0 * A.qs, A.qs, n);
  };

  const int nch = L.nch;
  float rg = 0.0f;                         // light wave: the next step's log decays
  double Gsum = 0.0;                       // and the segment's sum
  if (w == W::kLight && nch > 0) {
    Gsum += lin_gates<kRev>(sG[0], L.gate<kBack>(0, A.g_row), L.rows(L.chunk<kBack>(0)));
    rg = L.gate<kBack>(1, A.g_row);
  }
  // fp32 rows, which do not fit twice, wait for their tiles in registers
  uint4 xk[RowsK::kPer], xv[RowsV::kPer], xq[RowsK::kPer];
  auto fetch = [&](int it) {
    const int c = L.chunk<kBack>(it), n = L.rows(c);
    const int64_t r0 = (int64_t)kChunk * c;
    RowsK::fetch(xk, pK + r0 * A.ks, A.ks, n);
    RowsV::fetch(xv, pV + r0 * A.vs, A.vs, n);
    if constexpr (kOut) RowsK::fetch(xq, pQ + r0 * A.qs, A.qs, n);
  };
  if (nch > 0) {
    if constexpr (kDirect) {
      ask_k(0);
      ask(0);
    } else {
      fetch(0);
    }
  }
  S.load_state();
  if (kDirect) wait_vmem();                // the state is there: no wait for it inside the walk

#pragma unroll 1
  for (int it = 0; it < nch; ++it) {
    const int c = L.chunk<kBack>(it), n = L.rows(c);
    const int64_t r0 = (int64_t)kChunk * c;
    const auto& g = sG[it & 1];
    const char* sK = smem + Lds::K + (kDirect ? (it & 1) * W::TK::kBytes : 0);
    const char* sV = smem + Lds::V + (kDirect && !kOut ? (it & 1) * W::TV::kBytes : 0);
    if constexpr (kDirect) {
      // output passes: the chunk before this one was whole, its stores may go on
      if (kOut && it > 0) wait_rows<MODE == kLinDQ ? 4 + W::RT : 4>();
      else wait_vmem();
      barrier_lds();
      if (!kOut && it + 1 < nch) {
        ask_k(it + 1);
        ask(it + 1);
      }
    } else {
      RowsK::put(smem + Lds::K, xk);
      RowsV::put(smem + Lds::V, xv);
      if constexpr (kOut) RowsK::put(smem + Lds::Q, xq);
      barrier_lds();
      if (it + 1 < nch) fetch(it + 1);
    }
    // DQ: this lane's columns of E, on the way while the pairs are formed
    using E4 = std::conditional_t<sizeof(E) == 2, uint2, f32x4>;
    E4 er[kDots ? 4 : 1];
    if constexpr (kDots) {
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) {
        const int row = 16 * rt + S.ln;
        er[rt] = *reinterpret_cast<const E4*>(pE + (r0 + (row < n ? row : n - 1)) * A.es + 16 * w + 4 * S.gq);
      }
    }
    if constexpr (kOut) W::pairs(w, W::NW, smem + Lds::Q, sK, sV, nullptr, g, n, smem + Lds::P, nullptr);
    if (w == W::kLight && it + 1 < nch) {
      Gsum += lin_gates<kRev>(sG[(it + 1) & 1], rg, L.rows(L.chunk<kBack>(it + 1)), MODE == kLinStF ? Gsum : 0.0);
      rg = L.gate<kBack>(it + 2, A.g_row);
    }
    if (kDirect && kEarly && it + 1 < nch) ask_k(it + 1);
    S.take_v(sV);
    int bad_from = kChunk;
    bool bad = false;
    if constexpr (kOut) {
      S.state_part(smem + Lds::Q, g);
      if constexpr (kDots)
        S.dots(n, sR, [&](int rt) { return ld4((const E*)&er[rt]); });
      barrier_lds();
      if (kDirect && it + 1 < nch) {
        if constexpr (!kEarly) ask_k(it + 1);
        ask(it + 1);
      }
      if constexpr (MODE == kLinO) bad = S.clear_v(bad_from);
      S.pair_part(smem + Lds::P);
      if (bad) S.taint_out(bad_from);
      S.store_out(c, n);
      if (kDots && w == W::kLight) S.end_dots(c, n, g, sR, nullptr, nullptr);
    }
    S.update(sK, g);
    if (bad) S.taint_state(bad_from);
    if constexpr (MODE == kLinDQ) {
      if (it + 1 < nch) S.store_dump(c);
    }
    if constexpr (!kDirect) barrier_lds();
  }
  S.store_state();
  if (!kOut && w == W::kLight && S.l64 == 0) A.seg_decay[L.sv] = lin_pow(Gsum);
}

template <class Eng, int CK, int CV, int MODE>
__global__ __launch_bounds__(4 * CV, Eng::kSplit ? CV / 32 : CV / 64) void lin_scan_kernel(LinScan A) {
  lin_scan_walk<Eng, CK, CV, MODE>(A);
}

// Both state passes of the backward at once: the forward states' sums A and
// those of the states' gradients B (blockIdx.y).
template <class Eng, int CK, int CV>
__global__ __launch_bounds__(4 * CV, Eng::kSplit ? CV / 32 : CV / 64) void lin_sums_kernel(LinScan A, LinScan B) {
  if (blockIdx.y == 0) lin_scan_walk<Eng, CK, CV, kLinStF>(A);
  else lin_scan_walk<Eng, CK, CV, kLinStR>(B);
}

// The reverse passes of the backward, dk (with dg) and dv, as two roles of
// one workgroup: the first DK / 16 waves walk X = dS [TW, DK] for dk, the next
// TW / 16 waves X = dS^T [DK, TW] for dv.  They share the chunk's rows of q, k,
// v and d_o in LDS (q and d_o, which both still read after the second
// barrier, have two tiles), so each is read once.  Each role forms the other's
// pair products: dk's are two products and the sums of M, and its waves have
// the longer state part (11 ragged sequences, 8 heads of 64 x 128: 43 us for 47).
template <class Eng, int DK, int TW>
struct LinRevLds {
  using E = typename Eng::E;
  using WK = LinWalk<Eng, TW, DK, kLinDK>;
  using WV = LinWalk<Eng, DK, TW, kLinDV>;
  static constexpr bool kDirect = sizeof(E) == 2;
  static constexpr int kTiles = kDirect ? 2 : 1;
  static constexpr int TD = LinTile<E, DK>::kBytes, TV = LinTile<E, TW>::kBytes;
  static constexpr int Q = 0;
  static constexpr int O = Q + kTiles * TD;
  static constexpr int K = O + kTiles * TV;
  static constexpr int V = K + TD;
  static constexpr int PK = V + TV;
  static constexpr int PV = PK + WK::kPBytes;
  static constexpr int G = PV + WV::kPBytes;
  static constexpr int R = G + 2 * (int)sizeof(LinGatesRev);
  static constexpr int M = R + WK::NW * kChunk * 4;
  static constexpr int kSums = 384;
  static constexpr int Y = M + kSums * 4;
  static constexpr int kBytes = Y + WK::NW * 8;
};

// A: the dk pass (Q = v, K = d_o, V = q, E = k); B: the dv pass.
template <class Eng, int DK, int TW>
__global__ __launch_bounds__(4 * (DK + TW), (DK + TW) / 64 * (sizeof(typename Eng::E) == 2 && DK + TW == 128 ? 2 : 1))
void lin_rev_kernel(LinScan A, LinScan B) {
  using E = typename Eng::E;
  using Lds = LinRevLds<Eng, DK, TW>;
  using WK = typename Lds::WK;
  using WV = typename Lds::WV;
  constexpr int NT = 4 * (DK + TW);
  constexpr bool kDirect = Lds::kDirect;
  using RowsD = LinRows<E, DK, NT>;
  using RowsT = LinRows<E, TW, NT>;

  extern __shared__ char smem[];
  LinGatesRev* sG = reinterpret_cast<LinGatesRev*>(smem + Lds::G);
  float* sR = reinterpret_cast<float*>(smem + Lds::R);
  float* sM = reinterpret_cast<float*>(smem + Lds::M);
  double* sY = reinterpret_cast<double*>(smem + Lds::Y);
  const uint32_t lds0 = lds_base_u32(smem);

  for (int i = threadIdx.x; i < Lds::kSums; i += NT) sM[i] = 0.0f;
  LinPlace L;
  if (!L.find(A)) {
    // an unused slot's part of dg (a bad index array leaves it unread)
    if (A.dg_part != nullptr && threadIdx.x == 0) A.dg_part[(int64_t)blockIdx.x] = 0.0;
    return;
  }
  const int w = uniform(threadIdx.x >> 6);
  const int64_t t0 = L.sg.t0;
  const E* pQ = (const E*)A.V + t0 * A.vs + (int64_t)(L.vh / A.vd) * DK;
  const E* pK = (const E*)A.E + t0 * A.es + (int64_t)(L.vh / A.ed) * DK;
  const E* pV = (const E*)A.Q + t0 * A.qs + (int64_t)(L.vh / A.qd) * TW;
  const E* pO = (const E*)A.K + t0 * A.ks + (int64_t)(L.vh / A.kd) * TW;
  const int nch = L.nch;
  auto ask = [&](int it) {
    const int c = L.chunk<true>(it), n = L.rows(c);
    const int64_t r0 = (int64_t)kChunk * c;
    RowsD::ask(lds0 + Lds::Q + (it & 1) * Lds::TD, pQ + r0 * A.vs, A.vs, n);
    RowsT::ask(lds0 + Lds::O + (it & 1) * Lds::TV, pO + r0 * A.ks, A.ks, n);
    RowsD::ask(lds0 + Lds::K, pK + r0 * A.es, A.es, n);
    RowsT::ask(lds0 + Lds::V, pV + r0 * A.qs, A.qs, n);
  };
  auto begin = [&](int it) {               // the chunk's tiles and gates are there
    if constexpr (kDirect) {
      // from the third chunk on the one before was whole: its four stores may go on
      if (it > 1) wait_rows<4>();
      else wait_vmem();
      barrier_lds();
    } else {
      const int c = L.chunk<true>(it), n = L.rows(c);
      const int64_t r0 = (int64_t)kChunk * c;
      auto copy = [&](auto rows, char* t, const E* p, int stride) {
        uint4 x[decltype(rows)::kPer];
        rows.fetch(x, p + r0 * stride, stride, n);
        rows.put(t, x);
      };
      copy(RowsD(), smem + Lds::Q, pQ, A.vs);
      copy(RowsT(), smem + Lds::O, pO, A.ks);
      copy(RowsD(), smem + Lds::K, pK, A.es);
      copy(RowsT(), smem + Lds::V, pV, A.qs);
      __syncthreads();
    }
  };
  auto middle = [&](int it) {              // P, the dots and the next gates are there; k and v are free
    barrier_lds();
    if (kDirect && it + 1 < nch) ask(it + 1);
  };

  if (w < WK::NW) {
    if (kDirect && nch > 0) ask(0);
    WK S(A, L, w);
    S.load_state();
    if (kDirect) wait_vmem();
#pragma unroll 1
    for (int it = 0; it < nch; ++it) {
      const int c = L.chunk<true>(it), n = L.rows(c);
      const LinGatesRev& g = sG[it & 1];
      const char* sQ = smem + Lds::Q + (kDirect ? (it & 1) * Lds::TD : 0);
      const char* sO = smem + Lds::O + (kDirect ? (it & 1) * Lds::TV : 0);
      begin(it);
      S.begin_dg(c, n, sY);
      WV::pairs(w, WK::NW, smem + Lds::K, sQ, sO, nullptr, g, n, smem + Lds::PV, nullptr);
      S.take_v(sQ);
      S.state_part(smem + Lds::V, g);
      S.dots(n, sR, [&](int rt) { return WK::TV::row4(smem + Lds::K, 16 * rt + S.ln, 16 * w + 4 * S.gq); });
      asm volatile("" ::"v"(S.rdot), "v"(S.gate));   // their loads end before the next chunk's are asked for
      middle(it);
      S.pair_part(smem + Lds::PK);
      S.store_out(c, n);
      if (w == WK::kLight) S.end_dots(c, n, g, sR, sM, sY);
      S.update(sO, g);
      if constexpr (!kDirect) __syncthreads();
    }
    if (A.dg_part != nullptr && w == WK::kLight) {
      const double s = last_lane(wave_prefix_f64(S.dg_sum));
      if (S.l64 == 0) A.dg_part[L.sv] = s;
    }
  } else {
    const int wv = w - WK::NW;
    float rg = 0.0f;
    if (wv == WV::kLight && nch > 0) {
      lin_gates<true>(sG[0], L.gate<true>(0, A.g_row), L.rows(L.chunk<true>(0)));
      rg = L.gate<true>(1, A.g_row);
    }
    if (kDirect && nch > 0) ask(0);
    WV S(B, L, wv);
    S.load_state();
    if (kDirect) wait_vmem();
#pragma unroll 1
    for (int it = 0; it < nch; ++it) {
      const int c = L.chunk<true>(it), n = L.rows(c);
      const LinGatesRev& g = sG[it & 1];
      const char* sQ = smem + Lds::Q + (kDirect ? (it & 1) * Lds::TD : 0);
      const char* sO = smem + Lds::O + (kDirect ? (it & 1) * Lds::TV : 0);
      begin(it);
      WK::pairs(wv, WV::NW, smem + Lds::V, sO, sQ, smem + Lds::K, g, n, smem + Lds::PK, sM);
      if (wv == WV::kLight && it + 1 < nch) {
        lin_gates<true>(sG[(it + 1) & 1], rg, L.rows(L.chunk<true>(it + 1)));
        rg = L.gate<true>(it + 2, A.g_row);
      }
      S.take_v(sO);
      S.state_part(smem + Lds::K, g);
      middle(it);
      S.pair_part(smem + Lds::PV);
      S.store_out(c, n);
      S.update(sQ, g);
      if constexpr (!kDirect) __syncthreads();
    }
    S.store_state();
  }
}

template <class Eng, int CK, int CV, int MODE>
static hipError_t lin_scan_go(const LinScan& A, int64_t slots, hipStream_t stream) {
  static PerDeviceOnce once;
  constexpr int lds = LinLds<Eng, CK, CV, MODE>::kBytes;
  const auto kern = lin_scan_kernel<Eng, CK, CV, MODE>;
  const hipError_t e = set_dyn_lds_once(once, (const void*)kern, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)(slots * A.VH)), dim3(4 * CV), lds, stream, A);
  return hipGetLastError();
}

template <class Eng, int CK, int CV>
static hipError_t lin_sums_go(const LinScan& A, const LinScan& B, int64_t slots, hipStream_t stream) {
  static PerDeviceOnce once;
  constexpr int lds = LinLds<Eng, CK, CV, kLinStF>::kBytes, ldsR = LinLds<Eng, CK, CV, kLinStR>::kBytes;
  const auto kern = lin_sums_kernel<Eng, CK, CV>;
  const hipError_t e = set_dyn_lds_once(once, (const void*)kern, lds > ldsR ? lds : ldsR);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)(slots * A.VH), 2), dim3(4 * CV), lds > ldsR ? lds : ldsR, stream, A, B);
  return hipGetLastError();
}
template <class Eng>
static hipError_t lin_sums(const LinScan& A, const LinScan& B, int64_t slots, hipStream_t stream) {
  if (A.dk == 64) return A.tw == 64 ? lin_sums_go<Eng, 64, 64>(A, B, slots, stream)
                                    : lin_sums_go<Eng, 64, 128>(A, B, slots, stream);
  return A.tw == 64 ? lin_sums_go<Eng, 128, 64>(A, B, slots, stream)
                    : lin_sums_go<Eng, 128, 128>(A, B, slots, stream);
}

// CK, CV: the key channels and the value rows of a virtual head, in the order
// the mode takes them.
template <class Eng, int MODE>
static hipError_t lin_scan_mode(const LinScan& A, int64_t slots, hipStream_t stream) {
  constexpr bool swap = MODE == kLinDQ;
  const int ck = swap ? A.tw : A.dk, cv = swap ? A.dk : A.tw;
  if (ck == 64) return cv == 64 ? lin_scan_go<Eng, 64, 64, MODE>(A, slots, stream)
                                : lin_scan_go<Eng, 64, 128, MODE>(A, slots, stream);
  return cv == 64 ? lin_scan_go<Eng, 128, 64, MODE>(A, slots, stream)
                  : lin_scan_go<Eng, 128, 128, MODE>(A, slots, stream);
}

// The dk and dv passes in one launch.
template <class Eng, int DK, int TW>
static hipError_t lin_rev_go(const LinScan& A, const LinScan& B, int64_t slots, hipStream_t stream) {
  static PerDeviceOnce once;
  constexpr int lds = LinRevLds<Eng, DK, TW>::kBytes;
  const auto kern = lin_rev_kernel<Eng, DK, TW>;
  const hipError_t e = set_dyn_lds_once(once, (const void*)kern, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)(slots * A.VH)), dim3(4 * (DK + TW)), lds, stream, A, B);
  return hipGetLastError();
}
template <class Eng>
static hipError_t lin_rev(const LinScan& A, const LinScan& B, int64_t slots, hipStream_t stream) {
  if (A.dk == 64) return A.tw == 64 ? lin_rev_go<Eng, 64, 64>(A, B, slots, stream)
                                    : lin_rev_go<Eng, 64, 128>(A, B, slots, stream);
  return A.tw == 64 ? lin_rev_go<Eng, 128, 64>(A, B, slots, stream)
                    : lin_rev_go<Eng, 128, 128>(A, B, slots, stream);
}

}  // namespace gdn
