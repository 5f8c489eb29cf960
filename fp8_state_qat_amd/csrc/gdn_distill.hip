// gdn_distill.hip -- distillation from a teacher's top logits, with cross
// entropy: losses, gradients, or both in one pass over the logits.
//
// Mathematics.  A row of logits z (V of them), the teacher's kept logits t_j at
// ids i_j, h the temperature, q = softmax(z / h):
//   p_j = e^(t_j / h - c)      c: logsumexp of the kept t / h, or the given one
//                              of the teacher's whole row
//   kd  = sum_j p_j (ln p_j - ln q_(i_j)) [+ r (ln r - ln q_r)]
//         with a given c: r = 1 - sum p, q_r = the rest's mass, v not in I
//   ce  = logsumexp(z) - z_target
//   loss = kd_weight kd + ce_weight ce
// and for w = d loss, a = w kd_weight / h, b = w ce_weight
//   dz_v = a (m q_v - p_v) + b (softmax(z)_v - [v = target]),  m = sum p + r
//   with a given c, off I: a (m q_r - r) e^(z_v / h) / sum_(u not in I) e^(z_u / h)
// (m is 1 but where 1 - sum p is negative, where no column is left for the rest,
// and, 0, where nothing is kept.)
// The rest's sum is formed without the kept entries, as the difference of the
// whole sum and theirs would cancel: a bitmap of I in LDS, a byte for each eight
// columns.  All sums relative to their maximum; the few values of a row beyond
// its sums (p, c, r, the loss) in fp64, as 1 - sum p cancels, and from differences
// of logits only: a logsumexp is kept as a logit x and the rest of it, for next to
// logits of 1e16 and more nothing is left of it in one number.  The backward reads
// it as one fp32 number, off by 2^-24 of it and every probability by as much of
// itself times it: rows where that passes 2^-15 are summed again.
//
// Memory bound: a row belongs to one workgroup, thread i of TPB to the octets of
// eight columns i, i + TPB, ..; U octets a thread are asked for at once and
// held in registers, so a row of up to 8 TPB U columns is read once for its
// loss and its gradient.  Octets start at 16-byte addresses, whatever the row's.
// The kept entries and the target are written after the others by one wave.
#include "gdn_rows.hpp"

namespace gdn {

namespace {

constexpr int kMaxTop = 256, kMaxVocab = 1 << 20;
constexpr float kLog2ef = 1.4426950408889634f;

struct DistillArgs {
  const void* z;
  const int32_t* ids;
  const float* top;
  const float* teacher_lse;   // null: c is of the kept entries
  const int64_t* targets;     // null: no cross entropy
  const float* d_loss;        // null: 1
  float* loss;
  float* stats;               // forward: written (null in the joint pass); backward: read
  void* dz;
  int64_t row0, stride, d_stride, ignore;
  int V, K;
  float h, kd, ce;
  double ih;                  // 1 / h
};

enum DistillMode { kDisFwd = 0, kDisBwd = 1, kDisBoth = 2 };

// Eight columns as they are stored.
template <typename T>
struct Oct;
template <>
struct Oct<uint16_t> {
  uint4 u;
  static constexpr uint16_t kNone = 0xff80;   // -inf
  __device__ __forceinline__ void none() { u = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
  __device__ __forceinline__ void ld(const uint16_t* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void ld_some(const uint16_t* p, int lo, int hi) {
    uint32_t x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i >= lo && i < hi ? p[i] : kNone;
    u = make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
    x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z); x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
  }
  // columns of a set of bits to -inf
  __device__ __forceinline__ void clear(uint32_t b) {
    uint32_t* p[4] = {&u.x, &u.y, &u.z, &u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (b >> (2 * i) & 1) *p[i] = (*p[i] & 0xffff0000u) | 0xff80u;
      if (b >> (2 * i + 1) & 1) *p[i] = (*p[i] & 0xffffu) | 0xff800000u;
    }
  }
  // their largest value, exactly: an odd column with its neighbour's bits below it would be a NaN for +inf, and off by
  // more than exponentials bear from |z / h| = 1e4 on
  __device__ __forceinline__ float largest() const {
    const float a = fmaxf(fmaxf(bf16_lo(u.x), bf16_hi(u.x)), fmaxf(bf16_lo(u.y), bf16_hi(u.y)));
    return fmaxf(fmaxf(a, fmaxf(bf16_lo(u.z), bf16_hi(u.z))), fmaxf(bf16_lo(u.w), bf16_hi(u.w)));
  }
  // unpacked anew from here on: the compiler would keep the values of an earlier get() instead, twice the registers
  __device__ __forceinline__ void hide() { asm volatile("" : "+v"(u.x), "+v"(u.y), "+v"(u.z), "+v"(u.w)); }
};
template <>
struct Oct<float> {
  float4 a, b;
  __device__ __forceinline__ void none() { a = b = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
  __device__ __forceinline__ void ld(const float* p) { ld(p, p + 4); }
  __device__ __forceinline__ void ld(const float* p, const float* q) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(q);
  }
  __device__ __forceinline__ void ld_some(const float* p, int lo, int hi) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i >= lo && i < hi ? p[i] : -INFINITY;
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ __forceinline__ void clear(uint32_t m) {
    float* p[8] = {&a.x, &a.y, &a.z, &a.w, &b.x, &b.y, &b.z, &b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (m >> i & 1) *p[i] = -INFINITY;
  }
  __device__ __forceinline__ float largest() const {
    return fmaxf(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)), fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w)));
  }
  __device__ __forceinline__ void hide() {}
};

// A whole octet, past the caches: the gradient is not read here again (16384 x
// 32000: 441 us for 468).
__device__ __forceinline__ void st_row(uint16_t* p, uint16_t*, const float (&x)[8]) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const u32x4 u = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
  __builtin_nontemporal_store(u, reinterpret_cast<u32x4*>(p));
}
__device__ __forceinline__ void st_row(float* p, float* q, const float (&x)[8]) {   // in halves
  st_stream(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
  st_stream(reinterpret_cast<float4*>(q), make_float4(x[4], x[5], x[6], x[7]));
}
template <typename T>
__device__ __forceinline__ void st_some(T* p, int lo, int hi, const float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i >= lo && i < hi) {
      if constexpr (sizeof(T) == 2) p[i] = (T)(pack_bf16x2(x[i], x[i]) & 0xffffu);
      else p[i] = x[i];
    }
}

// 2^x by the hardware; results below 2^-126 are 0.
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ double sum_f64(double x) { return last_lane(wave_prefix_f64(x)); }

constexpr float kFar = 1024.0f;   // logsumexps above it are not taken from fp32 statistics

// What a row's gradient is made of; exponentials in base 2.
struct DistillRow {
  float A, x;        // A 2^((z - x) c / h) of every column (c = log2 e) ..
  float B, x1;       // + B 2^((z - x1) c); h = 2: + B (2^((z - x) c / h))^2
  float q, xh;       // kept columns beside a rest: q 2^((z - xh) c / h) ..
  float b;           // .. + b 2^((z - x1) c)
  float a, t;        // factors of p and of the target
  int bad;
};

// A logsumexp of z / h: x / h + s; f = e^-s (large, not infinite, where there is no value).
struct DistillLse {
  double x, s, f;
  // from an fp32 number of at most kFar: |s| <= 2^-14, so f has an error of 2^-44
  __device__ __forceinline__ void read(float l, double h, double ih) {
    x = (double)(float)((double)l * h);
    s = (double)l - x * ih;
    f = fma(s, fma(s, 0.5, -1.0), 1.0);
  }
};
// A lane's value in every lane: wave 0 forms its few logarithms and exponentials one to a lane.
__device__ __forceinline__ double of_lane(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

constexpr int kHash = 1024;

struct DistillShared {
  double p[kMaxTop];                // p_j, a column's whole at its first entry, else 0 (0: unused)
  int id[kMaxTop];                  // -1: unused, or not the column's first entry
  float zj[kMaxTop];
  float zt;                         // the target's logit
  float red[3][16];
  DistillRow row;
  alignas(16) uint32_t hash[kHash];   // id + 1, 0: free
};
static_assert(sizeof(DistillShared) % 16 == 0, "the bitmap behind it");

// The kept entries of a row, one wave: p, the sums over them that the row's
// values need, and the columns that come twice, found by a table of the ids (a
// search through all pairs only where there are any).
struct DistillKept {
  double c, mass, rest;   // c, sum p, r
  double m;               // the largest z_j (0: none is above -inf)
  double kd;              // sum p_j (ln p_j - (z_j - m) / h)
  double e1, eh;          // of the columns, sums of e^(z_j - m), e^((z_j - m) / h) (distill_sums)
  int n;                  // columns
  bool bad;
};

template <typename T>
__device__ __forceinline__ DistillKept distill_kept(const DistillArgs& A, int64_t r, const T* z, DistillShared& sh,
                                                    uint32_t* bits, int shift) {
  constexpr int kPer = kMaxTop / 64;
  const int lane = threadIdx.x & 63, K = A.K;
  const bool tail = A.teacher_lse != nullptr;
  const double ih = A.ih;
  DistillKept o;
#pragma unroll
  for (int i = 0; i < kHash / 256; ++i) reinterpret_cast<uint4*>(sh.hash)[lane + 64 * i] = make_uint4(0, 0, 0, 0);
  int id[kPer];
  float t[kPer], zj[kPer];
  bool out = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int j = lane + 64 * i;
    id[i] = j < K ? A.ids[r * K + j] : -1;
    out |= id[i] >= A.V;
    if (id[i] >= A.V) id[i] = -1;
    t[i] = id[i] >= 0 ? A.top[r * K + j] : -INFINITY;
    zj[i] = id[i] >= 0 ? io<T>::ld(z + id[i]) : -INFINITY;
  }
  bool dup = false;
  float tm = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (64 * i >= K) break;
    tm = fmaxf(tm, t[i]);
    if (id[i] < 0) continue;
    const uint32_t me = (uint32_t)id[i] + 1;
    for (uint32_t at = (me * 2654435761u) >> 22;; at = (at + 1) & (kHash - 1)) {   // at most kMaxTop entries: ends
      const uint32_t was = atomicCAS(&sh.hash[at], 0u, me);
      dup |= was == me;
      if (was == 0u || was == me) break;
    }
    if (bits != nullptr) {
      const int b = id[i] + shift;
      atomicOr(bits + (b >> 5), 1u << (b & 31));
    }
  }
  double m = 0.0;   // ln p_j = (t_j - m) / h - le (in one number c next to t / h of 1e12 nothing is left of le)
  double le;
  if (tail) {
    o.c = le = (double)A.teacher_lse[r];
  } else {
    m = (double)wave_max_dpp(tm);
    double e = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (64 * i < K && t[i] > -INFINITY) e += exp(((double)t[i] - m) * ih);
    e = sum_f64(e);
    le = log(e);
    o.c = e > 0.0 ? m * ih + le : -INFINITY;
  }
  float zm = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPer; ++i) zm = fmaxf(zm, zj[i]);
  zm = wave_max_dpp(zm);
  o.m = zm > -INFINITY ? (double)zm : 0.0;
  double p[kPer], sp = 0.0, kd = 0.0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    p[i] = 0.0;
    if (64 * i >= K) continue;
    out |= id[i] >= 0 && !(t[i] < INFINITY && (!tail || fabs(o.c) < INFINITY));   // not finite, of the teacher's
    const double l = ((double)t[i] - m) * ih - le;
    if (t[i] > -INFINITY) p[i] = exp(l);
    if (p[i] > 0.0) kd += p[i] * (l - ((double)zj[i] - o.m) * ih);
    sp += p[i];
    sh.id[lane + 64 * i] = id[i];
    sh.p[lane + 64 * i] = p[i];
    sh.zj[lane + 64 * i] = zj[i];
  }
  o.bad = __ballot(out) != 0;
  o.mass = sum_f64(sp);
  o.kd = sum_f64(kd);
  if (__ballot(dup) != 0) {   // the first entry of a column takes the others' p
    int keep[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      keep[i] = id[i];
      if (id[i] < 0) continue;
      const int j = lane + 64 * i;
      p[i] = 0.0;
      for (int e = 0; e < K; ++e)
        if (sh.id[e] == id[i]) {
          if (e < j) keep[i] = -1;
          p[i] += sh.p[e];
        }
      if (keep[i] < 0) p[i] = 0.0;
    }
    __builtin_amdgcn_wave_barrier();   // every lane has read before the first writes: one wave, in order
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (64 * i < K) {
        id[i] = keep[i];
        sh.id[lane + 64 * i] = id[i];
        sh.p[lane + 64 * i] = p[i];
      }
  }
  o.rest = 0.0;
  o.n = 0;
  if (tail) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) o.n += __popcll(__ballot(id[i] >= 0));
    o.rest = o.n < A.V ? fmax(0.0, 1.0 - o.mass) : 0.0;   // no column is left: no rest
  } else {
    o.mass = o.c > -INFINITY ? 1.0 : 0.0;
  }
  return o;
}

// The sums over the kept columns, where they are beside a rest.
__device__ __forceinline__ void distill_sums(DistillKept& o, const DistillShared& sh, int K, double ih) {
  double e1 = 0.0, eh = 0.0;
#pragma unroll
  for (int i = 0; i < kMaxTop / 64; ++i) {
    const int j = (int)(threadIdx.x & 63) + 64 * i;
    if (64 * i < K && sh.id[j] >= 0) {
      e1 += exp((double)sh.zj[j] - o.m);
      eh += exp(((double)sh.zj[j] - o.m) * ih);
    }
  }
  o.e1 = sum_f64(e1);
  o.eh = sum_f64(eh);
}

}  // namespace

template <typename T, int TPB, int U, int MODE>
__global__ __launch_bounds__(TPB) void distill_kernel(DistillArgs A) {
  constexpr bool kStats = MODE != kDisBwd, kGrad = MODE != kDisFwd;
  constexpr int NW = TPB / 64;
  extern __shared__ __align__(16) char smem[];
  DistillShared& sh = *reinterpret_cast<DistillShared*>(smem);
  uint8_t* bits = reinterpret_cast<uint8_t*>(smem + sizeof(DistillShared));
  const int64_t r = A.row0 + blockIdx.x;
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int V = A.V, K = A.K;
  const T* z = (const T*)A.z + r * A.stride;
  T* dz = kGrad ? (T*)A.dz + r * A.d_stride : nullptr;
  const bool tail = A.teacher_lse != nullptr;
  const int64_t target = A.targets ? A.targets[r] : 0;
  const bool ignored = A.targets != nullptr && target == A.ignore;
  const bool two = A.targets != nullptr && A.h != 1.0f;   // a second exponential:
  const bool square = A.h == 2.0f;                        // with h = 2 the first one's square
  const float ch = (float)(1.4426950408889634 * A.ih);

  // octet o: columns 8 o - shift .. + 7; whole ones from o0 to o1 - 1, at 16-byte addresses; the columns before and
  // behind them are thread 0's and 1's edge octet, from column e0 with e_lo .. e_hi - 1 of it in the row
  constexpr int kPer = 16 / (int)sizeof(T);
  const int head = (kPer - (int)((uintptr_t)z / sizeof(T) % kPer)) % kPer;
  const int shift = (8 - head) % 8;
  const int o0 = shift > 0 ? 1 : 0, o1 = (V + shift) / 8;
  const int tiles = max(1, (o1 - o0 + TPB * U - 1) / (TPB * U));
  const int e_oct = tid == 0 ? 0 : o1, e0 = 8 * e_oct - shift;
  const bool edge = tid == 0 ? shift > 0 : tid == 1 && (V + shift) % 8 != 0 && o1 >= o0;
  const int e_lo = edge && tid == 0 ? shift : 0, e_hi = edge ? min(8, V - e0) : 0;

  if (ignored) {
    if (kStats && tid == 0) A.loss[r] = 0.0f;
    if (MODE == kDisFwd && tid < 4) A.stats[4 * r + tid] = 0.0f;
    if constexpr (kGrad) {
      const float zero[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      const bool vec = (uintptr_t)(dz + head) % 16 == 0;
      for (int o = o0 + tid; o < o1; o += TPB) {
        if (vec) st_oct<T, true>(dz + 8 * o - shift, 8, zero);
        else st_some(dz + 8 * o - shift, 0, 8, zero);
      }
      if (edge) st_some(dz + e0, e_lo, e_hi, zero);
    }
    return;
  }

  Oct<T> x[U], xe;
  const T* zo = z + 8 * o0 - shift;   // octet o0
  T* dzo = kGrad ? dz + 8 * o0 - shift : nullptr;
  // fp32: a whole wave's octets as two runs of 1 KiB, 16 bytes a lane, so that each access fills its lines (gradient
  // of 1000 x 50001 by 256 threads a row, not in a cache: 83 us for 92)
  auto runs = [&](uint32_t o) { return sizeof(T) == 4 && (int)(o - lane) + 64 <= o1 - o0; };
  auto run_at = [&](uint32_t o) { return (o - lane) * 32u + 16u * lane; };   // the first's bytes from octet o0
  auto load = [&](int tile) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t o = (uint32_t)((tile * U + u) * TPB + tid);
      if constexpr (sizeof(T) == 4) {
        if (runs(o)) {
          x[u].ld((const T*)((const char*)zo + run_at(o)), (const T*)((const char*)zo + run_at(o) + 1024));
          continue;
        }
      }
      if ((int)o < o1 - o0) x[u].ld((const T*)((const char*)zo + o * (uint32_t)(8 * sizeof(T))));
      else x[u].none();
    }
  };
  load(0);
  xe.none();
  if (edge) xe.ld_some(z + e0, e_lo, e_hi);

  const bool mark = tail && kStats;
  if (mark) {
    for (int i = tid; i < (V + shift + 31) / 32; i += TPB) reinterpret_cast<uint32_t*>(bits)[i] = 0u;
    __syncthreads();
  }
  DistillKept kp;   // wave 0's
  if (w == 0) {
    kp = distill_kept<T>(A, r, z, sh, mark ? reinterpret_cast<uint32_t*>(bits) : nullptr, shift);
    if (mark) distill_sums(kp, sh, K, A.ih);
    const bool aim = A.targets != nullptr && target >= 0 && target < V;
    if (A.targets != nullptr && !aim) kp.bad = true;
    if (lane == 0 && aim) sh.zt = io<T>::ld(z + target);
  }
  if (mark) __syncthreads();

  // sums of 2^((z - top) c / h) and 2^((z - top) c), top the largest value so far: exactly subtracted before it is
  // scaled, so that no argument is above 0, however large the logits (a thread whose columns are all masked by the
  // type's lowest value sums theirs, until a real one leaves 0 of the sum).  Both are 0 where there is no value yet
  float top = -INFINITY, sum_h = 0.0f, sum_1 = 0.0f;
  auto reference = [](float m) { return m > -INFINITY ? m : 0.0f; };
  auto raise = [&](float m) {   // a sum over no value is 0, or NaN
    sum_h *= exp2_hw((top - m) * ch);
    sum_1 *= exp2_hw((top - m) * kLog2ef);
    top = m;
  };
  bool again = kStats;
  if constexpr (kStats) {
    for (int tile = 0; tile < tiles; ++tile) {
      if (tile > 0) load(tile);
      float m = top;
      if (mark) {   // kept columns are not of the rest: -inf (their gradient is written by itself)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int o = (tile * U + u) * TPB + tid;
          uint32_t b = 0u;
          if (runs(o)) {
            const uint8_t* half = bits + o0 + (o - lane) + lane / 2;
            b = (half[0] >> 4 * (lane & 1) & 15u) | (half[32] >> 4 * (lane & 1) & 15u) << 4;
          } else if (o < o1 - o0) {
            b = bits[o0 + o];
          }
          if (b != 0u) x[u].clear(b);
        }
        if (edge) xe.clear(bits[e_oct]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) m = fmaxf(m, x[u].largest());
      if (tile == 0) m = fmaxf(m, xe.largest());
      if (m > top) raise(m);
      const float to = reference(top);
      auto add = [&](const Oct<T>& y) {
        float v[8];
        y.get(v);
        if (!two) {
#pragma unroll
          for (int i = 0; i < 8; ++i) sum_h += exp2_hw((v[i] - to) * ch);
        } else if (square) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float e = exp2_hw((v[i] - to) * ch);
            sum_h += e;
            sum_1 = fmaf(e, e, sum_1);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            sum_h += exp2_hw((v[i] - to) * ch);
            sum_1 += exp2_hw((v[i] - to) * kLog2ef);
          }
        }
      };
#pragma unroll
      for (int u = 0; u < U; ++u) {
        x[u].hide();
        add(x[u]);
        __builtin_amdgcn_sched_barrier(0);   // octet by octet: mixed, they take twice the registers
      }
      if (tile == 0 && edge) add(xe);
    }
  } else {
    const float* s = A.stats + 4 * r;
    const bool none = s[3] == -INFINITY && A.h >= 1.0f;   // of the rest (h < 1: or a logsumexp below fp32's)
    again = fabsf(s[1]) > kFar || (A.targets != nullptr && fabsf(s[0]) > kFar) ||
            (tail && !none && fabsf(s[3]) > kFar);
    if (again) {
      __syncthreads();   // the table of the kept columns
      auto kept = [&](int i) {
        const uint32_t me = (uint32_t)i + 1;
        for (uint32_t at = (me * 2654435761u) >> 22;; at = (at + 1) & (kHash - 1)) {   // at most kMaxTop entries: ends
          const uint32_t was = sh.hash[at];
          if (was == me || was == 0u) return was == me;
        }
      };
#pragma unroll 1
      for (int i = tid; i < V; i += TPB) {
        if (tail && kept(i)) continue;
        const float v = io<T>::ld(z + i);
        if (v > top) raise(v);
        const float to = reference(top);
        sum_h += exp2_hw((v - to) * ch);
        sum_1 += exp2_hw((v - to) * kLog2ef);
      }
    }
  }
  if (again) {   // over the wave, then the workgroup
    const float m = wave_max_dpp(top);
    raise(reference(m));
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      sum_h += __shfl_xor(sum_h, o, 64);
      sum_1 += __shfl_xor(sum_1, o, 64);
    }
    if (lane == 0) {
      sh.red[0][w] = m;
      sh.red[1][w] = sum_h;
      sh.red[2][w] = sum_1;
    }
    __syncthreads();
  }

  // the row's few values: wave 0
  if (w == 0) {
    const double ih = A.ih;
    DistillLse all, one, rest;   // of z / h, of z, of z / h over the rest (s = -inf: no value)
    if (again) {
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < NW; ++i) m = fmaxf(m, sh.red[0][i]);
      const bool none = !(m > -INFINITY);
      m = reference(m);
      double ah = 0.0, a1 = 0.0;
#pragma unroll
      for (int i = 0; i < NW; ++i) {   // a wave without any value has sums of 0, or NaN
        const float below = sh.red[0][i] - m;
        ah += (double)(sh.red[1][i] * exp2_hw(below * ch));
        a1 += (double)(sh.red[2][i] * exp2_hw(below * kLog2ef));
      }
      rest.x = all.x = (double)m;
      double sh_ = ah, s1 = a1;
      if (!kStats && tail) distill_sums(kp, sh, K, ih);
      if (tail && kp.n > 0) {   // and the kept columns', relative to the larger maximum
        const double x = none ? kp.m : kp.eh == 0.0 ? rest.x : fmax(rest.x, kp.m);
        const double e = exp(lane == 0 ? (rest.x - x) * ih : lane == 1 ? (kp.m - x) * ih : lane == 2 ? rest.x - x : kp.m - x);
        auto moved = [](double s, double by) { return s == 0.0 ? 0.0 : s * by; };
        all.x = x;
        sh_ = moved(ah, of_lane(e, 0)) + moved(kp.eh, of_lane(e, 1));
        s1 = moved(a1, of_lane(e, 2)) + moved(kp.e1, of_lane(e, 3));
      }
      const double l = log(lane == 0 ? ah : lane == 1 ? sh_ : lane == 2 ? s1 : kp.rest);
      rest.s = of_lane(l, 0);
      all.s = of_lane(l, 1);
      one.x = all.x;
      one.s = two ? of_lane(l, 2) : all.s;
      if constexpr (kGrad) {
        const double s = lane == 0 ? all.s : lane == 1 ? rest.s : one.s;
        const double f = exp(s < -700.0 ? 700.0 : -s);
        all.f = of_lane(f, 0);
        rest.f = of_lane(f, 1);
        one.f = of_lane(f, 2);
      }
      if constexpr (kStats) {
        double kd = kp.kd + (kp.mass > 0.0 ? kp.mass * ((all.x - kp.m) * ih + all.s) : 0.0);
        if (tail && kp.rest > 0.0)
          kd += kp.rest * (of_lane(l, 3) - ((rest.x - all.x) * ih + (rest.s - all.s)));
        double loss = (double)A.kd * kd;
        if (A.targets != nullptr && !kp.bad) loss += (double)A.ce * ((one.x - (double)sh.zt) + one.s);
        if (lane == 0) A.loss[r] = kp.bad ? NAN : (float)loss;
        if constexpr (MODE == kDisFwd) {
          if (lane < 4) {
            const double s = lane == 0 ? (A.targets ? one.x + one.s : 0.0)
                             : lane == 1 ? all.x * ih + all.s : lane == 2 ? kp.c : tail ? rest.x * ih + rest.s : 0.0;
            A.stats[4 * r + lane] = kp.bad ? NAN : (float)s;
          }
        }
      }
    } else {
      one.read(A.stats[4 * r], 1.0, 1.0);
      all.read(A.stats[4 * r + 1], (double)A.h, ih);
      rest.read(A.stats[4 * r + 3], (double)A.h, ih);
      if (A.stats[4 * r + 3] == -INFINITY) rest = DistillLse{0.0, -INFINITY, 1.0};   // no value of the rest
    }
    if constexpr (kGrad) {
      const double wt = A.d_loss ? (double)A.d_loss[r] : 1.0;
      const double a = wt * (double)A.kd * ih, b = A.targets ? wt * (double)A.ce : 0.0;
      const double m = kp.mass + kp.rest;
      // of every column: ea e^(z / h - l) + eb e^(z - one), l the rest's logsumexp where there is one
      const DistillLse l = tail ? rest : all;
      const double e = exp(lane == 0 ? (rest.x - all.x) * ih + (rest.s - all.s) : (l.x - one.x) - one.s);
      double ea = a * m, eb = b;
      if (tail) {
        const bool any = rest.s != -INFINITY;   // a NaN is a value
        ea = any ? a * (m * of_lane(e, 0) - kp.rest) : 0.0;
        eb = any ? b : 0.0;   // none but -inf: no column takes them, and e^(l - one) may be infinite
      }
      DistillRow d;
      d.a = (float)a;
      d.t = (float)b;
      d.xh = (float)all.x;
      d.q = (float)(a * m * all.f);
      d.x1 = (float)one.x;
      d.b = (float)(b * one.f);
      d.x = (float)l.x;
      d.A = (float)(ea * l.f);
      d.B = (float)(eb * one.f);
      if (eb != 0.0 && (!two || square)) {   // one exponential for both
        const double be = eb * of_lane(e, 1);
        d.B = two ? (float)be : 0.0f;
        if (!two) d.A = (float)(ea * l.f + be);
      }
      d.bad = kp.bad;
      if (kp.bad) d.A = NAN;
      if (lane == 0) sh.row = d;
    }
  }

  if constexpr (kGrad) {
    __syncthreads();
    const DistillRow d = sh.row;
    // wave 0: what the kept columns and the target get (from logits read before any store: dz may be z)
    constexpr int kMine = kMaxTop / 64;
    int to[kMine + 1];
    float val[kMine + 1];
    if (w == 0) {
      auto column = [&](float zv) {
        const float e = exp2_hw((zv - d.x) * ch);
        float g = d.A * e;
        if (d.B != 0.0f) g += d.B * (square ? e * e : exp2_hw((zv - d.x1) * kLog2ef));
        return g;
      };
      bool met = false;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int j = lane + 64 * i;
        to[i] = j < K && !d.bad ? sh.id[j] : -1;
        if (to[i] < 0) continue;
        const float zv = sh.zj[j];
        float g;
        if (tail) {
          g = d.q * exp2_hw((zv - d.xh) * ch);
          if (d.b != 0.0f) g += d.b * exp2_hw((zv - d.x1) * kLog2ef);
        } else {
          g = column(zv);
        }
        g -= d.a * (float)sh.p[j];
        if (A.targets != nullptr && to[i] == (int)target) {
          g -= d.t;
          met = true;
        }
        val[i] = g;
      }
      to[kMine] = -1;
      if (__ballot(met) == 0 && lane == 0 && A.targets != nullptr && !d.bad) {
        to[kMine] = (int)target;
        val[kMine] = column(sh.zt) - d.t;
      }
    }
    const bool vec = (uintptr_t)(dz + head) % 16 == 0;
    auto grads = [&](const Oct<T>& y, float (&g)[8]) {
      float v[8];
      y.get(v);
      if (d.B == 0.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = d.A * exp2_hw((v[i] - d.x) * ch);
      } else if (square) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float e = exp2_hw((v[i] - d.x) * ch);
          g[i] = e * fmaf(d.B, e, d.A);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          g[i] = fmaf(d.B, exp2_hw((v[i] - d.x1) * kLog2ef), d.A * exp2_hw((v[i] - d.x) * ch));
      }
    };
    // the last tile first where both passes run: it is still in registers
    for (int i = 0; i < tiles; ++i) {
      const int tile = MODE == kDisBoth ? tiles - 1 - i : i;
      if (i > 0) load(tile);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t o = (uint32_t)((tile * U + u) * TPB + tid);
        x[u].hide();
        if ((int)o < o1 - o0) {
          float g[8];
          grads(x[u], g);
          T* to_o = (T*)((char*)dzo + o * (uint32_t)(8 * sizeof(T)));
          T* to_q = to_o + 4;
          if (runs(o)) {
            to_o = (T*)((char*)dzo + run_at(o));
            to_q = to_o + 256;
          }
          if (vec) st_row(to_o, to_q, g);
          else st_some(to_o, 0, 4, g), st_some(to_q - 4, 4, 8, g);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (edge) {
      float g[8];
      grads(xe, g);
      st_some(dz + e0, e_lo, e_hi, g);
    }
    __syncthreads();   // the kept columns' and the target's values replace the others
    if (w == 0) {
#pragma unroll
      for (int i = 0; i <= kMine; ++i)
        if (to[i] >= 0) io<T>::st(dz + to[i], val[i]);
    }
  }
}

namespace {

template <typename T, int TPB, int U, int MODE>
hipError_t launch_row(const gdn_distill_t& s, DistillArgs a, hipStream_t stream) {
  // the bitmap only where sums are formed beside a rest
  const size_t lds = sizeof(DistillShared) +
                     (a.teacher_lse != nullptr && MODE != kDisBwd ? ((size_t)(a.V + 14) / 8 + 3) / 4 * 4 : 0);
  constexpr size_t most = sizeof(DistillShared) + ((size_t)kMaxVocab + 14) / 8 + 4;
  static_assert(most <= 160 * 1024, "LDS budget exceeded");
  auto kern = distill_kernel<T, TPB, U, MODE>;
  static PerDeviceOnce once;
  hipError_t e = set_dyn_lds_once(once, (const void*)kern, most);
  if (e != hipSuccess) return e;
  for (int64_t r0 = 0; r0 < s.rows; r0 += max_blocks(TPB)) {
    a.row0 = r0;
    const int64_t n = s.rows - r0 < max_blocks(TPB) ? s.rows - r0 : max_blocks(TPB);
    hipLaunchKernelGGL(kern, dim3((unsigned)n), dim3(TPB), lds, stream, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, int TPB, int U>
hipError_t launch_rows(const gdn_distill_t& s, const DistillArgs& a, int mode, hipStream_t stream) {
  if (mode == kDisFwd) return launch_row<T, TPB, U, kDisFwd>(s, a, stream);
  return mode == kDisBwd ? launch_row<T, TPB, U, kDisBwd>(s, a, stream) : launch_row<T, TPB, U, kDisBoth>(s, a, stream);
}

}  // namespace

hipError_t launch_distill(const gdn_distill_t& s, const void* logits, const int32_t* ids, const float* top,
                          const float* teacher_lse, const int64_t* targets, const float* d_loss, float* loss,
                          float* stats, void* d_logits, hipStream_t stream) {
  const int mode = d_logits == nullptr ? kDisFwd : loss == nullptr ? kDisBwd : kDisBoth;
  DistillArgs a{};
  a.z = logits; a.ids = ids; a.top = top; a.teacher_lse = teacher_lse; a.targets = targets;
  a.d_loss = d_loss; a.loss = loss; a.stats = stats; a.dz = d_logits;
  a.stride = s.row_stride; a.d_stride = s.d_row_stride; a.ignore = s.ignore_index;
  a.V = s.vocab; a.K = s.topk;
  a.h = s.temperature; a.ih = 1.0 / (double)s.temperature; a.kd = s.kd_weight; a.ce = s.ce_weight;
  // Threads a row and octets a thread.  The losses: four octets on the way, many workgroups a compute unit (16384 x
  // 32000 bf16: 192 us; 16 octets took 256 registers and 670 us), and 1024 threads for a long row where each has a
  // compute unit to itself (256 x 131072: bf16 19 us for 35 with 256 threads, fp32 25.4 for 26.5; 1024 x 131072 would
  // take 65 for 51 and 97 for 89, 4096 rows in bf16 283 for 193).  Both: as much of the row in registers as leaves two
  // workgroups a compute unit, the rest read again from the last-level cache (4096 x 131072 bf16: 438 us with 512
  // threads and half a row, 612 with 1024 and all of it, 484 with 256 and a quarter).  The gradient alone, bf16: 417 us
  // with 16 octets, 441 with four (16384 x 32000); fp32: as below.
  const int octs = s.vocab / 8 + 2;
  const bool alone = octs > 8192 && s.rows <= device_cu_count();
  if (s.dtype == GDN_BF16) {
    if (octs <= 64 * 4) return launch_rows<uint16_t, 64, 4>(s, a, mode, stream);
    if (octs <= 256 * 4) return launch_rows<uint16_t, 256, 4>(s, a, mode, stream);
    if (mode == kDisFwd)
      return alone ? launch_row<uint16_t, 1024, 4, kDisFwd>(s, a, stream)
                   : launch_row<uint16_t, 256, 4, kDisFwd>(s, a, stream);
    if (mode == kDisBwd) return launch_row<uint16_t, 256, 16, kDisBwd>(s, a, stream);
    return octs <= 256 * 16 ? launch_row<uint16_t, 256, 16, kDisBoth>(s, a, stream)
                            : launch_row<uint16_t, 512, 16, kDisBoth>(s, a, stream);
  }
  if (octs <= 64 * 4) return launch_rows<float, 64, 4>(s, a, mode, stream);
  if (octs <= 256 * 4) return launch_rows<float, 256, 4>(s, a, mode, stream);
  if (mode == kDisFwd)
    return alone ? launch_row<float, 1024, 4, kDisFwd>(s, a, stream) : launch_row<float, 256, 4, kDisFwd>(s, a, stream);
  // the gradient alone: a row in the fewest turns once it fills most of 1024 threads (4000 x 32000: 174 us for 199
  // with 256 threads, 1000 x 50001 77 for 83; 1000 x 20011 would take 36.5 for 34.8)
  if (mode == kDisBwd)
    return octs < 3584 ? launch_row<float, 256, 4, kDisBwd>(s, a, stream)
                       : launch_row<float, 1024, 4, kDisBwd>(s, a, stream);
  // both, fp32: 256 threads while they hold the row (4000 x 16000: 90 us for 105 with 512), else 512 (2000 x 50001: 163
  // us; 256 threads 182, 256 and 1024 threads of four octets 193)
  return octs <= 256 * 8 ? launch_row<float, 256, 8, kDisBoth>(s, a, stream)
                         : launch_row<float, 512, 8, kDisBoth>(s, a, stream);
}

}  // namespace gdn
