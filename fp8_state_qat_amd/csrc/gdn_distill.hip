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
// its sums (p, c, r, the loss) in fp64, as 1 - sum p cancels.
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
constexpr double kLn2d = 0.6931471805599453;
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
};
template <>
struct Oct<float> {
  float4 a, b;
  __device__ __forceinline__ void none() { a = b = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
  __device__ __forceinline__ void ld(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
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
};

template <typename T>
__device__ __forceinline__ void st_some(T* p, int lo, int hi, const float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i >= lo && i < hi) {
      if constexpr (sizeof(T) == 2) p[i] = (T)(pack_bf16x2(x[i], x[i]) & 0xffffu);
      else p[i] = x[i];
    }
}

// e^x by the hardware's 2^x; x <= a few, results below 2^-126 are 0.
__device__ __forceinline__ float exp_hw(float x) { return __builtin_amdgcn_exp2f(x * kLog2ef); }

__device__ __forceinline__ double wave_max_f64(double x) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) x = fmax(x, __shfl_xor(x, o, 64));
  return x;
}
__device__ __forceinline__ double wave_sum_f64(double x) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) x += __shfl_xor(x, o, 64);
  return x;
}

// What a row's gradient is made of.
struct DistillRow {
  float A, L;        // A e^(z / h - L) of every column ..
  float B, lse;      // + B e^(z - lse)
  float q, lse_h;    // kept columns beside a rest: q e^(z / h - lse_h) in place of the first
  float a, b;        // factors of p and of [v = target]
  int bad;
};

struct DistillShared {
  double p[kMaxTop], lt[kMaxTop];   // p_j and ln p_j (0 and 0 where unused)
  int id[kMaxTop];                  // -1: unused
  float zj[kMaxTop];
  float zt;                         // the target's logit
  float red[3][16];
  DistillRow row;
};

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
  const bool two = A.targets != nullptr && A.h != 1.0f;   // a second exponential
  const float ih = 1.0f / A.h;

  // octet o: columns 8 o - shift .. + 7
  constexpr int kPer = 16 / (int)sizeof(T);
  const int head = (kPer - (int)((uintptr_t)z / sizeof(T) % kPer)) % kPer;
  const int shift = (8 - head) % 8;
  const int octs = (V + shift + 7) / 8;
  const int tiles = (octs + TPB * U - 1) / (TPB * U);

  if (ignored) {
    if (kStats && tid == 0) A.loss[r] = 0.0f;
    if (MODE == kDisFwd && tid < 4) A.stats[4 * r + tid] = 0.0f;
    if constexpr (kGrad) {
      const float zero[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      const bool vec = (uintptr_t)(dz + head) % 16 == 0;
      for (int o = tid; o < octs; o += TPB) {
        const int v0 = 8 * o - shift;
        if (vec && v0 >= 0 && v0 + 8 <= V) st_oct<T, true>(dz + v0, 8, zero);
        else st_some(dz + v0, max(0, -v0), min(8, V - v0), zero);
      }
    }
    return;
  }

  Oct<T> x[U];
  auto load = [&](int tile) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int o = (tile * U + u) * TPB + tid, v0 = 8 * o - shift;
      if (o >= octs) x[u].none();
      else if (v0 >= 0 && v0 + 8 <= V) x[u].ld(z + v0);
      else x[u].ld_some(z + v0, max(0, -v0), min(8, V - v0));
    }
  };
  load(0);

  // the kept entries
  if (tail && kStats) {
    for (int i = tid; i < (octs + 3) / 4; i += TPB) reinterpret_cast<uint32_t*>(bits)[i] = 0u;
    __syncthreads();
  }
  double c = 0.0, mass = 0.0, rest = 0.0;   // wave 0's: c, sum p, r
  bool bad = A.targets != nullptr && (target < 0 || target >= V);
  if (w == 0) {
    if (lane == 0 && A.targets != nullptr && !bad) sh.zt = io<T>::ld(z + target);
    double m = -INFINITY;
    bool out = false;
    for (int j = lane; j < K; j += 64) {
      const int id = A.ids[r * K + j];
      out |= id >= V;
      const int use = id >= 0 && id < V ? id : -1;
      const double t = use >= 0 ? (double)A.top[r * K + j] / (double)A.h : -INFINITY;
      sh.id[j] = use;
      sh.zj[j] = use >= 0 ? io<T>::ld(z + use) : -INFINITY;
      sh.lt[j] = t;
      m = fmax(m, t);
      if (tail && kStats && use >= 0) {
        const int at = use + shift;
        atomicOr(reinterpret_cast<uint32_t*>(bits) + (at >> 5), 1u << (at & 31));
      }
    }
    bad |= __ballot(out) != 0;
    if (tail) {
      c = (double)A.teacher_lse[r];
    } else {
      m = wave_max_f64(m);
      double s = 0.0;
      if (m > -INFINITY)
        for (int j = lane; j < K; j += 64) s += exp(sh.lt[j] - m);
      s = wave_sum_f64(s);
      c = m > -INFINITY ? m + log(s) : -INFINITY;
    }
    double sum = 0.0;
    for (int j = lane; j < K; j += 64) {
      const double l = sh.lt[j] - c, p = sh.lt[j] > -INFINITY ? exp(l) : 0.0;
      sh.p[j] = p;
      sh.lt[j] = p > 0.0 ? l : 0.0;
      sum += p;
    }
    mass = wave_sum_f64(sum);
    if (tail) rest = fmax(0.0, 1.0 - mass);
    else mass = c > -INFINITY ? 1.0 : 0.0;
  }
  __syncthreads();

  float mx = -INFINITY, s1 = 0.0f, sh_ = 0.0f;   // maximum, sums of e^(z - mx), e^((z - mx) / h)
  if constexpr (kStats) {
    for (int tile = 0; tile < tiles; ++tile) {
      if (tile > 0) load(tile);
      float m = mx;
      uint32_t ex[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int o = (tile * U + u) * TPB + tid;
        ex[u] = tail && o < octs ? bits[o] : 0u;
        float v[8];
        x[u].get(v);
        if (ex[u] != 0u) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = ex[u] >> i & 1 ? -INFINITY : v[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, v[i]);
      }
      const float ref = m > -INFINITY ? m : 0.0f;
      if (m > mx) {
        s1 *= exp_hw(mx - ref);
        sh_ *= exp_hw((mx - ref) * ih);
        mx = m;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[8];
        x[u].get(v);
        if (ex[u] != 0u) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = ex[u] >> i & 1 ? -INFINITY : v[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sh_ += exp_hw((v[i] - ref) * ih);
        if (two) {
#pragma unroll
          for (int i = 0; i < 8; ++i) s1 += exp_hw(v[i] - ref);
        }
      }
    }
    // over the wave, then the workgroup
    float m = mx;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
    const float ref = m > -INFINITY ? m : 0.0f;
    s1 *= exp_hw(mx - ref);
    sh_ *= exp_hw((mx - ref) * ih);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      s1 += __shfl_xor(s1, o, 64);
      sh_ += __shfl_xor(sh_, o, 64);
    }
    if (lane == 0) {
      sh.red[0][w] = m;
      sh.red[1][w] = s1;
      sh.red[2][w] = sh_;
    }
    __syncthreads();
  }

  // the row's few values: wave 0
  if (w == 0) {
    const double h = (double)A.h;
    double lse, lse_h, lse_r;   // of z, of z / h, of z / h over the rest
    if constexpr (kStats) {
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < NW; ++i) m = fmaxf(m, sh.red[0][i]);
      double a1 = 0.0, ah = 0.0;
#pragma unroll
      for (int i = 0; i < NW; ++i) {   // a wave without any value has sums of 0, or NaN
        const float d = sh.red[0][i] > -INFINITY ? sh.red[0][i] - m : 0.0f;
        a1 += (double)(sh.red[1][i] * exp_hw(d));
        ah += (double)(sh.red[2][i] * exp_hw(d * ih));
      }
      if (!two) a1 = ah;
      lse_r = lse_h = ah > 0.0 || ah != ah ? (double)m / h + log(ah) : -INFINITY;
      lse = a1 > 0.0 || a1 != a1 ? (double)m + log(a1) : -INFINITY;
      if (tail) {
        // the kept entries (each column once) join the rest
        double mh = -INFINITY;
        for (int j = lane; j < K; j += 64) mh = fmax(mh, (double)sh.zj[j]);
        mh = fmax(wave_max_f64(mh), (double)m);
        double e1 = 0.0, eh = 0.0;
        int n = 0;
        if (mh > -INFINITY) {
          for (int j = lane; j < K; j += 64) {
            const int id = sh.id[j];
            bool first = id >= 0;
            for (int i = 0; i < j; ++i) first &= sh.id[i] != id;
            if (!first) continue;
            ++n;
            e1 += exp((double)sh.zj[j] - mh);
            eh += exp(((double)sh.zj[j] - mh) / h);
          }
          e1 = wave_sum_f64(e1) + exp(lse - mh);
          eh = wave_sum_f64(eh) + exp(lse_r - mh / h);
          n = (int)wave_sum_f64((double)n);
          lse = mh + log(e1);
          lse_h = mh / h + log(eh);
        }
        if (n == V) rest = 0.0;   // no column is left
      }
      double kd = 0.0;
      for (int j = lane; j < K; j += 64)
        if (sh.p[j] > 0.0) kd += sh.p[j] * (sh.lt[j] - ((double)sh.zj[j] / h - lse_h));
      kd = wave_sum_f64(kd);
      if (rest > 0.0) kd += rest * (log(rest) - (lse_r - lse_h));
      double loss = (double)A.kd * kd;
      if (A.targets != nullptr && !bad) loss += (double)A.ce * (lse - (double)sh.zt);
      if (lane == 0) A.loss[r] = bad ? NAN : (float)loss;
      if constexpr (MODE == kDisFwd) {
        if (lane < 4) {
          const double s = lane == 0 ? (A.targets ? lse : 0.0) : lane == 1 ? lse_h : lane == 2 ? c : tail ? lse_r : 0.0;
          A.stats[4 * r + lane] = bad ? NAN : (float)s;
        }
      }
    } else {
      lse = (double)A.stats[4 * r];
      lse_h = (double)A.stats[4 * r + 1];
      lse_r = (double)A.stats[4 * r + 3];
      if (tail) {
        int n = 0;
        if (K >= V) {   // every column may be kept
          for (int j = lane; j < K; j += 64) {
            bool first = sh.id[j] >= 0;
            for (int i = 0; i < j; ++i) first &= sh.id[i] != sh.id[j];
            n += first ? 1 : 0;
          }
          n = (int)wave_sum_f64((double)n);
        }
        if (n == V) rest = 0.0;
      }
    }
    if constexpr (kGrad) {
      const double wt = A.d_loss ? (double)A.d_loss[r] : 1.0;
      const double a = wt * (double)A.kd / h, b = A.targets ? wt * (double)A.ce : 0.0, m = mass + rest;
      DistillRow d;
      d.a = (float)a;
      d.b = (float)b;
      d.lse_h = (float)lse_h;
      d.lse = (float)lse;
      d.B = (float)b;
      d.q = d.A = (float)(a * m);
      d.L = d.lse_h;
      if (tail) {
        d.A = lse_r > -INFINITY ? (float)(a * (m * exp(lse_r - lse_h) - rest)) : 0.0f;
        d.L = lse_r > -INFINITY ? (float)lse_r : 0.0f;
      }
      if (A.targets == nullptr) {
        d.B = 0.0f;
        d.lse = 0.0f;
      } else if (!two) {   // one exponential for both
        if (!tail) {
          d.A = (float)(a * m + b);
        } else if (lse_r > -INFINITY) {
          d.A = (float)(a * (m * exp(lse_r - lse_h) - rest) + b * exp(lse_r - lse));
        }
        d.B = 0.0f;
      }
      d.bad = bad;
      if (bad) d.A = NAN;
      if (lane == 0) sh.row = d;
    }
  }

  if constexpr (kGrad) {
    __syncthreads();
    const DistillRow d = sh.row;
    // wave 0: what the kept columns and the target get (from logits read before any store: dz may be z)
    constexpr int kMine = (kMaxTop + 1 + 63) / 64;
    int to[kMine];
    float val[kMine];
    if (w == 0) {
      const int n = K + (A.targets != nullptr ? 1 : 0);
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int j = lane + 64 * i;
        to[i] = -1;
        if (j >= n || d.bad) continue;
        const int id = j < K ? sh.id[j] : (int)target;
        if (id < 0) continue;
        bool first = true, kept = j < K;
        double sum = 0.0;
        for (int e = 0; e < K; ++e)
          if (sh.id[e] == id) {
            first &= e >= j;
            kept = true;
            sum += sh.p[e];
          }
        if (!first) continue;
        const float zv = j < K ? sh.zj[j] : sh.zt;
        float g;
        if (tail && kept) {
          g = d.q * exp_hw(fmaf(zv, ih, -d.lse_h));
          if (d.b != 0.0f) g += d.b * exp_hw(zv - d.lse);
        } else {
          g = d.A * exp_hw(fmaf(zv, ih, -d.L));
          if (d.B != 0.0f) g += d.B * exp_hw(zv - d.lse);
        }
        g -= d.a * (float)sum;
        if (A.targets != nullptr && id == (int)target) g -= d.b;
        to[i] = id;
        val[i] = g;
      }
    }
    const bool vec = (uintptr_t)(dz + head) % 16 == 0;
    for (int tile = 0; tile < tiles; ++tile) {
      if (tiles > 1 && (MODE == kDisBoth || tile > 0)) load(tile);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int o = (tile * U + u) * TPB + tid, v0 = 8 * o - shift;
        if (o >= octs) continue;
        float v[8], g[8];
        x[u].get(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = d.A * exp_hw(fmaf(v[i], ih, -d.L));
        if (d.B != 0.0f) {
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] = fmaf(d.B, exp_hw(v[i] - d.lse), g[i]);
        }
        if (vec && v0 >= 0 && v0 + 8 <= V) st_oct<T, true>(dz + v0, 8, g);
        else st_some(dz + v0, max(0, -v0), min(8, V - v0), g);
      }
    }
    __syncthreads();   // the kept columns' and the target's values replace the others
    if (w == 0) {
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        if (to[i] >= 0) io<T>::st(dz + to[i], val[i]);
    }
  }
}

namespace {

template <typename T, int TPB, int U>
hipError_t launch_rows(const gdn_distill_t& s, DistillArgs a, int mode, hipStream_t stream) {
  // the bitmap only where sums are formed beside a rest
  const size_t lds = sizeof(DistillShared) +
                     (a.teacher_lse != nullptr && mode != kDisBwd ? ((size_t)(a.V + 14) / 8 + 3) / 4 * 4 : 0);
  auto go = [&](auto kern, PerDeviceOnce& once) {
    constexpr size_t most = sizeof(DistillShared) + ((size_t)kMaxVocab + 14) / 8 + 4;
    static_assert(most <= 160 * 1024, "LDS budget exceeded");
    hipError_t e = set_dyn_lds_once(once, (const void*)kern, most);
    if (e != hipSuccess) return e;
    for (int64_t r0 = 0; r0 < s.rows; r0 += max_blocks(TPB)) {
      a.row0 = r0;
      const int64_t n = s.rows - r0 < max_blocks(TPB) ? s.rows - r0 : max_blocks(TPB);
      hipLaunchKernelGGL(kern, dim3((unsigned)n), dim3(TPB), lds, stream, a);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
  };
  static PerDeviceOnce once[3];
  if (mode == kDisFwd) return go(distill_kernel<T, TPB, U, kDisFwd>, once[0]);
  if (mode == kDisBwd) return go(distill_kernel<T, TPB, U, kDisBwd>, once[1]);
  return go(distill_kernel<T, TPB, U, kDisBoth>, once[2]);
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
  a.h = s.temperature; a.kd = s.kd_weight; a.ce = s.ce_weight;
  const int octs = s.vocab / 8 + 2;
  if (s.dtype == GDN_BF16) {
    if (octs <= 64 * 4) return launch_rows<uint16_t, 64, 4>(s, a, mode, stream);
    if (octs <= 256 * 4) return launch_rows<uint16_t, 256, 4>(s, a, mode, stream);
    if (octs <= 256 * 16) return launch_rows<uint16_t, 256, 16>(s, a, mode, stream);
    return launch_rows<uint16_t, 1024, 16>(s, a, mode, stream);
  }
  if (octs <= 64 * 4) return launch_rows<float, 64, 4>(s, a, mode, stream);
  if (octs <= 256 * 8) return launch_rows<float, 256, 8>(s, a, mode, stream);
  return launch_rows<float, 1024, 8>(s, a, mode, stream);
}

}  // namespace gdn
