// gdn_lin.hip -- host side of linear attention: segment length, workspace,
// the order of the scan passes, and the small kernels between them.
#include "gdn_lin_scan.hpp"

namespace gdn {

namespace {

// Segment sums to segment starts: seg[s] holds the segment's own sum and
// becomes the state at its start (forward: before the first token; reverse:
// after the last), cur <- e^(its decays) cur + sum.  One thread per four
// state values, blockIdx.y: sequence, blockIdx.z: direction.
struct LinStarts {
  float* seg;
  const float* decay;
  const float* first;
};
template <bool kRev>
__device__ __forceinline__ void lin_starts(const LinStarts& P, const LinSeg& q, int VH, int st4) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  const int vh = i / st4, e = i % st4;
  if (vh >= VH) return;
  float4* S = reinterpret_cast<float4*>(P.seg);
  float4 cur = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (P.first != nullptr) cur = reinterpret_cast<const float4*>(P.first)[((int64_t)q.n * VH + vh) * st4 + e];
  auto at = [&](int j) { return (int64_t)(q.slot0 + (kRev ? q.nseg - 1 - j : j)) * VH + vh; };
  constexpr int kAhead = 8;
  float4 own[kAhead];
  float dec[kAhead];
  for (int j0 = 0; j0 < q.nseg; j0 += kAhead) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (j0 + k < q.nseg - 1) {   // the last segment of the walk has no sum
        own[k] = S[at(j0 + k) * st4 + e];
        dec[k] = P.decay[at(j0 + k)];
      }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int j = j0 + k;
      if (j >= q.nseg) break;
      S[at(j) * st4 + e] = cur;
      if (j < q.nseg - 1) {
        cur.x = fmaf(cur.x, dec[k], own[k].x);
        cur.y = fmaf(cur.y, dec[k], own[k].y);
        cur.z = fmaf(cur.z, dec[k], own[k].z);
        cur.w = fmaf(cur.w, dec[k], own[k].w);
      }
    }
  }
}
__global__ __launch_bounds__(kThreads) void lin_starts_kernel(LinStarts F, LinStarts R,
                                                              const int32_t* __restrict__ cu, int N, int64_t T,
                                                              int seglen, int VH, int st4) {
  const LinSeg q = lin_find(cu, N, T, seglen, blockIdx.y, true);
  if (q.bad) return;
  if (blockIdx.z == 0) lin_starts<false>(F, q, VH, st4);
  else lin_starts<true>(R, q, VH, st4);
}

// The sums that end a backward, one launch.  blockIdx.y 0, 1: dq and dk, where
// R virtual heads share a query/key head, in fp32 and in order, four values a
// thread, rows [cu[0], cu[N]) only.  blockIdx.y 2: dg, from the tiles of a
// token's value rows, or for fixed decays from the segments' sums in fp64, one
// workgroup a head.  The caller leaves out what it does not need.
struct LinReduce {
  const float* part_q;
  const float* part_k;
  void* dq;
  void* dk;
  const float* dg_tok;
  const double* dg_part;
  float* dg;
  const int32_t* cu;
  const int32_t* status;
  int64_t slots, row4;
  int N, R, d4, H, VH, tiles;
  int y0;               // blockIdx.y of the launch's first part
};

template <typename T>
__device__ __forceinline__ void lin_reduce_qk(const LinReduce& A, const float* part, T* out0) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x + (int64_t)A.cu[0] * A.row4;
  if (i >= (int64_t)A.cu[A.N] * A.row4) return;
  const int64_t head = i / A.d4;           // row * qk_heads + head
  const float4* p = reinterpret_cast<const float4*>(part) + head * A.R * A.d4 + i % A.d4;
  float4 s = p[0];
  for (int r = 1; r < A.R; ++r) {
    const float4 x = p[(int64_t)r * A.d4];
    s.x += x.x;
    s.y += x.y;
    s.z += x.z;
    s.w += x.w;
  }
  T* out = out0 + 4 * i;
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  else
    *reinterpret_cast<float4*>(out) = s;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void lin_reduce_kernel(LinReduce A) {
  __shared__ double sum[kThreads];
  if (*A.status != 0) return;
  const int y = blockIdx.y + A.y0;
  if (y < 2) {
    lin_reduce_qk<T>(A, y ? A.part_k : A.part_q, (T*)(y ? A.dk : A.dq));
  } else if (A.dg_tok != nullptr) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x + (int64_t)A.cu[0] * A.H;
    if (i >= (int64_t)A.cu[A.N] * A.H) return;
    float s = A.dg_tok[i * A.tiles];
    for (int t = 1; t < A.tiles; ++t) s += A.dg_tok[i * A.tiles + t];
    A.dg[i] = s;
  } else if ((int)blockIdx.x < A.H) {
    double a = 0.0;
    for (int64_t i = threadIdx.x; i < A.slots * A.tiles; i += kThreads)
      a += A.dg_part[(i / A.tiles) * A.VH + (int64_t)blockIdx.x * A.tiles + i % A.tiles];
    sum[threadIdx.x] = a;
    __syncthreads();
    for (int off = kThreads / 2; off >= 1; off >>= 1) {
      if ((int)threadIdx.x < off) sum[threadIdx.x] += sum[threadIdx.x + off];
      __syncthreads();
    }
    if (threadIdx.x == 0) A.dg[blockIdx.x] = (float)sum[0];
  }
}

// Value rows are taken in tiles of 128 where they divide into them, else 64.
int lin_tile(int dv) { return dv % 128 == 0 ? 128 : 64; }

// Rows of a segment: whole sequences when the (sequence, head) pairs alone
// fill the card, else enough segments for that, down to single chunks (with
// two chunks at least, 4 heads of 512 tokens took 25 us forward and 53 backward
// instead of 21 and 40, ragged fp32 prompts 64 instead of 53).  The
// scan's workgroups fit a compute unit twice, with fp32 tiles of 128 key
// channels once (8 heads of 128 x 128, 6000 fp32 tokens: 106 us forward and
// 328 backward with 256 units, 119 and 374 with 512; 16 bf16 heads, 32k
// tokens: 239 with 256, 231 with 512).  In the backward the dq and state
// passes fit twice and the reverse passes, but for bf16 heads of 64 x 64, once:
// with 256 units and 512, 8 ragged bf16 heads of 64 x 128 take 102 and 99 us, 16
// of 64 x 64 193 and 180, 8 of 128 x 192 508 and 426, but 16 of 128 x 128 400
// and 421, and 8 fp32 heads of 64 x 128 183 and 198.
int64_t lin_units(const gdn_lin_t& s) { return s.io_dtype == GDN_F32 && s.dk == 128 ? 256 : 512; }
// Forward calls of up to four chunks stay whole: one kernel instead of three
// (130 tokens 12 us instead of 16.5, 192: 16.5 and 20, 256: 20 either way).
// The backward's chain a chunk is longer: 256 tokens take 65 us whole and 38
// in segments.
constexpr int64_t kLinWhole = 256;
int lin_seglen(const gdn_lin_t& s, bool bwd) {
  const int64_t VH = (int64_t)s.n_heads * (s.dv / lin_tile(s.dv));
  const int64_t units = lin_units(s);
  const int64_t whole = (s.total_tokens / kChunk + 1) * kChunk;
  if ((int64_t)s.n_seqs * VH >= units || (!bwd && s.total_tokens <= kLinWhole)) return (int)whole;
  int64_t len = (s.total_tokens * VH + units - 1) / units;
  len = len < kChunk ? kChunk : (len + kChunk - 1) / kChunk * kChunk;
  return (int)(len < whole ? len : whole);
}

struct LinLayout {
  int tw, tiles, VH, R, seglen;
  int64_t slots;       // segments at most
  bool split;          // more than one segment a sequence can occur
  int32_t* status;
  float* segF;
  float* decF;
  float* segR;
  float* decR;
  float* dump;
  float* rdot;
  float* dgt;
  double* dgp;
  float* part_q;
  float* part_k;
  size_t bytes;
};

LinLayout lin_layout(const gdn_lin_t& s, void* ws, bool bwd) {
  LinLayout L{};
  L.tw = lin_tile(s.dv);
  L.tiles = s.dv / L.tw;
  L.VH = s.n_heads * L.tiles;
  L.R = L.VH / s.qk_heads;
  L.seglen = lin_seglen(s, bwd);
  L.slots = s.total_tokens / L.seglen + s.n_seqs;
  L.split = s.total_tokens > L.seglen;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += (n + 255) & ~(size_t)255;
    return ws != nullptr ? (char*)ws + here : nullptr;
  };
  const size_t heads = (size_t)L.slots * L.VH, state = (size_t)L.tw * s.dk * 4;
  L.status = (int32_t*)take(kStatusBytes);
  if (L.split) {
    L.segF = (float*)take(heads * state);
    L.decF = (float*)take(heads * 4);
  }
  if (bwd) {
    if (L.split) {
      L.segR = (float*)take(heads * state);
      L.decR = (float*)take(heads * 4);
    }
    L.dump = (float*)take((size_t)(s.total_tokens / kChunk) * L.VH * state);
    L.rdot = (float*)take((size_t)s.total_tokens * L.VH * 4);
    if (s.gate_per_token && L.tiles > 1) L.dgt = (float*)take((size_t)s.total_tokens * L.VH * 4);
    if (!s.gate_per_token) L.dgp = (double*)take(heads * 8);
    if (L.R > 1) {
      L.part_q = (float*)take((size_t)s.total_tokens * L.VH * s.dk * 4);
      L.part_k = (float*)take((size_t)s.total_tokens * L.VH * s.dk * 4);
    }
  }
  L.bytes = at;
  return L;
}

struct Operand {
  const void* p;
  int stride, div;
};

hipError_t run_scan(const gdn_lin_t& s, const LinScan& A, LinMode m, const LinLayout& L, hipStream_t stream) {
  return s.io_dtype == GDN_BF16 ? launch_lin_scan_bf16(A, m, L.slots, stream)
                                : launch_lin_scan_f32(A, m, L.slots, stream);
}

LinScan lin_base(const gdn_lin_t& s, const LinLayout& L, const float* g, const int32_t* cu) {
  LinScan A{};
  A.g = g;
  A.cu = cu;
  A.g_row = s.gate_per_token ? s.n_heads : 0;
  A.VH = L.VH;
  A.tiles = L.tiles;
  A.dk = s.dk;
  A.tw = L.tw;
  A.N = s.n_seqs;
  A.seglen = L.seglen;
  A.T = s.total_tokens;
  return A;
}

void set_q(LinScan& A, const Operand& o) { A.Q = o.p; A.qs = o.stride; A.qd = o.div; }
void set_k(LinScan& A, const Operand& o) { A.K = o.p; A.ks = o.stride; A.kd = o.div; }
void set_v(LinScan& A, const Operand& o) { A.V = o.p; A.vs = o.stride; A.vd = o.div; }
void set_e(LinScan& A, const Operand& o) { A.E = o.p; A.es = o.stride; A.ed = o.div; }

// dirs: forward alone, or both
void starts(const gdn_lin_t& s, const LinLayout& L, const LinStarts& F, const LinStarts& R, int dirs,
            const int32_t* cu, hipStream_t stream) {
  const int st4 = L.tw * s.dk / 4;
  const dim3 grid((unsigned)(((int64_t)L.VH * st4 + kThreads - 1) / kThreads), s.n_seqs, dirs);
  hipLaunchKernelGGL(lin_starts_kernel, grid, dim3(kThreads), 0, stream, F, R, cu, s.n_seqs, s.total_tokens,
                     L.seglen, L.VH, st4);
}

}  // namespace

bool lin_fits(const gdn_lin_t& s, bool bwd) {
  const LinLayout L = lin_layout(s, nullptr, bwd);
  const int64_t scan = L.slots * L.VH * 4 * (bwd ? s.dk + L.tw : L.tw);
  const int64_t sums = s.total_tokens * (L.R > 1 ? (int64_t)s.qk_heads * (s.dk / 4) : 0);
  const int64_t dg = s.total_tokens * (L.tiles > 1 ? s.n_heads : 0);
  const int64_t most = (int64_t)1 << 32;
  return scan < most && (!bwd || (sums + kThreads < most && dg + kThreads < most));
}
size_t lin_fwd_workspace_bytes(const gdn_lin_t& s) { return lin_layout(s, nullptr, false).bytes; }
size_t lin_bwd_workspace_bytes(const gdn_lin_t& s) { return lin_layout(s, nullptr, true).bytes; }

#define GDN_TRY(x)                       \
  do {                                   \
    const hipError_t e_ = (x);           \
    if (e_ != hipSuccess) return e_;     \
  } while (0)

hipError_t launch_lin_fwd(const gdn_lin_t& s, const void* q, const void* k, const void* v, const float* g,
                          const int32_t* cu_seqlens, const float* initial_state, void* o, float* final_state,
                          void* workspace, hipStream_t stream) {
  const LinLayout L = lin_layout(s, workspace, false);
  const int qk = s.qk_heads * s.dk, vv = s.n_heads * s.dv;
  const Operand oq{q, qk, L.R}, ok{k, qk, L.R}, ov{v, vv, 1};
  LinScan A = lin_base(s, L, g, cu_seqlens);
  set_k(A, ok);
  set_v(A, ov);
  A.status = L.status;
  if (L.split) {
    A.seg = L.segF;
    A.seg_decay = L.decF;
    GDN_TRY(run_scan(s, A, kLinStF, L, stream));
    starts(s, L, {L.segF, L.decF, initial_state}, {}, 1, cu_seqlens, stream);
    A.status = nullptr;
  }
  set_q(A, oq);
  A.first = initial_state;
  A.last = final_state;
  A.out = o;
  A.os = vv;
  return run_scan(s, A, kLinO, L, stream);
}

hipError_t launch_lin_bwd(const gdn_lin_t& s, const void* q, const void* k, const void* v, const float* g,
                          const int32_t* cu_seqlens, const void* d_o, const float* initial_state,
                          const float* d_final_state, void* dq, void* dk, void* d_v, float* dg,
                          float* d_initial_state, void* workspace, hipStream_t stream) {
  const LinLayout L = lin_layout(s, workspace, true);
  const int qk = s.qk_heads * s.dk, vv = s.n_heads * s.dv;
  const Operand oq{q, qk, L.R}, ok{k, qk, L.R}, ov{v, vv, 1}, od{d_o, vv, 1};
  LinScan B = lin_base(s, L, g, cu_seqlens);
  B.status = L.status;
  if (L.split) {
    LinScan A = B, R = B;
    set_k(A, ok);
    set_v(A, ov);
    A.seg = L.segF;
    A.seg_decay = L.decF;
    set_k(R, oq);
    set_v(R, od);
    R.status = nullptr;
    R.seg = L.segR;
    R.seg_decay = L.decR;
    GDN_TRY(s.io_dtype == GDN_BF16 ? launch_lin_sums_bf16(A, R, L.slots, stream)
                                   : launch_lin_sums_f32(A, R, L.slots, stream));
    B.status = nullptr;
    starts(s, L, {L.segF, L.decF, initial_state}, {L.segR, L.decR, d_final_state}, 2, cu_seqlens, stream);
  }
  const bool sum = L.R > 1;
  const int qrow = sum ? L.VH * s.dk : qk;
  {
    LinScan A = B;   // dq = forward pass of (do, v, k)
    set_q(A, od);
    set_k(A, ov);
    set_v(A, ok);
    set_e(A, oq);
    A.seg = L.segF;
    A.first = initial_state;
    A.dump = L.dump;
    A.rdot = L.rdot;
    A.out = sum ? (void*)L.part_q : dq;
    A.os = qrow;
    A.out_f32 = sum;
    GDN_TRY(run_scan(s, A, kLinDQ, L, stream));
    B.status = nullptr;
  }
  LinScan V = B;     // dv = reverse pass of (k, q, do)
  set_q(V, ok);
  set_k(V, oq);
  set_v(V, od);
  V.seg = L.segR;
  V.first = d_final_state;
  V.last = d_initial_state;
  V.out = d_v;
  V.os = vv;
  LinScan K = B;     // dk = reverse pass of (v, do, q)
  set_q(K, ov);
  set_k(K, od);
  set_v(K, oq);
  set_e(K, ok);
  K.seg = L.segR;
  K.first = d_final_state;
  K.dump = L.dump;
  K.seg_in = L.segF;
  K.first_in = initial_state;
  K.rdot = L.rdot;
  K.out = sum ? (void*)L.part_k : dk;
  K.os = qrow;
  K.out_f32 = sum;
  if (s.gate_per_token) K.dg_tok = L.tiles > 1 ? L.dgt : dg;
  else K.dg_part = L.dgp;
  GDN_TRY(s.io_dtype == GDN_BF16 ? launch_lin_rev_bf16(K, V, L.slots, stream)
                                 : launch_lin_rev_f32(K, V, L.slots, stream));
  const bool qk_sum = sum && s.total_tokens > 0;
  const bool dg_sum = !s.gate_per_token || (L.tiles > 1 && s.total_tokens > 0);
  if (qk_sum || dg_sum) {
    LinReduce A{};
    A.part_q = L.part_q; A.part_k = L.part_k; A.dq = dq; A.dk = dk;
    A.dg_tok = L.dgt; A.dg_part = L.dgp; A.dg = dg;
    A.cu = cu_seqlens; A.status = L.status;
    A.slots = L.slots;
    A.N = s.n_seqs; A.R = L.R; A.d4 = s.dk / 4; A.row4 = (int64_t)s.qk_heads * A.d4;
    A.H = s.n_heads; A.VH = L.VH; A.tiles = L.tiles;
    A.y0 = qk_sum ? 0 : 2;
    auto blocks = [](int64_t n) { return (n + kThreads - 1) / kThreads; };
    const int64_t bq = qk_sum ? blocks(s.total_tokens * A.row4) : 0;
    const int64_t bg = !dg_sum ? 0 : s.gate_per_token ? blocks(s.total_tokens * s.n_heads) : s.n_heads;
    const dim3 grid((unsigned)(bq > bg ? bq : bg), (qk_sum ? 2 : 0) + (dg_sum ? 1 : 0));
    hipLaunchKernelGGL(s.io_dtype == GDN_BF16 ? lin_reduce_kernel<uint16_t> : lin_reduce_kernel<float>, grid,
                       dim3(kThreads), 0, stream, A);
  }
  return hipGetLastError();
}

}  // namespace gdn
