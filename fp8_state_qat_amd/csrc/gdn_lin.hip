// gdn_lin.hip -- host side of linear attention: segment length, workspace,
// the order of the scan passes, and the small kernels between them.
#include "gdn_lin_scan.hpp"

namespace gdn {

namespace {

// Segment sums to segment starts: seg[s] holds the segment's own sum and
// becomes the state at its start (forward: before the first token; reverse:
// after the last), cur <- e^(its decays) cur + sum.  One thread per four
// state values, blockIdx.y: sequence.
template <bool kRev>
__global__ __launch_bounds__(kThreads) void lin_starts_kernel(float* __restrict__ seg,
                                                              const float* __restrict__ decay,
                                                              const float* __restrict__ first,
                                                              const int32_t* __restrict__ cu, int N, int64_t T,
                                                              int seglen, int VH, int st4) {
  const LinSeg q = lin_find(cu, N, T, seglen, blockIdx.y, true);
  if (q.bad) return;
  const int i = blockIdx.x * kThreads + threadIdx.x;
  const int vh = i / st4, e = i % st4;
  if (vh >= VH) return;
  float4* S = reinterpret_cast<float4*>(seg);
  float4 cur = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (first != nullptr) cur = reinterpret_cast<const float4*>(first)[((int64_t)q.n * VH + vh) * st4 + e];
  auto at = [&](int j) { return (int64_t)(q.slot0 + (kRev ? q.nseg - 1 - j : j)) * VH + vh; };
  constexpr int kAhead = 4;
  float4 own[kAhead];
  float dec[kAhead];
  for (int j0 = 0; j0 < q.nseg; j0 += kAhead) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (j0 + k < q.nseg - 1) {   // the last segment of the walk has no sum
        own[k] = S[at(j0 + k) * st4 + e];
        dec[k] = decay[at(j0 + k)];
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

// Sums of the R virtual heads that share a query/key head, in fp32 and in
// order, for dq (blockIdx.y 0) and dk (1): four values a thread, rows
// [cu[0], cu[N]) only.
template <typename T>
__global__ __launch_bounds__(kThreads) void lin_reduce_qk_kernel(const float* __restrict__ part_q,
                                                                 const float* __restrict__ part_k,
                                                                 T* __restrict__ dq, T* __restrict__ dk,
                                                                 const int32_t* __restrict__ cu,
                                                                 const int32_t* __restrict__ status, int N, int R,
                                                                 int d4, int64_t row4) {
  if (*status != 0) return;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x + (int64_t)cu[0] * row4;
  if (i >= (int64_t)cu[N] * row4) return;
  const int64_t head = i / d4;             // row * qk_heads + head
  const float4* p = reinterpret_cast<const float4*>(blockIdx.y ? part_k : part_q) + head * R * d4 + i % d4;
  float4 s = p[0];
  for (int r = 1; r < R; ++r) {
    const float4 x = p[(int64_t)r * d4];
    s.x += x.x;
    s.y += x.y;
    s.z += x.z;
    s.w += x.w;
  }
  T* out = (blockIdx.y ? dk : dq) + 4 * i;
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  else
    *reinterpret_cast<float4*>(out) = s;
}

// dg of a token's head from the tiles of its value rows.
__global__ __launch_bounds__(kThreads) void lin_reduce_dg_kernel(const float* __restrict__ part,
                                                                 float* __restrict__ dg,
                                                                 const int32_t* __restrict__ cu,
                                                                 const int32_t* __restrict__ status, int N, int H,
                                                                 int tiles) {
  if (*status != 0) return;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x + (int64_t)cu[0] * H;
  if (i >= (int64_t)cu[N] * H) return;
  float s = part[i * tiles];
  for (int t = 1; t < tiles; ++t) s += part[i * tiles + t];
  dg[i] = s;
}

// dg of a head's fixed decay: the segments' sums in fp64, one workgroup a head.
__global__ __launch_bounds__(kThreads) void lin_reduce_dg_head_kernel(const double* __restrict__ part,
                                                                      float* __restrict__ dg,
                                                                      const int32_t* __restrict__ status,
                                                                      int64_t slots, int VH, int tiles) {
  __shared__ double s[kThreads];
  if (*status != 0) return;
  double a = 0.0;
  for (int64_t i = threadIdx.x; i < slots * tiles; i += kThreads)
    a += part[(i / tiles) * VH + (int64_t)blockIdx.x * tiles + i % tiles];
  s[threadIdx.x] = a;
  __syncthreads();
  for (int off = kThreads / 2; off >= 1; off >>= 1) {
    if ((int)threadIdx.x < off) s[threadIdx.x] += s[threadIdx.x + off];
    __syncthreads();
  }
  if (threadIdx.x == 0) dg[blockIdx.x] = (float)s[0];
}

// Value rows are taken in tiles of 128 where they divide into them, else 64.
int lin_tile(int dv) { return dv % 128 == 0 ? 128 : 64; }

// Rows of a segment: whole sequences when the (sequence, head) pairs alone
// fill the card, else enough segments for that, of at least 128 rows.  The
// scan's workgroups fit a compute unit twice, with fp32 tiles of 128 key
// channels once (8 heads of 128 x 128, 6000 fp32 tokens: 106 us forward and
// 328 backward with 256 units, 119 and 374 with 512; 16 bf16 heads, 32k
// tokens: 239 with 256, 231 with 512).
int64_t lin_units(const gdn_lin_t& s) { return s.io_dtype == GDN_F32 && s.dk == 128 ? 256 : 512; }
constexpr int64_t kLinMinSeg = 128;
int lin_seglen(const gdn_lin_t& s) {
  const int64_t VH = (int64_t)s.n_heads * (s.dv / lin_tile(s.dv));
  const int64_t units = lin_units(s);
  const int64_t whole = (s.total_tokens / kChunk + 1) * kChunk;
  if ((int64_t)s.n_seqs * VH >= units) return (int)whole;
  int64_t len = (s.total_tokens * VH + units - 1) / units;
  if (len < kLinMinSeg) len = kLinMinSeg;
  len = (len + kChunk - 1) / kChunk * kChunk;
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
  L.seglen = lin_seglen(s);
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
    const size_t groups = (size_t)(s.total_tokens / (kAnchor * kChunk) + L.slots);
    L.dump = (float*)take(groups * L.VH * state);
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

void starts(const gdn_lin_t& s, const LinLayout& L, float* seg, const float* dec, const float* first,
            const int32_t* cu, bool rev, hipStream_t stream) {
  const int st4 = L.tw * s.dk / 4;
  const dim3 grid((unsigned)(((int64_t)L.VH * st4 + kThreads - 1) / kThreads), s.n_seqs);
  hipLaunchKernelGGL(rev ? lin_starts_kernel<true> : lin_starts_kernel<false>, grid, dim3(kThreads), 0, stream, seg,
                     dec, first, cu, s.n_seqs, s.total_tokens, L.seglen, L.VH, st4);
}

}  // namespace

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
    starts(s, L, L.segF, L.decF, initial_state, cu_seqlens, false, stream);
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
    LinScan A = B;
    set_k(A, ok);
    set_v(A, ov);
    A.seg = L.segF;
    A.seg_decay = L.decF;
    GDN_TRY(run_scan(s, A, kLinStF, L, stream));
    A.status = B.status = nullptr;
    set_k(A, oq);
    set_v(A, od);
    A.seg = L.segR;
    A.seg_decay = L.decR;
    GDN_TRY(run_scan(s, A, kLinStR, L, stream));
    starts(s, L, L.segF, L.decF, initial_state, cu_seqlens, false, stream);
    starts(s, L, L.segR, L.decR, d_final_state, cu_seqlens, true, stream);
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
  K.rdot = L.rdot;
  K.out = sum ? (void*)L.part_k : dk;
  K.os = qrow;
  K.out_f32 = sum;
  if (s.gate_per_token) K.dg_tok = L.tiles > 1 ? L.dgt : dg;
  else K.dg_part = L.dgp;
  GDN_TRY(s.io_dtype == GDN_BF16 ? launch_lin_rev_bf16(K, V, L.slots, stream)
                                 : launch_lin_rev_f32(K, V, L.slots, stream));
  if (sum && s.total_tokens > 0) {
    const int d4 = s.dk / 4;
    const int64_t row4 = (int64_t)s.qk_heads * d4;
    const dim3 grid((unsigned)((s.total_tokens * row4 + kThreads - 1) / kThreads), 2);
    if (s.io_dtype == GDN_BF16)
      hipLaunchKernelGGL(lin_reduce_qk_kernel<uint16_t>, grid, dim3(kThreads), 0, stream, L.part_q, L.part_k,
                         (uint16_t*)dq, (uint16_t*)dk, cu_seqlens, L.status, s.n_seqs, L.R, d4, row4);
    else
      hipLaunchKernelGGL(lin_reduce_qk_kernel<float>, grid, dim3(kThreads), 0, stream, L.part_q, L.part_k,
                         (float*)dq, (float*)dk, cu_seqlens, L.status, s.n_seqs, L.R, d4, row4);
  }
  if (!s.gate_per_token)
    hipLaunchKernelGGL(lin_reduce_dg_head_kernel, dim3(s.n_heads), dim3(kThreads), 0, stream, L.dgp, dg, L.status,
                       L.slots, L.VH, L.tiles);
  else if (L.tiles > 1 && s.total_tokens > 0)
    hipLaunchKernelGGL(lin_reduce_dg_kernel, dim3((unsigned)((s.total_tokens * s.n_heads + kThreads - 1) / kThreads)),
                       dim3(kThreads), 0, stream, L.dgt, dg, cu_seqlens, L.status, s.n_seqs, s.n_heads, L.tiles);
  return hipGetLastError();
}

}  // namespace gdn
