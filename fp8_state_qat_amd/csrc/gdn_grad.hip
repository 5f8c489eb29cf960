// gdn_grad.hip -- host side of the gated delta rule's gradients: the workspace
// and the launches (mathematics in gdn_grad.hpp, kernels in
// gdn_grad_kernels.hpp).
//
// Workspace: the status word and the chunk offsets (as in gdn_chunk_fwd's),
// one record for each (chunk, head), the gradients of the states after every
// chunk, the tokens' errors and their gradients, and without given states those
// entering every chunk.  With the state's QDQ in the chunks and no given states,
// the forward runs again, its own code with the boundary record, so that the
// gradients are taken at the very states it had.  Its workspace is then the first
// part, with the status word and the offsets that the whole call uses (what it
// finds on the device is the call's), and its outputs and last states the last.
#include "gdn_grad.hpp"

namespace gdn {

namespace {

struct GradLayout {
  size_t rec, R, E, Y, S, o, fin, bytes;
  int64_t chunks, items;
  bool again;   // the forward runs again
};

size_t pad256(size_t x) { return (x + 255) / 256 * 256; }

// The forward as the call runs it again.
gdn_shape_t again(const gdn_shape_t& s) {
  gdn_shape_t f = s;
  f.o_dtype = s.io_dtype;
  return f;
}

GradLayout grad_layout(const gdn_shape_t& s, bool given) {
  GradLayout l{};
  l.chunks = (s.total_tokens + kChunk - 1) / kChunk + s.n_seqs;
  l.items = l.chunks * s.n_heads;
  const size_t rec = s.io_dtype == GDN_BF16 ? GradRec<EngBF16>::kBytes : GradRec<EngF32>::kBytes;
  const size_t states = (size_t)l.items * s.dv * s.dk * 4;
  l.again = !given && (s.qdq_flags & GDN_QDQ_CHUNK);
  l.rec = l.again ? pad256(prep_workspace_bytes(again(s))) : kStatusBytes + pad256((size_t)(s.n_seqs + 2) * 4);
  l.R = l.rec + pad256((size_t)l.items * rec);
  l.E = l.R + states;
  l.Y = l.E + (size_t)l.items * s.dv * kChunk * 4;
  l.S = l.Y + (size_t)l.items * s.dv * kChunk * 4;
  l.o = l.S + (given ? 0 : states);
  l.bytes = l.o;
  if (l.again) {
    l.fin = l.o + pad256((size_t)s.total_tokens * s.n_heads * s.dv * (s.io_dtype == GDN_BF16 ? 2 : 4));
    l.bytes = l.fin + pad256((size_t)s.n_seqs * s.n_heads * s.dv * s.dk * 4);
  }
  return l;
}

}  // namespace

bool grad_fits(const gdn_shape_t& s) {
  const int64_t chunks = (s.total_tokens + kChunk - 1) / kChunk + s.n_seqs;
  return chunks * s.n_heads < ((int64_t)1 << 32) / 512 &&
         (int64_t)s.n_seqs * s.n_heads * (s.dv / 64) < ((int64_t)1 << 32) / (4 * kThreads);   // two directions, 512 threads
}

size_t grad_workspace_bytes(const gdn_shape_t& s, bool given) { return grad_layout(s, given).bytes; }

hipError_t launch_chunk_grad(const gdn_shape_t& s, const void* q, const void* k, const void* v, const float* beta,
                             const float* g, const int32_t* cu_seqlens, const int32_t* seq_lens,
                             const float* initial_state, const float* states, int64_t n_states, const void* d_o,
                             const float* d_final_state, void* dq, void* dk, void* d_v, float* d_beta, float* dg,
                             float* d_initial_state, void* workspace, hipStream_t stream) {
  const GradLayout l = grad_layout(s, states != nullptr);
  char* w = reinterpret_cast<char*>(workspace);
  PrepLayout L{};
  L.status = reinterpret_cast<int32_t*>(w);
  L.offs = reinterpret_cast<int32_t*>(w + kStatusBytes);
  L.items = l.items;
  hipError_t e;
  if (l.again) {
    gdn_debug_t d{};
    d.bound_offsets = L.offs;
    d.bound_post = reinterpret_cast<float*>(w + l.S);
    e = launch_chunk_fwd(again(s), q, k, v, beta, g, cu_seqlens, seq_lens, nullptr, initial_state, w + l.o,
                         reinterpret_cast<float*>(w + l.fin), w, &d, stream);
    states = d.bound_post;
    n_states = l.chunks;
  } else {
    e = launch_prep(s, q, k, beta, g, cu_seqlens, seq_lens, nullptr, L, false, nullptr, nullptr, stream);
  }
  if (e != hipSuccess) return e;
  GradArgs a{};
  a.q = q; a.k = k; a.v = v; a.d_o = d_o;
  a.beta = beta; a.g = g;
  a.cu = cu_seqlens; a.seq_lens = seq_lens; a.offs = L.offs; a.status = L.status;
  a.init = initial_state;
  a.kept = states;
  a.n_kept = n_states;
  a.d_fin = d_final_state;
  a.rec = w + l.rec;
  a.S = states == nullptr ? reinterpret_cast<float*>(w + l.S) : nullptr;
  a.R = reinterpret_cast<float*>(w + l.R);
  a.E = reinterpret_cast<float*>(w + l.E);
  a.Y = reinterpret_cast<float*>(w + l.Y);
  a.dq = dq; a.dk = dk; a.d_v = d_v;
  a.d_beta = d_beta; a.dg = dg; a.d_init = d_initial_state;
  a.N = s.n_seqs; a.H = s.n_heads; a.dv = s.dv;
  return s.io_dtype == GDN_BF16 ? launch_grad_bf16(s, a, l.items, stream) : launch_grad_f32(s, a, l.items, stream);
}

}  // namespace gdn
