// gdn_lin.hpp -- arguments and host entry of the linear-attention scan kernels.
#pragma once

#include "gdn_launch.hpp"

namespace gdn {

// The passes of the scan (see gdn_lin_scan.hpp); kLinStR runs with kLinStF, kLinDV with kLinDK.
enum LinMode : int { kLinO = 0, kLinStF = 1, kLinDQ = 2, kLinStR = 3, kLinDV = 4, kLinDK = 5 };

struct LinScan {
  const void* Q;          // rows of the output side of a pair (null: state only)
  const void* K;          // rows contracted with Q and, transposed, with V into the state
  const void* V;
  const void* E;          // DQ: q, DK: k -- the rows the outputs' state part is dotted with
  void* out;
  const float* g;
  const int32_t* cu;
  const float* first;     // state at the pass's start of a sequence (null: zero)
  float* last;            // state at its end (null: not wanted)
  float* seg;             // [slot][VH][tw][dk]: state at the pass's start of a segment, or (state
                          // passes) the segment's own sum; null: one segment a sequence
  float* seg_decay;       // state passes: e^(sum of g) of each (slot, head)
  float* dump;            // DQ writes, DK reads: raw accumulators after each chunk but a segment's last
  const float* seg_in;    // DK: seg and first of the DQ pass
  const float* first_in;
  float* rdot;            // [T][VH]: DQ writes, DK reads: q_i . (state part of dq_i)
  float* dg_tok;          // DK: [T][VH], or null
  double* dg_part;        // DK: [slot][VH] sums over the segment's tokens, or null
  int32_t* status;        // written by the first kernel of a call, read by its reduction
  int qs, ks, vs, es, os; // row strides (elements)
  int qd, kd, vd, ed;     // head of operand X = virtual head / xd
  int64_t g_row;          // gate row stride: n_heads, or 0
  int VH, tiles, dk, tw;
  int N, seglen;
  int64_t T;
  int out_f32;            // out is an fp32 partial
};

hipError_t launch_lin_scan_bf16(const LinScan& A, LinMode mode, int64_t slots, hipStream_t stream);
hipError_t launch_lin_scan_f32(const LinScan& A, LinMode mode, int64_t slots, hipStream_t stream);
// The state passes of the backward together: A forward, B reverse.
hipError_t launch_lin_sums_bf16(const LinScan& A, const LinScan& B, int64_t slots, hipStream_t stream);
hipError_t launch_lin_sums_f32(const LinScan& A, const LinScan& B, int64_t slots, hipStream_t stream);
// The reverse passes together: A the dk pass, B the dv pass.
hipError_t launch_lin_rev_bf16(const LinScan& A, const LinScan& B, int64_t slots, hipStream_t stream);
hipError_t launch_lin_rev_f32(const LinScan& A, const LinScan& B, int64_t slots, hipStream_t stream);

}  // namespace gdn
