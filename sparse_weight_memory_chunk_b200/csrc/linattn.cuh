// linattn.cuh -- shared declarations of the linear-attention kernels (not part of the ABI).
#pragma once

#include "fwpkm_internal.cuh"

namespace fwpkm {

// One pass of the recurrence over every (sequence, head):
//   S_t = a S_{t-1} + k_t v_t^T,   o_t = out_scale S_t^T q_t      (t ascending, or descending)
// with q, k of width d and v, o of width dv.  The forward pass and all three gradients are
// this pass with other operands (see linattn.cu).
struct ScanArgs {
  fwpkm_heads q, k, v, o;
  const float* log_decay;  // [H]
  const int32_t* lens;     // [B] or null
  int B, H, T, d, dv;
  int reverse;
  float out_scale;
  // State in and out: element (i, j) of (b, h) at s[(b H + h) d dv + i si + j sj].  in_ready:
  // the first token adds to s_in as it is (else to a s_in).  out_decay: s_out is a S_last
  // instead of S_last.  in_scale multiplies s_in, st_scale s_out.
  const float* s_in;
  float* s_out;
  long long si, sj;
  float in_scale, st_scale;
  int in_ready, out_decay;
  // Segments of seg_len tokens, each from its own start state (nseg > 1): slots [B H][nseg]
  // of d x dv (row-major) in the workspace.
  int nseg, seg_len;
  float* slots;
};

// a^e in fp32 from a log decay (a^0 = 1 for every a).
__device__ __forceinline__ float decay_pow(float log_decay, float e) { return e == 0.f ? 1.f : expf(log_decay * e); }
// a^e in two fp32 parts, whose sum is exact to 2^-48: for a state that is multiplied by it again and again,
// so that the rounding of one part does not compound.
__device__ __forceinline__ float2 decay_parts(float log_decay, int e) {
  const double w = e == 0 ? 1.0 : exp((double)log_decay * e);
  const float hi = (float)w;
  return make_float2(hi, (float)(w - (double)hi));
}

// Length of sequence b.
__device__ __forceinline__ int scan_len(const ScanArgs& a, int b) {
  if (!a.lens) return a.T;
  const int n = a.lens[b];
  return n < 0 ? 0 : n > a.T ? a.T : n;
}

// Tensor-core pass (linattn_tc.cu): whether it takes passes of this shape, and this pass (its
// pointers and strides too); the launch (the number of kernels, or < 0 on a CUDA error); the
// status its kernels latched since the last call (a DEV_* value, cleared; < 0: CUDA error).
bool scan_tc_shape(const ScanArgs& a, int dtype);
bool scan_tc_takes(const ScanArgs& a, int dtype);
int scan_tc_segments(const ScanArgs& a);
int launch_scan_tc(const ScanArgs& a, cudaStream_t s);
int take_scan_status();
int launch_scan_combine(const ScanArgs& a, cudaStream_t s);

}  // namespace fwpkm
