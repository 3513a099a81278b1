// linattn.cu -- linear attention with a decay for each head: the dense fast-weight memory
// beside the sparse one.
//
// Per sequence and head, with decay a = exp(log_decay[head]) and state S [d][d_v]:
//   S_t = a S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t.
// Gradients (D_t = dL/dS_t, D after the last token = dL/dS_T):
//   dq_t = scale S_t do_t,   D_t = a D_{t+1} + scale q_t do_t^T  (the last token: + dS_T, undecayed),
//   dk_t = D_t v_t,   dv_t = D_t^T k_t,   dS_0 = a D_first.
// Each of them is the same pass with other operands: dq is the pass (q: do, k: v, v: k) from
// S_0^T; dk the descending pass (q: v, k: do, v: q) from dS_T^T; dv the descending pass
// (q: k, k: q, v: do) from dS_T.  So one kernel serves prompts, single tokens and training.
//
// This file holds the CUDA-core pass, for every type, width up to 256, stride, alignment and
// length, and the entry points; linattn_tc.cu the tensor-core pass for bf16 prompts.
//
// The CUDA-core pass keeps S in fp32 registers: a CTA of 256 threads owns up to 128 columns
// of one head's state, thread (row group, column quad) NI x 4 of its elements, and takes the
// tokens of a batch in order: 2 FMA per state element and token.  The next batch's rows come by
// asynchronous copies meanwhile.  Inside a batch of SC_TB tokens the state is kept relative to
// the batch's start (v_u enters as a^-u v_u, o_u leaves as a^u o_u), so the decay costs one
// multiplication per batch and its rounding does not compound over the tokens; a head whose
// a^-SC_TB would leave fp32's range takes batches of one token.  Bound: instruction issue
// (194 a warp and token at d = d_v = 128, of them 64 packed FMAs): 256 heads of 512 tokens in
// 350 us, 24.5 TFLOP/s.  (With rows staged by plain loads between two barriers the loads'
// latency bounded it: 128 such heads in 665 us, now 232.)
#include <cmath>
#include <cstdio>
#include <initializer_list>

#include "linattn.cuh"
#include "sm100.cuh"

namespace fwpkm {
namespace {

constexpr int SC_THREADS = 256;
constexpr int SC_WARPS = SC_THREADS / 32;
constexpr int SC_TB = 8;         // tokens per batch
constexpr int SC_STEP = 16;      // tokens that the kernel for a few of them takes at most
constexpr int SC_MAX_D = 256;    // rows of the state at most
constexpr int SC_SEGS = 2 * 148; // CTAs that the GPU holds at once, and segments of a pass at most
constexpr int SC_SPLIT = 256;    // tokens from which a prompt is split
constexpr int SC_SEG_MIN = 64;   // tokens per segment at least
constexpr float SC_RANGE = 40.f; // largest |log a^SC_TB| kept relative to the batch

__device__ __forceinline__ float sc_f(float x) { return x; }
__device__ __forceinline__ float sc_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void sc_put(float* p, float x) { *p = x; }
__device__ __forceinline__ void sc_put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename T>
__device__ __forceinline__ const T* head_row(const fwpkm_heads& x, int b, int h) {
  return (const T*)x.p + (long long)b * x.sb + (long long)h * x.sh;
}

// One row of `bytes` bytes into shared memory by a warp, in units of 16 or 4 bytes without waiting
// (both ends on that grid; a last unit may be shorter), or of 2 bytes where a row of bf16 is on no
// such grid.
__device__ __forceinline__ void copy_row(uint32_t dst, const char* src, int bytes, int unit, int lane) {
  if (unit == 16) {
    for (int o = lane * 16; o < bytes; o += 512)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + o), "l"(src + o), "r"(min(16, bytes - o))
                   : "memory");
  } else if (unit == 4) {
    for (int o = lane * 4; o < bytes; o += 128)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + o), "l"(src + o), "r"(min(4, bytes - o))
                   : "memory");
  } else {
    unsigned short x[SC_MAX_D / 32];
#pragma unroll
    for (int i = 0; i < SC_MAX_D / 32; ++i) {
      const int o = (i * 32 + lane) * 2;
      x[i] = o < bytes ? __ldg(reinterpret_cast<const unsigned short*>(src + o)) : (unsigned short)0;
    }
#pragma unroll
    for (int i = 0; i < SC_MAX_D / 32; ++i) {
      const int o = (i * 32 + lane) * 2;
      if (o < bytes) asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst + o), "h"(x[i]) : "memory");
    }
  }
}

// N (even) values in a row of shared memory, which start on a grid of N.
template <int N>
__device__ __forceinline__ void get_row(const float* p, float (&x)[N]) {
  constexpr int V = N % 4 == 0 ? 4 : 2;  // values per load
#pragma unroll
  for (int i = 0; i < N; i += V) {
    if (V == 4) {
      const float4 y = *reinterpret_cast<const float4*>(p + i);
      x[i] = y.x; x[i + 1] = y.y; x[(i + 2) % N] = y.z; x[(i + 3) % N] = y.w;
    } else {
      const float2 y = *reinterpret_cast<const float2*>(p + i);
      x[i] = y.x; x[i + 1] = y.y;
    }
  }
}
template <int N>
__device__ __forceinline__ void get_row(const __nv_bfloat16* p, float (&x)[N]) {
  constexpr int V = N % 8 == 0 ? 4 : N % 4 == 0 ? 2 : 1;  // words per load
#pragma unroll
  for (int i = 0; i < N; i += 2 * V) {
    uint32_t w[4];
    if (V == 4) {
      const uint4 y = *reinterpret_cast<const uint4*>(p + i);
      w[0] = y.x; w[1] = y.y; w[2] = y.z; w[3] = y.w;
    } else if (V == 2) {
      const uint2 y = *reinterpret_cast<const uint2*>(p + i);
      w[0] = y.x; w[1] = y.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(p + i);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      x[(i + 2 * j) % N] = __uint_as_float(w[j] << 16);
      x[(i + 2 * j + 1) % N] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}

// local: the segment's own state from zero into its slot, no output.  unit: bytes per copy of
// the rows of q, k and v.
template <typename T, int NI>
__global__ void __launch_bounds__(SC_THREADS, 2)
scan_kernel(ScanArgs a, int lj, int unit, int local) {
  extern __shared__ __align__(16) float sm[];
  __shared__ float s_in[SC_TB], s_out[SC_TB];        // a^-u and a^u
  pdl_wait();
  pdl_trigger();
  const int rgn = SC_THREADS / lj, dp = rgn * NI;   // row groups, padded d
  const int cols = 4 * lj, tiles = (a.dv + cols - 1) / cols;
  const int row = 2 * dp + cols;                     // k, q and v of a token
  float* sr = sm;                                    // [SC_TB][SC_WARPS][cols] partial outputs
  T* raw = reinterpret_cast<T*>(sr + SC_TB * SC_WARPS * cols);  // [2][SC_TB][row]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int jl = tid & (lj - 1), rg = tid / lj;
  const long long bh = blockIdx.x / tiles;
  const int tile = (int)(blockIdx.x - bh * tiles);
  const int b = (int)(bh / a.H), h = (int)(bh - (long long)b * a.H);
  const int g = blockIdx.y;
  const int c0 = tile * cols, j0 = c0 + 4 * jl, i0 = rg * NI;
  const int n = scan_len(a, b);
  const int t0 = min(n, g * a.seg_len), t1 = min(n, t0 + a.seg_len);
  const float ld = a.log_decay[h];
  // tokens per batch: one where a^-SC_TB would leave fp32's range
  const int tb = fabsf(ld) * (float)SC_TB <= SC_RANGE ? SC_TB : 1;
  const size_t cells = (size_t)a.d * a.dv;

  const T* qp = head_row<T>(a.q, b, h);
  const T* kp = head_row<T>(a.k, b, h);
  const T* vp = head_row<T>(a.v, b, h) + c0;
  static_assert(SC_TB == SC_WARPS, "a warp copies one token of a batch");
  // a batch's rows on their way: warp u takes token u
  auto fetch = [&](int tb0, int buf) {
    if (warp < min(tb, t1 - tb0)) {
      const long long t = a.reverse ? n - 1 - (tb0 + warp) : tb0 + warp;
      const uint32_t dst = sm100::smem_u32(raw + (buf * SC_TB + warp) * row);
      copy_row(dst, (const char*)(kp + t * a.k.st), a.d * (int)sizeof(T), unit, lane);
      if (!local) copy_row(dst + dp * (int)sizeof(T), (const char*)(qp + t * a.q.st), a.d * (int)sizeof(T), unit, lane);
      copy_row(dst + 2 * dp * (int)sizeof(T), (const char*)(vp + t * a.v.st), min(cols, a.dv - c0) * (int)sizeof(T), unit,
               lane);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // the padding of a row is zero throughout
  for (int x = tid * 16; x < 2 * SC_TB * row * (int)sizeof(T); x += SC_THREADS * 16)
    *reinterpret_cast<uint4*>(reinterpret_cast<char*>(raw) + x) = make_uint4(0u, 0u, 0u, 0u);
  if (tid < SC_TB) {
    s_in[tid] = decay_pow(-ld, (float)tid);   // (a batch of one token reads the first only)
    s_out[tid] = decay_pow(ld, (float)tid) * a.out_scale;
  }
  __syncthreads();
  fetch(t0, 0);

  // start state, decayed for the first token
  float S[NI][4];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) S[i][e] = 0.f;
  if (!local) {
    const bool slot = a.nseg > 1;
    // segment 0 starts from the copy of s_in in the last slot, segment g from slot g - 1
    const float* src = slot ? a.slots + ((size_t)bh * a.nseg + (g == 0 ? a.nseg - 1 : g - 1)) * cells
                            : (a.s_in ? a.s_in + (size_t)bh * cells : nullptr);
    if (src) {
      const long long si = slot ? a.dv : a.si, sj = slot ? 1 : a.sj;
      const float f = slot || n == 0 ? 1.f : a.in_scale;
      const bool vec = sj == 1 && (a.dv & 3) == 0 && (((uintptr_t)src) & 15) == 0;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (i0 + i < a.d) {
          if (vec) {
            if (j0 < a.dv) {
              const float4 x = *reinterpret_cast<const float4*>(src + (i0 + i) * si + j0);
              S[i][0] = x.x; S[i][1] = x.y; S[i][2] = x.z; S[i][3] = x.w;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (j0 + e < a.dv) S[i][e] = src[(i0 + i) * si + (j0 + e) * sj];
          }
        }
      }
      const float w = (t1 > t0 && !(g == 0 && a.in_ready)) ? f * decay_pow(ld, 1.f) : f;
      if (w != 1.f) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) S[i][e] *= w;
      }
    }
  }

  T* op = (T*)a.o.p + (long long)b * a.o.sb + (long long)h * a.o.sh + c0;
  const float a1 = decay_pow(ld, 1.f);
  const float2 whole = decay_parts(ld, tb);
  int buf = 0;
  for (int tb0 = t0; tb0 < t1; tb0 += tb, buf ^= 1) {
    const int m = min(tb, t1 - tb0);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    if (tb0 + tb < t1) fetch(tb0 + tb, buf ^ 1);
    const bool last = tb0 + m >= t1;
    const T* rows = raw + buf * SC_TB * row;
#pragma unroll 1
    for (int u = 0; u < m; ++u, rows += row) {
      float x[NI], v[4];
      get_row<NI>(rows + i0, x);
      get_row<4>(rows + 2 * dp + 4 * jl, v);
      const float w = s_in[u];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= w;
#pragma unroll
      for (int i = 0; i < NI; i += 2)
#pragma unroll
        for (int e = 0; e < 4; ++e) sm100::fma2(S[i][e], S[i + 1][e], x[i], x[i + 1], v[e], v[e]);
      if (!local) {
        float o[4] = {0.f, 0.f, 0.f, 0.f}, o1[4] = {0.f, 0.f, 0.f, 0.f};  // even and odd rows
        get_row<NI>(rows + dp + i0, x);
#pragma unroll
        for (int i = 0; i < NI; i += 2)
#pragma unroll
          for (int e = 0; e < 4; ++e) sm100::fma2(o[e], o1[e], x[i], x[i + 1], S[i][e], S[i + 1][e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += o1[e];
        for (int off = lj; off < 32; off <<= 1)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] += __shfl_xor_sync(0xffffffffu, o[e], off);
        if (lane < lj)
          *reinterpret_cast<float4*>(sr + (u * SC_WARPS + warp) * cols + 4 * jl) = make_float4(o[0], o[1], o[2], o[3]);
      }
    }
    // back to absolute: a^tb for the next batch's first token, a^(m-1) after the last token
    const float2 f = last ? decay_parts(ld, m - 1) : whole;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x) S[i][x] = fmaf(S[i][x], f.x, S[i][x] * f.y);
    if (!local) {
      __syncthreads();
      // warp u writes token u
      if (warp < m) {
        const long long t = a.reverse ? n - 1 - (tb0 + warp) : tb0 + warp;
        const float f = s_out[warp];
        for (int j = lane; j < cols && c0 + j < a.dv; j += 32) {
          float x = 0.f;
#pragma unroll
          for (int w = 0; w < SC_WARPS; ++w) x += sr[(warp * SC_WARPS + w) * cols + j];
          sc_put(op + t * a.o.st + j, x * f);
        }
      }
    }
  }

  // the segment's last state: its slot, or (last segment) the caller's
  float* dst = local ? a.slots + ((size_t)bh * a.nseg + g) * cells
                     : (a.s_out && g == a.nseg - 1 ? a.s_out + (size_t)bh * cells : nullptr);
  if (!dst) return;
  const long long si = local ? a.dv : a.si, sj = local ? 1 : a.sj;
  const float w = local || n == 0 ? 1.f : a.st_scale * (a.out_decay ? a1 : 1.f);
  const bool vec = sj == 1 && (a.dv & 3) == 0 && (((uintptr_t)dst) & 15) == 0;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    if (i0 + i >= a.d) continue;
    if (vec) {
      if (j0 < a.dv)
        *reinterpret_cast<float4*>(dst + (i0 + i) * si + j0) =
            make_float4(S[i][0] * w, S[i][1] * w, S[i][2] * w, S[i][3] * w);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j0 + e < a.dv) dst[(i0 + i) * si + (j0 + e) * sj] = S[i][e] * w;
    }
  }
}

// A few tokens of every sequence: bound by the state, read and written once.  The pass above
// without its batches: thread (row group, column quad) holds NI x 4 of the state, takes its rows'
// k and q straight from their row (one address per row group) and the row groups' partial
// outputs meet in shared memory.  The decay is exp in two fp32 parts, so that its rounding does
// not compound over thousands of tokens.  (The batched pass needed 1146 instructions a warp for
// one token and was bound by them: 61 us for 2048 heads of 128 x 128, 42 at the copy bandwidth.)
template <typename T, int NI>
__global__ void __launch_bounds__(SC_THREADS, 4)
step_kernel(ScanArgs a, int lj) {
  __shared__ __align__(16) float sr[2][SC_WARPS][128];
  __shared__ float sa[2];
  pdl_wait();
  pdl_trigger();
  const int cols = 4 * lj, tiles = (a.dv + cols - 1) / cols;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int jl = tid & (lj - 1), i0 = (tid / lj) * NI;
  const long long bh = blockIdx.x / tiles;
  const int c0 = (int)(blockIdx.x - bh * tiles) * cols, j0 = c0 + 4 * jl;
  const int b = (int)(bh / a.H), h = (int)(bh - (long long)b * a.H);
  const int n = scan_len(a, b);
  const size_t cells = (size_t)a.d * a.dv;
  const float* src = a.s_in + (size_t)bh * cells + (size_t)i0 * a.dv + j0;
  float4 S[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i)
    S[i] = i0 + i < a.d && j0 < a.dv ? *reinterpret_cast<const float4*>(src + (size_t)i * a.dv)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
  if (tid == 0) {
    const float2 w = decay_parts(a.log_decay[h], 1);
    sa[0] = w.x;
    sa[1] = w.y;
  }
  __syncthreads();
  const float hi = sa[0], lo = sa[1];
  const T* qp = head_row<T>(a.q, b, h) + i0;
  const T* kp = head_row<T>(a.k, b, h) + i0;
  const T* vp = head_row<T>(a.v, b, h) + j0;
  T* op = (T*)a.o.p + (long long)b * a.o.sb + (long long)h * a.o.sh;
  for (int t = 0; t < n; ++t) {
    float kk[NI], qq[NI], v[4];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      kk[i] = i0 + i < a.d ? sc_f(kp[t * a.k.st + i]) : 0.f;
      qq[i] = i0 + i < a.d ? sc_f(qp[t * a.q.st + i]) : 0.f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = j0 + e < a.dv ? sc_f(vp[t * a.v.st + e]) : 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      S[i].x = fmaf(S[i].x, hi, fmaf(S[i].x, lo, kk[i] * v[0]));
      S[i].y = fmaf(S[i].y, hi, fmaf(S[i].y, lo, kk[i] * v[1]));
      S[i].z = fmaf(S[i].z, hi, fmaf(S[i].z, lo, kk[i] * v[2]));
      S[i].w = fmaf(S[i].w, hi, fmaf(S[i].w, lo, kk[i] * v[3]));
      o.x = fmaf(qq[i], S[i].x, o.x);
      o.y = fmaf(qq[i], S[i].y, o.y);
      o.z = fmaf(qq[i], S[i].z, o.z);
      o.w = fmaf(qq[i], S[i].w, o.w);
    }
    for (int off = lj; off < 32; off <<= 1) {
      o.x += __shfl_xor_sync(0xffffffffu, o.x, off);
      o.y += __shfl_xor_sync(0xffffffffu, o.y, off);
      o.z += __shfl_xor_sync(0xffffffffu, o.z, off);
      o.w += __shfl_xor_sync(0xffffffffu, o.w, off);
    }
    float(*buf)[128] = sr[t & 1];  // two buffers: one barrier per token
    if (lane < lj) *reinterpret_cast<float4*>(&buf[warp][4 * jl]) = o;
    __syncthreads();
    if (tid < cols && c0 + tid < a.dv) {
      float x = 0.f;
#pragma unroll
      for (int w = 0; w < SC_WARPS; ++w) x += buf[w][tid];
      sc_put(op + t * a.o.st + c0 + tid, x * a.out_scale);
    }
  }
  float* dst = a.s_out + (size_t)bh * cells + (size_t)i0 * a.dv + j0;
#pragma unroll
  for (int i = 0; i < NI; ++i)
    if (i0 + i < a.d && j0 < a.dv) *reinterpret_cast<float4*>(dst + (size_t)i * a.dv) = S[i];
}

// Slots of local states -> states after each segment: E_g = a^len_g E_{g-1} + local_g, with
// E_{-1} = s_in; the last slot receives a copy of s_in (in_scale applied) for segment 0.
__global__ void __launch_bounds__(256)
scan_combine_kernel(ScanArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ float2 decay[SC_SEGS];  // a^len of every segment, in two parts
  const size_t cells = (size_t)a.d * a.dv;
  const size_t x = (size_t)blockIdx.x * 256 + threadIdx.x;
  const long long bh = blockIdx.y;
  const int b = (int)(bh / a.H), h = (int)(bh - (long long)b * a.H);
  const int n = scan_len(a, b);
  const float ld = a.log_decay[h];
  for (int g = threadIdx.x; g < a.nseg - 1; g += 256) {
    const int len = max(0, min(n - g * a.seg_len, a.seg_len));
    decay[g] = decay_parts(ld, len - (g == 0 && a.in_ready && len > 0 ? 1 : 0));
  }
  __syncthreads();
  if (x >= cells) return;
  const int i = (int)(x / a.dv), j = (int)(x - (size_t)i * a.dv);
  float* slot = a.slots + (size_t)bh * a.nseg * cells + x;
  float E = a.s_in ? a.s_in[(size_t)bh * cells + i * a.si + j * a.sj] * (n == 0 ? 1.f : a.in_scale) : 0.f;
  slot[(size_t)(a.nseg - 1) * cells] = E;
  for (int g0 = 0; g0 < a.nseg - 1; g0 += 8) {
    float loc[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) loc[u] = g0 + u < a.nseg - 1 ? slot[(size_t)(g0 + u) * cells] : 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int g = g0 + u;
      if (g >= a.nseg - 1) break;
      const float2 w = decay[g];
      E = fmaf(E, w.x, fmaf(E, w.y, loc[u]));
      slot[(size_t)g * cells] = E;
    }
  }
}

bool la_al(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
int pow2_ceil(int x) {
  int p = 1;
  while (p < x) p <<= 1;
  return p;
}

struct ScanShape {
  int lj, ni, tiles;
};
// Column quads per CTA: as wide as 16 rows per thread allow.  Narrower tiles (each re-reads q and
// k) where the heads and the segments that T allows leave half of the GPU's places empty and
// narrower ones fill them: 10 heads of 72 x 100 with 1003 tokens 91 -> 65 us, 8 of 128 x 128 with
// 100 tokens 51 -> 35; but with four rows a thread or fewer a token costs its latency, not its
// work, so there only a quarter counts (128 heads of 64 x 64, 512 tokens: 147 us wide, 172 narrow).
ScanShape scan_shape(const ScanArgs& a) {
  int lj = SC_THREADS * 16 / (pow2_ceil(a.d) < 16 ? 16 : pow2_ceil(a.d));
  if (lj > 32) lj = 32;
  const int need = pow2_ceil((a.dv + 3) / 4);
  if (lj > need) lj = need < 4 ? 4 : need;
  auto ctas = [&](int l) {  // with as many segments as fit
    const long long base = (long long)a.B * a.H * ((a.dv + 4 * l - 1) / (4 * l));
    long long n = a.T < SC_SPLIT || base > SC_SEGS / 3 ? 1 : SC_SEGS / base;
    if (n > a.T / SC_SEG_MIN) n = a.T / SC_SEG_MIN;
    return base * (n < 1 ? 1 : n);
  };
  auto rows = [&](int l) {
    for (int ni : {2, 4, 6, 8, 12})
      if (ni * (SC_THREADS / l) >= a.d) return ni;
    return 16;
  };
  while (lj > 4 && ctas(lj) <= (rows(lj) > 4 ? 150 : 75) && 2 * ctas(lj / 2) >= 3 * ctas(lj)) lj >>= 1;
  const int ni = rows(lj);
  return {lj, ni, (a.dv + 4 * lj - 1) / (4 * lj)};
}

// Segments of the CUDA-core pass: one when the heads' tiles fill the GPU, else enough for
// about two CTAs per SM, of at least 64 tokens each.
int scan_segments(const ScanArgs& a) {
  const long long base = (long long)a.B * a.H * scan_shape(a).tiles;
  if (base > SC_SEGS / 3 || a.T < SC_SPLIT) return 1;
  long long n = SC_SEGS / base;
  const long long most = a.T / SC_SEG_MIN;
  if (n > most) n = most;
  return n < 2 ? 1 : (int)n;
}

// Bytes per asynchronous copy: the largest grid that every row starts on.
template <typename T>
int copy_unit(const ScanArgs& a, int cols) {
  const int es = (int)sizeof(T);
  unsigned long long bits = (unsigned long long)cols * es;
  for (const fwpkm_heads* x : {&a.q, &a.k, &a.v})
    bits |= (unsigned long long)(uintptr_t)x->p | (unsigned long long)((x->sb | x->sh | x->st) * es);
  return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2;
}

template <typename T>
int go_scan(const ScanArgs& a, int local, cudaStream_t s) {
  const ScanShape sh = scan_shape(a);
  const int rg = SC_THREADS / sh.lj, dp = rg * sh.ni, cols = 4 * sh.lj;
  const size_t smem = SC_TB * ((size_t)4 * SC_WARPS * cols + 2 * sizeof(T) * (2 * dp + cols));
  const int unit = copy_unit<T>(a, cols);
  // (the 48 KB that need no leave hold the kernel's static tables too)
  const dim3 grid((unsigned)((long long)a.B * a.H * sh.tiles), local ? a.nseg - 1 : a.nseg);
#define FWPKM_SCAN(NI)                                                                           \
  case NI:                                                                                       \
    if (smem > 47 * 1024 && !raise_smem_limit((const void*)scan_kernel<T, NI>, smem)) return -1; \
    launch_k(scan_kernel<T, NI>, grid, SC_THREADS, smem, s, a, sh.lj, unit, local);               \
    break;
  switch (sh.ni) {
    FWPKM_SCAN(2)
    FWPKM_SCAN(4)
    FWPKM_SCAN(6)
    FWPKM_SCAN(8)
    FWPKM_SCAN(12)
    FWPKM_SCAN(16)
    default: return -1;
  }
#undef FWPKM_SCAN
  return 1;
}

// Whether the kernel for a few tokens takes this pass (states in whole 16-byte vectors).
bool step_takes(const ScanArgs& a) {
  return a.T <= SC_STEP && a.dv % 4 == 0 && a.s_in && a.s_out && la_al(a.s_in, 16) && la_al(a.s_out, 16);
}
int launch_step(const ScanArgs& a, int dtype, cudaStream_t s) {
  // eight rows of the state per thread; narrower column tiles when the heads do not fill the GPU
  int lj = SC_THREADS * 8 / (pow2_ceil(a.d) < 64 ? 64 : pow2_ceil(a.d));
  const int need = pow2_ceil((a.dv + 3) / 4);
  if (lj > need) lj = need < 4 ? 4 : need;
  while (lj > 4 && (long long)a.B * a.H * ((a.dv + 4 * lj - 1) / (4 * lj)) < 148) lj >>= 1;
  const unsigned grid = (unsigned)((long long)a.B * a.H * ((a.dv + 4 * lj - 1) / (4 * lj)));
  int ni = 1;
  while (ni * (SC_THREADS / lj) < a.d) ni <<= 1;
#define FWPKM_STEP(NI)                                                                            \
  case NI:                                                                                        \
    if (dtype == FWPKM_BF16) launch_k(step_kernel<__nv_bfloat16, NI>, grid, SC_THREADS, 0, s, a, lj); \
    else launch_k(step_kernel<float, NI>, grid, SC_THREADS, 0, s, a, lj);                         \
    break;
  switch (ni) {
    FWPKM_STEP(1)
    FWPKM_STEP(2)
    FWPKM_STEP(4)
    FWPKM_STEP(8)
    default: return -1;
  }
#undef FWPKM_STEP
  return 1;
}

// One pass on the CUDA cores.
int launch_scan(ScanArgs a, int dtype, int nseg, cudaStream_t s) {
  a.nseg = nseg;
  a.seg_len = a.T < 1 ? 1 : a.T;
  if (nseg > 1) a.seg_len = ((a.T + nseg - 1) / nseg + SC_TB - 1) / SC_TB * SC_TB;
  int nl = 0;
  auto go = [&](int local) { return dtype == FWPKM_BF16 ? go_scan<__nv_bfloat16>(a, local, s) : go_scan<float>(a, local, s); };
  if (nseg > 1) {
    if (go(1) < 0) return -1;
    nl += 1 + launch_scan_combine(a, s);
  }
  if (go(0) < 0) return -1;
  return nl + 1;
}

fwpkm_status check_la(const fwpkm_linattn_config* c, int T) {
  if (!c || c->B < 1 || c->H < 1 || c->d < 1 || c->d_v < 1 || T < 0 || !std::isfinite(c->scale) ||
      !std::isfinite(1.f / c->scale))  // (the gradients' descending passes run on states / scale)
    return FWPKM_ERR_INVALID_ARG;
  if (c->dtype != FWPKM_F32 && c->dtype != FWPKM_BF16) return FWPKM_ERR_INVALID_ARG;
  if (c->d > SC_MAX_D || c->d_v > SC_MAX_D || (long long)c->B * c->H > (1 << 24) || T > (1 << 28)) return FWPKM_ERR_UNSUPPORTED;
  return FWPKM_OK;
}

bool heads_ok(const fwpkm_heads* x, const fwpkm_linattn_config& c, bool out, int width) {
  if (!x || !x->p || !la_al(x->p, c.dtype == FWPKM_BF16 ? 2 : 4) || x->sb < 0 || x->sh < 0 || x->st < 0) return false;
  // an output's rows must not share memory (inputs may be broadcast with a stride of 0)
  if (out && (x->st < width || (c.B > 1 && x->sb == 0) || (c.H > 1 && x->sh == 0))) return false;
  return true;
}

// Whether an output begins where an input does: another CTA may still have to read what it writes.
bool shares(const fwpkm_heads* out, std::initializer_list<const fwpkm_heads*> in) {
  for (const fwpkm_heads* x : in)
    if (x->p == out->p) return true;
  return false;
}

ScanArgs base_args(const fwpkm_linattn_config& c, int T, const float* log_decay, const int32_t* lens) {
  ScanArgs a = {};
  a.log_decay = log_decay; a.lens = lens;
  a.B = c.B; a.H = c.H; a.T = T;
  a.in_scale = 1.f; a.st_scale = 1.f;
  return a;
}
ScanArgs forward_args(const fwpkm_linattn_config& c, int T, const float* log_decay, const int32_t* lens) {
  ScanArgs a = base_args(c, T, log_decay, lens);
  a.d = c.d; a.dv = c.d_v; a.si = c.d_v; a.sj = 1;
  a.out_scale = c.scale;
  return a;
}

// Segments a pass of this shape may use, whatever its pointers and strides.
int most_segments(const ScanArgs& a, int dtype) {
  const int cc = scan_segments(a), tc = scan_tc_shape(a, dtype) ? scan_tc_segments(a) : 1;
  return cc > tc ? cc : tc;
}
size_t slot_bytes(const ScanArgs& a, int nseg) {
  return nseg > 1 ? ((size_t)a.B * a.H * nseg * a.d * a.dv * 4 + 255) / 256 * 256 : 0;
}
int run_pass(ScanArgs a, int dtype, float* slots, cudaStream_t s) {
  a.slots = slots;
  if (scan_tc_takes(a, dtype)) return launch_scan_tc(a, s);
  return launch_scan(a, dtype, scan_segments(a), s);
}

fwpkm_status la_done(int launches) {
  if (launches > 0) count_launches(launches);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) fprintf(stderr, "fwpkm: CUDA error: %s\n", cudaGetErrorString(e));
  return e == cudaSuccess && launches >= 0 ? FWPKM_OK : FWPKM_ERR_CUDA;
}

// Shapes of the three gradient passes.
void grad_args(const fwpkm_linattn_config& c, int T, const float* log_decay, const int32_t* lens, ScanArgs (&p)[3]) {
  for (int i = 0; i < 3; ++i) {
    p[i] = base_args(c, T, log_decay, lens);
    p[i].reverse = i > 0;
  }
  p[0].d = c.d_v; p[0].dv = c.d; p[0].si = 1; p[0].sj = c.d_v;   // dq: state S^T
  p[1].d = c.d_v; p[1].dv = c.d; p[1].si = 1; p[1].sj = c.d_v;   // dk: state D^T
  p[2].d = c.d; p[2].dv = c.d_v; p[2].si = c.d_v; p[2].sj = 1;   // dv: state D
  p[0].out_scale = c.scale;
  for (int i = 1; i < 3; ++i) {
    // the pass runs on D / scale: sums of unscaled q do^T
    p[i].out_scale = c.scale;
    p[i].in_scale = 1.f / c.scale;
    p[i].st_scale = c.scale;
    p[i].in_ready = 1;
    p[i].out_decay = 1;
  }
}

}  // namespace

int launch_scan_combine(const ScanArgs& a, cudaStream_t s) {
  const size_t cells = (size_t)a.d * a.dv;
  launch_k(scan_combine_kernel, dim3((unsigned)((cells + 255) / 256), (unsigned)(a.B * a.H)), 256, 0, s, a);
  return 1;
}

}  // namespace fwpkm

using namespace fwpkm;

extern "C" {

fwpkm_status fwpkm_linear_attention_workspace_size(const fwpkm_linattn_config* cfg, int T, int backward,
                                                   size_t* bytes) {
  const fwpkm_status cs = check_la(cfg, T);
  if (cs != FWPKM_OK) return cs;
  if (!bytes) return FWPKM_ERR_INVALID_ARG;
  size_t most = 0;
  if (backward) {
    ScanArgs p[3];
    grad_args(*cfg, T, nullptr, nullptr, p);
    for (int i = 0; i < 3; ++i) {
      const size_t b = slot_bytes(p[i], most_segments(p[i], cfg->dtype));
      if (b > most) most = b;
    }
  } else {
    const ScanArgs a = forward_args(*cfg, T, nullptr, nullptr);
    most = slot_bytes(a, most_segments(a, cfg->dtype));
  }
  *bytes = most;
  return FWPKM_OK;
}

fwpkm_status fwpkm_linear_attention(const fwpkm_linattn_config* cfg, const fwpkm_heads* q, const fwpkm_heads* k,
                                    const fwpkm_heads* v, int T, const float* log_decay, const int32_t* lens,
                                    const float* s0, const fwpkm_heads* o, float* sT, void* workspace,
                                    size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("fwpkm_linear_attention");
  const fwpkm_status cs = check_la(cfg, T);
  if (cs != FWPKM_OK) return cs;
  if (!log_decay || !la_al(log_decay, 4) || (lens && !la_al(lens, 4)) || (s0 && !la_al(s0, 4)) || (sT && !la_al(sT, 4)))
    return FWPKM_ERR_INVALID_ARG;
  ScanArgs a = forward_args(*cfg, T, log_decay, lens);
  if (T > 0) {
    if (!heads_ok(q, *cfg, false, cfg->d) || !heads_ok(k, *cfg, false, cfg->d) || !heads_ok(v, *cfg, false, cfg->d_v) ||
        !heads_ok(o, *cfg, true, cfg->d_v))
      return FWPKM_ERR_INVALID_ARG;
    a.q = *q; a.k = *k; a.v = *v; a.o = *o;
  } else if (!sT) {
    return FWPKM_OK;
  }
  a.s_in = s0;
  a.s_out = sT;
  size_t need = 0;
  fwpkm_linear_attention_workspace_size(cfg, T, 0, &need);
  if (need > 0 && (!workspace || !la_al(workspace, 256))) return FWPKM_ERR_INVALID_ARG;
  if (ws_bytes < need) return FWPKM_ERR_WORKSPACE;
  if (T > 0 && shares(o, {q, k, v})) return FWPKM_ERR_INVALID_ARG;
  cudaGetLastError();
  PdlScope pdl(true);
  return la_done(run_pass(a, cfg->dtype, (float*)workspace, (cudaStream_t)stream));
}

fwpkm_status fwpkm_linear_attention_backward(const fwpkm_linattn_config* cfg, const fwpkm_heads* q,
                                             const fwpkm_heads* k, const fwpkm_heads* v, int T,
                                             const float* log_decay, const int32_t* lens, const float* s0,
                                             const fwpkm_heads* d_o, const float* d_sT, const fwpkm_heads* dq,
                                             const fwpkm_heads* dk, const fwpkm_heads* dv, float* ds0,
                                             void* workspace, size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("fwpkm_linear_attention_backward");
  const fwpkm_status cs = check_la(cfg, T);
  if (cs != FWPKM_OK) return cs;
  if (!log_decay || !la_al(log_decay, 4) || (lens && !la_al(lens, 4)) || (s0 && !la_al(s0, 4)) ||
      (d_sT && !la_al(d_sT, 4)) || (ds0 && !la_al(ds0, 4)))
    return FWPKM_ERR_INVALID_ARG;
  ScanArgs p[3];
  grad_args(*cfg, T, log_decay, lens, p);
  if (T > 0) {
    if (!heads_ok(q, *cfg, false, cfg->d) || !heads_ok(k, *cfg, false, cfg->d) || !heads_ok(v, *cfg, false, cfg->d_v) ||
        !heads_ok(d_o, *cfg, false, cfg->d_v) || !heads_ok(dq, *cfg, true, cfg->d) ||
        !heads_ok(dk, *cfg, true, cfg->d) || !heads_ok(dv, *cfg, true, cfg->d_v))
      return FWPKM_ERR_INVALID_ARG;
    p[0].q = *d_o; p[0].k = *v; p[0].v = *k; p[0].o = *dq;
    p[1].q = *v; p[1].k = *d_o; p[1].v = *q; p[1].o = *dk;
    p[2].q = *k; p[2].k = *q; p[2].v = *d_o; p[2].o = *dv;
  }
  p[0].s_in = s0;
  p[1].s_in = d_sT;
  p[2].s_in = d_sT;
  p[2].s_out = ds0;
  if (T == 0 && !ds0) return FWPKM_OK;
  size_t need = 0;
  fwpkm_linear_attention_workspace_size(cfg, T, 1, &need);
  if (need > 0 && (!workspace || !la_al(workspace, 256))) return FWPKM_ERR_INVALID_ARG;
  if (ws_bytes < need) return FWPKM_ERR_WORKSPACE;
  if (T > 0 && (shares(dq, {q, k, v, d_o, dk, dv}) || shares(dk, {q, k, v, d_o, dv}) || shares(dv, {q, k, v, d_o})))
    return FWPKM_ERR_INVALID_ARG;
  cudaGetLastError();
  PdlScope pdl(true);
  int nl = 0;
  // dv last: it alone writes ds0, which may be d_sT's own memory
  for (int i = T > 0 ? 0 : 2; i < 3; ++i) {
    const int r = run_pass(p[i], cfg->dtype, (float*)workspace, (cudaStream_t)stream);
    if (r < 0) return la_done(-1);
    nl += r;
  }
  return la_done(nl);
}

fwpkm_status fwpkm_linear_attention_step(const fwpkm_linattn_config* cfg, const fwpkm_heads* q, const fwpkm_heads* k,
                                         const fwpkm_heads* v, int n_tok, const float* log_decay,
                                         const int32_t* lens, const float* state, const fwpkm_heads* o,
                                         float* state_out, void* stream) {
  NvtxRange nvtx_range("fwpkm_linear_attention_step");
  const fwpkm_status cs = check_la(cfg, n_tok);
  if (cs != FWPKM_OK) return cs;
  if (!log_decay || !la_al(log_decay, 4) || (lens && !la_al(lens, 4)) || !state || !state_out || !la_al(state, 4) ||
      !la_al(state_out, 4))
    return FWPKM_ERR_INVALID_ARG;
  if (n_tok == 0 && state == state_out) return FWPKM_OK;
  ScanArgs a = forward_args(*cfg, n_tok, log_decay, lens);
  if (n_tok > 0) {
    if (!heads_ok(q, *cfg, false, cfg->d) || !heads_ok(k, *cfg, false, cfg->d) || !heads_ok(v, *cfg, false, cfg->d_v) ||
        !heads_ok(o, *cfg, true, cfg->d_v))
      return FWPKM_ERR_INVALID_ARG;
    a.q = *q; a.k = *k; a.v = *v; a.o = *o;
  }
  if (n_tok > 0 && shares(o, {q, k, v})) return FWPKM_ERR_INVALID_ARG;
  a.s_in = state;
  a.s_out = state_out;
  cudaGetLastError();
  PdlScope pdl(true);
  return la_done(step_takes(a) ? launch_step(a, cfg->dtype, (cudaStream_t)stream)
                               : launch_scan(a, cfg->dtype, 1, (cudaStream_t)stream));
}

fwpkm_status fwpkm_linear_attention_sync(void* stream) {
  if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return la_done(-1);
  const int st = take_scan_status();
  return st < 0 ? la_done(-1) : status_of_device(st);
}

}  // extern "C"
