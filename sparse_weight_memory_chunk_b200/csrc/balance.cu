// balance.cu -- how evenly a router uses its experts (sub-keys, slots): a balance loss on its
// logits, the experts' counts, and the loss's gradient.
//
// Per group (a layer, a sequence, one half of a memory's codebook) with logits x [T][E]:
//   P_t = softmax(x_t),  u = mean_t P_t (usage),  c_e = selections of expert e (counts)
//   load:     L = coef E sum_e f_e u_e,   f = c / sum c       (a_e = E f_e)
//   entropy:  L = coef sum_e u_e log u_e  (= -coef H(u), the memory's own anti-collapse loss,
//             Fast-weight Product Key Memory (paperlayer summary) §3.4; a_e = log u_e + 1)
//   dx_t[e] = dL coef / T P_t[e] (a_e - sum_e' a_e' P_t[e'])
// over the T tokens that the mask leaves (counts are constants of the gradient).  A row whose
// logits are all -inf has no softmax: it is left out like a masked one, but its selections
// count.  The gradient does not see a constant added to a, so the forward stores the slope
// coef (a - const) / T with the constant that a balanced router has (E f - 1, log(E u)):
// what is left in the bracket then does not cancel in fp32.
//
// Bytes: x read once per direction, dx written once; ~8 operations per logit: bound by HBM.
// Forward: CTAs over blocks of a group's rows, a team of lanes per row with the row in
// registers (one read), column sums in registers over the team's rows, joined over the
// CTA's teams in team order; a second launch joins the CTAs' partial sums in a fixed order, in fp64.
// No float atomics, so the results are deterministic; the counts are integer sums.
#include <cmath>
#include <cstdio>

#include "fwpkm_internal.cuh"

namespace fwpkm {
namespace {

constexpr int BL_THREADS = 256;
constexpr int BL_MAX_E = 4096;
constexpr int BL_JOIN = 512;

struct BalArgs {
  const void* x;
  long long ld, gs;        // elements between a group's rows, and between groups
  const int32_t* idx;      // [G][T][k] or null
  const uint8_t* mask;     // [G][T] or null
  int G, E, k, ctas;       // ctas: per group
  long long T, rows_cta;   // rows per CTA
  float* part;             // [G][ctas][E] partial usage sums
  int32_t* cpart;          // [G][ctas][E] partial counts
  int32_t* npart;          // [G][ctas] rows with a softmax
  double* usum;            // [G][E] their sums over the CTAs
  int32_t* csum;           // [G][E]
  int* done;               // [G] CTAs of the join that have written theirs
};

template <typename T, int VEC>
struct __align__(sizeof(T) * VEC) BPack {
  T v[VEC];
};
__device__ __forceinline__ float bal_f(float x) { return x; }
__device__ __forceinline__ float bal_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void bal_put(float& d, float x) { d = x; }
__device__ __forceinline__ void bal_put(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }

// A row of E logits over a team of L lanes (L <= 32: lanes of a warp; L = BL_THREADS: the
// CTA): thread `l` holds elements (j L + l) VEC .. +VEC-1, j < NCH; -inf past E.  fetch_row
// issues the loads of row t (false: behind `end`, or masked: nothing is read).
template <typename T, int VEC, int NCH, int L>
__device__ __forceinline__ bool fetch_row(const T* __restrict__ x, const uint8_t* __restrict__ mask, long long t,
                                          long long end, long long ld, int E, int l, BPack<T, VEC> (&p)[NCH]) {
  if (t >= end || (mask && !mask[t])) return false;
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    const int e = (j * L + l) * VEC;
    if (e < E) p[j] = *reinterpret_cast<const BPack<T, VEC>*>(x + t * ld + e);
  }
  return true;
}
template <typename T, int VEC, int NCH, int L>
__device__ __forceinline__ void take_row(const BPack<T, VEC> (&p)[NCH], bool on, int E, int l,
                                         float (&v)[VEC * NCH]) {
#pragma unroll
  for (int j = 0; j < NCH; ++j)
#pragma unroll
    for (int u = 0; u < VEC; ++u) v[j * VEC + u] = on && (j * L + l) * VEC < E ? bal_f(p[j].v[u]) : -INFINITY;
}

template <int L, bool MAX>
__device__ __forceinline__ float team_reduce(float x, float* red) {
  constexpr int W = L < 32 ? L : 32;
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, x, o);
    x = MAX ? fmaxf(x, y) : x + y;
  }
  if (L > 32) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    x = red[0];
#pragma unroll
    for (int w = 1; w < L / 32; ++w) x = MAX ? fmaxf(x, red[w]) : x + red[w];
  }
  return x;
}

// v -> exp(v - max) over the team; returns 1 / their sum, 0 (v = 0) for a row of -inf.  The maximum
// passes NaN by, but the sum keeps it.  exp is 2^((v - max) log2 e) by the hardware's 2^x (2^-22
// relative): with expf, 32 values a lane, the instructions and not the loads bounded both
// directions.  The difference comes first, so that the row's largest term is 1 whatever its logits:
// max log2 e rounded by itself is off by more than 2^x can hold from 4e9 on, and overflows for a row
// filled with the type's lowest value.
template <int NV, int L>
__device__ __forceinline__ float team_exp(float (&v)[NV], float* red) {
  constexpr float LOG2E = 1.4426950408889634f;
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) m = fmaxf(m, v[i]);
  m = team_reduce<L, true>(m, red);
  const float top = m == -INFINITY ? 0.f : m;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(v[i]) : "f"((v[i] - top) * LOG2E));
    s += v[i];
  }
  s = team_reduce<L, false>(s, red);
  return s == 0.f ? 0.f : 1.f / s;
}

template <typename T, int VEC, int NCH, int L>
__global__ void __launch_bounds__(BL_THREADS, L > 32 ? 4 : 1)
balance_sum_kernel(BalArgs a) {
  constexpr int NV = VEC * NCH;
  constexpr int TEAMS = BL_THREADS / L;
  extern __shared__ float sm[];               // [TEAMS][L * NV] usage sums, then counts [E]
  __shared__ float red[BL_THREADS / 32];
  __shared__ int s_n;
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.y, cta = blockIdx.x;
  const int team = threadIdx.x / L, l = threadIdx.x % L;
  const long long t0 = (long long)cta * a.rows_cta;
  const long long t1 = t0 + a.rows_cta < a.T ? t0 + a.rows_cta : a.T;
  const T* x = (const T*)a.x + (long long)g * a.gs;
  const uint8_t* mask = a.mask ? a.mask + (long long)g * a.T : nullptr;
  int* cnt = (int*)(sm + TEAMS * L * NV);
  if (threadIdx.x == 0) s_n = 0;
  if (a.idx)
    for (int e = threadIdx.x; e < a.E; e += BL_THREADS) cnt[e] = 0;
  float acc[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) acc[i] = 0.f;
  int n = 0;
  __syncthreads();
  // every team of a warp takes part in the warp's shuffles, so the loop's trip count is the CTA's;
  // a team's next row is on its way while it works on this one
  BPack<T, VEC> next[NCH];
  bool next_on = fetch_row<T, VEC, NCH, L>(x, mask, t0 + team, t1, a.ld, a.E, l, next);
  for (long long tb = t0; tb < t1; tb += TEAMS) {
    float v[NV];
    take_row<T, VEC, NCH, L>(next, next_on, a.E, l, v);
    next_on = fetch_row<T, VEC, NCH, L>(x, mask, tb + TEAMS + team, t1, a.ld, a.E, l, next);
    const float inv = team_exp<NV, L>(v, red);
    if (inv != 0.f) {
#pragma unroll
      for (int i = 0; i < NV; ++i) acc[i] = fmaf(v[i], inv, acc[i]);
      n += l == 0;
    }
  }
  if (n) atomicAdd(&s_n, n);
  if (a.idx) {
    const int32_t* ix = a.idx + (long long)g * a.T * a.k;
    for (long long p = t0 * a.k + threadIdx.x; p < t1 * a.k; p += BL_THREADS) {
      const int e = ix[p];
      if (e >= 0 && e < a.E && (!mask || mask[p / a.k])) atomicAdd(&cnt[e], 1);
    }
  }
#pragma unroll
  for (int j = 0; j < NCH; ++j)
#pragma unroll
    for (int u = 0; u < VEC; ++u) sm[team * (L * NV) + (j * L + l) * VEC + u] = acc[j * VEC + u];
  __syncthreads();
  float* part = a.part + ((long long)g * a.ctas + cta) * a.E;
  for (int e = threadIdx.x; e < a.E; e += BL_THREADS) {
    float s = 0.f;
    for (int q = 0; q < TEAMS; ++q) s += sm[q * (L * NV) + e];
    part[e] = s;
    if (a.idx) a.cpart[((long long)g * a.ctas + cta) * a.E + e] = cnt[e];
  }
  if (threadIdx.x == 0) {
    a.npart[(long long)g * a.ctas + cta] = s_n;
    if (cta == 0) a.done[g] = 0;
  }
}

__device__ __forceinline__ double block_sum(double x, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  x = (threadIdx.x & 31) < BL_JOIN / 32 ? red[threadIdx.x & 31] : 0.0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The CTAs' partial sums -> usage, counts, loss, slope.  A CTA takes BL_JOIN / slices columns of a
// group: slice i of its threads adds CTAs i, i + slices, .. and the slices are added in order.  The
// group's last CTA to finish has all columns' sums before it and forms the results.  (By one
// CTA per group the chain of loads took 30 us for 2 groups of 256 experts from 295 CTAs each,
// and by a cluster of eight 58 us for one of 4096.)
__global__ void __launch_bounds__(BL_JOIN)
balance_join_kernel(BalArgs a, int slices, int kind, float coef, double log_e, float* __restrict__ loss, int32_t* __restrict__ counts,
                    float* __restrict__ usage, float* __restrict__ slope) {
  __shared__ double red[BL_JOIN / 32];
  __shared__ double su[BL_JOIN];
  __shared__ int sc[BL_JOIN];
  __shared__ int s_last;
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.y, tid = threadIdx.x;
  const int cols = BL_JOIN / slices, col = tid & (cols - 1), slice = tid / cols;
  const int e = blockIdx.x * cols + col;
  double s = 0.0;
  int c = 0;
  if (e < a.E) {
    // (addresses clamped and values masked, so that the loads of a round go out together)
    const float* part = a.part + (long long)g * a.ctas * a.E + e;
    const int32_t* cp = (a.idx ? a.cpart : reinterpret_cast<const int32_t*>(a.part)) + (long long)g * a.ctas * a.E + e;
    const int counted = a.idx ? -1 : 0;
    constexpr int U = 8;
    for (int q = slice; q < a.ctas; q += U * slices) {
      float f[U];
      int k[U];
#pragma unroll
      for (int v = 0; v < U; ++v) {
        const int at = min(q + v * slices, a.ctas - 1) * a.E;
        f[v] = __ldcg(part + at);
        k[v] = __ldcg(cp + at);
      }
#pragma unroll
      for (int v = 0; v < U; ++v) {
        const bool in = q + v * slices < a.ctas;
        s += in ? f[v] : 0.f;
        c += in ? k[v] & counted : 0;
      }
    }
  }
  su[tid] = s;
  sc[tid] = c;
  __syncthreads();
  if (slice == 0 && e < a.E) {
    for (int q = 1; q < slices; ++q) {
      s += su[q * cols + col];
      c += sc[q * cols + col];
    }
    a.usum[(long long)g * a.E + e] = s;
    a.csum[(long long)g * a.E + e] = c;
    __threadfence();
  }
  __syncthreads();
  if (tid == 0) s_last = atomicAdd(&a.done[g], 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();

  double n = 0.0;
  for (int q = tid; q < a.ctas; q += BL_JOIN) n += a.npart[(long long)g * a.ctas + q];
  n = block_sum(n, red);
  const double inv_n = n > 0.0 ? 1.0 / n : 0.0;
  constexpr int PER = BL_MAX_E / BL_JOIN;        // columns per thread at most
  double u[PER];
  int cc[PER];
  double csum = 0.0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int x = i * BL_JOIN + tid;
    const long long o = (long long)g * a.E + x;
    u[i] = x < a.E ? __ldcg(a.usum + o) : 0.0;
    cc[i] = x < a.E ? __ldcg(a.csum + o) : 0;
    csum += cc[i];
  }
  csum = block_sum(csum, red);
  const double inv_c = csum > 0.0 ? 1.0 / csum : 0.0;
  double l = 0.0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int x = i * BL_JOIN + tid;
    if (x < a.E) {
      const double ue = u[i] * inv_n;
      double ae;
      if (kind == FWPKM_BALANCE_LOAD) {
        const double f = cc[i] * inv_c;
        l += a.E * f * ue;
        ae = csum > 0.0 ? a.E * f - 1.0 : 0.0;
      } else {
        ae = ue > 0.0 ? log(ue * a.E) : (ue == 0.0 ? 0.0 : ue);  // NaN stays
        l += ue * (ae - log_e);
      }
      const long long o = (long long)g * a.E + x;
      usage[o] = (float)ue;
      if (counts) counts[o] = cc[i];
      slope[o] = (float)(coef * ae * inv_n);
    }
  }
  l = block_sum(l, red);
  if (tid == 0) loss[g] = (float)(coef * l);
}

template <typename T, int VEC, int NCH, int L>
__global__ void __launch_bounds__(BL_THREADS, L > 32 ? 4 : 1)
balance_grad_kernel(BalArgs a, const float* __restrict__ slope, const float* __restrict__ d_loss, T* __restrict__ dx) {
  constexpr int NV = VEC * NCH;
  constexpr int TEAMS = BL_THREADS / L;
  __shared__ float red[BL_THREADS / 32];
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.y;
  const int team = threadIdx.x / L, l = threadIdx.x % L;
  const T* x = (const T*)a.x + (long long)g * a.gs;
  const uint8_t* mask = a.mask ? a.mask + (long long)g * a.T : nullptr;
  T* d = dx + (long long)g * a.T * a.E;
  float s[NV];
#pragma unroll
  for (int j = 0; j < NCH; ++j)
#pragma unroll
    for (int u = 0; u < VEC; ++u) {
      const int e = (j * L + l) * VEC + u;
      s[j * VEC + u] = e < a.E ? slope[(long long)g * a.E + e] : 0.f;
    }
  const float gl = d_loss ? d_loss[g] : 1.f;
  const long long step = (long long)gridDim.x * TEAMS;
  BPack<T, VEC> next[NCH];
  bool next_on = fetch_row<T, VEC, NCH, L>(x, mask, (long long)blockIdx.x * TEAMS + team, a.T, a.ld, a.E, l, next);
  for (long long tb = (long long)blockIdx.x * TEAMS; tb < a.T; tb += step) {
    const long long t = tb + team;
    const bool in = t < a.T;
    float v[NV];
    take_row<T, VEC, NCH, L>(next, next_on, a.E, l, v);
    next_on = fetch_row<T, VEC, NCH, L>(x, mask, t + step, a.T, a.ld, a.E, l, next);
    const float inv = team_exp<NV, L>(v, red);
    float c = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) c = fmaf(v[i], s[i], c);
    c = team_reduce<L, false>(c, red) * inv;
    const float f = gl * inv;
    if (in) {
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const int e = (j * L + l) * VEC;
        if (e < a.E) {
          BPack<T, VEC> p;
#pragma unroll
          for (int u = 0; u < VEC; ++u)
            bal_put(p.v[u], inv != 0.f ? f * v[j * VEC + u] * (s[j * VEC + u] - c) : 0.f);
          *reinterpret_cast<BPack<T, VEC>*>(d + t * a.E + e) = p;
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
size_t b256(size_t x) { return (x + 255) / 256 * 256; }
bool bal_al(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t bal_es(int dt) { return dt == FWPKM_BF16 ? 2 : 4; }

// CTAs that the GPU holds at once: a row of up to 1024 logits sits in the registers of a warp
// twice (its values and the next row's loads); wider ones are spread over the CTA, whose
// threads hold 16 of their values (16384 rows of 4096 bf16: 200 us for both directions with two
// CTAs per SM, 152 with the four that 64 registers a thread allow).
int bal_resident(int E) { return 148 * (E > 1024 ? 4 : E > 512 ? 2 : E > 256 ? 3 : 4); }

// Rows per CTA of the forward: no more CTAs over all groups than are resident (a second wave of
// a few doubles the time: 123 us instead of 70 for 16 groups of 4096 x 1024 fp32), and at
// least 32 rows each (a CTA costs a row of partial sums).
void split_rows(const fwpkm_balance_config& c, int* ctas, long long* rows) {
  long long n = bal_resident(c.experts) / c.groups;
  const long long most = (c.tokens + 31) / 32;
  if (n > most) n = most;
  if (n < 1) n = 1;
  *rows = (c.tokens + n - 1) / n;
  if (*rows < 1) *rows = 1;
  *ctas = (int)((c.tokens + *rows - 1) / *rows);
  if (*ctas < 1) *ctas = 1;
}

size_t bal_carve(const fwpkm_balance_config& c, char* base, BalArgs* a) {
  int ctas;
  long long rows;
  split_rows(c, &ctas, &rows);
  const size_t cells = (size_t)c.groups * ctas;
  const size_t p = b256(4 * cells * c.experts), cols = (size_t)c.groups * c.experts;
  if (a) {
    a->part = (float*)base;
    a->cpart = (int32_t*)(base + p);
    a->npart = (int32_t*)(base + 2 * p);
    a->usum = (double*)(base + 2 * p + b256(4 * cells));
    a->csum = (int32_t*)(base + 2 * p + b256(4 * cells) + b256(8 * cols));
    a->done = (int*)(base + 2 * p + b256(4 * cells) + b256(8 * cols) + b256(4 * cols));
    a->ctas = ctas;
    a->rows_cta = rows;
  }
  return 2 * p + b256(4 * cells) + b256(8 * cols) + b256(4 * cols) + b256(4 * (size_t)c.groups);
}

fwpkm_status check_balance(const fwpkm_balance_config* c) {
  if (!c || c->groups < 1 || c->tokens < 0 || c->experts < 1 || c->k < 0 || c->ld < c->experts || c->group_stride < 0)
    return FWPKM_ERR_INVALID_ARG;
  if (c->dtype != FWPKM_F32 && c->dtype != FWPKM_BF16) return FWPKM_ERR_INVALID_ARG;
  if (c->kind != FWPKM_BALANCE_LOAD && c->kind != FWPKM_BALANCE_ENTROPY) return FWPKM_ERR_INVALID_ARG;
  // counts are 32-bit: a group's selections must fit
  if (c->experts > BL_MAX_E || c->groups > 65535 || c->k > BL_MAX_E ||
      (c->k > 0 && c->tokens > 0x7fffffffLL / c->k))
    return FWPKM_ERR_UNSUPPORTED;
  return FWPKM_OK;
}

BalArgs bal_args(const fwpkm_balance_config& c, const void* x, const int32_t* idx, const uint8_t* mask) {
  BalArgs a = {};
  a.x = x; a.ld = c.ld; a.gs = c.group_stride; a.idx = idx; a.mask = mask;
  a.G = c.groups; a.E = c.experts; a.k = c.k; a.T = c.tokens;
  return a;
}

fwpkm_status bal_done(int launches) {
  count_launches(launches);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return FWPKM_OK;
  fprintf(stderr, "fwpkm: CUDA error: %s\n", cudaGetErrorString(e));
  return FWPKM_ERR_CUDA;
}

struct BalRun {
  bool grad;
  BalArgs a;
  const float* slope;
  const float* d_loss;
  void* dx;
  cudaStream_t s;
};

template <typename T, int VEC, int NCH, int L>
bool bal_go(const BalRun& r) {
  if (!r.grad) {
    const size_t smem = 4 * ((size_t)BL_THREADS * VEC * NCH) + (r.a.idx ? 4 * (size_t)r.a.E : 0);
    if (smem > 47 * 1024 && !raise_smem_limit((const void*)balance_sum_kernel<T, VEC, NCH, L>, smem)) return false;
    launch_k(balance_sum_kernel<T, VEC, NCH, L>, dim3(r.a.ctas, r.a.G), BL_THREADS, smem, r.s, r.a);
  } else {
    constexpr int TEAMS = BL_THREADS / L;
    long long gx = (r.a.T + TEAMS - 1) / TEAMS;
    const int all = bal_resident(r.a.E) / r.a.G;
    const long long most = all < 1 ? 1 : all;
    if (gx > most) gx = most;
    launch_k(balance_grad_kernel<T, VEC, NCH, L>, dim3((unsigned)gx, r.a.G), BL_THREADS, 0, r.s, r.a, r.slope,
             r.d_loss, (T*)r.dx);
  }
  return true;
}

// Lanes per row: as few as hold the row in one vector each up to a warp, then more vectors
// per lane (the row stays in registers), then the whole CTA.
template <typename T, int VEC>
bool bal_shape(const BalRun& r) {
  const int v = (r.a.E + VEC - 1) / VEC;  // vectors of a row
  if (v <= 2) return bal_go<T, VEC, 1, 2>(r);
  if (v <= 8) return bal_go<T, VEC, 1, 8>(r);
  if (v <= 32) return bal_go<T, VEC, 1, 32>(r);
  if (v <= 64) return bal_go<T, VEC, 2, 32>(r);
  if (v <= 128) return bal_go<T, VEC, 4, 32>(r);
  if (VEC < 8 && v <= 256) return bal_go<T, VEC, 8, 32>(r);
  if (VEC > 1) return bal_go<T, VEC, (BL_MAX_E / VEC + BL_THREADS - 1) / BL_THREADS, BL_THREADS>(r);
  if (v <= 1024) return bal_go<T, VEC, VEC == 1 ? 32 : 1, 32>(r);
  return bal_go<T, VEC, VEC == 1 ? BL_MAX_E / BL_THREADS : 1, BL_THREADS>(r);
}

template <typename T>
bool bal_type(const BalRun& r) {
  constexpr int VEC = 16 / (int)sizeof(T);
  const bool vec = bal_al(r.a.x, 16) && r.a.E % VEC == 0 && r.a.ld % VEC == 0 && r.a.gs % VEC == 0 &&
                   (!r.grad || bal_al(r.dx, 16));
  return vec ? bal_shape<T, VEC>(r) : bal_shape<T, 1>(r);
}

}  // namespace
}  // namespace fwpkm

using namespace fwpkm;

extern "C" {

fwpkm_status fwpkm_balance_workspace_size(const fwpkm_balance_config* cfg, size_t* bytes) {
  const fwpkm_status cs = check_balance(cfg);
  if (cs != FWPKM_OK) return cs;
  if (!bytes) return FWPKM_ERR_INVALID_ARG;
  *bytes = bal_carve(*cfg, nullptr, nullptr);
  return FWPKM_OK;
}

fwpkm_status fwpkm_balance_loss(const fwpkm_balance_config* cfg, const void* x, const int32_t* idx,
                                const uint8_t* mask, void* workspace, size_t ws_bytes, float* loss, int32_t* counts,
                                float* usage, float* slope, void* stream) {
  NvtxRange nvtx_range("fwpkm_balance_loss");
  const fwpkm_status cs = check_balance(cfg);
  if (cs != FWPKM_OK) return cs;
  if (!loss || !usage || !slope || !bal_al(loss, 4) || !bal_al(usage, 4) || !bal_al(slope, 4) ||
      (counts && !bal_al(counts, 4)))
    return FWPKM_ERR_INVALID_ARG;
  if (cfg->tokens > 0 && (!x || !bal_al(x, bal_es(cfg->dtype)))) return FWPKM_ERR_INVALID_ARG;
  if (idx && (cfg->k < 1 || !bal_al(idx, 4))) return FWPKM_ERR_INVALID_ARG;
  if (cfg->kind == FWPKM_BALANCE_LOAD && !idx && cfg->tokens > 0) return FWPKM_ERR_INVALID_ARG;
  if (!workspace || !bal_al(workspace, 256)) return FWPKM_ERR_INVALID_ARG;
  if (ws_bytes < bal_carve(*cfg, nullptr, nullptr)) return FWPKM_ERR_WORKSPACE;
  cudaGetLastError();
  PdlScope pdl(true);
  BalRun r = {};
  r.a = bal_args(*cfg, x, cfg->tokens > 0 ? idx : nullptr, mask);
  r.s = (cudaStream_t)stream;
  bal_carve(*cfg, (char*)workspace, &r.a);
  const bool ok = cfg->dtype == FWPKM_BF16 ? bal_type<__nv_bfloat16>(r) : bal_type<float>(r);
  if (!ok) return FWPKM_ERR_CUDA;
  int slices = 1;  // about eight CTAs' sums per thread, whole warps per slice
  while (slices < BL_JOIN / 32 && slices * 8 < r.a.ctas) slices <<= 1;
  const int cols = BL_JOIN / slices;
  launch_k(balance_join_kernel, dim3((cfg->experts + cols - 1) / cols, cfg->groups), BL_JOIN, 0, r.s, r.a, slices,
           cfg->kind, cfg->coef, log((double)cfg->experts), loss, counts, usage, slope);
  return bal_done(2);
}

fwpkm_status fwpkm_balance_loss_backward(const fwpkm_balance_config* cfg, const void* x, const uint8_t* mask,
                                         const float* slope, const float* d_loss, void* dx, void* stream) {
  NvtxRange nvtx_range("fwpkm_balance_loss_backward");
  const fwpkm_status cs = check_balance(cfg);
  if (cs != FWPKM_OK) return cs;
  if (cfg->tokens == 0) return FWPKM_OK;
  const size_t es = bal_es(cfg->dtype);
  if (!x || !slope || !dx || !bal_al(x, es) || !bal_al(dx, es) || !bal_al(slope, 4) || (d_loss && !bal_al(d_loss, 4)))
    return FWPKM_ERR_INVALID_ARG;
  // (in place a row is read and written by the same threads, but only where dx's rows are x's)
  if (dx == x && ((cfg->ld != cfg->experts && cfg->tokens > 1) ||
                  (cfg->group_stride != cfg->tokens * cfg->experts && cfg->groups > 1)))
    return FWPKM_ERR_INVALID_ARG;
  cudaGetLastError();
  PdlScope pdl(true);
  BalRun r = {};
  r.grad = true;
  r.a = bal_args(*cfg, x, nullptr, mask);
  r.slope = slope;
  r.d_loss = d_loss;
  r.dx = dx;
  r.s = (cudaStream_t)stream;
  const bool ok = cfg->dtype == FWPKM_BF16 ? bal_type<__nv_bfloat16>(r) : bal_type<float>(r);
  if (!ok) return FWPKM_ERR_CUDA;
  return bal_done(1);
}

}  // extern "C"
