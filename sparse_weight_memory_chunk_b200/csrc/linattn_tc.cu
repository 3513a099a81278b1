// linattn_tc.cu -- the linear-attention pass of linattn.cu on the tensor cores: bf16 operands,
// widths up to 128, chunks of 128 tokens (tcgen05.mma, TMEM accumulators, TMA-fed tiles).
//
// With E the state after the previous chunk, a the head's decay and t, s positions inside the
// chunk, a chunk of m tokens is four products:
//   P  = Q K^T                                           [t][s]
//   O  = diag(a^(t+1)) Q E + (P . a^(t-s), s <= t) V     [t][dv]
//   U  = sum_s a^(m-1-s) k_s v_s^T                       [d][dv]
//   E' = a^m E + U
// The descending pass is the same with the rows of the tile mirrored: its tiles end at the
// chunk's first token, so every formula takes u = 127 - row.
//
// Precision: the inputs are bf16, exact operands.  What is not exact in bf16 enters as pieces:
// P (weighted) and E as hi + lo (2^-18 left out; O is rounded to bf16 afterwards), the
// weighted keys of U as hi + mid + lo (exact to fp32, so the fp32 state that is handed on
// agrees with fp32 arithmetic).  E is kept in fp32 registers and U is a fresh accumulator per
// chunk, so the tensor cores' running sums span one chunk only.
//
// CTA = one head (and segment): warp 0 issues TMA loads (K, V two stages, Q one), warp 1 owns
// TMEM and issues the MMAs (one thread), warps 2-9 do the elementwise work: warp w reads
// TMEM lanes 32 (w % 4).. and column half (w - 2) / 4.  TMEM (512 columns): P fp32, overwritten
// in place by its two bf16 pieces (operand A of P V); O; U; two pieces of the weighted,
// transposed keys (operand A of U; the high piece waits in registers and takes the low one's
// place: U's large terms come last, so few of the accumulator's roundings are at full size,
// 2e-7 of the state instead of 6e-7 the other way round).  Per chunk, in order:
//   MMA    P(c)   Q E(c)          U lo, mid           U hi, P V              P(c+1) ..
//   math       K pieces(c) ......  P pieces, O scale ...  E update, E pieces, O out
// Bound: HBM for d = d_v = 128 (1 KB per token and head against 8 tensor products of
// 128 x 128 per token: 0.5 us of MMA and ~0.5 us of elementwise work per 0.7 us of HBM time
// per chunk and SM at the measured rates).
#include <cstdio>

#include "linattn.cuh"
#include "sm100.cuh"

namespace fwpkm {

using namespace sm100;

namespace {

constexpr int LC = 128;                  // tokens per chunk
constexpr int LA_MATH_WARPS = 8;
constexpr int LA_THREADS = (2 + LA_MATH_WARPS) * 32;
constexpr uint64_t LA_TIMEOUT_NS = 200ull * 1000 * 1000;  // any single wait
constexpr int LA_BLOCK = LC * 128;       // bytes of a 64-column block of 128 rows

__device__ int g_la_status = DEV_OK;     // latched by a kernel whose wait ran out

// TMEM columns
constexpr uint32_t TM_P = 0, TM_O = 128, TM_U = 256, TM_K0 = 384, TM_K1 = 448, TM_COLS = 512;

struct TcBars {
  uint64_t full_q, full_kv[2], p, o1, kt, u1, mid, u2, o2[2], next, drain, stall;
};

template <int DK, int DV>
struct TcSmem {
  static constexpr int Q = LC * DK * 2, K = LC * DK * 2, V = LC * DV * 2, E = DK * DV * 2;
  static constexpr int off_k = Q, off_v = off_k + 2 * K, off_e = off_v + 2 * V, off_tab = off_e + 2 * E;
  static constexpr int need = off_tab + 4 * (LC + 4) + (int)sizeof(TcBars) + 16 + 1024;
  // one CTA per SM: each holds all of TMEM
  static constexpr int bytes = need > 120 * 1024 ? need : 120 * 1024;
};

// Wait for a phase; false once any role gave up (or this wait ran out, which raises abort).
__device__ __forceinline__ bool la_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  uint32_t n = 0;
  uint64_t t0 = 0;
  while (!mbar_try_wait(bar, parity)) {
    if ((++n & 255u) == 0) {
      if (*abort) return false;
      const uint64_t t = globaltimer();
      if (t0 == 0) t0 = t;
      else if (t - t0 > LA_TIMEOUT_NS) {
        *abort = 1;
        return false;
      }
    }
  }
  return true;
}
// The same for a whole warp: one lane waits, all learn the verdict (and stay converged).
__device__ __forceinline__ bool la_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, int lane) {
  int ok = lane == 0 ? (la_wait(bar, parity, abort) ? 1 : 0) : 0;
  ok = __shfl_sync(0xffffffffu, ok, 0);
  return ok != 0;
}
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer() - t0 > LA_TIMEOUT_NS) return;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float low_f(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float high_f(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

// Byte of element (row, col) in a tile of 64-column blocks of `rows` 128-byte rows, swizzled.
__device__ __forceinline__ uint32_t sw_off(int row, int col, int rows) {
  return (uint32_t)((col >> 6) * rows * 128 + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4) + (col & 7) * 2);
}

struct TcCoord {
  int h, b;  // 1, or 0 where the tensor is broadcast along the axis
};
struct TcPass {
  ScanArgs a;
  TcCoord cq, ck, cv;
  int local, stall;
};

template <int DK, int DV>
__global__ void __launch_bounds__(LA_THREADS, 1)
scan_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, const TcPass ps) {
  using SM = TcSmem<DK, DV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *sq = smem, *sk = smem + SM::off_k, *sv = smem + SM::off_v, *se = smem + SM::off_e;
  float* pw = (float*)(smem + SM::off_tab);  // [LC + 1] a^j
  TcBars* bar = (TcBars*)(pw + LC + 4);
  uint32_t* tmem_slot = (uint32_t*)(bar + 1);
  volatile int* abort = (volatile int*)(tmem_slot + 1);

  const ScanArgs& a = ps.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool local = ps.local != 0;
  const int bh = blockIdx.x, g = blockIdx.y;
  const int b = bh / a.H, h = bh - b * a.H;

  if (threadIdx.x == 0) {
    mbar_init(&bar->full_q, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->full_kv[i], 1);
      mbar_init(&bar->o2[i], 1);
    }
    mbar_init(&bar->p, 1);
    mbar_init(&bar->o1, 1);
    mbar_init(&bar->kt, LA_MATH_WARPS);
    mbar_init(&bar->u1, 1);
    mbar_init(&bar->mid, LA_MATH_WARPS);
    mbar_init(&bar->u2, 1);
    mbar_init(&bar->next, LA_MATH_WARPS);
    mbar_init(&bar->drain, 1);
    mbar_init(&bar->stall, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  const int n = scan_len(a, b);
  const int t0 = min(n, g * a.seg_len), t1 = min(n, t0 + a.seg_len);  // positions along the pass
  const int chunks = (t1 - t0 + LC - 1) / LC;
  const float ld = a.log_decay[h];
  const float* init = nullptr;
  long long isi = a.dv, isj = 1;
  float in_scale = 1.f;
  const size_t cells = (size_t)a.d * a.dv;
  if (!local) {
    if (a.nseg > 1) {
      init = a.slots + ((size_t)bh * a.nseg + (g == 0 ? a.nseg - 1 : g - 1)) * cells;
    } else if (a.s_in) {
      init = a.s_in + (size_t)bh * cells;
      isi = a.si;
      isj = a.sj;
      in_scale = n == 0 ? 1.f : a.in_scale;
    }
  }
  // first token row of the tile of chunk c: ascending, or ending at the chunk's first token
  auto tile_t = [&](int c) { return a.reverse ? n - (t0 + c * LC) - LC : t0 + c * LC; };

  int kv_loads = 0, q_loads = 0;  // producer: chunks whose loads were issued
  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer ----------------
      auto load = [&](const CUtensorMap* m, uint8_t* dst, int width, uint64_t* fb, const TcCoord& cc, int c) {
        for (int x = 0; x < width; x += 64)
          tma_load_4d(dst + (x >> 6) * LA_BLOCK, m, fb, x, tile_t(c), h * cc.h, b * cc.b);
      };
      bool ok = true;
      for (int c = 0; c <= chunks && ok; ++c) {
        const int cq = c - 1;  // Q of the chunk before, once Q of the one before that was read
        if (!local && cq >= 0) {
          if (cq >= 1 && !(ok = la_wait(&bar->o1, (cq - 1) & 1, abort))) break;
          mbar_expect_tx(&bar->full_q, SM::Q);
          load(&mq, sq, DK, &bar->full_q, ps.cq, cq);
          ++q_loads;
        }
        if (c < chunks) {
          // K, V of chunk c once the products of chunk c - 2 have read their stage
          if (c >= 2 && !(ok = la_wait(&bar->o2[c & 1], ((c - 2) >> 1) & 1, abort))) break;
          mbar_expect_tx(&bar->full_kv[c & 1], SM::K + SM::V);
          load(&mk, sk + (c & 1) * SM::K, DK, &bar->full_kv[c & 1], ps.ck, c);
          load(&mv, sv + (c & 1) * SM::V, DV, &bar->full_kv[c & 1], ps.cv, c);
          ++kv_loads;
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && chunks > 0) {
      // ---------------- MMA issuer ----------------
      constexpr uint32_t id_p = idesc_bf16_f32(LC, LC), id_v = idesc_bf16_f32(LC, DV) | IDESC_B_MN;
      const uint32_t q0 = smem_u32(sq), e0 = smem_u32(se);
      bool ok = !(ps.stall && !la_wait(&bar->stall, 0, abort));
      for (int c = 0; c < chunks && ok; ++c) {
        const uint32_t ph = c & 1;
        const uint32_t k0 = smem_u32(sk + ph * SM::K), v0 = smem_u32(sv + ph * SM::V);
        auto u_piece = [&](uint32_t at, bool first) {
#pragma unroll
          for (int kk = 0; kk < LC / 16; ++kk)
            umma_bf16_ta(tmem + TM_U, tmem + at + kk * 8, sdesc_mn_sw128(v0 + kk * 2048, LA_BLOCK), id_v,
                         (first && kk == 0) ? 0u : 1u);
        };
        if (!(ok = la_wait(&bar->full_kv[ph], (c >> 1) & 1, abort))) break;
        const bool state = init != nullptr || c > 0;
        if (!local) {
          if (!(ok = la_wait(&bar->full_q, ph, abort))) break;
          if (c > 0 && !(ok = la_wait(&bar->o2[ph ^ 1], ((c - 1) >> 1) & 1, abort))) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk) {
            const uint32_t o = (kk >> 2) * LA_BLOCK + (kk & 3) * 32;
            umma_bf16(tmem + TM_P, sdesc_k_sw128(q0 + o), sdesc_k_sw128(k0 + o), id_p, kk != 0 ? 1u : 0u);
          }
          umma_commit(&bar->p);
          if (!(ok = la_wait(&bar->next, ph, abort))) break;
          tc_fence_after();
          if (state) {
#pragma unroll
            for (int pc = 0; pc < 2; ++pc)
#pragma unroll
              for (int kk = 0; kk < DK / 16; ++kk)
                umma_bf16(tmem + TM_O, sdesc_k_sw128(q0 + (kk >> 2) * LA_BLOCK + (kk & 3) * 32),
                          sdesc_mn_sw128(e0 + pc * SM::E + kk * 2048, DK * 128), id_v, (pc | kk) != 0 ? 1u : 0u);
          }
          umma_commit(&bar->o1);
        }
        if (!(ok = la_wait(&bar->kt, ph, abort))) break;
        tc_fence_after();
        u_piece(TM_K0, true);
        u_piece(TM_K1, false);
        umma_commit(&bar->u1);
        if (!(ok = la_wait(&bar->mid, ph, abort))) break;
        tc_fence_after();
        u_piece(TM_K0, false);
        umma_commit(&bar->u2);
        if (!local) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int pc = 0; pc < 2; ++pc)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_bf16_ta(tmem + TM_O, tmem + TM_P + hf * 64 + pc * 32 + kk * 8,
                             sdesc_mn_sw128(v0 + (hf * 4 + kk) * 2048, LA_BLOCK), id_v,
                             (state || (hf | pc | kk) != 0) ? 1u : 0u);
        }
        umma_commit(&bar->o2[ph]);  // also: this chunk's K and V have been read
      }
      umma_commit(&bar->drain);  // completes once every MMA issued above has finished
      drain_wait(&bar->drain, 0);
    }
  } else {
    // ---------------- elementwise work ----------------
    const int quad = warp & 3, hf = (warp - 2) >> 2;
    const int row = quad * 32 + lane;               // TMEM lane: token row, or state row
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    constexpr int EC = DV / 2;                      // columns of the state and of O per thread
    const int j0 = hf * EC;
    const int mt = threadIdx.x - 64;                // 0 .. 255
    for (int j = mt; j <= LC; j += LA_MATH_WARPS * 32) pw[j] = decay_pow(ld, (float)j);

    float S[EC];
#pragma unroll
    for (int j = 0; j < EC; ++j) S[j] = 0.f;
    if (init && row < a.d) {
#pragma unroll
      for (int j = 0; j < EC; ++j)
        if (j0 + j < a.dv) S[j] = init[row * isi + (j0 + j) * isj] * in_scale;
    }
    auto put_state = [&]() {  // E as two bf16 pieces, the second operand of Q E
      if (row < DK) {
#pragma unroll
        for (int j = 0; j < EC; j += 8) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            hi[u] = pack_bf16(S[j + 2 * u], S[j + 2 * u + 1]);
            lo[u] = pack_bf16(S[j + 2 * u] - low_f(hi[u]), S[j + 2 * u + 1] - high_f(hi[u]));
          }
          const uint32_t o = sw_off(row, j0 + j, DK);
          *reinterpret_cast<uint4*>(se + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(se + SM::E + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_async_smem();
    };
    if (init) put_state();
    // the decay table is shared by the math warps only
    asm volatile("bar.sync 1, %0;" ::"n"(LA_MATH_WARPS * 32) : "memory");
    if (lane == 0) mbar_arrive(&bar->next);

    const char* const op = (const char*)a.o.p + ((long long)b * a.o.sb + (long long)h * a.o.sh) * 2;
    for (int c = 0; c < chunks; ++c) {
      const uint32_t ph = c & 1;
      const int m = min(LC, t1 - t0 - c * LC);      // tokens of this chunk
      const int r0 = a.reverse ? LC - m : 0;        // their rows: [r0, r0 + m)
      const bool ready = c == 0 && g == 0 && a.in_ready;
      if (!la_wait_warp(&bar->full_kv[ph], (c >> 1) & 1, abort, lane)) break;
      const uint8_t* kt = sk + ph * SM::K;
      uint8_t* vt = sv + ph * SM::V;

      // weighted keys a^(m-1-s) k_s, transposed: thread = state row, 64 of the tokens
      uint32_t khi[32];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t md[16], lo[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float x[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int s = hf * 64 + q * 32 + 2 * i + u;
            const int e = a.reverse ? s - r0 : m - 1 - s;   // exponent; < 0 outside the chunk
            float kv = 0.f;
            if (DK == 128 || row < DK)
              kv = __uint_as_float((uint32_t)(*reinterpret_cast<const uint16_t*>(kt + sw_off(s, row, LC))) << 16);
            x[u] = e >= 0 ? kv * pw[e < 0 ? 0 : e] : 0.f;
          }
          const uint32_t hi = pack_bf16(x[0], x[1]);
          khi[q * 16 + i] = hi;
          x[0] -= low_f(hi);
          x[1] -= high_f(hi);
          md[i] = pack_bf16(x[0], x[1]);
          lo[i] = pack_bf16(x[0] - low_f(md[i]), x[1] - high_f(md[i]));
        }
        tmem_st16(lanes + TM_K0 + hf * 32 + q * 16, lo);
        tmem_st16(lanes + TM_K1 + hf * 32 + q * 16, md);
      }
      if (m < LC && !a.reverse) {
        // rows behind the sequence's end may hold anything, NaN included, which a weight of
        // zero does not remove: V's rows are cleared (the weights above drop K's)
        for (int x = mt; x < (LC - m) * (DV / 8); x += LA_MATH_WARPS * 32) {
          const int r = m + x / (DV / 8), cj = (x % (DV / 8)) * 8;
          *reinterpret_cast<uint4*>(vt + sw_off(r, cj, LC)) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_async_smem();
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->kt);

      if (!local) {
        // P pieces in place: thread = token row, 64 of the columns
        if (!la_wait_warp(&bar->p, ph, abort, lane)) break;
        tc_fence_after();
        uint32_t hi[32], lo[32];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t v[32];
          tmem_ld32(lanes + TM_P + hf * 64 + q * 32, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int s = hf * 64 + q * 32 + 2 * i + u;
              const int e = a.reverse ? s - row : row - s;
              x[u] = e >= 0 ? __uint_as_float(v[2 * i + u]) * pw[e < 0 ? 0 : e] : 0.f;
            }
            hi[q * 16 + i] = pack_bf16(x[0], x[1]);
            lo[q * 16 + i] = pack_bf16(x[0] - low_f(hi[q * 16 + i]), x[1] - high_f(hi[q * 16 + i]));
          }
        }
        tmem_st32(lanes + TM_P + hf * 64, hi);
        tmem_st32(lanes + TM_P + hf * 64 + 32, lo);
        // O = Q E so far: decay each token's row
        if (init != nullptr || c > 0) {
          if (!la_wait_warp(&bar->o1, ph, abort, lane)) break;
          tc_fence_after();
          const int u = a.reverse ? LC - 1 - row : row;
          const float f = pw[u + (ready ? 0 : 1)];
#pragma unroll
          for (int q = 0; q < EC; q += 32) {
            uint32_t v[32];
            tmem_ld32(lanes + TM_O + j0 + q, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
            tmem_st32(lanes + TM_O + j0 + q, v);
          }
        }
      }
      // the keys' high piece takes the low one's place once that has been read
      if (!la_wait_warp(&bar->u1, ph, abort, lane)) break;
      tc_fence_after();
      tmem_st32(lanes + TM_K0 + hf * 32, khi);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->mid);

      // E' = a^len E + U
      if (!la_wait_warp(&bar->u2, ph, abort, lane)) break;
      tc_fence_after();
      {
        const float e = (float)(m - (ready ? 1 : 0));
        const float fhi = decay_pow(ld, e);
#pragma unroll
        for (int q = 0; q < EC; q += 32) {
          uint32_t v[32];
          tmem_ld32(lanes + TM_U + j0 + q, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) S[q + i] = fmaf(S[q + i], fhi, __uint_as_float(v[i]));
        }
      }
      if (!local) {
        if (c + 1 < chunks) put_state();
        if (!la_wait_warp(&bar->o2[ph], (c >> 1) & 1, abort, lane)) break;
        tc_fence_after();
        const long long t = tile_t(c) + row;
        char* dst = const_cast<char*>(op) + t * a.o.st * 2;
        const bool live = row >= r0 && row < r0 + m;
#pragma unroll
        for (int q = 0; q < EC; q += 32) {
          uint32_t v[32];
          tmem_ld32(lanes + TM_O + j0 + q, v);
          tmem_wait_ld();
          if (live) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              if (j0 + q + i < a.dv) {
                uint32_t y[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                  y[u] = pack_bf16(__uint_as_float(v[i + 2 * u]) * a.out_scale,
                                   __uint_as_float(v[i + 2 * u + 1]) * a.out_scale);
                *reinterpret_cast<uint4*>(dst + (j0 + q + i) * 2) = make_uint4(y[0], y[1], y[2], y[3]);
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->next);
      }
    }
    // last state: the segment's slot, or the caller's
    float* dst = local ? a.slots + ((size_t)bh * a.nseg + g) * cells
                       : (a.s_out && g == a.nseg - 1 ? a.s_out + (size_t)bh * cells : nullptr);
    if (dst && row < a.d && !*abort) {
      const long long osi = local ? a.dv : a.si, osj = local ? 1 : a.sj;
      const float w = local || n == 0 ? 1.f : a.st_scale * (a.out_decay ? decay_pow(ld, 1.f) : 1.f);
#pragma unroll
      for (int j = 0; j < EC; ++j)
        if (j0 + j < a.dv) dst[row * osi + (j0 + j) * osj] = S[j] * w;
    }
  }

  // ---------------- teardown ----------------
  __syncwarp();
  if (warp == 0 && lane == 0 && *abort) {
    // let the copies this CTA issued land before its shared memory goes away
    for (int c = kv_loads < 2 ? 0 : kv_loads - 2; c < kv_loads; ++c) drain_wait(&bar->full_kv[c & 1], (c >> 1) & 1);
    if (q_loads > 0) drain_wait(&bar->full_q, (q_loads - 1) & 1);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TM_COLS);
  }
  if (threadIdx.x == 0 && *abort) raise_status(&g_la_status, nullptr, DEV_TIMEOUT);
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return (EncodeFn)p;
  }();
  return fn;
}

// bf16 heads [B][H][T][w] as a 4-D map, box 64 x 128 tokens, 128-byte swizzle, zeros outside
// (columns past w, tokens past T or before 0).  A broadcast axis becomes an axis of 1.
bool heads_map(CUtensorMap* map, const fwpkm_heads& x, const ScanArgs& a, int w, TcCoord* cc) {
  EncodeFn fn = encoder();
  if (!fn) return false;
  cc->h = a.H > 1 && x.sh != 0;
  cc->b = a.B > 1 && x.sb != 0;
  cuuint64_t dims[4] = {(cuuint64_t)w, (cuuint64_t)a.T, (cuuint64_t)(cc->h ? a.H : 1), (cuuint64_t)(cc->b ? a.B : 1)};
  cuuint64_t strides[3] = {(cuuint64_t)(a.T > 1 ? x.st * 2 : 16), (cuuint64_t)(cc->h ? x.sh * 2 : 16),
                           (cuuint64_t)(cc->b ? x.sb * 2 : 16)};
  cuuint32_t box[4] = {64, LC, 1, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, x.p, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows on the 16-byte grid along every axis in use; a token stride of 0 is not taken (TMA has
// no such axis) and strides stay below TMA's 2^40 bytes.
bool grid16(const fwpkm_heads& x, const ScanArgs& a) {
  const long long most = 1ll << 38;
  return ((uintptr_t)x.p & 15) == 0 && (a.T <= 1 || (x.st % 8 == 0 && x.st > 0 && x.st < most)) &&
         (a.H <= 1 || (x.sh % 8 == 0 && x.sh < most)) && (a.B <= 1 || (x.sb % 8 == 0 && x.sb < most));
}

template <int DK, int DV>
int go_tc(const TcPass& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
  if (!raise_smem_limit((const void*)scan_tc_kernel<DK, DV>, TcSmem<DK, DV>::bytes)) return -1;
  launch_k(scan_tc_kernel<DK, DV>, dim3((unsigned)(p.a.B * p.a.H), p.local ? p.a.nseg - 1 : p.a.nseg), LA_THREADS,
           TcSmem<DK, DV>::bytes, s, q, k, v, p);
  return 1;
}

int go_tc_shape(const TcPass& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
  if (p.a.d <= 64) return p.a.dv <= 64 ? go_tc<64, 64>(p, q, k, v, s) : go_tc<64, 128>(p, q, k, v, s);
  return p.a.dv <= 64 ? go_tc<128, 64>(p, q, k, v, s) : go_tc<128, 128>(p, q, k, v, s);
}

}  // namespace

// bf16, widths up to 128 in whole 16-byte vectors, rows on the 16-byte grid, and enough
// tokens that a chunk of 128 is not mostly padding.
bool scan_tc_shape(const ScanArgs& a, int dtype) {
  return dtype == FWPKM_BF16 && a.d <= 128 && a.dv <= 128 && a.d % 8 == 0 && a.dv % 8 == 0 && a.T >= 32;
}
bool scan_tc_takes(const ScanArgs& a, int dtype) {
  return scan_tc_shape(a, dtype) && grid16(a.q, a) && grid16(a.k, a) && grid16(a.v, a) && grid16(a.o, a);
}

// Segments: one when the heads fill half the GPU (a second wave or the extra pass over K and
// V would cost more), else one CTA per SM, of at least two chunks each.
int scan_tc_segments(const ScanArgs& a) {
  const int heads = a.B * a.H;
  if (heads > 148 / 2) return 1;
  int n = 148 / heads;
  const int most = a.T / (2 * LC);
  if (n > most) n = most;
  return n < 2 ? 1 : n;
}

int launch_scan_tc(const ScanArgs& a0, cudaStream_t s) {
  TcPass p = {};
  p.a = a0;
  p.a.nseg = scan_tc_segments(a0);
  p.a.seg_len = p.a.nseg > 1 ? ((a0.T + p.a.nseg - 1) / p.a.nseg + LC - 1) / LC * LC : a0.T;
  CUtensorMap q, k, v;
  if (!heads_map(&q, a0.q, a0, a0.d, &p.cq) || !heads_map(&k, a0.k, a0, a0.d, &p.ck) ||
      !heads_map(&v, a0.v, a0, a0.dv, &p.cv)) {
    fprintf(stderr, "fwpkm: cuTensorMapEncodeTiled failed\n");
    return -1;
  }
  int nl = 0;
  p.stall = take_test_stall();
  if (p.a.nseg > 1) {
    p.local = 1;
    if (go_tc_shape(p, q, k, v, s) < 0) return -1;
    nl += 1 + launch_scan_combine(p.a, s);
    p.local = 0;
    p.stall = 0;
  }
  if (go_tc_shape(p, q, k, v, s) < 0) return -1;
  return nl + 1;
}

int take_scan_status() {
  int st = DEV_OK;
  if (cudaMemcpyFromSymbol(&st, g_la_status, sizeof(int)) != cudaSuccess) return -1;
  if (st != DEV_OK) {
    const int ok = DEV_OK;
    if (cudaMemcpyToSymbol(g_la_status, &ok, sizeof(int)) != cudaSuccess) return -1;
  }
  return st;
}

}  // namespace fwpkm
