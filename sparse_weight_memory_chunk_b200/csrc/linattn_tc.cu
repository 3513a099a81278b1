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
// a^(t-s) = R_t B_s with B_s = a^(63-s), R_t = a^(t-63), so P is weighted by column, E enters
// as a^64 E, and R_t multiplies the finished row of O.  (About the middle of the chunk the weights
// reach e^30 either way at most; about its end they reached e^-60, where scores of 1e-12 left
// fp32's range.)  A head whose a^128 is out of range (|log a^128| > LA_RANGE) takes the weights
// element by element and scales Q E in place.
//
// Precision: the inputs are bf16, exact operands.  P (weighted) and E enter their products as two
// bf16 pieces, the upper half of the float and what that leaves (2^-16 left out at most), so O is off by
// its own rounding on the way out (1.66e-3 of its norm; rounded once each, P and E made it 2.35e-3, and a
// chunk 0.5 us shorter).  The weighted keys of U are hi + mid + lo where the state is handed on in fp32 (exact to fp32),
// else two pieces.  U adds the small pieces first, so few of the accumulator's roundings (which
// truncate) are at full size: the state is 9e-8 off against 6e-7 the other way round.  E is
// kept in fp32 registers, a chunk's decay a number whose rounding is carried into the next chunk's (the same number
// every time was off by up to 2^-25 a chunk, always the same way), and U is a fresh accumulator per chunk, so the tensor cores' running
// sums span one chunk only.
//
// CTA = one head (and segment): warp 0 issues TMA loads and stores (K, V two stages, Q one, the
// rows of O from the room of the chunk's V; a pass that only forms segment states: K, V three stages), warp 1 owns TMEM and issues the MMAs (one thread),
// warps 4-11 weight the keys, 12-19 the scores, 20-27 carry the state and the output: a warp
// reads TMEM lanes 32 (w % 4).. and one half of the columns.  TMEM (512 columns): P fp32,
// overwritten in place by its pieces' bf16 pairs (operand A of P V); O; U; two pieces of the
// weighted, transposed keys (operand A of U; the high piece waits in registers and takes the
// low one's place).  Per chunk c, in order:
//   MMA     U lo, mid(c)   P(c)   U hi(c)        Q E lo, hi(c)        P V lo, hi(c)
//   keys          K hi(c)              K pieces(c+1)
//   scores                        P pieces(c)
//   state   O out(c-1)                 E(c)      E pieces(c+1)
// so the MMAs of a chunk (8 products of 128^3, 512 cycles each at the dense rate; 7 where no state
// leaves) follow one another while the groups work beside them.  (With the groups' steps done in
// turn by the same warps a chunk took the sum of their latencies, 5.5 us of 148 heads at
// d = d_v = 128.)  A pass that only forms segment states has TMEM to spare and keeps two sets of
// key pieces, so that weighting a chunk's keys overlaps the products of the one before.
// Bound: for d = d_v = 128 a chunk is 128 KB, 3.0 us of an SM's share of the copy bandwidth; 148
// heads of 8192 tokens take 4.8 us a chunk (62% of it), 5.2 with the final state: what is left is
// the chain state -> E pieces -> Q E -> next state, and keys -> U -> next keys.
#include <cstdio>

#include "linattn.cuh"
#include "sm100.cuh"

namespace fwpkm {

using namespace sm100;

namespace {

constexpr int LC = 128;                  // tokens per chunk
// Warps by warpgroups (register shares go by warpgroup): four of roles (two idle), eight for the
// weighted keys, eight for the scores, eight for the state and the output.  896 threads launch
// at 72 registers and redistribute them.
constexpr int LA_ROLE_WARPS = 4, LA_GROUP_WARPS = 8, LA_GROUP = LA_GROUP_WARPS * 32;
constexpr int LA_THREADS = LA_ROLE_WARPS * 32 + 3 * LA_GROUP;
constexpr int LA_ROLE_REGS = 56, LA_KEY_REGS = 64, LA_SCORE_REGS = 64, LA_STATE_REGS = 96;
static_assert(LA_ROLE_WARPS * 32 * LA_ROLE_REGS + LA_GROUP * (LA_KEY_REGS + LA_SCORE_REGS + LA_STATE_REGS) <=
                  LA_THREADS * 72, "registers");
constexpr uint64_t LA_TIMEOUT_NS = 200ull * 1000 * 1000;  // any single wait
constexpr int LA_MID = LC / 2 - 1;       // the position that column weights count from
constexpr float LA_RANGE = 60.f;         // largest |log a^128| taken through column weights
constexpr int LA_BLOCK = LC * 128;       // bytes of a 64-column block of 128 rows

__device__ int g_la_status = DEV_OK;     // latched by a kernel whose wait ran out

// TMEM columns
constexpr uint32_t TM_P = 0, TM_O = 128, TM_U = 256, TM_K0 = 384, TM_COLS = 512;  // (a piece: 64)

struct TcBars {
  uint64_t full_q, full_k[3], full_v[3], free_k[3], o2[2], kt[2], u2[2];
  uint64_t p, o1, staged, khi, u1, mid, est, ofree, ufree, cleared, drain, stall;
};

template <int DK, int DV>
struct TcSmem {
  static constexpr int Q = LC * DK * 2, K = LC * DK * 2, V = LC * DV * 2, E = DK * DV * 2;
  // E's two pieces; in between, states pass through their room in fp32.  (The low one's place is as
  // large as a stage of V, whose third it is where only states are formed.)
  static constexpr int off_k = Q, off_v = off_k + 2 * K, off_elo = off_v + 2 * V, off_e = off_elo + V;
  static constexpr int off_tab = off_e + E;
  static_assert(V >= E && V + E >= DK * DV * 4, "room for a state in fp32");
  static constexpr int need = off_tab + 4 * (3 * LC + 4) + (int)sizeof(TcBars) + 16 + 1024;
  // one CTA per SM: each holds all of TMEM
  static constexpr int bytes = need > 120 * 1024 ? need : 120 * 1024;
};

// Wait for a phase; false once any role gave up (or this wait ran out, which raises abort).
__device__ __forceinline__ bool la_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  uint32_t n = 0;
  uint64_t t0 = 0;
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if ((++n & 255u) == 0) {
      const uint64_t t = globaltimer();
      if (t0 == 0) t0 = t;
      if (*abort || t - t0 > LA_TIMEOUT_NS) {
        *abort = 1;
        return false;
      }
    }
  }
  return true;
}
// The same for a whole warp, converged afterwards: true only if every lane saw the phase.
__device__ __forceinline__ bool la_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, la_wait(bar, parity, abort)) != 0;
}
// Several waits at once by a converged warp: lane i < n waits for the i-th (bar, parity).
struct Wait {
  uint64_t* bar;
  uint32_t parity;
};
__device__ __forceinline__ bool la_wait_each(int lane, volatile int* abort, Wait a, Wait b, Wait c, Wait d) {
  const Wait w = lane == 0 ? a : lane == 1 ? b : lane == 2 ? c : d;
  return __all_sync(0xffffffffu, la_wait(w.bar, w.parity, abort)) != 0;
}
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer() - t0 > LA_TIMEOUT_NS) return;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {  // rounded to nearest
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The upper halves of two floats (bf16, truncated) as a pair, and what truncation leaves.
__device__ __forceinline__ uint32_t pack_high(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}
// x, y less the pair of bf16 in p, exact (one mixed-precision operation each).
__device__ __forceinline__ void below_high(uint32_t p, float& x, float& y) {
  asm("{\n .reg .b16 l, u, m;\n mov.b32 {l, u}, %2;\n mov.b16 m, 0xBF80;\n fma.rn.f32.bf16 %0, l, m, %0;\n "
      "fma.rn.f32.bf16 %1, u, m, %1;\n}\n"
      : "+f"(x), "+f"(y)
      : "r"(p));
}

// Byte of element (row, col) in a tile of 64-column blocks of `rows` 128-byte rows, swizzled.
__device__ __forceinline__ uint32_t sw_off(int row, int col, int rows) {
  return (uint32_t)((col >> 6) * rows * 128 + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4) + (col & 7) * 2);
}

struct TcCoord {
  int h, b;  // 1, or 0 where the tensor is broadcast along the axis
};
struct TcPass {
  ScanArgs a;
  TcCoord cq, ck, cv, co;
  int local, stall;
};

template <int DK, int DV>
__global__ void __launch_bounds__(LA_THREADS, 1)
scan_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo, const TcPass ps) {
  using SM = TcSmem<DK, DV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *sq = smem, *sk = smem + SM::off_k, *sv = smem + SM::off_v, *selo = smem + SM::off_elo, *se = smem + SM::off_e;
  float* bw = (float*)(smem + SM::off_tab);  // [LC] column weights B_s
  float* kw = bw + LC;                       // [LC] weights of the chunk's keys
  float* pw = kw + LC;                       // [LC + 1] a^j
  TcBars* bar = (TcBars*)(pw + LC + 4);
  uint32_t* tmem_slot = (uint32_t*)(bar + 1);
  volatile int* abort = (volatile int*)(tmem_slot + 1);

  const ScanArgs& a = ps.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool local = ps.local != 0;
  // whether this segment's state leaves in fp32 (by itself, or through the states after it)
  const bool three = a.s_out != nullptr && (local || (int)blockIdx.y == a.nseg - 1);
  const int bh = blockIdx.x, g = blockIdx.y;
  const int b = bh / a.H, h = bh - b * a.H;

  if (threadIdx.x == 0) {
    mbar_init(&bar->full_q, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&bar->full_k[i], 1);
      mbar_init(&bar->full_v[i], 1);
      mbar_init(&bar->free_k[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->o2[i], 1);
      mbar_init(&bar->kt[i], LA_GROUP_WARPS);
      mbar_init(&bar->u2[i], 1);
    }
    mbar_init(&bar->p, 1);
    mbar_init(&bar->o1, 1);
    mbar_init(&bar->khi, LA_GROUP_WARPS);
    mbar_init(&bar->u1, 1);
    mbar_init(&bar->mid, LA_GROUP_WARPS);
    mbar_init(&bar->est, LA_GROUP_WARPS);
    mbar_init(&bar->ofree, LA_GROUP_WARPS);
    mbar_init(&bar->ufree, LA_GROUP_WARPS);
    mbar_init(&bar->cleared, LA_GROUP_WARPS);
    mbar_init(&bar->staged, LA_GROUP_WARPS);
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
  const bool fast = fabsf(ld) * (float)LC <= LA_RANGE;
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
  // first token row of the tile of chunk c (ascending, or ending at the chunk's first token),
  // and the chunk's tokens
  auto tile_t = [&](int c) { return a.reverse ? n - (t0 + c * LC) - LC : t0 + c * LC; };
  auto tokens = [&](int c) { return min(LC, t1 - t0 - c * LC); };

  // K and V: two stages, and where only states are formed a third in the room of Q and of E's low piece
  const int stages = local ? 3 : 2;
  auto stage = [&](int c) { return local ? c % 3 : c & 1; };
  auto stage_ph = [&](int c) { return (uint32_t)((local ? c / 3 : c >> 1) & 1); };
  auto k_rows = [&](int st) { return st == 2 ? sq : sk + st * SM::K; };
  auto v_rows = [&](int st) { return st == 2 ? selo : sv + st * SM::V; };

  int k_loads = 0, v_loads = 0, q_loads = 0;  // producer: chunks whose loads were issued
  if (warp < LA_ROLE_WARPS) regs_dec<LA_ROLE_REGS>();
  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA: loads of K, V, Q; stores of O ----------------
      auto load = [&](const CUtensorMap* m, uint8_t* dst, int width, uint64_t* fb, const TcCoord& cc, int c) {
        mbar_expect_tx(fb, (uint32_t)(LC * width * 2));
        for (int x = 0; x < width; x += 64)
          tma_load_4d(dst + (x >> 6) * LA_BLOCK, m, fb, x, tile_t(c), h * cc.h, b * cc.b);
      };
      auto load_k = [&](int c) {
        if (c >= chunks) return;
        load(&mk, k_rows(stage(c)), DK, &bar->full_k[stage(c)], ps.ck, c);
        ++k_loads;
      };
      auto load_v = [&](int c) {
        if (c >= chunks) return;
        load(&mv, v_rows(stage(c)), DV, &bar->full_v[stage(c)], ps.cv, c);
        ++v_loads;
      };
      auto load_q = [&](int c) {
        if (local || c >= chunks) return;
        load(&mq, sq, DK, &bar->full_q, ps.cq, c);
        ++q_loads;
      };
      load_k(0);
      load_v(0);
      load_q(0);
      for (int c = 1; c < stages; ++c) {
        load_k(c);
        load_v(c);
      }
      for (int c = 0; c < chunks; ++c) {
        if (!la_wait(&bar->free_k[stage(c)], stage_ph(c), abort)) break;
        load_k(c + stages);
        if (local) {
          load_v(c + stages);
          continue;
        }
        if (!la_wait(&bar->o1, c & 1, abort)) break;
        load_q(c + 1);
        // O's rows lie in the chunk's stage of V, which is loaded again once they have left
        if (!la_wait(&bar->staged, c & 1, abort)) break;
        if (tokens(c) == LC) {  // (the rows of a partial chunk, the last, are written by the state warps)
          for (int x = 0; x < DV; x += 64)
            tma_store_4d(&mo, v_rows(stage(c)) + (x >> 6) * LA_BLOCK, x, tile_t(c), h * ps.co.h, b * ps.co.b);
          bulk_commit();
          bulk_wait_read();
        }
        load_v(c + 2);
      }
      bulk_wait_all();
    }
  } else if (warp == 1) {
    if (chunks > 0) {
      // ---------------- MMA issuer: the warp waits together, one lane issues ----------------
      constexpr uint32_t id_p = idesc_bf16_f32(LC, LC), id_v = idesc_bf16_f32(LC, DV) | IDESC_B_MN;
      const uint32_t q0 = smem_u32(sq), e0 = smem_u32(se), elo0 = smem_u32(selo);
      bool ok = !(ps.stall && !la_wait_warp(&bar->stall, 0, abort));
      for (int c = 0; c < chunks && ok; ++c) {
        const uint32_t ph = c & 1, ph2 = (c >> 1) & 1;
        const int st = stage(c);
        const uint32_t k0 = smem_u32(k_rows(st)), v0 = smem_u32(v_rows(st)), st_ph = stage_ph(c);
        const uint64_t vd = sdesc_mn_sw128(v0, LA_BLOCK);   // + 128 per 16 tokens (16-byte units)
        auto u_piece = [&](uint32_t at, bool first) {
#pragma unroll 2
          for (int kk = 0; kk < LC / 16; ++kk)
            umma_bf16_ta(tmem + TM_U, tmem + at + kk * 8, vd + kk * 128, id_v, (first && kk == 0) ? 0u : 1u);
        };
        const bool state = init != nullptr || c > 0;
        {  // (ufree: the U of the chunk before has been taken up by the state)
          const Wait kt{&bar->kt[ph], ph2};
          ok = la_wait_each(lane, abort, kt, {&bar->full_v[st], st_ph}, {&bar->full_k[st], st_ph},
                            c == 0 ? kt : Wait{&bar->ufree, ph ^ 1});
        }
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t at = local && ph ? TM_P : TM_K0;
          u_piece(at, true);
          u_piece(at + 64, false);
          if (local && three) u_piece(TM_O + ph * 64, false);
          umma_commit(three && !local ? &bar->u1 : &bar->u2[ph]);
          if (local) umma_commit(&bar->free_k[st]);  // K and V
        }
        __syncwarp();
        if (local) continue;
        {
          // (o2 of the chunk before: P's columns are free)
          const Wait q{&bar->full_q, ph};
          ok = la_wait_each(lane, abort, q, c == 0 ? q : Wait{&bar->o2[ph ^ 1], (uint32_t)(((c - 1) >> 1) & 1)}, q, q);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t qd = sdesc_k_sw128(q0), kd = sdesc_k_sw128(k0);
#pragma unroll
            for (int x = 0; x < DK / 64; ++x)
#pragma unroll 2
              for (int kk = 0; kk < 4; ++kk)
                umma_bf16(tmem + TM_P, qd + x * (LA_BLOCK >> 4) + kk * 2, kd + x * (LA_BLOCK >> 4) + kk * 2, id_p,
                          (x | kk) != 0 ? 1u : 0u);
            umma_commit(&bar->p);
            umma_commit(&bar->free_k[st]);
          }
          __syncwarp();
        }
        if (three) {
          if (!(ok = la_wait_warp(&bar->khi, ph, abort))) break;
          tc_fence_after();
          if (elect_one()) {
            u_piece(TM_K0, false);
            umma_commit(&bar->u2[ph]);
          }
          __syncwarp();
        }
        // E in bf16, and O's columns (the rows of the previous chunk have left)
        const Wait est{&bar->est, ph};
        ok = la_wait_each(lane, abort, est, c == 0 ? est : Wait{&bar->ofree, ph ^ 1}, est, est);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          if (state) {
            const uint64_t qd = sdesc_k_sw128(q0);
#pragma unroll
            for (int piece = 0; piece < 2; ++piece) {
              const uint64_t ed = sdesc_mn_sw128(piece == 0 ? elo0 : e0, DK * 128);
#pragma unroll 2
              for (int kk = 0; kk < DK / 16; ++kk)
                umma_bf16(tmem + TM_O, qd + (kk >> 2) * (LA_BLOCK >> 4) + (kk & 3) * 2, ed + kk * 128, id_v,
                          (piece | kk) != 0 ? 1u : 0u);
            }
          }
          umma_commit(&bar->o1);  // also: Q and E have been read
        }
        __syncwarp();
        if (!(ok = la_wait_warp(&bar->mid, ph, abort))) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int piece = 0; piece < 2; ++piece)
#pragma unroll 2
            for (int kk = 0; kk < LC / 16; ++kk)  // (of every 32 columns of P, 16 of high and 16 of low pieces)
              umma_bf16_ta(tmem + TM_O, tmem + TM_P + (kk >> 1) * 32 + (1 - piece) * 16 + (kk & 1) * 8, vd + kk * 128,
                           id_v, (state || (piece | kk) != 0) ? 1u : 0u);
          umma_commit(&bar->o2[ph]);
        }
        __syncwarp();
      }
      if (elect_one()) umma_commit(&bar->drain);  // completes once every MMA issued above has finished
      __syncwarp();
      drain_wait(&bar->drain, 0);
    }
  } else if (warp >= LA_ROLE_WARPS && warp < LA_ROLE_WARPS + LA_GROUP_WARPS) {
    regs_dec<LA_KEY_REGS>();
    // ---------------- weighted keys a^(m-1-s) k_s, transposed: 32 state rows x 64 tokens a warp
    const int quad = warp & 3, hf = (warp - LA_ROLE_WARPS) >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16) + hf * 32;
    const int mt = threadIdx.x - LA_ROLE_WARPS * 32;
    const uint32_t k_at = (uint32_t)((quad >> 1) * LA_BLOCK + (hf * 64 + (lane & 7)) * 128 +
                                     ((((quad & 1) * 4 + (lane >> 3)) ^ (lane & 7)) << 4));
    // weights of a chunk of m tokens (descending: by rows from the other end)
    auto put_weights = [&](int m) {
      if (mt < LC) {
        const int e = a.reverse ? mt - (LC - m) : m - 1 - mt;
        kw[mt] = e < 0 ? 0.f : decay_pow(ld, (float)e);
      }
    };
    put_weights(LC);
    asm volatile("bar.sync 3, %0;" ::"n"(LA_GROUP) : "memory");
    for (int c = 0; c < chunks; ++c) {
      const uint32_t ph = c & 1, ph2 = (c >> 1) & 1;
      const int m = tokens(c);
      const int st = stage(c);
      if (!la_wait_warp(&bar->full_k[st], stage_ph(c), abort)) break;
      uint8_t* kb = k_rows(st);
      if (m < LC) {
        // (a head has one such chunk, its last.)  Rows behind the sequence's end may hold
        // anything, NaN included, which a weight of zero does not remove: they are cleared
        // (before a sequence's start, where descending tiles end, TMA fills zeros)
        if (!la_wait_warp(&bar->full_v[st], stage_ph(c), abort)) break;
        if (!a.reverse) {
          for (int x = mt; x < (LC - m) * (DK / 8); x += LA_GROUP)
            *reinterpret_cast<uint4*>(kb + sw_off(m + x / (DK / 8), (x % (DK / 8)) * 8, LC)) = make_uint4(0u, 0u, 0u, 0u);
          for (int x = mt; x < (LC - m) * (DV / 8); x += LA_GROUP)
            *reinterpret_cast<uint4*>(v_rows(st) + sw_off(m + x / (DV / 8), (x % (DV / 8)) * 8, LC)) =
                make_uint4(0u, 0u, 0u, 0u);
        }
        // every warp has read the full chunks' weights before any passes the first barrier
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->cleared);
        if (!la_wait_warp(&bar->cleared, 0, abort)) break;
        put_weights(m);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->cleared);
        if (!la_wait_warp(&bar->cleared, 1, abort)) break;
      }
      // the U that read the pieces' columns before has finished: the chunk before's, or of a pass
      // that forms states only, which has two sets of columns, the one's before that
      if (local ? c > 1 && !la_wait_warp(&bar->u2[ph], ph2 ^ 1, abort)
                : c > 0 && !la_wait_warp(&bar->u2[ph ^ 1], ((c - 1) >> 1) & 1, abort))
        break;
      tc_fence_after();
      const uint32_t kt = smem_u32(kb) + k_at, pieces = local && ph ? TM_P : TM_K0;
      uint32_t khi[8][4];                           // [16 tokens, lane half][.]
#pragma unroll
      for (int q = 0; q < 4; ++q) {                 // 16 tokens
        uint32_t md[2][4], lo[2][4];
#pragma unroll
        for (int sb = 0; sb < 2; ++sb) {
          uint32_t x4[4] = {0u, 0u, 0u, 0u};
          if (DK == 128 || quad < 2) ldmatrix_x4_trans(kt + (q * 2 + sb) * 1024, x4);
          const float2 w = *reinterpret_cast<const float2*>(kw + hf * 64 + (q * 2 + sb) * 8 + 2 * (lane & 3));
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float x0 = __uint_as_float(x4[u] << 16), x1 = __uint_as_float(x4[u] & 0xffff0000u);
            mul2(x0, x1, w.x, w.y);
            const int at = sb * 2 + (u & 1);
            const uint32_t hi = pack_high(x0, x1);
            khi[q * 2 + (u >> 1)][at] = hi;
            below_high(hi, x0, x1);
            md[u >> 1][at] = hi;
            if (three) {
              md[u >> 1][at] = pack_high(x0, x1);
              below_high(md[u >> 1][at], x0, x1);
            }
            lo[u >> 1][at] = pack_bf16(x0, x1);
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t at = lanes + ((uint32_t)(u * 16) << 16) + q * 8 + pieces;
          tmem_st_16x128_x2(at, lo[u]);
          tmem_st_16x128_x2(at + 64, md[u]);
        }
      }
      if (three && local) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          tmem_st_16x128_x2(lanes + ((uint32_t)((i & 1) * 16) << 16) + (i >> 1) * 8 + TM_O + ph * 64, khi[i]);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->kt[ph]);
      if (three && !local) {
        // the keys' high piece takes the low one's place once that has been read
        if (!la_wait_warp(&bar->u1, ph, abort)) break;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          tmem_st_16x128_x2(lanes + ((uint32_t)((i & 1) * 16) << 16) + (i >> 1) * 8 + TM_K0, khi[i]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->khi);
      }
    }
  } else if (warp >= LA_ROLE_WARPS && warp < LA_ROLE_WARPS + 2 * LA_GROUP_WARPS) {
    // ---------------- scores: weighted, to bf16 in place ----------------
    regs_dec<LA_SCORE_REGS>();
    const int quad = warp & 3, hf = (warp - LA_ROLE_WARPS - LA_GROUP_WARPS) >> 2;
    const int row = quad * 32 + lane;               // TMEM lane: token row
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const int mt = threadIdx.x - LA_ROLE_WARPS * 32 - LA_GROUP;
    for (int j = mt; j <= LC; j += LA_GROUP) {
      pw[j] = decay_pow(ld, (float)j);
      if (j < LC) bw[j] = fast ? decay_pow(ld, (float)(LA_MID - (a.reverse ? LC - 1 - j : j))) : 1.f;
    }
    asm volatile("bar.sync 1, %0;" ::"n"(LA_GROUP) : "memory");
    for (int c = 0; c < chunks && !local; ++c) {
      const uint32_t ph = c & 1;
      if (!la_wait_warp(&bar->p, ph, abort)) break;
      tc_fence_after();
      // a warp's two 32 x 32 blocks are behind the tokens, ahead of them (zero), or on the
      // diagonal; the halves interleave the blocks, so that their work is even
#pragma unroll 1
      for (int blk = hf; blk < 4; blk += 2) {       // 32 columns become 16 of high and 16 of low pairs
        const int dq = a.reverse ? blk - quad : quad - blk, s0 = blk * 32;
        uint32_t v[32];
        if (dq < 0) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0u;
        } else {
          tmem_ld32(lanes + TM_P + s0, v);
          tmem_wait_ld();
          if (!fast) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int e = a.reverse ? s0 + i - row : row - s0 - i;
              v[i] = __float_as_uint(__uint_as_float(v[i]) * pw[e < 0 ? 0 : e]);
            }
          }
          if (dq == 0) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (a.reverse ? i < lane : i > lane) v[i] = 0u;
          }
          uint32_t lo[16];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 w = *reinterpret_cast<const float4*>(bw + s0 + 4 * i);
            float x0 = __uint_as_float(v[4 * i]), x1 = __uint_as_float(v[4 * i + 1]);
            float x2 = __uint_as_float(v[4 * i + 2]), x3 = __uint_as_float(v[4 * i + 3]);
            mul2(x0, x1, w.x, w.y);
            mul2(x2, x3, w.z, w.w);
            v[2 * i] = pack_high(x0, x1);
            v[2 * i + 1] = pack_high(x2, x3);
            below_high(v[2 * i], x0, x1);
            below_high(v[2 * i + 1], x2, x3);
            lo[2 * i] = pack_bf16(x0, x1);
            lo[2 * i + 1] = pack_bf16(x2, x3);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) v[16 + i] = lo[i];
        }
        tmem_st32(lanes + TM_P + s0, v);
      }
      if (!fast && (init != nullptr || c > 0)) {
        // O = Q E so far: decay each token's row
        if (!la_wait_warp(&bar->o1, ph, abort)) break;
        tc_fence_after();
        const int u = a.reverse ? LC - 1 - row : row;
        const float f = pw[u + (c == 0 && g == 0 && a.in_ready ? 0 : 1)];
#pragma unroll 1
        for (int q = hf * (DV / 2); q < (hf + 1) * (DV / 2); q += 16) {
          uint32_t v[16];
          tmem_ld16(lanes + TM_O + q, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
          tmem_st16(lanes + TM_O + q, v);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->mid);
    }
  } else if (warp >= LA_ROLE_WARPS + 2 * LA_GROUP_WARPS) {
    // ---------------- state and output ----------------
    regs_inc<LA_STATE_REGS>();
    const int quad = warp & 3, hf = (warp - LA_ROLE_WARPS - 2 * LA_GROUP_WARPS) >> 2;
    const int row = quad * 32 + lane;               // TMEM lane: state row, or token row of O
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    constexpr int EC = DV / 2;                      // columns of the state and of O per thread
    const int j0 = hf * EC;
    const int mt = threadIdx.x - LA_ROLE_WARPS * 32 - 2 * LA_GROUP;
    auto st_sync = [] { asm volatile("bar.sync 2, %0;" ::"n"(LA_GROUP) : "memory"); };

    // States in global memory go through the room of E's pieces when their rows are contiguous
    // (fp32 d x DV, 16-byte chunks swizzled by row: a thread's own row directly would touch 32
    // rows per access); transposed ones are contiguous across the lanes.
    constexpr int CH = DV / 4;
    auto chunk_at = [&](int r, int ch) { return reinterpret_cast<float4*>(selo + r * DV * 4 + ((ch ^ (r & (CH - 1))) << 4)); };
    float S[EC];
    if (init) {
      if (isj == 1 && (a.dv & 3) == 0 && ((uintptr_t)init & 15) == 0 && (isi & 3) == 0) {
        // (eight loads in flight: one after the other they took 10 us)
#pragma unroll 1
        for (int x0 = mt; x0 < a.d * CH; x0 += 8 * LA_GROUP) {
          float4 y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int x = x0 + i * LA_GROUP, r = x / CH, ch = x - r * CH;
            y[i] = r < a.d && 4 * ch < a.dv ? *reinterpret_cast<const float4*>(init + r * isi + 4 * ch)
                                            : make_float4(0.f, 0.f, 0.f, 0.f);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int x = x0 + i * LA_GROUP, r = x / CH;
            if (r < a.d) *chunk_at(r, x - r * CH) = y[i];
          }
        }
        st_sync();
#pragma unroll
        for (int j = 0; j < EC; j += 4) {
          const float4 x = row < a.d ? *chunk_at(row, (j0 + j) >> 2) : make_float4(0.f, 0.f, 0.f, 0.f);
          S[j] = x.x; S[j + 1] = x.y; S[j + 2] = x.z; S[j + 3] = x.w;
        }
        st_sync();
      } else {
#pragma unroll
        for (int j = 0; j < EC; ++j) S[j] = row < a.d && j0 + j < a.dv ? init[row * isi + (j0 + j) * isj] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < EC; ++j) S[j] *= in_scale;
    } else {
#pragma unroll
      for (int j = 0; j < EC; ++j) S[j] = 0.f;
    }
    auto put_state = [&](float f) {  // f E in two bf16 pieces, the second operand of Q E
      if (row < DK) {
#pragma unroll
        for (int j = 0; j < EC; j += 8) {
          uint32_t y[4], lo[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float x0 = S[j + 2 * u], x1 = S[j + 2 * u + 1];
            mul2(x0, x1, f, f);
            y[u] = pack_high(x0, x1);
            below_high(y[u], x0, x1);
            lo[u] = pack_bf16(x0, x1);
          }
          const uint32_t at = sw_off(row, j0 + j, DK);
          *reinterpret_cast<uint4*>(se + at) = make_uint4(y[0], y[1], y[2], y[3]);
          *reinterpret_cast<uint4*>(selo + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->est);
    };
    const bool ready0 = g == 0 && a.in_ready;       // the first chunk's E is decayed already
    // (without a chunk nothing reads E, whose room the last state passes through)
    if (!local && chunks > 0) {
      if (init) put_state(fast ? decay_pow(ld, (float)(LA_MID + 1 - (ready0 ? 1 : 0))) : 1.f);
      else if (lane == 0) mbar_arrive(&bar->est);
    }
    // a^128 is rounded for each chunk to where the chunks' product is nearest: what a rounding leaves is
    // carried into the next one, so that it does not compound
    const float2 a_full = decay_parts(ld, LC);
    float left = 0.f;
    const float a_mid = decay_pow(ld, (float)(LA_MID + 1));
    // what multiplies a finished row of O
    const float r_out = fast ? a.out_scale * expf(ld * (float)((a.reverse ? LC - 1 - row : row) - LA_MID)) : a.out_scale;

    for (int c = 0; c < chunks; ++c) {
      const uint32_t ph = c & 1;
      const int m = tokens(c);
      // E' = a^len E + U
      if (!la_wait_warp(&bar->u2[ph], (c >> 1) & 1, abort)) break;
      tc_fence_after();
      {
        const int len = m - (c == 0 && ready0 ? 1 : 0);
        float f;
        if (len == LC) {
          const float x = a_full.y + left;
          f = a_full.x + x;
          left = (a_full.x - f) + x;
        } else {
          f = decay_pow(ld, (float)len);
        }
#pragma unroll
        for (int q = 0; q < EC; q += 16) {
          uint32_t v[16];
          tmem_ld16(lanes + TM_U + j0 + q, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; i += 2)
            fma2(S[q + i], S[q + i + 1], f, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->ufree);
      if (local) continue;
      if (c + 1 < chunks) {  // E in bf16, once Q E has read the one before
        if (!la_wait_warp(&bar->o1, ph, abort)) break;
        put_state(fast ? a_mid : 1.f);
      }
      // O leaves: through the room of the chunk's V, which P V was the last to read, and TMA, or
      // (partial chunk) straight to its rows
      if (!la_wait_warp(&bar->o2[ph], (c >> 1) & 1, abort)) break;
      tc_fence_after();
      uint8_t* so = v_rows(stage(c));
      const int r0 = a.reverse ? LC - m : 0;
#pragma unroll 1
      for (int q = 0; q < EC; q += 16) {
        uint32_t v[16];
        tmem_ld16(lanes + TM_O + j0 + q, v);
        tmem_wait_ld();
        const int j = j0 + q;
        const long long t = (long long)tile_t(c) + row;
        char* dst = (char*)a.o.p + ((long long)b * a.o.sb + (long long)h * a.o.sh + t * a.o.st + j) * 2;
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
          uint32_t y[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float x0 = __uint_as_float(v[i + 2 * u]), x1 = __uint_as_float(v[i + 2 * u + 1]);
            mul2(x0, x1, r_out, r_out);
            y[u] = pack_bf16(x0, x1);
          }
          if (m == LC) *reinterpret_cast<uint4*>(so + sw_off(row, j + i, LC)) = make_uint4(y[0], y[1], y[2], y[3]);
          else if (row >= r0 && row < r0 + m && j + i < a.dv)
            *reinterpret_cast<uint4*>(dst + i * 2) = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bar->staged);
        mbar_arrive(&bar->ofree);
      }
    }
    // last state: the segment's slot, or the caller's
    float* dst = local ? a.slots + ((size_t)bh * a.nseg + g) * cells
                       : (a.s_out && g == a.nseg - 1 ? a.s_out + (size_t)bh * cells : nullptr);
    if (dst) {
      const long long osi = local ? a.dv : a.si, osj = local ? 1 : a.sj;
      const float w = local || n == 0 ? 1.f : a.st_scale * (a.out_decay ? decay_pow(ld, 1.f) : 1.f);
      if (osj == 1 && (a.dv & 3) == 0 && ((uintptr_t)dst & 15) == 0 && (osi & 3) == 0) {
        // (the last chunk's O was waited for, so Q E has read E; where only states are formed, its last U
        // was, which reads the third stage of V)
        if (row < a.d) {
#pragma unroll
          for (int j = 0; j < EC; j += 4)
            *chunk_at(row, (j0 + j) >> 2) = make_float4(S[j] * w, S[j + 1] * w, S[j + 2] * w, S[j + 3] * w);
        }
        st_sync();
        for (int x = mt; x < a.d * CH; x += LA_GROUP) {
          const int r = x / CH, ch = x - r * CH;
          if (4 * ch < a.dv && !*abort) *reinterpret_cast<float4*>(dst + r * osi + 4 * ch) = *chunk_at(r, ch);
        }
      } else if (row < a.d && !*abort) {
#pragma unroll
        for (int j = 0; j < EC; ++j)
          if (j0 + j < a.dv) dst[row * osi + (j0 + j) * osj] = S[j] * w;
      }
    }
  }

  // ---------------- teardown ----------------
  __syncwarp();
  if (warp == 0 && lane == 0 && *abort) {
    // let the copies this CTA issued land before its shared memory goes away
    for (int i = max(0, k_loads - stages); i < k_loads; ++i) drain_wait(&bar->full_k[stage(i)], stage_ph(i));
    for (int i = max(0, v_loads - stages); i < v_loads; ++i) drain_wait(&bar->full_v[stage(i)], stage_ph(i));
    if (q_loads > 0) drain_wait(&bar->full_q, (q_loads - 1) & 1);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TM_COLS);
  }
  if (*abort) {
    // what this CTA owes is NaN, so that nothing passes for a result before the status is read (the
    // rows' stores have been waited for by the warp that issued them).  Where it is, is found anew:
    // kept in registers until here, it would cost the passes 1%
    int bh, g;
    asm volatile("mov.u32 %0, %%ctaid.x;\n mov.u32 %1, %%ctaid.y;" : "=r"(bh), "=r"(g));
    const int b = bh / a.H, h = bh - b * a.H, n = scan_len(a, b);
    const int t0 = min(n, g * a.seg_len), t1 = min(n, t0 + a.seg_len), first = a.reverse ? n - t1 : t0;
    const size_t cells = (size_t)a.d * a.dv;
    for (long long x = threadIdx.x; !local && x < (long long)(t1 - t0) * a.dv; x += LA_THREADS) {
      const long long t = first + x / a.dv;
      const int j = (int)(x % a.dv);
      ((unsigned short*)a.o.p)[(long long)b * a.o.sb + (long long)h * a.o.sh + t * a.o.st + j] = 0x7fff;
    }
    float* dst = local ? a.slots + ((size_t)bh * a.nseg + g) * cells
                       : (a.s_out && g == a.nseg - 1 ? a.s_out + (size_t)bh * cells : nullptr);
    for (size_t x = threadIdx.x; dst && x < cells; x += LA_THREADS) dst[x] = __int_as_float(0x7fffffff);
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
int go_tc(const TcPass& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& o,
          cudaStream_t s) {
  if (!raise_smem_limit((const void*)scan_tc_kernel<DK, DV>, TcSmem<DK, DV>::bytes)) return -1;
  launch_k(scan_tc_kernel<DK, DV>, dim3((unsigned)(p.a.B * p.a.H), p.local ? p.a.nseg - 1 : p.a.nseg), LA_THREADS,
           TcSmem<DK, DV>::bytes, s, q, k, v, o, p);
  return 1;
}

int go_tc_shape(const TcPass& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& o,
          cudaStream_t s) {
  if (p.a.d <= 64) return p.a.dv <= 64 ? go_tc<64, 64>(p, q, k, v, o, s) : go_tc<64, 128>(p, q, k, v, o, s);
  return p.a.dv <= 64 ? go_tc<128, 64>(p, q, k, v, o, s) : go_tc<128, 128>(p, q, k, v, o, s);
}

}  // namespace

// bf16, widths up to 128 in whole 16-byte vectors, rows on the 16-byte grid, and more tokens than
// the kernel for a few of them takes: from 32 on the pass costs one chunk (8 heads of 64 x 64:
// 8.4 us for 32 to 128 tokens, on the CUDA cores 14.5 for 32 and 48 for 128; 256 heads of
// 128 x 128: 26 us against 35 for 32 tokens and 115 for 128).
bool scan_tc_shape(const ScanArgs& a, int dtype) {
  return dtype == FWPKM_BF16 && a.d <= 128 && a.dv <= 128 && a.d % 8 == 0 && a.dv % 8 == 0 && a.T >= 32;
}
bool scan_tc_takes(const ScanArgs& a, int dtype) {
  return scan_tc_shape(a, dtype) && grid16(a.q, a) && grid16(a.k, a) && grid16(a.v, a) && grid16(a.o, a);
}

// Segments: one when the heads fill half the GPU, else one CTA per SM, of at least two chunks
// each.  (The extra pass over K and V costs half of the other: with two segments 74 heads of 8192
// tokens take 216 us, 75 whole ones 243.)
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
  CUtensorMap q, k, v, o;
  if (!heads_map(&q, a0.q, a0, a0.d, &p.cq) || !heads_map(&k, a0.k, a0, a0.d, &p.ck) ||
      !heads_map(&v, a0.v, a0, a0.dv, &p.cv) || !heads_map(&o, a0.o, a0, a0.dv, &p.co)) {
    fprintf(stderr, "fwpkm: cuTensorMapEncodeTiled failed\n");
    return -1;
  }
  int nl = 0;
  p.stall = take_test_stall();
  if (p.a.nseg > 1) {
    p.local = 1;
    if (go_tc_shape(p, q, k, v, o, s) < 0) return -1;
    nl += 1 + launch_scan_combine(p.a, s);
    p.local = 0;
    p.stall = 0;
  }
  if (go_tc_shape(p, q, k, v, o, s) < 0) return -1;
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
