// lookup.cu -- weighted lookups of a learned table and their gradients.
//
//   out_t    = scale * sum_r w[t,r] table[idx[t,r]]            (r < R; w absent: ones)
//   dtable_i = scale * sum_{(t,r): idx[t,r] = i} w[t,r] dout_t
//   dw[t,r]  = scale * <dout_t, table[idx[t,r]]>
//
// With R = 1 and no w this is a token embedding; with the slots and weights of a
// product-key selection it is the read of a slow value table.  Entries outside [0, rows)
// contribute nothing (their dw is 0).
//
// All three are bound by HBM: the forward reads every used row once and writes out once; the
// gradient reads dout once per pair and writes (or updates) every row of dtable once.
// No float atomics: the (row, pair) list is sorted by row with a stable radix sort, so each
// row's terms are summed in pair order and the results are deterministic.
#include <cooperative_groups.h>

#include <atomic>
#include <cstdio>

#include "fwpkm_internal.cuh"
#include "sm100.cuh"

namespace fwpkm {
namespace {

constexpr int LK_THREADS = 256;

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// VEC consecutive elements as one load or store (VEC * sizeof(T) = 16 bytes, or one element).
template <typename T, int VEC>
struct __align__(sizeof(T) * VEC) Pack {
  T v[VEC];
};

template <typename I>
__device__ __forceinline__ long long load_idx(const I* p, long long i) { return (long long)__ldg(p + i); }

// Threads across a row's vectors (a power of two) for a row of `vecs` vectors.
int row_threads(long long vecs) {
  int t = 1;
  while (t < LK_THREADS && t < vecs) t <<= 1;
  return t;
}

// One thread per vector of an output row, TU tokens per thread: their indices, then their
// rows, are in flight together.
template <typename T, typename I, int VEC, int TU>
__global__ void __launch_bounds__(LK_THREADS)
lookup_row_kernel(const T* __restrict__ table, long long rows, long long ld, const I* __restrict__ idx,
                  const float* __restrict__ w, long long n, int vecs, int tx_n, float scale, T* __restrict__ out,
                  long long out_ld) {
  pdl_wait();
  pdl_trigger();
  const int ty_n = LK_THREADS / tx_n;
  const int tx = threadIdx.x & (tx_n - 1), ty = threadIdx.x / tx_n;
  const int c = blockIdx.y * tx_n + tx;
  if (c >= vecs) return;
  const long long t0 = (long long)blockIdx.x * ty_n * TU + ty;
  long long row[TU];
  Pack<T, VEC> x[TU];
#pragma unroll
  for (int u = 0; u < TU; ++u) {
    const long long t = t0 + (long long)u * ty_n;
    row[u] = t < n ? load_idx(idx, t) : -1;
  }
#pragma unroll
  for (int u = 0; u < TU; ++u)
    if (row[u] >= 0 && row[u] < rows)
      x[u] = *reinterpret_cast<const Pack<T, VEC>*>(table + row[u] * ld + (long long)c * VEC);
#pragma unroll
  for (int u = 0; u < TU; ++u) {
    const long long t = t0 + (long long)u * ty_n;
    if (t >= n) return;
    const bool ok = row[u] >= 0 && row[u] < rows;
    const float f = w ? __ldg(w + t) * scale : scale;
    Pack<T, VEC> y;
#pragma unroll
    for (int e = 0; e < VEC; ++e) y.v[e] = from_f<T>(ok ? to_f<T>(x[u].v[e]) * f : 0.f);
    *reinterpret_cast<Pack<T, VEC>*>(out + t * out_ld + (long long)c * VEC) = y;
  }
}

// One thread per vector of an output row; the bag's rows four at a time, added in rank order.
template <typename T, typename I, int VEC>
__global__ void __launch_bounds__(LK_THREADS)
lookup_bag_kernel(const T* __restrict__ table, long long rows, long long ld, const I* __restrict__ idx,
                  const float* __restrict__ w, long long n, int R, int vecs, int tx_n, float scale,
                  T* __restrict__ out, long long out_ld) {
  pdl_wait();
  pdl_trigger();
  constexpr int U = 4;
  const int ty_n = LK_THREADS / tx_n;
  const int tx = threadIdx.x & (tx_n - 1), ty = threadIdx.x / tx_n;
  const int c = blockIdx.y * tx_n + tx;
  const long long t = (long long)blockIdx.x * ty_n + ty;
  if (c >= vecs || t >= n) return;
  float acc[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
  for (int r0 = 0; r0 < R; r0 += U) {
    long long row[U];
    float f[U];
    Pack<T, VEC> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      row[u] = r0 + u < R ? load_idx(idx, t * R + r0 + u) : -1;
      if (row[u] >= rows) row[u] = -1;
      f[u] = row[u] >= 0 ? (w ? __ldg(w + t * R + r0 + u) : 1.f) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (row[u] >= 0) x[u] = *reinterpret_cast<const Pack<T, VEC>*>(table + row[u] * ld + (long long)c * VEC);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (row[u] >= 0) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] = fmaf(f[u], to_f<T>(x[u].v[e]), acc[e]);
      }
  }
  Pack<T, VEC> y;
#pragma unroll
  for (int e = 0; e < VEC; ++e) y.v[e] = from_f<T>(acc[e] * scale);
  *reinterpret_cast<Pack<T, VEC>*>(out + t * out_ld + (long long)c * VEC) = y;
}

// dw: one warp per (token, DW_U ranks): the token's dout vectors are loaded once for them.
constexpr int DW_U = 4;
struct DwArgs {
  const void* table;
  const void* d_out;
  float* dw;           // null: not wanted
  long long rows, ld, out_ld, n;
  int R, vecs;
  float scale;
};
template <typename T, typename I, int VEC>
__device__ __forceinline__ void dw_job(const DwArgs& a, const I* __restrict__ idx, long long job, int lane) {
  const T* table = (const T*)a.table;
  const T* d_out = (const T*)a.d_out;
  const int groups = (a.R + DW_U - 1) / DW_U;
  const long long t = job / groups;
  if (t >= a.n) return;
  const int r0 = (int)(job - t * groups) * DW_U;
  long long row[DW_U];
  float acc[DW_U];
#pragma unroll
  for (int u = 0; u < DW_U; ++u) {
    row[u] = r0 + u < a.R ? load_idx(idx, t * a.R + r0 + u) : -1;
    if (row[u] >= a.rows) row[u] = -1;
    acc[u] = 0.f;
  }
  for (int c = lane; c < a.vecs; c += 32) {
    const Pack<T, VEC> g = *reinterpret_cast<const Pack<T, VEC>*>(d_out + t * a.out_ld + (long long)c * VEC);
    Pack<T, VEC> x[DW_U];
#pragma unroll
    for (int u = 0; u < DW_U; ++u)
      if (row[u] >= 0) x[u] = *reinterpret_cast<const Pack<T, VEC>*>(table + row[u] * a.ld + (long long)c * VEC);
#pragma unroll
    for (int u = 0; u < DW_U; ++u)
      if (row[u] >= 0) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[u] = fmaf(to_f<T>(g.v[e]), to_f<T>(x[u].v[e]), acc[u]);
      }
  }
#pragma unroll
  for (int u = 0; u < DW_U; ++u) acc[u] = warp_sum(acc[u]);
  if (lane == 0) {
#pragma unroll
    for (int u = 0; u < DW_U; ++u)
      if (r0 + u < a.R) a.dw[t * a.R + r0 + u] = row[u] >= 0 ? acc[u] * a.scale : 0.f;
  }
}
template <typename T, typename I, int VEC>
__global__ void __launch_bounds__(LK_THREADS)
lookup_dw_kernel(DwArgs a, const I* __restrict__ idx) {
  pdl_wait();
  pdl_trigger();
  dw_job<T, I, VEC>(a, idx, (long long)blockIdx.x * (LK_THREADS / 32) + (threadIdx.x >> 5), threadIdx.x & 31);
}

// ---------------------------------------------------------------------------
// Stable radix sort of the pairs by row.  Key: the row, or `rows` for an entry outside the
// table (sorted last and dropped).  Payload: the pair's index.  Least significant digit
// first, one counting pass per digit of up to RS_BITS bits.
// ---------------------------------------------------------------------------
constexpr int RS_THREADS = 512;
constexpr int RS_WARPS = RS_THREADS / 32;
constexpr int RS_BITS = 11;                 // 2048 bins: two passes up to 2^22 rows
constexpr int RS_MAX_BINS = 1 << RS_BITS;
constexpr int RS_ITEMS = 8;                 // items per thread of a tile
constexpr int RS_TILE = RS_THREADS * RS_ITEMS;
// Up to this many tiles every scatter CTA forms its own offsets from the tiles' counts;
// beyond it a scan launch does (the counts read by all CTAs grow with tiles^2).
constexpr int RS_OWN_SCAN = 32;

template <typename I>
__device__ __forceinline__ uint32_t pair_key(const I* idx, long long p, long long rows) {
  const long long r = load_idx(idx, p);
  return r >= 0 && r < rows ? (uint32_t)r : (uint32_t)rows;
}

// Where a pass reads its keys: the indices themselves (first pass) or the previous pass.
template <typename I>
struct Source {
  const I* idx;
  const uint2* item;  // (key, pair)
  long long rows;
  __device__ __forceinline__ uint2 at(long long p) const {
    return item ? item[p] : make_uint2(pair_key(idx, p, rows), (uint32_t)p);
  }
};

// Counts of one tile's digits: hist[tile][bin].
template <typename I>
__global__ void __launch_bounds__(RS_THREADS)
sort_hist_kernel(Source<I> src, long long P, int shift, int bins, uint32_t* __restrict__ hist) {
  __shared__ uint32_t s[RS_MAX_BINS];
  pdl_wait();
  pdl_trigger();
  for (int b = threadIdx.x; b < bins; b += RS_THREADS) s[b] = 0u;
  __syncthreads();
  const long long base = (long long)blockIdx.x * RS_TILE;
#pragma unroll
  for (int i = 0; i < RS_ITEMS; ++i) {
    const long long p = base + i * RS_THREADS + threadIdx.x;
    if (p < P) atomicAdd(&s[(src.at(p).x >> shift) & (bins - 1)], 1u);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += RS_THREADS) hist[(long long)blockIdx.x * bins + b] = s[b];
}

// hist[tile][bin] -> its exclusive sum over the tiles; total[bin] = the bin's count.
__global__ void __launch_bounds__(128)
sort_scan_kernel(uint32_t* __restrict__ hist, uint32_t* __restrict__ total, int tiles, int bins) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x * 128 + threadIdx.x;
  if (b >= bins) return;
  uint32_t run = 0;
  for (int t0 = 0; t0 < tiles; t0 += 16) {
    uint32_t x[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) x[u] = t0 + u < tiles ? hist[(long long)(t0 + u) * bins + b] : 0u;
#pragma unroll
    for (int u = 0; u < 16; ++u)
      if (t0 + u < tiles) {
        hist[(long long)(t0 + u) * bins + b] = run;
        run += x[u];
      }
  }
  total[b] = run;
}

// Exclusive sum over `bins` values in shared memory (bins <= MAXB, THREADS threads).
template <int THREADS, int MAXB>
__device__ __forceinline__ void block_exclusive(uint32_t* s, int bins, uint32_t* warp_tot) {
  constexpr int PER = MAXB / THREADS < 1 ? 1 : MAXB / THREADS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = threadIdx.x * PER + i;
    x[i] = b < bins ? s[b] : 0u;
    sum += x[i];
  }
  uint32_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_tot[warp] = inc;
  __syncthreads();
  uint32_t before = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) before += w < warp ? warp_tot[w] : 0u;
  uint32_t run = before + inc - sum;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = threadIdx.x * PER + i;
    if (b < bins) s[b] = run;
    run += x[i];
  }
  __syncthreads();
}

// Stable ranks of a tile's items inside their bins: warp w holds items [w, w+1) * 32 ITEMS
// of the tile in order, 32 at a time; lanes with equal digits rank each other by lane.
// wh[warp][bin] (uint16) ends as the number of earlier items of the tile in the bin from
// earlier warps, count[bin] (if given) as the tile's; rank[i] counts those of the same warp.
template <int WARPS, int ITEMS>
__device__ __forceinline__ void tile_ranks(const uint32_t (&digit)[ITEMS], const bool (&live)[ITEMS], uint16_t* wh,
                                           int bins, uint32_t (&rank)[ITEMS], uint32_t* count, int items = ITEMS) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int b = threadIdx.x; b < bins * WARPS / 2; b += WARPS * 32) reinterpret_cast<uint32_t*>(wh)[b] = 0u;
  __syncthreads();
  uint16_t* mine = wh + (size_t)warp * bins;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    if (i >= items) break;
    // lanes with the same digit, bit by bit (a match instruction over the warp is slower)
    unsigned peers = __ballot_sync(0xffffffffu, live[i]);
    if (!live[i]) peers = ~peers;
    for (int b = 0; (1 << b) < bins; ++b) {
      const bool set = (digit[i] >> b) & 1u;
      const unsigned with = __ballot_sync(0xffffffffu, set);
      peers &= set ? with : ~with;
    }
    const unsigned below = __popc(peers & ((1u << lane) - 1u));
    uint32_t old = 0;
    if (live[i]) old = mine[digit[i]];
    __syncwarp();
    if (live[i] && below == 0) mine[digit[i]] = (uint16_t)(old + __popc(peers));
    __syncwarp();
    rank[i] = old + below;
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += WARPS * 32) {
    uint32_t run = 0;
#pragma unroll
    for (int w8 = 0; w8 < WARPS; w8 += 8) {
      uint32_t c[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) c[u] = wh[(size_t)(w8 + u) * bins + b];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        wh[(size_t)(w8 + u) * bins + b] = (uint16_t)run;
        run += c[u];
      }
    }
    if (count) count[b] = run;
  }
  __syncthreads();
}

// Scatter one tile to its sorted places.  own_scan: hist holds plain counts and this CTA
// forms its offsets (tiles <= RS_OWN_SCAN); else hist is already the exclusive sum over tiles.
template <typename I>
__global__ void __launch_bounds__(RS_THREADS)
sort_scatter_kernel(Source<I> src, long long P, int shift, int bins, const uint32_t* __restrict__ hist,
                    const uint32_t* __restrict__ total, int tiles, int own_scan, uint2* __restrict__ out) {
  extern __shared__ uint32_t sm[];
  uint32_t* base = sm;                              // [bins]
  uint32_t* before = sm + bins;                     // [bins] earlier tiles' items of the bin
  uint16_t* wh = (uint16_t*)(sm + 2 * bins);        // [RS_WARPS][bins]
  __shared__ uint32_t warp_tot[RS_WARPS];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tile = blockIdx.x;
  uint32_t key[RS_ITEMS], pos[RS_ITEMS], digit[RS_ITEMS], rank[RS_ITEMS];
  bool live[RS_ITEMS];
#pragma unroll
  for (int i = 0; i < RS_ITEMS; ++i) {
    const long long p = (long long)tile * RS_TILE + (warp * RS_ITEMS + i) * 32 + lane;
    live[i] = p < P;
    const uint2 x = live[i] ? src.at(p) : make_uint2(0u, 0u);
    key[i] = x.x;
    pos[i] = x.y;
    digit[i] = (key[i] >> shift) & (bins - 1);
  }
  for (int b = threadIdx.x; b < bins; b += RS_THREADS) {
    uint32_t tot = 0, bef = 0;
    if (own_scan) {
      for (int t8 = 0; t8 < tiles; t8 += 8) {
        uint32_t c[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) c[u] = t8 + u < tiles ? hist[(long long)(t8 + u) * bins + b] : 0u;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (t8 + u == tile) bef = tot;
          tot += c[u];
        }
      }
    } else {
      tot = total[b];
      bef = hist[(long long)tile * bins + b];
    }
    base[b] = tot;
    before[b] = bef;
  }
  __syncthreads();
  block_exclusive<RS_THREADS, RS_MAX_BINS>(base, bins, warp_tot);
  tile_ranks<RS_WARPS, RS_ITEMS>(digit, live, wh, bins, rank, nullptr);
#pragma unroll
  for (int i = 0; i < RS_ITEMS; ++i)
    if (live[i]) {
      const uint32_t d = digit[i];
      out[base[d] + before[d] + wh[(size_t)warp * bins + d] + rank[i]] = make_uint2(key[i], pos[i]);
    }
}

// Up to CS_MAX pairs: the whole sort in one launch, by one cluster of up to sixteen CTAs that
// keeps the pairs in its shared memory (each pass: ranks in the CTA's tile, the tiles' counts
// read from one another, the items stored to their place in whichever CTA holds it).  The
// launch's other clusters form dw meanwhile, which needs no sorting.  (The launches of the
// general sort took 40 us for 16384 pairs, most of it latency.)
constexpr int CS_THREADS = 1024, CS_WARPS = CS_THREADS / 32, CS_ITEMS = 8, CS_TILE = CS_THREADS * CS_ITEMS;
// Digits of up to ten bits: one pass less than with nine for tables of 512 to 1023 rows (2000 pairs
// 11.1 -> 9.5 us); with eleven, 65536 pairs of 2^20 rows take two passes of 2048 bins in 37.8 us,
// with ten three of 128 in 30.8.
constexpr int CS_BITS = 10, CS_MAX_BINS = 1 << CS_BITS, CS_CLUSTER = 16;
constexpr long long CS_MAX = (long long)CS_TILE * 8;  // eight CTAs hold them; sixteen, where a GPC has them, in half the time
constexpr size_t CS_SMEM = 8 * (size_t)CS_TILE + 4 * 3 * (size_t)CS_MAX_BINS + 2 * (size_t)CS_WARPS * CS_MAX_BINS;

template <typename T, typename I, int VEC>
__global__ void __launch_bounds__(CS_THREADS, 1)
sort_cluster_kernel(const I* __restrict__ idx, int P, long long rows, int per, int passes, int ctas, int items,
                    uint2* __restrict__ out, DwArgs dw) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint8_t cs_raw[];
  uint2* item = (uint2*)cs_raw;                              // [CS_TILE] (key, pair)
  uint32_t* count = (uint32_t*)(item + CS_TILE);             // [CS_MAX_BINS] this tile's
  uint32_t* base = count + CS_MAX_BINS;                      // [CS_MAX_BINS]
  uint32_t* before = base + CS_MAX_BINS;                     // [CS_MAX_BINS] earlier tiles'
  uint16_t* wh = (uint16_t*)(before + CS_MAX_BINS);          // [CS_WARPS][bins]
  __shared__ uint32_t warp_tot[CS_WARPS];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if ((int)blockIdx.x >= ctas) {
    const long long jobs = dw.n * ((dw.R + DW_U - 1) / DW_U);
    const long long step = (long long)(gridDim.x - ctas) * CS_WARPS;
    for (long long j = (long long)(blockIdx.x - ctas) * CS_WARPS + warp; j < jobs; j += step)
      dw_job<T, I, VEC>(dw, idx, j, lane);
    return;
  }
  cg::cluster_group cluster = cg::this_cluster();
  const int tile = blockIdx.x, bins = 1 << per, tile_items = items * CS_THREADS;  // `items` per thread
  uint32_t key[CS_ITEMS], pos[CS_ITEMS], digit[CS_ITEMS], rank[CS_ITEMS];
  bool live[CS_ITEMS];
#pragma unroll
  for (int i = 0; i < CS_ITEMS; ++i) {
    const int p = tile * tile_items + (warp * items + i) * 32 + lane;
    live[i] = i < items && p < P;
    key[i] = live[i] ? pair_key(idx, p, rows) : 0u;
    pos[i] = (uint32_t)p;
  }
  for (int pass = 0; pass < passes; ++pass) {
#pragma unroll
    for (int i = 0; i < CS_ITEMS; ++i) digit[i] = (key[i] >> (pass * per)) & (bins - 1);
    tile_ranks<CS_WARPS, CS_ITEMS>(digit, live, wh, bins, rank, count, items);
    cluster.sync();  // every tile's counts are there, and its items in registers
    // (as a loop, though a thread has one bin at most: 2 us a call less than with an if)
    for (int b = threadIdx.x; b < bins; b += CS_THREADS) {
      uint32_t tot = 0, bef = 0;
#pragma unroll
      for (int r = 0; r < CS_CLUSTER; ++r) {
        const uint32_t c = r < ctas ? cluster.map_shared_rank(count, r < ctas ? r : 0)[b] : 0u;
        if (r < tile) bef += c;
        tot += c;
      }
      base[b] = tot;
      before[b] = bef;
    }
    __syncthreads();
    block_exclusive<CS_THREADS, CS_MAX_BINS>(base, bins, warp_tot);
    const bool last = pass == passes - 1;
#pragma unroll
    for (int i = 0; i < CS_ITEMS; ++i)
      if (live[i]) {
        const uint32_t d = digit[i];
        const uint32_t at = base[d] + before[d] + wh[(size_t)warp * bins + d] + rank[i];
        const uint32_t cta = at / (uint32_t)tile_items;
        if (last) out[at] = make_uint2(key[i], pos[i]);
        else cluster.map_shared_rank(item, cta)[at - cta * tile_items] = make_uint2(key[i], pos[i]);
      }
    cluster.sync();  // the items are in place (last pass: nobody reads this tile's counts any more)
    if (!last) {
#pragma unroll
      for (int i = 0; i < CS_ITEMS; ++i)
        if (live[i]) {
          const uint2 x = item[(warp * items + i) * 32 + lane];
          key[i] = x.x;
          pos[i] = x.y;
        }
    }
  }
}

// ---------------------------------------------------------------------------
// Segmented sum of the sorted pairs.  A team of tx_n threads (one vector of columns each)
// owns `seg` consecutive sorted pairs.  A row whose pairs lie inside the range is written at
// once; a row cut by the range's ends leaves a partial sum, and the second launch adds a
// cut row's partials in order.  The serial work on a row that everything reads is seg terms
// plus its partials: short ranges for few pairs (1761 pairs of 240 rows of 512 fp32, sums and
// join: 19 us with 32, 15 with 16), long ones for many (32768 pairs of 100 rows: 33 and 42).
// ---------------------------------------------------------------------------
int seg_pairs(long long P) { return P <= 2048 ? 8 : P <= 8192 ? 16 : 32; }
constexpr int ZERO_BYTES = 8192;

struct SegArgs {
  const uint2* item;  // sorted (row, pair)
  const float* w;
  long long P, rows, out_ld, grad_ld;
  int R, vecs, tx_n, width;
  float scale;
  int accumulate, seg;
  float* part;        // [ranges][2][width] fp32: the sums cut at the range's start and end
  long long ranges;
};

// A team thread's columns of a row of d_table, in 16-byte accesses (or one element).
template <typename G, int VEC>
struct GRow {
  static constexpr int GV = (sizeof(G) * VEC > 16) ? 16 / (int)sizeof(G) : VEC;
  Pack<G, GV> p[VEC / GV];
  __device__ __forceinline__ void load(const G* d_table, const SegArgs& a, uint32_t row, int c) {
    const G* src = d_table + (long long)row * a.grad_ld + (long long)c * VEC;
#pragma unroll
    for (int h = 0; h < VEC / GV; ++h) p[h] = *reinterpret_cast<const Pack<G, GV>*>(src + h * GV);
  }
};

template <typename G, int VEC, bool ACC>
__device__ __forceinline__ void put_row(G* d_table, const SegArgs& a, uint32_t row, int c, const float (&acc)[VEC],
                                        const GRow<G, VEC>& old) {
  G* dst = d_table + (long long)row * a.grad_ld + (long long)c * VEC;
  constexpr int GV = GRow<G, VEC>::GV;
#pragma unroll
  for (int h = 0; h < VEC / GV; ++h) {
    Pack<G, GV> y;
#pragma unroll
    for (int e = 0; e < GV; ++e) {
      const float s = acc[h * GV + e] * a.scale;
      y.v[e] = from_f<G>(ACC ? to_f<G>(old.p[h].v[e]) + s : s);
    }
    *reinterpret_cast<Pack<G, GV>*>(dst + h * GV) = y;
  }
}

// A team thread's columns of a partial sum (VEC > 1: the width is a multiple of VEC >= 4, so
// they lie on the 16-byte grid).
template <int VEC>
__device__ __forceinline__ void put_part(float* d, const float (&x)[VEC]) {
  constexpr int W = VEC < 4 ? 1 : 4;
#pragma unroll
  for (int e = 0; e < VEC; e += W) {
    Pack<float, W> y;
#pragma unroll
    for (int u = 0; u < W; ++u) y.v[u] = x[e + u];
    *reinterpret_cast<Pack<float, W>*>(d + e) = y;
  }
}
template <int VEC>
__device__ __forceinline__ void get_part(const float* d, float (&x)[VEC]) {
  constexpr int W = VEC < 4 ? 1 : 4;
#pragma unroll
  for (int e = 0; e < VEC; e += W) {
    const Pack<float, W> y = *reinterpret_cast<const Pack<float, W>*>(d + e);
#pragma unroll
    for (int u = 0; u < W; ++u) x[e + u] = y.v[u];
  }
}

// Whether `row` occurs in the sorted keys [lo, end).
__device__ __forceinline__ bool has_row(const uint2* __restrict__ item, long long lo, long long end, uint32_t row) {
  long long hi = end;
  while (lo < hi) {
    const long long mid = (lo + hi) >> 1;
    if (__ldg(&item[mid].x) < row) lo = mid + 1;
    else hi = mid;
  }
  return lo < end && __ldg(&item[lo].x) == row;
}
// The first of the sorted keys [lo, hi) that is not below `row` (hi: none), by a whole warp: 32
// probes a step.
__device__ __forceinline__ long long first_key(const uint2* __restrict__ item, long long lo, long long hi,
                                               long long row, int lane) {
  while (hi - lo > 32) {
    const long long step = (hi - lo + 31) / 32, at = lo + lane * step + step - 1;
    lo += __popc(__ballot_sync(0xffffffffu, at < hi && (long long)__ldg(&item[at].x) < row)) * step;
    if (lo + step - 1 < hi) hi = lo + step - 1;
  }
  return lo + __popc(__ballot_sync(0xffffffffu, lo + lane < hi && (long long)__ldg(&item[lo + lane].x) < row));
}
// Rows that a warp of the zeroing CTAs takes at once: about 64 KB of wide ones (their stores are
// the work), else one per lane (finding them is: 408100 rows of 64 fp32 that 12149 pairs leave
// took 98 us with eight rows, each searched for among all pairs, 61 with 32 among the pairs of the
// warp's rows).
__host__ __device__ constexpr int zero_rows(long long row_bytes) { return row_bytes >= 2048 ? 8 : 32; }

// ACC: added to d_table, whose rows are loaded with the pairs (SEG_U pairs in flight per team).
template <typename T, typename G, int VEC, bool ACC>
__global__ void __launch_bounds__(LK_THREADS, 2)
lookup_sum_kernel(SegArgs a, const T* __restrict__ d_out, G* __restrict__ d_table, int sum_blocks) {
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x >= sum_blocks) {
    // ---- rows no pair reads: zero (dense gradient only).  A warp takes a few rows, finds the
    // sorted keys among them, a lane looks each row up there, and the missing ones are written: by
    // bulk copies of zeros from shared memory where rows are on the 16-byte grid
    __shared__ __align__(16) uint8_t zeros[VEC == 1 ? 16 : ZERO_BYTES];
    if (VEC > 1) {
      for (int i = threadIdx.x * 16; i < ZERO_BYTES; i += LK_THREADS * 16)
        *reinterpret_cast<uint4*>(zeros + i) = make_uint4(0u, 0u, 0u, 0u);
      sm100::fence_async_smem();
      __syncthreads();
    }
    const int lane = threadIdx.x & 31;
    const long long warps = (long long)(gridDim.x - sum_blocks) * (LK_THREADS / 32);
    const long long w0 = (long long)(blockIdx.x - sum_blocks) * (LK_THREADS / 32) + (threadIdx.x >> 5);
    const int each = zero_rows((long long)a.width * sizeof(G));
    for (long long r0 = w0 * each; r0 < a.rows; r0 += warps * each) {
      const long long r = r0 + lane;
      const long long lo = first_key(a.item, 0, a.P, r0, lane), hi = first_key(a.item, lo, a.P, r0 + each, lane);
      const bool zero = lane < each && r < a.rows && !has_row(a.item, lo, hi, (uint32_t)r);
      if (VEC > 1) {
        if (zero) {
          const long long bytes = (long long)a.width * sizeof(G);
          uint8_t* dst = (uint8_t*)(d_table + r * a.grad_ld);
          for (long long o = 0; o < bytes; o += ZERO_BYTES)
            sm100::bulk_store(dst + o, zeros, (uint32_t)(bytes - o < ZERO_BYTES ? bytes - o : ZERO_BYTES));
          sm100::bulk_commit();
        }
      } else {
        unsigned todo = __ballot_sync(0xffffffffu, zero);
        while (todo) {
          const int l = __ffs(todo) - 1;
          todo &= todo - 1;
          G* dst = d_table + (r0 + l) * a.grad_ld;
          for (int c = lane; c < a.width; c += 32) dst[c] = from_f<G>(0.f);
        }
      }
    }
    if (VEC > 1) sm100::bulk_wait_all();
    return;
  }
  const int ty_n = LK_THREADS / a.tx_n;
  const int tx = threadIdx.x & (a.tx_n - 1), ty = threadIdx.x / a.tx_n;
  const int c = blockIdx.y * a.tx_n + tx;
  const long long range = (long long)blockIdx.x * ty_n + ty;
  if (c >= a.vecs || range >= a.ranges) return;
  const long long p0 = range * a.seg, p1 = p0 + a.seg < a.P ? p0 + a.seg : a.P;
  constexpr int SEG_U = ACC && VEC == 8 ? 4 : 8;
  const uint32_t none = (uint32_t)a.rows;
  float acc[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
  uint32_t cur = a.item[p0].x;
  const bool cut_start = p0 > 0 && a.item[p0 - 1].x == cur;
  const bool cut_end = p1 < a.P && a.item[p1].x == a.item[p1 - 1].x;
  bool first = true;  // still in the range's first row
  GRow<G, VEC> last;  // (accumulate) the row of the pair before, if it was its row's last
  for (long long q0 = p0; q0 < p1; q0 += SEG_U) {
    uint32_t k[SEG_U];
    float f[SEG_U];
    Pack<T, VEC> x[SEG_U];
    uint32_t pr[SEG_U];
#pragma unroll
    for (int u = 0; u < SEG_U; ++u) {
      const long long p = q0 + u;
      const uint2 x2 = p < p1 ? a.item[p] : make_uint2(none, 0u);
      k[u] = x2.x;
      pr[u] = x2.y;
    }
    const uint32_t after = q0 + SEG_U < p1 ? a.item[q0 + SEG_U].x : none;
    GRow<G, VEC> old[SEG_U];
#pragma unroll
    for (int u = 0; u < SEG_U; ++u) {
      // (in vectors also for a pair that is none, so that the loads go out together: 5000 pairs of
      // 1000 bf16 30 -> 21 us; by elements that took 102 us instead of 86 for 16000 pairs of 1291)
      f[u] = 0.f;
      if (VEC > 1 || k[u] != none) {
        f[u] = a.w ? __ldg(a.w + pr[u]) : 1.f;
        x[u] = *reinterpret_cast<const Pack<T, VEC>*>(d_out + (long long)(pr[u] / a.R) * a.out_ld + (long long)c * VEC);
        // the row's last pair here: what the gradient is added to, loaded with the pairs
        if (ACC && k[u] != none && k[u] != (u + 1 < SEG_U ? k[(u + 1) % SEG_U] : after)) old[u].load(d_table, a, k[u], c);
      }
    }
#pragma unroll
    for (int u = 0; u < SEG_U; ++u) {
      if (q0 + u < p1) {
        if (ACC && u > 0) last = old[(u + SEG_U - 1) % SEG_U];
        if (k[u] != cur) {
          if (cur != none) {
            if (first && cut_start) {
              put_part<VEC>(a.part + (range * 2) * a.width + (long long)c * VEC, acc);
            } else {
              put_row<G, VEC, ACC>(d_table, a, cur, c, acc, last);
            }
          }
#pragma unroll
          for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
          cur = k[u];
          first = false;
        }
        if (cur != none) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) acc[e] = fmaf(f[u], to_f<T>(x[u].v[e]), acc[e]);
        }
        if (ACC && (u == SEG_U - 1 || q0 + u + 1 == p1)) last = old[u];
      }
    }
  }
  if (cur == none) return;
  if ((first && cut_start) || cut_end) {
    // a row cut at both ends is one partial, kept as the start's
    put_part<VEC>(a.part + (range * 2 + ((first && cut_start) ? 0 : 1)) * a.width + (long long)c * VEC, acc);
  } else {
    put_row<G, VEC, ACC>(d_table, a, cur, c, acc, last);
  }
}

// Rows cut by range ends: the team of the range where the row begins adds its partials.
template <typename G, int VEC, bool ACC>
__global__ void __launch_bounds__(LK_THREADS)
lookup_join_kernel(SegArgs a, G* __restrict__ d_table) {
  pdl_wait();
  pdl_trigger();
  const int ty_n = LK_THREADS / a.tx_n;
  const int tx = threadIdx.x & (a.tx_n - 1), ty = threadIdx.x / a.tx_n;
  const int c = blockIdx.y * a.tx_n + tx;
  const long long range = (long long)blockIdx.x * ty_n + ty;
  if (c >= a.vecs || range + 1 >= a.ranges) return;
  const long long p0 = range * a.seg, p1 = p0 + a.seg;  // not the last range: full
  const uint32_t row = a.item[p1 - 1].x;
  if (row == (uint32_t)a.rows || a.item[p1].x != row) return;     // nothing cut at the end
  if (a.item[p0].x == row && p0 > 0 && a.item[p0 - 1].x == row) return;  // the row began earlier
  // last range that holds the row: the ranges after this one whose first key is the row
  long long lo = range + 1, hi = a.ranges;
  while (lo < hi) {
    const long long mid = (lo + hi) >> 1;
    if (a.item[mid * a.seg].x == row) lo = mid + 1;
    else hi = mid;
  }
  float acc[VEC];
  get_part<VEC>(a.part + (range * 2 + 1) * a.width + (long long)c * VEC, acc);
  constexpr int U = VEC > 4 ? 4 : 8;
  for (long long q0 = range + 1; q0 < lo; q0 += U) {
    float x[U][VEC];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (q0 + u < lo) get_part<VEC>(a.part + ((q0 + u) * 2) * a.width + (long long)c * VEC, x[u]);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (q0 + u < lo) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] += x[u][e];
      }
  }
  GRow<G, VEC> old;
  if (ACC) old.load(d_table, a, row, c);
  put_row<G, VEC, ACC>(d_table, a, row, c, acc, old);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }
bool ptr_al(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t dsize(int dt) { return dt == FWPKM_BF16 ? 2 : 4; }

int key_bits(long long rows) {  // bits of the largest key, `rows`
  int b = 1;
  while (b < 32 && (rows >> b) != 0) ++b;
  return b;
}

struct SortPlan {
  int bits, passes, per, bins, tiles;
};
SortPlan sort_plan(long long rows, long long P) {
  SortPlan s;
  s.bits = key_bits(rows);
  s.passes = (s.bits + RS_BITS - 1) / RS_BITS;
  s.per = (s.bits + s.passes - 1) / s.passes;
  s.bins = 1 << s.per;
  s.tiles = (int)((P + RS_TILE - 1) / RS_TILE);
  return s;
}

struct BackWork {
  uint2* item[2];
  uint32_t *hist, *total;
  float* part;
};
size_t back_carve(const fwpkm_lookup_config& c, long long P, char* base, BackWork* w) {
  const SortPlan sp = sort_plan(c.rows, P);
  const int seg = seg_pairs(P);
  const long long ranges = (P + seg - 1) / seg;
  size_t off = 0;
  auto take = [&](size_t bytes) -> char* {
    char* p = base ? base + off : nullptr;
    off += up256(bytes);
    return p;
  };
  BackWork b;
  for (int i = 0; i < 2; ++i) {
    b.item[i] = (uint2*)take(8 * (size_t)P);
  }
  b.hist = (uint32_t*)take(4 * (size_t)sp.tiles * sp.bins);
  b.total = (uint32_t*)take(4 * (size_t)sp.bins);
  b.part = (float*)take(4 * 2 * (size_t)ranges * c.width);
  if (w) *w = b;
  return off;
}

fwpkm_status check_lookup(const fwpkm_lookup_config* c, long long n) {
  if (!c || n < 0 || c->rows < 1 || c->width < 1 || c->R < 1 || c->table_ld < c->width || c->out_ld < c->width)
    return FWPKM_ERR_INVALID_ARG;
  if (c->dtype != FWPKM_F32 && c->dtype != FWPKM_BF16) return FWPKM_ERR_INVALID_ARG;
  if (c->idx_dtype != FWPKM_I32 && c->idx_dtype != FWPKM_I64) return FWPKM_ERR_INVALID_ARG;
  if (c->rows > 0x7ffffffeLL || c->width > (1 << 20) || c->R > 1024 || n > 0x7fffffffLL / c->R)
    return FWPKM_ERR_UNSUPPORTED;
  return FWPKM_OK;
}

fwpkm_status done(int launches) {
  count_launches(launches);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return FWPKM_OK;
  fprintf(stderr, "fwpkm: CUDA error: %s\n", cudaGetErrorString(e));
  return FWPKM_ERR_CUDA;
}

// Rows are taken 16 bytes at a time when every row starts on a 16-byte boundary and holds
// whole vectors; one element at a time otherwise (any width, stride or alignment).
template <typename T>
bool rows_vec(const void* p, long long ld, int width) {
  return ptr_al(p, 16) && (ld * sizeof(T)) % 16 == 0 && (width * sizeof(T)) % 16 == 0;
}

template <typename T, typename I, int VEC>
void go_lookup(const fwpkm_lookup_config& c, const void* table, const void* idx, const float* w, long long n,
               void* out, cudaStream_t s) {
  const int vecs = c.width / VEC, tx = row_threads(vecs), ty = LK_THREADS / tx;
  const unsigned gy = (unsigned)((vecs + tx - 1) / tx);
  if (c.R == 1) {
    constexpr int TU = 2;
    const unsigned gx = (unsigned)((n + (long long)ty * TU - 1) / ((long long)ty * TU));
    launch_k(lookup_row_kernel<T, I, VEC, TU>, dim3(gx, gy), LK_THREADS, 0, s, (const T*)table, c.rows, c.table_ld,
             (const I*)idx, w, n, vecs, tx, c.scale, (T*)out, c.out_ld);
  } else {
    const unsigned gx = (unsigned)((n + ty - 1) / ty);
    launch_k(lookup_bag_kernel<T, I, VEC>, dim3(gx, gy), LK_THREADS, 0, s, (const T*)table, c.rows, c.table_ld,
             (const I*)idx, w, n, c.R, vecs, tx, c.scale, (T*)out, c.out_ld);
  }
}

template <typename T, typename I>
void go_lookup_v(const fwpkm_lookup_config& c, const void* table, const void* idx, const float* w, long long n,
                 void* out, cudaStream_t s) {
  if (rows_vec<T>(table, c.table_ld, c.width) && rows_vec<T>(out, c.out_ld, c.width))
    go_lookup<T, I, 16 / (int)sizeof(T)>(c, table, idx, w, n, out, s);
  else
    go_lookup<T, I, 1>(c, table, idx, w, n, out, s);
}

// A launch in clusters of `cluster` CTAs.
template <typename... KArgs, typename... Args>
void launch_cluster(void (*kern)(KArgs...), unsigned grid, unsigned block, unsigned cluster, size_t smem,
                    cudaStream_t s, Args... args) {
  cudaLaunchAttribute attr[2];
  unsigned na = 0;
  attr[na].id = cudaLaunchAttributeClusterDimension;
  attr[na].val.clusterDim.x = cluster;
  attr[na].val.clusterDim.y = 1;
  attr[na++].val.clusterDim.z = 1;
  if (pdl_enabled()) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na++].val.programmaticStreamSerializationAllowed = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = na;
  cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// Whether clusters of 16 CTAs of this kernel fit the current device (they are not portable).
template <typename T, typename I, int VEC>
bool wide_clusters() {
  auto kern = sort_cluster_kernel<T, I, VEC>;
  static std::atomic<int> known[64];  // by device: 0 not asked, 1 no, 2 yes
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  int k = known[dev].load();
  if (k == 0) {
    k = 1;
    if (cudaFuncSetAttribute((const void*)kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) {
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = CS_CLUSTER;
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(CS_CLUSTER);
      cfg.blockDim = dim3(CS_THREADS);
      cfg.dynamicSmemBytes = CS_SMEM;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n > 0) k = 2;
    }
    cudaGetLastError();
    known[dev].store(k);
  }
  return k == 2;
}

// The sorted pairs end in w.item[*sorted].  Up to CS_MAX pairs: one launch, which forms
// dw too (dw.dw is cleared to say so).
template <typename T, typename I, int VEC>
int go_sort(const fwpkm_lookup_config& c, const void* idx, long long P, const BackWork& w, int* sorted, DwArgs* dw,
            cudaStream_t s) {
  const SortPlan sp = sort_plan(c.rows, P);
  if (P <= CS_MAX) {
    const void* kern = (const void*)sort_cluster_kernel<T, I, VEC>;
    if (!raise_smem_limit(kern, CS_SMEM)) return -1;
    // as many CTAs as there are thousands of pairs, up to the largest cluster that fits
    int ctas = 1;
    while (ctas < 8 && (long long)ctas * CS_THREADS < P) ctas <<= 1;
    if (P > 8 * CS_THREADS && wide_clusters<T, I, VEC>()) ctas = 16;
    const int items = (int)((P + (long long)ctas * CS_THREADS - 1) / ((long long)ctas * CS_THREADS));
    const int passes = (sp.bits + CS_BITS - 1) / CS_BITS, per = (sp.bits + passes - 1) / passes;
    long long more = 0;
    if (dw->dw) {
      more = (dw->n * ((dw->R + DW_U - 1) / DW_U) + CS_WARPS - 1) / CS_WARPS;
      if (more > 148 - ctas) more = 148 - ctas;
      more = (more + ctas - 1) / ctas * ctas;
    }
    launch_cluster(sort_cluster_kernel<T, I, VEC>, (unsigned)(ctas + more), CS_THREADS, (unsigned)ctas, CS_SMEM, s,
                   (const I*)idx, (int)P, c.rows, per, passes, ctas, items, w.item[0], *dw);
    dw->dw = nullptr;
    *sorted = 0;
    return 1;
  }
  const size_t smem = 4 * 2 * (size_t)sp.bins + 2 * (size_t)RS_WARPS * sp.bins;
  if (!raise_smem_limit((const void*)sort_scatter_kernel<I>, smem)) return -1;
  const int own = sp.tiles <= RS_OWN_SCAN;
  int nl = 0;
  for (int pass = 0; pass < sp.passes; ++pass) {
    const int from = (pass + 1) & 1, to = pass & 1;
    Source<I> src{(const I*)idx, pass ? w.item[from] : nullptr, c.rows};
    launch_k(sort_hist_kernel<I>, sp.tiles, RS_THREADS, 0, s, src, P, pass * sp.per, sp.bins, w.hist);
    ++nl;
    if (!own) {
      launch_k(sort_scan_kernel, (sp.bins + 127) / 128, 128, 0, s, w.hist, w.total, sp.tiles, sp.bins);
      ++nl;
    }
    launch_k(sort_scatter_kernel<I>, sp.tiles, RS_THREADS, smem, s, src, P, pass * sp.per, sp.bins,
             (const uint32_t*)w.hist, (const uint32_t*)w.total, sp.tiles, own, w.item[to]);
    ++nl;
    *sorted = to;
  }
  return nl;
}

template <typename T, typename G, int VEC, bool ACC>
int go_sum(const fwpkm_lookup_config& c, SegArgs a, const void* d_out, void* d_table, cudaStream_t s) {
  a.vecs = c.width / VEC;
  a.tx_n = row_threads(a.vecs);
  const int ty = LK_THREADS / a.tx_n;
  const unsigned gy = (unsigned)((a.vecs + a.tx_n - 1) / a.tx_n);
  const unsigned sb = (unsigned)((a.ranges + ty - 1) / ty);
  // dense gradient: CTAs that zero the rows nothing reads, a few rows per warp (up to 16 per SM's
  // place, then more; column blocks share one row split: only blockIdx.y == 0 has them)
  long long zb = 0;
  if (!ACC) {
    const int each = LK_THREADS / 32 * zero_rows((long long)c.width * sizeof(G));
    zb = (a.rows + each - 1) / each;
    if (zb > 148 * 32) zb = 148 * 32;
  }
  if (sb + zb == 0) return 0;
  int nl = 0;
  if (gy == 1) {
    launch_k(lookup_sum_kernel<T, G, VEC, ACC>, dim3(sb + (unsigned)zb), LK_THREADS, 0, s, a, (const T*)d_out,
             (G*)d_table, (int)sb);
    ++nl;
  } else {
    if (zb) {
      launch_k(lookup_sum_kernel<T, G, VEC, ACC>, dim3((unsigned)zb), LK_THREADS, 0, s, a, (const T*)d_out, (G*)d_table, 0);
      ++nl;
    }
    if (sb) {
      launch_k(lookup_sum_kernel<T, G, VEC, ACC>, dim3(sb, gy), LK_THREADS, 0, s, a, (const T*)d_out, (G*)d_table,
               (int)sb);
      ++nl;
    }
  }
  if (a.ranges > 1) {
    launch_k(lookup_join_kernel<G, VEC, ACC>, dim3(sb, gy), LK_THREADS, 0, s, a, (G*)d_table);
    ++nl;
  }
  return nl;
}

template <typename T, typename G, int VEC>
int go_sum_a(const fwpkm_lookup_config& c, const SegArgs& a, const void* d_out, void* d_table, cudaStream_t s) {
  return a.accumulate ? go_sum<T, G, VEC, true>(c, a, d_out, d_table, s)
                      : go_sum<T, G, VEC, false>(c, a, d_out, d_table, s);
}

template <typename T, typename G>
int go_sum_v(const fwpkm_lookup_config& c, const SegArgs& a, const void* d_out, void* d_table, cudaStream_t s) {
  if (rows_vec<T>(d_out, c.out_ld, c.width) && rows_vec<G>(d_table, a.grad_ld, c.width))
    return go_sum_a<T, G, 16 / (int)sizeof(T)>(c, a, d_out, d_table, s);
  return go_sum_a<T, G, 1>(c, a, d_out, d_table, s);
}

// Sort (if there is a d_table to form) and dw, by the table's and the indices' types.
template <typename T, typename I, int VEC>
int go_pairs(const fwpkm_lookup_config& c, const void* idx, long long P, const BackWork* w, int* sorted, DwArgs dw,
             cudaStream_t s) {
  dw.vecs = c.width / VEC;
  int nl = 0;
  if (w) {
    nl = go_sort<T, I, VEC>(c, idx, P, *w, sorted, &dw, s);
    if (nl < 0) return -1;
  }
  if (dw.dw) {
    const long long jobs = dw.n * ((c.R + DW_U - 1) / DW_U);
    const unsigned g = (unsigned)((jobs + LK_THREADS / 32 - 1) / (LK_THREADS / 32));
    launch_k(lookup_dw_kernel<T, I, VEC>, g, LK_THREADS, 0, s, dw, (const I*)idx);
    ++nl;
  }
  return nl;
}

template <typename T>
int go_pairs_t(const fwpkm_lookup_config& c, const void* idx, long long P, const BackWork* w, int* sorted,
               const DwArgs& dw, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  const bool vec = !dw.dw || (rows_vec<T>(dw.table, c.table_ld, c.width) && rows_vec<T>(dw.d_out, c.out_ld, c.width));
  if (c.idx_dtype == FWPKM_I64)
    return vec ? go_pairs<T, long long, V>(c, idx, P, w, sorted, dw, s)
               : go_pairs<T, long long, 1>(c, idx, P, w, sorted, dw, s);
  return vec ? go_pairs<T, int, V>(c, idx, P, w, sorted, dw, s) : go_pairs<T, int, 1>(c, idx, P, w, sorted, dw, s);
}

}  // namespace
}  // namespace fwpkm

using namespace fwpkm;

extern "C" {

fwpkm_status fwpkm_lookup(const fwpkm_lookup_config* cfg, const void* table, const void* idx, const float* w,
                          long long n, void* out, void* stream) {
  NvtxRange nvtx_range("fwpkm_lookup");
  const fwpkm_status cs = check_lookup(cfg, n);
  if (cs != FWPKM_OK) return cs;
  if (n == 0) return FWPKM_OK;
  const size_t es = dsize(cfg->dtype);
  if (!table || !idx || !out || !ptr_al(table, es) || !ptr_al(out, es) || (w && !ptr_al(w, 4)) ||
      !ptr_al(idx, cfg->idx_dtype == FWPKM_I64 ? 8 : 4) || out == table || out == w)
    return FWPKM_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  cudaGetLastError();
  PdlScope pdl(true);
  const bool i64 = cfg->idx_dtype == FWPKM_I64;
  if (cfg->dtype == FWPKM_BF16) {
    if (i64) go_lookup_v<__nv_bfloat16, long long>(*cfg, table, idx, w, n, out, s);
    else go_lookup_v<__nv_bfloat16, int>(*cfg, table, idx, w, n, out, s);
  } else {
    if (i64) go_lookup_v<float, long long>(*cfg, table, idx, w, n, out, s);
    else go_lookup_v<float, int>(*cfg, table, idx, w, n, out, s);
  }
  return done(1);
}

fwpkm_status fwpkm_lookup_backward_workspace_size(const fwpkm_lookup_config* cfg, long long n, size_t* bytes) {
  const fwpkm_status cs = check_lookup(cfg, n);
  if (cs != FWPKM_OK) return cs;
  if (!bytes) return FWPKM_ERR_INVALID_ARG;
  *bytes = back_carve(*cfg, n * cfg->R, nullptr, nullptr);
  return FWPKM_OK;
}

fwpkm_status fwpkm_lookup_backward(const fwpkm_lookup_config* cfg, const void* table, const void* idx, const float* w,
                                   const void* d_out, long long n, void* d_table, long long grad_ld, int grad_dtype,
                                   int accumulate, float* dw, void* workspace, size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("fwpkm_lookup_backward");
  const fwpkm_status cs = check_lookup(cfg, n);
  if (cs != FWPKM_OK) return cs;
  if (d_table && (grad_ld < cfg->width || (grad_dtype != FWPKM_F32 && grad_dtype != FWPKM_BF16)))
    return FWPKM_ERR_INVALID_ARG;
  const size_t es = dsize(cfg->dtype);
  if (d_table && !ptr_al(d_table, dsize(grad_dtype))) return FWPKM_ERR_INVALID_ARG;
  if (n > 0) {
    if (!idx || !d_out || !ptr_al(d_out, es) || (w && !ptr_al(w, 4)) || (dw && (!table || !ptr_al(table, es) || !ptr_al(dw, 4))) ||
        !ptr_al(idx, cfg->idx_dtype == FWPKM_I64 ? 8 : 4))
      return FWPKM_ERR_INVALID_ARG;
    if (d_table) {
      if (!workspace || !ptr_al(workspace, 256)) return FWPKM_ERR_INVALID_ARG;
      if (ws_bytes < back_carve(*cfg, n * cfg->R, nullptr, nullptr)) return FWPKM_ERR_WORKSPACE;
    }
    // outputs in the memory of what is still to be read (the table is not, once dw is formed)
    const uintptr_t w0 = (uintptr_t)w, dw0 = (uintptr_t)dw, bytes = 4 * (uintptr_t)(n * cfg->R);
    if (d_table && (d_table == d_out || d_table == w || (w && dw && dw0 < w0 + bytes && w0 < dw0 + bytes)))
      return FWPKM_ERR_INVALID_ARG;
    if (dw && (dw == d_out || dw == table)) return FWPKM_ERR_INVALID_ARG;
  }
  if (n == 0 && (!d_table || accumulate)) return FWPKM_OK;
  cudaStream_t s = (cudaStream_t)stream;
  cudaGetLastError();
  PdlScope pdl(true);
  const bool bf = cfg->dtype == FWPKM_BF16;
  const long long P = n * cfg->R;
  BackWork bw = {};
  int nl = 0, at = 0;
  if (P > 0) {
    if (d_table) back_carve(*cfg, P, (char*)workspace, &bw);
    DwArgs g = {};
    g.table = table; g.d_out = d_out; g.dw = dw;
    g.rows = cfg->rows; g.ld = cfg->table_ld; g.out_ld = cfg->out_ld; g.n = n; g.R = cfg->R; g.scale = cfg->scale;
    const BackWork* w = d_table ? &bw : nullptr;
    nl = bf ? go_pairs_t<__nv_bfloat16>(*cfg, idx, P, w, &at, g, s) : go_pairs_t<float>(*cfg, idx, P, w, &at, g, s);
    if (nl < 0) return FWPKM_ERR_CUDA;
    // (the sums take rows to write from the sorted pairs: where a launch above was refused, those are
    // whatever the workspace held)
    if (cudaPeekAtLastError() != cudaSuccess) return done(0);
  }
  if (d_table) {
    SegArgs a = {};
    a.P = P;
    a.rows = cfg->rows; a.out_ld = cfg->out_ld; a.grad_ld = grad_ld;
    a.R = cfg->R; a.width = cfg->width; a.scale = cfg->scale; a.accumulate = accumulate != 0;
    a.seg = seg_pairs(P);
    a.ranges = (P + a.seg - 1) / a.seg;
    a.w = w;
    a.item = bw.item[at];
    a.part = bw.part;
    if (bf)
      nl += grad_dtype == FWPKM_BF16 ? go_sum_v<__nv_bfloat16, __nv_bfloat16>(*cfg, a, d_out, d_table, s)
                                     : go_sum_v<__nv_bfloat16, float>(*cfg, a, d_out, d_table, s);
    else
      nl += grad_dtype == FWPKM_BF16 ? go_sum_v<float, __nv_bfloat16>(*cfg, a, d_out, d_table, s)
                                     : go_sum_v<float, float>(*cfg, a, d_out, d_table, s);
  }
  return done(nl);
}

}  // extern "C"
