// Embedding lookup and its gradient.
//
//   forward   out[i] = scale * table[id_i]            (zeros for an id outside [0, vocab))
//   gradient  dtable[v] = scale * sum_{i : id_i = v} dout[i]
//
// Both are bound by memory: the lookup reads each distinct row once and writes
// every output row; the gradient reads every dout row once and writes every
// row of the table's gradient, most of them zeros for a large vocabulary.
//
// The gradient sorts the (id, position) pairs, stably, so that each row's
// terms lie together in the order of their positions: one sum per row in that
// order, in fp32, with no atomics on values, so results repeat bit for bit.
// The order comes from one kernel up to 65,536 tokens: by counting the pairs
// before each (n^2 comparisons, no passes), or a radix sort by one cluster of
// blocks; above that from a device-wide radix sort.  The sorted list is cut into
// chunks of equal length, one warp per chunk and column segment, so that a
// frequent token's many rows are shared by many warps: a run that crosses a
// chunk's border leaves fp32 partial sums, which a second kernel adds in order.
// The blocks after those of the sums clear the rows that no token names, found
// by a search in the sorted list.
#include <stdint.h>

#include "internal.hpp"
#include "lm.hpp"
#include "prims.cuh"

namespace snack {
namespace {

// A warp per row and segment of it, kFwdUnroll accesses in flight per lane, so
// that a few rows still spread over the SMs.  32768 rows of 4096 bf16 out of
// 131072: 56 us, 6.5 TB/s; 8 rows of 1024 fp32: 1.6 us.
constexpr int kFwdUnroll = 4;

template <typename T, int B>
__global__ void __launch_bounds__(256) k_embed_fwd(TokenSrc ids, int64_t n, const T *__restrict__ table,
                                                   int64_t table_ld, int32_t width, float scale, T *__restrict__ out,
                                                   int64_t out_ld) {
  pdl_wait();
  typedef Pack<T, B> P;
  const int64_t row = (int64_t)blockIdx.x * 8 + threadIdx.y;
  if (row >= n) return;
  const uint32_t id = ids.key(row);
  const int acc = width / P::kN;
  const int a0 = blockIdx.y * (32 * kFwdUnroll) + threadIdx.x;
  T *o = out + row * out_ld;
  const T *t = table + (int64_t)id * table_ld;
  P v[kFwdUnroll];
#pragma unroll
  for (int u = 0; u < kFwdUnroll; ++u) {
    const int a = a0 + u * 32;
    if (a < acc && id < ids.vocab) v[u].raw = __ldg(reinterpret_cast<const typename P::R *>(t) + a);
  }
#pragma unroll
  for (int u = 0; u < kFwdUnroll; ++u) {
    const int a = a0 + u * 32;
    if (a >= acc) continue;
#pragma unroll
    for (int i = 0; i < P::kN; ++i) v[u].set(i, id < ids.vocab ? scale * v[u].get(i) : 0.f);
    reinterpret_cast<typename P::R *>(o)[a] = v[u].raw;
  }
}

// ------------------------------------------------------------ sorted order

constexpr int kRankMax = 4096;
constexpr int kRankRows = 32;  // tokens per block
constexpr int kRankThreads = 256;

// Place of token i among all: the number of (id, position) pairs before its
// own.  Lane l of every warp holds token 32 blockIdx.x + l; the eight warps
// count over interleaved groups of 32 tokens, whose ids they read from shared
// memory (every lane the same word).
__global__ void __launch_bounds__(kRankThreads) k_rank(TokenSrc ids, int n, uint32_t *__restrict__ keys,
                                                       uint32_t *__restrict__ pos) {
  pdl_wait();
  __shared__ __align__(16) uint32_t s_ids[kRankMax];
  __shared__ int cnt[kRankThreads / 32][kRankRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = (n + 31) / 32;
  for (int i = threadIdx.x; i < groups * 32; i += kRankThreads) s_ids[i] = i < n ? ids.key(i) : 0xFFFFFFFFu;
  __syncthreads();
  const int own = blockIdx.x;
  const int i = own * 32 + lane;
  const uint32_t mine = s_ids[i];
  int c = 0;
  for (int g = warp; g < groups; g += kRankThreads / 32) {
    if (g == own) {
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const uint32_t k = s_ids[g * 32 + j];
        c += (k < mine || (k == mine && j < lane)) ? 1 : 0;
      }
    } else {
      const uint4 *q = reinterpret_cast<const uint4 *>(s_ids + g * 32);
      const uint32_t lim = g < own ? mine + 1u : mine;  // an earlier token of the same id comes first
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint4 k = q[j];
        c += (k.x < lim) + (k.y < lim) + (k.z < lim) + (k.w < lim);
      }
    }
  }
  cnt[warp][lane] = c;
  __syncthreads();
  if (warp == 0 && i < n) {
    int r = 0;
#pragma unroll
    for (int w = 0; w < kRankThreads / 32; ++w) r += cnt[w][lane];
    keys[r] = mine;
    pos[r] = (uint32_t)i;
  }
}

// Rows of the table's gradient to clear, in 16-byte accesses where they allow it.
struct ZeroRows {
  uint8_t *base;
  int64_t row_bytes, ld_bytes, rows;
  int wide;
};
__device__ __forceinline__ void clear_row(const ZeroRows &z, int64_t r) {  // a warp
  const int lane = threadIdx.x & 31;
  uint8_t *row = z.base + r * z.ld_bytes;
  if (z.wide) {
    uint4 *o = reinterpret_cast<uint4 *>(row);
    for (int64_t i = lane; i < z.row_bytes / 16; i += 32) __stcs(o + i, make_uint4(0, 0, 0, 0));
  } else {
    uint16_t *o = reinterpret_cast<uint16_t *>(row);
    for (int64_t i = lane; i < z.row_bytes / 2; i += 32) o[i] = 0;
  }
}

// A stable LSD radix sort of up to 65,536 pairs by one cluster, in one launch.
// Each of its eight blocks holds `tile` pairs in shared memory; a pass of up to
// nine bits ranks them (a warp's equal digits by ballots, its counts before them in
// its own histogram), the blocks read each other's digit totals, and every pair
// goes straight to its place in the shared memory of the block that holds it.
// About 16 us at 32768 tokens; the other SMs clear the table's first rows, as
// many as that takes.
constexpr int kSortBlocks = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortRounds = 8;  // pairs per thread
constexpr int kSortMost = kSortBlocks * kSortThreads * kSortRounds;
constexpr size_t kSortTile = (size_t)kSortThreads * kSortRounds;
// two buffers of pairs, and the warps' histograms
constexpr int kSortBins = 512;  // digits of up to nine bits: two passes up to 2^18 ids
constexpr size_t kSortSmem = 2 * kSortTile * 8 + (size_t)kSortWarps * kSortBins * 4;

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t block) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(block));
  return r;
}

__global__ void __cluster_dims__(kSortBlocks, 1, 1) __launch_bounds__(kSortThreads, 1)
    k_sort(TokenSrc ids, int n, int tile_bits, int passes, int digit_bits, uint32_t *__restrict__ keys, uint32_t *__restrict__ pos,
           const ZeroRows zero) {
  pdl_wait();
  if (blockIdx.x >= kSortBlocks) {  // the clusters after the first clear rows meanwhile
    const int warp = threadIdx.x >> 5;
    for (int64_t r = (int64_t)(blockIdx.x - kSortBlocks) * kSortWarps + warp; r < zero.rows;
         r += (int64_t)(gridDim.x - kSortBlocks) * kSortWarps)
      clear_row(zero, r);
    return;
  }
  extern __shared__ __align__(16) uint8_t sort_smem[];
  uint2 *buf = reinterpret_cast<uint2 *>(sort_smem);  // [2][tile]
  uint32_t(*hist)[kSortBins] = reinterpret_cast<uint32_t(*)[kSortBins]>(sort_smem + 2 * kSortTile * 8);
  __shared__ uint32_t totals[kSortBins];  // this block's pairs by digit
  __shared__ uint32_t base[kSortBins];    // where they start in the whole order
  __shared__ uint32_t warp_sum[kSortBins / 32];
  const uint32_t bins = 1u << digit_bits, mask = bins - 1u;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t block = blockIdx.x;
  const int tile = 1 << tile_bits;
  const int first = (int)block * tile, mine = max(0, min(tile, n - first));
  const int rounds = tile / kSortThreads;  // a warp's pairs, 32 at a time
  const uint32_t below = (1u << lane) - 1u;
  for (int i = threadIdx.x; i < mine; i += kSortThreads) buf[i] = make_uint2(ids.key(first + i), (uint32_t)(first + i));
  for (int p = 0; p < passes; ++p) {
    uint2 *in = buf + (p & 1) * tile, *out = buf + ((p & 1) ^ 1) * tile;
    for (int i = threadIdx.x; i < kSortWarps * kSortBins; i += kSortThreads) (&hist[0][0])[i] = 0;
    __syncthreads();
    uint2 pair[kSortRounds];
    uint32_t rank[kSortRounds];
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
      if (r >= rounds) break;
      const int at = (warp * rounds + r) * 32 + lane;
      const bool here = at < mine;
      if (here) pair[r] = in[at];
      const uint32_t digit = here ? (pair[r].x >> (digit_bits * p)) & mask : bins;
      unsigned peers = 0xffffffffu;
#pragma unroll
      for (int bit = 0; bit < 10; ++bit) {
        if (bit > digit_bits) break;
        const bool on = (digit >> bit) & 1;
        const unsigned bal = __ballot_sync(0xffffffffu, on);
        peers &= on ? bal : ~bal;
      }
      const uint32_t c = here ? hist[warp][digit] : 0u;
      rank[r] = c + (uint32_t)__popc(peers & below);
      __syncwarp();
      if (here && (peers >> lane) == 1u) hist[warp][digit] = c + (uint32_t)__popc(peers);
      __syncwarp();
    }
    __syncthreads();
    if (threadIdx.x < kSortBins) {  // pairs of earlier warps, and the block's total
      uint32_t t = 0;
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = hist[w][threadIdx.x];
        hist[w][threadIdx.x] = t;
        t += c;
      }
      totals[threadIdx.x] = t;
    }
    cluster_sync();
    if (threadIdx.x < kSortBins) {
      uint32_t all = 0, before = 0;
#pragma unroll
      for (uint32_t b = 0; b < kSortBlocks; ++b) {
        uint32_t t;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(t) : "r"(cluster_addr(&totals[threadIdx.x], b)) : "memory");
        all += t;
        if (b < block) before += t;
      }
      const uint32_t inc = warp_inclusive_scan(all);
      if (lane == 31) warp_sum[warp] = inc;
      base[threadIdx.x] = before + inc - all;
    }
    __syncthreads();
    if (threadIdx.x < kSortBins) {
      uint32_t o = 0;
      for (int w = 0; w < warp; ++w) o += warp_sum[w];
      base[threadIdx.x] += o;
    }
    __syncthreads();
    const bool last = p + 1 == passes;
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
      if (r >= rounds) break;
      const int at = (warp * rounds + r) * 32 + lane;
      if (at < mine) {
        const uint32_t digit = (pair[r].x >> (digit_bits * p)) & mask;
        const uint32_t to = base[digit] + hist[warp][digit] + rank[r];
        if (last) {
          keys[to] = pair[r].x;
          pos[to] = pair[r].y;
        } else {
          const uint32_t b = to >> tile_bits;
          asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(cluster_addr(&out[to & (uint32_t)(tile - 1)], b)),
                       "r"(pair[r].x), "r"(pair[r].y)
                       : "memory");
        }
      }
    }
    cluster_sync();  // the next pass's input is in place; after the last, no block's memory is read any more
  }
}

// ------------------------------------------------------------ gradient

struct EmbedGrad {
  const uint32_t *keys, *pos;  // [n] sorted ids (vocab: none) and their positions
  int64_t n;
  const void *dout;
  int64_t dout_ld;
  void *dtable;
  int64_t table_ld;
  uint32_t vocab;
  int32_t width;
  float scale;
  int accumulate;
  float *part;      // [chunks][2][part_ld] sums of the runs that a chunk begins with (0) and ends with (1);
                    //  element i of a lane's access a at i * accesses + a, so a warp's stores are whole lines
  int64_t part_ld;
  int chunk;        // sorted entries per chunk
  int64_t n_chunks;
  int n_seg;        // column segments
  int64_t sum_blocks;
  ZeroRows zero;    // the rows that no token names, from `cleared` on,
  int64_t cleared;
  int zero_rows;    // so many per warp
};

constexpr int kGradWarps = 8;
constexpr int kGradVecs = 2;   // accesses per lane
constexpr int kGradBatch = 4;  // rows in flight per lane
constexpr int kZeroMost = 8;   // rows per warp of the clearing, at most

__device__ __forceinline__ int64_t lower_bound(const uint32_t *__restrict__ k, int64_t n, uint32_t v) {
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (__ldg(k + mid) < v)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

template <typename T>
__device__ __forceinline__ T *table_row(const EmbedGrad &g, uint32_t row) {
  return reinterpret_cast<T *>(g.dtable) + (int64_t)row * g.table_ld;
}

// this lane's accesses of a row as it is (accumulate)
template <typename T, int B>
__device__ __forceinline__ void get_row(const EmbedGrad &g, uint32_t row, int a0, int acc_n, Pack<T, B> (&old)[kGradVecs]) {
  const typename Pack<T, B>::R *o = reinterpret_cast<const typename Pack<T, B>::R *>(table_row<T>(g, row));
#pragma unroll
  for (int u = 0; u < kGradVecs; ++u)
    if (a0 + 32 * u < acc_n) old[u].raw = o[a0 + 32 * u];
}

// this lane's accesses of one row of the gradient: scale * acc (+ what was there)
template <typename T, int B>
__device__ __forceinline__ void put_row(const EmbedGrad &g, uint32_t row, int a0, int acc_n,
                                        const float (&acc)[kGradVecs][Pack<T, B>::kN], bool add,
                                        const Pack<T, B> (&old)[kGradVecs]) {
  typedef Pack<T, B> P;
  typename P::R *o = reinterpret_cast<typename P::R *>(table_row<T>(g, row));
#pragma unroll
  for (int u = 0; u < kGradVecs; ++u) {
    const int a = a0 + 32 * u;
    if (a >= acc_n) continue;
    P v;
#pragma unroll
    for (int i = 0; i < P::kN; ++i) {
      const float t = g.scale * acc[u][i];
      v.set(i, add ? old[u].get(i) + t : t);
    }
    o[a] = v.raw;
  }
}

// kAdd: the sums are added to the rows that are there, which are read with the
// batch in which their run begins.  With the clearing, 6.5 TB/s for 32768 rows of
// 4096 bf16 over a table of 131072 (227 us with the sort, 16, and the join, 15).
template <typename T, int B, bool kAdd>
__global__ void __launch_bounds__(kGradWarps * 32) k_embed_sum(const EmbedGrad g) {
  pdl_wait();
  typedef Pack<T, B> P;
  constexpr int kBatch = kAdd ? kGradBatch / 2 : kGradBatch;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int acc_n = g.width / P::kN;
  const bool sums = (int64_t)blockIdx.x < g.sum_blocks;
  const int64_t own = sums ? (int64_t)blockIdx.x : (int64_t)blockIdx.x - g.sum_blocks;
  if (!sums) {  // ---- rows that no token names
    const int64_t v0 = g.cleared + (own * kGradWarps + warp) * g.zero_rows;
    bool absent = false;
    if (lane < g.zero_rows && v0 + lane < (int64_t)g.vocab) {
      const uint32_t v = (uint32_t)(v0 + lane);
      const int64_t at = lower_bound(g.keys, g.n, v);
      absent = at >= g.n || __ldg(g.keys + at) != v;
    }
    const unsigned rows = __ballot_sync(0xffffffffu, absent);
    for (int r = 0; r < g.zero_rows; ++r)
      if ((rows >> r) & 1u) clear_row(g.zero, v0 + r);
    return;
  }
  const int64_t gw = own * kGradWarps + warp;
  const int64_t c = gw / g.n_seg;
  if (c >= g.n_chunks) return;
  const int seg = (int)(gw - c * g.n_seg);
  const int a0 = seg * (32 * kGradVecs) + lane;
  const int64_t j0 = c * g.chunk, j1 = min(j0 + (int64_t)g.chunk, g.n);
  const uint32_t first = __ldg(g.keys + j0);
  if (first >= g.vocab) return;  // only tokens outside the vocabulary from here on
  const bool from_before = j0 > 0 && __ldg(g.keys + j0 - 1) == first;
  const uint32_t after = j1 < g.n ? __ldg(g.keys + j1) : 0xFFFFFFFFu;
  const T *dout = reinterpret_cast<const T *>(g.dout);
  float acc[kGradVecs][P::kN];
#pragma unroll
  for (int u = 0; u < kGradVecs; ++u)
#pragma unroll
    for (int i = 0; i < P::kN; ++i) acc[u][i] = 0.f;
  uint32_t cur = first;
  bool head = from_before;  // the current run began in an earlier chunk
  P old[kGradVecs];         // the current run's row (kAdd)
  if (kAdd) get_row<T, B>(g, cur, a0, acc_n, old);
  auto keep_part = [&](int which) {
    float *p = g.part + (c * 2 + which) * g.part_ld;
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u)
      if (a0 + 32 * u < acc_n)
#pragma unroll
        for (int i = 0; i < P::kN; ++i) p[(int64_t)i * acc_n + a0 + 32 * u] = acc[u][i];
  };
  for (int64_t b = j0; b < j1 && cur < g.vocab; b += 32) {
    const uint32_t my_key = b + lane < j1 ? __ldg(g.keys + b + lane) : 0xFFFFFFFFu;
    const uint32_t my_pos = b + lane < j1 ? __ldg(g.pos + b + lane) : 0u;
    const int m = (int)min((int64_t)32, j1 - b);
    for (int e0 = 0; e0 < m && cur < g.vocab; e0 += kBatch) {
      P v[kBatch][kGradVecs], was[kAdd ? kBatch : 1][kGradVecs];
      uint32_t prev = cur;
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const uint32_t k = __shfl_sync(0xffffffffu, my_key, e0 + e), p = __shfl_sync(0xffffffffu, my_pos, e0 + e);
        if (kAdd && k != prev && k < g.vocab) get_row<T, B>(g, k, a0, acc_n, was[kAdd ? e : 0]);
        prev = k;
        const typename P::R *src = reinterpret_cast<const typename P::R *>(dout + (int64_t)p * g.dout_ld);
#pragma unroll
        for (int u = 0; u < kGradVecs; ++u)
          if (k < g.vocab && a0 + 32 * u < acc_n) v[e][u].raw = __ldcs(src + a0 + 32 * u);
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const uint32_t k = __shfl_sync(0xffffffffu, my_key, e0 + e);
        if (k != cur) {
          if (cur >= g.vocab) break;
          if (e0 + e >= m) break;  // the chunk's end: its last run is finished below
          if (head)
            keep_part(0);
          else
            put_row<T, B>(g, cur, a0, acc_n, acc, kAdd, old);
          head = false;
          cur = k;
          if (cur >= g.vocab) break;
          if (kAdd)
#pragma unroll
            for (int u = 0; u < kGradVecs; ++u) old[u].raw = was[kAdd ? e : 0][u].raw;
#pragma unroll
          for (int u = 0; u < kGradVecs; ++u)
#pragma unroll
            for (int i = 0; i < P::kN; ++i) acc[u][i] = 0.f;
        }
#pragma unroll
        for (int u = 0; u < kGradVecs; ++u)
          if (a0 + 32 * u < acc_n)
#pragma unroll
            for (int i = 0; i < P::kN; ++i) acc[u][i] += v[e][u].get(i);
      }
    }
  }
  if (cur >= g.vocab) return;
  if (head)
    keep_part(0);
  else if (after == cur)
    keep_part(1);
  else
    put_row<T, B>(g, cur, a0, acc_n, acc, kAdd, old);
}

// A run that crosses chunk borders: the chunk it begins in adds the partial
// sums of the chunks it covers, in order.  A warp does so for a run of up to
// kJoinShort chunks; for a longer one the block's warps take an equal stretch
// of it each, and their sums are added in the stretches' order.  (A block's
// warps hold neighbouring chunks of one segment: few long runs begin in them.)
constexpr int kJoinShort = 24;

template <typename T, int B>
__device__ __forceinline__ void add_parts(const EmbedGrad &g, int64_t q0, int64_t q1, int a0, int acc_n,
                                          float (&acc)[kGradVecs][Pack<T, B>::kN]) {
  constexpr int kN = Pack<T, B>::kN;
  constexpr int kJoinBatch = kN >= 8 ? 4 : 8;
  for (; q0 < q1; q0 += kJoinBatch) {  // loads of several chunks in flight
    float v[kJoinBatch][kGradVecs][kN];
#pragma unroll
    for (int e = 0; e < kJoinBatch; ++e) {
      const float *p = g.part + (q0 + e) * 2 * g.part_ld;
#pragma unroll
      for (int u = 0; u < kGradVecs; ++u)
#pragma unroll
        for (int i = 0; i < kN; ++i)
          v[e][u][i] = q0 + e < q1 && a0 + 32 * u < acc_n ? __ldcg(p + (int64_t)i * acc_n + a0 + 32 * u) : 0.f;
    }
#pragma unroll
    for (int e = 0; e < kJoinBatch; ++e)
#pragma unroll
      for (int u = 0; u < kGradVecs; ++u)
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (q0 + e < q1) acc[u][i] += v[e][u][i];
  }
}

template <typename T, int B>
__global__ void __launch_bounds__(kGradWarps * 32) k_embed_join(const EmbedGrad g) {
  pdl_wait();
  constexpr int kN = Pack<T, B>::kN;
  __shared__ int64_t s_last[kGradWarps];  // a long run's last chunk, else -1
  __shared__ uint32_t s_key[kGradWarps];
  __shared__ float s_sum[kGradWarps][32 * kGradVecs * kN];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int acc_n = g.width / kN;
  float acc[kGradVecs][kN];
  Pack<T, B> old[kGradVecs];
  auto clear = [&] {
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u)
#pragma unroll
      for (int i = 0; i < kN; ++i) acc[u][i] = 0.f;
  };
  auto tail = [&](int64_t c, int a0) {  // what the chunk the run begins in left over
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u)
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (a0 + 32 * u < acc_n) acc[u][i] = g.part[(c * 2 + 1) * g.part_ld + (int64_t)i * acc_n + a0 + 32 * u];
  };
  const int64_t w0 = (int64_t)blockIdx.x * kGradWarps;
  int64_t last_long = -1;
  {
    const int64_t gw = w0 + warp, seg = gw / g.n_chunks, c = gw - seg * g.n_chunks;
    if (seg < g.n_seg && c + 1 < g.n_chunks) {
      const int64_t j0 = c * g.chunk, j1 = j0 + g.chunk;
      const uint32_t cur = __ldg(g.keys + j1 - 1);
      const bool crosses = cur < g.vocab && __ldg(g.keys + j1) == cur;
      const bool earlier = j0 > 0 && __ldg(g.keys + j0) == cur && __ldg(g.keys + j0 - 1) == cur;
      if (crosses && !earlier) {
        int64_t last = c;  // the chunk it ends in: those after c that begin with it, 32 looked at per step
        for (;;) {
          const int64_t q = last + 1 + lane;
          const unsigned same = __ballot_sync(0xffffffffu, q < g.n_chunks && __ldg(g.keys + q * g.chunk) == cur);
          last += __popc(same);
          if (same != 0xffffffffu) break;
        }
        if (last - c > kJoinShort) {
          last_long = last;
          if (lane == 0) s_key[warp] = cur;
        } else {
          const int a0 = (int)seg * (32 * kGradVecs) + lane;
          clear();
          tail(c, a0);
          add_parts<T, B>(g, c + 1, last + 1, a0, acc_n, acc);
          if (g.accumulate) get_row<T, B>(g, cur, a0, acc_n, old);
          put_row<T, B>(g, cur, a0, acc_n, acc, g.accumulate != 0, old);
        }
      }
    }
  }
  if (lane == 0) s_last[warp] = last_long;
  if (!__syncthreads_or(last_long >= 0)) return;
  for (int k = 0; k < kGradWarps; ++k) {
    const int64_t last = s_last[k];
    if (last < 0) continue;
    const int64_t gw = w0 + k, seg = gw / g.n_chunks, c = gw - seg * g.n_chunks, n = last - c;
    const int a0 = (int)seg * (32 * kGradVecs) + lane;
    clear();
    if (warp == 0) tail(c, a0);
    add_parts<T, B>(g, c + 1 + n * warp / kGradWarps, c + 1 + n * (warp + 1) / kGradWarps, a0, acc_n, acc);
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u)
#pragma unroll
      for (int i = 0; i < kN; ++i) s_sum[warp][(u * kN + i) * 32 + lane] = acc[u][i];
    __syncthreads();
    if (warp == 0) {
      for (int q = 1; q < kGradWarps; ++q)
#pragma unroll
        for (int u = 0; u < kGradVecs; ++u)
#pragma unroll
          for (int i = 0; i < kN; ++i) acc[u][i] += s_sum[q][(u * kN + i) * 32 + lane];
      if (g.accumulate) get_row<T, B>(g, s_key[k], a0, acc_n, old);
      put_row<T, B>(g, s_key[k], a0, acc_n, acc, g.accumulate != 0, old);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------ host side

int key_bits(uint32_t vocab) {
  int b = 0;
  while (b < 32 && (vocab >> b)) ++b;
  return b;  // keys are 0 .. vocab
}

constexpr int kSegElems = 32 * kGradVecs;  // accesses per segment

struct GradWs {
  size_t keys, pos, k0, v0, k1, v1, temp, part, total;
  int chunk;
  int64_t n_chunks, part_ld;
};

// Chunks short enough that a small call still has some thousand warps; the
// partial sums of a run that covers many chunks are added by one warp per
// segment, so long calls get longer chunks.
GradWs grad_ws(int64_t n, int32_t width) {
  GradWs w;
  const int64_t segs = ceil_div(width, 512);  // at 16-byte accesses; narrower ones have more
  int64_t chunk = 8;
  while (chunk < 4096 && n / chunk * segs > 4096) chunk *= 2;
  w.chunk = (int)chunk;
  w.n_chunks = n > 0 ? (n + chunk - 1) / chunk : 0;
  w.part_ld = (int64_t)align_up((size_t)width, 4);
  size_t o = 0;
  w.keys = o;
  o += align_up((size_t)n * 4, kAlign);
  w.pos = o;
  o += align_up((size_t)n * 4, kAlign);
  const bool radix = n > kSortMost;
  w.k0 = o;
  if (radix) o += align_up((size_t)n * 4, kAlign);
  w.v0 = o;
  if (radix) o += align_up((size_t)n * 4, kAlign);
  w.k1 = o;
  if (radix) o += align_up((size_t)n * 4, kAlign);
  w.v1 = o;
  if (radix) o += align_up((size_t)n * 4, kAlign);
  w.temp = o;
  if (radix) o += align_up(radix_temp_bytes(n), kAlign);
  w.part = o;
  o += align_up((size_t)w.n_chunks * 2 * (size_t)w.part_ld * 4, kAlign);
  w.total = o;
  return w;
}

bool embed_sizes_ok(int64_t n, int64_t vocab, int32_t width) {
  return n >= 0 && n < INT32_MAX && vocab >= 1 && vocab < INT32_MAX && width >= 1;
}

template <typename T, int B>
cudaError_t launch_fwd(TokenSrc ids, int64_t n, const void *table, int64_t table_ld, int32_t width, float scale,
                       void *out, int64_t out_ld, cudaStream_t s) {
  const int acc = width / Pack<T, B>::kN;
  const dim3 grid((unsigned)ceil_div(n, 8), (unsigned)ceil_div(acc, 32 * kFwdUnroll));
  return launch_pdl(k_embed_fwd<T, B>, grid, dim3(32, 8), 0, s, ids, n, reinterpret_cast<const T *>(table), table_ld,
                    width, scale, reinterpret_cast<T *>(out), out_ld);
}

template <typename T, int B>
cudaError_t launch_grad(EmbedGrad g, cudaStream_t s) {
  const int acc = g.width / Pack<T, B>::kN;
  g.n_seg = (int)ceil_div(acc, kSegElems);
  g.sum_blocks = ceil_div(g.n_chunks * g.n_seg, kGradWarps);
  const int64_t rows = g.accumulate ? 0 : (int64_t)g.vocab - g.cleared;
  g.zero_rows = (int)(rows / 4096 < 1 ? 1 : rows / 4096 > kZeroMost ? kZeroMost : rows / 4096);
  const int64_t blocks = g.sum_blocks + ceil_div(rows, (int64_t)kGradWarps * g.zero_rows);
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  if (blocks == 0) return cudaSuccess;
  cudaError_t e = g.accumulate
                      ? launch_pdl(k_embed_sum<T, B, true>, (unsigned)blocks, kGradWarps * 32, 0, s, (const EmbedGrad)g)
                      : launch_pdl(k_embed_sum<T, B, false>, (unsigned)blocks, kGradWarps * 32, 0, s, (const EmbedGrad)g);
  if (e != cudaSuccess || g.n_chunks < 2) return e;
  return launch_pdl(k_embed_join<T, B>, (unsigned)g.sum_blocks, kGradWarps * 32, 0, s, (const EmbedGrad)g);
}

}  // namespace
}  // namespace snack

using namespace snack;

extern "C" {

snack_status snack_embed_fwd(const void *ids, snack_index ids_t, int64_t n, const void *table, int64_t table_ld,
                             int64_t vocab, int32_t width, snack_dtype t, float scale, void *out, int64_t out_ld,
                             snack_stream_t stream) {
  if (!lm_dtype_ok(t) || !lm_index_ok(ids_t) || !embed_sizes_ok(n, vocab, width)) return SNACK_ERR_INVALID_ARG;
  if (table_ld < width || out_ld < width) return SNACK_ERR_INVALID_ARG;
  if (n == 0) return SNACK_OK;
  const size_t es = dtype_size(t);
  if (!ids || !table || !out || !ptr_aligned(ids, index_size(ids_t)) || !ptr_aligned(table, es) || !ptr_aligned(out, es))
    return SNACK_ERR_INVALID_ARG;
  if (spans_overlap(out, span_bytes(n, width, out_ld, es), table, span_bytes(vocab, width, table_ld, es)) ||
      spans_overlap(out, span_bytes(n, width, out_ld, es), ids, (size_t)n * index_size(ids_t)))
    return SNACK_ERR_INVALID_ARG;
  const TokenSrc src{ids, ids_t == SNACK_I64, (uint32_t)vocab};
  const int b = access_bytes((uintptr_t)table | (uintptr_t)out | (uintptr_t)(table_ld * es) | (uintptr_t)(out_ld * es) |
                             (uintptr_t)((size_t)width * es));
  if (ceil_div((int64_t)width * (int64_t)es, (int64_t)b * 32 * kFwdUnroll) > 65535) return SNACK_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
#define SNACK_FWD(T, B) e = launch_fwd<T, B>(src, n, table, table_ld, width, scale, out, out_ld, s)
  if (t == SNACK_F32) {
    if (b == 16)
      SNACK_FWD(float, 16);
    else if (b == 8)
      SNACK_FWD(float, 8);
    else
      SNACK_FWD(float, 4);
  } else {
    if (b == 16)
      SNACK_FWD(bf16, 16);
    else if (b == 8)
      SNACK_FWD(bf16, 8);
    else if (b == 4)
      SNACK_FWD(bf16, 4);
    else
      SNACK_FWD(bf16, 2);
  }
#undef SNACK_FWD
  return e == cudaSuccess ? SNACK_OK : SNACK_ERR_CUDA;
}

snack_status snack_embed_grad_workspace_size(int64_t n, int64_t vocab, int32_t width, size_t *bytes) {
  if (!bytes || !embed_sizes_ok(n, vocab, width)) return SNACK_ERR_INVALID_ARG;
  *bytes = grad_ws(n, width).total;
  return SNACK_OK;
}

snack_status snack_embed_grad(const void *ids, snack_index ids_t, int64_t n, const void *dout, int64_t dout_ld,
                              int64_t vocab, int32_t width, snack_dtype t, float scale, int accumulate, void *dtable,
                              int64_t dtable_ld, void *ws, size_t ws_bytes, snack_stream_t stream) {
  if (!lm_dtype_ok(t) || !lm_index_ok(ids_t) || !embed_sizes_ok(n, vocab, width)) return SNACK_ERR_INVALID_ARG;
  if (dout_ld < width || dtable_ld < width || !dtable) return SNACK_ERR_INVALID_ARG;
  const size_t es = dtype_size(t);
  if (!ptr_aligned(dtable, es)) return SNACK_ERR_INVALID_ARG;
  const GradWs W = grad_ws(n, width);
  if (n > 0) {
    if (!ids || !dout || !ws || !ptr_aligned(ids, index_size(ids_t)) || !ptr_aligned(dout, es) || !ptr_aligned(ws, kAlign))
      return SNACK_ERR_INVALID_ARG;
    const size_t nd = span_bytes(vocab, width, dtable_ld, es);
    if (spans_overlap(dtable, nd, dout, span_bytes(n, width, dout_ld, es)) ||
        spans_overlap(dtable, nd, ids, (size_t)n * index_size(ids_t)) || spans_overlap(dtable, nd, ws, ws_bytes))
      return SNACK_ERR_INVALID_ARG;
    if (ws_bytes < W.total) return SNACK_ERR_WORKSPACE;
    if (spans_overlap(ws, W.total, dout, span_bytes(n, width, dout_ld, es)) ||
        spans_overlap(ws, W.total, ids, (size_t)n * index_size(ids_t)))
      return SNACK_ERR_INVALID_ARG;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t *w = reinterpret_cast<uint8_t *>(ws);
  EmbedGrad g = {};
  g.n = n;
  g.dout = dout;
  g.dout_ld = dout_ld;
  g.dtable = dtable;
  g.table_ld = dtable_ld;
  g.vocab = (uint32_t)vocab;
  g.width = width;
  g.scale = scale;
  g.accumulate = accumulate != 0;
  g.chunk = W.chunk;
  g.n_chunks = W.n_chunks;
  g.part_ld = W.part_ld;
  ZeroRows z = {reinterpret_cast<uint8_t *>(dtable), (int64_t)width * (int64_t)es, dtable_ld * (int64_t)es, vocab, 0};
  z.wide = access_bytes((uintptr_t)dtable | (uintptr_t)z.ld_bytes | (uintptr_t)z.row_bytes) == 16;
  g.zero = z;
  cudaError_t e = cudaSuccess;
  if (n > 0) {
    uint32_t *keys = reinterpret_cast<uint32_t *>(w + W.keys), *pos = reinterpret_cast<uint32_t *>(w + W.pos);
    g.keys = keys;
    g.pos = pos;
    g.part = reinterpret_cast<float *>(w + W.part);
    const TokenSrc src{ids, ids_t == SNACK_I64, (uint32_t)vocab};
    const int bits = key_bits((uint32_t)vocab);
    try {
      if (n <= kRankMax) {
        e = launch_pdl(k_rank, (unsigned)ceil_div(n, kRankRows), kRankThreads, 0, s, src, (int)n, keys, pos);
      } else if (n <= kSortMost) {
        const int passes = (bits + 8) / 9;
        int tile_bits = 10;
        while (((int64_t)kSortBlocks << tile_bits) < n) ++tile_bits;
        // the rows that the rest of the GPU clears in the sort's time, at 5 TB/s (none: 235 us for 32768 tokens
        // of 4096 over 131072 rows, and 121 us for 65536 of 1024; so many: 226 and 103 us)
        z.rows = g.accumulate ? 0 : (int64_t)(5e6 * (5.0 + 3.4e-4 * (double)n)) / z.row_bytes;
        if (z.rows > vocab) z.rows = vocab;
        g.cleared = z.rows;
        const int sms = current_sms(), clusters = z.rows > 0 && sms >= 2 * kSortBlocks ? sms / kSortBlocks : 1;
        if (clusters == 1) g.cleared = 0;
        e = raise_smem_limit(k_sort, kSortSmem);
        if (e == cudaSuccess)
          e = launch_pdl(k_sort, (unsigned)(clusters * kSortBlocks), kSortThreads, kSortSmem, s, src, (int)n, tile_bits, passes,
                         (bits + passes - 1) / passes, keys, pos, z);
      } else {
        e = radix_sort_custom<uint32_t>(src, ArrayDst<uint32_t>{keys, pos}, n, bits,
                                        reinterpret_cast<uint32_t *>(w + W.k0), reinterpret_cast<uint32_t *>(w + W.v0),
                                        reinterpret_cast<uint32_t *>(w + W.k1), reinterpret_cast<uint32_t *>(w + W.v1),
                                        w + W.temp, s);
      }
    } catch (...) {  // the shared-memory table could not grow
      return SNACK_ERR_CUDA;
    }
    if (e != cudaSuccess) return SNACK_ERR_CUDA;
  }
  const int b = access_bytes((uintptr_t)dtable | (n > 0 ? (uintptr_t)dout : 0) | (uintptr_t)(dtable_ld * es) |
                             (uintptr_t)(dout_ld * es) | (uintptr_t)((size_t)width * es));
  if (t == SNACK_F32)
    e = b == 16 ? launch_grad<float, 16>(g, s) : b == 8 ? launch_grad<float, 8>(g, s) : launch_grad<float, 4>(g, s);
  else
    e = b == 16  ? launch_grad<bf16, 16>(g, s)
        : b == 8 ? launch_grad<bf16, 8>(g, s)
        : b == 4 ? launch_grad<bf16, 4>(g, s)
                 : launch_grad<bf16, 2>(g, s);
  return e == cudaSuccess ? SNACK_OK : SNACK_ERR_CUDA;
}

}  // extern "C"
