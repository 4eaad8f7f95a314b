// Low-rank adapters of many requests beside a shared projection, and their
// gradients.  Row i belongs to a request with the adapter a = which[i]:
//
//   h_i  = A_a x_i                       [rank], fp32
//   y_i  = base_i + s_a B_a h_i
//   dh_i = s_a B_a^T dy_i
//   dx_i (+)= A_a^T dh_i
//   dA_a = sum_i dh_i x_i^T              over the adapter's rows
//   dB_a = s_a sum_i dy_i h_i^T
//
// All of it is bound by memory for the ranks that adapters have: x, base and y
// (dy, dx) go over the bus once each, an adapter's matrices once per tile, out of
// L2.  One block first files the rows by adapter, stably, into tiles of rows of one
// adapter (k_adapt_group).  Three kernels do the products:
//   down   h, dh: a tile against one adapter's matrix, K split over a cluster's
//          blocks, whose sums meet in shared memory;
//   up     y, dx: rank is the K, so a tile's h stays in shared memory for all
//          columns; the product is added to the base and rounded once;
//   outer  dA, dB: sums over an adapter's rows, in their order.
// bf16 goes through tcgen05 in tiles of 128 rows (adapt_tc.cuh).  fp32, in tiles of
// 64, and few rows of either type (down and up in one launch, k_adapt_few) through
// mma.sync, operands as they lie: which columns of a group a lane holds does not
// matter to a sum as long as both operands agree, so every lane reads 16
// consecutive bytes of a row.  fp32 operands are cut into three bf16 parts in
// registers, six part products down to 2^-16 of the leading one.  The tensor core's
// sums round towards zero: 16 of K at a time here, runs of them by tcgen05, are added
// in fp32.  h and dh are fp32 in memory and go into products as two bf16 parts (bf16
// operands: 2^-17 of an entry, far below the output's rounding) or three.  Every sum
// has one order: results repeat bit for bit.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "internal.hpp"
#include "lm.hpp"

namespace snack {
namespace {

constexpr int kTile = 64;         // rows of a tile
constexpr int kMostRank = 256;
constexpr int kMostAdapters = 32768;
constexpr int kMostCluster = 8;

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_blocks() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}
// a float of another block's shared memory, at the place of `p` in this one's
__device__ __forceinline__ float ld_cluster(const float *p, uint32_t block) {
  uint32_t at;
  float v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(block));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

// ------------------------------------------------------------ rows by adapter

// A tile: up to kTile rows of one adapter, at order[first ..]; the rows without
// an adapter are the last group's.
struct Tile {
  int32_t adapter, first, count, pad;
};

constexpr int kGroupThreads = 1024;
constexpr int kGroupKeep = 8;                    // keys a lane keeps between the two passes
constexpr int kGroupBytes = 208 * 1024;          // of counts in shared memory

int group_warps(int groups, int n) {
  const int w = std::min(kGroupBytes / 4 / groups, (n + 31) / 32);
  return w < 1 ? 1 : w > kGroupThreads / 32 ? kGroupThreads / 32 : w;
}

// Each warp counts a stretch of the rows by adapter; the counts, added up over
// adapters and warps, say where its rows go.  8192 rows, 16 adapters: 6 us, a chain of
// latencies on one SM.
__global__ void __launch_bounds__(kGroupThreads, 1)
    k_adapt_group(TokenSrc which, int n, int warps, int32_t *__restrict__ order, int32_t *__restrict__ start,
                  Tile *__restrict__ tiles, int tile_cap, int tile_rows) {
  pdl_wait();
  extern __shared__ __align__(16) int32_t hist[];  // [warps][groups]
  __shared__ int2 warp_sum[32];
  const int groups = (int)which.vocab + 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rounds = (n + 32 * warps - 1) / (32 * warps);
  const int64_t first = (int64_t)warp * rounds * 32;
  const unsigned below = (1u << lane) - 1u;
  for (int i = threadIdx.x; i < warps * groups; i += kGroupThreads) hist[i] = 0;
  __syncthreads();
  uint32_t kept[kGroupKeep];
  unsigned peers[kGroupKeep];
  auto pass = [&](bool place) {
    if (warp >= warps) return;
    int32_t *mine = hist + (int64_t)warp * groups;
    for (int r0 = 0; r0 < rounds; r0 += kGroupKeep) {
      if (!place || rounds > kGroupKeep) {
#pragma unroll
        for (int u = 0; u < kGroupKeep; ++u) {
          const int64_t i = first + (int64_t)(r0 + u) * 32 + lane;
          kept[u] = r0 + u < rounds && i < n ? which.key(i) : 0xFFFFFFFFu;
        }
#pragma unroll
        for (int u = 0; u < kGroupKeep; ++u)
          if (r0 + u < rounds) peers[u] = __match_any_sync(0xffffffffu, kept[u]);
      }
#pragma unroll
      for (int u = 0; u < kGroupKeep; ++u) {
        if (r0 + u >= rounds) break;
        const bool here = kept[u] != 0xFFFFFFFFu;
        const int at = here ? mine[kept[u]] : 0;
        __syncwarp();
        if (here && (peers[u] & below) == 0) mine[kept[u]] = at + __popc(peers[u]);
        if (here && place) order[at + __popc(peers[u] & below)] = (int32_t)(first + (int64_t)(r0 + u) * 32 + lane);
        __syncwarp();
      }
    }
  };
  pass(false);
  __syncthreads();
  int2 carry = make_int2(0, 0);  // rows and tiles of the groups before
  for (int g0 = 0; g0 < groups; g0 += kGroupThreads) {
    const int g = g0 + threadIdx.x;
    int count = 0;
    if (g < groups)
      for (int w0 = 0; w0 < warps; w0 += 8) {  // eight reads in flight
        int c[8];
#pragma unroll
        for (int w = 0; w < 8; ++w) c[w] = w0 + w < warps ? hist[(w0 + w) * groups + g] : 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          if (w0 + w < warps) hist[(w0 + w) * groups + g] = count;
          count += c[w];
        }
      }
    const int own = (count + tile_rows - 1) / tile_rows;
    int2 inc = make_int2(count, own);
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int a = __shfl_up_sync(0xffffffffu, inc.x, d), b = __shfl_up_sync(0xffffffffu, inc.y, d);
      if (lane >= d) {
        inc.x += a;
        inc.y += b;
      }
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int2 sums = warp_sum[lane], before = carry;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int a = __shfl_up_sync(0xffffffffu, sums.x, d), b = __shfl_up_sync(0xffffffffu, sums.y, d);
      if (lane >= d) {
        sums.x += a;
        sums.y += b;
      }
    }
    if (warp) {
      before.x += __shfl_sync(0xffffffffu, sums.x, warp - 1);
      before.y += __shfl_sync(0xffffffffu, sums.y, warp - 1);
    }
    carry.x += __shfl_sync(0xffffffffu, sums.x, 31);
    carry.y += __shfl_sync(0xffffffffu, sums.y, 31);
    const int from = before.x + inc.x - count, tile = before.y + inc.y - own;
    if (g < groups) {
      start[g] = from;
      for (int w0 = 0; w0 < warps; w0 += 8) {
        int c[8];
#pragma unroll
        for (int w = 0; w < 8; ++w) c[w] = w0 + w < warps ? hist[(w0 + w) * groups + g] : 0;
#pragma unroll
        for (int w = 0; w < 8; ++w)
          if (w0 + w < warps) hist[(w0 + w) * groups + g] = c[w] + from;
      }
      for (int t = 0; t < own; ++t)
        tiles[tile + t] = Tile{g, from + t * tile_rows, min(tile_rows, count - t * tile_rows), 0};
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    start[groups] = n;
    start[groups + 1] = carry.y;  // tiles
  }
  for (int t = carry.y + threadIdx.x; t < tile_cap; t += kGroupThreads) tiles[t] = Tile{-1, 0, 0, 0};
  pass(true);
}

// Some rows are filed by every block of the first kernel for itself, which saves a launch; one block writes down what the
// others need (1023 rows of 768, rank 8, fp32, with gradients, from cold caches: seven launches 54 us, five 49; 2048 rows
// of 6208 to 1024, rank 16, bf16: 80 and 77).
constexpr int kFileRows = 2048, kFileAdapters = 255;
struct FileArgs {
  TokenSrc which;  // ids null: the rows are filed already
  int32_t n, tile_rows, tile_cap;
  int32_t *order, *start;
  Tile *tiles;
};

// Tile `b` of the rows, its rows in `rows`; scratch: kThreads / 32 x (adapters + 1) words.  All of a block.
template <int kThreads>
__device__ __forceinline__ Tile file_tile(const FileArgs &f, int b, bool writer, int32_t *scratch, int32_t *rows) {
  constexpr int kWarps = kThreads / 32, kRounds = kFileRows / kThreads;
  static_assert(kFileAdapters < kThreads, "a group per thread");
  __shared__ int2 warp_sum[kWarps];
  __shared__ Tile found;
  const int groups = (int)f.which.vocab + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rounds = (f.n + kThreads - 1) / kThreads, first = warp * rounds * 32 + lane;
  const unsigned below = (1u << lane) - 1u;
  uint32_t key[kRounds];
  int place[kRounds];
#pragma unroll
  for (int u = 0; u < kRounds; ++u) key[u] = u < rounds && first + 32 * u < f.n ? f.which.key(first + 32 * u) : 0xFFFFFFFFu;
  for (int i = threadIdx.x; i < kWarps * groups; i += kThreads) scratch[i] = 0;
  if (threadIdx.x == 0) found = Tile{-1, 0, 0, 0};
  __syncthreads();
  int32_t *mine = scratch + warp * groups;
#pragma unroll
  for (int u = 0; u < kRounds; ++u) {
    if (u >= rounds) break;
    const unsigned peers = __match_any_sync(0xffffffffu, key[u]);
    const bool here = key[u] != 0xFFFFFFFFu;
    const int at = here ? mine[key[u]] : 0;
    __syncwarp();
    if (here && (peers & below) == 0) mine[key[u]] = at + __popc(peers);
    place[u] = at + __popc(peers & below);
    __syncwarp();
  }
  __syncthreads();
  const int g = threadIdx.x;
  int before_warp[kWarps], count = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before_warp[w] = count;
    count += g < groups ? scratch[w * groups + g] : 0;
  }
  const int own = (count + f.tile_rows - 1) / f.tile_rows;
  int2 inc = make_int2(count, own);
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int r = __shfl_up_sync(0xffffffffu, inc.x, d), t = __shfl_up_sync(0xffffffffu, inc.y, d);
    if (lane >= d) {
      inc.x += r;
      inc.y += t;
    }
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int from = inc.x - count, tile = inc.y - own, tiles = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) {
      from += warp_sum[w].x;
      tile += warp_sum[w].y;
    }
    tiles += warp_sum[w].y;
  }
  if (g < groups) {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) scratch[w * groups + g] = from + before_warp[w];
    if (b >= tile && b < tile + own) found = Tile{g, from + (b - tile) * f.tile_rows, min(f.tile_rows, count - (b - tile) * f.tile_rows), 0};
    if (writer) {
      f.start[g] = from;
      for (int t = 0; t < own; ++t) f.tiles[tile + t] = Tile{g, from + t * f.tile_rows, min(f.tile_rows, count - t * f.tile_rows), 0};
    }
  }
  if (writer) {
    if (threadIdx.x == 0) {
      f.start[groups] = f.n;
      f.start[groups + 1] = tiles;
    }
    for (int t = tiles + threadIdx.x; t < f.tile_cap; t += kThreads) f.tiles[t] = Tile{-1, 0, 0, 0};
  }
  __syncthreads();
  const Tile t = found;
#pragma unroll
  for (int u = 0; u < kRounds; ++u) {
    if (key[u] == 0xFFFFFFFFu) continue;
    const int at = mine[key[u]] + place[u], d = at - t.first;
    if (d >= 0 && d < t.count) rows[d] = first + 32 * u;
    if (writer) f.order[at] = first + 32 * u;
  }
  __syncthreads();
  return Tile{t.adapter, 0, t.count, 0};
}

// ------------------------------------------------------------ operands

// What of a group of K a lane holds: 16 bytes of a row that runs along K, four
// consecutive elements for each step of 16.
template <typename T>
struct Op;
template <>
struct Op<bf16> {
  static constexpr int kSteps = 2, kParts = 1, kLane = 8, kGroup = 32;  // elements per lane, K per group
  static constexpr int kOwnParts = 2;                                   // of h and dh
};
template <>
struct Op<float> {
  static constexpr int kSteps = 1, kParts = 3, kLane = 4, kGroup = 16;
  static constexpr int kOwnParts = 3;
};

// V consecutive elements as they are; zeros from `left` on
template <typename T, int V>
__device__ __forceinline__ Pack<T, V * (int)sizeof(T)> load_vec(const T *p, int left, bool wide) {
  Pack<T, V * (int)sizeof(T)> r;
  if (wide && left >= V) {
    r.raw = __ldg(reinterpret_cast<const typename Raw<V * (int)sizeof(T)>::type *>(p));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (sizeof(T) == 4)
        r.w[i] = i < left ? __float_as_uint(__ldg(p + i)) : 0u;
      else
        r.h[i] = i < left ? __ldg(reinterpret_cast<const uint16_t *>(p) + i) : (uint16_t)0;
    }
  }
  return r;
}

// The same into shared memory, on its way while the lane works on.  A lane reads what
// it wrote there itself, or what the same lane of its pair's other warp did.  kWide: the
// address is aligned to V elements; bf16 that are not are read at once.
template <int kBytes>
__device__ __forceinline__ void copy_async(void *to, const void *from, int bytes) {
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(at), "l"(from), "r"(bytes), "n"(kBytes) : "memory");
}
template <int kBytes>
__device__ __forceinline__ void copy_whole(void *to, const void *from) {
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(kBytes) : "memory");
}
template <typename T, int V, bool kWide>
__device__ __forceinline__ void fetch_vec(void *to, const T *p, int left) {
  constexpr int kBytes = V * (int)sizeof(T);
  if constexpr (kWide) {
    copy_async<kBytes>(to, p, max(0, min(left, V)) * (int)sizeof(T));
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) copy_async<4>(reinterpret_cast<float *>(to) + i, p + (i < left ? i : 0), i < left ? 4 : 0);
  } else {
    Pack<T, kBytes> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.h[i] = i < left ? reinterpret_cast<const uint16_t *>(p)[i] : (uint16_t)0;
    *reinterpret_cast<typename Raw<kBytes>::type *>(to) = r.raw;
  }
}
// of kernels for rows that are not all aligned: these may be
template <typename T, int V, bool kWide>
__device__ __forceinline__ void fetch_some(void *to, const T *p, int left, int wide) {
  if (kWide || wide)
    fetch_vec<T, V, true>(to, p, left);
  else
    fetch_vec<T, V, false>(to, p, left);
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void fetch_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// two warps that share what they read
__device__ __forceinline__ void pair_sync(int pair) { asm volatile("bar.sync %0, 64;" ::"r"(1 + pair) : "memory"); }

// The upper halves of two words, as a pair of bf16.
__device__ __forceinline__ uint32_t upper_halves(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}
__device__ __forceinline__ float without_top(float v) { return v - __uint_as_float(__float_as_uint(v) & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A pair of values as words of two bf16: three parts cut off, 8 significant bits
// each, or two rounded.
template <int kParts>
__device__ __forceinline__ void cut_pair(float a, float b, uint32_t (&w)[kParts]) {
  if constexpr (kParts == 2) {
    w[0] = pack_pair(a, b);
    w[1] = pack_pair(a - bf16_lo(w[0]), b - bf16_hi(w[0]));
  } else {
    static_assert(kParts == 3, "two or three parts");
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      if (p) {
        a = without_top(a);
        b = without_top(b);
      }
      w[p] = upper_halves(a, b);
    }
  }
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// acc[i] += a[i] b[i] over 16 of K for kN independent sums: rows g (lo) and g + 8 (hi)
// of a, in parts; the small products first, summed apart from what is there, which the
// tensor core would cut off at the same side each time (nearly 2^20 terms of one sign
// were off by 3e-4).  One part after the other for all sums: none waits for its own.
template <int kN, int kA, int kB, typename FA, typename FB, typename FAcc>
__device__ __forceinline__ void mma_all(FAcc acc, FA a, FB b) {
  typedef const uint32_t(&Rows)[2][2][kA];  // [row half][pair of K][part]
  typedef const uint32_t(&Cols)[2][kB];     // [pair of K][part]
  static_assert(kB == 1 || kA == kB, "parts");
  float d[kN][4];
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) d[n][e] = 0.f;
#pragma unroll
  for (int sum = kA - 1; sum >= 0; --sum)
#pragma unroll
    for (int i = sum; i >= 0; --i) {
      if (sum - i >= kB) break;
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        Rows w = a(n);
        Cols v = b(n);
        mma(d[n], w[0][0][i], w[1][0][i], w[0][1][i], w[1][1][i], v[0][sum - i], v[1][sum - i]);
      }
    }
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc(n)[e] += d[n][e];
}

// a lane's words of four consecutive elements of a row along K: [pair][part]
template <typename T, int B>
__device__ __forceinline__ void along(const Pack<T, B> &v, int s, uint32_t (&w)[2][Op<T>::kParts]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (sizeof(T) == 2)
      w[h][0] = v.w[2 * s + h];
    else
      cut_pair<3>(v.get(4 * s + 2 * h), v.get(4 * s + 2 * h + 1), w[h]);
  }
}
// the pair of elements j of two rows that follow one another along K; bf16 matrices that lie so go through tcgen05
template <int B>
__device__ __forceinline__ void across(const Pack<float, B> &a, const Pack<float, B> &b, int j, uint32_t (&w)[3]) {
  cut_pair<3>(a.get(j), b.get(j), w);
}

// ------------------------------------------------------------ h and dh

struct DownArgs {
  const void *x;   // [n][k] rows of the tiles' tokens: x, or dy
  int64_t x_ld;
  const void *m;   // the adapters' matrices: [rank][k] each (along K), or [k][rank]
  int32_t k, rank;
  const int32_t *order;
  const Tile *tiles;
  int32_t adapters;
  const float *scales;  // null: 1
  float *h;             // [n][rank]
  int x_wide, m_wide;   // the rows, the matrices are aligned to whole accesses
};

constexpr int kDownParts = 8;   // shares of K in a block: a warp each, or a pair that shares the rows' part and has half of the ranks each
constexpr int kDownStages = 4;  // groups of K that are on their way or in hand
__host__ __device__ constexpr int down_smem(int cols) {
  const int ring = kDownParts * kDownStages * (kTile / 8 + cols / 8) * 512, sums = 4 * kTile * cols * 4;
  return ring > sums ? ring : sums;
}

// The sums of the block's shares of K, and of the cluster's blocks; NT: a warp's ranks / 8.
template <typename T, int MT, int NT, int kHalves, bool kAlong, bool kWide>
__device__ __forceinline__ void down_tile(const DownArgs &a, const Tile &tile, int slice, float *smem) {
  typedef Op<T> O;
  constexpr int kRows = 16 * MT, kCols = 8 * NT * kHalves, kStages = kDownStages, kSlots = kTile / 8 + NT * kHalves;
  constexpr int kThreads = kDownParts * kHalves * 32;
  typedef Pack<T, NT * (int)sizeof(T)> Cross;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = warp / kHalves, half = warp % kHalves;
  const int g = lane >> 2, q = lane & 3;
  const int r0 = slice * kCols + half * 8 * NT;
  const uint32_t rank = cluster_rank(), blocks = cluster_blocks();
  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.f;
  // the rows that this warp reads of the tile (8 i + g for its share of i); past the end the last one again, and not kept
  constexpr int kRead = 2 * MT / kHalves;
  const T *row[kRead];
#pragma unroll
  for (int i = 0; i < kRead; ++i)
    row[i] = reinterpret_cast<const T *>(a.x) +
             (int64_t)a.order[tile.first + min(8 * (half * kRead + i) + g, tile.count - 1)] * a.x_ld + O::kLane * q;
  const T *mat = reinterpret_cast<const T *>(a.m) + (int64_t)tile.adapter * a.rank * a.k;
  // the part's ring: kStages x (of the rows 16 bytes of every 8th per lane; then each warp's of the matrix NT of them, or
  // the same bytes in smaller pieces)
  uint4 *ring = reinterpret_cast<uint4 *>(smem) + part * kStages * kSlots * 32;
  // two neighbouring groups, a line of the rows, then the two so many further on
  const int step = (int)blocks * kDownParts * 2 * O::kGroup;
  const int k_first = (int)(rank * kDownParts + part) * 2 * O::kGroup;
  int next = k_first, odd = 0;
  auto fetch = [&](int stage) {
    if (next < a.k) {
      uint4 *to = ring + stage * kSlots * 32 + lane;
      const int left = a.k - next - O::kLane * q;
#pragma unroll
      for (int i = 0; i < kRead; ++i) fetch_some<T, O::kLane, kWide>(to + (half * kRead + i) * 32, row[i] + next, left, a.x_wide);
      to += (kTile / 8 + half * NT) * 32;
      if constexpr (kAlong) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int r = r0 + 8 * j + g;
          fetch_some<T, O::kLane, kWide>(to + j * 32, mat + (int64_t)min(r, a.rank - 1) * a.k + next + O::kLane * q, r < a.rank ? left : 0, a.m_wide);
        }
      } else {  // rows next + kLane q + i: ranks NT g .. NT g + NT - 1
        typename Cross::R *piece = reinterpret_cast<typename Cross::R *>(to - lane) + lane;
        const int ranks = a.rank - r0 - NT * g;
#pragma unroll
        for (int i = 0; i < O::kLane; ++i)
          fetch_some<T, NT, kWide>(piece + i * 32, mat + (int64_t)min(next + O::kLane * q + i, a.k - 1) * a.rank + (ranks > 0 ? r0 + NT * g : 0),
                                   i < left ? ranks : 0, a.m_wide);
      }
    }
    fetch_commit();
    next += odd ? step - O::kGroup : O::kGroup;
    odd ^= 1;
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(s);
  int stage = 0, odd_now = 0;
  for (int k0 = k_first; k0 < a.k; k0 += odd_now ? step - O::kGroup : O::kGroup, odd_now ^= 1) {
    fetch_wait<kStages - 2>();
    if (kHalves > 1) pair_sync(part);  // the other warp's part is there, and it has done with the stage that is filled next
    fetch(stage == 0 ? kStages - 1 : stage - 1);
    const uint4 *from = ring + stage * kSlots * 32 + lane;
    uint32_t xa[O::kSteps][MT][2][2][O::kParts];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {
      Pack<T, 16> v;
      v.raw = from[i * 32];
#pragma unroll
      for (int s = 0; s < O::kSteps; ++s) along<T>(v, s, xa[s][i >> 1][i & 1]);
    }
    from += (kTile / 8 + half * NT) * 32;
    const typename Cross::R *piece = reinterpret_cast<const typename Cross::R *>(from - lane) + lane;
    uint32_t bw[O::kSteps][NT][2][O::kParts];
    if constexpr (kAlong) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        Pack<T, 16> v;
        v.raw = from[j * 32];
#pragma unroll
        for (int s = 0; s < O::kSteps; ++s) along<T>(v, s, bw[s][j]);
      }
    }
#pragma unroll
    for (int s = 0; s < O::kSteps; ++s) {
      if constexpr (!kAlong) {
        Cross v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i].raw = piece[(4 * s + i) * 32];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) across(v[2 * h], v[2 * h + 1], j, bw[s][j][h]);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
        mma_all<MT, O::kParts, O::kParts>([&](int m) -> float(&)[4] { return acc[m][j]; },
                                          [&](int m) -> const uint32_t(&)[2][2][O::kParts] { return xa[s][m]; },
                                          [&](int) -> const uint32_t(&)[2][O::kParts] { return bw[s][j]; });
    }
    if (++stage == kStages) stage = 0;
  }
  fetch_wait<0>();
  __syncthreads();  // the ring becomes the sums
  // the parts' sums: the upper half's to the lower half, then those of the four
  float *own = smem + (part & 3) * (kRows * kCols) + half * 8 * NT;
  auto each = [&](auto f) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int n = 2 * q + (e & 1), c = kAlong ? 8 * j + n : NT * n + j;
          f(own[(16 * m + 8 * (e >> 1) + g) * kCols + c], acc[m][j][e]);
        }
  };
  if (part >= 4) each([](float &s, float &v) { s = v; });
  __syncthreads();
  if (part < 4) each([](float &s, float &v) { s += v; });
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * kCols; i += kThreads)
    smem[i] = (smem[i] + smem[kRows * kCols + i]) + (smem[2 * kRows * kCols + i] + smem[3 * kRows * kCols + i]);
  if (blocks > 1)
    cluster_sync();
  else
    __syncthreads();
  const float scale = a.scales ? a.scales[tile.adapter] : 1.f;
  for (int i = (int)rank * kThreads + threadIdx.x; i < tile.count * kCols; i += (int)blocks * kThreads) {
    const int t = i / kCols, r = slice * kCols + i % kCols;
    float s = smem[i];
    if (blocks > 1) {
      s = ld_cluster(smem + i, 0);
      for (uint32_t b = 1; b < blocks; ++b) s += ld_cluster(smem + i, b);
    }
    if (r < a.rank) a.h[(int64_t)a.order[tile.first + t] * a.rank + r] = s * scale;
  }
  if (blocks > 1) cluster_sync();  // no block's memory is read any more
}

template <int NT, int kHalves, bool kAlong, bool kWide>
__global__ void __launch_bounds__(kDownParts * kHalves * 32, 1) k_adapt_down(const DownArgs args, const FileArgs f) {
  pdl_wait();
  extern __shared__ __align__(16) float down_ring[];
  __shared__ int32_t rows[kTile];
  DownArgs a = args;
  const int b = (int)(blockIdx.x / cluster_blocks());
  Tile tile;
  if (f.which.ids) {
    tile = file_tile<kDownParts * kHalves * 32>(f, b, blockIdx.x == 0 && blockIdx.y == 0, reinterpret_cast<int32_t *>(down_ring), rows);
    a.order = rows;
  } else {
    tile = a.tiles[b];
  }
  if (tile.adapter < 0 || tile.adapter >= a.adapters) return;  // the whole cluster's
  if (tile.count <= 16)
    down_tile<float, 1, NT, kHalves, kAlong, kWide>(a, tile, blockIdx.y, down_ring);
  else
    down_tile<float, 4, NT, kHalves, kAlong, kWide>(a, tile, blockIdx.y, down_ring);
}

// ------------------------------------------------------------ y and dx

struct UpArgs {
  const float *h;  // [n][rank]
  const void *m;   // the adapters' matrices: [n_cols][rank] each (along K), or [rank][n_cols]
  int32_t cols, rank;
  const int32_t *order;
  const Tile *tiles;
  int32_t adapters;
  const float *scales;   // null: 1
  const void *base;      // null: 0
  int64_t base_ld;
  void *out;
  int64_t out_ld;
  int groups;            // of 32 columns, per warp
  const int32_t *n_tiles;
  int h_wide, m_wide;    // h, the matrices are aligned to four elements
};

constexpr int kUpWarps = 8;     // pairs of them: half of the tile's rows each
constexpr int kUpCols = 32;  // columns of a pair at a time

// Of a row of h in shared memory, in elements: rows start 16 bytes apart modulo 128 as
// bf16 (its two parts), 64 as fp32 (which is cut into parts as it is read); the
// highest ranks of fp32 have no room for that.
template <typename T>
__host__ __device__ constexpr int up_ld(int rank) {
  return sizeof(T) == 2 ? (rank + 63) / 64 * 64 + 8 : rank > 192 ? kMostRank + 8 : (rank + 63) / 64 * 64 + 16;
}
template <typename T>
constexpr size_t up_h_bytes(int rank) { return (size_t)kTile * up_ld<T>(rank) * 4; }
// shared memory of a pair's lane: its 16-byte pieces of the base, and its pieces of the matrix (8 bytes of bf16, 16 of fp32)
template <typename T>
__host__ __device__ constexpr int up_base_bytes() { return kTile / 8 * 8 * (int)sizeof(T); }
template <typename T, int kSteps>
__host__ __device__ constexpr int up_stage_bytes() { return up_base_bytes<T>() + kSteps * 4 * 4 * (int)sizeof(T); }
template <typename T>
__host__ __device__ constexpr int up_stages() { return sizeof(T) == 2 ? 3 : 2; }

static_assert(kUpWarps * up_stages<bf16>() * up_stage_bytes<bf16, 2>() * 32 + up_h_bytes<bf16>(kMostRank) <= 232448 &&
                  kUpWarps * up_stages<float>() * up_stage_bytes<float, 1>() * 32 + up_h_bytes<float>(kMostRank) <= 232448 &&
                  kUpWarps * up_stages<float>() * up_stage_bytes<float, 1>() * 32 + up_h_bytes<float>(193) <= 232448 &&
                  kUpWarps * up_stages<float>() * up_stage_bytes<float, 1>() * 32 + up_h_bytes<float>(192) <= 232448,
              "shared memory of one block");

// four values of h, which another block of the cluster may have written
__device__ __forceinline__ Pack<float, 16> load_h(const float *p, int left, bool wide) {
  Pack<float, 16> r;
  if (wide && left >= 4) {
    r.raw = __ldcg(reinterpret_cast<const uint4 *>(p));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = i < left ? __float_as_uint(__ldcg(p + i)) : 0u;
  }
  return r;
}

// where the pieces of a stage have column `col` of a warp's row 8 i + r
template <typename T>
__device__ __forceinline__ int place_of(int i, int r, int col) {
  constexpr int kPer = 16 / (int)sizeof(T);
  return ((i * (8 / kPer) + (col & 7) / kPer) * 32 + 4 * r + (col >> 3)) * 16 + (col & 7) % kPer * (int)sizeof(T);
}

// A pair of warps takes 32 columns of the tile after 32 others; what it reads of the base
// and the matrix is on its way one or two turns before, kSteps of 16 of the rank per turn.
// The sums begin with the base, so the result is rounded as it leaves; h has its
// scale before it is cut into parts.
//
// kWhole: 64 rows, whole groups of columns and steps of the rank: nothing to check.
template <typename T, bool kAlong, int kSteps, bool kWide, bool kWhole>
__device__ __forceinline__ void up_tile(const UpArgs &a, const Tile &tile, int slice, uint8_t *up_ring) {
  constexpr int kHp = Op<T>::kOwnParts, kBp = Op<T>::kParts, MT = kTile / 32, NT = 4, kStages = up_stages<T>();
  typedef Pack<T, 16> P;
  typedef Pack<T, 4 * (int)sizeof(T)> P4;
  constexpr int kPer = P::kN, kVecs = 8 / kPer;  // accesses for a lane's 8 columns
  constexpr int kStage = up_stage_bytes<T, kSteps>() * 32;
  const bool none = !kWhole && tile.adapter >= a.adapters;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, pair = warp >> 1, half = warp & 1;
  const int g = lane >> 2, q = lane & 3;
  const int ld = up_ld<T>(a.rank) / 2, plane = kTile * ld;  // in words
  const int steps = none ? 1 : (a.rank + 15) / 16, turns = (steps + kSteps - 1) / kSteps;
  const int first_row = 32 * half, m_tiles = kWhole ? MT : max(0, min(MT, (tile.count - first_row + 15) / 16));
  uint8_t *ring = up_ring + pair * kStages * kStage;
  uint32_t *hs = reinterpret_cast<uint32_t *>(up_ring + kUpWarps * kStages * kStage);
  const T *mat = reinterpret_cast<const T *>(a.m) + (none ? 0 : (int64_t)tile.adapter * a.rank * a.cols);
  const int col0 = (slice * a.groups * kUpWarps + pair) * kUpCols;
  // this lane's rows, from its 8 columns on
  int32_t token[2 * MT];
  const T *base[2 * MT];
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i) {
    const int t = first_row + 8 * i + g;
    token[i] = kWhole || t < tile.count ? a.order[tile.first + t] : -1;
    base[i] = reinterpret_cast<const T *>(a.base) + (int64_t)max(token[i], 0) * a.base_ld + col0 + 8 * q;
  }
  const int items = (a.cols <= col0 ? 0 : min(a.groups, (a.cols - col0 + kUpWarps * kUpCols - 1) / (kUpWarps * kUpCols))) * turns;
  int next_col = col0, next_turn = 0, next_stage = 0, next_item = 0;
  auto fetch = [&] {
    if (next_item < items) {
      uint8_t *to = ring + next_stage * kStage;
      const int left = a.cols - next_col - 8 * q;
      if (next_turn == 0 && a.base) {
        uint8_t *part = to + half * (2 * MT * kVecs) * 512;
        if constexpr (kWide) {
          uint4 *at = reinterpret_cast<uint4 *>(part) + lane;
#pragma unroll
          for (int i = 0; i < 2 * MT; ++i) {
            if (i >= 2 * m_tiles) break;
            const T *from = base[i] + (next_col - col0);
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
              if constexpr (kWhole)
                copy_whole<16>(at + (i * kVecs + v) * 32, from + v * kPer);
              else
                fetch_vec<T, kPer, true>(at + (i * kVecs + v) * 32, from + v * kPer, left - v * kPer);
            }
          }
        } else {  // a row's 32 columns by the warp, one each
          const int c = next_col + lane;
#pragma unroll
          for (int i = 0; i < 2 * MT; ++i) {
            if (i >= 2 * m_tiles) break;
            T kept[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
              const int row = __shfl_sync(0xffffffffu, token[i], 4 * r);
              const bool in = row >= 0 && c < a.cols;
              const T *from = reinterpret_cast<const T *>(a.base) + (in ? row * a.base_ld + c : 0);
              if constexpr (sizeof(T) == 4)
                copy_async<4>(part + place_of<T>(i, r, lane), from, in ? 4 : 0);
              else
                kept[r] = in ? *from : from_f32<T>(0.f);
            }
            if constexpr (sizeof(T) == 2)
#pragma unroll
              for (int r = 0; r < 8; ++r) *reinterpret_cast<T *>(part + place_of<T>(i, r, lane)) = kept[r];
          }
        }
      }
      if (!none) {
        typename P4::R *at = reinterpret_cast<typename P4::R *>(to + up_base_bytes<T>() * 32) + lane;
        const int r0 = 16 * next_turn * kSteps + 4 * q;
#pragma unroll
        for (int jj = 0; jj < 2; ++jj)  // the other two are the pair's other warp's
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {
            const int j = 2 * half + jj;
            if constexpr (kAlong) {  // lane g has column 8 (g / 2) + 2 j + g % 2: a lane's sums are 8 neighbours
              const int col = next_col + 8 * (g >> 1) + 2 * j + (g & 1), r = r0 + 16 * s;
              if constexpr (kWhole)
                copy_whole<4 * (int)sizeof(T)>(at + (4 * s + j) * 32, mat + (int64_t)col * a.rank + r);
              else
                fetch_some<T, 4, kWide>(at + (4 * s + j) * 32, mat + (int64_t)min(col, a.cols - 1) * a.rank + (r < a.rank ? r : 0),
                                        col < a.cols ? a.rank - r : 0, a.m_wide);
            } else {  // columns 4 g .. 4 g + 3
              const int r = r0 + 16 * s + j, col = next_col + 4 * g;
              if constexpr (kWhole)
                copy_whole<4 * (int)sizeof(T)>(at + (4 * s + j) * 32, mat + (int64_t)r * a.cols + col);
              else
                fetch_some<T, 4, kWide>(at + (4 * s + j) * 32, mat + (int64_t)min(r, a.rank - 1) * a.cols + (col < a.cols ? col : 0),
                                        r < a.rank ? a.cols - col : 0, a.m_wide);
            }
          }
      }
      if (++next_turn == turns) {
        next_turn = 0;
        next_col += kUpWarps * kUpCols;
      }
    }
    fetch_commit();
    ++next_item;
    if (++next_stage == kStages) next_stage = 0;
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch();
  if (!none) {
    const float scale = a.scales ? a.scales[tile.adapter] : 1.f;
    const int quads = steps * 4, rows = (tile.count + 15) / 16 * 16;
    for (int i = threadIdx.x; i < rows * quads; i += kUpWarps * 64) {
      const int t = i / quads, r = (i - t * quads) * 4;
      const bool in = t < tile.count;
      const Pack<float, 16> v = load_h(a.h + (int64_t)(in ? a.order[tile.first + t] : 0) * a.rank + r, in ? a.rank - r : 0, a.h_wide);
      if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4 *>(hs + t * up_ld<T>(a.rank) + r) =
            make_float4(scale * v.get(0), scale * v.get(1), scale * v.get(2), scale * v.get(3));
      } else {  // the pairs of a step of 16: the lanes' first ones, then their second ones, as ldmatrix hands them out
        uint32_t w[2][kHp];
#pragma unroll
        for (int h = 0; h < 2; ++h) cut_pair<kHp>(scale * v.get(2 * h), scale * v.get(2 * h + 1), w[h]);
#pragma unroll
        for (int p = 0; p < kHp; ++p)
#pragma unroll
          for (int h = 0; h < 2; ++h) hs[p * plane + t * ld + (r >> 4) * 8 + 4 * h + ((r >> 2) & 3)] = w[h][p];
      }
    }
  }
  __syncthreads();
  // ldmatrix: lanes 0 to 15 name rows 0 to 15 of their first pairs, lanes 16 to 31 of the second
  const uint32_t h_at = static_cast<uint32_t>(__cvta_generic_to_shared(hs)) + (uint32_t)((first_row + (lane & 15)) * ld * 4 + (lane >> 4) * 16);
  float acc[MT][NT][4];
  // a lane's 8 columns: which sum has column e of row half h
  auto sum_at = [&](int m, int h, int e) -> float & { return kAlong ? acc[m][e >> 1][2 * h + (e & 1)] : acc[m][e & 3][2 * h + (e >> 2)]; };
  int c = col0 + 8 * q, turn = 0, stage = 0;
  for (int item = 0; item < items; ++item) {
    fetch_wait<kStages - 2>();
    pair_sync(pair);  // the other warp's part is there, and it has done with the stage that is filled next
    fetch();
    const uint8_t *from = ring + stage * kStage;
    if (turn == 0) {
      const uint4 *at = reinterpret_cast<const uint4 *>(from) + half * (2 * MT * kVecs) * 32 + lane;
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) {
        if (i >= 2 * m_tiles) break;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
          P old;
          old.raw = a.base ? at[(i * kVecs + v) * 32] : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int e = 0; e < kPer; ++e) sum_at(i >> 1, i & 1, v * kPer + e) = old.get(e);
        }
      }
    }
    if (!none) {
      const typename P4::R *at = reinterpret_cast<const typename P4::R *>(from + up_base_bytes<T>() * 32) + lane;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int k = turn * kSteps + s;
        if (!kWhole && k >= steps) break;
        P4 mv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) mv[j].raw = at[(4 * s + j) * 32];
        uint32_t b[NT][2][kBp];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if constexpr (kAlong) {
            along<T>(mv[j], 0, b[j]);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) across(mv[2 * h], mv[2 * h + 1], j, b[j][h]);
          }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if (m >= m_tiles) break;
          uint32_t w[2][2][kHp];  // rows g and g + 8
          if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float4 v = *reinterpret_cast<const float4 *>(hs + (first_row + 16 * m + 8 * h + g) * up_ld<T>(a.rank) + 16 * k + 4 * q);
              cut_pair<kHp>(v.x, v.y, w[h][0]);
              cut_pair<kHp>(v.z, v.w, w[h][1]);
            }
          } else {
#pragma unroll
            for (int p = 0; p < kHp; ++p)
              asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                           : "=r"(w[0][0][p]), "=r"(w[1][0][p]), "=r"(w[0][1][p]), "=r"(w[1][1][p])
                           : "r"(h_at + (uint32_t)(p * plane + 16 * m * ld + 8 * k) * 4));
          }
          mma_all<NT, kHp, kBp>([&](int j) -> float(&)[4] { return acc[m][j]; },
                                [&](int) -> const uint32_t(&)[2][2][kHp] { return w; },
                                [&](int j) -> const uint32_t(&)[2][kBp] { return b[j]; });
        }
      }
    }
    if (++stage == kStages) stage = 0;
    if (++turn < turns) continue;
    turn = 0;
    const int left = a.cols - c;
    uint8_t *part = const_cast<uint8_t *>(from) + half * (2 * MT * kVecs) * 512;  // !kWide: the stage's, read already
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {
      if (i >= 2 * m_tiles) break;
      if (kWide && !kWhole && (token[i] < 0 || left <= 0)) continue;
      T *out = reinterpret_cast<T *>(a.out) + token[i] * a.out_ld + c;
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        P o;
        if constexpr (sizeof(T) == 2) {
#pragma unroll
          for (int e = 0; e < 4; ++e) o.w[e] = pack_pair(sum_at(i >> 1, i & 1, 2 * e), sum_at(i >> 1, i & 1, 2 * e + 1));
        } else {
#pragma unroll
          for (int e = 0; e < kPer; ++e) o.set(e, sum_at(i >> 1, i & 1, v * kPer + e));
        }
        if constexpr (!kWide) {
          reinterpret_cast<uint4 *>(part)[(i * kVecs + v) * 32 + lane] = o.raw;
        } else if (kWhole || left >= (v + 1) * kPer) {
          *reinterpret_cast<uint4 *>(out + v * kPer) = o.raw;
        } else {
#pragma unroll
          for (int e = 0; e < kPer; ++e)
            if (v * kPer + e < left) {
              if constexpr (sizeof(T) == 4)
                out[v * kPer + e] = o.get(e);
              else
                reinterpret_cast<uint16_t *>(out)[v * kPer + e] = o.h[e];
            }
        }
      }
    }
    if constexpr (!kWide) {  // a row's 32 columns by the warp, one each
      __syncwarp();
      const int own = c - 8 * q + lane;
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) {
        if (i >= 2 * m_tiles) break;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const int row = __shfl_sync(0xffffffffu, token[i], 4 * r);
          if (row >= 0 && own < a.cols)
            reinterpret_cast<T *>(a.out)[row * a.out_ld + own] = *reinterpret_cast<const T *>(part + place_of<T>(i, r, lane));
        }
      }
      __syncwarp();
    }
    c += kUpWarps * kUpCols;
  }
}

template <bool kAlong, bool kWide>
__global__ void __launch_bounds__(kUpWarps * 64, 1) k_adapt_up(const UpArgs a) {
  pdl_wait();
  extern __shared__ __align__(16) uint8_t up_ring[];
  const Tile tile = a.tiles[blockIdx.x];
  if (tile.adapter < 0) return;
  const bool none = tile.adapter >= a.adapters;
  if (none && a.base == a.out) return;
  if constexpr (kWide) {
    if (!none && tile.count == kTile && a.cols % kUpCols == 0 && a.rank % 16 == 0) {
      up_tile<float, kAlong, 1, true, true>(a, tile, blockIdx.y, up_ring);
      return;
    }
  }
  up_tile<float, kAlong, 1, kWide, false>(a, tile, blockIdx.y, up_ring);
}

// ------------------------------------------------------------ few rows

// Of few rows both products in one launch, without the rows' order in memory: a cluster per row, which goes on if its row
// is the first of up to 64 with its adapter; its blocks share K, then the columns.  bf16 of 4096 to 4096, from cold caches:
// one row of rank 16 11 us, 64 of 64 requests 15 (the three launches 22 and 32); 256 rows of two requests, rank 64, 33 (26):
// more rows of a higher rank are for the others.
constexpr int kFewRows = 256;
constexpr int kFewThreads = 512;
static_assert(kFewThreads == kUpWarps * 64 && kFewThreads == kDownParts * 64, "both products' threads");

template <typename T, int NT, int kSteps, bool kWide>
__global__ void __launch_bounds__(kFewThreads, 1) k_adapt_few(const DownArgs down, const UpArgs up, TokenSrc which, int n) {
  pdl_wait();
  extern __shared__ __align__(16) uint8_t few_ring[];
  __shared__ int32_t rows[kTile];
  __shared__ int32_t found[kFewRows / 32];
  const int i = (int)(blockIdx.x / cluster_blocks()), j = threadIdx.x, lane = j & 31, warp = j >> 5;
  const uint32_t own = which.key(i);
  const bool same = j < n && which.key(j) == own;
  if (__syncthreads_count(same && j < i) % kTile != 0) return;  // the whole cluster's
  const bool mine = same && j >= i;
  const unsigned peers = __ballot_sync(0xffffffffu, mine);
  if (lane == 0 && warp < kFewRows / 32) found[warp] = __popc(peers);
  __syncthreads();
  int at = __popc(peers & ((1u << lane) - 1u)), count = 0;
#pragma unroll
  for (int w = 0; w < kFewRows / 32; ++w) {
    if (w < warp) at += found[w];
    count += found[w];
  }
  if (mine && at < kTile) rows[at] = j;
  __syncthreads();
  const Tile tile = {(int32_t)own, 0, min(count, kTile), 0};
  if (tile.adapter < down.adapters) {
    DownArgs a = down;
    a.order = rows;
    for (int slice = 0; slice * 16 * NT < a.rank; ++slice) {
      if (tile.count <= 16)
        down_tile<T, 1, NT, 2, true, kWide>(a, tile, slice, reinterpret_cast<float *>(few_ring));
      else
        down_tile<T, 4, NT, 2, true, kWide>(a, tile, slice, reinterpret_cast<float *>(few_ring));
      __syncthreads();
    }
  } else if (up.base == up.out) {
    return;
  }
  UpArgs a = up;  // h is there: down_tile ends with the cluster's barrier
  a.order = rows;
  up_tile<T, true, kSteps, kWide, false>(a, tile, (int)cluster_rank(), few_ring);
}

// ------------------------------------------------------------ dA and dB

struct OuterArgs {
  const float *v;  // [n][rank]: dh, or h
  const void *x;   // [n][cols]: x, or dy
  int64_t x_ld;
  int32_t rank, cols;
  const int32_t *order, *start;
  const float *scales;  // null: 1
  void *out;            // [rank][cols] of each adapter, or [cols][rank]
  int turned;           // the latter
  int v_wide;
};
// dA and dB, one beside the other: the first `slices` of the grid's columns are dA's
struct OuterPair {
  OuterArgs a[2];
  int32_t slices;
};

constexpr int kOuterWarps = 8;
constexpr int kOuterRows = 32;    // rows of v in shared memory at a time: two steps of 16
constexpr int kOuterStages = 4;   // of x, on its way
__host__ __device__ constexpr int outer_cols(int lane) { return kOuterWarps * 8 * lane; }  // of a block
template <int MT>
constexpr int outer_v_words() { return Op<float>::kOwnParts * 2 * MT * 128; }  // a fragment: 4 words of 32 lanes
template <int MT>
constexpr size_t outer_smem() {
  const size_t ring = (size_t)kOuterWarps * kOuterStages * 8 * 512 + 2 * (size_t)outer_v_words<MT>() * 4;
  const size_t sums = (size_t)16 * MT * (outer_cols(Op<float>::kLane) + 1) * 4;
  return ring > sums ? ring : sums;
}

// The cluster's sums [kRank][kCols] to the output, this block's share of them.
template <int kRank, int kCols, int kThreads>
__device__ __forceinline__ void outer_write(const OuterArgs &a, const float *sums, int pitch, uint32_t block, uint32_t blocks, int adapter,
                                            int r0, int b0, bool empty) {
  const float scale = a.scales ? a.scales[adapter] : 1.f;
  float *out = reinterpret_cast<float *>(a.out) + (int64_t)adapter * a.rank * a.cols;
  for (int i = (int)block * kThreads + threadIdx.x; i < kCols * kRank; i += (int)blocks * kThreads) {
    int r, c;  // of the block's
    if (a.turned) {
      r = i % kRank;
      c = i / kRank;
    } else {
      c = i % kCols;
      r = i / kCols;
    }
    if (r0 + r >= a.rank || b0 + c >= a.cols) continue;
    const float *at = sums + r * pitch + c;
    float s = *at;
    if (blocks > 1) {
      s = ld_cluster(at, 0);
      for (uint32_t b = 1; b < blocks; ++b) s += ld_cluster(at, b);
    }
    // an adapter without rows has no gradient, whatever its scale
    out[a.turned ? (int64_t)(b0 + c) * a.rank + r0 + r : (int64_t)(r0 + r) * a.cols + b0 + c] = empty ? 0.f : s * scale;
  }
}

// An adapter's sums over its rows, 32 at a time, for 16 MT of the rank: a warp has 8
// kLane columns, the cluster's blocks have every so many of the rows.  The block's
// warps share the rows' v, cut into parts and laid out as mma.sync reads it.
template <int MT, bool kWide>
__global__ void __launch_bounds__(kOuterWarps * 32, 1) k_adapt_outer(const OuterPair pair) {
  pdl_wait();
  const uint32_t block = cluster_rank(), blocks = cluster_blocks();
  const int slice = (int)(blockIdx.x / blocks), second = slice >= pair.slices ? 1 : 0;
  const OuterArgs &a = pair.a[second];
  typedef float T;
  typedef Op<T> O;
  constexpr int NT = O::kLane, kCols = 8 * NT, kRank = 16 * MT, kVp = O::kOwnParts, kThreads = kOuterWarps * 32;
  constexpr int kVWords = outer_v_words<MT>(), kPitch = outer_cols(NT) + 1;
  extern __shared__ __align__(16) uint32_t outer_ring[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int adapter = blockIdx.y, r0 = blockIdx.z * kRank;
  const int b0 = (slice - second * pair.slices) * kOuterWarps * kCols;
  const int first = a.start[adapter], end = a.start[adapter + 1];
  const int lane_c = b0 + warp * kCols + NT * g, left = a.cols - lane_c;
  uint4 *ring = reinterpret_cast<uint4 *>(outer_ring) + warp * kOuterStages * 8 * 32 + lane;
  uint32_t *vs = outer_ring + kOuterWarps * kOuterStages * 8 * 128;  // [2][step][part][m tile][lane][4]
  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.f;
  const int step = (int)blocks * kOuterRows;
  const int p_first = first + (int)block * kOuterRows;
  // lane l: the row at place l of the 32 from p0 on (-1 past the end)
  auto tokens_at = [&](int p0) { return p0 + lane < end ? __ldg(a.order + p0 + lane) : -1; };
  // x: rows 16 s + 4 q + i; zeros past the end
  auto fetch = [&](int tokens, bool any, int stage) {
    if (any) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int token = __shfl_sync(0xffffffffu, tokens, 16 * (i >> 2) + 4 * q + (i & 3));
        fetch_vec<T, NT, kWide>(ring + (stage * 8 + i) * 32, reinterpret_cast<const T *>(a.x) + max(token, 0) * a.x_ld + (left > 0 ? lane_c : 0),
                                token >= 0 ? left : 0);
      }
    }
    fetch_commit();
  };
  // v: a thread has four ranks of two neighbouring rows, several times for the larger ranks
  constexpr int kQuads = kRank / 4, kJobs = kOuterRows / 2 * kQuads, kOwn = (kJobs + kThreads - 1) / kThreads;
  Pack<float, 16> held[kOwn][2];
  auto read_v = [&](int tokens) {
#pragma unroll
    for (int o = 0; o < kOwn; ++o) {
      const int job = threadIdx.x + o * kThreads, r = r0 + job % kQuads * 4;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int token = __shfl_sync(0xffffffffu, tokens, (job / kQuads * 2 + k) & 31);
        const bool in = (kJobs % kThreads == 0 || job < kJobs) && token >= 0;
        held[o][k] = load_vec<float, 4>(a.v + (in ? (int64_t)token * a.rank + r : 0), in ? a.rank - r : 0, a.v_wide);
      }
    }
  };
  auto put_v = [&](uint32_t *to) {
#pragma unroll
    for (int o = 0; o < kOwn; ++o) {
      const int job = threadIdx.x + o * kThreads;
      if (kJobs % kThreads != 0 && job >= kJobs) break;
      // row 16 s + 4 q' + 2 k of the pair; rank 16 m + 8 h + g'; the lanes' places turned so that a warp's words
      // fall on all banks
      const int row = job / kQuads * 2, s = row >> 4, qq = (row >> 2) & 3, k = (row >> 1) & 1;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = job % kQuads * 4 + e, m = r >> 4, h = (r >> 3) & 1, gg = r & 7;
        uint32_t w[kVp];
        cut_pair<kVp>(held[o][0].get(e), held[o][1].get(e), w);
#pragma unroll
        for (int p = 0; p < kVp; ++p) to[(((s * kVp + p) * MT + m) * 32 + ((gg * 4 + qq) ^ (m | (gg & 4)))) * 4 + 2 * k + h] = w[p];
      }
    }
  };
  if (p_first < end) {
    int ahead[kOuterStages];  // the rows of the steps to come: of the next one, ..., of the one to fetch
    {
      const int now = tokens_at(p_first);
#pragma unroll
      for (int s = 0; s < kOuterStages; ++s) ahead[s] = tokens_at(p_first + (s + 1) * step);
      fetch(now, true, 0);
      read_v(now);
#pragma unroll
      for (int s = 1; s < kOuterStages - 1; ++s) fetch(ahead[s - 1], p_first + s * step < end, s);
    }
    int stage = 0, turn = 0;
    for (int p0 = p_first; p0 < end; p0 += step, turn ^= 1) {
      put_v(vs + turn * kVWords);
      fetch(ahead[kOuterStages - 2], p0 + (kOuterStages - 1) * step < end, stage == 0 ? kOuterStages - 1 : stage - 1);
      if (p0 + step < end) read_v(ahead[0]);
#pragma unroll
      for (int s = 0; s + 1 < kOuterStages; ++s) ahead[s] = ahead[s + 1];
      ahead[kOuterStages - 1] = tokens_at(p0 + (kOuterStages + 1) * step);
      __syncthreads();  // one per turn: a buffer is written again after the other one's
      fetch_wait<kOuterStages - 1>();
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Pack<T, 16> xv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) xv[i].raw = ring[(stage * 8 + 4 * s + i) * 32];
        uint32_t w[MT][2][2][kVp];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int p = 0; p < kVp; ++p) {
            const uint4 f = reinterpret_cast<const uint4 *>(vs + turn * kVWords)[((s * kVp + p) * MT + m) * 32 + (lane ^ (m | (g & 4)))];
            w[m][0][0][p] = f.x;
            w[m][1][0][p] = f.y;
            w[m][0][1][p] = f.z;
            w[m][1][1][p] = f.w;
          }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint32_t b[2][O::kParts];
#pragma unroll
          for (int k = 0; k < 2; ++k) across(xv[2 * k], xv[2 * k + 1], j, b[k]);
          mma_all<MT, kVp, O::kParts>([&](int m) -> float(&)[4] { return acc[m][j]; },
                                      [&](int m) -> const uint32_t(&)[2][2][kVp] { return w[m]; },
                                      [&](int) -> const uint32_t(&)[2][O::kParts] { return b; });
        }
      }
      if (++stage == kOuterStages) stage = 0;
    }
    fetch_wait<0>();
  }
  __syncthreads();  // the rings become the sums
  float *sums = reinterpret_cast<float *>(outer_ring);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sums[(16 * m + 8 * (e >> 1) + g) * kPitch + warp * kCols + NT * (2 * q + (e & 1)) + j] = acc[m][j][e];
  if (blocks > 1)
    cluster_sync();
  else
    __syncthreads();
  outer_write<kRank, outer_cols(NT), kThreads>(a, sums, kPitch, block, blocks, adapter, r0, b0, first == end);
  if (blocks > 1) cluster_sync();
}

// ------------------------------------------------------------ host side

struct AdaptWs {
  size_t order, start, tiles, h, total;
  int tile_cap;
};

AdaptWs adapt_ws(int64_t n, int32_t adapters, int32_t rank) {
  AdaptWs w;
  size_t o = 0;
  w.order = o;
  o += align_up((size_t)n * 4, kAlign);
  w.start = o;
  o += align_up(((size_t)adapters + 3) * 4, kAlign);
  // every adapter's last tile, and the rows' without one, may be short
  w.tile_cap = (int)(ceil_div(n, kTile) + std::min<int64_t>(n, (int64_t)adapters + 1));
  w.tiles = o;
  o += align_up((size_t)w.tile_cap * sizeof(Tile), kAlign);
  w.h = o;
  o += align_up((size_t)n * (size_t)rank * 4, kAlign);
  w.total = o;
  return w;
}

const int32_t *tile_count(const uint8_t *ws, const AdaptWs &W, int32_t adapters) {
  return reinterpret_cast<const int32_t *>(ws + W.start) + adapters + 2;
}

bool row_wide(const void *p, int64_t ld, size_t es) { return ptr_aligned(p, 16) && (size_t)ld * es % 16 == 0; }

cudaError_t launch_group(const TokenSrc &which, int n, int tile_rows, uint8_t *b, const AdaptWs &W, cudaStream_t s) {
  const int groups = (int)which.vocab + 1, warps = group_warps(groups, n);
  const size_t smem = (size_t)warps * groups * 4;
  cudaError_t e = raise_smem_limit(k_adapt_group, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_adapt_group, 1, kGroupThreads, smem, s, which, n, warps, reinterpret_cast<int32_t *>(b + W.order),
                    reinterpret_cast<int32_t *>(b + W.start), reinterpret_cast<Tile *>(b + W.tiles), W.tile_cap, tile_rows);
}

// tiles that a call is likely to have: half of the short ones
int64_t likely_tiles(int64_t n, int32_t adapters, int tile_rows) {
  return ceil_div(n, tile_rows) + std::min<int64_t>(n, adapters) / 2;
}

// blocks of a cluster: as many as the SMs have room for at a block each, and each with some of the shares
unsigned cluster_for(int64_t blocks, int64_t shares, int sms) {
  unsigned c = 1;
  while (c < kMostCluster && blocks * 2 * c <= (int64_t)sms && shares >= 2 * (int64_t)c) c *= 2;
  return c;
}

}  // namespace
}  // namespace snack
#include "adapt_tc.cuh"
namespace snack {
namespace {

template <int NT, int kHalves, bool kAlong, bool kWide>
cudaError_t launch_down(const DownArgs &a, const FileArgs &f, int64_t n, int tile_cap, int sms, cudaStream_t s) {
  constexpr int kCols = 8 * NT * kHalves;
  const size_t smem = down_smem(kCols);
  const auto kernel = k_adapt_down<NT, kHalves, kAlong, kWide>;
  cudaError_t e = raise_smem_limit(kernel, smem);
  if (e != cudaSuccess) return e;
  const unsigned slices = (unsigned)ceil_div(a.rank, kCols);
  const unsigned c = cluster_for(likely_tiles(n, a.adapters, kTile) * slices, ceil_div(a.k, Op<float>::kGroup * kDownParts), sms);
  return launch_cluster(c, kernel, dim3((unsigned)tile_cap * c, slices), kDownParts * kHalves * 32, smem, s, a, f);
}
// whole accesses of 16 bytes of the rows and of a matrix that runs along K, of `across` elements of one that does not
template <typename T, bool kAlong>
bool down_wide(DownArgs *a, int across) {
  const size_t es = sizeof(T);
  a->x_wide = row_wide(a->x, a->x_ld, es);
  a->m_wide = kAlong ? row_wide(a->m, a->k, es) : ptr_aligned(a->m, across * es) && a->rank % across == 0;
  return a->x_wide && a->m_wide;
}
template <int NT, int kHalves, bool kAlong>
cudaError_t down_by(DownArgs a, const FileArgs &f, int64_t n, int tile_cap, int sms, cudaStream_t s) {
  return down_wide<float, kAlong>(&a, NT) ? launch_down<NT, kHalves, kAlong, true>(a, f, n, tile_cap, sms, s)
                                          : launch_down<NT, kHalves, kAlong, false>(a, f, n, tile_cap, sms, s);
}
template <typename T, bool kAlong>
cudaError_t down(const DownArgs &a, const FileArgs &f, int64_t n, int tile_cap, int sms, cudaStream_t s) {
  if constexpr (sizeof(T) == 2)
    return down_tc<kAlong>(a, f, likely_tiles(n, a.adapters, kTcTile), tile_cap, sms, s);
  else
    return a.rank <= 16 ? down_by<2, 1, kAlong>(a, f, n, tile_cap, sms, s) : down_by<2, 2, kAlong>(a, f, n, tile_cap, sms, s);
}

template <bool kAlong, bool kWide>
cudaError_t launch_up(UpArgs a, int64_t n, int tile_cap, int sms, cudaStream_t s) {
  const size_t smem = (size_t)kUpWarps * up_stages<float>() * up_stage_bytes<float, 1>() * 32 + up_h_bytes<float>(a.rank);
  const auto kernel = k_adapt_up<kAlong, kWide>;
  cudaError_t e = raise_smem_limit(kernel, smem);
  if (e != cudaSuccess) return e;
  const int64_t all = ceil_div(a.cols, kUpWarps * kUpCols);
  // a block that has more columns reads its rows of h for all of them, as long as there are four blocks per SM
  int64_t groups = std::max<int64_t>(1, likely_tiles(n, a.adapters, kTile) * all / (4 * (int64_t)sms));
  groups = std::min<int64_t>(groups, 16);
  if (ceil_div(all, groups) > 65535) groups = ceil_div(all, 65535);
  a.groups = (int)groups;
  return launch_pdl(kernel, dim3((unsigned)tile_cap, (unsigned)ceil_div(all, groups)), kUpWarps * 64, smem, s, (const UpArgs)a);
}
// whole accesses of 16 bytes of the rows, of four elements of the matrix
template <typename T, bool kAlong>
bool up_wide(UpArgs *a) {
  const size_t es = sizeof(T);
  a->m_wide = ptr_aligned(a->m, 4 * es) && (kAlong ? a->rank : a->cols) % 4 == 0;
  return row_wide(a->base, a->base_ld, es) && row_wide(a->out, a->out_ld, es) && a->m_wide;
}
template <bool kAlong>
cudaError_t up_by(UpArgs a, int64_t n, int tile_cap, int sms, cudaStream_t s) {
  return up_wide<float, kAlong>(&a) ? launch_up<kAlong, true>(a, n, tile_cap, sms, s) : launch_up<kAlong, false>(a, n, tile_cap, sms, s);
}
template <typename T, bool kAlong>
cudaError_t up(const UpArgs &a, int64_t n, int tile_cap, int sms, cudaStream_t s) {
  if constexpr (sizeof(T) == 2)
    return up_tc<kAlong>(a, tile_cap, sms, s);
  else
    return up_by<kAlong>(a, n, tile_cap, sms, s);
}

template <typename T, int NT, int kSteps, bool kWide>
cudaError_t launch_few(const DownArgs &d, UpArgs u, const TokenSrc &which, int n, int sms, cudaStream_t s) {
  const size_t smem = std::max((size_t)down_smem(16 * NT),
                               (size_t)kUpWarps * up_stages<T>() * up_stage_bytes<T, kSteps>() * 32 + up_h_bytes<T>(u.rank));
  const auto kernel = k_adapt_few<T, NT, kSteps, kWide>;
  cudaError_t e = raise_smem_limit(kernel, smem);
  if (e != cudaSuccess) return e;
  const int64_t shares = std::max(ceil_div(d.k, Op<T>::kGroup * kDownParts), ceil_div(u.cols, kUpWarps * kUpCols));
  const unsigned c = cluster_for(std::min<int64_t>(n, (int64_t)d.adapters + 1), shares, sms);
  u.groups = (int)ceil_div(u.cols, (int64_t)c * kUpWarps * kUpCols);
  return launch_cluster(c, kernel, dim3((unsigned)n * c), kFewThreads, smem, s, d, (const UpArgs)u, which, n);
}
template <typename T>
cudaError_t few(DownArgs d, UpArgs u, const TokenSrc &which, int n, int sms, cudaStream_t s) {
  const bool wide_in = down_wide<T, true>(&d, 8), wide = up_wide<T, true>(&u) && wide_in;
  constexpr int kSteps = sizeof(T) == 2 ? 2 : 1;
  if (d.rank <= 16) return wide ? launch_few<T, 1, 1, true>(d, u, which, n, sms, s) : launch_few<T, 1, 1, false>(d, u, which, n, sms, s);
  return wide ? launch_few<T, 2, kSteps, true>(d, u, which, n, sms, s) : launch_few<T, 2, kSteps, false>(d, u, which, n, sms, s);
}

template <int MT, bool kWide>
cudaError_t launch_outer(OuterPair p, int64_t n, int32_t adapters, int sms, cudaStream_t s) {
  const size_t smem = outer_smem<MT>();
  const auto kernel = k_adapt_outer<MT, kWide>;
  cudaError_t e = raise_smem_limit(kernel, smem);
  if (e != cudaSuccess) return e;
  constexpr int kCols = outer_cols(Op<float>::kLane);
  p.slices = p.a[0].out ? (int32_t)ceil_div(p.a[0].cols, kCols) : 0;
  const int64_t slices = p.slices + (p.a[1].out ? ceil_div(p.a[1].cols, kCols) : 0);
  const int32_t rank = p.a[p.slices ? 0 : 1].rank;
  const int64_t ranks = ceil_div(rank, 16 * MT);
  const unsigned c = cluster_for(slices * ranks * adapters, ceil_div(n, (int64_t)adapters * kOuterRows), sms);
  return launch_cluster(c, kernel, dim3((unsigned)(slices * c), (unsigned)adapters, (unsigned)ranks), kOuterWarps * 32, smem, s,
                        (const OuterPair)p);
}
template <typename T>
cudaError_t outer(const OuterPair &p, int32_t rank, int64_t n, int32_t adapters, int sms, cudaStream_t s) {
  const auto aligned = [](const OuterArgs &a) { return !a.out || row_wide(a.x, a.x_ld, sizeof(T)); };
  const bool wide = aligned(p.a[0]) && aligned(p.a[1]);
  if constexpr (sizeof(T) == 2) {
    if (rank <= 32) return wide ? launch_outer_tc<32, true>(p, n, adapters, sms, s) : launch_outer_tc<32, false>(p, n, adapters, sms, s);
    return wide ? launch_outer_tc<64, true>(p, n, adapters, sms, s) : launch_outer_tc<64, false>(p, n, adapters, sms, s);
  } else {
    if (rank <= 16) return wide ? launch_outer<1, true>(p, n, adapters, sms, s) : launch_outer<1, false>(p, n, adapters, sms, s);
    if (rank <= 32) return wide ? launch_outer<2, true>(p, n, adapters, sms, s) : launch_outer<2, false>(p, n, adapters, sms, s);
    return wide ? launch_outer<4, true>(p, n, adapters, sms, s) : launch_outer<4, false>(p, n, adapters, sms, s);
  }
}

snack_status adapt_check(int64_t n, int32_t adapters, int32_t rank, int32_t in_f, int32_t out_f, snack_dtype t) {
  if (!lm_dtype_ok(t) || n < 0 || adapters < 1 || rank < 1 || in_f < 1 || out_f < 1) return SNACK_ERR_INVALID_ARG;
  if (n >= (1 << 24) || adapters > kMostAdapters || rank > kMostRank || in_f >= (1 << 20) || out_f >= (1 << 20))
    return SNACK_ERR_UNSUPPORTED;
  return SNACK_OK;
}

struct Span {
  const void *p;
  size_t bytes;
};
bool overlaps(const Span &a, const Span &b) { return spans_overlap(a.p, a.bytes, b.p, b.bytes); }

int tile_rows(snack_dtype t) { return t == SNACK_BF16 ? kTcTile : kTile; }
// how the first kernel files the rows itself; without ids where they are too many
FileArgs file_args(const TokenSrc &which, int n, snack_dtype t, uint8_t *ws, const AdaptWs &W) {
  FileArgs f = {};
  if (n > kFileRows || which.vocab > (uint32_t)kFileAdapters) return f;
  f.which = which;
  f.n = n;
  f.tile_rows = tile_rows(t);
  f.tile_cap = W.tile_cap;
  f.order = reinterpret_cast<int32_t *>(ws + W.order);
  f.start = reinterpret_cast<int32_t *>(ws + W.start);
  f.tiles = reinterpret_cast<Tile *>(ws + W.tiles);
  return f;
}

template <typename T>
cudaError_t run_fwd(const DownArgs &d, const UpArgs &u, const FileArgs &f, int64_t n, const AdaptWs &W, int sms, cudaStream_t s) {
  cudaError_t e = down<T, true>(d, f, n, W.tile_cap, sms, s);
  return e != cudaSuccess ? e : up<T, true>(u, n, W.tile_cap, sms, s);
}

int sms_here() {
  const int n = current_sms();
  return n < 1 ? 152 : n;
}

}  // namespace
}  // namespace snack

using namespace snack;

#define ADAPT_CUDA(...)                                      \
  do {                                                       \
    if ((__VA_ARGS__) != cudaSuccess) return SNACK_ERR_CUDA; \
  } while (0)

extern "C" {

snack_status snack_adapt_workspace_size(int64_t n, int32_t n_adapters, int32_t rank, size_t *bytes) {
  if (!bytes) return SNACK_ERR_INVALID_ARG;
  const snack_status st = adapt_check(n, n_adapters, rank, 1, 1, SNACK_F32);
  if (st != SNACK_OK) return st;
  *bytes = n == 0 ? 0 : adapt_ws(n, n_adapters, rank).total;
  return SNACK_OK;
}

snack_status snack_adapt_fwd(const void *x, int64_t x_ld, int64_t n, const void *a, const void *b, int32_t n_adapters,
                             int32_t rank, int32_t in_f, int32_t out_f, snack_dtype t, const void *which,
                             snack_index which_t, const float *scales, const void *base, int64_t base_ld, void *y,
                             int64_t y_ld, float *h, void *ws, size_t ws_bytes, snack_stream_t stream) try {
  const snack_status ck = adapt_check(n, n_adapters, rank, in_f, out_f, t);
  if (ck != SNACK_OK) return ck;
  if (!lm_index_ok(which_t) || x_ld < in_f || y_ld < out_f || (base && base_ld < out_f)) return SNACK_ERR_INVALID_ARG;
  if (n == 0) return SNACK_OK;
  const size_t es = dtype_size(t);
  if (!x || !a || !b || !which || !y || !ws || !ptr_aligned(x, es) || !ptr_aligned(a, es) || !ptr_aligned(b, es) ||
      !ptr_aligned(y, es) || !ptr_aligned(base, es) || !ptr_aligned(scales, 4) || !ptr_aligned(h, 4) ||
      !ptr_aligned(which, index_size(which_t)) || !ptr_aligned(ws, kAlign))
    return SNACK_ERR_INVALID_ARG;
  const AdaptWs W = adapt_ws(n, n_adapters, rank);
  const Span sy = {y, span_bytes(n, out_f, y_ld, es)}, sh = {h, h ? (size_t)n * rank * 4 : 0}, sw = {ws, W.total};
  const Span sbase = {base, base ? span_bytes(n, out_f, base_ld, es) : 0};
  const Span read[] = {{x, span_bytes(n, in_f, x_ld, es)},
                       {a, (size_t)n_adapters * rank * in_f * es},
                       {b, (size_t)n_adapters * rank * out_f * es},
                       {which, (size_t)n * index_size(which_t)},
                       {scales, scales ? (size_t)n_adapters * 4 : 0}};
  for (const Span &r : read)
    if (overlaps(sy, r) || overlaps(sh, r) || overlaps(sw, r)) return SNACK_ERR_INVALID_ARG;
  const bool in_place = base == y && (n == 1 || base_ld == y_ld);  // of one row the step means nothing
  if ((!in_place && overlaps(sy, sbase)) || overlaps(sh, sbase) || overlaps(sw, sbase) || overlaps(sy, sh) || overlaps(sy, sw) ||
      overlaps(sh, sw))
    return SNACK_ERR_INVALID_ARG;
  if (ws_bytes < W.total) return SNACK_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t *w = reinterpret_cast<uint8_t *>(ws);
  const int sms = sms_here();
  DownArgs d = {};
  d.x = x;
  d.x_ld = x_ld;
  d.m = a;
  d.k = in_f;
  d.rank = rank;
  d.order = reinterpret_cast<const int32_t *>(w + W.order);
  d.tiles = reinterpret_cast<const Tile *>(w + W.tiles);
  d.adapters = n_adapters;
  d.h = h ? h : reinterpret_cast<float *>(w + W.h);
  UpArgs u = {};
  u.h = d.h;
  u.m = b;
  u.cols = out_f;
  u.rank = rank;
  u.order = d.order;
  u.tiles = d.tiles;
  u.n_tiles = tile_count(w, W, n_adapters);
  u.adapters = n_adapters;
  u.scales = scales;
  u.base = base;
  u.base_ld = base_ld;
  u.out = y;
  u.out_ld = y_ld;
  u.h_wide = rank % 4 == 0 && ptr_aligned(d.h, 16);
  const TokenSrc ids{which, which_t == SNACK_I64, (uint32_t)n_adapters};
  if (n <= (rank <= 32 ? kFewRows : kFewRows / 4)) {
    ADAPT_CUDA(t == SNACK_F32 ? few<float>(d, u, ids, (int)n, sms, s) : few<bf16>(d, u, ids, (int)n, sms, s));
    return SNACK_OK;
  }
  const FileArgs f = file_args(ids, (int)n, t, w, W);
  if (!f.which.ids) ADAPT_CUDA(launch_group(ids, (int)n, tile_rows(t), w, W, s));
  ADAPT_CUDA(t == SNACK_F32 ? run_fwd<float>(d, u, f, n, W, sms, s) : run_fwd<bf16>(d, u, f, n, W, sms, s));
  return SNACK_OK;
} catch (...) {  // a host allocation failed
  return SNACK_ERR_CUDA;
}

snack_status snack_adapt_bwd(const void *x, int64_t x_ld, int64_t n, const void *a, const void *b, int32_t n_adapters,
                             int32_t rank, int32_t in_f, int32_t out_f, snack_dtype t, const void *which,
                             snack_index which_t, const float *scales, const float *h, const void *dy, int64_t dy_ld,
                             int accumulate, void *dx, int64_t dx_ld, void *da, void *db, void *ws, size_t ws_bytes,
                             snack_stream_t stream) try {
  const snack_status ck = adapt_check(n, n_adapters, rank, in_f, out_f, t);
  if (ck != SNACK_OK) return ck;
  const size_t es = dtype_size(t);
  if (!lm_index_ok(which_t) || (dx && (dx_ld < in_f || !ptr_aligned(dx, es))) || !ptr_aligned(da, es) || !ptr_aligned(db, es))
    return SNACK_ERR_INVALID_ARG;
  const size_t na = (size_t)n_adapters * rank * in_f * es, nb = (size_t)n_adapters * rank * out_f * es;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (n == 0) {
    if (da) ADAPT_CUDA(cudaMemsetAsync(da, 0, na, s));
    if (db) ADAPT_CUDA(cudaMemsetAsync(db, 0, nb, s));
    return SNACK_OK;
  }
  if (x_ld < in_f || dy_ld < out_f) return SNACK_ERR_INVALID_ARG;
  if (!x || !a || !b || !which || !dy || !ws || (db && !h) || !ptr_aligned(x, es) || !ptr_aligned(a, es) || !ptr_aligned(b, es) ||
      !ptr_aligned(dy, es) || !ptr_aligned(scales, 4) || !ptr_aligned(h, 4) || !ptr_aligned(which, index_size(which_t)) ||
      !ptr_aligned(ws, kAlign))
    return SNACK_ERR_INVALID_ARG;
  const AdaptWs W = adapt_ws(n, n_adapters, rank);
  const Span written[] = {{dx, dx ? span_bytes(n, in_f, dx_ld, es) : 0}, {da, da ? na : 0}, {db, db ? nb : 0}, {ws, W.total}};
  const Span read[] = {{x, span_bytes(n, in_f, x_ld, es)},
                       {a, na},
                       {b, nb},
                       {which, (size_t)n * index_size(which_t)},
                       {scales, scales ? (size_t)n_adapters * 4 : 0},
                       {h, h ? (size_t)n * rank * 4 : 0},
                       {dy, span_bytes(n, out_f, dy_ld, es)}};
  for (int i = 0; i < 4; ++i) {
    for (int j = i + 1; j < 4; ++j)
      if (overlaps(written[i], written[j])) return SNACK_ERR_INVALID_ARG;
    for (const Span &r : read)
      if (overlaps(written[i], r)) return SNACK_ERR_INVALID_ARG;
  }
  if (ws_bytes < W.total) return SNACK_ERR_WORKSPACE;
  if (!dx && !da && !db) return SNACK_OK;
  uint8_t *w = reinterpret_cast<uint8_t *>(ws);
  const int sms = sms_here();
  const bool wide32 = t == SNACK_F32;
  const int32_t *order = reinterpret_cast<const int32_t *>(w + W.order), *start = reinterpret_cast<const int32_t *>(w + W.start);
  float *dh = reinterpret_cast<float *>(w + W.h);
  DownArgs d = {};
  d.x = dy;
  d.x_ld = dy_ld;
  d.m = b;
  d.k = out_f;
  d.rank = rank;
  d.order = order;
  d.tiles = reinterpret_cast<const Tile *>(w + W.tiles);
  d.adapters = n_adapters;
  d.scales = scales;
  d.h = dh;
  UpArgs u = {};
  u.h = dh;
  u.m = a;
  u.cols = in_f;
  u.rank = rank;
  u.order = order;
  u.tiles = d.tiles;
  u.n_tiles = tile_count(w, W, n_adapters);
  u.adapters = n_adapters;
  u.base = accumulate ? dx : nullptr;
  u.base_ld = dx_ld;
  u.out = dx;
  u.out_ld = dx_ld;
  u.h_wide = rank % 4 == 0;
  const TokenSrc ids{which, which_t == SNACK_I64, (uint32_t)n_adapters};
  const FileArgs f = dx || da ? file_args(ids, (int)n, t, w, W) : FileArgs{};
  if (!f.which.ids) ADAPT_CUDA(launch_group(ids, (int)n, tile_rows(t), w, W, s));
  if (dx || da)
    ADAPT_CUDA(wide32 ? down<float, false>(d, f, n, W.tile_cap, sms, s) : down<bf16, false>(d, f, n, W.tile_cap, sms, s));
  if (dx) ADAPT_CUDA(wide32 ? up<float, false>(u, n, W.tile_cap, sms, s) : up<bf16, false>(u, n, W.tile_cap, sms, s));
  if (da || db) {
    OuterPair p = {};
    for (OuterArgs &o : p.a) {
      o.rank = rank;
      o.order = order;
      o.start = start;
    }
    p.a[0].v = dh;
    p.a[0].v_wide = rank % 4 == 0;
    p.a[0].x = x;
    p.a[0].x_ld = x_ld;
    p.a[0].cols = in_f;
    p.a[0].out = da;
    p.a[1].v = h;
    p.a[1].v_wide = rank % 4 == 0 && ptr_aligned(h, 16);
    p.a[1].x = dy;
    p.a[1].x_ld = dy_ld;
    p.a[1].cols = out_f;
    p.a[1].out = db;
    p.a[1].turned = 1;
    p.a[1].scales = scales;
    ADAPT_CUDA(wide32 ? outer<float>(p, rank, n, n_adapters, sms, s) : outer<bf16>(p, rank, n, n_adapters, sms, s));
  }
  return SNACK_OK;
} catch (...) {  // a host allocation failed
  return SNACK_ERR_CUDA;
}

}  // extern "C"
