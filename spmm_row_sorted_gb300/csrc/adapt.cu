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
// (dy, dx) go over the bus once each, an adapter's matrices once per 64 rows,
// out of L2.  One block first files the rows by adapter, stably, into tiles of up
// to 64 rows of one adapter (k_adapt_group).  Three kernels do the products:
//   down   h, dh: a tile against one adapter's matrix, K split over a block's
//          warps and a cluster's blocks, whose sums meet in shared memory;
//   up     y, dx: rank is the K, so a tile's h stays in shared memory and each
//          warp has 32 columns; the product is added to the base and rounded once;
//   outer  dA, dB: sums over an adapter's rows, in their order.
// The products run on the tensor cores by mma.sync, operands straight from global
// memory: which columns of a group a lane holds does not matter to a sum as long as
// both operands agree, so every lane reads 16 consecutive bytes of a row.  (tcgen05
// would want 128 rows of one adapter and a rank of 64 at least, and both operands
// laid out in shared memory, to save arithmetic that is not the bound.)  fp32
// operands are cut into three bf16 parts in registers, six part products down to
// 2^-16 of the leading one, 16 of K on the tensor core at a time: its sums round
// towards zero.  h and dh are fp32 in memory and go into products as two bf16 parts
// (bf16 operands: 2^-17 of an entry, far below the output's rounding) or three.
// Every sum has one order: results repeat bit for bit.
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

int group_warps(int groups) {
  const int w = kGroupBytes / 4 / groups;
  return w < 1 ? 1 : w > kGroupThreads / 32 ? kGroupThreads / 32 : w;
}

// Each warp counts a stretch of the rows by adapter; the counts, added up over
// adapters and warps, say where its rows go.  8192 rows: see adapt_fwd's figures.
__global__ void __launch_bounds__(kGroupThreads, 1)
    k_adapt_group(TokenSrc which, int n, int warps, int32_t *__restrict__ order, int32_t *__restrict__ start,
                  Tile *__restrict__ tiles, int tile_cap) {
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
      }
#pragma unroll
      for (int u = 0; u < kGroupKeep; ++u) {
        if (r0 + u >= rounds) break;
        const unsigned peers = __match_any_sync(0xffffffffu, kept[u]);
        const bool here = kept[u] != 0xFFFFFFFFu;
        const int at = here ? mine[kept[u]] : 0;
        __syncwarp();
        if (here && (peers & below) == 0) mine[kept[u]] = at + __popc(peers);
        if (here && place) order[at + __popc(peers & below)] = (int32_t)(first + (int64_t)(r0 + u) * 32 + lane);
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
      for (int w = 0; w < warps; ++w) {
        const int c = hist[w * groups + g];
        hist[w * groups + g] = count;
        count += c;
      }
    const int own = (count + kTile - 1) / kTile;
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
    int2 before = carry;
    for (int w = 0; w < kGroupThreads / 32; ++w) {
      if (w < warp) {
        before.x += warp_sum[w].x;
        before.y += warp_sum[w].y;
      }
      carry.x += warp_sum[w].x;
      carry.y += warp_sum[w].y;
    }
    const int from = before.x + inc.x - count, tile = before.y + inc.y - own;
    if (g < groups) {
      start[g] = from;
      for (int w = 0; w < warps; ++w) hist[w * groups + g] += from;
      for (int t = 0; t < own; ++t)
        tiles[tile + t] = Tile{g, from + t * kTile, min(kTile, count - t * kTile), 0};
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) start[groups] = n;
  for (int t = carry.y + threadIdx.x; t < tile_cap; t += kGroupThreads) tiles[t] = Tile{-1, 0, 0, 0};
  pass(true);
}

// ------------------------------------------------------------ operands

// What of a group of K a lane holds: 16 bytes of a row that runs along K, four
// consecutive elements for each step of 16.
template <typename T>
struct Op;
template <>
struct Op<bf16> {
  static constexpr int kSteps = 2, kParts = 1, kLane = 8, kGroup = 32;  // elements per lane, K per group
};
template <>
struct Op<float> {
  static constexpr int kSteps = 1, kParts = 3, kLane = 4, kGroup = 16;
};

// V consecutive elements as they are; zeros from `left` on.  kConst: of memory that
// the kernel does not write.
template <typename T, int V, bool kConst = true>
__device__ __forceinline__ Pack<T, V * (int)sizeof(T)> load_vec(const T *p, int left, bool wide) {
  Pack<T, V * (int)sizeof(T)> r;
  auto get = [](auto *at) { return kConst ? __ldg(at) : *at; };
  if (wide && left >= V) {
    r.raw = get(reinterpret_cast<const typename Raw<V * (int)sizeof(T)>::type *>(p));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (sizeof(T) == 4)
        r.w[i] = i < left ? __float_as_uint(get(p + i)) : 0u;
      else
        r.h[i] = i < left ? get(reinterpret_cast<const uint16_t *>(p) + i) : (uint16_t)0;
    }
  }
  return r;
}
// the same of more than 16 bytes
template <typename T, int V>
struct Many {
  static constexpr int kPer = V * (int)sizeof(T) > 16 ? 16 / (int)sizeof(T) : V;
  Pack<T, kPer * (int)sizeof(T)> p[V / kPer];
  __device__ __forceinline__ void load(const T *at, int left, bool wide) {
#pragma unroll
    for (int i = 0; i < V / kPer; ++i) p[i] = load_vec<T, kPer>(at + i * kPer, left - i * kPer, wide);
  }
  __device__ __forceinline__ float get(int i) const { return p[i / kPer].get(i % kPer); }
};

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

// A pair of values as kParts words of two bf16: three cut off, 8 significant bits
// each, or two rounded.
template <int kParts>
__device__ __forceinline__ void cut_pair(float a, float b, uint32_t (&w)[kParts]) {
  if constexpr (kParts == 1) {
    w[0] = upper_halves(a, b);  // values that are bf16
  } else if constexpr (kParts == 2) {
    w[0] = pack_pair(a, b);
    w[1] = pack_pair(a - bf16_lo(w[0]), b - bf16_hi(w[0]));
  } else {
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
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// acc += a b over 16 of K: rows g (lo) and g + 8 (hi) of a, in parts; the small
// products first, and those of fp32 operands summed apart from what is there.
template <int kA, int kB>
__device__ __forceinline__ void mma_step(float (&acc)[4], const uint32_t (&lo)[2][kA], const uint32_t (&hi)[2][kA],
                                         const uint32_t (&b)[2][kB]) {
  if constexpr (kA == 3 && kB == 3) {
    float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int sum = 2; sum >= 0; --sum)
#pragma unroll
      for (int i = sum; i >= 0; --i) mma(d, lo[0][i], hi[0][i], lo[1][i], hi[1][i], b[0][sum - i], b[1][sum - i]);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] += d[e];
  } else {
    static_assert(kB == 1, "one part");
#pragma unroll
    for (int i = kA - 1; i >= 0; --i) mma(acc, lo[0][i], hi[0][i], lo[1][i], hi[1][i], b[0][0], b[1][0]);
  }
}

// a lane's words of a row along K: [step][half of the step's pairs][part]
template <typename T>
struct Along {
  uint32_t w[Op<T>::kSteps][2][Op<T>::kParts];
  __device__ __forceinline__ void set(const Pack<T, 16> &v) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) w[s][h][0] = v.w[2 * s + h];
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) cut_pair<3>(v.get(2 * h), v.get(2 * h + 1), w[0][h]);
    }
  }
};
// pairs of element j of two rows that follow one another along K
template <typename T, typename V>
__device__ __forceinline__ void across(const V &a, const V &b, int j, uint32_t (&w)[Op<T>::kParts]) {
  cut_pair<Op<T>::kParts>(a.get(j), b.get(j), w);
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
  int x_wide, m_wide;
};

constexpr int kDownWarps = 8;

// The sums of kDownWarps warps over their parts of K, and of the cluster's blocks.
template <typename T, int MT, int NT, bool kAlong>
__device__ __forceinline__ void down_tile(const DownArgs &a, const Tile &tile, float *smem) {
  typedef Op<T> O;
  constexpr int kRows = 16 * MT, kCols = 8 * NT;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int r0 = blockIdx.y * kCols;
  const uint32_t rank = cluster_rank(), blocks = cluster_blocks();
  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.f;
  const T *row[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // the rows past the tile's end are the last one's again, and not kept
      const int at = min(16 * m + 8 * h + g, tile.count - 1);
      row[m][h] = reinterpret_cast<const T *>(a.x) + (int64_t)__ldg(a.order + tile.first + at) * a.x_ld + O::kLane * q;
    }
  const T *mat = reinterpret_cast<const T *>(a.m) + (int64_t)tile.adapter * a.rank * a.k;
  for (int k0 = (int)(rank * kDownWarps + warp) * O::kGroup; k0 < a.k; k0 += (int)blocks * kDownWarps * O::kGroup) {
    const int left = a.k - k0 - O::kLane * q;
    Pack<T, 16> xv[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) xv[m][h] = load_vec<T, O::kLane>(row[m][h] + k0, left, a.x_wide);
    if constexpr (kAlong) {
      Pack<T, 16> mv[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int r = r0 + 8 * j + g;
        mv[j] = load_vec<T, O::kLane>(mat + (int64_t)min(r, a.rank - 1) * a.k + k0 + O::kLane * q, r < a.rank ? left : 0, a.m_wide);
      }
      Along<T> xa[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) xa[m][h].set(xv[m][h]);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        Along<T> b;
        b.set(mv[j]);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int s = 0; s < O::kSteps; ++s) mma_step(acc[m][j], xa[m][0].w[s], xa[m][1].w[s], b.w[s]);
      }
    } else {
      Many<T, NT> mv[O::kLane];  // rows k0 + kLane q + i: ranks NT g .. NT g + NT - 1
#pragma unroll
      for (int i = 0; i < O::kLane; ++i)
        mv[i].load(mat + (int64_t)min(k0 + O::kLane * q + i, a.k - 1) * a.rank + r0 + NT * g, i < left ? a.rank - r0 - NT * g : 0, a.m_wide);
      Along<T> xa[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) xa[m][h].set(xv[m][h]);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int s = 0; s < O::kSteps; ++s) {
          uint32_t b[2][O::kParts];
#pragma unroll
          for (int h = 0; h < 2; ++h) across<T>(mv[4 * s + 2 * h], mv[4 * s + 2 * h + 1], j, b[h]);
#pragma unroll
          for (int m = 0; m < MT; ++m) mma_step(acc[m][j], xa[m][0].w[s], xa[m][1].w[s], b);
        }
    }
  }
  // the warps' sums: the upper half's to the lower half, then those of the four
  float *own = smem + (warp & 3) * (kRows * kCols);
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
  if (warp >= 4) each([](float &s, float &v) { s = v; });
  __syncthreads();
  if (warp < 4) each([](float &s, float &v) { s += v; });
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * kCols; i += kDownWarps * 32)
    smem[i] = (smem[i] + smem[kRows * kCols + i]) + (smem[2 * kRows * kCols + i] + smem[3 * kRows * kCols + i]);
  if (blocks > 1)
    cluster_sync();
  else
    __syncthreads();
  const float scale = a.scales ? a.scales[tile.adapter] : 1.f;
  for (int i = (int)rank * kDownWarps * 32 + threadIdx.x; i < tile.count * kCols; i += (int)blocks * kDownWarps * 32) {
    const int t = i / kCols, r = r0 + i % kCols;
    float s = smem[i];
    if (blocks > 1) {
      s = ld_cluster(smem + i, 0);
      for (uint32_t b = 1; b < blocks; ++b) s += ld_cluster(smem + i, b);
    }
    if (r < a.rank) a.h[(int64_t)a.order[tile.first + t] * a.rank + r] = s * scale;
  }
  if (blocks > 1) cluster_sync();  // no block's memory is read any more
}

template <typename T, int NT, bool kAlong>
__global__ void __launch_bounds__(kDownWarps * 32) k_adapt_down(const DownArgs a) {
  pdl_wait();
  extern __shared__ __align__(16) float down_smem[];
  const Tile tile = a.tiles[blockIdx.x / cluster_blocks()];
  if (tile.adapter < 0 || tile.adapter >= a.adapters) return;  // the whole cluster's
  if (tile.count <= 16)
    down_tile<T, 1, NT, kAlong>(a, tile, down_smem);
  else
    down_tile<T, 4, NT, kAlong>(a, tile, down_smem);
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
  int m_wide, base_wide, out_wide;
};

constexpr int kUpWarps = 4;
constexpr int kUpCols = 32;  // columns of a warp at a time

// of a row of h's parts in shared memory, in elements: rows start 32 bytes apart modulo 128
__host__ __device__ __forceinline__ int up_ld(int rank) { return (rank + 63) / 64 * 64 + 16; }

template <typename T, bool kAlong>
__global__ void __launch_bounds__(kUpWarps * 32) k_adapt_up(const UpArgs a) {
  pdl_wait();
  constexpr int kHp = sizeof(T) == 2 ? 2 : 3, kBp = Op<T>::kParts, MT = kTile / 16, NT = 4;
  typedef Pack<T, 16> P;
  constexpr int kPer = P::kN, kVecs = 8 / kPer;  // accesses for a lane's 8 columns
  extern __shared__ __align__(16) uint32_t up_smem[];
  const Tile tile = a.tiles[blockIdx.x];
  if (tile.adapter < 0) return;
  const bool none = tile.adapter >= a.adapters;
  if (none && a.base == a.out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int ld = up_ld(a.rank) / 2, plane = kTile * ld;  // in words
  const int steps = (a.rank + 15) / 16;
  const int m_tiles = (tile.count + 15) / 16;
  if (!none) {
    const int pairs = steps * 8;
    for (int i = threadIdx.x; i < m_tiles * 16 * pairs; i += kUpWarps * 32) {
      const int t = i / pairs, r = (i - t * pairs) * 2;
      const float *at = a.h + (int64_t)(t < tile.count ? a.order[tile.first + t] : 0) * a.rank + r;
      const float lo = t < tile.count && r < a.rank ? __ldg(at) : 0.f, hi = t < tile.count && r + 1 < a.rank ? __ldg(at + 1) : 0.f;
      uint32_t w[kHp];
      cut_pair<kHp>(lo, hi, w);
#pragma unroll
      for (int p = 0; p < kHp; ++p) up_smem[p * plane + t * ld + (r >> 1)] = w[p];
    }
  }
  __syncthreads();
  const float scale = none ? 0.f : a.scales ? a.scales[tile.adapter] : 1.f;
  const T *mat = reinterpret_cast<const T *>(a.m) + (none ? 0 : (int64_t)tile.adapter * a.rank * a.cols);
  for (int u = 0; u < a.groups; ++u) {
    const int n0 = ((blockIdx.y * a.groups + u) * kUpWarps + warp) * kUpCols;
    if (n0 >= a.cols) break;
    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.f;
    for (int s = 0; s < (none ? 0 : steps); ++s) {
      uint32_t b[NT][2][kBp];
      if constexpr (kAlong) {  // lane g has column 8 (g / 2) + 2 j + g % 2: a lane's sums are 8 neighbours
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int c = n0 + 8 * (g >> 1) + 2 * j + (g & 1), r = 16 * s + 4 * q;
          const auto v = load_vec<T, 4>(mat + (int64_t)min(c, a.cols - 1) * a.rank + r, c < a.cols ? a.rank - r : 0, a.m_wide);
#pragma unroll
          for (int h = 0; h < 2; ++h) cut_pair<kBp>(v.get(2 * h), v.get(2 * h + 1), b[j][h]);
        }
      } else {  // column 4 g + j
        Pack<T, 4 * (int)sizeof(T)> v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 16 * s + 4 * q + i;
          v[i] = load_vec<T, 4>(mat + (int64_t)min(r, a.rank - 1) * a.cols + n0 + 4 * g, r < a.rank ? a.cols - n0 - 4 * g : 0, a.m_wide);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) across<T>(v[2 * h], v[2 * h + 1], j, b[j][h]);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (m >= m_tiles) break;
        uint32_t w[2][2][kHp];  // rows g and g + 8
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int p = 0; p < kHp; ++p) {
            const uint2 v = *reinterpret_cast<const uint2 *>(up_smem + p * plane + (16 * m + 8 * h + g) * ld + 8 * s + 2 * q);
            w[h][0][p] = v.x;
            w[h][1][p] = v.y;
          }
#pragma unroll
        for (int j = 0; j < NT; ++j) mma_step(acc[m][j], w[0], w[1], b[j]);
      }
    }
    const int c = n0 + 8 * q, left = a.cols - c;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m >= m_tiles) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = 16 * m + 8 * h + g;
        if (t >= tile.count || left <= 0) continue;
        const int64_t token = a.order[tile.first + t];
        const T *base = reinterpret_cast<const T *>(a.base) + token * a.base_ld + c;
        T *out = reinterpret_cast<T *>(a.out) + token * a.out_ld + c;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
          P o;
          if (a.base)
            o = load_vec<T, kPer, false>(base + v * kPer, left - v * kPer, a.base_wide);
          else
            o.raw = make_uint4(0, 0, 0, 0);
          if (!none)
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
              const int e = v * kPer + i;  // of the lane's 8 columns
              const float d = kAlong ? acc[m][e >> 1][2 * h + (e & 1)] : acc[m][e & 3][2 * h + (e >> 2)];
              o.set(i, fmaf(scale, d, o.get(i)));
            }
          if (a.out_wide && left >= (v + 1) * kPer) {
            *reinterpret_cast<uint4 *>(out + v * kPer) = o.raw;
          } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
              if (v * kPer + i < left) {
                if constexpr (sizeof(T) == 4)
                  out[v * kPer + i] = o.get(i);
                else
                  reinterpret_cast<uint16_t *>(out)[v * kPer + i] = o.h[i];
              }
          }
        }
      }
    }
  }
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
  int v_wide, x_wide;
};

constexpr int kOuterWarps = 8, kOuterSlices = 4;  // slices of columns x shares of the rows

// An adapter's sums over its rows for up to 16 MT of the rank and four slices of 8
// kLane columns: a warp has one slice and every other 16 rows of the block's, the
// cluster's blocks have stretches of the rows.
template <typename T, int MT>
__global__ void __launch_bounds__(kOuterWarps * 32) k_adapt_outer(const OuterArgs a) {
  pdl_wait();
  typedef Op<T> O;
  constexpr int NT = O::kLane, kCols = 8 * NT, kRank = 16 * MT, kPer = 2 * MT;  // ranks of a lane
  constexpr int kVp = sizeof(T) == 2 ? 2 : 3;
  extern __shared__ __align__(16) float outer_smem[];  // [kOuterSlices][kRank][kCols]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const uint32_t block = cluster_rank(), blocks = cluster_blocks();
  const int slice = warp % kOuterSlices, share = warp / kOuterSlices;
  constexpr int kShares = kOuterWarps / kOuterSlices;
  const int adapter = blockIdx.y, r0 = blockIdx.z * kRank;
  const int c0 = ((int)(blockIdx.x / blocks) * kOuterSlices + slice) * kCols;
  const int first = a.start[adapter], end = a.start[adapter + 1];
  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.f;
  const int lane_c = c0 + NT * g, left = a.cols - lane_c, lane_r = r0 + kPer * g, r_left = a.rank - lane_r;
  if (c0 < a.cols)
    for (int p0 = first + (int)(block * kShares + share) * 16; p0 < end; p0 += (int)blocks * kShares * 16) {
      Pack<T, 16> xv[4];
      Many<float, kPer> vv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // rows 4 q + i of the 16; zeros past the end
        const int p = p0 + 4 * q + i;
        const int64_t token = a.order[min(p, end - 1)];
        xv[i] = load_vec<T, NT>(reinterpret_cast<const T *>(a.x) + token * a.x_ld + lane_c, p < end ? left : 0, a.x_wide);
        vv[i].load(a.v + token * a.rank + lane_r, p < end ? r_left : 0, a.v_wide);
      }
      uint32_t w[MT][2][2][kVp];  // m tile, rows g and g + 8 of it: ranks 2 m and 2 m + 1 of the lane's
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int k = 0; k < 2; ++k) cut_pair<kVp>(vv[2 * k].get(2 * m + h), vv[2 * k + 1].get(2 * m + h), w[m][h][k]);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint32_t b[2][O::kParts];
#pragma unroll
        for (int k = 0; k < 2; ++k) across<T>(xv[2 * k], xv[2 * k + 1], j, b[k]);
#pragma unroll
        for (int m = 0; m < MT; ++m) mma_step(acc[m][j], w[m][0], w[m][1], b);
      }
    }
  float *own = outer_smem + slice * kRank * kCols;
  auto each = [&](auto f) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          f(own[(kPer * g + 2 * m + (e >> 1)) * kCols + NT * (2 * q + (e & 1)) + j], acc[m][j][e]);
  };
#pragma unroll
  for (int s = 0; s < kShares; ++s) {
    if (share == s) {
      if (s == 0)
        each([](float &t, float &v) { t = v; });
      else
        each([](float &t, float &v) { t += v; });
    }
    __syncthreads();
  }
  if (blocks > 1) cluster_sync();
  const float scale = a.scales ? a.scales[adapter] : 1.f;
  T *out = reinterpret_cast<T *>(a.out) + (int64_t)adapter * a.rank * a.cols;
  const int b0 = (int)(blockIdx.x / blocks) * kOuterSlices * kCols;
  for (int i = (int)block * kOuterWarps * 32 + threadIdx.x; i < kOuterSlices * kCols * kRank; i += (int)blocks * kOuterWarps * 32) {
    int r, c;  // of the block's
    if (a.turned) {
      r = i % kRank;
      c = i / kRank;
    } else {
      c = i % (kOuterSlices * kCols);
      r = i / (kOuterSlices * kCols);
    }
    if (r0 + r >= a.rank || b0 + c >= a.cols) continue;
    const float *at = outer_smem + (c / kCols * kRank + r) * kCols + c % kCols;
    float s;
    if (blocks > 1) {
      s = ld_cluster(at, 0);
      for (uint32_t b = 1; b < blocks; ++b) s += ld_cluster(at, b);
    } else {
      s = *at;
    }
    // an adapter without rows has no gradient, whatever its scale
    const float v = first == end ? 0.f : s * scale;
    out[a.turned ? (int64_t)(b0 + c) * a.rank + r0 + r : (int64_t)(r0 + r) * a.cols + b0 + c] = from_f32<T>(v);
  }
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
  o += align_up(((size_t)adapters + 2) * 4, kAlign);
  // every adapter's last tile, and the rows' without one, may be short
  w.tile_cap = (int)(ceil_div(n, kTile) + std::min<int64_t>(n, (int64_t)adapters + 1));
  w.tiles = o;
  o += align_up((size_t)w.tile_cap * sizeof(Tile), kAlign);
  w.h = o;
  o += align_up((size_t)n * (size_t)rank * 4, kAlign);
  w.total = o;
  return w;
}

bool row_wide(const void *p, int64_t ld, size_t es) { return ptr_aligned(p, 16) && (size_t)ld * es % 16 == 0; }

cudaError_t launch_group(const TokenSrc &which, int n, uint8_t *b, const AdaptWs &W, cudaStream_t s) {
  const int groups = (int)which.vocab + 1, warps = group_warps(groups);
  const size_t smem = (size_t)warps * groups * 4;
  cudaError_t e = raise_smem_limit(k_adapt_group, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_adapt_group, 1, kGroupThreads, smem, s, which, n, warps, reinterpret_cast<int32_t *>(b + W.order),
                    reinterpret_cast<int32_t *>(b + W.start), reinterpret_cast<Tile *>(b + W.tiles), W.tile_cap);
}

// tiles that a call is likely to have: half of the short ones
int64_t likely_tiles(int64_t n, int32_t adapters) {
  return ceil_div(n, kTile) + std::min<int64_t>(n, adapters) / 2;
}

// blocks of a cluster so that about two blocks per SM share the work, and each has some of it
unsigned cluster_for(int64_t blocks, int64_t shares, int sms) {
  unsigned c = 1;
  while (c < kMostCluster && blocks * c < 2 * (int64_t)sms && shares >= 2 * (int64_t)c) c *= 2;
  return c;
}

template <typename T, int NT, bool kAlong>
cudaError_t launch_down(const DownArgs &a, int64_t n, int tile_cap, int sms, cudaStream_t s) {
  const size_t smem = (size_t)4 * kTile * 8 * NT * 4;
  cudaError_t e = raise_smem_limit(k_adapt_down<T, NT, kAlong>, smem);
  if (e != cudaSuccess) return e;
  const unsigned slices = (unsigned)ceil_div(a.rank, 8 * NT);
  const unsigned c = cluster_for(likely_tiles(n, a.adapters) * slices, ceil_div(a.k, Op<T>::kGroup * kDownWarps), sms);
  return launch_cluster(c, k_adapt_down<T, NT, kAlong>, dim3((unsigned)tile_cap * c, slices), kDownWarps * 32, smem, s, a);
}
template <typename T, bool kAlong>
cudaError_t down(const DownArgs &a, int64_t n, int tile_cap, int sms, cudaStream_t s) {
  constexpr int kMost = sizeof(T) == 2 ? 8 : 4;
  if (a.rank <= 8) return launch_down<T, 1, kAlong>(a, n, tile_cap, sms, s);
  if (a.rank <= 16) return launch_down<T, 2, kAlong>(a, n, tile_cap, sms, s);
  if (a.rank <= 32 || kMost == 4) return launch_down<T, 4, kAlong>(a, n, tile_cap, sms, s);
  return launch_down<T, kMost, kAlong>(a, n, tile_cap, sms, s);
}

template <typename T, bool kAlong>
cudaError_t up(UpArgs a, int64_t n, int tile_cap, int sms, cudaStream_t s) {
  constexpr int kParts = sizeof(T) == 2 ? 2 : 3;
  const size_t smem = (size_t)kParts * kTile * up_ld(a.rank) * 2;
  cudaError_t e = raise_smem_limit(k_adapt_up<T, kAlong>, smem);
  if (e != cudaSuccess) return e;
  const int64_t all = ceil_div(a.cols, kUpWarps * kUpCols);
  // a block that has more columns reads its rows of h for all of them, as long as there are eight blocks per SM
  int64_t groups = std::max<int64_t>(1, likely_tiles(n, a.adapters) * all / (8 * (int64_t)sms));
  groups = std::min<int64_t>(groups, 8);
  if (ceil_div(all, groups) > 65535) groups = ceil_div(all, 65535);
  a.groups = (int)groups;
  return launch_pdl(k_adapt_up<T, kAlong>, dim3((unsigned)tile_cap, (unsigned)ceil_div(all, groups)), kUpWarps * 32, smem, s,
                    (const UpArgs)a);
}

template <typename T, int MT>
cudaError_t launch_outer(const OuterArgs &a, int64_t n, int32_t adapters, int sms, cudaStream_t s) {
  constexpr int kCols = 8 * Op<T>::kLane;
  const size_t smem = (size_t)kOuterSlices * 16 * MT * kCols * 4;
  cudaError_t e = raise_smem_limit(k_adapt_outer<T, MT>, smem);
  if (e != cudaSuccess) return e;
  const int64_t slices = ceil_div(a.cols, kOuterSlices * kCols), ranks = ceil_div(a.rank, 16 * MT);
  const unsigned c = cluster_for(slices * ranks * adapters, ceil_div(n, (int64_t)adapters * 32), sms);
  return launch_cluster(c, k_adapt_outer<T, MT>, dim3((unsigned)(slices * c), (unsigned)adapters, (unsigned)ranks), kOuterWarps * 32,
                        smem, s, a);
}
template <typename T>
cudaError_t outer(const OuterArgs &a, int64_t n, int32_t adapters, int sms, cudaStream_t s) {
  if (a.rank <= 16) return launch_outer<T, 1>(a, n, adapters, sms, s);
  if (a.rank <= 32) return launch_outer<T, 2>(a, n, adapters, sms, s);
  return launch_outer<T, 4>(a, n, adapters, sms, s);
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

template <typename T>
cudaError_t run_fwd(const DownArgs &d, const UpArgs &u, int64_t n, const AdaptWs &W, int sms, cudaStream_t s) {
  cudaError_t e = down<T, true>(d, n, W.tile_cap, sms, s);
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
  const bool in_place = base == y && base_ld == y_ld;
  if ((!in_place && overlaps(sy, sbase)) || overlaps(sh, sbase) || overlaps(sw, sbase) || overlaps(sy, sh) || overlaps(sy, sw) ||
      overlaps(sh, sw))
    return SNACK_ERR_INVALID_ARG;
  if (ws_bytes < W.total) return SNACK_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t *w = reinterpret_cast<uint8_t *>(ws);
  const int sms = sms_here();
  ADAPT_CUDA(launch_group(TokenSrc{which, which_t == SNACK_I64, (uint32_t)n_adapters}, (int)n, w, W, s));
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
  d.x_wide = row_wide(x, x_ld, es);
  d.m_wide = row_wide(a, in_f, es);
  UpArgs u = {};
  u.h = d.h;
  u.m = b;
  u.cols = out_f;
  u.rank = rank;
  u.order = d.order;
  u.tiles = d.tiles;
  u.adapters = n_adapters;
  u.scales = scales;
  u.base = base;
  u.base_ld = base_ld;
  u.out = y;
  u.out_ld = y_ld;
  u.m_wide = ptr_aligned(b, 4 * es) && rank % 4 == 0;
  u.base_wide = row_wide(base, base_ld, es);
  u.out_wide = row_wide(y, y_ld, es);
  ADAPT_CUDA(t == SNACK_F32 ? run_fwd<float>(d, u, n, W, sms, s) : run_fwd<bf16>(d, u, n, W, sms, s));
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
  ADAPT_CUDA(launch_group(TokenSrc{which, which_t == SNACK_I64, (uint32_t)n_adapters}, (int)n, w, W, s));
  const int32_t *order = reinterpret_cast<const int32_t *>(w + W.order), *start = reinterpret_cast<const int32_t *>(w + W.start);
  float *dh = reinterpret_cast<float *>(w + W.h);
  const int ranks = rank <= 8 ? 1 : rank <= 16 ? 2 : rank <= 32 || wide32 ? 4 : 8;  // a lane's of a row of b
  if (dx || da) {
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
    d.x_wide = row_wide(dy, dy_ld, es);
    d.m_wide = ptr_aligned(b, ranks * es) && rank % ranks == 0;
    ADAPT_CUDA(wide32 ? down<float, false>(d, n, W.tile_cap, sms, s) : down<bf16, false>(d, n, W.tile_cap, sms, s));
  }
  if (dx) {
    UpArgs u = {};
    u.h = dh;
    u.m = a;
    u.cols = in_f;
    u.rank = rank;
    u.order = order;
    u.tiles = reinterpret_cast<const Tile *>(w + W.tiles);
    u.adapters = n_adapters;
    u.base = accumulate ? dx : nullptr;
    u.base_ld = dx_ld;
    u.out = dx;
    u.out_ld = dx_ld;
    u.m_wide = ptr_aligned(a, 4 * es) && in_f % 4 == 0;
    u.base_wide = u.out_wide = row_wide(dx, dx_ld, es);
    ADAPT_CUDA(wide32 ? up<float, false>(u, n, W.tile_cap, sms, s) : up<bf16, false>(u, n, W.tile_cap, sms, s));
  }
  OuterArgs o = {};
  o.rank = rank;
  o.order = order;
  o.start = start;
  if (da) {
    o.v = dh;
    o.v_wide = rank % 4 == 0;
    o.x = x;
    o.x_ld = x_ld;
    o.cols = in_f;
    o.out = da;
    o.x_wide = row_wide(x, x_ld, es);
    ADAPT_CUDA(wide32 ? outer<float>(o, n, n_adapters, sms, s) : outer<bf16>(o, n, n_adapters, sms, s));
  }
  if (db) {
    o.v = h;
    o.v_wide = rank % 4 == 0 && ptr_aligned(h, 16);
    o.x = dy;
    o.x_ld = dy_ld;
    o.cols = out_f;
    o.out = db;
    o.turned = 1;
    o.scales = scales;
    o.x_wide = row_wide(dy, dy_ld, es);
    ADAPT_CUDA(wide32 ? outer<float>(o, n, n_adapters, sms, s) : outer<bf16>(o, n, n_adapters, sms, s));
  }
  return SNACK_OK;
} catch (...) {  // a host allocation failed
  return SNACK_ERR_CUDA;
}

}  // extern "C"
