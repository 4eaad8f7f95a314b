// Cross entropy of some fp32 tokens (up to 64): logits, of the loss and of the
// gradient's dz, on the tensor cores with w cut into bf16 parts in registers, as it
// is read.  Laying w's parts out in
// memory first (xent.cu) moves 16 bytes per weight before the product's own
// reads, which only pays where many tokens share it, and its tiles of 256 tokens
// stay mostly empty here; with mma.sync the vocabulary is the product's rows, a
// few tokens its columns, and w's fragments come straight from global memory.
// Bound by issuing instructions up to 16 tokens (the cuts: 4.3 TB/s of w), by the
// rate of mma.sync, below that of tcgen05, from there on.  Losses, us, against the
// way through memory (17 tokens and more) and the CUDA cores (below):
//   tokens x vocabulary x width    here     other
//    8 x 119598 x 2176              217       263
//   16 x 119598 x 2176              287       382
//   32 x 119598 x 2176              417       957
//   16 x 32768 x 1024                42        76
//   32 x 32768 x 1024                58       128
//   32 x 500 x 1024                  21        26
// (dz of 17 tokens and more, where w's parts have to be in memory for dx anyway, would be
// faster from them: gradients of 32 x 119598 x 2176 take 1956 us, so 1751, of 64 x 119598
// x 512 550 and 440; but then loss and dz would come from different sums.)
// Included by xent.cu.
#pragma once

#include "lm.hpp"
#include "xent_small.cuh"

namespace snack {
namespace {

constexpr int kCutWarps = 16;
constexpr int kCutXBytes = 184 * 1024;  // of x's parts in shared memory
constexpr int kCutPad = 16;             // elements: neighbouring tokens' rows start 32 bytes apart modulo 128

struct CutArgs {
  const float *x, *w;
  int64_t x_ld, w_ld;
  int32_t n, width;
  int64_t vocab;
  int32_t chunk;  // of the width in shared memory at a time: a multiple of 64
  int split;      // warps that share a row's columns
  int x_wide, w_wide;
  TokenSrc targets;
  float2 *part;  // [blocks][n] (maximum, sum of exp(z - maximum))
  float *zt;     // [n]
  // gradient
  const float *lse, *weight;  // weight: of each row, or null
  int32_t v0;                 // first vocabulary row of w here, which may be a piece of it
  float *dz;                  // [vocab][tokens built for],
  bf16 *dz_parts;             //  or its three bf16 parts [3][n][dz_ld], `plane` elements apart
  int64_t dz_ld, plane;
};

// fp32 losses that run here.  Above 32 tokens two warps read (and cut) each row of
// w, which pays for narrow rows only: 48 tokens, 4096 x 256, 18 us (20 by way of
// memory), 65536 x 128, 38 us (66); 10000 x 768, 53 us (43).
inline bool cut_fits(int n, int32_t width) { return n <= 32 || (n <= 64 && width <= 512); }
// tokens a kernel is built for
inline int cut_tokens(int n) { return n <= 8 ? 8 : n <= 16 ? 16 : n <= 32 ? 32 : 64; }
// of the width in shared memory at a time
inline int cut_chunk(int n, int32_t width) {
  const int most = (kCutXBytes / 6 / cut_tokens(n) - kCutPad) / 64 * 64, all = (width + 63) / 64 * 64;
  return all < most ? all : most;
}

// A block's 16 warps have 16 rows of w each (two of them the same ones above 32
// tokens), or `split` of them share the columns of 16 rows: a small vocabulary
// then still spreads over the SMs, and the last wave of tiles is shorter.  8
// tokens, 2000 x 4096: 21 us, whole rows 81; 119598 x 2176: 217 and 241 us.  A
// tile costs its steps of 32 columns, about five more, and where x does not stay in
// shared memory its staging (32 tokens, 20000 x 4096: whole rows 199 us, shared
// 340).
inline int cut_rows(int n, int split) { return kCutWarps / (n > 32 ? 2 : 1) / split * 16; }
inline int cut_split(int n, int64_t vocab, int32_t width, int sms) {
  const int64_t chunks = (width + cut_chunk(n, width) - 1) / cut_chunk(n, width);
  const int64_t staging = chunks > 1 ? (int64_t)cut_tokens(n) * width / 10000 + 3 * chunks : 0;
  int best = 1;
  int64_t best_cost = INT64_MAX;
  for (int s = 1; s <= kCutWarps / (n > 32 ? 2 : 1); s *= 2) {
    const int64_t tiles = (vocab + cut_rows(n, s) - 1) / cut_rows(n, s);
    const int64_t cost = (tiles + sms - 1) / sms * ((width + 31) / 32 / s + 5 + staging);
    if (cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

// Shared memory: x's parts, the block's statistics, the sums of warps that share rows.
inline size_t cut_smem_bytes(const CutArgs &a, int tiles, int across) {
  const size_t tokens = 8 * (size_t)tiles * across;
  return tokens * (size_t)(a.chunk + kCutPad) * 6 + kCutWarps / across * tokens * 8 +
         (a.split > 1 ? (size_t)kCutWarps * 4 * tiles * 32 * 4 : 0);
}
static_assert(kCutXBytes + 4096 + kCutWarps * 16 * 32 * 4 <= 232448, "shared memory of one block");

// d += a b for 16 rows of w, 16 of K and 8 tokens
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The upper halves of two words, as a pair of bf16.
__device__ __forceinline__ uint32_t upper_halves(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}
// v becomes what its leading 8 significant bits leave over (NaN of an infinity, whose logits are then NaN).
__device__ __forceinline__ void drop_top(float &v) { v -= __uint_as_float(__float_as_uint(v) & 0xFFFF0000u); }

// A block's tile is kCutWarps / kAcross / split groups of 16 rows of w; each warp
// has one, 8 kTiles of the tokens, and every split-th 32 columns.  A lane reads four columns in a row of a w row at a
// time: which columns of 16 a lane of mma.sync holds does not matter to the sum
// as long as both operands agree, so no fragment is shuffled.  x's parts (rounded,
// so that their remainders have either sign) lie in shared memory in the order of
// x; w's are cut off without rounding, three of 8 bits.  The tensor core rounds
// sums towards zero, so it only adds up 32 of K, the ten small part products
// before the two leading ones; those sums are added in fp32.  kGrad: dz instead of
// the loss's statistics, from the very same logits: a confident token's dz = p - 1
// shows what two ways of summing them differ by (17 to 64 tokens against logits of
// the large products: 1e-5 where 1 - p was 2e-3).
template <int kTiles, int kAcross, bool kGrad>
__global__ void __launch_bounds__(kCutWarps * 32, 1) k_xent_cut(const CutArgs a) {
  pdl_wait();
  constexpr int kTokens = 8 * kTiles * kAcross, kDown = kCutWarps / kAcross;
  constexpr int kDepth = kTiles <= 2 ? 2 : 1;  // steps of 32 columns read ahead
  extern __shared__ __align__(16) uint8_t cut_smem[];
  bf16 *xs = reinterpret_cast<bf16 *>(cut_smem);  // [3][kTokens][ld]
  const int ld = a.chunk + kCutPad, plane = kTokens * ld;
  float2(*red)[kTokens] = reinterpret_cast<float2(*)[kTokens]>(cut_smem + 6 * plane);               // [kDown]
  float(*part_sum)[4 * kTiles][32] = reinterpret_cast<float(*)[4 * kTiles][32]>(red + kDown);  // [kCutWarps], split
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;  // row of 8, and columns 4 q .. 4 q + 3 of 16
  const int down = warp / kAcross / a.split, part = warp / kAcross % a.split, tok0 = (warp % kAcross) * 8 * kTiles;
  const int groups = kDown / a.split, rows = 16 * groups, k_first = 32 * part, k_step = 32 * a.split;
  const int64_t tiles = (a.vocab + rows - 1) / rows;
  float run_max[kTiles][2], run_sum[kTiles][2];
#pragma unroll
  for (int j = 0; j < kTiles; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      run_max[j][e] = -INFINITY;
      run_sum[j][e] = 0.f;
    }
  struct Step {
    float4 v[2][2];  // rows g and g + 8, 16 columns twice
  };
  // the next step to read: its tile, its columns and this lane's place in its rows (the last row's, past the end)
  int64_t next_tile = k_first < a.width ? (int64_t)blockIdx.x : tiles;
  int next_k = k_first;
  const float *next_row[2];
  auto rows_of = [&] {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t r = next_tile * rows + down * 16 + 8 * h + g;
      next_row[h] = a.w + (r < a.vocab ? r : a.vocab - 1) * a.w_ld + 4 * q;
    }
  };
  auto fetch = [&](Step &s) {
    if (next_tile >= tiles) return;
    if (a.w_wide && next_k + 32 <= a.width) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 2; ++c) s.v[h][c] = __ldg(reinterpret_cast<const float4 *>(next_row[h] + next_k + 16 * c));
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          s.v[h][c] = load4(next_row[h] + next_k + 16 * c, a.width - next_k - 16 * c - 4 * q, a.w_wide);
    }
    next_k += k_step;
    if (next_k >= a.width) {
      next_k = k_first;
      next_tile += gridDim.x;
      rows_of();
    }
  };
  Step ahead[kDepth];
  rows_of();
#pragma unroll
  for (int d = 0; d < kDepth; ++d) fetch(ahead[d]);
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    float acc[kTiles][4];
#pragma unroll
    for (int j = 0; j < kTiles; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    int kc = k_first;  // this warp's columns
    for (int k0 = 0; k0 < a.width; k0 += a.chunk) {
      const int len = min(a.chunk, (a.width - k0 + 31) / 32 * 32);
      if (tile == (int64_t)blockIdx.x || a.width > a.chunk) {  // a single chunk stays for all tiles
        __syncthreads();
        for (int i = threadIdx.x; i < kTokens * (len / 4); i += kCutWarps * 32) {
          const int t = i / (len / 4), k = (i - t * (len / 4)) * 4;
          const float4 f = t < a.n ? load4(a.x + t * a.x_ld + k0 + k, a.width - k0 - k, a.x_wide) : make_float4(0.f, 0.f, 0.f, 0.f);
          float v[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
          for (int p = 0; p < 3; ++p) {
            Pack<bf16, 8> o;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float h = __bfloat162float(__float2bfloat16_rn(v[e]));
              if (isinf(h) && !isinf(v[e])) h = __uint_as_float(__float_as_uint(v[e]) & 0xFFFF0000u);  // rounded past the largest
              o.set(e, h);
              v[e] = isfinite(v[e]) ? v[e] - h : 0.f;
            }
            *reinterpret_cast<uint2 *>(xs + p * plane + t * ld + k) = o.raw;
          }
        }
        __syncthreads();
      }
      for (; kc < k0 + len; kc += k_step) {
        uint32_t wp[2][3][4];  // 16 columns, part, fragment
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4 f = ahead[0].v[h][c];
            float v[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int p = 0; p < 3; ++p) {
              if (p)
#pragma unroll
                for (int e = 0; e < 4; ++e) drop_top(v[e]);
              wp[c][p][h] = upper_halves(v[0], v[1]);
              wp[c][p][2 + h] = upper_halves(v[2], v[3]);
            }
          }
        if (kDepth == 2) ahead[0] = ahead[kDepth - 1];
        fetch(ahead[kDepth - 1]);
        const bf16 *at = xs + (tok0 + g) * ld + (kc - k0) + 4 * q;
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
          uint2 xp[2][3];
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int p = 0; p < 3; ++p) xp[c][p] = *reinterpret_cast<const uint2 *>(at + p * plane + 8 * j * ld + 16 * c);
          float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            mma16816(d, wp[c][2], xp[c][0].x, xp[c][0].y);
            mma16816(d, wp[c][1], xp[c][1].x, xp[c][1].y);
            mma16816(d, wp[c][0], xp[c][2].x, xp[c][2].y);
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            mma16816(d, wp[c][1], xp[c][0].x, xp[c][0].y);
            mma16816(d, wp[c][0], xp[c][1].x, xp[c][1].y);
          }
          mma16816(d, wp[0][0], xp[0][0].x, xp[0][0].y);
          mma16816(d, wp[1][0], xp[1][0].x, xp[1][0].y);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[j][i] += d[i];
        }
      }
    }
    if (a.split > 1) {  // the first of a group's warps adds the others' sums in order
      if (part) {
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) part_sum[warp][4 * j + i][lane] = acc[j][i];
      }
      __syncthreads();
      if (part == 0)
        for (int p = 1; p < a.split; ++p)
#pragma unroll
          for (int j = 0; j < kTiles; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][i] += part_sum[warp + kAcross * p][4 * j + i][lane];
      __syncthreads();
      if (part) continue;
    }
    const int64_t r0 = tile * rows + down * 16 + g;
#pragma unroll
    for (int j = 0; j < kTiles; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = tok0 + 8 * j + 2 * q + e;
        const uint32_t id = t < a.n ? a.targets.key(t) : a.targets.vocab;
        if (kGrad) {
          const float u = id < a.targets.vocab ? (a.weight ? a.weight[t] : 1.f) : 0.f;
          const float lse = u != 0.f ? a.lse[t] : 0.f;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int64_t r = r0 + 8 * h;
            if (r >= a.vocab) continue;
            const float p = expf(acc[j][2 * h + e] - lse);
            float d = u != 0.f ? u * ((int64_t)id == a.v0 + r ? p - 1.f : p) : 0.f;
            if (!a.dz_parts) {
              a.dz[r * kTokens + t] = d;
            } else if (t < a.n) {
#pragma unroll
              for (int k = 0; k < 3; ++k) {
                const bf16 part = __float2bfloat16_rn(d);
                a.dz_parts[k * a.plane + t * a.dz_ld + r] = part;
                d -= __bfloat162float(part);
              }
            }
          }
          continue;
        }
        if (t >= a.n) continue;
        float z[2], top = run_max[j][e];
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // rows g and g + 8
          const int64_t r = r0 + 8 * h;
          z[h] = r < a.vocab ? acc[j][2 * h + e] : -INFINITY;
          top = fmaxf(top, z[h]);
          if (r < a.vocab && (int64_t)id == r) a.zt[t] = z[h];
        }
        const float base = top == -INFINITY ? 0.f : top;
        run_sum[j][e] = run_sum[j][e] * expf(run_max[j][e] - base) + (expf(z[0] - base) + expf(z[1] - base));
        run_max[j][e] = top;
      }
  }
  if (kGrad) return;
  auto join = [](float &m, float &s, float m2, float s2) {
    const float top = fmaxf(m, m2), base = top == -INFINITY ? 0.f : top;
    s = s * expf(m - base) + s2 * expf(m2 - base);
    m = top;
  };
#pragma unroll
  for (int j = 0; j < kTiles; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int d = 4; d < 32; d *= 2)
        join(run_max[j][e], run_sum[j][e], __shfl_xor_sync(0xffffffffu, run_max[j][e], d),
             __shfl_xor_sync(0xffffffffu, run_sum[j][e], d));
      if (g == 0 && part == 0) red[down][tok0 + 8 * j + 2 * q + e] = make_float2(run_max[j][e], run_sum[j][e]);
    }
  __syncthreads();
  if ((int)threadIdx.x < kTokens && (int)threadIdx.x < a.n) {
    float2 p = red[0][threadIdx.x];
    for (int w = 1; w < groups; ++w) join(p.x, p.y, red[w][threadIdx.x].x, red[w][threadIdx.x].y);
    a.part[(size_t)blockIdx.x * (size_t)a.n + threadIdx.x] = p;
  }
}

}  // namespace
}  // namespace snack
