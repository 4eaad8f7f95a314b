// Cross entropy of a few fp32 tokens: the logits and both gradients on the CUDA
// cores, reading w as it lies.  The tensor cores would need w cut into bf16
// parts first, 10 bytes moved per element to save arithmetic that a few tokens
// do not have; here every pass reads the 4 bytes once (bound by memory up to
// about 16 tokens, by fp32 arithmetic from there on).  Included by xent.cu.
#pragma once

#include "lm.hpp"

namespace snack {
namespace {

constexpr int kSmallMostTokens = 32;
constexpr int kSmallWarps = 8;
constexpr int kSmallK = 512;  // of the width in shared memory at a time

// tokens a kernel is built for, and the rows of w a warp works on at once: their
// sums stay in registers
__host__ __device__ constexpr int small_rows(int nt) { return nt <= 8 ? 8 : 4; }

// Four consecutive elements; zeros from `left` on.  `wide`: 16-byte aligned rows.
__device__ __forceinline__ float4 load4(const float *p, int left, bool wide) {
  if (left >= 4 && wide) return __ldg(reinterpret_cast<const float4 *>(p));
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (left > 0) v.x = __ldg(p);
  if (left > 1) v.y = __ldg(p + 1);
  if (left > 2) v.z = __ldg(p + 2);
  if (left > 3) v.w = __ldg(p + 3);
  return v;
}

struct SmallArgs {
  const float *x, *w;
  int64_t x_ld, w_ld;
  int32_t n, width;
  int64_t vocab;
  int w_wide;
  TokenSrc targets;
  // loss
  float2 *part;  // [blocks][n] (maximum, sum of exp(z - maximum))
  float *zt;     // [n]
  // gradient
  const float *lse, *weight;  // weight: of each row, or null
  float *dz;                  // [vocab][tokens built for]
};

// A block's warps take neighbouring groups of small_rows(kNt) rows of w; a
// lane adds the products of every 32nd four columns for all rows and tokens (x
// from shared memory, one read for all the rows), and the lanes' sums are added
// at the end.  kGrad: dz instead of the loss's statistics.
template <int kNt, bool kGrad>
__global__ void __launch_bounds__(kSmallWarps * 32) k_xent_few(const SmallArgs a) {
  pdl_wait();
  constexpr int kR = small_rows(kNt), kTile = kSmallWarps * kR;
  extern __shared__ __align__(16) float few_smem[];
  float *xs = few_smem;                   // [kNt][kSmallK]
  float *zs = few_smem + kNt * kSmallK;   // [kTile][kNt + 1]
  __shared__ float run_max[kNt], run_sum[kNt];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x < kNt) {
    run_max[threadIdx.x] = -INFINITY;
    run_sum[threadIdx.x] = 0.f;
  }
  const int64_t tiles = (a.vocab + kTile - 1) / kTile;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t v0 = tile * kTile + warp * kR;
    float acc[kR][kNt];
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
      for (int t = 0; t < kNt; ++t) acc[r][t] = 0.f;
    for (int k0 = 0; k0 < a.width; k0 += kSmallK) {
      if (k0 > 0 || tile == (int64_t)blockIdx.x || a.width > kSmallK) {  // one chunk stays for all tiles
        __syncthreads();
        for (int i = threadIdx.x * 4; i < kNt * kSmallK; i += kSmallWarps * 32 * 4) {
          const int t = i / kSmallK, k = i % kSmallK;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (t < a.n) v = load4(a.x + t * a.x_ld + k0 + k, a.width - k0 - k, false);
          *reinterpret_cast<float4 *>(xs + i) = v;
        }
        __syncthreads();
      }
#pragma unroll 2
      for (int k = lane * 4; k < kSmallK; k += 128) {
        const int left = a.width - k0 - k;
        if (left <= 0) break;
        float4 w[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r)
          w[r] = v0 + r < a.vocab ? load4(a.w + (v0 + r) * a.w_ld + k0 + k, left, a.w_wide) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int t = 0; t < kNt; ++t) {
          const float4 x = *reinterpret_cast<const float4 *>(xs + t * kSmallK + k);
#pragma unroll
          for (int r = 0; r < kR; ++r)
            acc[r][t] = fmaf(w[r].x, x.x, fmaf(w[r].y, x.y, fmaf(w[r].z, x.z, fmaf(w[r].w, x.w, acc[r][t]))));
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
      for (int t = 0; t < kNt; ++t) {
        float s = acc[r][t];
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        if (lane == ((r * kNt + t) & 31)) zs[(warp * kR + r) * (kNt + 1) + t] = s;
      }
    __syncthreads();
    const int rows = (int)(a.vocab - tile * kTile < kTile ? a.vocab - tile * kTile : kTile);
    if (kGrad) {
      for (int i = threadIdx.x; i < rows * kNt; i += kSmallWarps * 32) {
        const int r = i / kNt, t = i % kNt;
        float d = 0.f;
        if (t < a.n) {
          const uint32_t id = a.targets.key(t);
          const float g = id < a.targets.vocab ? (a.weight ? a.weight[t] : 1.f) : 0.f;
          if (g != 0.f) {
            const float p = expf(zs[r * (kNt + 1) + t] - a.lse[t]);
            d = g * ((int64_t)id == tile * kTile + r ? p - 1.f : p);
          }
        }
        a.dz[tile * kTile * kNt + i] = d;
      }
    } else {
      for (int t = warp; t < a.n; t += kSmallWarps) {  // a warp per token
        float m = -INFINITY;
        for (int r = lane; r < rows; r += 32) m = fmaxf(m, zs[r * (kNt + 1) + t]);
#pragma unroll
        for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float old = run_max[t], nm = fmaxf(m, old), base = nm == -INFINITY ? 0.f : nm;
        float s = 0.f;
        for (int r = lane; r < rows; r += 32) s += expf(zs[r * (kNt + 1) + t] - base);
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        __syncwarp();
        if (lane == 0) {
          run_sum[t] = run_sum[t] * expf(old - base) + s;
          run_max[t] = nm;
          const uint32_t id = a.targets.key(t);
          if (id < a.targets.vocab && (int64_t)id >= tile * kTile && (int64_t)id < tile * kTile + rows)
            a.zt[t] = zs[((int64_t)id - tile * kTile) * (kNt + 1) + t];
        }
        __syncwarp();
      }
    }
    __syncthreads();
  }
  if (!kGrad && threadIdx.x < kNt && (int)threadIdx.x < a.n)
    a.part[(size_t)blockIdx.x * (size_t)a.n + threadIdx.x] = make_float2(run_max[threadIdx.x], run_sum[threadIdx.x]);
}

struct SmallGrad {
  const float *x, *w, *dz;
  int64_t x_ld, w_ld, dw_ld;
  int32_t n, width;
  int64_t vocab, rows_per_split;
  int w_wide, dw_wide;
  TokenSrc targets;
  const float *weight;
  const float *factor_a, *factor_b;  // common factor of dw: their product (null: 1)
  float *acc;                        // [splits][n][acc_ld] sums of dx
  int32_t acc_ld;
  float *dw;
};

// 128 columns per block; its warps take every 8th row of a range of the
// vocabulary.  A lane holds four columns of all tokens: their sums of dx, and x
// for dw.  The warps' sums of dx meet in shared memory.
template <int kNt, bool kDxOut, bool kDwOut>
__global__ void __launch_bounds__(kSmallWarps * 32) k_xent_few_grad(const SmallGrad a) {
  pdl_wait();
  __shared__ float4 sum[kDxOut ? kSmallWarps : 1][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 128 + lane * 4, left = a.width - c;
  float4 acc[kDxOut ? kNt : 1], x[kDwOut ? kNt : 1];
  if (kDxOut)
#pragma unroll
    for (int t = 0; t < kNt; ++t) acc[kDxOut ? t : 0] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (kDwOut) {
    const float f = (a.factor_a ? *a.factor_a : 1.f) * (a.factor_b ? *a.factor_b : 1.f);
#pragma unroll
    for (int t = 0; t < kNt; ++t) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      // rows that are left out add nothing, whatever they hold
      if (t < a.n && a.targets.key(t) < a.targets.vocab && !(a.weight && a.weight[t] == 0.f))
        v = load4(a.x + t * a.x_ld + c, left, false);
      x[kDwOut ? t : 0] = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
    }
  }
  const int64_t r0 = (int64_t)blockIdx.y * a.rows_per_split;
  const int64_t r1 = r0 + a.rows_per_split < a.vocab ? r0 + a.rows_per_split : a.vocab;
  constexpr int kU = kNt <= 8 ? 4 : 2;  // rows in flight
  for (int64_t v0 = r0 + warp; v0 < r1; v0 += kU * kSmallWarps) {
    float4 w[kU];
    float4 d[kU][kNt / 4];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t v = v0 + u * kSmallWarps;
      if (kDxOut) w[u] = v < r1 ? load4(a.w + v * a.w_ld + c, left, a.w_wide) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < kNt / 4; ++q)
        d[u][q] = v < r1 ? __ldg(reinterpret_cast<const float4 *>(a.dz + v * kNt) + q) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t v = v0 + u * kSmallWarps;
      if (v >= r1) break;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int t = 0; t < kNt; ++t) {
        const float4 q = d[u][t / 4];
        const float z = (t & 3) == 0 ? q.x : (t & 3) == 1 ? q.y : (t & 3) == 2 ? q.z : q.w;
        if (kDxOut) {
          float4 &s = acc[kDxOut ? t : 0];
          s.x = fmaf(z, w[u].x, s.x);
          s.y = fmaf(z, w[u].y, s.y);
          s.z = fmaf(z, w[u].z, s.z);
          s.w = fmaf(z, w[u].w, s.w);
        }
        if (kDwOut) {
          const float4 b = x[kDwOut ? t : 0];
          o.x = fmaf(z, b.x, o.x);
          o.y = fmaf(z, b.y, o.y);
          o.z = fmaf(z, b.z, o.z);
          o.w = fmaf(z, b.w, o.w);
        }
      }
      if (kDwOut) {
        float *to = a.dw + v * a.dw_ld + c;
        if (left >= 4 && a.dw_wide) {
          __stcs(reinterpret_cast<float4 *>(to), o);
        } else {
          if (left > 0) to[0] = o.x;
          if (left > 1) to[1] = o.y;
          if (left > 2) to[2] = o.z;
          if (left > 3) to[3] = o.w;
        }
      }
    }
  }
  if constexpr (kDxOut) {
#pragma unroll
    for (int t = 0; t < kNt; ++t) {
      if (t >= a.n) break;
      sum[warp][lane] = acc[t];
      __syncthreads();
      if (warp == 0 && left > 0) {
        float4 s = sum[0][lane];
#pragma unroll
        for (int q = 1; q < kSmallWarps; ++q) {
          const float4 b = sum[q][lane];
          s.x += b.x;
          s.y += b.y;
          s.z += b.z;
          s.w += b.w;
        }
        // acc_ld is a multiple of four: columns past the width are its own
        *reinterpret_cast<float4 *>(a.acc + ((size_t)blockIdx.y * (size_t)a.n + t) * (size_t)a.acc_ld + c) = s;
      }
      __syncthreads();
    }
  }
}

}  // namespace
}  // namespace snack
