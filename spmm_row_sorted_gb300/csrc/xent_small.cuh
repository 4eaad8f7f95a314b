// Cross entropy of a few fp32 tokens on the CUDA cores, reading w as it lies: the
// logits of up to 4 tokens (of more: xent_cut.cuh), and both gradients of up to
// 16.  The tensor cores of the large products would need w cut into bf16 parts
// first, 10 bytes moved per element to save arithmetic that a few tokens do not
// have; here every pass reads the 4 bytes once (bound by memory up to about 8
// tokens, by fp32 arithmetic from there on).  Loss and gradients of 3 tokens
// against 129472 x 2784: 1192 us, by way of the tensor cores 3813 (w read three
// times and dw written, 5.8 GB: 4.8 TB/s).  Included by xent.cu.
#pragma once

#include "lm.hpp"

namespace snack {
namespace {

constexpr int kSmallMostTokens = 16;  // of the gradients
constexpr int kFewMostLogits = 4;     // of k_xent_few
constexpr int kSmallWarps = 16;
constexpr int kSmallXBytes = 192 * 1024;  // of x in shared memory
constexpr int kSmallRows = 8;             // rows of w a warp works on at once: their sums stay in registers

// Whether the CUDA cores form the logits: with fewer rows than one tile per SM, warps that share
// rows are faster (xent_cut.cuh; 4 tokens, 2000 x 4096: 20 us, here 36; 119598 x 2176: 217 and 189).
inline bool few_fits(int n, int64_t vocab, int sms) {
  return n <= kFewMostLogits && vocab >= (int64_t)kSmallWarps * kSmallRows * sms;
}

// of the width in shared memory at a time
inline int small_k(int32_t width) {
  const int most = kSmallXBytes / 4 / kFewMostLogits / 128 * 128, all = (width + 127) / 128 * 128;
  return all < most ? all : most;
}

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
  int32_t chunk;  // of the width in shared memory at a time
  int x_wide, w_wide;
  TokenSrc targets;
  // loss
  float2 *part;  // [blocks][n] (maximum, sum of exp(z - maximum))
  float *zt;     // [n]
  // gradient
  const float *lse, *weight;  // weight: of each row, or null
  float *dz;                  // [vocab][kFewMostLogits]
};

// A block's warps take neighbouring groups of kSmallRows rows of w; a
// lane adds the products of every 32nd four columns for all rows and tokens (x
// from shared memory, one read for all the rows), and the lanes' sums are added
// at the end.  kGrad: dz instead of the loss's statistics.
template <bool kGrad>
__global__ void __launch_bounds__(kSmallWarps * 32, 1) k_xent_few(const SmallArgs a) {
  pdl_wait();
  constexpr int kNt = kFewMostLogits, kR = kSmallRows, kTile = kSmallWarps * kR;
  extern __shared__ __align__(16) float few_smem[];
  float *xs = few_smem;                   // [kNt][chunk]
  float *zs = few_smem + kNt * a.chunk;   // [kTile][kNt + 1]
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
    for (int k0 = 0; k0 < a.width; k0 += a.chunk) {
      if (tile == (int64_t)blockIdx.x || a.width > a.chunk) {  // a single chunk stays for all tiles
        __syncthreads();
#pragma unroll
        for (int t = 0; t < kNt; ++t)
          for (int k = threadIdx.x * 4; k < a.chunk; k += kSmallWarps * 32 * 4)
            *reinterpret_cast<float4 *>(xs + t * a.chunk + k) =
                t < a.n ? load4(a.x + t * a.x_ld + k0 + k, a.width - k0 - k, a.x_wide) : make_float4(0.f, 0.f, 0.f, 0.f);
        __syncthreads();
      }
#pragma unroll 2
      for (int k = lane * 4; k < a.chunk; k += 128) {
        const int left = a.width - k0 - k;
        if (left <= 0) break;
        float4 w[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r)
          w[r] = v0 + r < a.vocab ? load4(a.w + (v0 + r) * a.w_ld + k0 + k, left, a.w_wide) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int t = 0; t < kNt; ++t) {
          const float4 x = *reinterpret_cast<const float4 *>(xs + t * a.chunk + k);
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

// A lane holds kC columns of all tokens: their sums of dx, and x for dw.  A
// block's warps share 32 kC columns and a range of the vocabulary, whose dz lies
// in shared memory 128 rows at a time (every lane reads the same words); their
// sums of dx meet in shared memory at the end.
constexpr int kFewWarps = 8;
constexpr int kFewRows = 128;
__host__ __device__ constexpr int few_cols(int nt) { return nt <= 8 ? 4 : 2; }

template <int kC>
struct Cols {
  float v[kC];
  __device__ __forceinline__ void load(const float *p, int left, bool wide) {
    if (left >= kC && wide) {
      if constexpr (kC == 4) {
        const float4 q = __ldg(reinterpret_cast<const float4 *>(p));
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
      } else {
        const float2 q = __ldg(reinterpret_cast<const float2 *>(p));
        v[0] = q.x, v[1] = q.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kC; ++i) v[i] = i < left ? __ldg(p + i) : 0.f;
    }
  }
  __device__ __forceinline__ void store(float *p, int left, bool wide) const {
    if (left >= kC && wide) {
      if constexpr (kC == 4)
        __stcs(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
      else
        __stcs(reinterpret_cast<float2 *>(p), make_float2(v[0], v[1]));
    } else {
#pragma unroll
      for (int i = 0; i < kC; ++i)
        if (i < left) p[i] = v[i];
    }
  }
};

template <int kNt, bool kDxOut, bool kDwOut>
__global__ void __launch_bounds__(kFewWarps * 32) k_xent_few_grad(const SmallGrad a) {
  pdl_wait();
  // rows in flight per warp (8 instead of 4: 4 tokens, 119598 x 2176, 698 -> 635 us with dz; of 8 tokens it costs a
  // block per SM, 767 -> 891 us)
  constexpr int kC = few_cols(kNt), kU = kNt <= 4 ? 8 : 4;
  __shared__ __align__(16) float dzs[kFewRows * kNt];
  __shared__ float sum[kDxOut ? kFewWarps : 1][32 * kC];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = (blockIdx.x * 32 + lane) * kC, left = a.width - c;
  float acc[kDxOut ? kNt : 1][kC];
  Cols<kC> x[kDwOut ? kNt : 1];
  if (kDxOut)
#pragma unroll
    for (int t = 0; t < kNt; ++t)
#pragma unroll
      for (int i = 0; i < kC; ++i) acc[kDxOut ? t : 0][i] = 0.f;
  if (kDwOut) {
    const float f = (a.factor_a ? *a.factor_a : 1.f) * (a.factor_b ? *a.factor_b : 1.f);
#pragma unroll
    for (int t = 0; t < kNt; ++t) {
      Cols<kC> &v = x[kDwOut ? t : 0];
      // rows that are left out add nothing, whatever they and the factor hold
      const bool in = t < a.n && a.targets.key(t) < a.targets.vocab && !(a.weight && a.weight[t] == 0.f);
      v.load(a.x + (in ? t : 0) * a.x_ld + c, in ? left : 0, false);
#pragma unroll
      for (int i = 0; i < kC; ++i) v.v[i] = in ? v.v[i] * f : 0.f;
    }
  }
  const int64_t r0 = (int64_t)blockIdx.y * a.rows_per_split;
  const int64_t r1 = r0 + a.rows_per_split < a.vocab ? r0 + a.rows_per_split : a.vocab;
  for (int64_t b = r0; b < r1; b += kFewRows) {
    const int rows = (int)(r1 - b < kFewRows ? r1 - b : kFewRows);
    __syncthreads();
    for (int i = threadIdx.x * 4; i < rows * kNt; i += kFewWarps * 32 * 4)
      *reinterpret_cast<float4 *>(dzs + i) = __ldg(reinterpret_cast<const float4 *>(a.dz + b * kNt + i));
    __syncthreads();
    for (int q = warp; q < rows; q += kU * kFewWarps) {
      Cols<kC> w[kU];
      if (kDxOut)
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (q + u * kFewWarps < rows) w[u].load(a.w + (b + q + u * kFewWarps) * a.w_ld + c, left, a.w_wide);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int r = q + u * kFewWarps;
        if (r >= rows) break;
        Cols<kC> o;
#pragma unroll
        for (int i = 0; i < kC; ++i) o.v[i] = 0.f;
#pragma unroll
        for (int t4 = 0; t4 < kNt / 4; ++t4) {
          const float4 z4 = *reinterpret_cast<const float4 *>(dzs + r * kNt + 4 * t4);
          const float z[4] = {z4.x, z4.y, z4.z, z4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = 4 * t4 + e;
#pragma unroll
            for (int i = 0; i < kC; ++i) {
              if (kDxOut) acc[kDxOut ? t : 0][i] = fmaf(z[e], w[u].v[i], acc[kDxOut ? t : 0][i]);
              if (kDwOut) o.v[i] = fmaf(z[e], x[kDwOut ? t : 0].v[i], o.v[i]);
            }
          }
        }
        if (kDwOut && left > 0) o.store(a.dw + (b + r) * a.dw_ld + c, left, a.dw_wide);
      }
    }
  }
  if constexpr (kDxOut) {
#pragma unroll
    for (int t = 0; t < kNt; ++t) {
      if (t >= a.n) break;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kC; ++i) sum[warp][lane * kC + i] = acc[t][i];
      __syncthreads();
      for (int i = threadIdx.x; i < 32 * kC; i += kFewWarps * 32) {
        const int col = blockIdx.x * 32 * kC + i;
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < kFewWarps; ++q) s += sum[q][i];
        if (col < a.acc_ld) a.acc[((size_t)blockIdx.y * (size_t)a.n + t) * (size_t)a.acc_ld + col] = s;
      }
    }
  }
}

}  // namespace
}  // namespace snack
