// Global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum g^2),   out = g * min(1, max_norm / (norm + 1e-6))
//
// Bound by memory: the norm has to be known before the first output, so the
// gradients are read twice and written once; the second pass walks the pieces
// from the last to the first, so that what the first pass read last is still
// in L2.  The tensors' addresses travel as kernel arguments (no table is laid
// out on the device).  The work is cut into pieces of kPiece bytes of one
// tensor, and a block finds a piece's tensor by a search in the pieces' prefix.
//
// Up to 65,536 elements in at most 16 tensors, one cluster of blocks does both
// passes in one launch, its elements in registers.
//
// Each thread adds its squares in fp32, in three levels (an access's batch, a
// piece, all its pieces): over 1e9 elements that is some 120 roundings in a row,
// not 4,500, which all err to one side where the elements are alike.  Blocks leave their sums in the
// workspace and one block adds them in order, in fp64, so no atomics are needed
// and results repeat.  Squares are summed at
// three scales (g, 2^-80 g and 2^100 g), which costs arithmetic that hides
// behind the loads: the plain sum is used unless it left fp32's range.
#include <stdint.h>

#include <algorithm>
#include <vector>

#include "internal.hpp"
#include "lm.hpp"

namespace snack {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kPiece = 64 * 1024;  // bytes of one tensor per piece of the norm
// and of the scaling (norm and scaling of 1e9 bf16 elements: 860 us, three passes
// at 7.0 TB/s): 64 KB where all of it is in place, and may have nothing to
// do (2 GB of fp32 with the factor 1: 286 us of norm, and 55 us of blocks that
// return at once at 16 KB each; where it has to be scaled, 2 GB of bf16 in place, 64 KB
// take 871 us and 16 KB 860)
constexpr int64_t kScalePiece = 16 * 1024, kScalePieceInPlace = 64 * 1024;
constexpr int kBlocksPerSm = 6;
constexpr float kDown = 8.271806125530277e-25f;   // 2^-80
constexpr float kUp = 1.2676506002282294e30f;     // 2^100
constexpr float kTiny = 7.888609052210118e-31f;   // 2^-100

// A launch's tensors, in kernel arguments: at most kMost of them.
template <int kMost>
struct ClipTable {
  const void *in[kMost];
  void *out[kMost];
  int64_t n[kMost];          // elements; bf16 tensors as -n - 1
  uint32_t first[kMost + 1];  // pieces before the tensor
  int count;
};
constexpr int kSmallTable = 16, kMidTable = 128, kBigTable = 768;
static_assert(sizeof(ClipTable<kBigTable>) < 32000, "kernel arguments hold 32764 bytes");

struct Sum3 {
  float mid, low, high;  // sums of g^2, (2^-80 g)^2, (2^100 g)^2
};

__device__ __forceinline__ void add_square(Sum3 &s, float v) {
  s.mid = fmaf(v, v, s.mid);
  const float a = v * kDown, b = v * kUp;
  s.low = fmaf(a, a, s.low);
  s.high = fmaf(b, b, s.high);
}

__device__ __forceinline__ void add_sum(Sum3 &s, const Sum3 &p) {
  s.mid += p.mid;
  s.low += p.low;
  s.high += p.high;
}

// A load that is issued where it stands: the batches below keep several in flight.
__device__ __forceinline__ uint4 load16(const uint4 *p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

template <int kMost>
__device__ __forceinline__ int find_tensor(const ClipTable<kMost> &t, uint32_t piece) {
  int lo = 0, hi = t.count;  // first[lo] <= piece < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= piece)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <typename T>
__device__ __forceinline__ void sum_piece(const T *__restrict__ p, int64_t m, Sum3 &s) {
  constexpr int kN = 16 / (int)sizeof(T);
  typedef Pack<T, 16> V;
  // elements before the first 16-byte boundary, 16-byte accesses, and the rest
  int64_t lead = (int64_t)((16 - ((uintptr_t)p & 15)) & 15) / (int64_t)sizeof(T);
  if (lead > m) lead = m;
  const int64_t vecs = (m - lead) / kN;
  const uint4 *v = reinterpret_cast<const uint4 *>(p + lead);
  int64_t i = threadIdx.x;
  for (; i + 3 * kThreads < vecs; i += 4 * kThreads) {
    V a[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) a[u].raw = load16(v + i + u * kThreads);
    Sum3 q = {0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int e = 0; e < kN; ++e) add_square(q, a[u].get(e));
    add_sum(s, q);
  }
  for (; i < vecs; i += kThreads) {
    V a;
    a.raw = __ldg(v + i);
#pragma unroll
    for (int e = 0; e < kN; ++e) add_square(s, a.get(e));
  }
  for (int64_t j = threadIdx.x; j < lead; j += kThreads) add_square(s, to_f32(p[j]));
  for (int64_t j = lead + vecs * kN + threadIdx.x; j < m; j += kThreads) add_square(s, to_f32(p[j]));
}

__device__ __forceinline__ Sum3 block_sum(Sum3 s) {
  __shared__ Sum3 part[kThreads / 32];
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    s.mid += __shfl_xor_sync(0xffffffffu, s.mid, d);
    s.low += __shfl_xor_sync(0xffffffffu, s.low, d);
    s.high += __shfl_xor_sync(0xffffffffu, s.high, d);
  }
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  Sum3 t = {0.f, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    t.mid += part[w].mid;
    t.low += part[w].low;
    t.high += part[w].high;
  }
  return t;
}

// sums[base + block] = this block's share of the launch's pieces
template <int kMost>
__global__ void __launch_bounds__(kThreads) k_clip_norm(const __grid_constant__ ClipTable<kMost> t, uint32_t pieces,
                                                        Sum3 *__restrict__ sums) {
  pdl_wait();
  Sum3 s = {0.f, 0.f, 0.f};
  for (uint32_t q = blockIdx.x; q < pieces; q += gridDim.x) {
    const int k = find_tensor(t, q);
    const int64_t at = (int64_t)(q - t.first[k]) * kPiece;
    const int64_t n = t.n[k];
    Sum3 piece = {0.f, 0.f, 0.f};
    if (n >= 0) {
      const int64_t e = at / 4;
      sum_piece(reinterpret_cast<const float *>(t.in[k]) + e, min(kPiece / 4, n - e), piece);
    } else {
      const int64_t e = at / 2;
      sum_piece(reinterpret_cast<const bf16 *>(t.in[k]) + e, min(kPiece / 2, -n - 1 - e), piece);
    }
    add_sum(s, piece);
  }
  const Sum3 b = block_sum(s);
  if (threadIdx.x == 0) sums[blockIdx.x] = b;
}

// The norm from all blocks' sums: one warp adds them in fp64 (which is slow
// here), the scaled sums only where they are needed.
__device__ __forceinline__ double warp_total(const float *p, int n_sums) {
  double m = 0;
  for (int i = threadIdx.x; i < n_sums; i += 32) m += (double)__ldg(p + 3 * i);
#pragma unroll
  for (int d = 16; d; d >>= 1) m += __shfl_xor_sync(0xffffffffu, m, d);
  return m;
}
__device__ __forceinline__ float root(double sum, float back) {
  // sqrt in fp32 of a value scaled into its range by an even power of two
  int e;
  double f = frexp(sum, &e);
  if (e & 1) {
    f *= 2.0;
    e -= 1;
  }
  return ldexpf(sqrtf((float)f), e / 2) * back;
}
__device__ __forceinline__ float norm_of(double mid, double low, double high) {
  if (isnan(mid)) return (float)mid;
  if (isinf(mid)) return isinf(low) ? INFINITY : root(low, 1.f / kDown);
  if (mid < (double)kTiny) return high > 0 ? root(high, 1.f / kUp) : 0.f;
  return root(mid, 1.f);
}
__device__ __forceinline__ float total_norm(const Sum3 *__restrict__ sums, int n_sums) {
  __shared__ float result;
  if (threadIdx.x < 32) {
    const float *p = reinterpret_cast<const float *>(sums);
    const double mid = warp_total(p, n_sums);
    double low = 0, high = 0;
    if (isinf(mid)) low = warp_total(p + 1, n_sums);
    if (mid < (double)kTiny) high = warp_total(p + 2, n_sums);
    if (threadIdx.x == 0) result = norm_of(mid, low, high);
  }
  __syncthreads();
  return result;
}

// Elements of an output before its first 16-byte boundary; its pieces start there.
__host__ __device__ inline int64_t lead_of(const void *out, int64_t n, int64_t es) {
  const int64_t lead = (int64_t)((16 - ((uintptr_t)out & 15)) & 15) / es;
  return lead < n ? lead : n;
}

// Piece `r` of out[0 .. n) = in[0 .. n) * f.  Both sides move in 16-byte accesses
// also where they lie at different offsets from a boundary: the elements of an
// aligned 16 bytes of `out` then lie in two neighbouring aligned 16 bytes of
// `in`, the second of which is the next lane's first (so it comes from L1), and
// a funnel shift by the offset, the same for the whole tensor, joins them.
template <typename T>
__device__ __forceinline__ void scale_piece(const T *in, T *out, int64_t n, int64_t r, int64_t bytes, float f) {
  constexpr int kN = 16 / (int)sizeof(T);
  constexpr int kU = 4;
  typedef Pack<T, 16> V;
  const int64_t lead = lead_of(out, n, sizeof(T)), per = bytes / (int64_t)sizeof(T);
  int64_t b = lead + r * per;
  const int64_t end = min(n, b + per);
  int64_t vecs = (end - b) / kN;
  const uint32_t off = (uint32_t)((uintptr_t)(in + b) & 15);  // bytes that the elements lie past a boundary
  // elements outside the accesses: before the first boundary, and at the ends of a shifted tensor, whose
  // aligned neighbours would lie outside it
  int64_t head = r == 0 ? 0 : b;
  if (off && (uintptr_t)(in + b) - off < (uintptr_t)in && vecs > 0) {
    b += kN;
    --vecs;
  }
  if (off && vecs > 0 && (uintptr_t)(in + b) - off + 16 * (uintptr_t)(vecs + 1) > (uintptr_t)(in + n)) --vecs;
  const uint4 *v = reinterpret_cast<const uint4 *>((uintptr_t)(in + b) - off);
  uint4 *w = reinterpret_cast<uint4 *>(out + b);
  const int words = (int)(off >> 2);
  const bool half = (off & 2) != 0;
  for (int64_t i = threadIdx.x; i < vecs; i += kU * kThreads) {
    uint4 x[kU], y[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (i + u * kThreads < vecs) {
        x[u] = load16(v + i + u * kThreads);
        if (off) y[u] = load16(v + i + u * kThreads + 1);
      }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (i + u * kThreads >= vecs) continue;
      V a;
      a.raw = x[u];
      if (off) {
        uint32_t t[8] = {x[u].x, x[u].y, x[u].z, x[u].w, y[u].x, y[u].y, y[u].z, y[u].w};
        if (words & 2) {
#pragma unroll
          for (int k = 0; k < 6; ++k) t[k] = t[k + 2];
        }
        if (words & 1) {
#pragma unroll
          for (int k = 0; k < 5; ++k) t[k] = t[k + 1];
        }
        if (half) {
#pragma unroll
          for (int k = 0; k < 4; ++k) t[k] = __funnelshift_r(t[k], t[k + 1], 16);
        }
        a.raw = make_uint4(t[0], t[1], t[2], t[3]);
      }
#pragma unroll
      for (int e = 0; e < kN; ++e) a.set(e, a.get(e) * f);
      w[i + u * kThreads] = a.raw;
    }
  }
  for (int64_t j = head + threadIdx.x; j < b; j += kThreads) out[j] = from_f32<T>(to_f32(in[j]) * f);
  for (int64_t j = b + vecs * kN + threadIdx.x; j < end; j += kThreads) out[j] = from_f32<T>(to_f32(in[j]) * f);
}

// the norm, and the factor beside it, for the scaling's blocks
__global__ void __launch_bounds__(kThreads) k_clip_total(const Sum3 *__restrict__ sums, int n_sums, float max_norm,
                                                         float *norm, float *factor) {
  pdl_wait();
  const float nrm = total_norm(sums, n_sums);
  if (threadIdx.x) return;
  if (norm) *norm = nrm;
  const float f = max_norm / (nrm + 1e-6f);
  *factor = f > 1.f ? 1.f : f;  // a NaN stays
}

// One block per piece, from the last piece to the first.  (Blocks that loop over
// pieces moved 6.3 TB/s here where one block per 16 KB moves 7.1.)
template <int kMost>
__global__ void __launch_bounds__(kThreads) k_clip_scale(const __grid_constant__ ClipTable<kMost> t, uint32_t pieces, int64_t bytes,
                                                         const float *__restrict__ factor) {
  pdl_wait();
  const uint32_t r = pieces - 1 - blockIdx.x;
  const float f = *factor;
  const int k = find_tensor(t, r);
  if (f == 1.f && t.out[k] == t.in[k]) return;
  const int64_t n = t.n[k];
  if (n >= 0)
    scale_piece(reinterpret_cast<const float *>(t.in[k]), reinterpret_cast<float *>(t.out[k]), n, r - t.first[k], bytes, f);
  else
    scale_piece(reinterpret_cast<const bf16 *>(t.in[k]), reinterpret_cast<bf16 *>(t.out[k]), -n - 1, r - t.first[k], bytes, f);
}

// A few small tensors: one cluster of kCluster blocks does it all in one
// launch.  Its threads keep their elements in registers between the norm and
// the scaling; the blocks' sums meet in every block's shared memory.  Bound by its
// latencies: 7.4 us for 51,026 elements in four tensors, launch included.
constexpr int kCluster = 8;
constexpr int kClusterThreads = 1024;
constexpr int kKeep = 8;  // elements per thread
constexpr int64_t kSmallMost = (int64_t)kCluster * kClusterThreads * kKeep;

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kClusterThreads)
    k_clip_small(const __grid_constant__ ClipTable<kSmallTable> t, int scale, float max_norm, float *norm) {
  pdl_wait();
  __shared__ Sum3 part[kClusterThreads / 32];
  __shared__ Sum3 all[kCluster];  // every block's sum
  __shared__ float result;
  uint32_t rank;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this block runs: its shared memory is there
  // first[k]: elements before tensor k
  const uint32_t total = t.first[t.count];
  const uint32_t i0 = rank * kClusterThreads + threadIdx.x;
  float v[kKeep];
  int owner[kKeep];
  Sum3 s = {0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < kKeep; ++j) {
    const uint32_t i = i0 + (uint32_t)j * (kCluster * kClusterThreads);
    v[j] = 0.f;
    owner[j] = 0;
    if (i < total) {
      int k = 0;
      while (k + 1 < t.count && t.first[k + 1] <= i) ++k;
      owner[j] = k;
      const uint32_t e = i - t.first[k];
      v[j] = t.n[k] >= 0 ? reinterpret_cast<const float *>(t.in[k])[e] : to_f32(reinterpret_cast<const bf16 *>(t.in[k])[e]);
    }
  }
#pragma unroll
  for (int j = 0; j < kKeep; ++j) add_square(s, v[j]);
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    s.mid += __shfl_xor_sync(0xffffffffu, s.mid, d);
    s.low += __shfl_xor_sync(0xffffffffu, s.low, d);
    s.high += __shfl_xor_sync(0xffffffffu, s.high, d);
  }
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (threadIdx.x < 32) {
    s = part[threadIdx.x];
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      s.mid += __shfl_xor_sync(0xffffffffu, s.mid, d);
      s.low += __shfl_xor_sync(0xffffffffu, s.low, d);
      s.high += __shfl_xor_sync(0xffffffffu, s.high, d);
    }
    if (threadIdx.x < kCluster) {  // into every block's copy of `all`, at this block's place
      uint32_t to;
      asm("mapa.shared::cluster.u32 %0, %1, %2;"
          : "=r"(to)
          : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(&all[rank]))), "r"(threadIdx.x));
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(s.mid) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4), "f"(s.low) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 8), "f"(s.high) : "memory");
    }
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (threadIdx.x == 0) {
    double m = 0, l = 0, h = 0;
    for (int b = 0; b < kCluster; ++b) {
      m += (double)all[b].mid;
      l += (double)all[b].low;
      h += (double)all[b].high;
    }
    result = norm_of(m, l, h);
    if (norm && rank == 0) *norm = result;
  }
  __syncthreads();
  if (!scale) return;
  float f = max_norm / (result + 1e-6f);
  if (f > 1.f) f = 1.f;
#pragma unroll
  for (int j = 0; j < kKeep; ++j) {
    const uint32_t i = i0 + (uint32_t)j * (kCluster * kClusterThreads);
    if (i >= total) continue;
    const int k = owner[j];
    if (f == 1.f && t.out[k] == t.in[k]) continue;
    const uint32_t e = i - t.first[k];
    if (t.n[k] >= 0)
      reinterpret_cast<float *>(t.out[k])[e] = v[j] * f;
    else
      reinterpret_cast<bf16 *>(t.out[k])[e] = from_f32<bf16>(v[j] * f);
  }
}

inline int64_t pieces_of(int64_t n, snack_dtype t) { return ceil_div(n * (int64_t)dtype_size(t), kPiece); }
inline int64_t scale_pieces_of(const void *out, int64_t n, snack_dtype t, int64_t bytes) {
  const int64_t es = (int64_t)dtype_size(t), p = ceil_div((n - lead_of(out, n, es)) * es, bytes);
  return p > 0 ? p : 1;
}

struct ClipCall {
  int32_t n;
  const void *const *grads;
  void *const *outs;
  const int64_t *numel;
  const snack_dtype *types;
  float max_norm;
  float *norm;
  Sum3 *sums;
  float *factor;
  int sms;
};

int64_t groups_of(int32_t n, int most) { return ceil_div((int64_t)n, (int64_t)most); }
int table_for(int32_t n) { return n <= kSmallTable ? kSmallTable : n <= kMidTable ? kMidTable : kBigTable; }

template <int kMost>
snack_status run_clip(const ClipCall &c, cudaStream_t s) {
  if (kMost == kSmallTable) {  // few enough to stay in one cluster's registers
    int64_t total = 0;
    for (int32_t k = 0; k < c.n && total <= kSmallMost; ++k) total += c.numel[k];
    if (total <= kSmallMost) {
      ClipTable<kSmallTable> t;
      t.count = 0;
      uint32_t at = 0;
      for (int32_t k = 0; k < c.n; ++k) {
        if (c.numel[k] == 0) continue;
        t.in[t.count] = c.grads[k];
        t.out[t.count] = c.outs ? c.outs[k] : nullptr;
        t.n[t.count] = c.types[k] == SNACK_F32 ? c.numel[k] : -c.numel[k] - 1;
        t.first[t.count++] = at;
        at += (uint32_t)c.numel[k];
      }
      t.first[t.count] = at;
      return launch_pdl(k_clip_small, kCluster, kClusterThreads, 0, s, t, c.outs ? 1 : 0, c.max_norm, c.norm) ==
                     cudaSuccess
                 ? SNACK_OK
                 : SNACK_ERR_CUDA;
    }
  }
  const int64_t groups = c.n > 0 ? groups_of(c.n, kMost) : 1;
  const int most_blocks = c.sms * kBlocksPerSm;
  bool in_place = c.outs != nullptr;
  for (int32_t k = 0; k < c.n && in_place; ++k) in_place = c.outs[k] == c.grads[k];
  const int64_t bytes = in_place ? kScalePieceInPlace : kScalePiece;
  int n_sums = 0;
  for (int pass = 0; pass < (c.outs ? 2 : 1); ++pass)
    for (int64_t g0 = 0; g0 < groups; ++g0) {
      const int64_t g = pass == 0 ? g0 : groups - 1 - g0;
      ClipTable<kMost> t;
      t.count = 0;
      int64_t pieces = 0;
      for (int64_t k = g * kMost; k < c.n && k < (g + 1) * kMost; ++k) {
        if (c.numel[k] == 0) continue;
        t.in[t.count] = c.grads[k];
        t.out[t.count] = c.outs ? c.outs[k] : nullptr;
        t.n[t.count] = c.types[k] == SNACK_F32 ? c.numel[k] : -c.numel[k] - 1;
        t.first[t.count++] = (uint32_t)pieces;
        pieces += pass == 0 ? pieces_of(c.numel[k], c.types[k]) : scale_pieces_of(c.outs[k], c.numel[k], c.types[k], bytes);
        if (pieces > INT32_MAX) return SNACK_ERR_UNSUPPORTED;
      }
      t.first[t.count] = (uint32_t)pieces;
      cudaError_t e = cudaSuccess;
      if (pass == 0) {
        const int blocks = pieces < 1 ? 1 : (int)(pieces < most_blocks ? pieces : most_blocks);
        e = launch_pdl(k_clip_norm<kMost>, (unsigned)blocks, kThreads, 0, s, t, (uint32_t)pieces, c.sums + n_sums);
        n_sums += blocks;
        if (e == cudaSuccess && g0 + 1 == groups)
          e = launch_pdl(k_clip_total, 1, kThreads, 0, s, (const Sum3 *)c.sums, n_sums, c.max_norm, c.norm, c.factor);
      } else if (pieces > 0) {
        e = launch_pdl(k_clip_scale<kMost>, (unsigned)pieces, kThreads, 0, s, t, (uint32_t)pieces, bytes,
                       (const float *)c.factor);
      }
      if (e != cudaSuccess) return SNACK_ERR_CUDA;
    }
  return SNACK_OK;
}

// Whether the norm or the workspace overlaps a tensor of the call, or each other.
bool clip_scratch_overlaps(int32_t n, const void *const *grads, void *const *outs, const int64_t *numel,
                           const snack_dtype *types, const float *norm, const void *ws, size_t ws_bytes) {
  const size_t norm_bytes = norm ? sizeof(float) : 0;
  if (spans_overlap(norm, norm_bytes, ws, ws_bytes)) return true;
  for (int32_t k = 0; k < n; ++k) {
    const size_t bytes = (size_t)numel[k] * dtype_size(types[k]);
    if (spans_overlap(grads[k], bytes, ws, ws_bytes) || spans_overlap(grads[k], bytes, norm, norm_bytes)) return true;
    if (outs && outs[k] != grads[k] &&
        (spans_overlap(outs[k], bytes, ws, ws_bytes) || spans_overlap(outs[k], bytes, norm, norm_bytes)))
      return true;
  }
  return false;
}

// Whether an output overlaps another tensor of the call: a gradient given twice
// in place would be scaled twice, or once, as its blocks happen to run.
bool clip_overlaps(int32_t n, const void *const *grads, void *const *outs, const int64_t *numel, const snack_dtype *types) {
  struct Span {
    uintptr_t begin, end;
    bool written;
  };
  std::vector<Span> spans;
  spans.reserve(2 * (size_t)n);
  for (int32_t k = 0; k < n; ++k) {
    if (numel[k] == 0) continue;
    const size_t bytes = (size_t)numel[k] * dtype_size(types[k]);
    const uintptr_t o = (uintptr_t)outs[k], g = (uintptr_t)grads[k];
    spans.push_back({o, o + bytes, true});
    if (g != o) spans.push_back({g, g + bytes, false});
  }
  const auto before = [](const Span &a, const Span &b) { return a.begin < b.begin; };
  if (!std::is_sorted(spans.begin(), spans.end(), before)) std::sort(spans.begin(), spans.end(), before);
  uintptr_t written = 0, any = 0;  // ends of the spans so far
  for (const Span &s : spans) {
    if (s.begin < (s.written ? any : written)) return true;
    any = std::max(any, s.end);
    if (s.written) written = std::max(written, s.end);
  }
  return false;
}

bool clip_sizes_ok(int32_t n, const int64_t *numel, const snack_dtype *types) {
  if (n < 0 || (n > 0 && (!numel || !types))) return false;
  for (int32_t k = 0; k < n; ++k)
    if (numel[k] < 0 || numel[k] > ((int64_t)1 << 45) || !lm_dtype_ok(types[k])) return false;
  return true;
}

// the factor, and the sums of every launch's blocks, on any device of up to 1024 multiprocessors
size_t clip_ws(int32_t n) {
  const int64_t groups = n > 0 ? groups_of(n, table_for(n)) : 1;
  return kAlign + align_up((size_t)groups * 1024 * kBlocksPerSm * sizeof(Sum3), kAlign);
}

}  // namespace
}  // namespace snack

using namespace snack;

extern "C" {

snack_status snack_clip_workspace_size(int32_t n_tensors, const int64_t *numel, const snack_dtype *types,
                                       size_t *bytes) {
  if (!bytes || !clip_sizes_ok(n_tensors, numel, types)) return SNACK_ERR_INVALID_ARG;
  *bytes = clip_ws(n_tensors);
  return SNACK_OK;
}

snack_status snack_clip_grad_norm(int32_t n_tensors, const void *const *grads, void *const *outs,
                                  const int64_t *numel, const snack_dtype *types, float max_norm, float *norm,
                                  void *ws, size_t ws_bytes, snack_stream_t stream) try {
  if (!clip_sizes_ok(n_tensors, numel, types) || !(max_norm >= 0.f)) return SNACK_ERR_INVALID_ARG;
  if (n_tensors > 0 && !grads) return SNACK_ERR_INVALID_ARG;
  for (int32_t k = 0; k < n_tensors; ++k) {
    if (numel[k] == 0) continue;
    const size_t es = dtype_size(types[k]);
    if (!grads[k] || !ptr_aligned(grads[k], es)) return SNACK_ERR_INVALID_ARG;
    if (!outs) continue;
    if (!outs[k] || !ptr_aligned(outs[k], es)) return SNACK_ERR_INVALID_ARG;
  }
  if (outs && clip_overlaps(n_tensors, grads, outs, numel, types)) return SNACK_ERR_INVALID_ARG;
  if (norm && !ptr_aligned(norm, 4)) return SNACK_ERR_INVALID_ARG;
  if (!ws || !ptr_aligned(ws, kAlign)) return SNACK_ERR_INVALID_ARG;
  if (ws_bytes < clip_ws(n_tensors)) return SNACK_ERR_WORKSPACE;
  if (clip_scratch_overlaps(n_tensors, grads, outs, numel, types, norm, ws, clip_ws(n_tensors))) return SNACK_ERR_INVALID_ARG;
  ClipCall c = {n_tensors, grads, outs, numel, types, max_norm, norm,
                reinterpret_cast<Sum3 *>(reinterpret_cast<uint8_t *>(ws) + kAlign), reinterpret_cast<float *>(ws),
                current_sms()};
  if (c.sms < 1) return SNACK_ERR_CUDA;
  if (c.sms > 1024) c.sms = 1024;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (table_for(n_tensors)) {
    case kSmallTable:
      return run_clip<kSmallTable>(c, s);
    case kMidTable:
      return run_clip<kMidTable>(c, s);
    default:
      return run_clip<kBigTable>(c, s);
  }
} catch (...) {  // a host allocation failed
  return SNACK_ERR_CUDA;
}

}  // extern "C"
