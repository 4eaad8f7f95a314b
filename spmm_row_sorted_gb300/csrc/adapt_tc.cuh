// The adapters' products of bf16 on the fifth generation tensor cores; few rows are
// k_adapt_few's.  Included by adapt.cu.
//
// Operands are gathered row by row into tiles with the 128-byte swizzle, by cp.async, or
// where they lie on no such access as the aligned pieces that hold them, shifted; the fp32
// one is cut into two bf16 parts on its way.  One thread issues tcgen05.mma.  The sums stay
// in tensor memory for a run of steps, whose sums are added in fp32 where there are several.
#pragma once

namespace snack {
namespace {

__device__ __forceinline__ uint32_t su32(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(bar)), "r"(count) : "memory");
}
constexpr int kSpinLimit = 1 << 20;  // about four seconds, far above any real wait
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity, int limit = kSpinLimit) {
  const uint32_t at = su32(bar);
  for (int i = 0; i < limit; ++i) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(at), "r"(parity)
        : "memory");
    if (done) return true;
  }
  return false;
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(su32(bar)) : "memory");
}
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// one full warp; the address lands in *dst
__device__ __forceinline__ void tmem_alloc(uint32_t *dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(dst)), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t at, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols) : "memory");
}
// Shared-memory descriptors of tiles with the 128-byte swizzle: start and leading offset
// in 16 bytes; stride 1024 from 8 rows to the next, version 1, layout 2.  MN-major: rows
// of K of 64 elements, `box` bytes from 64 elements to the next 64.
constexpr uint32_t kTcDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t tc_desc(uint32_t at, uint32_t box) { return ((at & 0x3FFFF) >> 4) | (box >> 4) << 16; }
// D (TMEM) (+)= A B^T of 16 of K
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t inst, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(inst), "r"(accumulate), "n"(kTcDescHi)
      : "memory");
}
// arrive on *bar once every MMA issued so far by this thread has completed
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(su32(bar)) : "memory");
}
// fp32 sums (bit 4) of bf16 operands (bits 7 and 10), MN-major A and B (bits 15 and 16), N / 8 at bit 17, M / 16 at bit 24
__host__ __device__ constexpr uint32_t tc_inst(int m, int n, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(m >> 4) << 24);
}
// 16 consecutive fp32 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_ld16(uint32_t at, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(at)
      : "memory");
}
// ties the registers of a load to the wait for it
__device__ __forceinline__ void tmem_wait(float (&a)[16], float (&b)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) asm volatile("" : "+f"(a[i]), "+f"(b[i]));
}

constexpr int kTcThreads = 256;

__device__ __forceinline__ float4 ld_cluster4(const float *p, uint32_t block) {
  uint32_t at;
  float4 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(su32(p)), "r"(block));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}

// ------------------------------------------------------------ h and dh

constexpr int kTcTile = 128;  // rows of a tile: the lanes of TMEM
constexpr int kTcK = 64;      // of K per stage: 128 bytes of a row
constexpr int kTcRowBox = kTcTile * 128;  // bytes of 64 elements of the rows

// of the rank: padded to steps of 16, and 64 of it per 128 bytes
__host__ __device__ constexpr int tc_steps(int rank) { return (rank + 15) / 16; }
__host__ __device__ constexpr int tc_blocks(int rank) { return (rank + 63) / 64; }
__host__ __device__ constexpr uint32_t tc_tmem_cols(int cols) { return cols <= 32 ? 32 : cols <= 64 ? 64 : cols <= 128 ? 128 : 256; }

constexpr int kTcDownStages = 4;
// Steps summed on the tensor core, which cuts off what does not fit (of terms of one sign 9e-8 of the sum at each of a step's
// four additions; nearly 2^20 of K were off by 7e-4), before their sum is added in fp32: 64 additions, 6e-6, less than
// the 2^-17 that h and dh are held to in the products after.  Runs have the two halves of a block's tensor memory in turn; the
// one before is read when its last step has been waited for anyway (8192 rows of 16384, rank 64, both calls of a pass: 331 us
// without runs, 335 with these, 341 with runs of 8).
constexpr int kTcDownRun = 16;
__host__ __device__ constexpr int tc_down_stage(int rank) { return kTcRowBox + tc_blocks(rank) * kTcK * 128; }
__host__ __device__ constexpr size_t tc_down_smem(int rank) {
  const size_t ring = (size_t)kTcDownStages * tc_down_stage(rank), sums = (size_t)kTcTile * (16 * tc_steps(rank) + 4) * 4;
  const size_t all = (ring > sums ? ring : sums) + 1024;
  // all of the tensor memory above a rank of 128: no room beside it for another kernel that wants some
  return rank > 128 && all < 200 * 1024 ? 200 * 1024 : all;
}

// How a matrix's or the rows' pieces of eight elements lie in memory
enum { kLoose = 0, kOn8 = 1, kOn16 = 2 };
__host__ inline int lies_on(const void *p, int64_t ld) {
  return ptr_aligned(p, 16) && ld % 8 == 0 ? kOn16 : ptr_aligned(p, 8) && ld % 4 == 0 ? kOn8 : kLoose;
}

// Eight elements from anywhere, `left` of them there, the others zeros: the two aligned pieces that hold them, shifted.
// kKept: read only while the kernel runs.
template <bool kKept>
__device__ __forceinline__ uint4 load_loose(const void *p, int left) {
  if (left <= 0) return make_uint4(0, 0, 0, 0);
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const int skip = (int)(at & 15), bytes = min(left, 8) * 2;
  const uint4 *from = reinterpret_cast<const uint4 *>(at - skip);
  uint4 lo, hi = make_uint4(0, 0, 0, 0);
  if constexpr (kKept) {
    lo = __ldg(from);
    if (skip + bytes > 16) hi = __ldg(from + 1);
  } else {
    lo = *from;
    if (skip + bytes > 16) hi = from[1];
  }
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if (skip & 8)
#pragma unroll
    for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
  if (skip & 4)
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
  uint32_t v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[k] = skip & 2 ? __byte_perm(w[k], w[k + 1], 0x5432) : w[k];
    v[k] = 2 * k + 1 < left ? v[k] : 2 * k < left ? v[k] & 0xFFFFu : 0u;
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}
// and to anywhere, by words where they are aligned
__device__ __forceinline__ void store_loose(uint16_t *p, uint4 v, int left) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if ((reinterpret_cast<uintptr_t>(p) & 2) == 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (2 * k + 1 < left)
        *reinterpret_cast<uint32_t *>(p + 2 * k) = w[k];
      else if (2 * k < left)
        p[2 * k] = (uint16_t)w[k];
    }
  } else {
    if (left > 0) p[0] = (uint16_t)w[0];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t pair = k < 3 ? __byte_perm(w[k], w[k + 1 < 4 ? k + 1 : 3], 0x5432) : w[k] >> 16;
      if (k < 3 && 2 * k + 2 < left)
        *reinterpret_cast<uint32_t *>(p + 2 * k + 1) = pair;
      else if (2 * k + 1 < left)
        p[2 * k + 1] = (uint16_t)pair;
    }
  }
}

// A piece of 16 bytes as 16 or, where it lies on 8, twice 8 of them; `bytes` of them are there.
__device__ __forceinline__ void copy_piece(void *to, const void *from, int bytes, bool wide) {
  if (wide) {
    copy_async<16>(to, from, bytes);
  } else {
    copy_async<8>(to, from, min(bytes, 8));
    copy_async<8>(reinterpret_cast<uint8_t *>(to) + 8, reinterpret_cast<const uint8_t *>(from) + (bytes > 8 ? 8 : 0), max(bytes - 8, 0));
  }
}
// Pieces of a matrix, place(k, to, from, bytes) naming the k-th of n: on their way, or, where they lie anywhere, read two at
// a time and there.
template <typename F>
__device__ __forceinline__ void copy_pieces(int n, int on, F place) {
  if (on != kLoose) {
#pragma unroll 2
    for (int k = 0; k < n; ++k) {
      uint8_t *to;
      const bf16 *from;
      int bytes;
      place(k, to, from, bytes);
      copy_piece(to, from, bytes, on == kOn16);
    }
    return;
  }
#pragma unroll 1
  for (int k = 0; k < n; k += 2) {
    uint8_t *to[2];
    uint4 v[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const bf16 *from;
      int bytes = 0;
      place(min(k + u, n - 1), to[u], from, bytes);
      v[u] = load_loose<true>(from, bytes / 2);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) *reinterpret_cast<uint4 *>(to[u]) = v[u];
  }
}

// A tile of 128 rows against an adapter's matrix, all of its ranks (N); the cluster's blocks have every so many 64 of K.
// kWide: the rows lie on 16 bytes.  kLong: a block may have more than a run of steps.
template <bool kAlong, bool kWide, bool kLong>
__global__ void __launch_bounds__(kTcThreads, 2) k_adapt_down_tc(const DownArgs args, const FileArgs f, int m_on) {
  pdl_wait();
  const uint32_t block = cluster_rank(), blocks = cluster_blocks();
  extern __shared__ uint8_t tc_raw[];
  __shared__ int32_t rows[kTcTile];
  DownArgs a = args;
  Tile tile;
  if (f.which.ids) {
    tile = file_tile<kTcThreads>(f, (int)(blockIdx.x / blocks), blockIdx.x == 0, reinterpret_cast<int32_t *>(tc_raw + (16 - (su32(tc_raw) & 15) & 15)), rows);
    a.order = rows;
  } else {
    tile = a.tiles[blockIdx.x / blocks];
  }
  if (tile.adapter < 0 || tile.adapter >= a.adapters) return;  // the whole cluster's
  __shared__ uint64_t done[kTcDownStages];
  __shared__ uint32_t tmem_at;
  uint8_t *ring = tc_raw + ((1024 - (su32(tc_raw) & 1023)) & 1023);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = a.rank, n_pad = 16 * tc_steps(rank), stage_bytes = tc_down_stage(rank);
  const uint32_t half = tc_tmem_cols(n_pad), tmem_cols = kLong ? 2 * half : half;
  if (warp == 0) tmem_alloc(&tmem_at, tmem_cols);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kTcDownStages; ++s) mbar_init(&done[s], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  bool ok = true;
  const int k_blocks = (a.k + kTcK - 1) / kTcK, steps = (int)block < k_blocks ? (k_blocks - (int)block + (int)blocks - 1) / (int)blocks : 0;
  // the rows: eight lanes have 128 bytes of one, a warp four at a time
  constexpr int kPasses = kTcTile / (kTcThreads / 8);
  const bf16 *row[kPasses];
#pragma unroll
  for (int u = 0; u < kPasses; ++u) {
    const int t = threadIdx.x / 8 + u * (kTcThreads / 8);
    row[u] = reinterpret_cast<const bf16 *>(a.x) + (int64_t)a.order[tile.first + min(t, tile.count - 1)] * a.x_ld + 8 * (lane & 7);
  }
  const bf16 *mat = reinterpret_cast<const bf16 *>(a.m) + (int64_t)tile.adapter * rank * a.k;
  auto fetch = [&](int i) {
    if (i < steps) {
      const int k0 = (i * (int)blocks + (int)block) * kTcK;
      uint8_t *to = ring + (i % kTcDownStages) * stage_bytes;
      const int left = a.k - k0, bytes = max(0, min(left - 8 * (lane & 7), 8)) * 2;
      auto place = [&](int u) { return to + (threadIdx.x / 8 + u * (kTcThreads / 8)) * 128 + (((lane & 7) ^ ((threadIdx.x / 8) & 7)) << 4); };
      if constexpr (kWide) {
#pragma unroll
        for (int u = 0; u < kPasses; ++u)
          if (threadIdx.x / 8 + u * (kTcThreads / 8) < tile.count) copy_async<16>(place(u), bytes ? row[u] + k0 : row[u], bytes);
      } else {
        uint4 v[kPasses];
#pragma unroll
        for (int u = 0; u < kPasses; ++u)
          v[u] = load_loose<true>(row[u] + k0, threadIdx.x / 8 + u * (kTcThreads / 8) < tile.count ? bytes / 2 : 0);
#pragma unroll
        for (int u = 0; u < kPasses; ++u) *reinterpret_cast<uint4 *>(place(u)) = v[u];
      }
      // the matrix: eight threads have 128 bytes of every 32nd row; zeros past the end
      const int c = lane & 7, r0 = threadIdx.x >> 3;
      uint8_t *box = to + kTcRowBox + r0 * 128 + ((c ^ (r0 & 7)) << 4);
      constexpr int kEvery = kTcThreads / 8;
      if constexpr (kAlong) {
        copy_pieces((n_pad - r0 + kEvery - 1) / kEvery, m_on, [&](int k, uint8_t *&at, const bf16 *&from, int &n) {
          const int r = r0 + k * kEvery;
          at = box + k * kEvery * 128;
          n = r < rank ? bytes : 0;
          from = n ? mat + (int64_t)r * a.k + k0 + 8 * c : mat;
        });
      } else {
        copy_pieces(8 * c < n_pad ? 2 * ((n_pad - 8 * c + 63) / 64) : 0, m_on, [&](int k, uint8_t *&at, const bf16 *&from, int &n) {
          static_assert(kTcK == 2 * kEvery, "two rows of each 64");
          const int b = 8 * c + 64 * (k >> 1), r = r0 + (k & 1) * kEvery;
          at = box + (k >> 1) * kTcK * 128 + (k & 1) * kEvery * 128;
          n = r < left ? max(0, min(rank - b, 8)) * 2 : 0;
          from = n ? mat + (int64_t)(k0 + r) * rank + b : mat;
        });
      }
    }
    fetch_commit();
  };
  // this warp's sums: rows 32 (warp % 4) + lane, 16 columns in 32
  const uint32_t own_sums = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
  const int own_c = 16 * (warp >> 2);
  float before[kLong ? kMostRank / 2 : 1];  // of the runs before the one before, in local memory
  auto keep = [&](int run) {
    tc_fence_after();
#pragma unroll 1
    for (int c = own_c; c < n_pad; c += 32) {
      float v[16];
      tmem_ld16(own_sums + (run & 1) * half + c, v);
      tmem_wait(v, v);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float &to = before[kLong ? (c >> 5) * 16 + e : 0];
        to = run ? to + v[e] : v[e];
      }
    }
    tc_fence_before();
  };
  // the rows past the tile's end stay as they are: a row's sums are its own
  if (steps) {
    const uint32_t inst = tc_inst(kTcTile, n_pad, false, !kAlong);
    for (int s = 0; s < kTcDownStages - 1; ++s) fetch(s);
    for (int i = 0; i < steps; ++i) {
      fetch_wait<kTcDownStages - 2>();
      fence_async_shared();
      __syncthreads();
      if (threadIdx.x == 0) {
        tc_fence_after();
        const uint32_t at = su32(ring) + (i % kTcDownStages) * stage_bytes, b = at + kTcRowBox;
        const uint32_t d = kLong ? tmem + (i / kTcDownRun & 1) * half : tmem;
#pragma unroll
        for (int s = 0; s < kTcK / 16; ++s)
          tc_mma(d, tc_desc(at + s * 32, 16), kAlong ? tc_desc(b + s * 32, 16) : tc_desc(b + s * 2048, kTcK * 128), inst,
                 (kLong ? i % kTcDownRun : i) > 0 || s > 0);
        tc_commit(&done[i % kTcDownStages]);
      }
      if (i > 0) ok = mbar_wait(&done[(i - 1) % kTcDownStages], ((i - 1) / kTcDownStages) & 1) && ok;
      fetch(i + kTcDownStages - 1);
      if (kLong && i > 0 && i % kTcDownRun == 0) keep(i / kTcDownRun - 1);
    }
    fetch_wait<0>();
    ok = mbar_wait(&done[(steps - 1) % kTcDownStages], ((steps - 1) / kTcDownStages) & 1) && ok;
    tc_fence_after();
  }
  ok = __syncthreads_and(ok);  // the ring becomes the sums; of a wait that gave up all of the block's are NaN
  float *sums = reinterpret_cast<float *>(ring);
  const int pitch = n_pad + 4;
  for (int c = own_c; c < n_pad; c += 32) {
    float v[16];
    if (steps) {
      tmem_ld16(own_sums + (kLong ? ((steps - 1) / kTcDownRun & 1) * half : 0) + c, v);
      tmem_wait(v, v);
    }
    float *to = sums + (32 * (warp & 3) + lane) * pitch + c;
    if (kLong && steps > kTcDownRun)
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] += before[kLong ? (c >> 5) * 16 + e : 0];
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = !ok ? NAN : steps ? v[e] : 0.f;
#pragma unroll
    for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4 *>(to + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
  }
  tc_fence_before();
  if (blocks > 1)
    cluster_sync();
  else
    __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols);
  }
  const float scale = a.scales ? a.scales[tile.adapter] : 1.f;
  const int quads = n_pad / 4;
  for (int i = (int)block * kTcThreads + threadIdx.x; i < tile.count * quads; i += (int)blocks * kTcThreads) {
    const int t = i / quads, r = (i - t * quads) * 4;
    if (r >= rank) continue;
    const float *at = sums + t * pitch + r;
    float4 s = *reinterpret_cast<const float4 *>(at);
    if (blocks > 1) {
      s = ld_cluster4(at, 0);
      for (uint32_t b = 1; b < blocks; ++b) {
        const float4 o = ld_cluster4(at, b);
        s.x += o.x;
        s.y += o.y;
        s.z += o.z;
        s.w += o.w;
      }
    }
    float *to = a.h + (int64_t)a.order[tile.first + t] * rank + r;
    const float w[4] = {s.x * scale, s.y * scale, s.z * scale, s.w * scale};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (r + e < rank) to[e] = w[e];
  }
  if (blocks > 1) cluster_sync();  // no block's memory is read any more
}

template <bool kAlong, bool kWide>
cudaError_t launch_down_tc(const DownArgs &a, const FileArgs &f, int64_t tiles, int tile_cap, int sms, cudaStream_t s) {
  const size_t smem = tc_down_smem(a.rank);
  const unsigned c = cluster_for(tiles, ceil_div(a.k, 2 * kTcK), 2 * sms);
  const auto kernel = ceil_div(a.k, (int64_t)c * kTcK) > kTcDownRun ? k_adapt_down_tc<kAlong, kWide, true> : k_adapt_down_tc<kAlong, kWide, false>;
  cudaError_t e = raise_smem_limit(kernel, smem);
  if (e != cudaSuccess) return e;
  return launch_cluster(c, kernel, dim3((unsigned)tile_cap * c), kTcThreads, smem, s, a, f, lies_on(a.m, kAlong ? a.k : a.rank));
}
template <bool kAlong>
cudaError_t down_tc(const DownArgs &a, const FileArgs &f, int64_t tiles, int tile_cap, int sms, cudaStream_t s) {
  return lies_on(a.x, a.x_ld) == kOn16 ? launch_down_tc<kAlong, true>(a, f, tiles, tile_cap, sms, s)
                                       : launch_down_tc<kAlong, false>(a, f, tiles, tile_cap, sms, s);
}

// ------------------------------------------------------------ y and dx

constexpr int kTcUpCols = 128;  // columns of a unit
constexpr int kTcUpEpi = 256;   // threads that write results; a warp more fetches the matrix, another one issues the products
constexpr int kTcUpThreads = kTcUpEpi + 64;
constexpr int kTcUpMostStages = 3;
constexpr int64_t kTcUpRun = 8; // units of a block that follow one another, about
__host__ __device__ constexpr int tc_up_stage(int rank) { return tc_blocks(rank) * kTcUpCols * 128; }
__host__ __device__ constexpr int tc_up_stages(int rank) { return tc_blocks(rank) <= 2 ? 3 : tc_blocks(rank) == 3 ? 2 : 1; }
__host__ __device__ constexpr size_t tc_up_smem(int rank) {
  return (size_t)2 * tc_blocks(rank) * kTcRowBox + (size_t)tc_up_stages(rank) * tc_up_stage(rank) + 1024;
}
static_assert(tc_up_smem(kMostRank) <= 232448 - 1024 && tc_up_smem(192) <= 232448 - 1024 && tc_up_smem(128) <= 232448 - 1024 &&
                  tc_down_smem(kMostRank) <= 232448 - 1024,
              "shared memory of one block");

// how often the warp that fetches, and those that issue and write, look for what they wait for: a test builds with fewer
#ifndef SNACK_UP_FETCH_WAITS
#define SNACK_UP_FETCH_WAITS kSpinLimit
#define SNACK_UP_WAITS kSpinLimit
#endif
constexpr int kFetchWaits = SNACK_UP_FETCH_WAITS, kUpWaits = SNACK_UP_WAITS;

// the warps that lay out h and the one that issues products: whether all are well
__device__ __forceinline__ bool tc_rows_sync(bool ok) {
  uint32_t all;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.and.pred p, 1, %2, q;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(all)
               : "r"(ok ? 1u : 0u), "n"(kTcUpEpi + 32)
               : "memory");
  return all != 0;
}

// 32 columns of 16 lanes of TMEM as a product's fragments: v[4 j + 2 h + e] is row 8 h + lane / 4, column 8 j + 2 (lane % 4) + e
__device__ __forceinline__ void tmem_ld_rows(uint32_t at, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(at)
      : "memory");
}
// the pairs (j, lane % 4) of a fragment turned into (lane % 4, j): a lane has eight neighbours of each row then
__device__ __forceinline__ void turn_pairs(float (&v)[16], int lane) {
#pragma unroll
  for (int d = 1; d <= 2; d *= 2) {
    const bool up = lane & d;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & d) continue;  // lanes without the bit keep chunk j and take their partner's j for their chunk j + d
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float mine = up ? v[4 * j + k] : v[4 * (j + d) + k];
        const float other = __shfl_xor_sync(0xffffffffu, mine, d);
        if (up)
          v[4 * j + k] = other;
        else
          v[4 * (j + d) + k] = other;
      }
    }
  }
}

// up to eight elements at the end of a row
__device__ __noinline__ uint4 read_some(const uint16_t *p, int left) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = (2 * j < left ? p[2 * j] : 0u) | (2 * j + 1 < left ? (uint32_t)p[2 * j + 1] << 16 : 0u);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __noinline__ void write_some(uint16_t *p, uint4 v, int left) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) p[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
}

// Units of a tile of 128 rows and 128 columns: h in its two parts (A, K-major) against the matrix's columns (B).  A block
// has runs of units; all blocks' runs one beside the other, so that what is read and written at a time are some tiles'
// rows.  One warp fetches the matrix, one issues the products into two sets of sums in turn, eight add the base, which
// they have read ahead, and write the result: 32 rows and 64 columns each, 64 bytes of a row from four lanes together.
// For that the matrix's rows lie in the order of a fragment's columns (kAlong), or pairs change lanes.
// A warp whose wait gives up hands on nothing more, so that the others' waits give up as well: a result is right or NaN.
// (Base and result through shared memory, 64 columns at a time: 143 us for y of 8192 x 16384 of rank 64, 41 % of shared
// memory's cycles; eight warps doing everything in turn 190, of a step's 3700 cycles 1200 waiting for the products.)
// kWide: the base's and the result's rows lie on 16 bytes.
template <bool kAlong, bool kWide>
__global__ void __launch_bounds__(kTcUpThreads, 2) k_adapt_up_tc(const UpArgs a, int m_on) {
  pdl_wait();
  extern __shared__ uint8_t tc_raw[];
  __shared__ uint64_t full[kTcUpMostStages], empty[kTcUpMostStages], done[2], taken[2];
  __shared__ uint32_t tmem_at;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int across = (a.cols + kTcUpCols - 1) / kTcUpCols;
  const int64_t units = (int64_t)__ldg(a.n_tiles) * across;
  const int64_t per = (units + gridDim.x - 1) / gridDim.x, rounds = max((int64_t)1, per / kTcUpRun), run = (per + rounds - 1) / rounds;
  int64_t u0 = blockIdx.x * run, u_end = min(units, u0 + run);
  if (u0 >= units) return;
  const int rank = a.rank, steps = tc_steps(rank), k_blocks = tc_blocks(rank), stages = tc_up_stages(rank), stage_bytes = tc_up_stage(rank);
  uint8_t *hs = tc_raw + ((1024 - (su32(tc_raw) & 1023)) & 1023), *ring = hs + 2 * k_blocks * kTcRowBox;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kTcUpMostStages; ++s) {
      mbar_init(&full[s], 32);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&done[s], 1);
      mbar_init(&taken[s], kTcUpEpi / 32);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kTcUpThreads / 32 - 1) tmem_alloc(&tmem_at, 2 * kTcUpCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  bool ok = true;
  int s = 0, turn = 0;       // the stage in hand and how often the ring has been round, modulo 2
  uint32_t g = 0;            // units with products so far; of the warp that issues them those issued
  while (u0 < units) {
    const int at = (int)(u0 / across), first = (int)(u0 - (int64_t)at * across);
    const int items = (int)min((int64_t)(across - first), u_end - u0), col0 = first * kTcUpCols;
    u0 += items;
    if (u0 == u_end) {
      u0 += (gridDim.x - 1) * run;
      u_end = min(units, u0 + run);
    }
    const Tile tile = a.tiles[at];
    const bool none = tile.adapter >= a.adapters;  // the base as it is
    if (none && a.base == a.out) continue;
    if (warp < kTcUpEpi / 32) {
      const int first_row = 32 * (warp & 3), q = lane & 3, col = col0 + 64 * (warp >> 2) + 8 * q;
      const uint16_t *from[4];  // this lane's rows, from its first eight columns on
      uint16_t *to[4];
      bool in[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = first_row + 8 * r + (lane >> 2);
        in[r] = t < tile.count;
        const int64_t token = __ldg(a.order + tile.first + (in[r] ? t : 0));
        from[r] = reinterpret_cast<const uint16_t *>(a.base) + token * a.base_ld + col;
        to[r] = reinterpret_cast<uint16_t *>(a.out) + token * a.out_ld + col;
      }
      uint4 base[2][4];
      auto read = [&](int past, bool whole, uint4 (&v)[4]) {  // columns `past` behind the first ones
        if (kWide && a.base && whole) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (in[r]) v[r] = *reinterpret_cast<const uint4 *>(from[r] + past);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int left = a.base && in[r] ? a.cols - col - past : 0;
            v[r] = kWide ? read_some(from[r] + past, left) : load_loose<false>(from[r] + past, left);
          }
        }
      };
      const bool whole_first = !a.base || col0 + kTcUpCols <= a.cols;
      if (a.base) {
        read(0, whole_first, base[0]);
        read(32, whole_first, base[1]);
      }
      if (!none) {  // h, when no product reads the tile's before any more: two threads have a row, eight ranks at a time; zeros
                    // past the tile's rows and the rank
        const float scale = a.scales ? a.scales[tile.adapter] : 1.f;
        const int t = threadIdx.x >> 1;
        const float *from = a.h + (int64_t)__ldg(a.order + tile.first + (t < tile.count ? t : 0)) * rank;
        for (int e0 = threadIdx.x & 1; ok && e0 < 2 * steps; e0 += 4) {
          Pack<float, 16> v[2][2];
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const int r = 8 * (e0 + 2 * u) + 4 * p;
              v[u][p] = load_vec<float, 4>(from + (r < rank ? r : 0), t < tile.count ? rank - r : 0, a.h_wide);
            }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int e8 = e0 + 2 * u;
            if (e8 >= 2 * steps) break;
            uint32_t w[4][2];
#pragma unroll
            for (int p = 0; p < 4; ++p) cut_pair<2>(scale * v[u][p >> 1].get(2 * (p & 1)), scale * v[u][p >> 1].get(2 * (p & 1) + 1), w[p]);
#pragma unroll
            for (int p = 0; p < 2; ++p)
              *reinterpret_cast<uint4 *>(hs + (p * k_blocks + (e8 >> 3)) * kTcRowBox + t * 128 + (((e8 & 7) ^ (t & 7)) << 4)) =
                  make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
          }
        }
        fence_async_shared();
        ok = tc_rows_sync(ok);
      }
      for (int i = 0; i < items; ++i) {
        if (!none) {
          ok = ok && mbar_wait(&done[g & 1], (g >> 1) & 1, kUpWaits);
          tc_fence_after();
        }
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
          const int past = i * kTcUpCols + 32 * sub;
          const bool whole = col0 + (i + 1) * kTcUpCols <= a.cols;
          if (!a.base) {
#pragma unroll
            for (int r = 0; r < 4; ++r) base[sub][r] = make_uint4(0, 0, 0, 0);
          }
          float v[2][16];
          if (!none) {
            const uint32_t at_sums = tmem + ((uint32_t)first_row << 16) + (g & 1) * kTcUpCols + 64 * (warp >> 2) + 32 * sub;
            tmem_ld_rows(at_sums, v[0]);
            tmem_ld_rows(at_sums + (16u << 16), v[1]);
            tmem_wait(v[0], v[1]);
            if (sub == 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0 && ok) mbar_arrive(&taken[g & 1]);
            }
            if constexpr (!kAlong) {
              turn_pairs(v[0], lane);
              turn_pairs(v[1], lane);
            }
            if (!ok)  // a wait gave up
#pragma unroll
              for (int e = 0; e < 16; ++e) v[0][e] = v[1][e] = NAN;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float *x = &v[r >> 1][2 * (r & 1)];
              uint32_t(&o)[4] = reinterpret_cast<uint32_t(&)[4]>(base[sub][r]);
#pragma unroll
              for (int j = 0; j < 4; ++j) o[j] = pack_pair(bf16_lo(o[j]) + x[4 * j], bf16_hi(o[j]) + x[4 * j + 1]);
            }
          }
          if (kWide && whole) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (in[r]) *reinterpret_cast<uint4 *>(to[r] + past) = base[sub][r];
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int left = in[r] ? a.cols - col - past : 0;
              if constexpr (kWide)
                write_some(to[r] + past, base[sub][r], left);
              else
                store_loose(to[r] + past, base[sub][r], left);
            }
          }
          if (a.base && i + 1 < items) read(past + kTcUpCols, col0 + (i + 2) * kTcUpCols <= a.cols, base[sub]);
        }
        if (!none) ++g;
      }
    } else if (none) {
      continue;
    } else if (warp == kTcUpEpi / 32) {
      const bf16 *mat = reinterpret_cast<const bf16 *>(a.m) + (int64_t)tile.adapter * rank * a.cols;
      for (int i = 0; i < items; ++i, ++g) {
        if (g >= (uint32_t)stages) {
          ok = __all_sync(0xffffffffu, ok && mbar_wait(&empty[s], turn ^ 1, kFetchWaits));
          if (!ok) continue;
        }
        uint8_t *to = ring + s * stage_bytes;
        const int col = col0 + i * kTcUpCols, left = a.cols - col;
        if constexpr (kAlong) {  // eight lanes have 128 bytes of a row, four rows at a time
          // row r = 4 u + r0 of the tile is column 32 (u / 8) + 16 (u % 2) + 2 (u / 2 % 4) + 8 (r0 / 2) + r0 % 2: a fragment's
          const int c = lane & 7, r0 = lane >> 3, n0 = 8 * (r0 >> 1) + (r0 & 1);
          for (int b = 0; b < k_blocks; ++b, to += kTcUpCols * 128) {
            if (64 * b + 8 * c >= 16 * steps) break;
            const int bytes = max(0, min(rank - 64 * b - 8 * c, 8)) * 2;
            const bf16 *p = mat + (int64_t)(col + n0) * rank + 64 * b + 8 * c;
            uint8_t *even = to + r0 * 128 + ((c ^ r0) << 4), *odd = to + (r0 + 4) * 128 + ((c ^ (r0 + 4)) << 4) - 512;
            if (left >= kTcUpCols && bytes == 16 && m_on == kOn16) {
#pragma unroll
              for (int u = 0; u < kTcUpCols / 4; ++u)
                copy_whole<16>((u & 1 ? odd : even) + u * 512, p + (32 * (u >> 3) + 16 * (u & 1) + 2 * ((u >> 1) & 3)) * rank);
            } else {
              copy_pieces(kTcUpCols / 4, m_on, [&](int u, uint8_t *&at, const bf16 *&piece, int &there) {
                const int n = 32 * (u >> 3) + 16 * (u & 1) + 2 * ((u >> 1) & 3);
                at = (u & 1 ? odd : even) + u * 512;
                there = n0 + n < left ? bytes : 0;
                piece = there ? p + n * rank : mat;
              });
            }
          }
        } else {  // 16 lanes have the 256 bytes of a row
          const int c = lane & 15, r0 = lane >> 4, bytes = max(0, min(left - 8 * c, 8)) * 2;
          to += (c >> 3) * k_blocks * 64 * 128;
          auto place = [&](int u, uint8_t *&at, const bf16 *&piece, int &there) {
            const int k = r0 + 2 * u;
            at = to + k * 128 + (((c & 7) ^ (k & 7)) << 4);
            there = k < rank ? bytes : 0;
            piece = there ? mat + (int64_t)k * a.cols + col + 8 * c : mat;
          };
          if (left >= kTcUpCols && rank % 16 == 0 && m_on == kOn16) {
#pragma unroll 8
            for (int u = 0; u < 8 * steps; ++u) {
              uint8_t *at;
              const bf16 *piece;
              int there;
              place(u, at, piece, there);
              copy_whole<16>(at, mat + (int64_t)(r0 + 2 * u) * a.cols + col + 8 * c);
            }
          } else {
            copy_pieces(8 * steps, m_on, place);
          }
        }
        fetch_commit();
        if (stages == 1) {
          fetch_wait<0>();
          fence_async_shared();
          mbar_arrive(&full[s]);
        } else if (g > 0) {  // the one before is there
          fetch_wait<1>();
          fence_async_shared();
          mbar_arrive(&full[s == 0 ? stages - 1 : s - 1]);
        }
        if (++s == stages) {
          s = 0;
          turn ^= 1;
        }
      }
    } else {
      ok = tc_rows_sync(ok);
      constexpr uint32_t kInst = tc_inst(kTcTile, kTcUpCols, false, !kAlong);
      for (int i = 0; i < items; ++i) {
        ok = __all_sync(0xffffffffu, ok && mbar_wait(&full[s], turn, kUpWaits) &&
                                         (g < 2 || mbar_wait(&taken[g & 1], ((g >> 1) & 1) ^ 1, kUpWaits)));
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t h_at = su32(hs), b = su32(ring) + s * stage_bytes, d = tmem + (g & 1) * kTcUpCols;
          for (int p = 1; p >= 0; --p)
            for (int k = 0; k < steps; ++k)
              tc_mma(d, tc_desc(h_at + (p * k_blocks + (k >> 2)) * kTcRowBox + (k & 3) * 32, 16),
                     kAlong ? tc_desc(b + (k >> 2) * kTcUpCols * 128 + (k & 3) * 32, 16) : tc_desc(b + k * 2048, k_blocks * 64 * 128), kInst,
                     p == 0 || k > 0);
          tc_commit(&empty[s]);
          tc_commit(&done[g & 1]);
        }
        __syncwarp();
        ++g;
        if (++s == stages) {
          s = 0;
          turn ^= 1;
        }
      }
    }
  }
  if (warp == kTcUpEpi / 32 && g > 0 && stages > 1) {
    fetch_wait<0>();
    fence_async_shared();
    if (ok) mbar_arrive(&full[s == 0 ? stages - 1 : s - 1]);
  }
  // no product is under way any more, also where the warps that write have given up
  if (warp == kTcUpThreads / 32 - 1 && g > 0) mbar_wait(&done[(g - 1) & 1], ((g - 1) >> 1) & 1, kUpWaits);
  tc_fence_before();
  __syncthreads();
  if (warp == kTcUpThreads / 32 - 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * kTcUpCols);
  }
}

template <bool kAlong, bool kWide>
cudaError_t launch_up_tc(const UpArgs &a, int tile_cap, int sms, cudaStream_t s) {
  const size_t smem = tc_up_smem(a.rank);
  const auto kernel = k_adapt_up_tc<kAlong, kWide>;
  cudaError_t e = raise_smem_limit(kernel, smem);
  if (e != cudaSuccess) return e;
  const int64_t most = tile_cap * ceil_div(a.cols, kTcUpCols), room = (int64_t)sms * (smem <= 113 * 1024 ? 2 : 1);
  return launch_pdl(kernel, (unsigned)std::min(most, room), kTcUpThreads, smem, s, a, lies_on(a.m, kAlong ? a.rank : a.cols));
}
template <bool kAlong>
cudaError_t up_tc(const UpArgs &a, int tile_cap, int sms, cudaStream_t s) {
  return (!a.base || lies_on(a.base, a.base_ld) == kOn16) && lies_on(a.out, a.out_ld) == kOn16 ? launch_up_tc<kAlong, true>(a, tile_cap, sms, s)
                                                                                              : launch_up_tc<kAlong, false>(a, tile_cap, sms, s);
}

// ------------------------------------------------------------ dA and dB

constexpr int kTcCols = 256;     // columns of a block: two tiles of 128, the lanes of TMEM
constexpr int kTcRows = 32;      // rows (of K) per stage
constexpr int kTcStages = 3;
constexpr int kTcBox = kTcRows * 128;  // bytes of 64 columns of a stage
// Steps summed on the tensor core, which cuts off what does not fit (of terms of one sign 5e-8 of the sum at each of a step's
// four additions; 2^21 rows of one adapter were off by 1.7e-3), before their sum is added in fp32: 528 additions, 2.7e-5 or
// a 72nd of half a step of bf16, 4096 rows and a bit.  An even number of rounds of the stages: the barriers' phases begin
// again with each run.
constexpr int kTcRun = 132;
static_assert(kTcRun % (2 * kTcStages) == 0, "whole phases");
__host__ __device__ constexpr int tc_outer_stage(int ranks) { return (kTcCols + 2 * ranks) / 64 * kTcBox; }
constexpr size_t tc_outer_smem(int ranks) {
  const size_t ring = (size_t)kTcStages * tc_outer_stage(ranks), sums = std::max((size_t)ranks * (kTcCols + 4), (size_t)kTcCols * (ranks + 4)) * 4;
  return (ring > sums ? ring : sums) + 1024;
}

// The cluster's sums, kMajor rows of kMinor + 4, to rows `at_major` on and columns `at_minor` on of [major][minor]: this
// block's share of them, four neighbours at a time, four of those in flight.
template <int kMinor, int kMajor>
__device__ __forceinline__ void tc_outer_write(const OuterArgs &a, const float *sums, uint32_t block, uint32_t blocks, int adapter,
                                               int at_major, int at_minor, int major, int minor, bool empty) {
  constexpr int kItems = kMajor * kMinor / 4, kEach = 4;
  static_assert(kItems % (kTcThreads * kMostCluster) == 0, "whole turns");
  const float scale = a.scales ? a.scales[adapter] : 1.f;
  bf16 *out = reinterpret_cast<bf16 *>(a.out) + (int64_t)adapter * major * minor;
  const bool wide = minor % 4 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 7) == 0;
  const int share = kItems / (int)blocks;
  for (int i0 = threadIdx.x; i0 < share; i0 += kEach * kTcThreads) {
    float4 v[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u) v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (uint32_t b = 0; b < blocks; ++b) {
#pragma unroll
      for (int u = 0; u < kEach; ++u) {
        const int i = i0 + u * kTcThreads + (int)block * share;
        if (i0 + u * kTcThreads >= share) break;
        const float *at = sums + i / (kMinor / 4) * (kMinor + 4) + i % (kMinor / 4) * 4;
        const float4 o = blocks > 1 ? ld_cluster4(at, b) : *reinterpret_cast<const float4 *>(at);
        v[u].x += o.x;
        v[u].y += o.y;
        v[u].z += o.z;
        v[u].w += o.w;
      }
    }
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int i = i0 + u * kTcThreads + (int)block * share;
      if (i0 + u * kTcThreads >= share) break;
      const int r = at_major + i / (kMinor / 4), c = at_minor + i % (kMinor / 4) * 4;
      if (r >= major || c >= minor) continue;
      // an adapter without rows has no gradient, whatever its scale
      const float w[4] = {empty ? 0.f : v[u].x * scale, empty ? 0.f : v[u].y * scale, empty ? 0.f : v[u].z * scale, empty ? 0.f : v[u].w * scale};
      bf16 *to = out + (int64_t)r * minor + c;
      if (wide) {
        *reinterpret_cast<uint2 *>(to) = make_uint2(pack_pair(w[0], w[1]), pack_pair(w[2], w[3]));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < minor) to[e] = from_f32<bf16>(w[e]);
      }
    }
  }
}

// An adapter's sums over its rows for 256 columns of x (A, as it lies) and kRanks of v
// (B: its second parts, then its first ones, into the same sums).
// kWide: the rows of x lie on 16 bytes.  kLong: a block may have more than a run of steps (8192 rows, rank 64, 4096 to 16384,
// four adapters, both calls: 331 us without, 339 with it, where no block has more).
template <int kRanks, bool kWide, bool kLong>
__global__ void __launch_bounds__(kTcThreads, kWide ? 3 : 2) k_adapt_outer_tc(const OuterPair pair) {
  pdl_wait();
  const uint32_t block = cluster_rank(), blocks = cluster_blocks();
  const int slices = (int)(blockIdx.x / blocks), second = slices >= pair.slices ? 1 : 0;
  const OuterArgs &a = pair.a[second];
  constexpr int kStage = tc_outer_stage(kRanks);
  constexpr int kTmem = kTcCols / 128 * kRanks;
  // of v: 64 ranks of a part to themselves, or the 32 of both beside each other
  constexpr uint32_t kPart = kRanks == 64 ? kTcBox : 64;
  extern __shared__ uint8_t tc_raw[];
  __shared__ uint64_t done[kTcStages];
  __shared__ uint32_t tmem_at;
  uint8_t *ring = tc_raw + ((1024 - (su32(tc_raw) & 1023)) & 1023);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int adapter = blockIdx.y, r0 = blockIdx.z * kRanks;
  const int b0 = (slices - second * pair.slices) * kTcCols;
  const int first = a.start[adapter], end = a.start[adapter + 1];
  const int step = (int)blocks * kTcRows;
  int p_first = first + (int)block * kTcRows;
  const int all_steps = p_first < end ? (end - p_first + step - 1) / step : 0;
  int steps = kLong ? min(all_steps, kTcRun) : all_steps, left_steps = all_steps;  // of the run, and from it on
  if (warp == 0) tmem_alloc(&tmem_at, kTmem);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kTcStages; ++s) mbar_init(&done[s], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  bool ok = true;
  // this warp's sums: column 32 (warp % 4) + lane of tile warp / 4
  const uint32_t own_sums = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (warp >> 2) * kRanks;
  float before[kLong ? kRanks : 1];  // of the runs before: in local memory, for registers would cost the SM's third block (360)

  // lane l: the row at place l of a step's 32 (-1 past the end)
  auto tokens_at = [&](int i) {
    const int p = p_first + i * step + lane;
    return i < steps && p < end ? __ldg(a.order + p) : -1;
  };
  // x: a warp has whole rows, a lane 8 columns; zeros past the end
  const int left = a.cols - b0 - 8 * lane;
  const bf16 *x = reinterpret_cast<const bf16 *>(a.x) + (left > 0 ? b0 + 8 * lane : 0);
  const int bytes = max(0, min(left, 8)) * 2;
  auto fetch = [&](int i, int tokens) {
    if (i < steps) {
      uint8_t *to = ring + (i % kTcStages) * kStage + (lane >> 3) * kTcBox;
      uint4 v[kTcRows / 8];
#pragma unroll
      for (int u = 0; u < kTcRows / 8; ++u) {
        const int k = warp + 8 * u, token = __shfl_sync(0xffffffffu, tokens, k);
        const bf16 *from = x + max(token, 0) * a.x_ld;
        if constexpr (kWide)
          copy_async<16>(to + k * 128 + (((lane & 7) ^ (k & 7)) << 4), from, token >= 0 ? bytes : 0);
        else
          v[u] = load_loose<true>(from, token >= 0 ? bytes / 2 : 0);
      }
      if constexpr (!kWide) {
#pragma unroll
        for (int u = 0; u < kTcRows / 8; ++u) {
          const int k = warp + 8 * u;
          *reinterpret_cast<uint4 *>(to + k * 128 + (((lane & 7) ^ (k & 7)) << 4)) = v[u];
        }
      }
    }
    fetch_commit();
  };
  // v: four ranks of a row at a time
  constexpr int kQuads = kRanks / 4, kJobs = kTcRows * kQuads / kTcThreads;
  static_assert(kJobs * kTcThreads == kTcRows * kQuads, "whole jobs");
  struct Held {
    Pack<float, 16> v[kJobs];
  };
  auto read_v = [&](int tokens, Held &held) {
#pragma unroll
    for (int u = 0; u < kJobs; ++u) {
      const int job = threadIdx.x + u * kTcThreads, k = job / kQuads, r = r0 + job % kQuads * 4;
      const int token = __shfl_sync(0xffffffffu, tokens, k);
      const bool in = token >= 0 && r < a.rank;
      held.v[u] = load_vec<float, 4>(a.v + (in ? (int64_t)token * a.rank + r : 0), in ? a.rank - r : 0, a.v_wide);
    }
  };
  auto put_v = [&](int i, const Held &held) {
    uint8_t *to = ring + (i % kTcStages) * kStage + kTcCols / 64 * kTcBox;
#pragma unroll
    for (int u = 0; u < kJobs; ++u) {
      const int job = threadIdx.x + u * kTcThreads, k = job / kQuads, r = job % kQuads * 4;
      uint32_t w[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) cut_pair<2>(held.v[u].get(2 * h), held.v[u].get(2 * h + 1), w[h]);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int c = p * kRanks + r;
        *reinterpret_cast<uint2 *>(to + (c >> 6) * kTcBox + k * 128 + ((((c >> 3) & 7) ^ (k & 7)) << 4) + (c & 7) * 2) =
            make_uint2(w[0][p], w[1][p]);
      }
    }
  };
  while (steps) {
    constexpr uint32_t kInst = tc_inst(128, kRanks, true, true);
    int ahead[kTcStages];  // the rows of steps i + 1, ..., i + kTcStages
    Held even, odd;        // v of the step in hand and of the next one
    {
      const int now = tokens_at(0);
#pragma unroll
      for (int s = 0; s < kTcStages; ++s) ahead[s] = tokens_at(s + 1);
      fetch(0, now);
      read_v(now, even);
      read_v(ahead[0], odd);
#pragma unroll
      for (int s = 1; s < kTcStages - 1; ++s) fetch(s, ahead[s - 1]);
    }
    auto step_on = [&](int i, Held &held) {
      put_v(i, held);
      fetch_wait<kTcStages - 2>();
      fence_async_shared();
      __syncthreads();
      if (threadIdx.x == 0) {
        tc_fence_after();
        const uint32_t at = su32(ring) + (i % kTcStages) * kStage;
#pragma unroll
        for (int s = 0; s < kTcRows / 16; ++s)
#pragma unroll
          for (int p = 1; p >= 0; --p)
#pragma unroll
            for (int m = 0; m < kTcCols / 128; ++m)
              tc_mma(tmem + m * kRanks, tc_desc(at + 2 * m * kTcBox + s * 2048, kTcBox),
                     tc_desc(at + kTcCols / 64 * kTcBox + s * 2048 + p * kPart, kTcBox), kInst, i > 0 || s > 0 || p == 0);
        tc_commit(&done[i % kTcStages]);
      }
      // the stage that step i - 1 has read is filled for step i + kTcStages - 1
      if (i > 0) ok = mbar_wait(&done[(i - 1) % kTcStages], ((i - 1) / kTcStages) & 1) && ok;
      fetch(i + kTcStages - 1, ahead[kTcStages - 2]);
      read_v(ahead[1], held);
#pragma unroll
      for (int s = 0; s + 1 < kTcStages; ++s) ahead[s] = ahead[s + 1];
      ahead[kTcStages - 1] = tokens_at(i + kTcStages + 1);
    };
    for (int i = 0; i < steps; i += 2) {
      step_on(i, even);
      if (i + 1 < steps) step_on(i + 1, odd);
    }
    fetch_wait<0>();
    ok = mbar_wait(&done[(steps - 1) % kTcStages], ((steps - 1) / kTcStages) & 1) && ok;
    tc_fence_after();
    if constexpr (!kLong) {
      break;
    } else {
      if (left_steps <= kTcRun) break;
      // read before the next step's barrier, behind which the next run begins
#pragma unroll 1
      for (int r = 0; r < kRanks; r += 16) {
        float v[16];
        tmem_ld16(own_sums + r, v);
        tmem_wait(v, v);
#pragma unroll
        for (int e = 0; e < 16; ++e) before[r + e] = left_steps < all_steps ? before[r + e] + v[e] : v[e];
      }
      tc_fence_before();
      left_steps -= kTcRun;
      steps = min(left_steps, kTcRun);
      p_first += kTcRun * step;
    }
  }
  ok = __syncthreads_and(ok);  // the ring becomes the sums; of a wait that gave up all of the block's are NaN
  float *sums = reinterpret_cast<float *>(ring);
  {
    const int c = 32 * warp + lane;
#pragma unroll
    for (int r = 0; r < kRanks; r += 32) {
      float v[2][16];
      if (all_steps) {
        tmem_ld16(own_sums + r, v[0]);
        tmem_ld16(own_sums + r + 16, v[1]);
        tmem_wait(v[0], v[1]);
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e >> 4][e & 15] = !ok ? NAN : all_steps ? v[e >> 4][e & 15] : 0.f;
      if (a.turned) {
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          *reinterpret_cast<float4 *>(sums + c * (kRanks + 4) + r + e) =
              make_float4(v[e >> 4][e & 15], v[e >> 4][(e & 15) + 1], v[e >> 4][(e & 15) + 2], v[e >> 4][(e & 15) + 3]);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) sums[(r + e) * (kTcCols + 4) + c] = v[e >> 4][e & 15];
      }
    }
    if (kLong && all_steps > kTcRun) {  // a loop of its own: otherwise `before` is read in any case
#pragma unroll 1
      for (int r = 0; r < kRanks; ++r) sums[a.turned ? c * (kRanks + 4) + r : r * (kTcCols + 4) + c] += before[kLong ? r : 0];
    }
  }
  tc_fence_before();
  if (blocks > 1)
    cluster_sync();
  else
    __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmem);
  }
  if (a.turned)
    tc_outer_write<kRanks, kTcCols>(a, sums, block, blocks, adapter, b0, r0, a.cols, a.rank, first == end);
  else
    tc_outer_write<kTcCols, kRanks>(a, sums, block, blocks, adapter, r0, b0, a.rank, a.cols, first == end);
  if (blocks > 1) cluster_sync();
}

template <int kRanks, bool kWide>
cudaError_t launch_outer_tc(OuterPair p, int64_t n, int32_t adapters, int sms, cudaStream_t s) {
  const size_t smem = tc_outer_smem(kRanks);
  p.slices = p.a[0].out ? (int32_t)ceil_div(p.a[0].cols, kTcCols) : 0;
  const int64_t slices = p.slices + (p.a[1].out ? ceil_div(p.a[1].cols, kTcCols) : 0);
  const int64_t ranks = ceil_div(p.a[0].rank, kRanks);
  // three blocks of an SM at a time; two rounds of them even out adapters that have more rows than others (8192 rows, rank 64,
  // 4096 to 16384, four adapters: 161 us in 320 blocks, 104 in 640, 113 in 1280; 95 with v read two steps ahead)
  const unsigned c = cluster_for(slices * ranks * adapters, ceil_div(n, (int64_t)adapters * kTcRows), 5 * sms);
  // all rows may be one adapter's
  const auto kernel = ceil_div(n, (int64_t)c * kTcRows) > kTcRun ? k_adapt_outer_tc<kRanks, kWide, true> : k_adapt_outer_tc<kRanks, kWide, false>;
  cudaError_t e = raise_smem_limit(kernel, smem);
  if (e != cudaSuccess) return e;
  return launch_cluster(c, kernel, dim3((unsigned)(slices * c), (unsigned)adapters, (unsigned)ranks), kTcThreads, smem, s,
                        (const OuterPair)p);
}

}  // namespace
}  // namespace snack
