// The adapters' products on the fifth generation tensor cores (bf16 whose rows lie on
// 16 bytes).  Included by adapt.cu.
//
// Operands are gathered row by row with cp.async into tiles with the 128-byte swizzle,
// the fp32 one cut into two bf16 parts on its way; one thread issues tcgen05.mma, the
// sums stay in tensor memory until the block's share of K is done.
#pragma once

namespace snack {
namespace {

__device__ __forceinline__ uint32_t su32(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(bar)), "r"(count) : "memory");
}
constexpr int kSpinLimit = 1 << 20;  // far above any real wait
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity) {
  const uint32_t at = su32(bar);
  for (int i = 0; i < kSpinLimit; ++i) {
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
constexpr uint32_t tc_inst(int m, int n, bool a_mn, bool b_mn) {
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

// ------------------------------------------------------------ dA and dB

constexpr int kTcCols = 256;     // columns of a block: two tiles of 128, the lanes of TMEM
constexpr int kTcRows = 32;      // rows (of K) per stage
constexpr int kTcStages = 3;
constexpr int kTcThreads = 256;
constexpr int kTcBox = kTcRows * 128;  // bytes of 64 columns of a stage
__host__ __device__ constexpr int tc_outer_stage(int ranks) { return (kTcCols + 2 * ranks) / 64 * kTcBox; }
constexpr size_t tc_outer_smem(int ranks) {
  const size_t ring = (size_t)kTcStages * tc_outer_stage(ranks), sums = std::max((size_t)ranks * (kTcCols + 4), (size_t)kTcCols * (ranks + 4)) * 4;
  return (ring > sums ? ring : sums) + 1024;
}

__device__ __forceinline__ float4 ld_cluster4(const float *p, uint32_t block) {
  uint32_t at;
  float4 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(su32(p)), "r"(block));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
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
template <int kRanks>
__global__ void __launch_bounds__(kTcThreads, 3) k_adapt_outer_tc(const OuterPair pair) {
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
  const int step = (int)blocks * kTcRows, p_first = first + (int)block * kTcRows;
  const int steps = p_first < end ? (end - p_first + step - 1) / step : 0;
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
#pragma unroll
      for (int u = 0; u < kTcRows / 8; ++u) {
        const int k = warp + 8 * u, token = __shfl_sync(0xffffffffu, tokens, k);
        copy_async<16>(to + k * 128 + (((lane & 7) ^ (k & 7)) << 4), x + max(token, 0) * a.x_ld, token >= 0 ? bytes : 0);
      }
    }
    fetch_commit();
  };
  // v: four ranks of a row at a time
  constexpr int kQuads = kRanks / 4, kJobs = kTcRows * kQuads / kTcThreads;
  static_assert(kJobs * kTcThreads == kTcRows * kQuads, "whole jobs");
  Pack<float, 16> held[kJobs];
  auto read_v = [&](int tokens) {
#pragma unroll
    for (int u = 0; u < kJobs; ++u) {
      const int job = threadIdx.x + u * kTcThreads, k = job / kQuads, r = r0 + job % kQuads * 4;
      const int token = __shfl_sync(0xffffffffu, tokens, k);
      const bool in = token >= 0 && r < a.rank;
      held[u] = load_vec<float, 4>(a.v + (in ? (int64_t)token * a.rank + r : 0), in ? a.rank - r : 0, a.v_wide);
    }
  };
  auto put_v = [&](int i) {
    uint8_t *to = ring + (i % kTcStages) * kStage + kTcCols / 64 * kTcBox;
#pragma unroll
    for (int u = 0; u < kJobs; ++u) {
      const int job = threadIdx.x + u * kTcThreads, k = job / kQuads, r = job % kQuads * 4;
      uint32_t w[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) cut_pair<2>(held[u].get(2 * h), held[u].get(2 * h + 1), w[h]);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int c = p * kRanks + r;
        *reinterpret_cast<uint2 *>(to + (c >> 6) * kTcBox + k * 128 + ((((c >> 3) & 7) ^ (k & 7)) << 4) + (c & 7) * 2) =
            make_uint2(w[0][p], w[1][p]);
      }
    }
  };
  if (steps) {
    constexpr uint32_t kInst = tc_inst(128, kRanks, true, true);
    int ahead[kTcStages];  // the rows of steps i + 1, ..., i + kTcStages
    {
      const int now = tokens_at(0);
#pragma unroll
      for (int s = 0; s < kTcStages; ++s) ahead[s] = tokens_at(s + 1);
      fetch(0, now);
      read_v(now);
#pragma unroll
      for (int s = 1; s < kTcStages - 1; ++s) fetch(s, ahead[s - 1]);
    }
    for (int i = 0; i < steps; ++i) {
      put_v(i);
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
      read_v(ahead[0]);
#pragma unroll
      for (int s = 0; s + 1 < kTcStages; ++s) ahead[s] = ahead[s + 1];
      ahead[kTcStages - 1] = tokens_at(i + kTcStages + 1);
    }
    fetch_wait<0>();
    ok = mbar_wait(&done[(steps - 1) % kTcStages], ((steps - 1) / kTcStages) & 1) && ok;
    tc_fence_after();
  }
  __syncthreads();  // the ring becomes the sums
  float *sums = reinterpret_cast<float *>(ring);
  {
    const int tile = warp >> 2, c = 128 * tile + 32 * (warp & 3) + lane;
    const uint32_t from = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + tile * kRanks;
#pragma unroll
    for (int r = 0; r < kRanks; r += 32) {
      float v[2][16];
      if (steps) {
        tmem_ld16(from + r, v[0]);
        tmem_ld16(from + r + 16, v[1]);
        tmem_wait(v[0], v[1]);
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e >> 4][e & 15] = !ok ? NAN : steps ? v[e >> 4][e & 15] : 0.f;
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

template <int kRanks>
cudaError_t launch_outer_tc(OuterPair p, int64_t n, int32_t adapters, int sms, cudaStream_t s) {
  const size_t smem = tc_outer_smem(kRanks);
  const auto kernel = k_adapt_outer_tc<kRanks>;
  cudaError_t e = raise_smem_limit(kernel, smem);
  if (e != cudaSuccess) return e;
  p.slices = p.a[0].out ? (int32_t)ceil_div(p.a[0].cols, kTcCols) : 0;
  const int64_t slices = p.slices + (p.a[1].out ? ceil_div(p.a[1].cols, kTcCols) : 0);
  const int64_t ranks = ceil_div(p.a[0].rank, kRanks);
  // three blocks of an SM at a time; two rounds of them even out adapters that have more rows than others (8192 rows, 64 of
  // 4096 to 16384, four adapters: 161 us in 320 blocks, 104 in 640, 113 in 1280)
  const unsigned c = cluster_for(slices * ranks * adapters, ceil_div(n, (int64_t)adapters * kTcRows), 5 * sms);
  return launch_cluster(c, kernel, dim3((unsigned)(slices * c), (unsigned)adapters, (unsigned)ranks), kTcThreads, smem, s,
                        (const OuterPair)p);
}

}  // namespace
}  // namespace snack
