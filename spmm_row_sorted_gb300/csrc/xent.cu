// Softmax cross entropy of a projection to a vocabulary, and its gradient,
// in pieces of the vocabulary; the logits are never kept.
//
//   z[i, v]  = sum_d x[i, d] w[v, d]
//   lse[i]   = log sum_v exp z[i, v],   loss[i] = lse[i] - z[i, t_i]
//   dz[i, v] = g_i (exp(z[i, v] - lse[i]) - [v = t_i])
//   dx = dz w,   dw = dz^T x
//
// Four matrix products of 2 n V D operations each on the tensor cores (the
// forward's logits, the same again for the gradient, dx and dw), all by one
// kernel with four epilogues:
//   stats  keeps of a logits tile only each row's maximum and sum of
//          exponentials, per half tile, without the target's;
//   dlog   turns a logits tile into dz, stored as bf16 for one piece of the
//          vocabulary (one part for bf16 operands, 2^-9 of an entry: dw of 4096 x
//          131072 x 2048 then lies 0.0019 from 64 bits, where its own rounding gives
//          0.0016; a second part would double both products that read dz; dx takes
//          what the target's entry lost at the end);
//   dx     adds dz w of the piece to fp32 sums (a TMA reduction: one addition
//          per element and piece, in the pieces' order);
//   dw     writes the piece's rows of dw.
// Bound by the tensor cores; for a few tokens by reading w once (a few fp32
// tokens: xent_small.cuh and xent_cut.cuh).
//
// A pair of CTAs, one per SM, works through output tiles of 256 x up to 256,
// 128 rows each.  In each CTA a warp loads its rows of A and its half of B by TMA
// into a ring of stages; one thread of the pair issues the tcgen05.mma, which
// read both halves of B (a third fewer bytes from L2 than a tile per CTA: dx and
// dw went from 1463 and 1509 to 1388 and 1362 us at 4096 x 131072 x 2048); and
// eight warps run the epilogue of one accumulator from one half of the tensor
// memory while the next one forms in the other.  Operands whose rows run along K
// are K-major tiles (128-byte swizzle), the others (w for dx, dz^T and x for dw)
// are read as they lie, as MN-major tiles: no transposes.
//
// The tensor core's fp32 accumulation rounds towards zero, which over a long K
// is a bias: a sum of 4096 products came out 5e-6 to 1.4e-5 of itself too small.
// So an accumulator takes at most 512 of K (32 instructions; 256 for the losses of
// fp32 operands) where that counts, and the epilogue's warps add the partial
// sums in registers, rounding to nearest, while the next one forms in the other
// half of the tensor memory.  What is left is at most 1e-6 of a logit (unit_of).
// The target's logit, of which loss and dz = p - 1 are small differences, does not
// come from there: a warp per row forms it in fp32 (target_logit), the same bits for
// the loss and the gradient.  (With it from the tensor core the losses of 2048 x 65536 x
// 4096 were 1.2e-6 of themselves off, so they are 1.8e-7.)
//
// fp32 operands are cut into three bf16 parts each (8 significant bits at a
// time, 24 in all), and a product is the sum of the six part products down to
// 2^-16 of the leading one, the smaller ones summed apart; what is left out is
// below 2^-24.  All six go over 512 of K before the next 512, so that the parts
// of w that the SMs work on stay in L2.
// The parts, and bf16 operands whose rows are not 16-byte aligned, are laid
// out in the workspace, w's by pieces of the vocabulary; so is the gradient's x,
// without the rows that are not trained on.
//
// Every wait on an mbarrier is bounded; when one runs out the CTA marks its
// error word, waits (bounded) for what it has in flight, frees its tensor
// memory and returns, and the kernel that finishes a call makes the losses, dx
// and the first row of dw NaN.
#include <cuda.h>
#include <math.h>

#include <algorithm>

#include "internal.hpp"
#include "lm.hpp"
#include "xent_cut.cuh"
#include "xent_small.cuh"

namespace snack {
namespace {

// ------------------------------------------------------------ PTX wrappers

__device__ __forceinline__ uint32_t su32(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t *bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// the address, in the cluster's shared memory, of the pair leader's copy of `p`
__device__ __forceinline__ uint32_t at_leader(const void *p) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(su32(p)));
  return r;
}
__device__ __forceinline__ void mbar_arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
constexpr int kSpinLimit = 1 << 20;  // try_wait rounds before a wait is declared stuck (far above any real wait)
__device__ __forceinline__ bool mbar_try(uint64_t *bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(done)
      : "r"(su32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity) {
  for (int i = 0; i < kSpinLimit; ++i)
    if (mbar_try(bar, parity)) return true;
  return false;
}
// the same for a converged warp, with one answer for all its lanes
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
  return __any_sync(0xffffffffu, mbar_wait(bar, parity));
}
// one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, q;\n}" : "=r"(p));
  return p != 0;
}
// into this CTA's shared memory; the bytes count on the barrier at `bar`, in either CTA of the pair
__device__ __forceinline__ void tma_load(void *dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3, %4}], [%5];" ::"r"(su32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap *map, const void *src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(su32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void tma_add(const CUtensorMap *map, const void *src, int x, int y, int z) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(su32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// all but the newest `kLeft` stores have read their shared memory
template <int kLeft>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_alloc(uint32_t *dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(dst)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Shared-memory descriptor of an operand tile with the 128-byte swizzle:
// start (16-byte units), leading and stride byte offsets, version 1, layout
// type 2.  K-major: 128-byte rows of 64 K elements, 8 rows to a 1024-byte
// atom, stride 1024 from atom to atom (the leading offset is not used).
// MN-major: boxes of 64 K rows of 64 MN elements (128 bytes each); 8 K rows
// to an atom, stride 1024 from one to the next along K, and the leading
// offset is the 8192 bytes from one box of 64 MN elements to the next.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // stride, version, layout
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, bool mn_major) {
  return ((saddr & 0x3FFFF) >> 4) | ((mn_major ? (8192u >> 4) : 1u) << 16);
}
// D (TMEM) (+)= A (smem) * B (smem)^T, bf16 with fp32 accumulation, over the
// pair of CTAs: 256 rows, 128 of A and of D in each; half of B's rows in each
__device__ __forceinline__ void umma(uint32_t taddr, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n}" ::"r"(taddr),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
// arrive on both CTAs' *bar once every MMA issued so far by this thread has completed
__device__ __forceinline__ void umma_commit(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(su32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// 32 consecutive fp32 columns of this thread's TMEM lane; not there before tmem_wait and tmem_ready
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// ties a load's registers to the wait before it: no use of them moves above
__device__ __forceinline__ void tmem_ready(float (&v)[32]) {
  asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]),
        "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]),
        "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]),
        "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));
}
__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Instruction descriptor of kind::f16: fp32 accumulator (bit 4), A and B bf16
// (bits 7 and 10), MN-major A and B (bits 15 and 16), N / 8 at bit 17, M / 16 at bit 24.
__device__ __forceinline__ uint32_t inst_desc(int m, int n, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// ------------------------------------------------------------------ kernel

constexpr int kM = 256;           // rows of an output tile: 128 (the TMEM lanes) in each CTA of the pair
constexpr int kMCta = kM / 2;
constexpr int kNMax = 256;        // columns of the widest output tile
constexpr int kKb = 64;           // K per stage
constexpr int kEpiWarps = 8;
constexpr int kChunks = kNMax / 2 / 32;  // 32-column chunks of an epilogue warp's half tile
constexpr int kThreads = (kEpiWarps + 4) * 32;  // and a warpgroup for the loads and the MMAs (two of its warps idle)
// An epilogue thread keeps 128 sums; launched with 168 registers each, the
// third warpgroup gives most of its own to the other two (384 * 168 in all).
constexpr int kEpiRegs = 232, kIssueRegs = 40;
static_assert(256 * kEpiRegs + 128 * kIssueRegs <= kThreads * 168, "the split stays within the launch's registers");
constexpr int kStageA = kMCta * kKb * 2;
constexpr int kRing = 6 * (kStageA + kNMax / 2 * kKb * 2);  // bytes of the ring of stages
constexpr int kMaxStages = 16;
constexpr int kStaging = 4096;    // an epilogue warp's 32 rows x 128 bytes on their way out
constexpr int kBarBytes = 512;
constexpr int kSmem = 1024 + kRing + kEpiWarps * kStaging + kBarBytes;
static_assert(kSmem <= 232448, "shared memory of one CTA");
static_assert(kStageA <= kEpiWarps * kStaging, "a short A tile's reads end within the CTA's shared memory");

enum { kStats = 0, kDlog = 1, kDx = 2, kDw = 3, kScore = 4 };  // kScore: score.cuh

// The factor common to all rows of dz (sum and mean): a product of up to two
// device values.  It is applied to the finished sums, so dz itself lies in
// [-1, 1] and its rounding to bf16 is not the same for every row.
struct Factor {
  const float *a, *b;  // null: 1
  __device__ __forceinline__ float get() const { return (a ? *a : 1.f) * (b ? *b : 1.f); }
};

// The vocabulary rows that are targets, for the rows of dw that are finished apart (score.cuh).
struct Hits {
  int32_t *first, *last;  // [vocab] the first and the last row of x with the target (first: beyond all rows, if none); null: none
  float *rows;            // [n][ld] such a row's sums, at its first row of x
  int64_t ld;
};

struct GemmArgs {
  int32_t m, n;             // rows and columns of the product
  int32_t nt;               // columns of a tile: a multiple of 32 (128 or 256 where B is MN-major)
  int32_t a_rows;           // rows of A loaded per CTA: 128, or fewer where m has fewer (K-major A)
  int32_t m_tiles, n_tiles, n_split;
  int32_t k_blocks;         // of 64
  int32_t products;         // part products per element (1: bf16, 6: fp32)
  uint32_t a_part, b_part;  // 4 bits per product: its parts
  int32_t unit;             // K stages summed on the tensor core before the sums move to registers: of the smaller
                            // part products together, then of the leading one
  int32_t stages;
  uint32_t *err;            // [256] error words, one per CTA
  int32_t first;            // the call's first launch writes every error word
  // stats
  float2 *part;             // [slots][m] (maximum, sum of exp(z - maximum)) per half tile
  int32_t slot0;
  // stats, dlog, dw
  TokenSrc targets;
  int32_t v0;               // first vocabulary row of the piece
  // dlog
  const float *lse, *hot;   // [m] each, hot: dz at the target
  Entropy ent;
  const float *dloss;       // upstream gradient of each row, or null (1: a common factor is applied to the sums)
  int32_t out_parts;        // bf16 parts of dz
  // dx
  int32_t add;              // add to the sums (else write them)
  // dw
  Factor factor;
  int32_t tokens;           // of `targets`
  void *out;                // first row of the piece; used where TMA cannot store
  int64_t out_ld;
  int32_t out_wide;         // fp32 (else bf16)
  int32_t out_tma;
  Hits hits;
  // score
  float4 *stats;            // [m][slots] (maximum, how often, sum of exp(z - maximum) of the others, sum of it times z - maximum)
  float *high;              // [m][high_ld] maximum of 32 neighbouring logits each, or null: then no logits are kept
  int64_t stats_ld, high_ld;
};

// the six part products, smallest first: parts (2,0) (1,1) (0,2) (1,0) (0,1) (0,0)
constexpr uint32_t kPartA = 0x001012u, kPartB = 0x010210u;

// Byte offset of 16-byte chunk c of row r in a warp's staging tile (32 rows
// of 128 bytes, 128-byte swizzle: what the store's tensor map undoes).
__device__ __forceinline__ uint32_t stage_off(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// Whether a row is trained on at all (a converged warp; mostly its first look answers).
__device__ __forceinline__ bool any_trained(const TokenSrc &targets, int32_t n) {
  for (int32_t i = threadIdx.x & 31; __any_sync(0xffffffffu, i < n); i += 32)
    if (__any_sync(0xffffffffu, i < n && targets.key(i) < targets.vocab)) return true;
  return false;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// One product.  4096 tokens against 131072 x 2048 bf16: 1.11 to 1.2 ms each of
// the four, 1.7 to 1.9 PFLOP/s as the power allows (90 % of the tensor cores'
// cycles; 80 to 88 % where partial sums are read).
template <int kMode>
__device__ __forceinline__ void product(const CUtensorMap &map_a, const CUtensorMap &map_b, const CUtensorMap &map_o,
                                        const GemmArgs &P) {
  pdl_wait();
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  constexpr bool kAmn = kMode == kDw, kBmn = kMode == kDx || kMode == kDw;
  const uint32_t rank = cta_rank();  // 0: the leader, which issues the pair's MMAs
  const int nb = P.nt / 2;           // rows of B in each CTA
  // With few rows a stage holds only those of A: the MMAs read 128 rows all the
  // same, whatever lies in the others' place, and those rows are never used.
  const uint32_t a_bytes = (uint32_t)(P.a_rows * kKb * 2);
  const uint32_t stage_bytes = a_bytes + (uint32_t)(nb * kKb * 2);
  uint8_t *staging = smem + kRing;
  uint64_t *full = reinterpret_cast<uint64_t *>(staging + kEpiWarps * kStaging);
  uint64_t *empty = full + kMaxStages;
  uint64_t *acc_full = empty + kMaxStages;  // [2]
  uint64_t *acc_free = acc_full + 2;        // [2]
  uint64_t *drained = acc_free + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drained + 1);
  int *bad = reinterpret_cast<int *>(tmem_slot + 1);
  static_assert(8 * (2 * kMaxStages + 5) + 16 <= kBarBytes, "barriers and flags fit their bytes");

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_free[b], 2 * kEpiWarps);
    }
    mbar_init(drained, 1);
    *bad = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  pair_sync();  // both CTAs' barriers are ready
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int tiles = P.m_tiles * P.n_tiles * P.n_split;
  const int per_split = (P.k_blocks + P.n_split - 1) / P.n_split;
  bool ok = true;
  // a tile: its row and column of tiles, its share of K; neighbours in the
  // order share the operand that the other dimension re-reads
  struct Tile {
    int m0, n0, split, k0, nk;
  };
  auto tile_at = [&](int t) {
    Tile r;
    r.split = t / (P.m_tiles * P.n_tiles);
    const int mn = t - r.split * (P.m_tiles * P.n_tiles);
    if (kMode == kDx || kMode == kDw) {  // columns (D) run fastest: a row of tiles shares its part of dz
      r.m0 = mn / P.n_tiles * kM;
      r.n0 = mn % P.n_tiles * P.nt;
    } else {
      r.m0 = mn % P.m_tiles * kM;
      r.n0 = mn / P.m_tiles * P.nt;
    }
    r.k0 = r.split * per_split;
    r.nk = max(0, min(P.k_blocks, r.k0 + per_split) - r.k0);
    return r;
  };

  if (warp >= kEpiWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    // The whole warp runs each loop, so that addresses and descriptors stay in
    // uniform registers, and one lane issues: with the loops inside a one-lane
    // branch the MMA warp needed 730 cycles for a stage's 512 of MMAs.
    const bool one = elect_one();
    int s = 0;           // stage
    uint32_t phase = 0;  // of its barriers
    if (warp == kEpiWarps) {  // ------------------------------------------- loads
      const uint32_t bar0 = at_leader(full);  // the leader's barriers count both CTAs' bytes
      for (int t = blockIdx.x / 2; t < tiles && ok; t += gridDim.x / 2) {
        const Tile q = tile_at(t);
        const int am = q.m0 + (int)rank * kMCta, bn = q.n0 + (int)rank * nb;
        for (int k0 = 0; k0 < q.nk && ok; k0 += P.unit) {
          const int k1 = min(q.nk, k0 + P.unit);
          for (int c = 0; c < P.products && ok; ++c) {
            const int za = (P.a_part >> (4 * c)) & 15, zb = (P.b_part >> (4 * c)) & 15;
            for (int k = (q.k0 + k0) * kKb; k < (q.k0 + k1) * kKb; k += kKb) {
              if (!warp_wait(&empty[s], phase ^ 1)) {
                ok = false;
                break;
              }
              if (one) {
                uint8_t *a = smem + (uint32_t)s * stage_bytes, *b = a + a_bytes;
                const uint32_t bar = bar0 + 8u * s;
                if (rank == 0) mbar_expect_tx(&full[s], 2 * stage_bytes);
                if (kAmn) {
                  tma_load(a, &map_a, am, k, za, bar);
                  tma_load(a + 8192, &map_a, am + 64, k, za, bar);
                } else {
                  tma_load(a, &map_a, k, am, za, bar);
                }
                if (kBmn) {
                  tma_load(b, &map_b, bn, k, zb, bar);
                  if (nb > 64) tma_load(b + 8192, &map_b, bn + 64, k, zb, bar);
                } else {
                  tma_load(b, &map_b, k, bn, zb, bar);
                }
              }
              __syncwarp();
              if (++s == P.stages) {
                s = 0;
                phase ^= 1;
              }
            }
          }
        }
      }
    } else if (warp == kEpiWarps + 1 && rank == 0) {  // ------------------- MMAs
      const uint32_t idesc = inst_desc(kM, P.nt, kAmn, kBmn);
      const uint32_t a_lo = desc_lo(su32(smem), kAmn), b_lo = desc_lo(su32(smem) + a_bytes, kBmn);
      constexpr uint32_t kA16 = kAmn ? 128 : 2, kB16 = kBmn ? 128 : 2;  // 16 of K in 16-byte units: 16 rows, or 32 bytes
      int n_acc = 0;
      for (int t = blockIdx.x / 2; t < tiles && ok; t += gridDim.x / 2) {
        const Tile q = tile_at(t);
        const int steps = P.products * q.nk;
        int i = 0;
        bool seen = false;  // the next stage's bytes are there
        for (int k0 = 0; k0 < q.nk && ok; k0 += P.unit) {
          const int len = min(P.unit, q.nk - k0);
          // the smaller part products (if any) in one accumulator, the leading one in the next
          for (int unit = P.products > 1 ? 0 : 1; unit < 2 && ok; ++unit, ++n_acc) {
            const int buf = n_acc & 1;
            if (!warp_wait(&acc_free[buf], ((n_acc >> 1) & 1) ^ 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t d = tmem + (uint32_t)(buf * kNMax);
            const int end = i + (unit ? len : (P.products - 1) * len);
            uint32_t more = 0;  // the unit's first MMA overwrites
            while (i < end) {
              if (!__any_sync(0xffffffffu, seen) && !warp_wait(&full[s], phase)) {
                ok = false;
                break;
              }
              const uint32_t off = (uint32_t)s * (stage_bytes >> 4);
              const int cur = s;
              if (++s == P.stages) {
                s = 0;
                phase ^= 1;
              }
              seen = ++i < steps && mbar_try(&full[s], phase);  // answered while the MMAs below are issued
              if (one) {
#pragma unroll
                for (int k = 0; k < kKb / 16; ++k)
                  umma(d, a_lo + off + k * kA16, b_lo + off + k * kB16, idesc, k == 0 ? more : 1u);
                umma_commit(&empty[cur]);
              }
              __syncwarp();
              more = 1;
            }
            if (ok && one) umma_commit(&acc_full[buf]);
            __syncwarp();
          }
        }
      }
      if (one) umma_commit(drained);
      __syncwarp();
    }
  } else {  // -------------------------------------------------------- epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    const int quarter = warp & 3, half = warp >> 2;  // TMEM lanes 32 quarter .. +31; half of the columns
    uint8_t *stage = staging + warp * kStaging;
    constexpr float kLog2e = 1.4426950408889634f;
    int n_acc = 0;
    uint32_t n_store = 0;
    for (int t = blockIdx.x / 2; t < tiles && ok; t += gridDim.x / 2) {
      const Tile q = tile_at(t);
      if (q.nk == 0) continue;
      const int m0 = q.m0 + (int)rank * kMCta;  // this CTA's rows
      const int row = m0 + quarter * 32 + lane;
      const bool row_ok = row < P.m;
      const int width0 = (P.nt / 32 + 1) / 2 * 32;  // columns of the first half
      const int c_end = half ? P.nt - width0 : width0;
      const int col0 = q.n0 + half * width0;
      // the target's column of this tile's half, or below zero
      int tcol = -1;
      float lse = 0.f, g = 0.f, hot = 0.f;
      float went = 0.f, ent = 0.f;
      if (kMode == kStats || kMode == kDlog || kMode == kScore) {
        if (row_ok && (kMode != kScore || P.targets.ids)) {
          const uint32_t id = P.targets.key(row);
          if (id < P.targets.vocab) {
            tcol = (int)id - P.v0 - col0;  // beyond c_end: another half's
            if (kMode == kDlog) {
              lse = P.lse[row];
              g = P.dloss ? P.dloss[row] : 1.f;
              hot = P.hot[row];
              if (P.ent.weight) {
                went = P.ent.weight[row];
                ent = P.ent.value[row];
              }
            }
          }
        }
      }
      // the tile's sums: one unit after the other, added in fp32
      float acc[kChunks][32];
      const int units = (q.nk + P.unit - 1) / P.unit * (P.products > 1 ? 2 : 1);
      for (int u = 0; u < units; ++u, ++n_acc) {
        const int buf = n_acc & 1;
        if (!warp_wait(&acc_full[buf], (n_acc >> 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t from = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(buf * kNMax + half * width0);
        const int chunks = c_end / 32;
        auto release = [&] {  // the accumulator has been read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_at(at_leader(&acc_free[buf]));
        };
        __syncwarp();
        if (u == 0) {  // all loads in flight at once; later units two at a time (their sums need registers too)
#pragma unroll
          for (int h = 0; h < kChunks; ++h)
            if (h < chunks) tmem_ld32(from + 32u * h, acc[h]);
          tmem_wait();
          release();
#pragma unroll
          for (int h = 0; h < kChunks; ++h) tmem_ready(acc[h]);
        } else {
#pragma unroll
          for (int h = 0; h < kChunks; h += 2) {
            if (h >= chunks) break;
            float v[2][32];
            tmem_ld32(from + 32u * h, v[0]);
            if (h + 1 < chunks) tmem_ld32(from + 32u * (h + 1), v[1]);
            tmem_wait();
            if (h + 2 >= chunks) release();
            tmem_ready(v[0]);
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[h][j] += v[0][j];
            if (h + 1 < chunks) {
              tmem_ready(v[1]);
#pragma unroll
              for (int j = 0; j < 32; ++j) acc[h + 1][j] += v[1][j];
            }
          }
        }
      }
      if (!ok) break;
      if (kMode == kStats) {
        float mx = -INFINITY, sum = 0.f;
#pragma unroll
        for (int h = 0; h < kChunks; ++h) {
          const int c = 32 * h;
          if (c >= c_end) break;
          float(&v)[32] = acc[h];
          const int valid = P.n - col0 - c;
          if (valid < 32) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j >= valid) v[j] = -INFINITY;
          }
          if (tcol >= c && tcol < c + 32) {  // joined later
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (tcol == c + j) v[j] = -INFINITY;
          }
          float m4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
          for (int j = 4; j < 32; ++j) m4[j & 3] = fmaxf(m4[j & 3], v[j]);
          const float nm = fmaxf(mx, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
          const float base = nm == -INFINITY ? 0.f : nm;  // a row of -inf so far: every term is 0
          float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 32; ++j) s4[j & 3] += ex2((v[j] - base) * kLog2e);
          sum = sum * ex2((mx - base) * kLog2e) + ((s4[0] + s4[1]) + (s4[2] + s4[3]));
          mx = nm;
        }
        if (row_ok)
          P.part[(size_t)(P.slot0 + 2 * (q.n0 / P.nt) + half) * (size_t)P.m + row] = make_float2(mx, sum);
      } else if (kMode == kScore) {
        const int slot = 2 * (q.n0 / P.nt) + half;
        float high[kChunks], mx = -INFINITY;
#pragma unroll
        for (int h = 0; h < kChunks; ++h) {
          const int c = 32 * h;
          high[h] = -INFINITY;
          if (c >= c_end) continue;
          float(&v)[32] = acc[h];
          if (P.high) {  // the logits as they are
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int ch = 0; ch < 8; ++ch)
              *reinterpret_cast<float4 *>(stage + stage_off(lane, ch)) =
                  make_float4(v[4 * ch], v[4 * ch + 1], v[4 * ch + 2], v[4 * ch + 3]);
            fence_async_shared();
            __syncwarp();
            if (lane == 0 && col0 + c < P.n && m0 + quarter * 32 < P.m) {
              tma_store(&map_o, stage, col0 + c, m0 + quarter * 32, 0);
              bulk_commit();
            }
          }
          const int valid = P.n - col0 - c;
          if (valid < 32) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j >= valid) v[j] = -INFINITY;
          }
          auto largest = [&] {
            float m4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
            for (int j = 4; j < 32; ++j) m4[j & 3] = fmaxf(m4[j & 3], v[j]);
            return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          };
          float top = largest();
          high[h] = top;
          if (tcol >= c && tcol < c + 32) {  // joined later
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (tcol == c + j) v[j] = -INFINITY;
            top = largest();
          }
          mx = fmaxf(mx, top);
        }
        // the maximum apart from the rest: of a confident row's sums the rest is what counts
        const float base = mx == -INFINITY ? 0.f : mx;
        float often = 0.f, rest[2] = {0.f, 0.f}, slope[2] = {0.f, 0.f};
#pragma unroll
        for (int h = 0; h < kChunks; ++h) {
          if (32 * h >= c_end) break;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float d = acc[h][j] - base, e = ex2(d * kLog2e);
            if (d == 0.f && mx != -INFINITY)
              often += 1.f;
            else
              rest[j & 1] += e;
            slope[j & 1] = fmaf(e, fmaxf(d, kFarBelow), slope[j & 1]);
          }
        }
        if (row_ok) {
          P.stats[(size_t)row * (size_t)P.stats_ld + P.slot0 + slot] = make_float4(mx, often, rest[0] + rest[1], slope[0] + slope[1]);
          if (P.high)
#pragma unroll
            for (int h = 0; h < kChunks; ++h)
              if (32 * h < c_end) P.high[(size_t)row * (size_t)P.high_ld + (col0 / 32 + h)] = high[h];
        }
      } else if (kMode == kDlog) {
#pragma unroll
        for (int h = 0; h < kChunks; ++h) {
          const int c = 32 * h;
          if (c >= c_end) break;
          float(&v)[32] = acc[h];
          if (P.ent.weight) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = ex2((v[j] - lse) * kLog2e) * entropy_slope(g, went, v[j] - lse, ent);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = g * ex2((v[j] - lse) * kLog2e);
          }
          if (tcol >= c && tcol < c + 32) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (tcol == c + j) v[j] = hot;
          }
          if (g == 0.f && went == 0.f) {  // not trained on, whatever its logits
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0.f;
          }
          // 32 rows x 64 bytes per store, from two buffers in turn
          for (int part = 0; part < P.out_parts; ++part) {
            uint8_t *to = stage + (n_store++ & 1) * (kStaging / 2);
            if (lane == 0) bulk_wait_read<1>();
            __syncwarp();
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
              uint4 u;
              u.x = pack_bf16(v[8 * ch], v[8 * ch + 1]);
              u.y = pack_bf16(v[8 * ch + 2], v[8 * ch + 3]);
              u.z = pack_bf16(v[8 * ch + 4], v[8 * ch + 5]);
              u.w = pack_bf16(v[8 * ch + 6], v[8 * ch + 7]);
              *reinterpret_cast<uint4 *>(to + lane * 64 + ((ch ^ ((lane >> 1) & 3)) << 4)) = u;
              if (P.out_parts > 1) {  // what the part leaves over
                v[8 * ch] -= bf16_lo(u.x);
                v[8 * ch + 1] -= bf16_hi(u.x);
                v[8 * ch + 2] -= bf16_lo(u.y);
                v[8 * ch + 3] -= bf16_hi(u.y);
                v[8 * ch + 4] -= bf16_lo(u.z);
                v[8 * ch + 5] -= bf16_hi(u.z);
                v[8 * ch + 6] -= bf16_lo(u.w);
                v[8 * ch + 7] -= bf16_hi(u.w);
              }
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0 && col0 + c < P.n && m0 + quarter * 32 < P.m) {
              tma_store(&map_o, to, col0 + c, m0 + quarter * 32, part);
            }
            if (lane == 0) bulk_commit();  // an empty group where nothing was stored keeps the buffers' turns
          }
        }
      } else {
        const bool wide = kMode == kDx || P.out_wide;
        if (kMode == kDw) {
          float f = P.factor.get();
          if (!isfinite(f) && !any_trained(P.targets, P.tokens)) f = 0.f;  // sums of nothing stay 0
#pragma unroll
          for (int h = 0; h < kChunks; ++h)
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[h][j] *= f;
          if (P.hits.first) {
            const int first = row_ok ? P.hits.first[P.v0 + row] : P.tokens;
            if (first < P.tokens) {
              float *to = P.hits.rows + (int64_t)first * P.hits.ld + col0;
#pragma unroll
              for (int h = 0; h < kChunks; ++h)
#pragma unroll
                for (int j = 0; j < 32; j += 4)
                  if (32 * h < c_end && col0 + 32 * h + j < P.n)
                    *reinterpret_cast<float4 *>(to + 32 * h + j) = make_float4(acc[h][j], acc[h][j + 1], acc[h][j + 2], acc[h][j + 3]);
            }
          }
        }
        const int step = wide ? 32 : 64;  // columns of 128 bytes
#pragma unroll
        for (int h = 0; h < kChunks; ++h) {
          const int c = 32 * h;
          if (c >= c_end) break;
          float(&v)[32] = acc[h];
          if (lane == 0 && (c % step) == 0) bulk_wait_read<0>();
          __syncwarp();
          if (wide) {
#pragma unroll
            for (int ch = 0; ch < 8; ++ch)
              *reinterpret_cast<float4 *>(stage + stage_off(lane, ch)) =
                  make_float4(v[4 * ch], v[4 * ch + 1], v[4 * ch + 2], v[4 * ch + 3]);
          } else {
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
              uint4 u;
              u.x = pack_bf16(v[8 * ch], v[8 * ch + 1]);
              u.y = pack_bf16(v[8 * ch + 2], v[8 * ch + 3]);
              u.z = pack_bf16(v[8 * ch + 4], v[8 * ch + 5]);
              u.w = pack_bf16(v[8 * ch + 6], v[8 * ch + 7]);
              *reinterpret_cast<uint4 *>(stage + stage_off(lane, ch + ((c & 32) >> 3))) = u;
            }
          }
          if ((c + 32) % step != 0) continue;  // the row's other half first
          const int x0 = col0 + c / step * step;
          if (kMode == kDx || P.out_tma) {
            fence_async_shared();
            __syncwarp();
            if (lane == 0 && x0 < P.n && m0 + quarter * 32 < P.m) {
              if (kMode == kDx && P.add)
                tma_add(&map_o, stage, x0, m0 + quarter * 32, q.split);
              else
                tma_store(&map_o, stage, x0, m0 + quarter * 32, kMode == kDx ? q.split : 0);
              bulk_commit();
            }
          } else {  // rows that TMA cannot address: a warp writes one after the other
            __syncwarp();
            const int rows = x0 < P.n ? min(32, P.m - (m0 + quarter * 32)) : 0;
            const int64_t first = (int64_t)(m0 + quarter * 32) * P.out_ld + x0;
            if (wide) {
#pragma unroll 4
              for (int r = 0; r < rows; ++r)
                if (x0 + lane < P.n)
                  reinterpret_cast<float *>(P.out)[first + r * P.out_ld + lane] =
                      *reinterpret_cast<const float *>(stage + stage_off(r, lane >> 2) + (lane & 3) * 4);
            } else {
              for (int r = 0; r < rows; ++r)
                for (int j = lane; j < step && x0 + j < P.n; j += 32)
                  reinterpret_cast<uint16_t *>(P.out)[first + r * P.out_ld + j] =
                      *reinterpret_cast<const uint16_t *>(stage + stage_off(r, j >> 3) + (j & 7) * 2);
            }
            __syncwarp();
          }
        }
      }
    }
    if (lane == 0) bulk_wait();
  }
  if (!ok) *bad = 1;
  __syncthreads();
  if (threadIdx.x == 0) {
    bool failed = *bad != 0;
    // the leader's last commit: every MMA of the pair and every arrival on this
    // CTA's barriers is done (bounded; after a failure, a millisecond more for
    // loads that are still in flight)
    const bool rest = mbar_wait(drained, 0);
    failed = failed || !rest;
    if (failed)
      for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    if (P.first) {
      for (int e = blockIdx.x; e < 256; e += gridDim.x) P.err[e] = failed ? 1u : 0u;
    } else if (failed) {
      P.err[blockIdx.x & 255] = 1u;
    }
  }
  tc_fence_before();
  __syncthreads();
  pair_sync();  // nothing of either CTA is still at work in the other's memory
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

template <int kMode>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) k_xent(const __grid_constant__ CUtensorMap map_a,
                                                      const __grid_constant__ CUtensorMap map_b,
                                                      const __grid_constant__ CUtensorMap map_o, const GemmArgs P) {
  product<kMode>(map_a, map_b, map_o, P);
}
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) k_score(const __grid_constant__ CUtensorMap map_a,
                                                      const __grid_constant__ CUtensorMap map_b,
                                                      const __grid_constant__ CUtensorMap map_o, const GemmArgs P) {
  product<kScore>(map_a, map_b, map_o, P);
}

__device__ __forceinline__ bool any_error(const uint32_t *err) {
  if (!err) return false;  // no product ran on the tensor cores
  uint32_t e = 0;
  for (int i = threadIdx.x; i < 256; i += blockDim.x) e |= err[i];
  return __syncthreads_or((int)e) != 0;
}

// The logit of a row's target, by a warp: 32 sums in fp32, added at the end, in an
// order that does not depend on how the rows lie.
struct TargetLogit {
  const void *x, *w;  // x null: there is none to form
  int64_t x_ld, w_ld;
  int32_t width;
  int bf, x_wide, w_wide;  // bf16 operands; rows 16-byte aligned
  template <typename T>
  static __device__ __forceinline__ Pack<T, 16> some(const T *row, int g, int32_t width, int wide) {
    constexpr int kN = 16 / (int)sizeof(T);
    Pack<T, 16> p;
    if (wide && (g + 1) * kN <= width) {
      p.raw = __ldg(reinterpret_cast<const uint4 *>(row) + g);
    } else {
#pragma unroll
      for (int e = 0; e < kN; ++e) p.set(e, g * kN + e < width ? to_f32(row[g * kN + e]) : 0.f);
    }
    return p;
  }
  template <typename T>
  __device__ __forceinline__ float dot(int64_t row, uint32_t id) const {
    constexpr int kN = 16 / (int)sizeof(T);
    const T *a = reinterpret_cast<const T *>(x) + row * x_ld, *b = reinterpret_cast<const T *>(w) + (int64_t)id * w_ld;
    const int groups = (width + kN - 1) / kN;
    float s = 0.f;
#pragma unroll 4
    for (int g = threadIdx.x & 31; g < groups; g += 32) {
      const Pack<T, 16> p = some(a, g, width, x_wide), q = some(b, g, width, w_wide);
      float t = 0.f;
#pragma unroll
      for (int e = 0; e < kN; ++e) t = fmaf(p.get(e), q.get(e), t);
      s += t;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    return s;
  }
  __device__ __forceinline__ float get(int64_t row, uint32_t id) const { return bf ? dot<bf16>(row, id) : dot<float>(row, id); }
};

// Per row: the maximum and sum over all slots, the loss, the kept state; 32
// threads per row, each over every 32nd slot.  Where the slots leave the target
// out (tl), its logit is formed here and joins them; else zt has it.  Blocks of eight rows; up to
// kJoinMost rows one block has them all and adds their losses too (kTotal; mean
// of 16 rows, 32768 x 1024 bf16: a launch for the total took 2.6 us more of 22).
constexpr int kJoinMost = 32;
template <int kRows, bool kTotal>
__global__ void __launch_bounds__(32 * kRows) k_xent_join(const float2 *__restrict__ part, int slots, int m,
                                                          const float *__restrict__ zt, const TargetLogit tl, TokenSrc targets,
                                                          float *__restrict__ loss, float *__restrict__ state,
                                                          const uint32_t *__restrict__ err, int mean) {
  pdl_wait();
  const bool bad = any_error(err);
  __shared__ float2 red[32][kRows + 1];
  __shared__ float row_loss[kRows];
  const int r = threadIdx.x % kRows, q = threadIdx.x / kRows;
  const int row = blockIdx.x * kRows + r;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int own = blockIdx.x * kRows + warp;  // a warp for each row
  const uint32_t id = own < m ? targets.key(own) : targets.vocab;
  const bool trained = id < targets.vocab;
  const float z = !trained ? 0.f : tl.x ? tl.get(own, id) : zt[own];
  float mx = -INFINITY, sum = 0.f;
  if (row < m) {
    for (int s = q; s < slots; s += 32) {
      const float2 p = part[(size_t)s * (size_t)m + row];
      const float nm = fmaxf(mx, p.x);
      if (nm != -INFINITY) {
        sum = sum * expf(mx - nm) + p.y * expf(p.x - nm);
        mx = nm;
      } else {
        sum += p.y;  // zero, or a NaN to keep
      }
    }
  }
  red[q][r] = make_float2(mx, sum);
  __syncthreads();
  const float2 p = red[lane][warp];
  float nm = p.x;
#pragma unroll
  for (int d = 16; d; d >>= 1) nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, d));
  sum = nm == -INFINITY ? p.y : p.y * expf(p.x - nm);
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane == 0 && own < m) {
    float rest;
    if (trained && tl.x) {
      const float top = fmaxf(nm, z);
      if (nm != -INFINITY) sum *= expf(nm - top);
      rest = z == top ? log1pf(sum) : logf(sum + expf(z - top));
      nm = top;
    } else {
      rest = logf(sum);
    }
    if (bad) rest = NAN;
    state[own] = nm + rest;
    // not lse - z: a confident token's loss is far below the spacing of lse
    const float l = trained ? (nm - z) + rest : 0.f;
    if (kTotal)
      row_loss[warp] = l;
    else
      loss[own] = l;
    if (!kTotal && own == 0) state[m] = 1.f;
  }
  if (!kTotal) return;
  __syncthreads();
  if (warp) return;
  const int count = max(1, __popc(__ballot_sync(0xffffffffu, lane < m && targets.key(lane) < targets.vocab)));
  double total = lane < m ? (double)row_loss[lane] : 0.0;
#pragma unroll
  for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
  if (lane == 0) {
    *loss = (float)(mean ? total / count : total);
    state[m] = mean ? 1.f / (float)count : 1.f;
  }
}

// The sum or mean of the losses, and 1 / count beside the rows' state.
__global__ void __launch_bounds__(1024) k_xent_total(const float *__restrict__ row_loss, int m, TokenSrc targets,
                                                     int mean, float *__restrict__ loss, float *__restrict__ state) {
  pdl_wait();
  __shared__ double sl[32];
  __shared__ int sc[32];
  double s = 0;
  int c = 0;
  for (int i = threadIdx.x; i < m; i += 1024) {
    s += (double)row_loss[i];
    c += targets.key(i) < targets.vocab ? 1 : 0;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, d);
    c += __shfl_xor_sync(0xffffffffu, c, d);
  }
  if ((threadIdx.x & 31) == 0) {
    sl[threadIdx.x >> 5] = s;
    sc[threadIdx.x >> 5] = c;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0;
    c = 0;
    for (int w = 0; w < 32; ++w) {
      s += sl[w];
      c += sc[w];
    }
    const int n = c > 0 ? c : 1;
    *loss = (float)(mean ? s / n : s);
    state[m] = mean ? 1.f / (float)n : 1.f;
  }
}

// Rows that the gradient leaves out: no target in the vocabulary, or the weight 0.
struct Drop {
  TokenSrc targets;     // ids null: none are
  const float *weight;  // per row, or null
  const float *went;    // of the rows' entropies, or null
  __device__ __forceinline__ bool row(int64_t r) const {
    return targets.ids && (targets.key(r) >= targets.vocab || (weight && weight[r] == 0.f && (!went || went[r] == 0.f)));
  }
};

// [rows][width] into `parts` planes of bf16 [rows][out_ld]: the value, what
// its rounding to bf16 leaves over, and what that leaves over.  A warp per row,
// four groups of eight elements per lane in flight.  Rows that are not trained
// on (drop) become zeros: dz^T x then holds nothing of them, NaN neither.  Where
// it is asked for, hot receives dz at every row's target, from its logit in fp32.
template <typename T>
__global__ void __launch_bounds__(256) k_xent_pack(const T *__restrict__ in, int64_t ld, int64_t rows, int32_t width,
                                                   int parts, bf16 *__restrict__ out, int32_t out_ld, int64_t plane, int vec, const Drop drop,
                                                   const TargetLogit tl, const float *__restrict__ lse,
                                                   const Entropy ent, float *__restrict__ hot) {
  pdl_wait();
  constexpr int kU = 4, kB = 16 / (int)sizeof(T);
  const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= rows) return;
  const bool dropped = drop.row(r);
  if (hot) {
    const float z = dropped ? 0.f : tl.get(r, drop.targets.key(r));
    if ((threadIdx.x & 31) == 0) {
      const float d = dropped ? 0.f : z - lse[r];
      float v = dropped ? 0.f : (drop.weight ? drop.weight[r] : 1.f) * expm1f(d);
      if (ent.weight && !dropped) v = fmaf(expf(d), entropy_slope(0.f, ent.weight[r], d, ent.value[r]), v);
      hot[r] = v;
    }
  }
  const int groups = out_ld / 8;
  for (int g0 = threadIdx.x & 31; g0 < groups; g0 += 32 * kU) {
    float v[kU][8];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int c = (g0 + 32 * u) * 8;
      const T *at = in + r * ld + c;
      if (dropped) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[u][j] = 0.f;
      } else if (vec && c + 8 <= width) {
#pragma unroll
        for (int h = 0; h < 8 / kB; ++h) {
          Pack<T, 16> q;
          q.raw = __ldg(reinterpret_cast<const uint4 *>(at) + h);
#pragma unroll
          for (int j = 0; j < kB; ++j) v[u][h * kB + j] = q.get(j);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[u][j] = c + j < width ? to_f32(at[j]) : 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int c = (g0 + 32 * u) * 8;
      if (c >= out_ld) break;
      if constexpr (sizeof(T) == 2) {  // bf16 is its own only part
        Pack<bf16, 16> o;
#pragma unroll
        for (int j = 0; j < 8; ++j) o.h[j] = (uint16_t)(__float_as_uint(v[u][j]) >> 16);
        *reinterpret_cast<uint4 *>(out + r * out_ld + c) = o.raw;
      } else {
        for (int p = 0; p < parts; ++p) {
          Pack<bf16, 16> o;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float x = v[u][j];
            float h = __bfloat162float(__float2bfloat16_rn(x));
            if (isinf(h) && !isinf(x)) h = __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);  // rounded past the largest
            o.set(j, h);
            v[u][j] = isfinite(x) ? x - h : 0.f;
          }
          *reinterpret_cast<uint4 *>(out + p * plane + r * out_ld + c) = o.raw;
        }
      }
    }
  }
}

// Rows of bf16 from 16-byte aligned ones to any others, two elements per store:
// where a row starts in the middle of a word, two neighbouring words of the
// source make one of it.  (Stores of single elements out of the product's
// epilogue took 440 us for 86926 rows of 1709, this and the aligned stores 190.)
__global__ void __launch_bounds__(256) k_xent_rows(const bf16 *__restrict__ in, int64_t in_ld, int64_t rows, int32_t width,
                                                   bf16 *__restrict__ out, int64_t out_ld) {
  pdl_wait();
  const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= rows) return;
  const int lane = threadIdx.x & 31;
  const uint32_t *from = reinterpret_cast<const uint32_t *>(in + r * in_ld);
  bf16 *row = out + r * out_ld;
  const int shift = (int)(((uintptr_t)row >> 1) & 1);
  uint32_t *to = reinterpret_cast<uint32_t *>(row + shift);
  const int words = (width - shift) / 2;
  const bf16 *single = in + r * in_ld;
#pragma unroll 4
  for (int k = lane; k < words; k += 32) {
    const uint32_t a = __ldg(from + k);
    to[k] = shift ? __funnelshift_r(a, __ldg(from + k + 1), 16) : a;
  }
  if (lane == 0 && shift) row[0] = single[0];
  if (lane == 1 && shift + 2 * words < width) row[width - 1] = single[width - 1];
}

// The rows of dw that are targets: their sums, with what rounding dz to bf16 lost of its
// entries there, mostly by far the largest: for each row of x with the target, in their
// order, that much of it.  A block per row of x and 256 columns, at work for the first
// of each target; its warps share the rows of a target (frequent tokens have hundreds).
constexpr int kHitRows = 512;  // rows of x looked at at a time
__global__ void __launch_bounds__(128) k_xent_hits(const Hits hits, TokenSrc targets, int32_t n, const float *__restrict__ hot,
                                                   const bf16 *__restrict__ x, int64_t x_ld, int32_t width, bf16 *__restrict__ dw,
                                                   int64_t dw_ld, int wide) {
  pdl_wait();
  __shared__ int rows[kHitRows];
  __shared__ int counts[4];
  __shared__ float part[3][32][9];
  const int i = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t id = targets.key(i);
  if (id >= targets.vocab || hits.first[id] != i) return;
  const int last = hits.last[id];
  const int c = blockIdx.y * 256 + lane * 8;
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.f;
  for (int r0 = i; r0 <= last; r0 += kHitRows) {
    constexpr int kOwn = kHitRows / 128;
    const int first = r0 + threadIdx.x * kOwn;
    unsigned here = 0;
#pragma unroll
    for (int u = 0; u < kOwn; ++u)
      if (first + u <= last && targets.key(first + u) == id) here |= 1u << u;
    int before = __popc(here);
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int o = __shfl_up_sync(0xffffffffu, before, d);
      if (lane >= d) before += o;
    }
    if (lane == 31) counts[warp] = before;
    before -= __popc(here);
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (w < warp) before += counts[w];
      all += counts[w];
    }
#pragma unroll
    for (int u = 0; u < kOwn; ++u)
      if ((here >> u) & 1) rows[before++] = first + u;
    __syncthreads();
    if (c < width) {
#pragma unroll 4
      for (int k = warp; k < all; k += 4) {
        const float h = hot[rows[k]], over = h - __bfloat162float(__float2bfloat16_rn(h));
        Pack<bf16, 16> v;
        v.raw = __ldg(reinterpret_cast<const uint4 *>(x + rows[k] * x_ld + c));
        if (over != 0.f)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] = fmaf(over, v.get(j), acc[j]);
      }
    }
    __syncthreads();
  }
  if (warp)
#pragma unroll
    for (int j = 0; j < 8; ++j) part[warp - 1][lane][j] = acc[j];
  __syncthreads();
  if (warp || c >= width) return;
#pragma unroll
  for (int w = 0; w < 3; ++w)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] += part[w][lane][j];
#pragma unroll
  for (int j = 0; j < 8; j += 4)
    if (c + j < width) {
      const float4 v = *reinterpret_cast<const float4 *>(hits.rows + (int64_t)i * hits.ld + c + j);
      acc[j] += v.x;
      acc[j + 1] += v.y;
      acc[j + 2] += v.z;
      acc[j + 3] += v.w;
    }
  bf16 *to = dw + (int64_t)id * dw_ld + c;
  if (wide && c + 8 <= width) {
    Pack<bf16, 16> o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o.set(j, acc[j]);
    *reinterpret_cast<uint4 *>(to) = o.raw;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < width) to[j] = __float2bfloat16_rn(acc[j]);
  }
}

// dx = the splits' sums, added in order and rounded once; rows that are left out
// stay 0 also where the factor is not finite.  With hot (dz rounded to bf16), what
// the rounding left over of the target's entry, mostly the largest of its row, times
// the target's row of w: dx of 4096 x 131072 x 2048 lies 0.0017 from 64 bits, as far as
// its own rounding to bf16 puts it, without that 0.0020.  The last kernel of a gradient: after an error it
// makes dx and the first row of dw NaN.
template <typename T>
__global__ void __launch_bounds__(256) k_xent_dx(const float *__restrict__ acc, int splits, int64_t plane, int32_t acc_ld,
                                                 int32_t m, int32_t width, T *__restrict__ dx, int64_t ld,
                                                 T *__restrict__ dw, Factor factor, const Drop drop,
                                                 const float *__restrict__ hot, const T *__restrict__ w, int64_t w_ld,
                                                 int w_vec, const uint32_t *__restrict__ err) {
  pdl_wait();
  const bool bad = any_error(err);
  const float f = bad ? NAN : factor.get();
  const bool look = !bad && !isfinite(f);
  if (bad && dw && blockIdx.x == 0)
    for (int i = threadIdx.x; i < width; i += 256) dw[i] = from_f32<T>(NAN);
  const int groups = acc_ld / 4;
  const int64_t total = (int64_t)m * groups;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / groups;
    const int c = (int)(i - r * groups) * 4;
    float4 s = *reinterpret_cast<const float4 *>(acc + r * acc_ld + c);
    for (int k = 1; k < splits; ++k) {
      const float4 b = *reinterpret_cast<const float4 *>(acc + k * plane + r * acc_ld + c);
      s.x += b.x;
      s.y += b.y;
      s.z += b.z;
      s.w += b.w;
    }
    if (hot) {
      const float h = hot[r], over = h - __bfloat162float(__float2bfloat16_rn(h));
      const uint32_t id = drop.targets.key(r);
      if (over != 0.f && id < drop.targets.vocab) {
        const T *at = w + (int64_t)id * w_ld + c;
        Pack<T, 4 * sizeof(T)> q;
        if (w_vec && c + 4 <= width) {
          q.raw = __ldg(reinterpret_cast<const typename Pack<T, 4 * sizeof(T)>::R *>(at));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) q.set(j, c + j < width ? to_f32(at[j]) : 0.f);
        }
        s.x = fmaf(over, q.get(0), s.x);
        s.y = fmaf(over, q.get(1), s.y);
        s.z = fmaf(over, q.get(2), s.z);
        s.w = fmaf(over, q.get(3), s.w);
      }
    }
    T *o = dx + r * ld + c;
    const float fr = look && drop.row(r) ? 0.f : f;
    const float e[4] = {s.x * fr, s.y * fr, s.z * fr, s.w * fr};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < width) o[j] = from_f32<T>(e[j]);
  }
}

// ------------------------------------------------------------ host side

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
  static const EncodeTiled fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// planes x rows x cols (cols contiguous, rows ld elements apart) in boxes of
// box_rows rows of box_cols columns; zero fill outside
bool make_map(CUtensorMap *m, const void *base, bool wide, uint64_t cols, uint64_t rows, uint64_t ld, uint64_t planes,
              uint64_t plane, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle) {
  EncodeTiled enc = encoder();
  if (!enc) return false;
  const uint64_t es = wide ? 4 : 2;
  const cuuint64_t dims[3] = {cols, rows, planes};
  const cuuint64_t strides[2] = {ld * es, plane * es};
  const cuuint32_t box[3] = {box_cols, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return with_context([&] {
    return enc(m, wide ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base),
               dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  });
}

// A matrix as the products read it: bf16, 16-byte aligned rows, one or three planes.
struct Operand {
  const void *p;
  int64_t rows, ld, plane;
  int32_t cols, planes;
};
bool load_map(CUtensorMap *m, const Operand &o, bool mn_major, uint32_t box_rows) {
  return make_map(m, o.p, false, (uint64_t)o.cols, (uint64_t)o.rows, (uint64_t)o.ld, (uint64_t)o.planes,
                  (uint64_t)(o.plane > 0 ? o.plane : o.rows * o.ld), 64, mn_major ? 64 : box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

constexpr size_t kPieceBytes = (size_t)256 << 20;  // of dz, or of w's parts, at a time

int sms_of() {
  const int n = current_sms();
  return n < 2 ? 152 : n > 256 ? 256 : n;
}

// Columns of a tile of a product with a K-major B: the width whose last wave of
// tiles wastes least, each tile counted as its columns and the fixed cost of 16
// more; the widest of equals.
int tile_cols(int64_t m_tiles, int64_t n, int sms) {
  int best = 256;
  int64_t best_cost = INT64_MAX;
  for (int nt = 256; nt >= 64; nt -= 32) {
    const int64_t cost = ceil_div(m_tiles * ceil_div(n, nt), sms / 2) * (nt + 16);
    if (cost < best_cost) {
      best_cost = cost;
      best = nt;
    }
  }
  return best;
}

// Pieces of the vocabulary of about equal size and at most kPieceBytes: a
// multiple of the rows that give every pair of SMs one 256-column tile (67 fp32
// tokens, 119598 x 2176: 78 tiles a piece on 76 pairs took two waves, 76 take
// one), or of 256 where those are too many.
int64_t piece_rows(int64_t vocab, int64_t row_bytes, int64_t m_tiles, int sms) {
  const int64_t pairs = sms / 2, wave = 256 * (m_tiles < pairs ? pairs / m_tiles : 1);
  int64_t most = (int64_t)(kPieceBytes / (size_t)row_bytes);
  const int64_t unit = most >= wave ? wave : 256;
  most = most / unit * unit;
  if (most < 1024) most = 1024;
  const int64_t equal = ceil_div(ceil_div(vocab, ceil_div(vocab, most)), unit) * unit;
  return equal < most ? equal : most;
}

// How many ways the K of a product is split: the choice whose last wave of
// tiles wastes least, each tile counted as its K stages (weight of them per K
// block, 0.27 us each) and the fixed cost of eight more, and the reading of the
// splits' sums at the end.
int pick_split(int64_t tiles, int64_t k_blocks, int64_t weight, int64_t sum_bytes, int sms) {
  int best = 1;
  double best_cost = 1e30;
  for (int s = 1; s <= 64; ++s) {
    const int64_t per = ceil_div(k_blocks, s);
    if (s > 1 && per * weight < 8) break;
    if ((s - 1) * per >= k_blocks) continue;  // a split without work
    const double cost = (double)(ceil_div(tiles * s, sms / 2) * (per * weight + 8)) +
                        (double)s * (double)sum_bytes / 6.5e6 / 0.27;
    if (cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

struct XentShape {
  int32_t n, width;
  int64_t vocab;
  snack_dtype t;
  bool pack_x, pack_w;
  bool pack_dw;  // bf16 rows of dw that TMA cannot store: by way of the workspace
  bool few_logits;  // the CUDA cores' logits of a few fp32 tokens,
  bool few;         // and all of a loss, or of the gradients, there
  bool cut;    // the logits of some more: w cut into parts in registers
  int parts;
  int32_t ld;  // row length of packed planes
  int sms;
};

struct XentWs {
  size_t err, zt, hot, row_loss, part, xp, wp, dz, acc, dwp, total;
  int nt;             // forward tile
  int64_t piece;      // vocabulary rows at a time (forward: of packed w; gradient: of dz)
  int64_t slots;
  int64_t dz_ld;
  int32_t acc_ld;
  int nt_d, split;    // dx, dw tile columns; K splits of dx
  int few_nt;         // few tokens: the number that the kernels are built for
  int64_t few_blocks, few_rows;  // blocks of the logits; vocabulary rows per split of dx
};

// blocks of k_xent_cut for `rows` of the vocabulary: one per SM
int64_t cut_blocks(const XentShape &s, int64_t rows) {
  const int64_t tiles = ceil_div(rows, (int64_t)cut_rows(s.n, cut_split(s.n, s.vocab, s.width, s.sms)));
  return tiles < s.sms ? tiles : s.sms;
}

XentWs xent_ws(const XentShape &s, bool grad) {
  XentWs w = {};
  size_t o = 0;
  const int64_t m_tiles = ceil_div(s.n, kM);
  w.err = o;
  o += align_up(256 * 4, kAlign);
  if (s.few) {
    w.few_nt = s.few_logits ? kFewMostLogits : s.n <= 8 ? 8 : 16;
    const int64_t tiles = ceil_div(s.vocab, (int64_t)kSmallWarps * kSmallRows);
    w.few_blocks = tiles < s.sms ? tiles : s.sms;
    w.slots = w.few_blocks;
    if (!grad) {
      w.zt = o;
      o += align_up((size_t)s.n * 4, kAlign);
      w.row_loss = o;
      o += align_up((size_t)s.n * 4, kAlign);
      w.part = o;
      o += align_up((size_t)w.slots * (size_t)s.n * 8, kAlign);
    } else {
      const int64_t groups = ceil_div(s.width, 32 * few_cols(w.few_nt));
      int64_t splits = ceil_div(4 * (int64_t)s.sms, groups);
      if (splits > ceil_div(s.vocab, 64)) splits = ceil_div(s.vocab, 64);
      w.few_rows = ceil_div(s.vocab, splits);
      w.split = (int)ceil_div(s.vocab, w.few_rows);
      w.acc_ld = (int32_t)align_up((size_t)s.width, 4);
      w.dz = o;
      o += align_up((size_t)s.vocab * (size_t)w.few_nt * 4, kAlign);
      w.acc = o;
      o += align_up((size_t)w.split * (size_t)s.n * (size_t)w.acc_ld * 4, kAlign);
    }
    w.total = o;
    return w;
  }
  if (s.cut && !grad) {
    w.slots = cut_blocks(s, s.vocab);
    w.zt = o;
    o += align_up((size_t)s.n * 4, kAlign);
    w.row_loss = o;
    o += align_up((size_t)s.n * 4, kAlign);
    w.part = o;
    o += align_up((size_t)w.slots * (size_t)s.n * 8, kAlign);
    w.total = o;
    return w;
  }
  const int64_t w_row = (int64_t)s.parts * s.ld * 2;
  w.xp = o;
  if (s.pack_x) o += align_up((size_t)s.parts * (size_t)s.n * (size_t)s.ld * 2, kAlign);
  if (!grad) {
    w.piece = s.pack_w ? piece_rows(s.vocab, w_row, m_tiles, s.sms) : s.vocab;
    if (w.piece > s.vocab) w.piece = s.vocab;
    w.nt = tile_cols(m_tiles, w.piece, s.sms);
    w.slots = 2 * (ceil_div(s.vocab, w.piece) * ceil_div(w.piece, w.nt));
    w.row_loss = o;
    o += align_up((size_t)s.n * 4, kAlign);
    w.part = o;
    o += align_up((size_t)w.slots * (size_t)s.n * 8, kAlign);
  } else {
    const int64_t dz_row = (int64_t)s.parts * s.n * 2;
    const int64_t dw_row = s.pack_dw ? (int64_t)s.ld * 2 : 0;
    w.piece = piece_rows(s.vocab, std::max(std::max(s.pack_w ? w_row : 0, dz_row), dw_row), m_tiles, s.sms);
    if (w.piece > s.vocab) w.piece = s.vocab;
    w.dz_ld = ceil_div(w.piece, 64) * 64;
    w.nt_d = s.width > 128 ? 256 : 128;  // a CTA's half of B is 64 columns at least
    w.acc_ld = (int32_t)align_up((size_t)s.width, 4);
    // the pieces' products are alike: all of them as one piece of so many times the K stages
    w.split = pick_split(m_tiles * ceil_div(s.width, w.nt_d), ceil_div(w.piece, kKb),
                         (s.parts == 3 ? 6 : 1) * ceil_div(s.vocab, w.piece), (int64_t)s.n * w.acc_ld * 4, s.sms);
    w.hot = o;
    o += align_up((size_t)s.n * 4, kAlign);
    w.dz = o;
    o += align_up((size_t)s.parts * (size_t)s.n * (size_t)w.dz_ld * 2, kAlign);
    w.acc = o;
    o += align_up((size_t)w.split * (size_t)s.n * (size_t)w.acc_ld * 4, kAlign);
  }
  w.dwp = o;
  if (grad && s.pack_dw) o += align_up((size_t)w.piece * (size_t)s.ld * 2, kAlign);
  w.wp = o;
  if (s.pack_w) o += align_up((size_t)s.parts * (size_t)w.piece * (size_t)s.ld * 2, kAlign);
  w.total = o;
  return w;
}

// Whether a bf16 matrix (w, and the forward's x) can be read as it lies.  TMA asks for 16-byte aligned
// rows; off a 128-byte line every box row costs it one line more, and the
// products run a fifth to a quarter slower (1999 x 50001 x 1000: gradient 499
// against 402 us, forward 235 against 199 us), so large products lay it out
// again first: the gradient reads an operand three times, the forward once.
bool rows_ready(const void *p, int64_t ld, int32_t n, bool grad) {
  if (!ptr_aligned(p, 16) || ld % 8 != 0) return false;
  const bool on_lines = ptr_aligned(p, 128) && ld % 64 == 0;
  return on_lines || n < (grad ? 1024 : 4096);
}

XentShape xent_shape(const void *x, int64_t x_ld, int32_t n, const void *wt, int64_t w_ld, int64_t vocab, int32_t width,
                     snack_dtype t, bool grad) {
  XentShape s;
  s.n = n;
  s.width = width;
  s.vocab = vocab;
  s.t = t;
  s.parts = t == SNACK_F32 ? 3 : 1;
  s.pack_x = grad || t == SNACK_F32 || !rows_ready(x, x_ld, n, grad);  // the gradient's leaves rows out
  s.pack_w = t == SNACK_F32 || !rows_ready(wt, w_ld, n, grad);
  s.few_logits = t == SNACK_F32 && few_fits(n, vocab, sms_of());
  s.few = t == SNACK_F32 && (grad ? n <= kSmallMostTokens : s.few_logits);
  s.cut = t == SNACK_F32 && !s.few && cut_fits(n, width);
  s.pack_dw = t == SNACK_BF16 && width % 8 != 0;
  s.ld = (int32_t)align_up((size_t)width, 64);
  s.sms = sms_of();
  return s;
}

// Units of K stages (64 each): see the note on rounding at the top.  Each unit
// costs an exchange of accumulators and a read of 128 KB of tensor memory per
// CTA (about 1900 cycles beside the MMAs, of 512 a stage and product).  Sums that
// become the loss or other fp32 results take units of at most eight stages, of
// equal length; the losses of fp32 operands take four (six part products hide most
// of the reads: 1024 x 16384 x 768, 5 us of 92).  What is rounded to bf16 (dz, dx
// and dw of bf16 operands) is far below half its ulp with long ones; dz at the
// target, p - 1, is not, and does not come from them: one accumulator over 4096 of K
// would make it wrong by 2e-4 at logits of 40, where 1 - p was 2e-3.  The entropy's
// gradient has log p + H, which is small where the logits are alike: there dz takes the
// units of the statistics, whose error is then common to both (1021 x 50001 x 1000 370
// and 374 us, 4096 x 131072 x 2048 5420 and 5545).
// Measured, relative error of logits of 40 (width 4096) on average, and the loss of
// 2048 x 65536 x 4096 bf16 and of 67 x 119598 x 2176 fp32, us:
//   unit   random    positive  nine of ten zero    bf16   fp32
//      8  -5.9e-7    -8.1e-7    -1.6e-7             568    961
//      4  -2.9e-7    -3.5e-7    -0.7e-7             678    984
//      2  -1.5e-7    -1.7e-7    -0.3e-7            1099   1033
int unit_of(int k_blocks, int most) { return (int)ceil_div(k_blocks, ceil_div(k_blocks, most)); }

template <int kMode>
cudaError_t launch_gemm(const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &o, GemmArgs &g, int sms,
                        cudaStream_t s) {
  static constexpr auto kernel = [] {
    if constexpr (kMode == kScore)
      return k_score;
    else
      return k_xent<kMode>;
  }();
  // the entropy's gradient has what a logit is above the row's mean: its logits have to be the statistics' own, to the bit
  const bool logits = kMode == kStats || kMode == kScore || (kMode == kDlog && g.ent.weight);
  cudaError_t e = raise_smem_limit(kernel, kSmem);
  if (e != cudaSuccess) return e;
  // the register split draws on what the launch gives: a kernel built with fewer would wait for ever
  static const bool enough = [] {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, kernel) == cudaSuccess &&
           a.numRegs * kThreads >= 256 * kEpiRegs + 128 * kIssueRegs;
  }();
  if (!enough) return cudaErrorInvalidDeviceFunction;
  g.m_tiles = (int32_t)ceil_div(g.m, kM);
  g.n_tiles = (int32_t)ceil_div(g.n, g.nt);
  g.unit = unit_of((int)ceil_div(g.k_blocks, g.n_split), g.products > 1 ? (logits ? 4 : 8) : logits ? 8 : 64);
  g.a_rows = kMode == kDw || g.m >= kMCta ? kMCta : (int32_t)align_up((size_t)g.m, 8);
  g.stages = kRing / ((g.a_rows + g.nt / 2) * kKb * 2);
  if (g.stages > kMaxStages) g.stages = kMaxStages;
  const int64_t tiles = (int64_t)g.m_tiles * g.n_tiles * g.n_split;
  if (tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
  e = launch_pdl(kernel, 2 * (unsigned)(tiles < sms / 2 ? tiles : sms / 2), kThreads, kSmem, s, a, b, o, (const GemmArgs)g);
  g.first = 0;
  return e;
}

// the targets of a gradient's rows, for x's layout
struct RowInfo {
  Drop drop;
  TargetLogit tl;
  const float *lse;
  Entropy ent;
  float *hot;
};

cudaError_t pack(const XentShape &s, const void *in, int64_t ld, int64_t rows, void *out, const RowInfo &ri, cudaStream_t st) {
  const int64_t blocks = ceil_div(rows, 8);
  const int vec = ptr_aligned(in, 16) && (size_t)ld * dtype_size(s.t) % 16 == 0;
  if (s.t == SNACK_F32)
    return launch_pdl(k_xent_pack<float>, (unsigned)blocks, 256, 0, st, reinterpret_cast<const float *>(in), ld, rows,
                      s.width, s.parts, reinterpret_cast<bf16 *>(out), s.ld, (int64_t)rows * s.ld, vec, ri.drop, ri.tl, ri.lse,
                    ri.ent, ri.hot);
  return launch_pdl(k_xent_pack<bf16>, (unsigned)blocks, 256, 0, st, reinterpret_cast<const bf16 *>(in), ld, rows,
                    s.width, s.parts, reinterpret_cast<bf16 *>(out), s.ld, (int64_t)rows * s.ld, vec, ri.drop, ri.tl, ri.lse,
                    ri.ent, ri.hot);
}

// x, or a piece of w from row v0 on, as the products read it
cudaError_t operand(const XentShape &s, bool packed, const void *p, int64_t ld, int64_t v0, int64_t rows, void *buf,
                    Operand *o, cudaStream_t st, const RowInfo &ri = RowInfo{}) {
  const size_t es = dtype_size(s.t);
  const uint8_t *at = reinterpret_cast<const uint8_t *>(p) + (size_t)v0 * (size_t)ld * es;
  o->rows = rows;
  o->cols = s.width;
  if (!packed) {
    o->p = at;
    o->ld = ld;
    o->planes = 1;
    o->plane = 0;
    return cudaSuccess;
  }
  o->p = buf;
  o->ld = s.ld;
  o->planes = s.parts;
  o->plane = rows * s.ld;
  return pack(s, at, ld, rows, buf, ri, st);
}

GemmArgs gemm_args(const XentShape &s, uint8_t *ws, const XentWs &W, int first) {
  GemmArgs g = {};
  g.n_split = 1;
  g.products = s.parts == 3 ? 6 : 1;
  g.a_part = s.parts == 3 ? kPartA : 0;
  g.b_part = s.parts == 3 ? kPartB : 0;
  g.err = reinterpret_cast<uint32_t *>(ws + W.err);
  g.first = first;
  return g;
}

TargetLogit target_logit(const XentShape &s, const void *x, int64_t x_ld, const void *w, int64_t w_ld) {
  const size_t es = dtype_size(s.t);
  const auto wide = [es](const void *p, int64_t ld) { return ptr_aligned(p, 16) && (size_t)ld * es % 16 == 0; };
  return {x, w, x_ld, w_ld, s.width, s.t == SNACK_BF16, wide(x, x_ld), wide(w, w_ld)};
}

cudaError_t finish_loss(const float2 *part, int slots, int32_t n, const float *zt, const TargetLogit &tl, const TokenSrc &tg,
                        snack_reduction reduction, float *row_loss, float *loss, float *state, const uint32_t *err,
                        cudaStream_t s) {
  if (n <= kJoinMost && reduction != SNACK_NONE)
    return launch_pdl(k_xent_join<kJoinMost, true>, 1, 32 * kJoinMost, 0, s, part, slots, n, zt, tl, tg, loss, state, err,
                      reduction == SNACK_MEAN ? 1 : 0);
  cudaError_t e = launch_pdl(k_xent_join<8, false>, (unsigned)ceil_div(n, 8), 256, 0, s, part, slots, n, zt, tl, tg, row_loss,
                             state, err, 0);
  if (e != cudaSuccess || reduction == SNACK_NONE) return e;
  return launch_pdl(k_xent_total, 1, 1024, 0, s, (const float *)row_loss, n, tg, reduction == SNACK_MEAN, loss, state);
}

template <bool kGrad>
cudaError_t launch_few(const SmallArgs &a, int64_t blocks, cudaStream_t s) {
  const size_t smem = (size_t)(kFewMostLogits * a.chunk + kSmallWarps * kSmallRows * (kFewMostLogits + 1)) * 4;
  cudaError_t e = raise_smem_limit(k_xent_few<kGrad>, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_xent_few<kGrad>, (unsigned)blocks, kSmallWarps * 32, smem, s, a);
}

template <int kTiles, int kAcross, bool kGrad>
cudaError_t launch_cut(const CutArgs &a, int64_t blocks, cudaStream_t s) {
  const size_t smem = cut_smem_bytes(a, kTiles, kAcross);
  cudaError_t e = raise_smem_limit(k_xent_cut<kTiles, kAcross, kGrad>, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_xent_cut<kTiles, kAcross, kGrad>, (unsigned)blocks, kCutWarps * 32, smem, s, a);
}

// the kernel for the call's tokens
template <bool kGrad>
cudaError_t launch_cut_for(const CutArgs &a, int64_t blocks, cudaStream_t s) {
  return a.n <= 8    ? launch_cut<1, 1, kGrad>(a, blocks, s)
         : a.n <= 16 ? launch_cut<2, 1, kGrad>(a, blocks, s)
         : a.n <= 32 ? launch_cut<4, 1, kGrad>(a, blocks, s)
                     : launch_cut<4, 2, kGrad>(a, blocks, s);
}

CutArgs cut_args(const XentShape &S, const void *x, int64_t x_ld, const void *w, int64_t w_ld, const TokenSrc &tg) {
  CutArgs a = {};
  a.x = reinterpret_cast<const float *>(x);
  a.w = reinterpret_cast<const float *>(w);
  a.x_ld = x_ld;
  a.w_ld = w_ld;
  a.n = S.n;
  a.width = S.width;
  a.vocab = S.vocab;
  a.chunk = cut_chunk(S.n, S.width);
  a.split = cut_split(S.n, S.vocab, S.width, S.sms);
  a.x_wide = ptr_aligned(x, 16) && x_ld % 4 == 0;
  a.w_wide = ptr_aligned(w, 16) && w_ld % 4 == 0;
  a.targets = tg;
  return a;
}

template <int kNt>
cudaError_t launch_few_grad(const SmallGrad &a, dim3 grid, bool dx, bool dw, cudaStream_t s) {
  auto kernel = dx && dw ? k_xent_few_grad<kNt, true, true>
                : dx     ? k_xent_few_grad<kNt, true, false>
                         : k_xent_few_grad<kNt, false, true>;
  return launch_pdl(kernel, grid, kFewWarps * 32, 0, s, a);
}

SmallArgs small_args(const XentShape &S, const void *x, int64_t x_ld, const void *w, int64_t w_ld, const TokenSrc &tg) {
  SmallArgs a = {};
  a.x = reinterpret_cast<const float *>(x);
  a.w = reinterpret_cast<const float *>(w);
  a.x_ld = x_ld;
  a.w_ld = w_ld;
  a.n = S.n;
  a.width = S.width;
  a.vocab = S.vocab;
  a.x_wide = ptr_aligned(x, 16) && x_ld % 4 == 0;
  a.w_wide = ptr_aligned(w, 16) && w_ld % 4 == 0;
  a.chunk = small_k(S.width);
  a.targets = tg;
  return a;
}

snack_status xent_check(const void *x, int64_t x_ld, int32_t n, const void *w, int64_t w_ld, int64_t vocab, int32_t width,
                        snack_dtype t) {
  if (!lm_dtype_ok(t) || n < 0 || vocab < 1 || width < 1 || x_ld < width || w_ld < width) return SNACK_ERR_INVALID_ARG;
  const size_t es = dtype_size(t);
  if (!ptr_aligned(x, es) || !ptr_aligned(w, es)) return SNACK_ERR_INVALID_ARG;
  // tile counts and the row steps of tensor maps stay within 31 and 40 bits
  if (vocab >= ((int64_t)1 << 30) || n >= (1 << 24) || width >= (1 << 20) || x_ld >= ((int64_t)1 << 36) ||
      w_ld >= ((int64_t)1 << 36))
    return SNACK_ERR_UNSUPPORTED;
  return SNACK_OK;
}

struct Span {
  const void *p;
  size_t bytes;
};
// Whether one of the buffers that a call writes overlaps any other of its buffers (absent ones have no bytes).
template <int kWritten, int kRead>
bool any_overlap(const Span (&written)[kWritten], const Span (&read)[kRead]) {
  for (int i = 0; i < kWritten; ++i) {
    for (int j = i + 1; j < kWritten; ++j)
      if (spans_overlap(written[i].p, written[i].bytes, written[j].p, written[j].bytes)) return true;
    for (const Span &r : read)
      if (spans_overlap(written[i].p, written[i].bytes, r.p, r.bytes)) return true;
  }
  return false;
}

#define XENT_CUDA(x)                               \
  do {                                             \
    if ((x) != cudaSuccess) return SNACK_ERR_CUDA; \
  } while (0)

// The gradients of a loss whose dz[i, v] is weight[i] (1 where weight is null) times
// (p - [v = target]), and with ent weights of the rows' entropies besides, all times
// factor.  state: the rows' log sums of exponentials.  hits: rows of dw to keep.
snack_status xent_gradient(const XentShape &S, const XentWs &W, const void *x, int64_t x_ld, const void *w, int64_t w_ld,
                           const TokenSrc &tg, const float *weight, const Entropy &ent, const Hits &hits, const Factor &factor,
                           const float *state, void *dx, int64_t dx_ld, void *dw, int64_t dw_ld, uint8_t *b, cudaStream_t s) {
  const int32_t n = S.n, width = S.width;
  const int64_t vocab = S.vocab;
  const size_t es = dtype_size(S.t);
  const bool wide = S.t == SNACK_F32;
  if (S.few) {
    SmallArgs a = small_args(S, x, x_ld, w, w_ld, tg);
    a.lse = state;
    a.weight = weight;
    a.ent = ent;
    a.dz = reinterpret_cast<float *>(b + W.dz);
    if (S.few_logits) {
      XENT_CUDA(launch_few<true>(a, W.few_blocks, s));
    } else {
      CutArgs c = cut_args(S, x, x_ld, w, w_ld, tg);
      c.lse = a.lse;
      c.weight = weight;
      c.ent = ent;
      c.dz = a.dz;
      XENT_CUDA(launch_cut_for<true>(c, cut_blocks(S, vocab), s));
    }
    SmallGrad g = {};
    g.x = a.x;
    g.w = a.w;
    g.dz = a.dz;
    g.x_ld = x_ld;
    g.w_ld = w_ld;
    g.dw_ld = dw_ld;
    g.n = n;
    g.width = width;
    g.vocab = vocab;
    g.rows_per_split = W.few_rows;
    g.w_wide = a.w_wide;
    g.dw_wide = ptr_aligned(dw, 16) && dw_ld % 4 == 0;
    g.targets = tg;
    g.weight = weight;
    g.went = ent.weight;
    g.factor_a = factor.a;
    g.factor_b = factor.b;
    g.acc = reinterpret_cast<float *>(b + W.acc);
    g.acc_ld = W.acc_ld;
    g.dw = reinterpret_cast<float *>(dw);
    const dim3 grid((unsigned)ceil_div(width, 32 * few_cols(W.few_nt)), (unsigned)W.split);
    XENT_CUDA(W.few_nt == 4   ? launch_few_grad<4>(g, grid, dx, dw, s)
              : W.few_nt == 8 ? launch_few_grad<8>(g, grid, dx, dw, s)
                              : launch_few_grad<16>(g, grid, dx, dw, s));
    if (dx)
      XENT_CUDA(launch_pdl(k_xent_dx<float>, (unsigned)ceil_div((int64_t)n * (W.acc_ld / 4), 256), 256, 0, s,
                           (const float *)g.acc, W.split, (int64_t)n * W.acc_ld, W.acc_ld, n, width,
                           reinterpret_cast<float *>(dx), dx_ld, (float *)nullptr, factor, Drop{tg, weight, ent.weight},
                           (const float *)nullptr, (const float *)nullptr, (int64_t)0, 0, (const uint32_t *)nullptr));
    return SNACK_OK;
  }
  const uint32_t a_rows = n >= kMCta ? kMCta : (uint32_t)align_up((size_t)n, 8);
  Operand ox, ow;
  float *hot = reinterpret_cast<float *>(b + W.hot);
  XENT_CUDA(operand(S, S.pack_x, x, x_ld, 0, n, b + W.xp, &ox, s,
                    RowInfo{Drop{tg, weight, ent.weight}, target_logit(S, x, x_ld, w, w_ld), state, ent, S.cut ? nullptr : hot}));
  CUtensorMap mx, mw, mxt, mwt, mdz, mdzt, mdz_out, macc, mdw;
  if (!load_map(&mx, ox, false, a_rows) || !load_map(&mxt, ox, true, 0)) return SNACK_ERR_CUDA;
  if (!make_map(&macc, b + W.acc, true, (uint64_t)width, (uint64_t)n, (uint64_t)W.acc_ld, (uint64_t)W.split,
                (uint64_t)n * (uint64_t)W.acc_ld, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B))
    return SNACK_ERR_CUDA;
  int first = 1;
  for (int64_t v0 = 0; v0 < vocab; v0 += W.piece) {
    const int64_t rows = vocab - v0 < W.piece ? vocab - v0 : W.piece;
    if (dx || !S.cut) XENT_CUDA(operand(S, S.pack_w, w, w_ld, v0, rows, b + W.wp, &ow, s));
    const Operand dz = {b + W.dz, n, W.dz_ld, (int64_t)n * W.dz_ld, (int32_t)rows, S.parts};
    if (!load_map(&mdz, dz, false, a_rows) || !load_map(&mdzt, dz, true, 0) || (dx && !load_map(&mwt, ow, true, 0)))
      return SNACK_ERR_CUDA;
    if (S.cut) {  // as the loss's were
      CutArgs c = cut_args(S, x, x_ld, reinterpret_cast<const float *>(w) + v0 * w_ld, w_ld, tg);
      c.vocab = rows;
      c.v0 = (int32_t)v0;
      c.lse = state;
      c.weight = weight;
      c.ent = ent;
      c.dz_parts = reinterpret_cast<bf16 *>(b + W.dz);
      c.dz_ld = W.dz_ld;
      c.plane = dz.plane;
      XENT_CUDA(launch_cut_for<true>(c, cut_blocks(S, rows), s));
    } else {
      const int nt = tile_cols(ceil_div(n, kM), rows, S.sms);
      if (!load_map(&mw, ow, false, (uint32_t)nt / 2) ||
          !make_map(&mdz_out, dz.p, false, (uint64_t)rows, (uint64_t)n, (uint64_t)W.dz_ld, (uint64_t)S.parts,
                    (uint64_t)dz.plane, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
        return SNACK_ERR_CUDA;
      GemmArgs g = gemm_args(S, b, W, first);
      g.m = n;
      g.n = (int32_t)rows;
      g.nt = nt;
      g.k_blocks = (int32_t)ceil_div(width, kKb);
      g.targets = tg;
      g.v0 = (int32_t)v0;
      g.lse = state;
      g.hot = hot;
      g.dloss = weight;
      g.ent = ent;
      g.out_parts = S.parts;
      XENT_CUDA(launch_gemm<kDlog>(mx, mw, mdz_out, g, S.sms, s));
      first = 0;
    }
    if (dx) {
      GemmArgs h = gemm_args(S, b, W, first);
      h.m = n;
      h.n = width;
      h.nt = W.nt_d;
      h.n_split = W.split;
      h.k_blocks = (int32_t)ceil_div(rows, kKb);
      h.add = v0 > 0;
      XENT_CUDA(launch_gemm<kDx>(mdz, mwt, macc, h, S.sms, s));
      first = 0;
    }
    if (dw) {
      GemmArgs h = gemm_args(S, b, W, first);
      h.m = (int32_t)rows;
      h.n = width;
      h.nt = W.nt_d;
      h.k_blocks = (int32_t)ceil_div(n, kKb);
      uint8_t *to = reinterpret_cast<uint8_t *>(dw) + (size_t)v0 * (size_t)dw_ld * es;
      // a TMA store writes whole 16 bytes at a row's end: of rows of other lengths it would write past them
      const bool direct = ptr_aligned(to, 16) && (size_t)dw_ld * es % 16 == 0 && (size_t)width * es % 16 == 0;
      const bool by_ws = !direct && S.pack_dw;
      uint8_t *out = by_ws ? b + W.dwp : to;
      const int64_t out_ld = by_ws ? S.ld : dw_ld;
      h.out = out;
      h.v0 = (int32_t)v0;
      h.hits = hits;
      h.factor = factor;
      h.targets = tg;
      h.tokens = n;
      h.out_ld = out_ld;
      h.out_wide = wide;
      h.out_tma = direct || by_ws;
      if (h.out_tma && !make_map(&mdw, out, wide, (uint64_t)width, (uint64_t)rows, (uint64_t)out_ld, 1,
                                 (uint64_t)rows * (uint64_t)out_ld, wide ? 32 : 64, 32, CU_TENSOR_MAP_SWIZZLE_128B))
        return SNACK_ERR_CUDA;
      XENT_CUDA(launch_gemm<kDw>(mdzt, mxt, h.out_tma ? mdw : mxt, h, S.sms, s));
      first = 0;
      if (by_ws)
        XENT_CUDA(launch_pdl(k_xent_rows, (unsigned)ceil_div(rows, 8), 256, 0, s, reinterpret_cast<const bf16 *>(out),
                             out_ld, rows, width, reinterpret_cast<bf16 *>(to), dw_ld));
    }
  }
  if (dw && hits.first)
    XENT_CUDA(launch_pdl(k_xent_hits, dim3((unsigned)n, (unsigned)ceil_div(width, 256)), 128, 0, s, hits, tg, n, (const float *)hot,
                         reinterpret_cast<const bf16 *>(ox.p), ox.ld, width, reinterpret_cast<bf16 *>(dw), dw_ld,
                         ptr_aligned(dw, 16) && dw_ld % 8 == 0 ? 1 : 0));
  const int64_t total = dx ? (int64_t)n * (W.acc_ld / 4) : 0;
  int64_t blocks = ceil_div(total, 256);
  if (blocks > (int64_t)S.sms * 16) blocks = (int64_t)S.sms * 16;
  if (blocks < 1) blocks = 1;
  const float *acc = reinterpret_cast<const float *>(b + W.acc);
  const uint32_t *err = reinterpret_cast<const uint32_t *>(b + W.err);
  if (wide)
    XENT_CUDA(launch_pdl(k_xent_dx<float>, (unsigned)blocks, 256, 0, s, acc, W.split, (int64_t)n * W.acc_ld, W.acc_ld,
                         dx ? n : 0, width, reinterpret_cast<float *>(dx), dx_ld, reinterpret_cast<float *>(dw), factor,
                         Drop{tg, weight, ent.weight}, (const float *)nullptr, (const float *)nullptr, (int64_t)0, 0, err));
  else
    XENT_CUDA(launch_pdl(k_xent_dx<bf16>, (unsigned)blocks, 256, 0, s, acc, W.split, (int64_t)n * W.acc_ld, W.acc_ld,
                         dx ? n : 0, width, reinterpret_cast<bf16 *>(dx), dx_ld, reinterpret_cast<bf16 *>(dw), factor,
                         Drop{tg, weight, ent.weight}, (const float *)hot, reinterpret_cast<const bf16 *>(w), w_ld,
                         ptr_aligned(w, 8) && w_ld % 4 == 0 ? 1 : 0, err));
  return SNACK_OK;
}

}  // namespace
}  // namespace snack

using namespace snack;

extern "C" {

snack_status snack_xent_workspace_size(const void *x, int64_t x_ld, int32_t n, const void *w, int64_t w_ld,
                                       int64_t vocab, int32_t width, snack_dtype t, int grad, size_t *bytes) {
  if (!bytes) return SNACK_ERR_INVALID_ARG;
  const snack_status st = xent_check(x, x_ld, n, w, w_ld, vocab, width, t);
  if (st != SNACK_OK) return st;
  *bytes = n == 0 ? 0 : xent_ws(xent_shape(x, x_ld, n, w, w_ld, vocab, width, t, grad != 0), grad != 0).total;
  return SNACK_OK;
}

snack_status snack_xent_fwd(const void *x, int64_t x_ld, int32_t n, const void *w, int64_t w_ld, int64_t vocab,
                            int32_t width, snack_dtype t, const void *targets, snack_index targets_t,
                            snack_reduction reduction, float *loss, float *state, void *ws, size_t ws_bytes,
                            snack_stream_t stream) try {
  const snack_status ck = xent_check(x, x_ld, n, w, w_ld, vocab, width, t);
  if (ck != SNACK_OK) return ck;
  if (!lm_index_ok(targets_t) || reduction < SNACK_NONE || reduction > SNACK_MEAN) return SNACK_ERR_INVALID_ARG;
  if (!loss || !state || !ptr_aligned(loss, 4) || !ptr_aligned(state, 4)) return SNACK_ERR_INVALID_ARG;
  if (n > 0 && (!x || !w || !targets || !ws || !ptr_aligned(targets, index_size(targets_t)) || !ptr_aligned(ws, kAlign)))
    return SNACK_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const TokenSrc tg{targets, targets_t == SNACK_I64, (uint32_t)vocab};
  if (n == 0) {
    if (reduction != SNACK_NONE)
      XENT_CUDA(launch_pdl(k_xent_total, 1, 1024, 0, s, (const float *)nullptr, 0, tg, reduction == SNACK_MEAN, loss, state));
    return SNACK_OK;
  }
  const XentShape S = xent_shape(x, x_ld, n, w, w_ld, vocab, width, t, false);
  const XentWs W = xent_ws(S, false);
  if (ws_bytes < W.total) return SNACK_ERR_WORKSPACE;
  const size_t es = dtype_size(t);
  const Span written[] = {{loss, (reduction == SNACK_NONE ? (size_t)n : 1) * 4}, {state, ((size_t)n + 1) * 4}, {ws, W.total}};
  const Span read[] = {{x, span_bytes(n, width, x_ld, es)}, {w, span_bytes(vocab, width, w_ld, es)},
                       {targets, (size_t)n * index_size(targets_t)}};
  if (any_overlap(written, read)) return SNACK_ERR_INVALID_ARG;
  uint8_t *b = reinterpret_cast<uint8_t *>(ws);
  float *zt = reinterpret_cast<float *>(b + W.zt);
  float2 *part = reinterpret_cast<float2 *>(b + W.part);
  float *row_loss = reduction == SNACK_NONE ? loss : reinterpret_cast<float *>(b + W.row_loss);
  if (S.few) {
    SmallArgs a = small_args(S, x, x_ld, w, w_ld, tg);
    a.part = part;
    a.zt = zt;
    XENT_CUDA(launch_few<false>(a, W.few_blocks, s));
    XENT_CUDA(finish_loss(part, (int)W.slots, n, zt, TargetLogit{}, tg, reduction, row_loss, loss, state, nullptr, s));
    return SNACK_OK;
  }
  if (S.cut) {
    CutArgs a = cut_args(S, x, x_ld, w, w_ld, tg);
    a.part = part;
    a.zt = zt;
    XENT_CUDA(launch_cut_for<false>(a, W.slots, s));
    XENT_CUDA(finish_loss(part, (int)W.slots, n, zt, TargetLogit{}, tg, reduction, row_loss, loss, state, nullptr, s));
    return SNACK_OK;
  }
  const uint32_t a_rows = n >= kMCta ? kMCta : (uint32_t)align_up((size_t)n, 8);
  Operand ox, ow;
  XENT_CUDA(operand(S, S.pack_x, x, x_ld, 0, n, b + W.xp, &ox, s));
  CUtensorMap mx, mw;
  if (!load_map(&mx, ox, false, a_rows)) return SNACK_ERR_CUDA;
  GemmArgs g = gemm_args(S, b, W, 1);
  g.m = n;
  g.nt = W.nt;
  g.k_blocks = (int32_t)ceil_div(width, kKb);
  g.part = part;
  g.targets = tg;
  for (int64_t v0 = 0; v0 < vocab; v0 += W.piece) {
    const int64_t rows = vocab - v0 < W.piece ? vocab - v0 : W.piece;
    XENT_CUDA(operand(S, S.pack_w, w, w_ld, v0, rows, b + W.wp, &ow, s));
    if (!load_map(&mw, ow, false, (uint32_t)W.nt / 2)) return SNACK_ERR_CUDA;
    g.n = (int32_t)rows;
    g.v0 = (int32_t)v0;
    XENT_CUDA(launch_gemm<kStats>(mx, mw, mx, g, S.sms, s));
    g.slot0 += 2 * g.n_tiles;
  }
  const bool copied = S.pack_x && t == SNACK_BF16;  // x laid out again, on better boundaries
  XENT_CUDA(finish_loss(part, g.slot0, n, nullptr, target_logit(S, copied ? ox.p : x, copied ? ox.ld : x_ld, w, w_ld), tg,
                        reduction, row_loss, loss, state, g.err, s));
  return SNACK_OK;
} catch (...) {  // a host allocation failed
  return SNACK_ERR_CUDA;
}

snack_status snack_xent_bwd(const void *x, int64_t x_ld, int32_t n, const void *w, int64_t w_ld, int64_t vocab,
                            int32_t width, snack_dtype t, const void *targets, snack_index targets_t,
                            snack_reduction reduction, const float *state, const float *dloss, void *dx, int64_t dx_ld,
                            void *dw, int64_t dw_ld, void *ws, size_t ws_bytes, snack_stream_t stream) try {
  const snack_status ck = xent_check(x, x_ld, n, w, w_ld, vocab, width, t);
  if (ck != SNACK_OK) return ck;
  const size_t es = dtype_size(t);
  if (!lm_index_ok(targets_t) || reduction < SNACK_NONE || reduction > SNACK_MEAN) return SNACK_ERR_INVALID_ARG;
  if ((dx && (dx_ld < width || !ptr_aligned(dx, es))) || (dw && (dw_ld < width || !ptr_aligned(dw, es))))
    return SNACK_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (n == 0) {
    if (dw) XENT_CUDA(cudaMemset2DAsync(dw, (size_t)dw_ld * es, 0, (size_t)width * es, (size_t)vocab, s));
    return SNACK_OK;
  }
  if (!x || !w || !targets || !state || !ws || !ptr_aligned(targets, index_size(targets_t)) || !ptr_aligned(state, 4) ||
      !ptr_aligned(ws, kAlign) || (dloss && !ptr_aligned(dloss, 4)) || (reduction == SNACK_NONE && !dloss))
    return SNACK_ERR_INVALID_ARG;
  const XentShape S = xent_shape(x, x_ld, n, w, w_ld, vocab, width, t, true);
  const XentWs W = xent_ws(S, true);
  const Span written[] = {{dx, dx ? span_bytes(n, width, dx_ld, es) : 0}, {dw, dw ? span_bytes(vocab, width, dw_ld, es) : 0},
                          {ws, std::min(ws_bytes, W.total)}};
  const Span read[] = {{x, span_bytes(n, width, x_ld, es)}, {w, span_bytes(vocab, width, w_ld, es)},
                       {targets, (size_t)n * index_size(targets_t)}, {state, ((size_t)n + 1) * 4},
                       {dloss, dloss ? (reduction == SNACK_NONE ? (size_t)n : 1) * 4 : 0}};
  if (any_overlap(written, read)) return SNACK_ERR_INVALID_ARG;
  if (ws_bytes < W.total) return SNACK_ERR_WORKSPACE;
  if (!dx && !dw) return SNACK_OK;
  const TokenSrc tg{targets, targets_t == SNACK_I64, (uint32_t)vocab};
  const float *weight = reduction == SNACK_NONE ? dloss : nullptr;
  const Factor factor = {reduction == SNACK_NONE ? nullptr : dloss, reduction == SNACK_MEAN ? state + n : nullptr};
  return xent_gradient(S, W, x, x_ld, w, w_ld, tg, weight, Entropy{}, Hits{}, factor, state, dx, dx_ld, dw, dw_ld,
                       reinterpret_cast<uint8_t *>(ws), s);
} catch (...) {  // a host allocation failed
  return SNACK_ERR_CUDA;
}

}  // extern "C"

#include "score.cuh"
