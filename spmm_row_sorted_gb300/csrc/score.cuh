// Log probabilities of given tokens under a projection to a vocabulary, the entropies
// of its distributions and their likeliest tokens; and the gradients of the first two.
//
//   z[i, v] = sum_d x[i, d] w[v, d],   M = max_v z,   S = sum_v e^(z - M)
//   logp[i] = (z[i, t_i] - M) - log S
//   H[i]    = log S - (sum_v e^(z - M) (z - M)) / S
//   dz[i, v] = g_i [v = t_i] - p (g_i + h_i (log p + H_i))
//
// The logits are the loss's (xent.cu; of a few fp32 tokens xent_small.cuh and
// xent_cut.cuh), with statistics of half a tile (of 32 logits there): the maximum, how
// often it occurs, and of the others the sums of e^(z - M) and of e^(z - M) (z - M), so
// that a confident row's log S and H, which are far below 1, keep their digits.  The
// target is left out of them and joins at the end with its logit in fp32.
//
// Likeliest tokens.  The `keep` largest logits lie in the `keep` groups of 32 logits
// with the largest maxima (of equal ones the first): each of those has a logit that
// comes before any of another group.  So the product writes the maxima, and the logits
// themselves for a piece of the vocabulary; a block per row then reads V / 32 maxima and
// `keep` lines of logits, whatever the data.  Eight more than asked for are kept, and
// neighbours in the order that are too close are ranked by their products summed again
// in twice fp32's precision.  What a logit is off by goes with the size of its terms, not
// with its own, where terms cancel: too close are two that are within 2^-15 of the largest
// sum |x w| of those kept (each is within 10^-5 of its own), or, where the rows are few or
// fp32, any two.  Equal logits rank by their ids.  Included by xent.cu.
#pragma once

namespace snack {
namespace {

constexpr int kMostTop = 24;
constexpr int kKeepMore = 8;
// of a block: four warps, or where the rows are few four for the likeliest tokens, four for the statistics beside them, one
// for the target's logit, and all 32 for what is summed again (8 rows of 32768, 20 tokens: the call 38.3 us, 40.4 with 17 warps;
// 2048 rows of 65536, 8 tokens: blocks of eight warps 841 us where those of four took 834)
constexpr int kTopWarps = 4, kTopThreads = kTopWarps * 32;
constexpr int kFinishThreads = 1024;
constexpr int kFoundFew = 256;  // keys that are ranked by counting
constexpr int kNoId = 0x7FFFFFFF;
constexpr int kFound = (kMostTop + kKeepMore) * 32;  // all logits of the groups that are looked at

// ------------------------------------------------------------ statistics

// (maximum, how often, rest, slope) of two sets of logits
__device__ __forceinline__ float4 join_stats(float4 a, float4 b) {
  if (b.x > a.x) {
    const float4 t = a;
    a = b;
    b = t;
  }
  if (b.x == a.x) {
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
  } else if (b.x == -INFINITY) {
    a.z += b.z;  // 0, or a NaN to keep
  } else {
    const float d = b.x - a.x, f = expf(d), all = b.y + b.z;
    a.z = fmaf(f, all, a.z);
    a.w = fmaf(f, fmaf(all, fmaxf(d, kFarBelow), b.w), a.w);
  }
  return a;
}

// Statistics and maxima of the logits of a few tokens, [vocab][tokens]: a thread for
// each group of 32 and token.
__global__ void __launch_bounds__(256) k_score_stats(const float *__restrict__ z, int32_t tokens, int32_t n, int64_t vocab,
                                                     int32_t groups, TokenSrc targets, float4 *__restrict__ stats,
                                                     float *__restrict__ high, float *__restrict__ zt) {
  pdl_wait();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int t = (int)(i % tokens);
  const int64_t group = i / tokens;
  if (group >= groups || t >= n) return;
  const uint32_t id = targets.ids ? targets.key(t) : (uint32_t)vocab;
  const int64_t v0 = group * 32;
  const int own = (int64_t)id >= v0 && (int64_t)id < v0 + 32 && id < (uint32_t)vocab ? (int)(id - v0) : -1;
  float v[32], top = -INFINITY, mx = -INFINITY;
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = v0 + j < vocab ? __ldg(z + (v0 + j) * tokens + t) : -INFINITY;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    top = fmaxf(top, v[j]);
    if (j == own) {  // joined later
      zt[t] = v[j];
      v[j] = -INFINITY;
    }
    mx = fmaxf(mx, v[j]);
  }
  const float base = mx == -INFINITY ? 0.f : mx;
  float often = 0.f, rest = 0.f, slope = 0.f;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const float d = v[j] - base, e = expf(d);
    if (d == 0.f && mx != -INFINITY)
      often += 1.f;
    else
      rest += e;
    slope = fmaf(e, fmaxf(d, kFarBelow), slope);
  }
  stats[(size_t)t * groups + group] = make_float4(mx, often, rest, slope);
  if (high) high[(size_t)t * groups + group] = top;
}

// ------------------------------------------------------------ likeliest tokens

struct FinishArgs {
  int32_t n;
  TokenSrc targets;  // ids null: none given
  // likeliest tokens: the piece's maxima and logits
  int32_t top, keep, groups, rows, v0;
  const float *high, *z;
  int64_t high_ld, z_row, z_col;  // steps of a logit's row and column
  unsigned long long *list;       // [n][32] what is kept from piece to piece
  int first, last;
  TargetLogit at;                 // x and w
  // statistics
  const float4 *stats;
  int64_t stats_ld;
  int32_t slots;
  const float *zt;                // the targets' logits (else formed here)
  // results
  float *logp, *entropy, *top_logp, *lse, *kept_entropy;
  int64_t *top_ids;
  const uint32_t *err;
};

// A logit and its id as one number, in the order of the likeliest: larger logits, of
// equal ones lower ids (0: none).  NaN counts as the lowest logit, -0 as 0.
typedef unsigned long long Key;
__device__ __forceinline__ uint32_t place_of_value(float v) {
  const uint32_t u = __float_as_uint((isnan(v) ? -INFINITY : v) + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ Key key_of(float v, int id) { return (Key)place_of_value(v) << 32 | (uint32_t)~id; }
__device__ __forceinline__ float key_value(Key k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ int key_id(Key k) { return (int)~(uint32_t)k; }

// Lists of 32 keys, lane l has the l-th largest; all of a converged warp.
__device__ __forceinline__ Key swap_step(Key k, int d, bool larger) {
  const Key o = __shfl_xor_sync(0xffffffffu, k, d);
  return larger == (k > o) ? k : o;
}
__device__ __forceinline__ Key sorted(Key k, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size *= 2)
#pragma unroll
    for (int d = size / 2; d; d /= 2) k = swap_step(k, d, ((lane & d) == 0) == ((lane & size) == 0 || size == 32));
  return k;
}
// the 32 largest of two sorted lists
__device__ __forceinline__ Key joined(Key a, Key b, int lane) {
  const Key o = __shfl_sync(0xffffffffu, b, 31 - lane);
  Key k = a > o ? a : o;
#pragma unroll
  for (int d = 16; d; d /= 2) k = swap_step(k, d, (lane & d) == 0);
  return k;
}
// the list with what each lane has to offer, if that is among its first `keep`
__device__ __noinline__ Key offered(Key list, Key k, int keep, int lane) {
  unsigned m = __ballot_sync(0xffffffffu, k > __shfl_sync(0xffffffffu, list, keep - 1));
  if (__popc(m) > 4) return joined(list, sorted(k, lane), lane);
  for (; m; m &= m - 1) {
    const Key n = __shfl_sync(0xffffffffu, k, __ffs(m) - 1), up = __shfl_up_sync(0xffffffffu, list, 1);
    const int at = __popc(__ballot_sync(0xffffffffu, list > n));
    list = lane < at ? list : lane == at ? n : up;
  }
  return list;
}

// the warps that look for the likeliest
__device__ __forceinline__ void top_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kTopThreads) : "memory"); }
// the `keep` largest of n distinct keys, in their order; all of them
__device__ __noinline__ void choose(const Key *keys, int n, Key *chosen, int keep) {
  for (int i = threadIdx.x; i < n; i += kTopThreads) {
    const Key own = keys[i];
    int place = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) place += keys[j] > own ? 1 : 0;
    if (place < keep) chosen[place] = own;
  }
}

// hi + lo += a * b, to about twice fp32's precision; kExact: the product fits fp32, as that of two bf16 does
template <bool kExact>
__device__ __forceinline__ void add_product(float &hi, float &lo, float a, float b) {
  const float p = __fmul_rn(a, b);
  const float s = __fadd_rn(hi, p), t = __fsub_rn(s, hi);
  const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(p, t));
  lo = __fadd_rn(lo, kExact ? e : __fadd_rn(__fmaf_rn(a, b, -p), e));
  hi = s;
}
// a number in the order of hi + lo, an integer (double's own comparisons and sums are slow here)
__device__ __forceinline__ long long order_of(float hi, float lo) {
  const long long bits = __double_as_longlong((double)(hi + 0.f) + (double)lo);  // -0 as 0
  return bits < 0 ? bits ^ 0x7FFFFFFFFFFFFFFFLL : bits;
}
// hi + lo += b, to about twice fp32's precision
__device__ __forceinline__ void add_two(float &hi, float &lo, float b_hi, float b_lo) {
  const float s = __fadd_rn(hi, b_hi), t = __fsub_rn(s, hi);
  const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(b_hi, t));
  lo = __fadd_rn(__fadd_rn(lo, b_lo), e);
  hi = s;
}
// the logit of a row and a token, by a warp: hi + lo
template <typename T>
__device__ __noinline__ float2 long_logit(const TargetLogit &at, int64_t row, int64_t id, int lane) {
  constexpr int kN = 16 / (int)sizeof(T);
  const T *a = reinterpret_cast<const T *>(at.x) + row * at.x_ld, *b = reinterpret_cast<const T *>(at.w) + id * at.w_ld;
  const int groups = (at.width + kN - 1) / kN;
  float hi = 0.f, lo = 0.f;
#pragma unroll 4
  for (int g = lane; g < groups; g += 32) {
    const Pack<T, 16> p = TargetLogit::some(a, g, at.width, at.x_wide), q = TargetLogit::some(b, g, at.width, at.w_wide);
#pragma unroll
    for (int e = 0; e < kN; ++e) add_product<sizeof(T) == 2>(hi, lo, p.get(e), q.get(e));
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const float o_hi = __shfl_xor_sync(0xffffffffu, hi, d), o_lo = __shfl_xor_sync(0xffffffffu, lo, d);
    add_two(hi, lo, o_hi, o_lo);
  }
  return make_float2(hi, lo);
}

// Of a row and kept tokens i0 .. i0 + 15 of bf16: a warp's share of their sums of |x w|, in .x of token i0 + lane / 4 and in .y
// of the eighth after it.  Tokens are the rows of mma.sync; which columns of 32 a lane holds does not matter to a sum.
__device__ __noinline__ float2 term_sizes(const TargetLogit &at, int64_t row, const Key *chosen, int keep, int i0, int warp, int lane) {
  constexpr uint32_t kNoSigns = 0x7FFF7FFFu;
  const int q = lane & 3, groups = (at.width + 7) / 8;
  const bf16 *x = reinterpret_cast<const bf16 *>(at.x) + row * at.x_ld, *w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = i0 + 8 * h + (lane >> 2);
    const Key k = i < keep && chosen[i] ? chosen[i] : chosen[0];
    w[h] = reinterpret_cast<const bf16 *>(at.w) + (int64_t)key_id(k) * at.w_ld;
  }
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int g0 = 4 * warp; g0 < groups; g0 += 4 * kTopWarps) {
    const Pack<bf16, 16> b = TargetLogit::some(x, g0 + q, at.width, at.x_wide), lo = TargetLogit::some(w[0], g0 + q, at.width, at.w_wide),
                         hi = TargetLogit::some(w[1], g0 + q, at.width, at.w_wide);
#pragma unroll
    for (int s = 0; s < 4; s += 2) {
      const uint32_t a[4] = {lo.w[s] & kNoSigns, hi.w[s] & kNoSigns, lo.w[s + 1] & kNoSigns, hi.w[s + 1] & kNoSigns};
      mma16816(acc, a, b.w[s] & kNoSigns, b.w[s + 1] & kNoSigns);
    }
  }
  return make_float2(acc[0], acc[2]);
}

// A block per row.  kFew: few rows, a large block each.
template <bool kFew>
__global__ void __launch_bounds__(kFew ? kFinishThreads : kTopThreads) k_score_finish(const FinishArgs a) {
  pdl_wait();
  __shared__ Key chosen[32];
  __shared__ __align__(16) uint32_t bests[kTopThreads];
  __shared__ uint32_t least_best;
  __shared__ __align__(16) Key found[kFound + 32];
  __shared__ float4 sums[kTopWarps];
  __shared__ float2 exact[32];
  __shared__ float sizes[kTopWarps][32];
  __shared__ float target_z;
  __shared__ int n_found;
  const int64_t row = blockIdx.x;
  constexpr int warps = (kFew ? kFinishThreads : kTopThreads) / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool bad = a.last && any_error(a.err);
  const uint32_t target = a.targets.ids ? a.targets.key(row) : a.targets.vocab;
  const bool given = target < a.targets.vocab;
  if (a.targets.ids && !given) {  // not scored
    if (!a.last) return;
    for (int i = threadIdx.x; i < a.top; i += 32 * warps) {
      a.top_ids[row * a.top + i] = -1;
      a.top_logp[row * a.top + i] = 0.f;
    }
    if (threadIdx.x == 0) {
      if (a.logp) a.logp[row] = 0.f;
      if (a.entropy) a.entropy[row] = 0.f;
      a.lse[row] = 0.f;
      a.kept_entropy[row] = 0.f;
    }
    return;
  }
  Key list = 0;
  if (warp < kTopWarps && a.top) {
    // The groups with the largest maxima: none of them is below what `keep` of the threads'
    // own largest ones reach, and few others reach it.
    const float *high = a.high + row * a.high_ld;
    uint32_t best = 0;
#pragma unroll 8
    for (int g = threadIdx.x; g < a.groups; g += kTopThreads) best = max(best, place_of_value(__ldg(high + g)));
    bests[threadIdx.x] = best;
    if (threadIdx.x < 32) chosen[threadIdx.x] = 0;
    if (threadIdx.x == 0) {
      n_found = 0;
      least_best = 0;
    }
    top_sync();
    int reached = 0;
#pragma unroll
    for (int i = 0; i < kTopThreads; i += 4) {
      const uint4 four = *reinterpret_cast<const uint4 *>(bests + i);
      reached += (four.x >= best ? 1 : 0) + (four.y >= best ? 1 : 0) + (four.z >= best ? 1 : 0) + (four.w >= best ? 1 : 0);
    }
    if (reached >= a.keep) atomicMax(&least_best, best);
    top_sync();
    const uint32_t from = least_best;
#pragma unroll 4
    for (int g = threadIdx.x; g < a.groups; g += kTopThreads) {
      const float v = __ldg(high + g);
      if (place_of_value(v) >= from) {
        const int at = atomicAdd(&n_found, 1);  // their order does not matter
        if (at < kFound) found[at] = key_of(v, g);
      }
    }
    top_sync();
    int n = n_found;
    if (n <= kFoundFew) {
      choose(found, n, chosen, a.keep);
    } else if (warp == 0) {
      if (n <= kFound) {
#pragma unroll 1
        for (int i = 0; i < n; i += 32) list = offered(list, i + lane < n ? found[i + lane] : 0, a.keep, lane);
      } else {  // a few threads have most of the large ones
#pragma unroll 1
        for (int g = lane; g - lane < a.groups; g += 32) list = offered(list, g < a.groups ? key_of(__ldg(high + g), g) : 0, a.keep, lane);
      }
      chosen[lane] = list;
    }
    top_sync();
    if (threadIdx.x == 0) n_found = 0;
    // and of their logits those that are not below the last group's maximum
    constexpr int kMost = (kMostTop + kKeepMore + kTopWarps - 1) / kTopWarps;
    const Key last_group = chosen[a.keep - 1];
    const Key least = last_group ? key_of(key_value(last_group), kNoId) : 0;
    Key k[kMost];
#pragma unroll
    for (int u = 0; u < kMost; ++u) {
      const int i = warp + u * kTopWarps;
      const Key of = i < a.keep ? chosen[i] : 0;
      const int col = of ? key_id(of) * 32 + lane : a.rows;
      k[u] = col < a.rows ? key_of(__ldg(a.z + row * a.z_row + col * a.z_col), a.v0 + col) : 0;
    }
    top_sync();
#pragma unroll
    for (int u = 0; u < kMost; ++u)
      if (k[u] && k[u] >= least) found[atomicAdd(&n_found, 1)] = k[u];
    if (!a.first && warp == 0) {
      const Key old = a.list[row * 32 + lane];
      if (old) found[atomicAdd(&n_found, 1)] = old;
    }
    if (warp == kTopWarps - 1) chosen[lane] = 0;  // read by all already
    top_sync();
    n = n_found;
    if (n <= kFoundFew) {
      choose(found, n, chosen, a.keep);
    } else if (warp == 0) {
      list = 0;
#pragma unroll 1
      for (int i = 0; i < n; i += 32) list = offered(list, i + lane < n ? found[i + lane] : 0, a.keep, lane);
      chosen[lane] = lane < a.keep ? list : 0;
    }
    top_sync();
    if (warp == 0) {
      list = chosen[lane];
      if (!a.last) a.list[row * 32 + lane] = list;
    }
  }
  if (!a.last) return;
  if (const int mine = warp - (kFew ? kTopWarps : 0); mine >= 0 && mine < kTopWarps) {  // the row's statistics
    float4 s = make_float4(-INFINITY, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 32 * mine + lane; i < a.slots; i += kTopThreads) s = join_stats(s, a.stats[row * a.stats_ld + i]);
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {  // lane by lane upwards: the same result in all
      float4 o;
      o.x = __shfl_xor_sync(0xffffffffu, s.x, d);
      o.y = __shfl_xor_sync(0xffffffffu, s.y, d);
      o.z = __shfl_xor_sync(0xffffffffu, s.z, d);
      o.w = __shfl_xor_sync(0xffffffffu, s.w, d);
      s = lane & d ? join_stats(o, s) : join_stats(s, o);
    }
    if (lane == 0) sums[mine] = s;
  }
  if (given && warp == warps - 1) {
    const float z = a.zt ? a.zt[row] : a.at.get(row, target);
    if (lane == 0) target_z = z;
  }
  __syncthreads();
  unsigned again = 0;  // what is summed again
  if (a.top) {
    float slack = INFINITY;
    if (!kFew && a.at.bf) {
      for (int i0 = 0; i0 < a.keep; i0 += 16) {
        const float2 size = term_sizes(a.at, row, chosen, a.keep, i0, warp, lane);
        if ((lane & 3) == 0) {
          sizes[warp][i0 + (lane >> 2)] = size.x;
          sizes[warp][i0 + 8 + (lane >> 2)] = size.y;
        }
      }
      __syncthreads();
      float size = 0.f;
#pragma unroll
      for (int w = 0; w < kTopWarps; ++w) size += lane < a.keep ? sizes[w][lane] : 0.f;
#pragma unroll
      for (int d = 16; d; d >>= 1) size = fmaxf(size, __shfl_xor_sync(0xffffffffu, size, d));
      slack = size * 0x1p-15f;
    }
    const Key own = chosen[lane];
    const float mine = own ? key_value(own) : -INFINITY, above = __shfl_up_sync(0xffffffffu, mine, 1);
    const bool close = lane > 0 && own && !(above - mine > slack);
    const unsigned with = __ballot_sync(0xffffffffu, close);  // bit l: l goes with l - 1
    // a run of them that begins before place `top`
    const int begin = 31 - __clz(~with & (0xffffffffu >> (31 - lane)));
    const bool run = close || (lane < 31 && (with >> (lane + 1)) & 1);
    again = __ballot_sync(0xffffffffu, run && begin < a.top);
    int k = 0;
    for (unsigned m = again; m; m &= m - 1, ++k) {
      if (k % warps != warp) continue;
      const int i = __ffs(m) - 1, id = key_id(chosen[i]);
      const float2 l = a.at.bf ? long_logit<bf16>(a.at, row, id, lane) : long_logit<float>(a.at, row, id, lane);
      if (lane == 0) exact[i] = l;
    }
    __syncthreads();
  }
  if (warp) return;
  float4 s = sums[0];
#pragma unroll
  for (int w = 1; w < kTopWarps; ++w) s = join_stats(s, sums[w]);
  const float z = given ? target_z : 0.f;
  // the largest logit with the target's, and of the sums relative to it what is over 1
  float high = s.x, over, slope;
  if (given && z >= s.x) {
    const float d = s.x - z, f = s.x == -INFINITY ? 0.f : expf(d), all = s.y + s.z;
    high = z;
    over = s.x == -INFINITY ? s.z : f * all;
    slope = s.x == -INFINITY ? 0.f : f * fmaf(all, fmaxf(d, kFarBelow), s.w);
  } else {
    const float d = z - s.x, f = given ? expf(d) : 0.f;
    over = (s.y - 1.f) + s.z + f;
    slope = given ? fmaf(f, fmaxf(d, kFarBelow), s.w) : s.w;
  }
  if (bad || !(high < INFINITY) || isnan(z)) over = NAN;
  const float log_sum = log1pf(over), logp = (z - high) - log_sum, entropy = log_sum - slope / (1.f + over);
  if (lane == 0) {
    if (a.logp) a.logp[row] = given ? logp : 0.f;
    if (a.entropy) a.entropy[row] = entropy;
    a.lse[row] = high + log_sum;
    a.kept_entropy[row] = entropy;
  }
  if (!a.top) return;
  const int id = key_id(list);
  float2 l = make_float2(key_value(list), 0.f);
  if ((again >> lane) & 1 && isfinite(exact[lane].x)) l = exact[lane];
  const long long mine = order_of(l.x, l.y);
  int place = 0;
  for (int j = 0; j < a.keep; ++j) {
    const long long other = __shfl_sync(0xffffffffu, mine, j);
    const int ij = __shfl_sync(0xffffffffu, id, j);
    place += other > mine || (other == mine && ij < id) ? 1 : 0;
  }
  // the first one's log probability by the statistics' own logits, whose errors it shares; the others' by what is between them
  const int best = __ffs(__ballot_sync(0xffffffffu, lane < a.keep && place == 0)) - 1;
  const bool of_target = given && id == (int)target;
  const float first = __shfl_sync(0xffffffffu, of_target ? logp : (key_value(list) - high) - log_sum, best);
  const float2 top_l = make_float2(__shfl_sync(0xffffffffu, l.x, best), __shfl_sync(0xffffffffu, l.y, best));
  if (lane < a.keep && place < a.top) {
    a.top_ids[row * a.top + place] = id;
    a.top_logp[row * a.top + place] = of_target ? logp : place ? ((l.x - top_l.x) + (l.y - top_l.y)) + first : first;
  }
}

// The gradients' weights as the loss's: of the log probability's negative, and of the
// entropy; targets where none are given; and which rows of x have which target.
__global__ void __launch_bounds__(256) k_score_weights(int32_t n, const float *__restrict__ dlogp, const float *__restrict__ dentropy,
                                                       float *__restrict__ weight, float *__restrict__ went, int32_t *__restrict__ ids,
                                                       TokenSrc targets, const Hits hits) {
  pdl_wait();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const float g = dlogp ? -dlogp[i] : 0.f, h = dentropy ? -dentropy[i] : 0.f;
  weight[i] = g;
  went[i] = h;
  if (ids) {
    ids[i] = 0;
  } else if (hits.first && g != 0.f) {
    const uint32_t id = targets.key(i);
    if (id < targets.vocab) {
      atomicMin(hits.first + id, i);
      atomicMax(hits.last + id, i);
    }
  }
}

// ------------------------------------------------------------ host side

// What the gradient takes besides the loss's: weights and targets, and for bf16 the
// targets' rows of dw.
struct ScoreGradWs {
  size_t weight, went, ids, first, last, rows, total;
  int64_t rows_ld;
};
ScoreGradWs score_grad_ws(const XentShape &s, const XentWs &x) {
  ScoreGradWs w = {};
  size_t o = x.total;
  auto take = [&o](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes, kAlign);
    return at;
  };
  w.weight = take((size_t)s.n * 4);
  w.went = take((size_t)s.n * 4);
  w.ids = take((size_t)s.n * 4);
  if (s.t == SNACK_BF16) {
    w.first = take((size_t)s.vocab * 4);
    w.last = take((size_t)s.vocab * 4);
    w.rows_ld = (int64_t)align_up((size_t)s.width, 4);
    w.rows = take((size_t)s.n * (size_t)w.rows_ld * 4);
  }
  w.total = o;
  return w;
}

struct ScoreWs {
  size_t err, zt, xp, wp, z, stats, high, list, total;
  int32_t tokens;             // few tokens: those that the logits' kernel is built for
  int64_t piece, slots;
  int64_t z_ld, high_ld;
  int nt;
};

ScoreWs score_ws(const XentShape &s, int32_t top) {
  ScoreWs w = {};
  size_t o = 0;
  auto take = [&o](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes, kAlign);
    return at;
  };
  const int64_t m_tiles = ceil_div(s.n, kM);
  w.err = take(256 * 4);
  w.zt = take((size_t)s.n * 4);
  if (s.few || s.cut) {
    w.tokens = s.few ? kFewMostLogits : cut_tokens(s.n);
    w.piece = s.vocab;
    w.high_ld = w.slots = ceil_div(s.vocab, 32);
    w.z = take((size_t)s.vocab * (size_t)w.tokens * 4);
  } else {
    // logits a gigabyte at a time, w's copies a quarter of that
    const int64_t w_row = (int64_t)s.parts * s.ld * 2, row = std::max(s.pack_w ? w_row : 0, top ? (int64_t)s.n : 0);
    if (s.pack_x) w.xp = take((size_t)s.parts * (size_t)s.n * (size_t)s.ld * 2);
    w.piece = row ? piece_rows(s.vocab, row, m_tiles, s.sms) : s.vocab;
    if (w.piece > s.vocab) w.piece = s.vocab;
    if (s.pack_w) w.wp = take((size_t)s.parts * (size_t)w.piece * (size_t)s.ld * 2);
    w.nt = tile_cols(m_tiles, w.piece, s.sms);
    w.slots = 2 * (ceil_div(s.vocab, w.piece) * ceil_div(w.piece, w.nt));
    w.z_ld = ceil_div(w.piece, 64) * 64;
    w.high_ld = ceil_div(w.piece, w.nt) * w.nt / 32;
    if (top) w.z = take((size_t)s.n * (size_t)w.z_ld * 4);
    if (top && w.piece < s.vocab) w.list = take((size_t)s.n * 32 * 8);
  }
  w.stats = take((size_t)s.n * (size_t)w.slots * 16);
  if (top) w.high = take((size_t)s.n * (size_t)w.high_ld * 4);
  w.total = o;
  return w;
}

cudaError_t score_logits_few(const XentShape &S, const ScoreWs &W, const void *x, int64_t x_ld, const void *w, int64_t w_ld,
                             const TokenSrc &tg, float *z, cudaStream_t s) {
  if (S.few) {
    SmallArgs a = small_args(S, x, x_ld, w, w_ld, tg);
    a.dz = z;
    const int64_t tiles = ceil_div(S.vocab, (int64_t)kSmallWarps * kSmallRows);
    return launch_few<true>(a, tiles < S.sms ? tiles : S.sms, s);
  }
  CutArgs c = cut_args(S, x, x_ld, w, w_ld, tg);
  c.dz = z;
  return launch_cut_for<true>(c, cut_blocks(S, S.vocab), s);
}

}  // namespace
}  // namespace snack

extern "C" {

snack_status snack_score_workspace_size(const void *x, int64_t x_ld, int32_t n, const void *w, int64_t w_ld,
                                        int64_t vocab, int32_t width, snack_dtype t, int32_t top, int grad, size_t *bytes) {
  if (!bytes) return SNACK_ERR_INVALID_ARG;
  const snack_status st = xent_check(x, x_ld, n, w, w_ld, vocab, width, t);
  if (st != SNACK_OK) return st;
  if (top < 0 || top > vocab) return SNACK_ERR_INVALID_ARG;
  if (top > kMostTop) return SNACK_ERR_UNSUPPORTED;
  const XentShape S = xent_shape(x, x_ld, n, w, w_ld, vocab, width, t, grad != 0);
  *bytes = n == 0 ? 0 : grad ? score_grad_ws(S, xent_ws(S, true)).total : score_ws(S, top).total;
  return SNACK_OK;
}

snack_status snack_score_fwd(const void *x, int64_t x_ld, int32_t n, const void *w, int64_t w_ld, int64_t vocab,
                             int32_t width, snack_dtype t, const void *targets, snack_index targets_t, float *logp,
                             float *entropy, int32_t top, int64_t *top_ids, float *top_logp, float *state, void *ws,
                             size_t ws_bytes, snack_stream_t stream) try {
  const snack_status ck = xent_check(x, x_ld, n, w, w_ld, vocab, width, t);
  if (ck != SNACK_OK) return ck;
  if (!lm_index_ok(targets_t) || top < 0 || top > vocab) return SNACK_ERR_INVALID_ARG;
  if (top > kMostTop) return SNACK_ERR_UNSUPPORTED;
  if (n == 0) return SNACK_OK;
  if (!x || !w || !state || !ws || (top > 0 && (!top_ids || !top_logp)) || (logp && !targets) ||
      !ptr_aligned(targets, index_size(targets_t)) || !ptr_aligned(logp, 4) || !ptr_aligned(entropy, 4) || !ptr_aligned(state, 4) ||
      !ptr_aligned(top_ids, 8) || !ptr_aligned(top_logp, 4) || !ptr_aligned(ws, kAlign))
    return SNACK_ERR_INVALID_ARG;
  const XentShape S = xent_shape(x, x_ld, n, w, w_ld, vocab, width, t, false);
  const ScoreWs W = score_ws(S, top);
  if (ws_bytes < W.total) return SNACK_ERR_WORKSPACE;
  const size_t es = dtype_size(t);
  const Span written[] = {{logp, logp ? (size_t)n * 4 : 0},
                          {entropy, entropy ? (size_t)n * 4 : 0},
                          {top_ids, (size_t)n * (size_t)top * 8},
                          {top_logp, (size_t)n * (size_t)top * 4},
                          {state, (size_t)n * 8},
                          {ws, W.total}};
  const Span read[] = {{x, span_bytes(n, width, x_ld, es)}, {w, span_bytes(vocab, width, w_ld, es)},
                       {targets, targets ? (size_t)n * index_size(targets_t) : 0}};
  if (any_overlap(written, read)) return SNACK_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t *b = reinterpret_cast<uint8_t *>(ws);
  const TokenSrc tg{targets, targets_t == SNACK_I64, (uint32_t)vocab};
  FinishArgs f = {};
  f.n = n;
  f.targets = tg;
  f.top = top;
  f.keep = (int32_t)std::min<int64_t>(top + kKeepMore, vocab);
  f.high = top ? reinterpret_cast<const float *>(b + W.high) : nullptr;
  f.high_ld = W.high_ld;
  f.z = reinterpret_cast<const float *>(b + W.z);
  f.list = reinterpret_cast<unsigned long long *>(b + W.list);
  f.first = f.last = 1;
  f.at = target_logit(S, x, x_ld, w, w_ld);
  f.stats = reinterpret_cast<const float4 *>(b + W.stats);
  f.stats_ld = W.slots;
  f.logp = logp;
  f.entropy = entropy;
  f.top_logp = top_logp;
  f.top_ids = top_ids;
  f.lse = state;
  f.kept_entropy = state + n;
  auto finish = [&] {
    return n <= S.sms ? launch_pdl(k_score_finish<true>, (unsigned)n, kFinishThreads, 0, s, (const FinishArgs)f)
                      : launch_pdl(k_score_finish<false>, (unsigned)n, kTopThreads, 0, s, (const FinishArgs)f);
  };
  if (W.tokens) {
    f.groups = f.slots = (int32_t)W.slots;
    f.rows = (int32_t)vocab;
    f.z_row = 1;
    f.z_col = W.tokens;
  }
  if (W.tokens) {
    float *z = reinterpret_cast<float *>(b + W.z), *zt = reinterpret_cast<float *>(b + W.zt);
    XENT_CUDA(score_logits_few(S, W, x, x_ld, w, w_ld, tg, z, s));
    const int64_t threads = W.slots * W.tokens;
    XENT_CUDA(launch_pdl(k_score_stats, (unsigned)ceil_div(threads, 256), 256, 0, s, (const float *)z, W.tokens, n, vocab,
                         (int32_t)W.slots, tg, reinterpret_cast<float4 *>(b + W.stats), top ? reinterpret_cast<float *>(b + W.high) : nullptr,
                         zt));
    f.zt = zt;  // of the same sums as the others, and the gradient's
    XENT_CUDA(finish());
    return SNACK_OK;
  }
  const uint32_t a_rows = n >= kMCta ? kMCta : (uint32_t)align_up((size_t)n, 8);
  Operand ox, ow;
  XENT_CUDA(operand(S, S.pack_x, x, x_ld, 0, n, b + W.xp, &ox, s));
  CUtensorMap mx, mw, mz;
  if (!load_map(&mx, ox, false, a_rows)) return SNACK_ERR_CUDA;
  GemmArgs g = gemm_args(S, b, XentWs{}, 1);
  g.err = reinterpret_cast<uint32_t *>(b + W.err);
  g.m = n;
  g.nt = W.nt;
  g.k_blocks = (int32_t)ceil_div(width, kKb);
  g.targets = tg;
  g.stats = reinterpret_cast<float4 *>(b + W.stats);
  g.stats_ld = W.slots;
  g.high = top ? reinterpret_cast<float *>(b + W.high) : nullptr;
  g.high_ld = W.high_ld;
  f.err = g.err;
  f.z_row = W.z_ld;
  f.z_col = 1;
  for (int64_t v0 = 0; v0 < vocab; v0 += W.piece) {
    const int64_t rows = vocab - v0 < W.piece ? vocab - v0 : W.piece;
    XENT_CUDA(operand(S, S.pack_w, w, w_ld, v0, rows, b + W.wp, &ow, s));
    if (!load_map(&mw, ow, false, (uint32_t)W.nt / 2)) return SNACK_ERR_CUDA;
    if (top && !make_map(&mz, f.z, true, (uint64_t)rows, (uint64_t)n, (uint64_t)W.z_ld, 1, (uint64_t)n * (uint64_t)W.z_ld, 32, 32,
                         CU_TENSOR_MAP_SWIZZLE_128B))
      return SNACK_ERR_CUDA;
    g.n = (int32_t)rows;
    g.v0 = (int32_t)v0;
    XENT_CUDA(launch_gemm<kScore>(mx, mw, top ? mz : mx, g, S.sms, s));
    g.slot0 += 2 * g.n_tiles;
    f.last = v0 + rows == vocab;
    f.slots = g.slot0;
    f.groups = (int32_t)ceil_div(rows, 32);
    f.rows = (int32_t)rows;
    f.v0 = (int32_t)v0;
    if (top || f.last) XENT_CUDA(finish());
    f.first = 0;
  }
  return SNACK_OK;
} catch (...) {  // a host allocation failed
  return SNACK_ERR_CUDA;
}

snack_status snack_score_bwd(const void *x, int64_t x_ld, int32_t n, const void *w, int64_t w_ld, int64_t vocab,
                             int32_t width, snack_dtype t, const void *targets, snack_index targets_t, const float *state,
                             const float *dlogp, const float *dentropy, void *dx, int64_t dx_ld, void *dw, int64_t dw_ld,
                             void *ws, size_t ws_bytes, snack_stream_t stream) try {
  const snack_status ck = xent_check(x, x_ld, n, w, w_ld, vocab, width, t);
  if (ck != SNACK_OK) return ck;
  const size_t es = dtype_size(t);
  if (!lm_index_ok(targets_t) || (dlogp && !targets)) return SNACK_ERR_INVALID_ARG;
  if ((dx && (dx_ld < width || !ptr_aligned(dx, es))) || (dw && (dw_ld < width || !ptr_aligned(dw, es))))
    return SNACK_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (n == 0) {
    if (dw) XENT_CUDA(cudaMemset2DAsync(dw, (size_t)dw_ld * es, 0, (size_t)width * es, (size_t)vocab, s));
    return SNACK_OK;
  }
  if (!x || !w || !state || !ws || !ptr_aligned(targets, index_size(targets_t)) || !ptr_aligned(state, 4) || !ptr_aligned(ws, kAlign) ||
      !ptr_aligned(dlogp, 4) || !ptr_aligned(dentropy, 4))
    return SNACK_ERR_INVALID_ARG;
  const XentShape S = xent_shape(x, x_ld, n, w, w_ld, vocab, width, t, true);
  const XentWs W = xent_ws(S, true);
  const ScoreGradWs E = score_grad_ws(S, W);
  const Span written[] = {{dx, dx ? span_bytes(n, width, dx_ld, es) : 0}, {dw, dw ? span_bytes(vocab, width, dw_ld, es) : 0},
                          {ws, std::min(ws_bytes, E.total)}};
  const Span read[] = {{x, span_bytes(n, width, x_ld, es)}, {w, span_bytes(vocab, width, w_ld, es)},
                       {targets, targets ? (size_t)n * index_size(targets_t) : 0}, {state, (size_t)n * 8},
                       {dlogp, dlogp ? (size_t)n * 4 : 0}, {dentropy, dentropy ? (size_t)n * 4 : 0}};
  if (any_overlap(written, read)) return SNACK_ERR_INVALID_ARG;
  if (ws_bytes < E.total) return SNACK_ERR_WORKSPACE;
  if (!dx && !dw) return SNACK_OK;
  uint8_t *b = reinterpret_cast<uint8_t *>(ws);
  float *weight = reinterpret_cast<float *>(b + E.weight), *went = reinterpret_cast<float *>(b + E.went);
  int32_t *ids = targets ? nullptr : reinterpret_cast<int32_t *>(b + E.ids);
  Hits hits = {};
  if (t == SNACK_BF16 && dw && dlogp) {
    hits = {reinterpret_cast<int32_t *>(b + E.first), reinterpret_cast<int32_t *>(b + E.last), reinterpret_cast<float *>(b + E.rows), E.rows_ld};
    XENT_CUDA(cudaMemsetAsync(hits.first, 0x7F, (size_t)vocab * 4, s));  // above every row
    XENT_CUDA(cudaMemsetAsync(hits.last, 0, (size_t)vocab * 4, s));
  }
  const TokenSrc tg = targets ? TokenSrc{targets, targets_t == SNACK_I64, (uint32_t)vocab} : TokenSrc{ids, 0, (uint32_t)vocab};
  XENT_CUDA(launch_pdl(k_score_weights, (unsigned)ceil_div(n, 256), 256, 0, s, n, dlogp, dentropy, weight, went, ids, tg, hits));
  return xent_gradient(S, W, x, x_ld, w, w_ld, tg, weight, Entropy{went, state + n}, hits, Factor{nullptr, nullptr}, state, dx, dx_ld, dw,
                       dw_ld, b, s);
} catch (...) {  // a host allocation failed
  return SNACK_ERR_CUDA;
}

}  // extern "C"
