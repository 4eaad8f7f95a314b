// Host-side checks and small device helpers shared by the language-model
// operators (embed.cu, xent.cu, clip.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace snack {

inline bool lm_dtype_ok(snack_dtype t) { return t == SNACK_F32 || t == SNACK_BF16; }
inline bool lm_index_ok(snack_index t) { return t == SNACK_I32 || t == SNACK_I64; }
inline size_t index_size(snack_index t) { return t == SNACK_I64 ? 8 : 4; }
inline bool ptr_aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// bytes from the first element of a [rows][width] matrix (rows ld elements apart) to past its last
inline size_t span_bytes(int64_t rows, int64_t width, int64_t ld, size_t es) {
  return rows > 0 ? ((size_t)(rows - 1) * (size_t)ld + (size_t)width) * es : 0;
}
inline bool spans_overlap(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return na && nb && x < y + nb && y < x + na;
}

// Streaming multiprocessors of the current device (0 when it cannot be read).
inline int current_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

// Widest access, in bytes (16, 8, 4 or 2), that every address, row step and
// row length given divides by.
inline int access_bytes(uintptr_t bits) {
  for (int a = 16; a > 1; a >>= 1)
    if (bits % (uintptr_t)a == 0) return a;
  return 1;
}

// A token id as a sort key: ids outside [0, vocab) become `vocab`, which
// sorts last and names no row.
struct TokenSrc {
  const void *ids;
  int wide;  // 64-bit ids
  uint32_t vocab;
  __device__ __forceinline__ uint32_t key(int64_t i) const {
    if (wide) {
      const int64_t v = reinterpret_cast<const int64_t *>(ids)[i];
      return (uint64_t)v < (uint64_t)vocab ? (uint32_t)v : vocab;
    }
    const int32_t v = reinterpret_cast<const int32_t *>(ids)[i];
    return (uint32_t)v < vocab ? (uint32_t)v : vocab;
  }
  __device__ __forceinline__ uint32_t val(int64_t i) const { return (uint32_t)i; }
};

// The entropies of the rows' distributions in a gradient: a weight per row (null: none)
// and the entropy itself.
struct Entropy {
  const float *weight, *value;
};
// exp(d) below this is 0, and d times it as well, also where d is infinite
constexpr float kFarBelow = -200.f;
// what exp(d) is multiplied by in dz, where d is a log probability: g of the loss, and
// of the entropy H, dH/dz = -p (d + H), with the weight's sign turned
__device__ __forceinline__ float entropy_slope(float g, float weight, float d, float entropy) {
  return fmaf(weight, fmaxf(d, kFarBelow) + entropy, g);
}

// B bytes of consecutive elements of T: one load or store of that width.
template <int B>
struct Raw;
template <>
struct Raw<16> {
  typedef uint4 type;
};
template <>
struct Raw<8> {
  typedef uint2 type;
};
template <>
struct Raw<4> {
  typedef uint32_t type;
};
template <>
struct Raw<2> {
  typedef uint16_t type;
};

template <typename T, int B>
struct Pack {
  static constexpr int kN = B / (int)sizeof(T);
  typedef typename Raw<B>::type R;
  union {
    R raw;
    uint16_t h[B / 2];
    uint32_t w[B / 4 > 0 ? B / 4 : 1];
  };
  __device__ __forceinline__ Pack() {}
  __device__ __forceinline__ float get(int i) const {
    if (sizeof(T) == 4) return __uint_as_float(w[i]);
    return __uint_as_float((uint32_t)h[i] << 16);
  }
  __device__ __forceinline__ void set(int i, float v) {
    if (sizeof(T) == 4)
      w[i] = __float_as_uint(v);
    else
      h[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
};

}  // namespace snack
