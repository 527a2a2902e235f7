// Vectors of fp32 and bf16 values at any address: the loads and stores of
// operators whose rows may begin anywhere.  The target takes vector accesses
// of any alignment, so a row of odd width needs no form of its own but for its
// last, shorter piece.
#pragma once

#include "common.h"
#include "mx4.h"

namespace moe {

template <class T>
__device__ __forceinline__ T load_any(const void* p) {
  T v;
  __builtin_memcpy(&v, p, sizeof(T));
  return v;
}
template <class T>
__device__ __forceinline__ void store_any(void* p, T v) {
  __builtin_memcpy(p, &v, sizeof(T));
}

// V values of a row as they lie in memory (V * size bytes).
template <bool F32, int V>
struct RowPiece {
  static constexpr int kSize = F32 ? 4 : 2, kWords = V * kSize / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; i++) w[i] = 0;
  }
  // n of the V values, the others 0.
  __device__ __forceinline__ void load(const void* p, int n) {
    if (n >= V) {
      if constexpr (kWords % 4 == 0) {
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
          const uint4 v = load_any<uint4>(static_cast<const char*>(p) + 4 * i);
          w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
        }
      } else if constexpr (kWords == 2) {
        const uint2 v = load_any<uint2>(p);
        w[0] = v.x, w[1] = v.y;
      } else {
#pragma unroll
        for (int i = 0; i < kWords; i++) w[i] = load_any<uint32_t>(static_cast<const char*>(p) + 4 * i);
      }
      return;
    }
    clear();
#pragma unroll
    for (int i = 0; i < V; i++) {
      if (i >= n) continue;
      if constexpr (F32) w[i] = static_cast<const uint32_t*>(p)[i];
      else w[i / 2] |= (uint32_t)static_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
    }
  }
  __device__ __forceinline__ void store(void* p, int n) const {
    if (n >= V) {
      if constexpr (kWords % 4 == 0) {
#pragma unroll
        for (int i = 0; i < kWords; i += 4)
          store_any(static_cast<char*>(p) + 4 * i, make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]));
      } else if constexpr (kWords == 2) {
        store_any(p, make_uint2(w[0], w[1]));
      } else {
#pragma unroll
        for (int i = 0; i < kWords; i++) store_any(static_cast<char*>(p) + 4 * i, w[i]);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < V; i++) {
      if (i >= n) continue;
      if constexpr (F32) static_cast<uint32_t*>(p)[i] = w[i];
      else static_cast<uint16_t*>(p)[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (F32) return __uint_as_float(w[i]);
    return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
  // Rounded once to the type, NaN kept.
  __device__ __forceinline__ void set(const float v[V]) {
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < V; i++) w[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2) w[i / 2] = f32_to_bf16_bits(v[i]) | f32_to_bf16_bits(v[i + 1]) << 16;
    }
  }
};

}  // namespace moe
