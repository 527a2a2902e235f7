// Quantisation to the microscaled 4-bit format and back (format: mx4.h).
//
// Both are bound by memory: 2.53 or 4.53 bytes a value (bf16 or fp32 on the
// wide side), a handful of instructions each.  131072 x 2048 bf16 values there
// and back take 269 us, 5.0 TB/s; a 2 GiB copy reaches 4.9.  A thread takes eight values, so
// a wave's wide side is 1 or 2 KB of consecutive bytes, its codes are one
// dword a lane, and the four lanes of a block find its largest magnitude with
// two lane moves.
#include "launch.h"
#include "mx4.h"

namespace moe {

constexpr int kMxThreads = 256;

// Eight consecutive values; `wide` loads need 16-byte alignment.
template <bool F32, bool Wide>
__device__ __forceinline__ void load8(const void* p, float v[8]) {
  if constexpr (F32) {
    const float* f = static_cast<const float*>(p);
    if constexpr (Wide) {
      const float4 a = *reinterpret_cast<const float4*>(f), b = *reinterpret_cast<const float4*>(f + 4);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = f[i];
    }
  } else {
    const uint16_t* h = static_cast<const uint16_t*>(p);
    if constexpr (Wide) {
      const uint4 a = *reinterpret_cast<const uint4*>(h);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; i++) {
        v[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
        v[2 * i + 1] = bf16_bits_to_f32(w[i] >> 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = bf16_bits_to_f32(h[i]);
    }
  }
}

template <bool F32, bool Wide>
__global__ __launch_bounds__(kMxThreads) void k_mx4_quantize(Mx4RowArgs A) {
  constexpr int kSize = F32 ? 4 : 2;
  const int64_t pieces = A.rows * (A.cols / 8);
  const int per_row = (int)(A.cols / 8);
  const int64_t step = (int64_t)gridDim.x * kMxThreads;
  // cols is a multiple of 32, so the four lanes of a block are all in or all out.
  for (int64_t i = (int64_t)blockIdx.x * kMxThreads + threadIdx.x; i < pieces; i += step) {
    const int64_t row = i / per_row;
    const int64_t col = (i - row * per_row) * 8;
    float v[8];
    load8<F32, Wide>(static_cast<const char*>(A.wide) + (row * A.ld + col) * kSize, v);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) m = max(m, f32_abs_bits(v[j]));
    const int s = mx4_scale_byte(quad_max(m));
    reinterpret_cast<uint32_t*>(A.codes)[i] = mx4_pack8(v, mx4_inv_scale(s));
    if ((i & 3) == 0) A.scales[i >> 2] = (uint8_t)s;
  }
}

template <bool F32, bool Wide>
__global__ __launch_bounds__(kMxThreads) void k_mx4_dequantize(Mx4RowArgs A) {
  const int64_t pieces = A.rows * (A.cols / 8);
  const int per_row = (int)(A.cols / 8);
  const int64_t step = (int64_t)gridDim.x * kMxThreads;
  for (int64_t i = (int64_t)blockIdx.x * kMxThreads + threadIdx.x; i < pieces; i += step) {
    const int64_t row = i / per_row;
    const int64_t col = (i - row * per_row) * 8;
    const uint4 b = mx4_unpack8_bf16(reinterpret_cast<const uint32_t*>(A.codes)[i], mx4_scale_f32(A.scales[i >> 2]));
    const uint32_t w[4] = {b.x, b.y, b.z, b.w};
    if constexpr (F32) {
      float* y = static_cast<float*>(A.wide) + row * A.ld + col;
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        v[2 * j] = bf16_bits_to_f32(w[j] & 0xFFFFu);
        v[2 * j + 1] = bf16_bits_to_f32(w[j] >> 16);
      }
      if constexpr (Wide) {
        *reinterpret_cast<float4*>(y) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(y + 4) = make_float4(v[4], v[5], v[6], v[7]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++) y[j] = v[j];
      }
    } else {
      uint16_t* y = static_cast<uint16_t*>(A.wide) + row * A.ld + col;
      if constexpr (Wide) {
        *reinterpret_cast<uint4*>(y) = b;
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++) y[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
      }
    }
  }
}

// Rows whose first value and stride are multiples of 16 bytes take the wide
// loads and stores; other addresses take them value by value.
static bool wide_rows(const Mx4RowArgs& A) {
  const int64_t size = A.f32 ? 4 : 2;
  return ((reinterpret_cast<uintptr_t>(A.wide) | (uintptr_t)(A.ld * size)) & 15) == 0;
}

static dim3 row_grid(const Mx4RowArgs& A) {
  const int64_t blocks = (A.rows * (A.cols / 8) + kMxThreads - 1) / kMxThreads;
  return dim3((unsigned)(blocks < 16384 ? blocks : 16384));
}

hipError_t launch_mx4_quantize(const Mx4RowArgs& A, hipStream_t s, const KTime& kt) {
  const bool w = wide_rows(A);
  auto* f = A.f32 ? (w ? k_mx4_quantize<true, true> : k_mx4_quantize<true, false>)
                  : (w ? k_mx4_quantize<false, true> : k_mx4_quantize<false, false>);
  MOE_LAUNCH(f, row_grid(A), dim3(kMxThreads), 0, s, kt.start, kt.stop, A);
  return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const Mx4RowArgs& A, hipStream_t s, const KTime& kt) {
  const bool w = wide_rows(A);
  auto* f = A.f32 ? (w ? k_mx4_dequantize<true, true> : k_mx4_dequantize<true, false>)
                  : (w ? k_mx4_dequantize<false, true> : k_mx4_dequantize<false, false>);
  MOE_LAUNCH(f, row_grid(A), dim3(kMxThreads), 0, s, kt.start, kt.stop, A);
  return hipGetLastError();
}

}  // namespace moe
