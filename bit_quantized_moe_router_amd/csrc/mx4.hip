// Quantisation to the microscaled 4-bit format and back (format: mx4.h).
//
// Both are bound by memory: 2.53 or 4.53 bytes a value (bf16 or fp32 on the
// wide side), a handful of instructions each.  131072 x 2048 values there and
// back take 224 us in bf16, 6.1 TB/s, and 602 us in fp32, 4.0 TB/s; a 2 GiB
// copy reaches 4.9.  A thread takes eight values, so a wave's wide side is 1 or
// 2 KB of consecutive bytes, its codes are one dword a lane, and the four lanes
// of a block find its largest magnitude with two lane moves.
#include "launch.h"
#include "mx4.h"

namespace moe {

constexpr int kMxThreads = 256;

// How a row's values are reached: one by one, by 16 bytes (which need that
// alignment), or, for more bf16 values than the caches hold, by 16 bytes past
// them: the codes and what is still to be read then keep their place there.
// us past the caches / through them, 2048 columns:
//   rows            quantised   read back   both in turn  read back, then a reader
//   16384   bf16     17 /  15    11 /  14     28 /  29       44 /  38
//   65536   bf16     56 /  59    50 /  63    107 / 138      134 / 144
//   131072  bf16    119 / 130   104 / 128    224 / 268      272 / 286
//   32768   fp32     58 /  46   101 /  76    162 / 134      154 / 140
//   131072  fp32    259 / 241   466 / 340    724 / 605      589 / 630
// fp32 goes through them: a lane's eight values are two 16-byte stores there, a
// wave's 32 bytes apart, which only the caches make whole lines of.
enum { kByOne = 0, kWide = 1, kPast = 2 };
constexpr int64_t kCacheBytes = (int64_t)256 << 20;  // the last-level cache

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

template <int Mode>
__device__ __forceinline__ uint4 load16(const void* p) {
  if constexpr (Mode == kPast) {
    const u32x4_t v = __builtin_nontemporal_load(static_cast<const u32x4_t*>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
  }
  return *static_cast<const uint4*>(p);
}
template <int Mode>
__device__ __forceinline__ void store16(void* p, uint4 v) {
  if constexpr (Mode == kPast) __builtin_nontemporal_store(u32x4_t{v.x, v.y, v.z, v.w}, static_cast<u32x4_t*>(p));
  else *static_cast<uint4*>(p) = v;
}

// Eight consecutive values.
template <bool F32, int Mode>
__device__ __forceinline__ void load8(const void* p, float v[8]) {
  if constexpr (F32) {
    const float* f = static_cast<const float*>(p);
    if constexpr (Mode != kByOne) {
      const float4 a = __builtin_bit_cast(float4, load16<Mode>(f)), b = __builtin_bit_cast(float4, load16<Mode>(f + 4));
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = f[i];
    }
  } else {
    const uint16_t* h = static_cast<const uint16_t*>(p);
    if constexpr (Mode != kByOne) {
      const uint4 a = load16<Mode>(h);
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

template <bool F32, int Mode>
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
    load8<F32, Mode>(static_cast<const char*>(A.wide) + (row * A.ld + col) * kSize, v);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) m = max(m, f32_abs_bits(v[j]));
    const int s = mx4_scale_byte(quad_max(m));
    reinterpret_cast<uint32_t*>(A.codes)[i] = mx4_pack8(v, mx4_inv_scale(s));
    if ((i & 3) == 0) A.scales[i >> 2] = (uint8_t)s;
  }
}

template <bool F32, int Mode>
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
      if constexpr (Mode != kByOne) {
        store16<Mode>(y, __builtin_bit_cast(uint4, make_float4(v[0], v[1], v[2], v[3])));
        store16<Mode>(y + 4, __builtin_bit_cast(uint4, make_float4(v[4], v[5], v[6], v[7])));
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++) y[j] = v[j];
      }
    } else {
      uint16_t* y = static_cast<uint16_t*>(A.wide) + row * A.ld + col;
      if constexpr (Mode != kByOne) {
        store16<Mode>(y, b);
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++) y[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
      }
    }
  }
}

// Rows whose first value and stride are multiples of 16 bytes go by 16 bytes;
// other addresses value by value.
static int row_mode(const Mx4RowArgs& A) {
  const int64_t size = A.f32 ? 4 : 2;
  if (((reinterpret_cast<uintptr_t>(A.wide) | (uintptr_t)(A.ld * size)) & 15) != 0) return kByOne;
  return !A.f32 && A.rows * A.cols * size >= kCacheBytes ? kPast : kWide;
}

static dim3 row_grid(const Mx4RowArgs& A) {
  const int64_t blocks = (A.rows * (A.cols / 8) + kMxThreads - 1) / kMxThreads;
  return dim3((unsigned)(blocks < 16384 ? blocks : 16384));
}

hipError_t launch_mx4_quantize(const Mx4RowArgs& A, hipStream_t s, const KTime& kt) {
  const int m = row_mode(A);
  auto* f = A.f32         ? (m == kWide ? k_mx4_quantize<true, kWide> : k_mx4_quantize<true, kByOne>)
            : m == kPast  ? k_mx4_quantize<false, kPast>
            : m == kWide  ? k_mx4_quantize<false, kWide>
                          : k_mx4_quantize<false, kByOne>;
  MOE_LAUNCH(f, row_grid(A), dim3(kMxThreads), 0, s, kt.start, kt.stop, A);
  return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const Mx4RowArgs& A, hipStream_t s, const KTime& kt) {
  const int m = row_mode(A);
  auto* f = A.f32         ? (m == kWide ? k_mx4_dequantize<true, kWide> : k_mx4_dequantize<true, kByOne>)
            : m == kPast  ? k_mx4_dequantize<false, kPast>
            : m == kWide  ? k_mx4_dequantize<false, kWide>
                          : k_mx4_dequantize<false, kByOne>;
  MOE_LAUNCH(f, row_grid(A), dim3(kMxThreads), 0, s, kt.start, kt.stop, A);
  return hipGetLastError();
}

}  // namespace moe
