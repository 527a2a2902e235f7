// Low-rank adapters, backward (adapters.h): dh and dx by the kernel of the
// forward pass, then the gradients of both factors,
//   dA_a = sum_i dh_i x_i^T,   dB_a = s_a sum_i dy_i h_i^T.
#include "adapters.h"

namespace moe {

// ---------------------------------------------------------------------------
// A workgroup takes 16 F columns of x (for dA) or of dy (for dB) and up to 64 ranks
// of one adapter, and its rows 32 at a time.  Lane (m, q) reads columns F m ..
// F m + F - 1 of rows 8 q .. 8 q + 7, which turned around are the operands of F
// fragments (row m of fragment f: column F m + f), and the same rows of rank m
// of dh or h from where k_adapters_rows has left them in three parts.  Even: the
// widths are multiples of 8, the rank of 4.
// The W waves of a workgroup take the rows in turn and join their sums through
// LDS in a fixed order.
//
// Bound by the chain offsets -> rows' names -> rows of each wave's few turns and the
// join: 256 adapters of rank 16 over 32768 rows, 2048 -> 1024 in bf16, 62 us at 3.6 TB/s;
// 3 of rank 64 over 2085 rows, 2048 -> 1000 in fp32, 19.9 us.  A wave with columns of its
// own that no other wave shares needs no join, but an adapter with many rows then takes
// as long as they do (skewed routing 118 us against 57).
// ---------------------------------------------------------------------------
template <bool WideF32, int NB, int F, int W, bool Even>
__device__ __forceinline__ void adapter_sum(const AdapterArgs& A, bool for_a, int e, int block, int rank0, int rpad,
                                            float (*s_sum)[16 * F + 4]) {
  constexpr int kIn = WideF32 ? 3 : 1;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int m = lane & 15, q = lane >> 4;
  const int r = A.r, wide_n = for_a ? A.K : A.N;
  const int lo = min(max(A.offsets[e], 0), A.P), hi = min(max(A.offsets[e + 1], lo), A.P);
  const char* wide = static_cast<const char*>(for_a ? (const void*)A.x : A.dy);
  const uint16_t* thin = A.thin + (for_a ? 0 : A.thin_h);
  const int32_t* names = for_a ? A.src_rows : A.dst_rows;
  const int c0 = block * 16 * F + F * m, left = wide_n - c0;
  f32x4_t acc[F][NB] = {};
  const int last = hi > lo ? (hi + 31) >> 5 : 0;
  // The eight rows' names, a step ahead of the rows.
  auto name = [&](int c, int (&to)[8]) {
    const int p = 32 * c + 8 * q;
    if (!names) {
#pragma unroll
      for (int j = 0; j < 8; j++) to[j] = p + j;
    } else if (p + 8 <= A.P) {
      const int4 u = load_any<int4>(names + p), v = load_any<int4>(names + p + 4);
      to[0] = u.x, to[1] = u.y, to[2] = u.z, to[3] = u.w, to[4] = v.x, to[5] = v.y, to[6] = v.z, to[7] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) to[j] = p + j < A.P ? names[p + j] : -1;
    }
  };
  int c = (lo >> 5) + wave;
  int row[8];
  if (c < last) name(c, row);
  for (; c < last; c += W) {
    int ahead[8];
    if (c + W < last) name(c + W, ahead);
    uint4 t[NB][3];
#pragma unroll
    for (int b = 0; b < NB; b++)
#pragma unroll
      for (int s = 0; s < 3; s++)
        t[b][s] = *reinterpret_cast<const uint4*>(thin + ((int64_t)c * rpad + rank0 + 16 * b + m) * kThinRank + 32 * s + 8 * q);
    RowPiece<WideF32, F> x[8];
    bool in[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const int p = 32 * c + 8 * q + j;
      int at = row[j];
      if (for_a && A.src_div > 1 && at >= 0) at = div_by(at, A.src);
      in[j] = p >= lo && p < hi && (unsigned)at < (unsigned)(for_a ? A.x_rows : A.y_rows);
      x[j].clear();
      if (in[j] && left > 0) x[j].load(wide + ((int64_t)at * wide_n + c0) * (WideF32 ? 4 : 2), Even ? F : left);
    }
    // Rows of other adapters, and rows outside x or dy, count as zeros whatever dh or h hold for them.
    uint32_t mask[4];
#pragma unroll
    for (int d = 0; d < 4; d++) mask[d] = (in[2 * d] ? 0xFFFFu : 0u) | (in[2 * d + 1] ? 0xFFFF0000u : 0u);
    bf16x8_t tv[NB][3];
#pragma unroll
    for (int b = 0; b < NB; b++)
#pragma unroll
      for (int s = 0; s < 3; s++)
        tv[b][s] = as_bf16x8(t[b][s].x & mask[0], t[b][s].y & mask[1], t[b][s].z & mask[2], t[b][s].w & mask[3]);
#pragma unroll
    for (int f = 0; f < F; f++) {
      bf16x8_t xv[kIn];
      if constexpr (!WideF32) {
        uint32_t d[4];
#pragma unroll
        for (int p = 0; p < 4; p++) {
          const uint32_t u = x[2 * p].w[f / 2], v = x[2 * p + 1].w[f / 2];
          d[p] = f & 1 ? high_halves(u, v) : low_halves(u, v);
        }
        xv[0] = as_bf16x8(d[0], d[1], d[2], d[3]);
      } else {
        uint32_t d[3][4];
#pragma unroll
        for (int p = 0; p < 4; p++) {
          // Cut off, so that each part is the upper half of what is left; the part of an infinity or NaN is its first.
          float u = x[2 * p].get(f), v = x[2 * p + 1].get(f);
#pragma unroll
          for (int s = 0; s < 3; s++) {
            d[s][p] = high_halves(__float_as_uint(u), __float_as_uint(v));
            const float ur = u - __uint_as_float(__float_as_uint(u) & 0xFFFF0000u);
            const float vr = v - __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
            u = ur == ur ? ur : 0.f;
            v = vr == vr ? vr : 0.f;
          }
        }
#pragma unroll
        for (int s = 0; s < 3; s++) xv[s] = as_bf16x8(d[s][0], d[s][1], d[s][2], d[s][3]);
      }
      // Products of parts below 2^-24 of the leading one are left out; small ones first.
#pragma unroll
      for (int b = 0; b < NB; b++)
#pragma unroll
        for (int sum = 2; sum >= 0; sum--)
#pragma unroll
          for (int s = 0; s <= sum; s++)
            if (sum - s < kIn) acc[f][b] = mfma_bf16(tv[b][s], xv[sum - s], acc[f][b]);
    }
#pragma unroll
    for (int j = 0; j < 8; j++) row[j] = ahead[j];
  }
  // The last wave to the first, each adding to what those before it left.  Ranks 4 q + i of column F m + f.
  const int waves = max(1, min(W, last - (lo >> 5)));
  for (int w = waves - 1; w > 0; w--) {
    if (wave == w) {
#pragma unroll
      for (int b = 0; b < NB; b++)
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
          for (int f = 0; f < F; f++) {
            float& at = s_sum[16 * b + 4 * q + i][F * m + f];
            at = w == waves - 1 ? acc[f][b][i] : at + acc[f][b][i];
          }
    }
    __syncthreads();
  }
  if (wave != 0) return;
  if (left <= 0) return;
  const float scale = !for_a && A.scales ? A.scales[e] : 1.f;
#pragma unroll
  for (int b = 0; b < NB; b++) {
    float v[4][F];
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int f = 0; f < F; f++)
        v[i][f] = scale * (waves > 1 ? acc[f][b][i] + s_sum[16 * b + 4 * q + i][F * m + f] : acc[f][b][i]);
    const int cr = rank0 + 16 * b + 4 * q;
    if (for_a) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        if (cr + i >= r) continue;
        RowPiece<true, F> o;
        o.set(v[i]);
        o.store(A.da + ((int64_t)e * r + cr + i) * wide_n + c0, Even ? F : left);
      }
    } else {
#pragma unroll
      for (int f = 0; f < F; f++) {
        if (f >= left || cr >= r) continue;
        const float u[4] = {v[0][f], v[1][f], v[2][f], v[3][f]};
        RowPiece<true, 4> o;
        o.set(u);
        o.store(A.db + ((int64_t)e * wide_n + c0 + f) * r + cr, Even ? 4 : r - cr);
      }
    }
  }
}

template <bool YF32, int NB, int F, int W, bool Even>
__global__ __launch_bounds__(64 * W) void k_adapters_sums(AdapterArgs A, int blocks_a, int blocks_b, int rank_blocks) {
  __shared__ float s_sum[16 * NB][16 * F + 4];
  const int per = (blocks_a + blocks_b) * rank_blocks;
  const int e = blockIdx.x / per;
  int u = blockIdx.x - e * per;
  const int rank0 = u % rank_blocks * 16 * NB, rpad = 16 * NB * rank_blocks;
  u /= rank_blocks;
  if (u < blocks_a) adapter_sum<false, NB, F, W, Even>(A, true, e, u, rank0, rpad, s_sum);
  else adapter_sum<YF32, NB, F, W, Even>(A, false, e, u - blocks_a, rank0, rpad, s_sum);
}

template <bool YF32, int NB, int F, int W, bool Even>
static void launch_sums(const AdapterArgs& A, hipStream_t s, const KTime& kt, hipEvent_t ev0) {
  constexpr int kCols = 16 * F;
  const int ba = (A.K + kCols - 1) / kCols, bb = (A.N + kCols - 1) / kCols, rb = (A.r + 16 * NB - 1) / (16 * NB);
  MOE_LAUNCH((k_adapters_sums<YF32, NB, F, W, Even>), dim3((unsigned)(A.n * (ba + bb) * rb)), dim3(64 * W), 0, s, ev0,
             kt.stop, A, ba, bb, rb);
}

template <bool YF32, int NB>
static void sums(const AdapterArgs& A, int cus, hipStream_t s, const KTime& kt, hipEvent_t ev0) {
  // 64 columns by 4 waves where those are workgroups enough, by 8 where the rows' turns would take longer than the rest, and
  // 32 columns by more waves still where many compute units would have none.  Both kernels of the backward pass, 4096 rows,
  // us with 32 by 16 (8 for rank 64) / 64 by 8 / 64 by 4 / 128 by 4:
  //   rank 16:  1 adapter of 512 -> 512  29 / 38 / 52 / 55     3 of 2048 -> 2048  37 / 36 / 45 / 48
  //             8 of 2048 -> 2048  39 / 34 / 40 / 42           64 of 2048 -> 2048  63 / 39 / 34 / 33
  //   rank 64:  1 of 512 -> 512  53 / 58 / 76 / 99             8 of 4096 -> 4096  87 / 84 / 80 / 111
  const int64_t blocks = (int64_t)A.n * ((A.K + 63) / 64 + (A.N + 63) / 64) * ((A.r + 16 * NB - 1) / (16 * NB));
  const bool even = A.K % 8 == 0 && A.N % 8 == 0 && A.r % 4 == 0;
  constexpr int kMost = NB == 4 ? 8 : 16;
  auto* f = blocks >= 8 * cus ? (even ? launch_sums<YF32, NB, 4, 4, true> : launch_sums<YF32, NB, 4, 4, false>)
            : blocks >= cus   ? (even ? launch_sums<YF32, NB, 4, 8, true> : launch_sums<YF32, NB, 4, 8, false>)
                              : (even ? launch_sums<YF32, NB, 2, kMost, true> : launch_sums<YF32, NB, 2, kMost, false>);
  f(A, s, kt, ev0);
}

hipError_t launch_adapters_backward(const AdapterArgs& A, bool y_f32, int cus, hipStream_t s, const KTime& kt) {
  hipEvent_t stop = A.da ? nullptr : kt.stop;
  hipError_t e = hipSuccess;
  if (A.P > 0)
    e = y_f32 ? adapters_rows_any<true, true>(A, cus, s, kt.start, stop)
              : adapters_rows_any<true, false>(A, cus, s, kt.start, stop);
  if (e != hipSuccess || !A.da) return e;
  hipEvent_t ev0 = A.P > 0 ? nullptr : kt.start;
  const int nr = adapter_frags(A.r);
  auto* f = y_f32 ? (nr == 1 ? sums<true, 1> : nr == 2 ? sums<true, 2> : sums<true, 4>)
                  : (nr == 1 ? sums<false, 1> : nr == 2 ? sums<false, 2> : sums<false, 4>);
  f(A, cus, s, kt, ev0);
  return hipGetLastError();
}

// Bytes of the two thin operands of `rows` positions.
size_t adapters_thin_bytes(int r, int64_t rows) {
  return (size_t)((rows + 31) / 32) * (16 * adapter_frags(r)) * kThinRank * 2 * sizeof(uint16_t);
}

}  // namespace moe
