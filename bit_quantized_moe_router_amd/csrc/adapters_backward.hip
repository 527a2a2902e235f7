// Low-rank adapters, backward (adapters.h): dh and dx by the kernel of the
// forward pass, then the gradients of both factors,
//   dA_a = sum_i dh_i x_i^T,   dB_a = s_a sum_i dy_i h_i^T.
#include "adapters.h"

namespace moe {

// ---------------------------------------------------------------------------
// A workgroup takes 128 columns of x (for dA) or of dy (for dB) and up to 64
// ranks of one adapter, and all of its rows: 32 rows an instruction, the waves
// taking them in turn and joining their sums through LDS in a fixed order.
// Lane (m, q) reads columns 8 m .. 8 m + 7 of rows 8 q .. 8 q + 7, which turned
// around are the operands of eight fragments (row m of fragment f: column 8 m +
// f), and the rank m of the same rows of dh or h, in three parts.
// ---------------------------------------------------------------------------
template <bool WideF32, int NB>
__device__ __forceinline__ void adapter_sum(const AdapterArgs& A, bool for_a, int e, int block, int rank0,
                                            float (&s_sum)[16 * NB][132]) {
  constexpr int kIn = WideF32 ? 3 : 1;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int m = lane & 15, q = lane >> 4;
  const int r = A.r, W = for_a ? A.K : A.N;
  const int lo = min(max(A.offsets[e], 0), A.P), hi = min(max(A.offsets[e + 1], lo), A.P);
  const void* wide = for_a ? (const void*)A.x : A.dy;
  const float* thin = for_a ? A.dh : A.h;
  const int c0 = block * 128 + 8 * m, left = W - c0;
  f32x4_t acc[8][NB] = {};
  for (int p0 = lo + 32 * wave; p0 < hi; p0 += 128) {
    int row[8];
    float t[8][NB];
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const int p = p0 + 8 * q + j;
      row[j] = -1;
      int raw;
      if (p < hi) row[j] = for_a ? adapter_src(A, p, &raw) : adapter_dst(A, p);
#pragma unroll
      for (int b = 0; b < NB; b++) {
        const int c = rank0 + 16 * b + m;
        t[j][b] = p < hi && c < r ? thin[(int64_t)p * r + c] : 0.f;
      }
    }
    RowPiece<WideF32, 8> x[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
      x[j].clear();
      if (row[j] >= 0 && left > 0)
        x[j].load(static_cast<const char*>(wide) + ((int64_t)row[j] * W + c0) * (WideF32 ? 4 : 2), left);
    }
    // A row outside x or dy counts as zeros, whatever dh or h hold for it.
    bf16x8_t tv[NB][3];
#pragma unroll
    for (int b = 0; b < NB; b++) {
      uint32_t d[3][4];
#pragma unroll
      for (int j = 0; j < 8; j++) {
        uint32_t part[3];
        split_parts<3>(row[j] >= 0 ? t[j][b] : 0.f, part);
#pragma unroll
        for (int s = 0; s < 3; s++) d[s][j / 2] = j & 1 ? d[s][j / 2] | part[s] << 16 : part[s];
      }
#pragma unroll
      for (int s = 0; s < 3; s++) tv[b][s] = as_bf16x8(d[s][0], d[s][1], d[s][2], d[s][3]);
    }
#pragma unroll
    for (int f = 0; f < 8; f++) {
      bf16x8_t xv[kIn];
      if constexpr (!WideF32) {
        uint32_t d[4];
#pragma unroll
        for (int p = 0; p < 4; p++) {
          const uint32_t a = x[2 * p].w[f / 2], b = x[2 * p + 1].w[f / 2];
          d[p] = f & 1 ? high_halves(a, b) : low_halves(a, b);
        }
        xv[0] = as_bf16x8(d[0], d[1], d[2], d[3]);
      } else {
        uint32_t d[3][4];
#pragma unroll
        for (int j = 0; j < 8; j++) {
          uint32_t part[3];
          split_parts<3>(x[j].get(f), part);
#pragma unroll
          for (int s = 0; s < 3; s++) d[s][j / 2] = j & 1 ? d[s][j / 2] | part[s] << 16 : part[s];
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
  }
  // Waves 3, 2, 1, 0, each adding to what those before it left.  Ranks 4 q + i of column 8 m + f.
  const int waves = min(4, (hi - lo + 31) / 32);
  for (int w = waves - 1; w > 0; w--) {
    if (wave == w) {
#pragma unroll
      for (int b = 0; b < NB; b++)
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
          for (int f = 0; f < 8; f++) {
            float& at = s_sum[16 * b + 4 * q + i][8 * m + f];
            at = w == waves - 1 ? acc[f][b][i] : at + acc[f][b][i];
          }
    }
    __syncthreads();
  }
  if (wave != 0) return;
  const float scale = !for_a && A.scales ? A.scales[e] : 1.f;
#pragma unroll
  for (int b = 0; b < NB; b++) {
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int f = 0; f < 8; f++)
        v[i][f] = scale * (waves > 1 ? acc[f][b][i] + s_sum[16 * b + 4 * q + i][8 * m + f] : acc[f][b][i]);
    const int c = rank0 + 16 * b + 4 * q;
    if (for_a) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        if (c + i >= r || left <= 0) continue;
        RowPiece<true, 8> o;
        o.set(v[i]);
        o.store(A.da + ((int64_t)e * r + c + i) * W + c0, left);
      }
    } else {
#pragma unroll
      for (int f = 0; f < 8; f++) {
        if (f >= left || c >= r) continue;
        const float u[4] = {v[0][f], v[1][f], v[2][f], v[3][f]};
        RowPiece<true, 4> o;
        o.set(u);
        o.store(A.db + ((int64_t)e * W + c0 + f) * r + c, r - c);
      }
    }
  }
}

template <bool YF32, int NB>
__global__ __launch_bounds__(kAdThreads) void k_adapters_sums(AdapterArgs A, int blocks_a, int blocks_b, int rank_blocks) {
  __shared__ float s_sum[16 * NB][132];
  const int per = (blocks_a + blocks_b) * rank_blocks;
  const int e = blockIdx.x / per;
  int u = blockIdx.x - e * per;
  const int rank0 = u % rank_blocks * 16 * NB;
  u /= rank_blocks;
  if (u < blocks_a) adapter_sum<false, NB>(A, true, e, u, rank0, s_sum);
  else adapter_sum<YF32, NB>(A, false, e, u - blocks_a, rank0, s_sum);
}

template <bool YF32, int NB>
static void launch_sums(const AdapterArgs& A, hipStream_t s, const KTime& kt, hipEvent_t ev0) {
  const int ba = (A.K + 127) / 128, bb = (A.N + 127) / 128, rb = (A.r + 16 * NB - 1) / (16 * NB);
  MOE_LAUNCH((k_adapters_sums<YF32, NB>), dim3((unsigned)(A.n * (ba + bb) * rb)), dim3(kAdThreads), 0, s, ev0, kt.stop, A,
             ba, bb, rb);
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
  auto* f = y_f32 ? (nr == 1 ? launch_sums<true, 1> : nr == 2 ? launch_sums<true, 2> : launch_sums<true, 4>)
                  : (nr == 1 ? launch_sums<false, 1> : nr == 2 ? launch_sums<false, 2> : launch_sums<false, 4>);
  f(A, s, kt, ev0);
  return hipGetLastError();
}

}  // namespace moe
