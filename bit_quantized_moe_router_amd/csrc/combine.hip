// The sum over each token's routed rows, and its gradients:
//   y_t = base_t + sum_j w_tj r_tj,   dr_tj = w_tj dy_t,   dw_tj = <dy_t, r_tj>
// over the j whose id is not negative.
//
// Bound by the bytes of the rows, in small calls by the way ids -> rows -> sum.
// Forward: threads split the columns, each sums its columns over j in order,
// with all of a token's rows in flight.  Backward: one pass over the rows
// gives both gradients; the lanes of a token hold its k dot products until the
// end.  Sums are fp32, each result is rounded once, and there are no atomics.
//
// Measured: 1 token of 8 rows of 2048 columns fp32 4.2 us; 4096 tokens of 8 rows
// of 2048 bf16 26.5 us, 6.4 TB/s with the last-level cache's share; 2085 tokens of
// 6 rows of 1999 columns bf16, 15 % of them left out, 16.9 us forward and 31.2
// backward (3.6 TB/s both), the rows' odd width leaving 7 of 8 unaligned.
#include <type_traits>

#include "launch.h"
#include "vec.h"

namespace moe {

constexpr int kCombThreads = 256, kCombBatch = 8;

// The columns of a thread: 16 bytes of a row.
template <bool RF32>
constexpr int kCombCols = RF32 ? 4 : 8;

// tpr threads a row (a power of two up to 256).  Whole: a wave has one row, so
// that ids and weights are read by the scalar unit and a left-out row is
// skipped by a branch of the whole wave.  Even: the width is a multiple of a
// thread's columns, and there is no shorter last piece.
template <bool RF32, bool YF32, bool Whole, bool Even>
__global__ __launch_bounds__(kCombThreads) void k_combine_rows(CombineArgs A, int tpr_log2) {
  constexpr int V = kCombCols<RF32>, kR = RF32 ? 4 : 2, kY = YF32 ? 4 : 2;
  const int tpr = 1 << tpr_log2, per = kCombThreads >> tpr_log2;
  const int part = threadIdx.x & (tpr - 1);
  const int64_t step = (int64_t)gridDim.x * per;
  const int64_t H = A.H;
  for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < A.T; t0 += step) {
    int sub = threadIdx.x >> tpr_log2;
    if constexpr (Whole) sub = __builtin_amdgcn_readfirstlane(sub);
    const int64_t t = t0 + sub;
    if (t >= A.T) break;
    for (int64_t c = (int64_t)part * V; c < H; c += (int64_t)tpr * V) {
      const int n = Even ? V : (int)min((int64_t)V, H - c);
      float acc[V] = {};
      if (A.base) {
        RowPiece<YF32, V> b;
        b.load(static_cast<const char*>(A.base) + (t * H + c) * kY, n);
#pragma unroll
        for (int i = 0; i < V; i++) acc[i] = b.get(i);
      }
      for (int j0 = 0; j0 < A.k; j0 += kCombBatch) {
        RowPiece<RF32, V> r[kCombBatch];
        float w[kCombBatch];
        bool on[kCombBatch];
#pragma unroll
        for (int u = 0; u < kCombBatch; u++) {
          const int64_t a = t * A.k + j0 + u;
          on[u] = j0 + u < A.k && (!A.ids || A.ids[a] >= 0);
          w[u] = on[u] && A.weights ? A.weights[a] : 1.f;
        }
#pragma unroll
        for (int u = 0; u < kCombBatch; u++) {
          r[u].clear();
          if (on[u]) r[u].load(static_cast<const char*>(A.rows) + ((t * A.k + j0 + u) * H + c) * kR, n);
        }
#pragma unroll
        for (int u = 0; u < kCombBatch; u++) {
          if (!on[u]) continue;
#pragma unroll
          for (int i = 0; i < V; i++) acc[i] = fmaf(w[u], r[u].get(i), acc[i]);
        }
      }
      RowPiece<YF32, V> y;
      y.set(acc);
      y.store(static_cast<char*>(A.y) + (t * H + c) * kY, n);
    }
  }
}

__device__ __forceinline__ float comb_wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// A token by `Waves` waves of a workgroup of four, or, where a row has fewer
// pieces than a wave has lanes, by 2^lanes_log2 lanes (Waves = 0); KB: k rounded up.
template <bool RF32, bool YF32, int KB, int Waves, bool Even>
__global__ __launch_bounds__(kCombThreads) void k_combine_grad(CombineArgs A, int lanes_log2) {
  constexpr int V = kCombCols<RF32>, kR = RF32 ? 4 : 2, kY = YF32 ? 4 : 2;
  __shared__ float s_dot[Waves > 1 ? Waves : 1][KB];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  // Lanes a token within a wave, this one's number among all of the token's, and tokens a workgroup.
  const int lanes = Waves == 0 ? 1 << lanes_log2 : 64, part = Waves == 0 ? lane & (lanes - 1) : Waves == 1 ? lane : threadIdx.x;
  const int tokens = Waves == 0 ? kCombThreads >> lanes_log2 : 4 / Waves;
  const int sub = Waves == 0 ? (int)(threadIdx.x >> lanes_log2) : Waves == 1 ? wave : 0;
  const int64_t H = A.H, step = (int64_t)gridDim.x * tokens;
  const int cols = (Waves > 1 ? kCombThreads : lanes) * V;
  // With Waves = 4 the loop's condition is the workgroup's, so that all of it meets at the barriers.
  for (int64_t t = (int64_t)blockIdx.x * tokens + sub; t < A.T; t += step) {
    float w[KB], dot[KB] = {};
    bool on[KB];
#pragma unroll
    for (int j = 0; j < KB; j++) {
      const int64_t a = t * A.k + j;
      on[j] = j < A.k && (!A.ids || A.ids[a] >= 0);
      w[j] = !on[j] ? 0.f : A.weights ? A.weights[a] : 1.f;
    }
    for (int64_t c = part * V; c < H; c += cols) {
      const int n = Even ? V : (int)min((int64_t)V, H - c);
      RowPiece<YF32, V> d;
      d.load(static_cast<const char*>(A.dy) + (t * H + c) * kY, n);
      RowPiece<RF32, V> r[KB];
      if (A.dweights) {
#pragma unroll
        for (int j = 0; j < KB; j++) {
          r[j].clear();
          if (on[j]) r[j].load(static_cast<const char*>(A.rows) + ((t * A.k + j) * H + c) * kR, n);
        }
#pragma unroll
        for (int j = 0; j < KB; j++) {
          if (!on[j]) continue;
#pragma unroll
          for (int i = 0; i < V; i++) dot[j] = fmaf(d.get(i), r[j].get(i), dot[j]);
        }
      }
      if (A.drows) {
#pragma unroll
        for (int j = 0; j < KB; j++) {
          if (j >= A.k) continue;
          float v[V];
#pragma unroll
          for (int i = 0; i < V; i++) v[i] = on[j] ? w[j] * d.get(i) : 0.f;
          r[j].set(v);
          r[j].store(static_cast<char*>(A.drows) + ((t * A.k + j) * H + c) * kR, n);
        }
      }
    }
    if (!A.dweights) continue;
    if constexpr (Waves == 0) {
      for (int d = 1; d < lanes; d <<= 1) {
#pragma unroll
        for (int j = 0; j < KB; j++) dot[j] += __shfl_xor(dot[j], d);
      }
#pragma unroll
      for (int j = 0; j < KB; j++)
        if (j < A.k && part == (j & (lanes - 1))) A.dweights[t * A.k + j] = dot[j];
      continue;
    }
#pragma unroll
    for (int j = 0; j < KB; j++) dot[j] = comb_wave_sum(dot[j]);
    if constexpr (Waves == 1) {
      float mine = 0.f;
#pragma unroll
      for (int j = 0; j < KB; j++) mine = lane == j ? dot[j] : mine;
      if (lane < A.k) A.dweights[t * A.k + lane] = mine;
    } else {
      if (lane == 0) {
#pragma unroll
        for (int j = 0; j < KB; j++) s_dot[wave][j] = dot[j];
      }
      __syncthreads();
      if (threadIdx.x < A.k) {
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < Waves; v++) sum += s_dot[v][threadIdx.x];
        A.dweights[t * A.k + threadIdx.x] = sum;
      }
      __syncthreads();
    }
  }
}

// At most this many workgroups; each goes through several tokens beyond them.
constexpr int64_t kCombGrid = 1 << 20;

hipError_t launch_combine_forward(const CombineArgs& A, hipStream_t s, const KTime& kt) {
  const int V = A.rows_f32 ? 4 : 8;
  const int64_t pieces = (A.H + V - 1) / V;
  int log2 = 0;
  while (log2 < 8 && (1 << log2) < pieces) log2++;
  const int64_t per = kCombThreads >> log2, groups = (A.T + per - 1) / per;
  const dim3 grid((unsigned)(groups < kCombGrid ? groups : kCombGrid));
  auto go = [&](auto rf, auto yf) {
    constexpr bool RF = rf.value, YF = yf.value;
    auto* f = A.H % V ? (log2 >= 6 ? k_combine_rows<RF, YF, true, false> : k_combine_rows<RF, YF, false, false>)
                      : (log2 >= 6 ? k_combine_rows<RF, YF, true, true> : k_combine_rows<RF, YF, false, true>);
    MOE_LAUNCH(f, grid, dim3(kCombThreads), 0, s, kt.start, kt.stop, A, log2);
  };
  using std::false_type;
  using std::true_type;
  if (A.rows_f32) A.y_f32 ? go(true_type{}, true_type{}) : go(true_type{}, false_type{});
  else A.y_f32 ? go(false_type{}, true_type{}) : go(false_type{}, false_type{});
  return hipGetLastError();
}

template <bool RF, bool YF>
static void launch_grad(const CombineArgs& A, hipStream_t s, const KTime& kt) {
  // Four waves a token where a row has pieces for more than one (8 bf16 rows of 2048, a wave or four a token: 1 token 15.6,
  // 7.2 us; 512 tokens 20.5, 11.3; 2048 tokens 30.3, 28.0); part of a wave where it has few (15920 tokens of 6 rows of 61,
  // a wave a token or 8 lanes: 42.7, 14.3).
  const int64_t pieces = (A.H + kCombCols<RF> - 1) / kCombCols<RF>;
  int log2 = 0;
  while (log2 < 6 && (1 << log2) < pieces) log2++;
  const int waves = log2 < 6 ? 0 : pieces > 64 ? 4 : 1;
  const int64_t tokens = waves == 0 ? kCombThreads >> log2 : waves == 1 ? 4 : 1, groups = (A.T + tokens - 1) / tokens;
  const dim3 grid((unsigned)(groups < kCombGrid ? groups : kCombGrid));
  auto go = [&](auto kb) {
    constexpr int KB = kb.value;
    auto* f = A.H % kCombCols<RF> ? (waves == 0   ? k_combine_grad<RF, YF, KB, 0, false>
                                     : waves == 1 ? k_combine_grad<RF, YF, KB, 1, false>
                                                  : k_combine_grad<RF, YF, KB, 4, false>)
                                  : (waves == 0   ? k_combine_grad<RF, YF, KB, 0, true>
                                     : waves == 1 ? k_combine_grad<RF, YF, KB, 1, true>
                                                  : k_combine_grad<RF, YF, KB, 4, true>);
    MOE_LAUNCH(f, grid, dim3(kCombThreads), 0, s, kt.start, kt.stop, A, log2);
  };
  if (A.k <= 4) go(std::integral_constant<int, 4>{});
  else if (A.k <= 8) go(std::integral_constant<int, 8>{});
  else go(std::integral_constant<int, 16>{});
}

hipError_t launch_combine_backward(const CombineArgs& A, hipStream_t s, const KTime& kt) {
  auto* f = A.rows_f32 ? (A.y_f32 ? launch_grad<true, true> : launch_grad<true, false>)
                       : (A.y_f32 ? launch_grad<false, true> : launch_grad<false, false>);
  f(A, s, kt);
  return hipGetLastError();
}

}  // namespace moe
