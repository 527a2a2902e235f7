// The router's balance loss with its per-expert counts, and its gradient.
//
// With p_t the softmax of token t's logits, n the valid tokens, c_e the valid
// assignments of expert e, P_e = sum_t p_te / n and f_e = c_e / (n k):
//   balance = E sum_e f_e P_e,   z = sum_t lse_t^2 / n,   loss = a balance + b z,
//   dloss/dl_te = p_te (a E / n (f_e - sum_j f_j p_tj) + 2 b lse_t / n)
// (f is made of counts and has no gradient).
//
// Forward: a group of lanes takes a row and adds its probabilities to per-lane
// sums and its ids to integer counters in LDS; each workgroup leaves one
// partial row.  A second launch sums the partial rows by expert in a fixed
// order in float64; its last workgroup to finish joins the balance sum, also
// in a fixed order, so repeated calls give identical bits.  Small inputs take
// one workgroup and one launch.  Backward: one pass that takes the softmax
// again from the logits.
//
// Both are bound by reading (and writing) the logits, next to them by the
// exchanges between lanes that a softmax needs.  So a row gets few lanes (16
// for more than 64 experts) with up to 32 values each: four rows share a
// wave's exchanges, loads are 16 bytes a lane, and the next rows are loaded
// before the present ones are worked on.
#include <type_traits>

#include "launch.h"
#include "mx4.h"

namespace moe {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Lane moves inside a row of 16 lanes: neighbours in a quad, mirrored halves, mirrored row.
template <int Ctrl>
__device__ __forceinline__ float lane_move(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), Ctrl, 0xF, 0xF, true));
}
// Sum / maximum over groups of G = 4, 8 or 16 consecutive lanes, in every lane of the group.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  v += lane_move<0xB1>(v);
  v += lane_move<0x4E>(v);
  if (G >= 8) v += lane_move<0x141>(v);
  if (G >= 16) v += lane_move<0x140>(v);
  return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
  v = fmaxf(v, lane_move<0xB1>(v));
  v = fmaxf(v, lane_move<0x4E>(v));
  if (G >= 8) v = fmaxf(v, lane_move<0x141>(v));
  if (G >= 16) v = fmaxf(v, lane_move<0x140>(v));
  return v;
}

// A row's values in a group of G lanes: value j of lane g is expert
// expert_of(g, j), in runs of 16 bytes (W values) a lane.
template <bool F32, int G, int N>
struct BalRow {
  static constexpr int kRun = F32 ? 4 : 8;
  static constexpr int kVecs = N / kRun;
  uint4 raw[kVecs];

  static __device__ __forceinline__ int expert_of(int g, int j) { return (g + G * (j / kRun)) * kRun + j % kRun; }

  // Wide: E is a multiple of the run and the rows are 16-byte aligned.
  template <bool Wide>
  __device__ __forceinline__ void load(const void* logits, int64_t t, int E, int g) {
    constexpr uint32_t kOut = F32 ? 0xFF800000u : 0xFF80FF80u;  // -inf past the last expert
#pragma unroll
    for (int v = 0; v < kVecs; v++) {
      const int e = (g + G * v) * kRun;
      raw[v] = make_uint4(kOut, kOut, kOut, kOut);
      if constexpr (Wide) {
        if (e < E) raw[v] = *reinterpret_cast<const uint4*>(static_cast<const char*>(logits) + (t * E + e) * (F32 ? 4 : 2));
      } else {
        uint32_t d[4] = {kOut, kOut, kOut, kOut};
#pragma unroll
        for (int i = 0; i < kRun; i++) {
          if (e + i >= E) continue;
          if constexpr (F32) d[i] = static_cast<const uint32_t*>(logits)[t * E + e + i];
          else {
            const uint32_t b = static_cast<const uint16_t*>(logits)[t * E + e + i];
            d[i / 2] = i & 1 ? (d[i / 2] & 0xFFFFu) | b << 16 : (d[i / 2] & 0xFFFF0000u) | b;
          }
        }
        raw[v] = make_uint4(d[0], d[1], d[2], d[3]);
      }
    }
  }

  // The row's softmax in p and its log-sum-exp.  A row of -inf alone has p = 0
  // and lse = 0; NaNs stay.
  __device__ __forceinline__ void softmax(float p[N], float* lse) const {
#pragma unroll
    for (int v = 0; v < kVecs; v++) {
      const uint32_t d[4] = {raw[v].x, raw[v].y, raw[v].z, raw[v].w};
#pragma unroll
      for (int i = 0; i < kRun; i++)
        p[v * kRun + i] = F32 ? __uint_as_float(d[F32 ? i : 0])
                              : __uint_as_float(i & 1 ? d[i / 2] & 0xFFFF0000u : d[i / 2] << 16);
    }
    float top = p[0];
#pragma unroll
    for (int j = 1; j < N; j++) top = fmaxf(top, p[j]);
    top = group_max<G>(top);
    // Of nothing but -inf, or of NaNs alone: any finite number will do.
    if (!(top > -INFINITY)) top = 0.f;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < N; j++) {
      p[j] = __builtin_amdgcn_exp2f((p[j] - top) * kLog2e);
      sum += p[j];
    }
    sum = group_sum<G>(sum);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int j = 0; j < N; j++) p[j] *= inv;
    *lse = sum == 0.f ? 0.f : top + __builtin_amdgcn_logf(sum) * kLn2;
  }
};

// The loss from the summed parts (one thread).
__device__ __forceinline__ void balance_finish(const BalanceArgs& A, double dot, double z, int n) {
  const double bal = n > 0 ? A.E * dot : 0.0, zz = n > 0 ? z / n : 0.0;
  A.losses[0] = (float)((double)A.balance_coef * bal + (double)A.z_coef * zz);
  A.losses[1] = (float)bal;
  A.losses[2] = (float)zz;
  A.n_valid[0] = n;
}

// One launch of `gridDim.x` workgroups over all rows.  With one workgroup it
// finishes the loss; otherwise it leaves a partial row in the workspace.
template <bool F32, int G, int N, bool Wide, int NT>
__global__ __launch_bounds__(NT) void k_balance_rows(BalanceArgs A) {
  constexpr int kBalThreads = NT, kBalWaves = NT / 64;
  constexpr int kRows = kBalThreads / G;  // rows in flight a workgroup
  __shared__ int s_count[512];
  __shared__ float s_p[kBalWaves][G * N];  // a wave's sums
  __shared__ double s_z[kBalWaves];
  __shared__ int s_n[kBalWaves];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, g = lane & (G - 1);
  const int E = A.E;
  if (blockIdx.x == 0 && tid == 0) *A.done = 0;  // the second launch's counter
  for (int e = tid; e < E; e += kBalThreads) s_count[e] = 0;
  __syncthreads();
  float acc[N] = {};
  double z = 0.0;
  int n = 0;
  using Row = BalRow<F32, G, N>;
  Row cur, next;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t t = (int64_t)blockIdx.x * kRows + tid / G;
  // Padding rows are loaded like the others, so that no load waits for `valid`.
  uint8_t on = 1, next_on = 1;
  if (t < A.T) {
    if (A.valid) on = A.valid[t];
    cur.template load<Wide>(A.logits, t, E, g);
  }
  // A group's lanes are in one wave and go through the same rows.
  for (; t < A.T; t += step) {
    if (t + step < A.T) {
      if (A.valid) next_on = A.valid[t + step];
      next.template load<Wide>(A.logits, t + step, E, g);
    }
    if (on) {
      float p[N], lse;
      cur.softmax(p, &lse);
#pragma unroll
      for (int j = 0; j < N; j++) acc[j] += p[j];
      if (g == 0) {
        z += (double)lse * lse;
        n += 1;
      }
      for (int j = g; j < A.k; j += G) {
        const int e = A.ids[t * A.k + j];
        if ((unsigned)e < (unsigned)E) atomicAdd(&s_count[e], 1);
      }
    }
    cur = next;
    on = next_on;
  }
  // Groups of a wave, then waves, in a fixed order.
#pragma unroll
  for (int d = G; d < 64; d <<= 1) {
#pragma unroll
    for (int j = 0; j < N; j++) acc[j] += __shfl_xor(acc[j], d);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    z += __shfl_xor(z, d);
    n += __shfl_xor(n, d);
  }
  if (lane < G) {
#pragma unroll
    for (int j = 0; j < N; j++) s_p[wave][Row::expert_of(g, j)] = acc[j];
  }
  if (lane == 0) s_z[wave] = z, s_n[wave] = n;
  __syncthreads();
  z = 0.0, n = 0;
#pragma unroll
  for (int w = 0; w < kBalWaves; w++) z += s_z[w], n += s_n[w];
  const int e = tid;  // E is at most the number of threads
  double sum = 0.0;
  if (e < E) {
#pragma unroll
    for (int w = 0; w < kBalWaves; w++) sum += (double)s_p[w][e];
  }
  if (gridDim.x > 1) {
    if (e < E) {
      A.part_p[(int64_t)blockIdx.x * E + e] = (float)sum;
      A.part_count[(int64_t)blockIdx.x * E + e] = s_count[e];
    }
    if (tid == 0) {
      A.part_z[blockIdx.x] = z;
      A.part_n[blockIdx.x] = n;
    }
    return;
  }
  double dot = 0.0;
  if (e < E) {
    const double pe = n > 0 ? sum / n : 0.0;
    A.mean_prob[e] = (float)pe;
    A.counts[e] = s_count[e];
    if (n > 0) dot = pe * s_count[e] / ((double)n * A.k);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) dot += __shfl_xor(dot, d);
  __syncthreads();
  if (lane == 0) s_z[wave] = dot;
  __syncthreads();
  if (tid != 0) return;
  dot = 0.0;
  for (int w = 0; w < kBalWaves; w++) dot += s_z[w];
  balance_finish(A, dot, z, n);
}

// Second launch: workgroup b sums the partial rows of 16 experts, 64 threads
// an expert; the last workgroup to arrive adds the workgroups' parts of the
// balance sum in order.
constexpr int kBalSumExperts = 16, kBalSumThreads = 1024;

__global__ __launch_bounds__(kBalSumThreads) void k_balance_sum(BalanceArgs A, int parts) {
  constexpr int kSlices = kBalSumThreads / kBalSumExperts;  // 64
  static_assert(kBalMaxParts % kSlices == 0, "every slice may hold the same number of parts");
  constexpr int kTurns = kBalMaxParts / kSlices;
  __shared__ double s_p[kSlices][kBalSumExperts + 1];
  __shared__ int s_c[kSlices][kBalSumExperts + 1];
  const int tid = threadIdx.x, x = tid & 15, slice = tid >> 4;
  const int e = blockIdx.x * kBalSumExperts + x;
  float pv[kTurns];
  int cv[kTurns];
#pragma unroll
  for (int i = 0; i < kTurns; i++) {
    const int g = slice + kSlices * i;
    const bool in = g < parts && e < A.E;
    pv[i] = in ? A.part_p[(int64_t)g * A.E + e] : 0.f;
    cv[i] = in ? A.part_count[(int64_t)g * A.E + e] : 0;
  }
  double p = 0.0;
  int c = 0;
#pragma unroll
  for (int i = 0; i < kTurns; i++) p += (double)pv[i], c += cv[i];
  s_p[slice][x] = p;
  s_c[slice][x] = c;
  // z and n by the first wave, kBalMaxParts / 64 parts a lane.
  double z = 0.0;
  int n = 0;
  if (tid < 64) {
#pragma unroll
    for (int i = 0; i < kBalMaxParts / 64; i++) {
      const int g = tid + 64 * i;
      if (g < parts) z += A.part_z[g], n += A.part_n[g];
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      z += __shfl_xor(z, d);
      n += __shfl_xor(n, d);
    }
  }
  __syncthreads();
  if (tid >= 64) return;
  // Lane (x, y): slices 16 y .. 16 y + 15 of expert x.
  p = 0.0, c = 0;
#pragma unroll
  for (int i = 0; i < 16; i++) {
    p += s_p[(tid >> 4) * 16 + i][x];
    c += s_c[(tid >> 4) * 16 + i][x];
  }
#pragma unroll
  for (int d = 16; d < 64; d <<= 1) {
    p += __shfl_xor(p, d);
    c += __shfl_xor(c, d);
  }
  double dot = 0.0;
  if (tid < 16 && e < A.E) {
    const double pe = n > 0 ? p / n : 0.0;
    A.mean_prob[e] = (float)pe;
    A.counts[e] = c;
    if (n > 0) dot = pe * c / ((double)n * A.k);
  }
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) dot += __shfl_xor(dot, d);
  int arrived = 0;
  if (tid == 0) {
    __hip_atomic_store(&A.dots[blockIdx.x], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    arrived = __hip_atomic_fetch_add(A.done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (__builtin_amdgcn_readfirstlane(arrived) != (int)gridDim.x - 1) return;
  // At most 32 workgroups, a lane each; the same exchanges give the same sum whoever is last.
  dot = tid < (int)gridDim.x ? __hip_atomic_load(&A.dots[tid], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) dot += __shfl_xor(dot, d);
  if (tid == 0) balance_finish(A, dot, z, n);
}

// At most 1024 workgroups of 256 threads, each going through several rows a
// group at large T: 25 us for 65536 x 512 bf16 logits (134 MB in and out, 5.3
// TB/s) against 28 with 512 workgroups and 29 with 2048.
constexpr int kGradThreads = 256;

template <bool F32, int G, int N, bool Wide>
__global__ __launch_bounds__(kGradThreads) void k_balance_grad(BalanceArgs A) {
  constexpr int kRows = kGradThreads / G;
  using Row = BalRow<F32, G, N>;
  const int lane = threadIdx.x & 63, g = lane & (G - 1);
  const int E = A.E, n = A.n_valid[0];
  const float up = A.grad ? A.grad[0] : 1.f;
  // grad a E / n f_e = c_e grad a E / (n^2 k), and the z term's grad 2 b / n.
  const float scale = n > 0 ? up / (float)n : 0.f;
  const float za = 2.f * A.z_coef * scale;
  const float fa = n > 0 ? A.balance_coef * E * scale / ((float)n * A.k) : 0.f;
  float f[N];
#pragma unroll
  for (int j = 0; j < N; j += 4) {
    const int e = Row::expert_of(g, j);
    int4 c = make_int4(0, 0, 0, 0);
    if constexpr (Wide) {
      if (e < E) c = *reinterpret_cast<const int4*>(A.counts + e);
    } else {
      if (e < E) c.x = A.counts[e];
      if (e + 1 < E) c.y = A.counts[e + 1];
      if (e + 2 < E) c.z = A.counts[e + 2];
      if (e + 3 < E) c.w = A.counts[e + 3];
    }
    f[j] = fa * (float)c.x, f[j + 1] = fa * (float)c.y, f[j + 2] = fa * (float)c.z, f[j + 3] = fa * (float)c.w;
  }
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t t = (int64_t)blockIdx.x * kRows + threadIdx.x / G;
  Row cur, next;
  uint8_t on = 1, next_on = 1;
  if (t < A.T) {
    if (A.valid) on = A.valid[t];
    cur.template load<Wide>(A.logits, t, E, g);
  }
  for (; t < A.T; t += step, cur = next, on = next_on) {
    if (t + step < A.T) {
      if (A.valid) next_on = A.valid[t + step];
      next.template load<Wide>(A.logits, t + step, E, g);
    }
    float p[N], lse = 0.f, dot = 0.f;
    if (on && n > 0) {
      cur.softmax(p, &lse);
#pragma unroll
      for (int j = 0; j < N; j++) dot += p[j] * f[j];
      dot = group_sum<G>(dot);
#pragma unroll
      for (int j = 0; j < N; j++) p[j] *= f[j] - dot + za * lse;
    } else {
#pragma unroll
      for (int j = 0; j < N; j++) p[j] = 0.f;
    }
#pragma unroll
    for (int v = 0; v < Row::kVecs; v++) {
      const int e = (g + G * v) * Row::kRun;
      const float* d = p + v * Row::kRun;
      if constexpr (Wide) {
        if (e >= E) continue;
        uint4 o;
        if constexpr (F32) {
          o = make_uint4(__float_as_uint(d[0]), __float_as_uint(d[1]), __float_as_uint(d[2]), __float_as_uint(d[3]));
        } else {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; i++) w[i] = f32_to_bf16_bits(d[2 * i]) | f32_to_bf16_bits(d[2 * i + 1]) << 16;
          o = make_uint4(w[0], w[1], w[2], w[3]);
        }
        *reinterpret_cast<uint4*>(static_cast<char*>(A.dlogits) + (t * E + e) * (F32 ? 4 : 2)) = o;
      } else {
#pragma unroll
        for (int i = 0; i < Row::kRun; i++) {
          if (e + i >= E) continue;
          if (F32)
            static_cast<float*>(A.dlogits)[t * E + e + i] = d[i];
          else
            static_cast<uint16_t*>(A.dlogits)[t * E + e + i] = (uint16_t)f32_to_bf16_bits(d[i]);
        }
      }
    }
  }
}

// Lanes a row (G) and values a lane (N) for E experts.
template <class F>
static void by_experts(int E, F f) {
  using std::integral_constant;
  if (E <= 32) f(integral_constant<int, 4>{}, integral_constant<int, 8>{});
  else if (E <= 64) f(integral_constant<int, 8>{}, integral_constant<int, 8>{});
  else if (E <= 128) f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
  else if (E <= 256) f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
  else f(integral_constant<int, 16>{}, integral_constant<int, 32>{});
}

// 16 bytes a lane where every row is 16-byte aligned (and what else is read or written by 16 bytes).
static bool wide_logits(const BalanceArgs& A, const void* b, const void* c) {
  return A.E % (A.f32 ? 4 : 8) == 0 &&
         ((reinterpret_cast<uintptr_t>(A.logits) | reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(c)) & 15) == 0;
}

// Workgroups of 512 threads, or of 1024 where there are more rows than kBalMaxParts
// of the small ones take at once: fewer partial rows make the second launch
// shorter (65536 x 512: 6.1 against 8.6 us), while few rows are done sooner by
// small workgroups (4096 x 256: 5.4 against 6.7 us).
static int64_t row_groups(int T, int E, int threads) {
  const int rows = threads / (E <= 32 ? 4 : E <= 64 ? 8 : 16);
  return ((int64_t)T + rows - 1) / rows;
}

int balance_parts(int T, int E) {
  const int64_t groups = row_groups(T, E, 512);
  return (int)(groups <= 4 ? 1 : groups < kBalMaxParts ? groups : kBalMaxParts);
}

template <bool F32, int G, int N, int NT>
static void launch_rows(const BalanceArgs& A, bool wide, int parts, hipStream_t s, const KTime& kt) {
  auto* f = wide ? k_balance_rows<F32, G, N, true, NT> : k_balance_rows<F32, G, N, false, NT>;
  MOE_LAUNCH(f, dim3(parts), dim3(NT), 0, s, kt.start, parts > 1 ? nullptr : kt.stop, A);
}

hipError_t launch_balance_forward(const BalanceArgs& A, hipStream_t s, const KTime& kt) {
  const int parts = balance_parts(A.T, A.E);
  const bool wide = wide_logits(A, nullptr, nullptr), big = row_groups(A.T, A.E, 512) > kBalMaxParts;
  by_experts(A.E, [&](auto g, auto n) {
    constexpr int G = g.value, N = n.value;
    auto* f = A.f32 ? (big ? launch_rows<true, G, N, 1024> : launch_rows<true, G, N, 512>)
                    : (big ? launch_rows<false, G, N, 1024> : launch_rows<false, G, N, 512>);
    f(A, wide, parts, s, kt);
  });
  if (parts > 1)
    MOE_LAUNCH(k_balance_sum, dim3((A.E + kBalSumExperts - 1) / kBalSumExperts), dim3(kBalSumThreads), 0, s, nullptr,
               kt.stop, A, parts);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceArgs& A, hipStream_t s, const KTime& kt) {
  const bool wide = wide_logits(A, A.dlogits, A.counts);
  by_experts(A.E, [&](auto g, auto n) {
    constexpr int G = g.value, N = n.value, rows = kGradThreads / G;
    const int64_t groups = ((int64_t)A.T + rows - 1) / rows;
    auto* f = A.f32 ? (wide ? k_balance_grad<true, G, N, true> : k_balance_grad<true, G, N, false>)
                    : (wide ? k_balance_grad<false, G, N, true> : k_balance_grad<false, G, N, false>);
    MOE_LAUNCH(f, dim3((unsigned)(groups < 1024 ? groups : 1024)), dim3(kGradThreads), 0, s, kt.start, kt.stop, A);
  });
  return hipGetLastError();
}

}  // namespace moe
