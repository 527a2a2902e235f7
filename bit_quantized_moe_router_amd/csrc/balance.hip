// The router's balance loss with its per-expert counts, and its gradient.
//
// With p_t the softmax of token t's logits, n the valid tokens, c_e the valid
// assignments of expert e, P_e = sum_t p_te / n and f_e = c_e / (n k):
//   balance = E sum_e f_e P_e,   z = sum_t lse_t^2 / n,   loss = a balance + b z,
//   dloss/dl_te = p_te (a E / n (f_e - sum_j f_j p_tj) + 2 b lse_t / n)
// (f is made of counts and has no gradient).
//
// Forward: a group of lanes takes a row (as many lanes as the experts need, at
// most a wave), adds its probabilities to per-lane sums and its ids to integer
// counters in LDS; each workgroup leaves one partial row.  A second launch
// sums the partial rows by expert in a fixed order in float64; its last
// workgroup to finish joins the balance sum, also in a fixed order, so repeated
// calls give identical bits.  Small inputs take one workgroup and one launch.
// Backward: one pass that takes the softmax again from the logits.  Both are
// bound by reading (and writing) the logits.
#include <type_traits>

#include "launch.h"
#include "mx4.h"

namespace moe {

constexpr int kBalThreads = 256;
constexpr int kBalWaves = kBalThreads / 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Sum / maximum over groups of G consecutive lanes, in every lane of the group.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int d = 1; d < G; d <<= 1) v += __shfl_xor(v, d);
  return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int d = 1; d < G; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

template <bool F32>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  return F32 ? static_cast<const float*>(p)[i] : bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// The row's softmax in p (lane `g` of the group holds experts g, g + G, ...)
// and its log-sum-exp.  A row of -inf alone has p = 0 and lse = 0; NaNs stay.
template <bool F32, int G, int V>
__device__ __forceinline__ void softmax_row(const void* logits, int64_t t, int E, int g, float p[V], float* lse) {
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < V; j++) {
    const int e = g + G * j;
    p[j] = e < E ? load_logit<F32>(logits, t * E + e) : -INFINITY;
    top = fmaxf(top, p[j]);
  }
  top = group_max<G>(top);
  if (top == -INFINITY) top = 0.f;
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < V; j++) {
    p[j] = __builtin_amdgcn_exp2f((p[j] - top) * kLog2e);
    sum += p[j];
  }
  sum = group_sum<G>(sum);
  if (sum == 0.f) {
    *lse = 0.f;
    return;
  }
  const float inv = 1.f / sum;
#pragma unroll
  for (int j = 0; j < V; j++) p[j] *= inv;
  *lse = top + __builtin_amdgcn_logf(sum) * kLn2;
}

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
template <bool F32, int G, int V>
__global__ __launch_bounds__(kBalThreads) void k_balance_rows(BalanceArgs A) {
  constexpr int kRows = kBalThreads / G;  // rows in flight a workgroup
  __shared__ int s_count[512];
  __shared__ float s_p[kBalWaves][G * V];
  __shared__ double s_z[kBalWaves];
  __shared__ int s_n[kBalWaves];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, g = lane & (G - 1);
  const int E = A.E;
  if (blockIdx.x == 0 && tid == 0) *A.done = 0;  // the second launch's counter
  for (int e = tid; e < E; e += kBalThreads) s_count[e] = 0;
  __syncthreads();
  float acc[V] = {};
  double z = 0.0;
  int n = 0;
  for (int64_t t = (int64_t)blockIdx.x * kRows + tid / G; t < A.T; t += (int64_t)gridDim.x * kRows) {
    if (A.valid && !A.valid[t]) continue;
    float p[V], lse;
    softmax_row<F32, G, V>(A.logits, t, E, g, p, &lse);
#pragma unroll
    for (int j = 0; j < V; j++) acc[j] += p[j];
    if (g == 0) {
      z += (double)lse * lse;
      n += 1;
    }
    for (int j = g; j < A.k; j += G) {
      const int e = A.ids[t * A.k + j];
      if ((unsigned)e < (unsigned)E) atomicAdd(&s_count[e], 1);
    }
  }
  // Groups of a wave, then waves, in a fixed order.
#pragma unroll
  for (int d = G; d < 64; d <<= 1) {
#pragma unroll
    for (int j = 0; j < V; j++) acc[j] += __shfl_xor(acc[j], d);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    z += __shfl_xor(z, d);
    n += __shfl_xor(n, d);
  }
  if (lane < G) {
#pragma unroll
    for (int j = 0; j < V; j++) s_p[wave][g + G * j] = acc[j];
  }
  if (lane == 0) s_z[wave] = z, s_n[wave] = n;
  __syncthreads();
  z = (s_z[0] + s_z[1]) + (s_z[2] + s_z[3]);
  n = (s_n[0] + s_n[1]) + (s_n[2] + s_n[3]);
  if (gridDim.x > 1) {
    for (int e = tid; e < E; e += kBalThreads) {
      A.part_p[(int64_t)blockIdx.x * E + e] = (s_p[0][e] + s_p[1][e]) + (s_p[2][e] + s_p[3][e]);
      A.part_count[(int64_t)blockIdx.x * E + e] = s_count[e];
    }
    if (tid == 0) {
      A.part_z[blockIdx.x] = z;
      A.part_n[blockIdx.x] = n;
    }
    return;
  }
  double dot = 0.0;
  for (int e = tid; e < E; e += kBalThreads) {
    const double pe = n > 0 ? ((double)s_p[0][e] + s_p[1][e] + s_p[2][e] + s_p[3][e]) / n : 0.0;
    A.mean_prob[e] = (float)pe;
    A.counts[e] = s_count[e];
    if (n > 0) dot += pe * s_count[e] / ((double)n * A.k);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) dot += __shfl_xor(dot, d);
  __syncthreads();
  if (lane == 0) s_z[wave] = dot;
  __syncthreads();
  if (tid == 0) balance_finish(A, (s_z[0] + s_z[1]) + (s_z[2] + s_z[3]), z, n);
}

// Second launch: workgroup b sums the partial rows of 16 experts, 16 threads
// an expert; the last workgroup to arrive adds the workgroups' parts of the
// balance sum in order.
constexpr int kBalSumExperts = 16;

__global__ __launch_bounds__(kBalThreads) void k_balance_sum(BalanceArgs A, int parts) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // Lane l: expert l & 15 of the workgroup's, slice (wave, l >> 4) of the parts.
  const int e = blockIdx.x * kBalSumExperts + (lane & 15), slice = wave * 4 + (lane >> 4);
  double p = 0.0, z = 0.0;
  int c = 0, n = 0;
  for (int g = slice; g < parts; g += 16) {
    if (e < A.E) {
      p += (double)A.part_p[(int64_t)g * A.E + e];
      c += A.part_count[(int64_t)g * A.E + e];
    }
    z += A.part_z[g];
    n += A.part_n[g];
  }
  __shared__ double s_p[16][17];
  __shared__ int s_c[16][17];
  __shared__ double s_z[16];
  __shared__ int s_n[16];
  s_p[slice][lane & 15] = p;
  s_c[slice][lane & 15] = c;
  if ((lane & 15) == 0) s_z[slice] = z, s_n[slice] = n;
  __syncthreads();
  if (wave != 0) return;
  p = 0.0, z = 0.0, c = 0, n = 0;
  for (int i = 0; i < 16; i++) {
    p += s_p[i][lane & 15];
    c += s_c[i][lane & 15];
    z += s_z[i];
    n += s_n[i];
  }
  double dot = 0.0;
  if (lane < 16 && e < A.E) {
    const double pe = n > 0 ? p / n : 0.0;
    A.mean_prob[e] = (float)pe;
    A.counts[e] = c;
    if (n > 0) dot = pe * c / ((double)n * A.k);
  }
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) dot += __shfl_xor(dot, d);
  int last = 0;
  if (lane == 0) {
    __hip_atomic_store(&A.dots[blockIdx.x], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = __hip_atomic_fetch_add(A.done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
  }
  if (lane != 0 || !last) return;
  dot = 0.0;
  for (int b = 0; b < (int)gridDim.x; b++)
    dot += __hip_atomic_load(&A.dots[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  balance_finish(A, dot, z, n);
}

template <bool F32, int G, int V>
__global__ __launch_bounds__(kBalThreads) void k_balance_grad(BalanceArgs A) {
  constexpr int kRows = kBalThreads / G;
  const int lane = threadIdx.x & 63, g = lane & (G - 1);
  const int E = A.E, n = A.n_valid[0];
  const float up = A.grad ? A.grad[0] : 1.f;
  // a E / n * f_e, with f_e = c_e / (n k), and the z term's 2 b / n.
  const float scale = n > 0 ? up / (float)n : 0.f;
  const float za = 2.f * A.z_coef * scale;
  float f[V];
#pragma unroll
  for (int j = 0; j < V; j++) {
    const int e = g + G * j;
    f[j] = e < E && n > 0 ? A.balance_coef * E * scale * ((float)A.counts[e] / ((float)n * A.k)) : 0.f;
  }
  for (int64_t t = (int64_t)blockIdx.x * kRows + threadIdx.x / G; t < A.T; t += (int64_t)gridDim.x * kRows) {
    const bool on = n > 0 && (!A.valid || A.valid[t]);
    float p[V], lse = 0.f, dot = 0.f;
    if (on) {
      softmax_row<F32, G, V>(A.logits, t, E, g, p, &lse);
#pragma unroll
      for (int j = 0; j < V; j++) dot += p[j] * f[j];
      dot = group_sum<G>(dot);
    }
#pragma unroll
    for (int j = 0; j < V; j++) {
      const int e = g + G * j;
      if (e >= E) continue;
      const float d = on ? p[j] * (f[j] - dot + za * lse) : 0.f;
      if (F32)
        static_cast<float*>(A.dlogits)[t * E + e] = d;
      else
        static_cast<uint16_t*>(A.dlogits)[t * E + e] = (uint16_t)f32_to_bf16_bits(d);
    }
  }
}

// Lanes a row and values a lane for E experts.
template <class F>
static void by_experts(int E, F f) {
  if (E <= 8) f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
  else if (E <= 16) f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
  else if (E <= 32) f(std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{});
  else if (E <= 64) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  else if (E <= 128) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  else if (E <= 256) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
  else f(std::integral_constant<int, 64>{}, std::integral_constant<int, 8>{});
}

int balance_parts(int T, int E) {
  const int rows = kBalThreads / (E <= 8 ? 8 : E <= 16 ? 16 : E <= 32 ? 32 : 64);
  const int64_t groups = ((int64_t)T + rows - 1) / rows;
  return (int)(groups <= 4 ? 1 : groups < kBalMaxParts ? groups : kBalMaxParts);
}

hipError_t launch_balance_forward(const BalanceArgs& A, hipStream_t s, const KTime& kt) {
  const int parts = balance_parts(A.T, A.E);
  by_experts(A.E, [&](auto g, auto v) {
    auto* f = A.f32 ? k_balance_rows<true, g.value, v.value> : k_balance_rows<false, g.value, v.value>;
    MOE_LAUNCH(f, dim3(parts), dim3(kBalThreads), 0, s, kt.start, parts > 1 ? nullptr : kt.stop, A);
  });
  if (parts > 1)
    MOE_LAUNCH(k_balance_sum, dim3((A.E + kBalSumExperts - 1) / kBalSumExperts), dim3(kBalThreads), 0, s, nullptr,
               kt.stop, A, parts);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceArgs& A, hipStream_t s, const KTime& kt) {
  by_experts(A.E, [&](auto g, auto v) {
    constexpr int rows = kBalThreads / g.value;
    const int64_t groups = ((int64_t)A.T + rows - 1) / rows;
    auto* f = A.f32 ? k_balance_grad<true, g.value, v.value> : k_balance_grad<false, g.value, v.value>;
    MOE_LAUNCH(f, dim3((unsigned)(groups < 4096 ? groups : 4096)), dim3(kBalThreads), 0, s, kt.start, kt.stop, A);
  });
  return hipGetLastError();
}

}  // namespace moe
