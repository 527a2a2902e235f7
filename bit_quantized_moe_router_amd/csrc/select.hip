// Routing from scores: the choice of k experts a token by softmax or sigmoid
// scores with a bias and groups, the order of the assignments by expert, and the
// gradient of the logits.
//
//   s = softmax(l) or sigmoid(l),  c = s + bias,  the top_groups groups with the
//   largest sums of their group_best largest c,  in them the k largest c,
//   w_j = scale s_j / sum_i s_i  or  scale s_j.
//
// A token's choice is one between numbers that may be close: the ids are those
// of c in float64.  Without a bias s grows with l, so that experts (and groups
// by their largest) are compared by l itself, exactly.
//
// The order by expert is a counting sort that keeps the order of the
// assignments: counts by part of the tokens, their prefix sums over the
// parts, then every part places its own.  Integer counts do not depend on the order
// in which they are added, so repeated calls give the same bits.
#include <type_traits>

#include "launch.h"
#include "small_route.h"
#include "vec.h"

namespace moe {

// ---- one token, exactly -------------------------------------------------------

// What a wave needs in LDS for one token.
struct SelectLds {
  double c[kMaxE];
};

__device__ __forceinline__ double shfl_xor_f64(double v, int d) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __shfl_xor((uint32_t)u, d), hi = __shfl_xor((uint32_t)(u >> 32), d);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

template <bool F32>
__device__ __forceinline__ float logit_at(const void* logits, int64_t i) {
  if constexpr (F32) return static_cast<const float*>(logits)[i];
  return bf16_bits_to_f32(static_cast<const uint16_t*>(logits)[i]);
}

// The groups that stay (bit g), from the choice scores in LDS: lane g sums its
// group's group_best largest, then counts the groups before it.  -inf is an
// expert that is not there; a group without one never stays.
__device__ __forceinline__ uint64_t groups_kept(const SelectArgs& A, const double* c) {
  const int lane = threadIdx.x & 63;
  double sum = -INFINITY;
  if (lane < A.groups) {
    double first = -INFINITY, second = -INFINITY;
    for (int i = 0; i < A.per; i++) {
      const double v = c[lane * A.per + i];
      second = fmax(second, fmin(first, v));
      first = fmax(first, v);
    }
    sum = A.best == 2 && second > -INFINITY ? first + second : first;
  }
  int before = 0;
  for (int g = 0; g < A.groups; g++) {
    const double v = lane_value_f64(sum, g);
    before += v > sum || (v == sum && g < lane) ? 1 : 0;
  }
  return __ballot(lane < A.groups && sum > -INFINITY && before < A.top_groups);
}

// The choice for token t by one wave: lane j < k returns place j's expert (or -1) and its logit; *top and *total are
// the row's largest logit and its sum of exp(l - top).  false: the row holds what no choice is made from (a NaN, with
// softmax +inf).
template <bool F32>
__device__ __forceinline__ bool select_exact(const SelectArgs& A, int64_t t, SelectLds& lds, int* id, float* chosen,
                                             float* top, float* total) {
  const int lane = threadIdx.x & 63;
  float l[kMaxEPerLane];
  double key[kMaxEPerLane];
  bool bad = false;
  float mx = -INFINITY;
#pragma unroll
  for (int j = 0; j < kMaxEPerLane; j++) {
    const int e = lane + 64 * j;
    l[j] = e < A.E ? logit_at<F32>(A.logits, t * A.E + e) : -INFINITY;
    bad = bad || l[j] != l[j] || (A.softmax && l[j] == INFINITY);
    mx = fmaxf(mx, l[j]);
  }
  mx = wave_max_f32(mx);
  *top = mx;
  *id = -1;
  *chosen = -INFINITY;
  if (__ballot(bad)) return false;
  const bool any = mx > -INFINITY;
  // Choice scores: l itself where that gives the same order.
  const bool scores = A.bias || (A.groups > 1 && A.best == 2);
  double s[kMaxEPerLane], sum = 0.0;
#pragma unroll
  for (int j = 0; j < kMaxEPerLane; j++) {
    s[j] = 0.0;
    if (any && l[j] > -INFINITY) s[j] = A.softmax ? exp((double)l[j] - (double)mx) : scores ? 1.0 / (1.0 + exp(-(double)l[j])) : 0.0;
    sum += s[j];
  }
  sum = wave_sum_f64(sum);
  *total = (float)sum;
  bool out[kMaxEPerLane];
#pragma unroll
  for (int j = 0; j < kMaxEPerLane; j++) {
    const int e = lane + 64 * j;
    out[j] = !(l[j] > -INFINITY);
    key[j] = scores ? (A.softmax ? s[j] / sum : s[j]) : (double)l[j];
    if (A.bias && e < A.E) {
      const float b = A.bias[e];
      out[j] = out[j] || !(b > -INFINITY);
      key[j] += (double)b;
    }
    if (out[j]) key[j] = -INFINITY;
  }
  if (A.groups > 1) {
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int j = 0; j < kMaxEPerLane; j++)
      if (lane + 64 * j < A.E) lds.c[lane + 64 * j] = key[j];
    __threadfence_block();
    __builtin_amdgcn_wave_barrier();
    const uint64_t kept = groups_kept(A, lds.c);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int j = 0; j < kMaxEPerLane; j++) {
      const int e = lane + 64 * j;
      out[j] = out[j] || e >= A.E || !((kept >> (min(e, A.E - 1) / A.per)) & 1);
      // In the groups the order is that of l where there is no bias.
      key[j] = out[j] ? -INFINITY : A.bias ? key[j] : (double)l[j];
    }
  }
  for (int i = 0; i < A.k; i++) {
    double best = -INFINITY;
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int j = 0; j < kMaxEPerLane; j++)
      if (!out[j] && (key[j] > best || at == 0x7FFFFFFF)) best = key[j], at = lane + 64 * j;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double v = shfl_xor_f64(best, d);
      const int w = __shfl_xor(at, d);
      // An absent candidate has the largest index and -inf.
      if (v > best || (v == best && w < at)) best = v, at = w;
    }
    if (at == 0x7FFFFFFF) break;
    float mine = 0.f;
#pragma unroll
    for (int j = 0; j < kMaxEPerLane; j++)
      if (lane + 64 * j == at) out[j] = true, mine = l[j];
    mine = __shfl(mine, at & 63);
    if (lane == i) *id = at, *chosen = mine;
  }
  return true;
}

// exp(l) / (1 + exp(l)) times exp(-shift), shift <= 0, for l <= 0 without underflow of what shift cancels; l > 0: shift = 0.
__device__ __forceinline__ float sigmoid_shifted(float l, float shift) {
  return l >= 0.f ? 1.f / (1.f + expf(-l)) : expf(l - shift) / (1.f + expf(l));
}

// Sum over the 16 lanes of a row of lanes.
__device__ __forceinline__ float sum16(float v) { return row_sum16(v); }
__device__ __forceinline__ float max16(float v) {
  v = fmaxf(v, dpp_f32<0xB1>(v));
  v = fmaxf(v, dpp_f32<0x4E>(v));
  v = fmaxf(v, dpp_f32<0x124>(v));
  return fmaxf(v, dpp_f32<0x128>(v));
}

// The weight of each place from its logit, in the first lanes of a row of 16; l = -inf for a place without an expert.
// A score is taken relative to the largest chosen one where it is divided by their sum, so that no logits are too
// small for it.
__device__ __forceinline__ float select_weight(const SelectArgs& A, float l, float top, float total) {
  const float largest = max16(l);
  if (!(largest > -INFINITY)) return 0.f;
  float u;
  if (A.softmax) u = l > -INFINITY ? expf(l - (A.renorm ? largest : top)) : 0.f;
  else u = l > -INFINITY ? sigmoid_shifted(l, A.renorm ? fminf(largest, 0.f) : 0.f) : 0.f;
  if (A.renorm) return A.scale * (u / sum16(u));
  return A.scale * (A.softmax ? u / total : u);
}

constexpr int kSelThreads = 256, kSelWaves = kSelThreads / 64;

template <bool F32>
__device__ __forceinline__ void select_token(const SelectArgs& A, int64_t t, SelectLds& lds, int* s_count) {
  const int lane = threadIdx.x & 63;
  int id = -1;
  float w = 0.f;
  if (!A.valid || A.valid[t]) {
    float l, top, total;
    if (select_exact<F32>(A, t, lds, &id, &l, &top, &total)) w = select_weight(A, l, top, total);
    else w = __builtin_nanf("");
  }
  if (lane < A.k) {
    A.ids[t * A.k + lane] = id;
    A.weights[t * A.k + lane] = w;
    if (s_count && id >= 0) atomicAdd(&s_count[id], 1);
  }
}

// Part b: tokens b * per_part .. ; its counts by expert go to the workspace.
template <bool F32>
__global__ __launch_bounds__(kSelThreads) void k_select(SelectArgs A) {
  __shared__ SelectLds lds[kSelWaves];
  __shared__ int s_count[kMaxE];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int e = threadIdx.x; e < A.E; e += kSelThreads) s_count[e] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * A.per_part, t1 = min((int64_t)A.T, t0 + A.per_part);
  for (int64_t t = t0 + wave; t < t1; t += kSelWaves) select_token<F32>(A, t, lds[wave], A.part_count ? s_count : nullptr);
  if (!A.part_count) return;
  __syncthreads();
  for (int e = threadIdx.x; e < A.E; e += kSelThreads) A.part_count[(int64_t)blockIdx.x * A.E + e] = s_count[e];
}

// ---- the order by expert ---------------------------------------------------------

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;

// Exclusive prefix sum over the workgroup's first 512 threads (0 beyond E).
__device__ __forceinline__ int sort_offsets(int v, int* s_wave) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int incl = wave_incl_scan(v);
  if (lane == 63 && wave < kMaxE / 64) s_wave[wave] = incl;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < kMaxE / 64; w++) base += w < wave ? s_wave[w] : 0;
  return base + incl - v;
}

// Assignments [lo, hi) into the order, stably: a wave has a run of them, 64 at a
// time; lanes with the same expert find each other by ballots.  first(e, n): the
// place of the range's first assignment of expert e, of which it has n (called by
// thread e < 512 of the whole workgroup, n = 0 for e >= E).
template <class First>
__device__ __forceinline__ void sort_range(const int32_t* __restrict__ ids, int64_t lo, int64_t hi, int E,
                                           int32_t* __restrict__ sorted, int (*s_cnt)[kMaxE], First first) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int nbits = E > 1 ? 32 - __clz(E - 1) : 0;
  const uint64_t below = lane == 0 ? 0ull : ~0ull >> (64 - lane);
  for (int i = tid; i < kSortWaves * kMaxE; i += kSortThreads) s_cnt[0][i] = 0;
  __syncthreads();
  const int64_t run = ((hi - lo + kSortWaves - 1) / kSortWaves + 63) & ~(int64_t)63;
  const int64_t a0 = min(hi, lo + wave * run), a1 = min(hi, a0 + run);
  for (int64_t a = a0 + lane; a < a1; a += 64) {
    const int e = ids[a];
    if ((unsigned)e < (unsigned)E) atomicAdd(&s_cnt[wave][e], 1);
  }
  __syncthreads();
  int n = 0;
  if (tid < E)
    for (int w = 0; w < kSortWaves; w++) n += s_cnt[w][tid];
  int at = first(tid, n);
  if (tid < E) {
    for (int w = 0; w < kSortWaves; w++) {
      const int c = s_cnt[w][tid];
      s_cnt[w][tid] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int64_t b = a0; b < a1; b += 64) {
    const int64_t a = b + lane;
    const int e = a < a1 ? ids[a] : -1;
    const bool in = (unsigned)e < (unsigned)E;
    const uint64_t same = match_mask(in ? e : 0, in, nbits);
    const int rank = __popcll(same & below);
    int place = 0;
    if (in && rank == 0) place = atomicAdd(&s_cnt[wave][e], __popcll(same));
    place = __shfl(place, same ? __builtin_ctzll(same) : 0);
    if (in) sorted[place + rank] = (int)a;
  }
}

__device__ __forceinline__ void sort_all(const SortArgs& A, int (*s_cnt)[kMaxE], int* s_wave) {
  sort_range(A.ids, 0, A.n, A.E, A.sorted, s_cnt, [&](int e, int n) {
    const int off = sort_offsets(n, s_wave);
    if (e < A.E) {
      A.counts[e] = n;
      A.offsets[e] = off;
      if (e == A.E - 1) A.offsets[A.E] = off + n;
    }
    return off;
  });
}

// Few assignments: one workgroup.
__global__ __launch_bounds__(kSortThreads) void k_sort_small(SortArgs A) {
  __shared__ int s_cnt[kSortWaves][kMaxE];
  __shared__ int s_wave[kMaxE / 64];
  sort_all(A, s_cnt, s_wave);
}

// Few tokens: the choice and the order in one workgroup.
template <bool F32>
__global__ __launch_bounds__(kSortThreads) void k_select_small(SelectArgs A, SortArgs S) {
  __shared__ SelectLds lds[kSortWaves];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int64_t t = wave; t < A.T; t += kSortWaves) select_token<F32>(A, t, lds[wave], nullptr);
  __syncthreads();
  int(*s_cnt)[kMaxE] = reinterpret_cast<int(*)[kMaxE]>(lds);
  static_assert(sizeof(lds) >= sizeof(int) * kSortWaves * kMaxE, "the counters take the scores' place");
  __shared__ int s_wave[kMaxE / 64];
  sort_all(S, s_cnt, s_wave);
}

// Counts of a part's assignments.
__global__ __launch_bounds__(kSortThreads) void k_sort_count(SortArgs A) {
  __shared__ int s_count[kMaxE];
  for (int e = threadIdx.x; e < A.E; e += kSortThreads) s_count[e] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * A.per_part, hi = min((int64_t)A.n, lo + A.per_part);
  for (int64_t a = lo + threadIdx.x; a < hi; a += kSortThreads) {
    const int e = A.ids[a];
    if ((unsigned)e < (unsigned)A.E) atomicAdd(&s_count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < A.E; e += kSortThreads) A.part_count[(int64_t)blockIdx.x * A.E + e] = s_count[e];
}

// Counts by part to the parts' prefix sums, in place, and to the experts' totals: 16 experts a workgroup, a wave each.
__global__ __launch_bounds__(kSortThreads) void k_sort_scan(SortArgs A) {
  constexpr int kPer = kSortMaxParts / 64;
  __shared__ int s[kSortMaxParts][17];
  const int e0 = blockIdx.x * 16, x = threadIdx.x & 15, y = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const int p = y + 64 * i;
    s[p][x] = p < A.parts && e0 + x < A.E ? A.part_count[(int64_t)p * A.E + e0 + x] : 0;
  }
  __syncthreads();
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int v[kPer], mine = 0;
#pragma unroll
  for (int i = 0; i < kPer; i++) mine += v[i] = s[lane * kPer + i][wave];
  int at = wave_incl_scan(mine);
  if (lane == 63 && e0 + wave < A.E) A.counts[e0 + wave] = at;
  at -= mine;
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    s[lane * kPer + i][wave] = at;
    at += v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const int p = y + 64 * i;
    if (p < A.parts && e0 + x < A.E) A.part_count[(int64_t)p * A.E + e0 + x] = s[p][x];
  }
}

__global__ __launch_bounds__(kSortThreads) void k_sort_place(SortArgs A) {
  __shared__ int s_cnt[kSortWaves][kMaxE];
  __shared__ int s_wave[kMaxE / 64];
  const int64_t lo = (int64_t)blockIdx.x * A.per_part, hi = min((int64_t)A.n, lo + A.per_part);
  const int e = threadIdx.x;
  const int total = e < A.E ? A.counts[e] : 0;
  const int before = e < A.E ? A.part_count[(int64_t)blockIdx.x * A.E + e] : 0;
  sort_range(A.ids, lo, hi, A.E, A.sorted, s_cnt, [&](int, int) {
    const int off = sort_offsets(total, s_wave);
    if (blockIdx.x == 0 && e < A.E) {
      A.offsets[e] = off;
      if (e == A.E - 1) A.offsets[A.E] = off + total;
    }
    return off + before;
  });
}

// ---- the gradient ------------------------------------------------------------------

// With D = sum_i dw_i w_i over the chosen:
//   renormalised  softmax dl_j = w_j (dw_j - D / scale),  sigmoid the same times 1 - s_j
//   as they are   sigmoid dl_j = w_j (1 - s_j) dw_j,      softmax dl_e = w_e dw_e - s_e D, for every expert.
template <bool F32>
__global__ __launch_bounds__(kSelThreads) void k_select_grad(SelectArgs A) {
  constexpr int V = F32 ? 4 : 8, kSize = F32 ? 4 : 2, kPieces = kMaxE / 64 / V;
  __shared__ float s_row[kSelWaves][kMaxE];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  float* row = s_row[wave];
  for (int i = lane; i < kMaxE; i += 64) row[i] = 0.f;
  const bool dense = A.softmax && !A.renorm, in_place = A.base && A.base == A.dlogits;
  const float inv_scale = 1.f / A.scale;
  for (int64_t t = (int64_t)blockIdx.x * kSelWaves + wave; t < A.T; t += (int64_t)gridDim.x * kSelWaves) {
    int id = -1;
    float w = 0.f, dw = 0.f;
    if (lane < A.k) {
      id = A.ids[t * A.k + lane];
      w = A.weights[t * A.k + lane];
      dw = A.dweights[t * A.k + lane];
      if ((unsigned)id >= (unsigned)A.E) id = -1, dw = 0.f;
    }
    const bool none = __ballot(id >= 0) == 0, bad = __ballot(w != w) != 0;
    // Every expert's logit is read before any place is written: dlogits may stand in the logits' place.
    RowPiece<F32, V> l[kPieces];
    float top = -INFINITY, total = 0.f;
    if (dense && !none) {
#pragma unroll
      for (int p = 0; p < kPieces; p++) {
        const int c = (lane + 64 * p) * V;
        l[p].clear();
        if (c < A.E) l[p].load(static_cast<const char*>(A.logits) + (t * A.E + c) * kSize, A.E - c);
#pragma unroll
        for (int i = 0; i < V; i++)
          if (c + i < A.E) top = fmaxf(top, l[p].get(i));
      }
      top = wave_max_f32(top);
#pragma unroll
      for (int p = 0; p < kPieces; p++)
#pragma unroll
        for (int i = 0; i < V; i++)
          if ((lane + 64 * p) * V + i < A.E) total += __expf(l[p].get(i) - top);
      total = wave_sum_f32(total);
    }
    const float D = sum16(id >= 0 ? dw * w : 0.f);
    float d = 0.f;
    if (id >= 0) {
      d = w * (A.renorm ? dw - D * inv_scale : dw);
      if (!A.softmax) {
        const float v = logit_at<F32>(A.logits, t * A.E + id);  // 1 - s = 1 / (1 + e^l)
        d *= v >= 0.f ? expf(-v) / (1.f + expf(-v)) : 1.f / (1.f + expf(v));
      }
    }
    if (in_place && !dense && !bad) {
      if (id >= 0) {
        char* p = static_cast<char*>(A.dlogits) + (t * A.E + id) * kSize;
        const float v = logit_at<F32>(A.dlogits, t * A.E + id) + d;
        if constexpr (F32) *reinterpret_cast<float*>(p) = v;
        else *reinterpret_cast<uint16_t*>(p) = (uint16_t)f32_to_bf16_bits(v);
      }
      continue;
    }
    if (id >= 0) row[id] = d;
    __threadfence_block();
    __builtin_amdgcn_wave_barrier();
    const float all = dense && !none ? lane_value(D, 0) / total : 0.f;
#pragma unroll
    for (int p = 0; p < kPieces; p++) {
      const int c = (lane + 64 * p) * V;
      if (c >= A.E) continue;
      float v[V];
#pragma unroll
      for (int i = 0; i < V; i++) {
        v[i] = row[c + i];
        if (dense && !none) v[i] -= all * __expf(l[p].get(i) - top);
        if (bad) v[i] = __builtin_nanf("");
      }
      RowPiece<F32, V> o;
      if (A.base) {
        o.load(static_cast<const char*>(A.base) + (t * A.E + c) * kSize, A.E - c);
#pragma unroll
        for (int i = 0; i < V; i++) v[i] += o.get(i);
      }
      o.set(v);
      o.store(static_cast<char*>(A.dlogits) + (t * A.E + c) * kSize, A.E - c);
    }
    __builtin_amdgcn_wave_barrier();
    if (id >= 0) row[id] = 0.f;
    __threadfence_block();
    __builtin_amdgcn_wave_barrier();
  }
}

// ---- launches ------------------------------------------------------------------------

// Assignments that one workgroup orders by itself.
constexpr int64_t kSortSmall = 4096;
// Tokens that one workgroup chooses for before it orders them.
constexpr int kSelectSmall = 32;

int sort_parts(int64_t n) {
  const int64_t parts = (n + kSortSmall - 1) / kSortSmall;
  return (int)(parts < 1 ? 1 : parts < kSortMaxParts ? parts : kSortMaxParts);
}

int select_parts(int T) {
  if (T <= kSelectSmall) return 1;
  const int parts = (T + 15) / 16;
  return parts < kSortMaxParts ? parts : kSortMaxParts;
}

static hipError_t launch_order(SortArgs S, hipStream_t s, hipEvent_t stop) {
  MOE_LAUNCH(k_sort_scan, dim3((S.E + 15) / 16), dim3(kSortThreads), 0, s, nullptr, nullptr, S);
  MOE_LAUNCH(k_sort_place, dim3(S.parts), dim3(kSortThreads), 0, s, nullptr, stop, S);
  return hipGetLastError();
}

hipError_t launch_sort(SortArgs S, hipStream_t s, const KTime& kt) {
  S.parts = sort_parts(S.n);
  if (S.parts == 1) {
    MOE_LAUNCH(k_sort_small, dim3(1), dim3(kSortThreads), 0, s, kt.start, kt.stop, S);
    return hipGetLastError();
  }
  S.per_part = (S.n + (int64_t)S.parts - 1) / S.parts;
  MOE_LAUNCH(k_sort_count, dim3(S.parts), dim3(kSortThreads), 0, s, kt.start, nullptr, S);
  return launch_order(S, s, kt.stop);
}

hipError_t launch_select_forward(SelectArgs A, SortArgs S, bool order, hipStream_t s, const KTime& kt) {
  const int parts = select_parts(A.T);
  if (parts == 1 && order) {
    auto* f = A.f32 ? k_select_small<true> : k_select_small<false>;
    MOE_LAUNCH(f, dim3(1), dim3(kSortThreads), 0, s, kt.start, kt.stop, A, S);
    return hipGetLastError();
  }
  A.per_part = (A.T + (int64_t)parts - 1) / parts;
  A.part_count = order ? S.part_count : nullptr;
  auto* f = A.f32 ? k_select<true> : k_select<false>;
  MOE_LAUNCH(f, dim3(parts), dim3(kSelThreads), 0, s, kt.start, order ? nullptr : kt.stop, A);
  if (!order) return hipGetLastError();
  S.parts = parts;
  S.per_part = A.per_part * A.k;
  return launch_order(S, s, kt.stop);
}

hipError_t launch_select_backward(const SelectArgs& A, hipStream_t s, const KTime& kt) {
  const int64_t groups = ((int64_t)A.T + kSelWaves - 1) / kSelWaves;
  auto* f = A.f32 ? k_select_grad<true> : k_select_grad<false>;
  MOE_LAUNCH(f, dim3((unsigned)(groups < 4096 ? groups : 4096)), dim3(kSelThreads), 0, s, kt.start, kt.stop, A);
  return hipGetLastError();
}

}  // namespace moe
