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

// What a wave needs in LDS for one token: the choice scores.
struct SelectLds {
  double c[kMaxE];
};

template <bool F32>
__device__ __forceinline__ float logit_at(const void* logits, int64_t i) {
  if constexpr (F32) return static_cast<const float*>(logits)[i];
  return bf16_bits_to_f32(static_cast<const uint16_t*>(logits)[i]);
}

// LDS that this wave has written may be read by its other lanes.
__device__ __forceinline__ void wave_lds() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ double lane_from_f64(double v, int from) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __shfl((uint32_t)u, from), hi = __shfl((uint32_t)(u >> 32), from);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// The groups that stay (bit g), from the choice scores in LDS: 64 / n_groups lanes a group find its group_best largest,
// then every group counts those before it.  -inf is an expert that is not there; a group without one never stays.
__device__ __forceinline__ uint64_t groups_kept(const SelectArgs& A, const double* c) {
  const int lane = threadIdx.x & 63, per = 64 / A.groups;
  const int group = lane / per, pos = lane - group * per;
  double first = -INFINITY, second = -INFINITY;
  if (group < A.groups)
    for (int i = pos; i < A.per; i += per) {
      const double v = c[group * A.per + i];
      second = fmax(second, fmin(first, v));
      first = fmax(first, v);
    }
  double a = first, b = second;
  for (int i = 1; i < per; i++) {
    const int from = lane - pos + (pos + i < per ? pos + i : pos + i - per);
    const double ga = lane_from_f64(first, from), gb = lane_from_f64(second, from);
    b = fmax(fmax(b, gb), fmin(a, ga));
    a = fmax(a, ga);
  }
  const double sum = A.best == 2 && b > -INFINITY ? a + b : a;
  int before = 0;
  for (int g = 0; g < A.groups; g++) {
    const double v = lane_value_f64(sum, g * per);
    before += v > sum || (v == sum && g < group) ? 1 : 0;
  }
  const uint64_t in = __ballot(pos == 0 && group < A.groups && sum > -INFINITY && before < A.top_groups);
  uint64_t kept = 0;
  for (uint64_t left = in; left; left &= left - 1) kept |= 1ull << (__builtin_ctzll(left) / per);
  return kept;
}

// The choice for token t by one wave, in float64: lane j < k returns place j's expert (or -1).  false: the row holds
// what no choice is made from (a NaN, with softmax +inf).  Taken for rows whose choice float32 leaves open, about one
// in a thousand of random ones.
template <bool F32>
__device__ __forceinline__ bool select_exact(const SelectArgs& A, int64_t t, double* c, int* id) {
  // The scores are kept in LDS and gone through by loops, so that this rare part asks for few registers.
  const int lane = threadIdx.x & 63;
  float mx = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < kMaxEPerLane; j++) {
    const int e = lane + 64 * j;
    const float l = e < A.E ? logit_at<F32>(A.logits, t * A.E + e) : -INFINITY;
    c[e] = (double)l;
    bad = bad || l != l || (A.softmax && l == INFINITY);
    mx = fmaxf(mx, l);
  }
  mx = wave_max_f32(mx);
  *id = -1;
  if (__ballot(bad)) return false;
  if (!(mx > -INFINITY)) return true;
  wave_lds();
  // Choice scores: l itself where that gives the same order.
  const bool scores = A.bias || (A.groups > 1 && A.best == 2);
  double sum = 0.0;
  if (scores) {
#pragma unroll 1
    for (int e = lane; e < A.E; e += 64) {
      const double l = c[e], v = exp(A.softmax ? l - (double)mx : -l);
      const double s = l == -INFINITY ? 0.0 : A.softmax ? v : 1.0 / (1.0 + v);
      sum += s;
      c[e] = s;
    }
    if (A.softmax) sum = wave_sum_f64(sum);
    wave_lds();
  }
  // With the bias; -inf for experts that are not there (a score of 0 may be one of them).
#pragma unroll 1
  for (int e = lane; e < A.E; e += 64) {
    double v = c[e];
    if (scores && A.softmax) v /= sum;
    bool out = !(logit_at<F32>(A.logits, t * A.E + e) > -INFINITY);
    if (A.bias) {
      const float b = A.bias[e];
      out = out || !(b > -INFINITY);
      v += (double)b;
    }
    c[e] = out ? -INFINITY : v;
  }
  wave_lds();
  if (A.groups > 1) {
    const uint64_t kept = groups_kept(A, c);
    wave_lds();
#pragma unroll 1
    for (int e = lane; e < A.E; e += 64) {
      // In the groups the order is that of l where there is no bias.
      if (!((kept >> (e / A.per)) & 1)) c[e] = -INFINITY;
      else if (!A.bias && c[e] > -INFINITY) c[e] = (double)logit_at<F32>(A.logits, t * A.E + e);
    }
    wave_lds();
  }
#pragma unroll 1
  for (int i = 0; i < A.k; i++) {
    double best = -INFINITY;
    int at = lane;
#pragma unroll
    for (int j = 0; j < kMaxEPerLane; j++) {
      const double v = c[lane + 64 * j];  // -inf behind the last expert
      if (v > best) best = v, at = lane + 64 * j;
    }
    const double top = wave_max_f64(best);
    if (!(top > -INFINITY)) break;
    // Of lanes with the same score the one with the lowest expert.
    uint64_t who = __ballot(best == top);
    int e = lane_value(at, __builtin_ctzll(who));
    for (who &= who - 1; who; who &= who - 1) e = min(e, lane_value(at, __builtin_ctzll(who)));
    if (lane == i) *id = e;
    if (lane == (e & 63)) c[e] = -INFINITY;
    wave_lds();
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

// ---- four tokens a wave ------------------------------------------------------------
//
// 16 lanes a token.  Each lane has a run of up to NB experts (of one group, where there are groups: 16 / n_groups
// lanes each), turned into keys of 32 bits: 23 bits of a score, then 4 bits of the lane and 5 of the place in its run,
// counted down.  One integer maximum then finds the best of the lanes and who it is, ties towards the lower index.  A
// lane sorts its keys down to its eight largest; k times the largest head of the 16 lanes is taken and its lane moves
// up.  Bound by the instructions: about 1400 for four tokens of 512 experts with k = 16, a third of them the scores (an
// exponential and a reciprocal each, four times a plain instruction's time), a third the sort and the rounds.  65536
// such tokens in 8 groups take 68 to 71 us (bf16, 67 MB read, 12 written).
//
// Logits that bf16 holds are compared by their 16 bits, exactly.  Other scores are in fixed point, from float32
// functions: they order nearly every row as float64 would.  Neighbours among the chosen that are closer than the scores'
// error are put in order by float64, and so are the last chosen and the first left out; a row goes to select_exact where
// that does not settle it, where a third one is that close to these two (on either side), where the last group that
// stays and the next are that close, where a lane ran out of sorted keys, and where a logit is NaN or +inf.
constexpr int kSelThreads = 256, kSelWaves = kSelThreads / 64;
constexpr int kSelPart = 16;  // tokens that a workgroup of kSelThreads takes at once
constexpr int kSelRuns = 8;     // a lane's sorted keys
constexpr int kSelMaxRun = 32;  // a lane's experts

// What a score is: the logit itself (no bias, no sums), its softmax or its sigmoid.
enum { kByLogit = 0, kBySoftmax = 1, kBySigmoid = 2, kByOne = 3 /* a wave a token */ };

__device__ __forceinline__ uint32_t umax16(uint32_t v) {
  v = max(v, (uint32_t)dpp_i32<0xB1>((int)v));
  v = max(v, (uint32_t)dpp_i32<0x4E>((int)v));
  v = max(v, (uint32_t)dpp_i32<0x141>((int)v));
  return max(v, (uint32_t)dpp_i32<0x140>((int)v));
}
__device__ __forceinline__ float min16(float v) { return -max16(-v); }

__device__ __forceinline__ void order2(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b), lo = min(a, b);
  a = hi, b = lo;
}
// Largest first (19 exchanges).
__device__ __forceinline__ void sort8(uint32_t* v) {
  order2(v[0], v[2]), order2(v[1], v[3]), order2(v[4], v[6]), order2(v[5], v[7]);
  order2(v[0], v[4]), order2(v[1], v[5]), order2(v[2], v[6]), order2(v[3], v[7]);
  order2(v[0], v[1]), order2(v[2], v[3]), order2(v[4], v[5]), order2(v[6], v[7]);
  order2(v[2], v[4]), order2(v[3], v[5]);
  order2(v[1], v[4]), order2(v[3], v[6]);
  order2(v[1], v[2]), order2(v[3], v[4]), order2(v[5], v[6]);
}
// The eight largest of two sorted runs, sorted: one against the other reversed is a bitonic run of the larger halves.
__device__ __forceinline__ void merge8(uint32_t* a, const uint32_t* b) {
#pragma unroll
  for (int i = 0; i < 8; i++) a[i] = max(a[i], b[7 - i]);
#pragma unroll
  for (int d = 4; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (!(i & d)) order2(a[i], a[i + d]);
}
// What the bias asks of all rows of a call.
struct BiasRange {
  bool exact;  // every row by select_exact
  // Keys of the scores with it: score * scale + offset, off by `step` a unit of the scores' error.
  float scale, offset, far, step;
};

__device__ __forceinline__ BiasRange bias_range(const SelectArgs& A) {
  BiasRange r{};
  if (!A.bias) return r;
  float low = INFINITY, high = -INFINITY;
  bool inf = false;
  for (int e = threadIdx.x & 63; e < A.E; e += 64) {
    const float b = A.bias[e];
    if (b > -INFINITY && b < INFINITY) low = fminf(low, b), high = fmaxf(high, b);
    else inf = inf || b == INFINITY;
  }
  low = -wave_max_f32(-low);
  high = wave_max_f32(high);
  if (!(low <= high)) low = high = 0.f;
  r.far = fmaxf(fabsf(low), fabsf(high));
  // +inf, and biases so far from zero next to their range that float32 sums do not tell scores apart.
  r.exact = __ballot(inf) != 0 || !(r.far < 1048576.f * (1.f + (high - low)));
  // 512 at least: the offset is off by half a step of low * scale or of what is added to it, and a sum in float32 is never
  // below its bias.  Keys beyond 2^32 are cut off there, which brings none nearer to another than `gap` unless they are.
  r.scale = 4294000000.f / (1.f + (high - low));
  r.offset = fmaf(-low, r.scale, fmaf(1.2e-7f * r.far, r.scale, 600.f));
  r.step = 2.f / 512 * r.scale;
  return r;
}

// Lanes whose numbers are next to each other in the order of (v, larger first; id, smaller first) change places in
// pairs (`odd`: lanes 1 and 2, 3 and 4, ...; else 0 and 1, ...), of the first k of 16.
__device__ __forceinline__ void swap_pairs(double& v, int& id, int k, bool odd) {
  const int g = threadIdx.x & 15;
  const bool left = (g & 1) == (odd ? 1 : 0);
  const int other = (threadIdx.x & 48) + ((left ? g + 1 : g - 1) & 15);
  const double w = __shfl(v, other);
  const int wid = __shfl(id, other);
  const bool pair = left ? g + 1 < k : g >= 1 && g < k;
  const bool before = v > w || (v == w && id < wid);  // this lane's comes first
  if (pair && before != left) v = w, id = wid;
}

// A lane's part of a token.
struct SelectLane {
  int group, pos, lanes;  // its group, its place in it, lanes a group
  int e0, n;              // its experts
};

__device__ __forceinline__ SelectLane select_lane(const SelectArgs& A) {
  const int g = threadIdx.x & 15;
  SelectLane L;
  L.lanes = A.lanes;
  L.group = g / A.lanes;
  L.pos = g - L.group * A.lanes;
  const int first = L.pos * A.run;
  L.e0 = L.group * A.per + first;
  L.n = L.group < A.groups ? max(0, min(A.run, A.per - first)) : 0;
  return L;
}

// Eight of a lane's logits, from number p of its run; places past its run hold -inf, a row that is not there zeros.
template <bool F32>
__device__ __forceinline__ RowPiece<F32, 8> select_piece(const char* at, bool row, int n, int p) {
  RowPiece<F32, 8> r;
#pragma unroll
  for (int i = 0; i < r.kWords; i++) r.w[i] = !row ? 0u : F32 ? 0xFF800000u : 0xFF80FF80u;
  at += p * (F32 ? 4 : 2);
  if (!row) return r;
  if (n >= p + 8) {
    r.load(at, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) {
      if (p + i >= n) continue;
      if constexpr (F32) r.w[i] = reinterpret_cast<const uint32_t*>(at)[i];
      else {
        const uint32_t v = reinterpret_cast<const uint16_t*>(at)[i];
        r.w[i / 2] = i & 1 ? (r.w[i / 2] & 0xFFFFu) | v << 16 : (r.w[i / 2] & 0xFFFF0000u) | v;
      }
    }
  }
  return r;
}

// v to an integer, cut off at 0 and 2^32; a NaN and -inf give 0.
__device__ __forceinline__ uint32_t to_u32(float v) {
  uint32_t u;
  asm("v_cvt_u32_f32 %0, %1" : "=v"(u) : "v"(v));
  return u;
}

typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

template <bool F32, int By, bool Biased>
__device__ __forceinline__ uint64_t select_four(const SelectArgs& A, int64_t t0, int64_t t1, const SelectLane& L,
                                                const BiasRange& B, const float4* s_bias, int* s_count, int* s_ids) {
  constexpr uint32_t kScore = 0xFFFFFE00u;  // a key's bits of the score
  const int lane = threadIdx.x & 63, g = lane & 15;
  const int64_t t = t0 + (lane >> 4);
  const bool row = t < t1 && (!A.valid || A.valid[t]);
  const char* at_row = static_cast<const char*>(A.logits) + (t * A.E + L.e0) * (F32 ? 4 : 2);
  constexpr float kLog2 = 1.4426950408889634f;
  // The lane's logits eight at a time, the next eight on their way.  A loop: unrolled, the code and its registers were
  // several times as long and as many, and slower.
  auto each = [&](auto f) {
    RowPiece<F32, 8> cur = select_piece<F32>(at_row, row, L.n, 0);
#pragma unroll 1
    for (int p = 0; p < A.run; p += 8) {
      RowPiece<F32, 8> next = cur;
      if (p + 8 < A.run) next = select_piece<F32>(at_row, row, L.n, p + 8);
      f(p, cur);
      cur = next;
    }
  };
  // What the row as a whole is asked for: its largest logit, the sum of exp(l - top), its smallest, whether bf16 holds
  // all of its values, and whether one is +inf or a NaN.
  float top = -INFINITY, low = INFINITY, total = 1.f;
  uint32_t bits = 0;
  bool bad = false;
  const bool sums = By == kBySoftmax || (A.softmax && !A.renorm);
  if (sums || (F32 && !Biased)) {
    each([&](int, const RowPiece<F32, 8>& r) {
#pragma unroll
      for (int i = 0; i < 8; i++) {
        top = fmaxf(top, r.get(i));
        if constexpr (F32 && !Biased) {
          low = fminf(low, r.get(i) > -INFINITY ? r.get(i) : INFINITY);
          bits |= __float_as_uint(r.get(i));
        }
      }
    });
    top = max16(top);
  }
  const float ref = top > -INFINITY ? top : 0.f;
  if (sums) {
    total = 0.f;
    each([&](int, const RowPiece<F32, 8>& r) {
#pragma unroll
      for (int i = 0; i < 8; i++) total += __builtin_amdgcn_exp2f((r.get(i) - ref) * kLog2);
    });
    total = sum16(total);
  }
  // One lane's for the whole row: the lanes' sums differ in their order, and equal logits are to have equal scores.
  const float inv = By == kBySoftmax ? __shfl(__builtin_amdgcn_rcpf(total), lane & 48) : 1.f;
  // Errors of float32 scores, absolute.  Sigmoid: with t = l log2 e off by 2^-23.4 |t| and one step each of exp2, the sum and
  // the reciprocal, s is off by s (1 - s) (|l| 2^-23.4 + 2^-23) + s 1.5 2^-23 < 2^-22.  Softmax: s (2 |l - top| +
  // terms a lane + 24) 2^-24, of which the sum's terms, |l - top| < 7 on their average, have 18; s |l - top| < 0.4 / total
  // and s <= 1 / total.  With a bias the sum's rounding.
  float err = By == kBySigmoid ? 2.5e-7f : By == kBySoftmax ? (float)(A.run + 26) * 6e-8f / fmaxf(total, 1.f) : 0.f;
  // Keys by the values' own bits (whole), or by v * scale + offset.
  bool whole = !F32 && !Biased;
  float offset = 0.f, scale = 0.f;
  uint32_t gap = 0;
  if constexpr (Biased) {
    err += 6e-8f * (1.f + B.far);
    scale = B.scale, offset = B.offset;
    // Two keys in order may be out of order by this many steps of 512: each score's error, the roundings of offset (of
    // |low| scale) and of the sum, and the cut.
    gap = to_u32(fminf((err + 6e-8f * B.far) * B.step + 6.f, 8e6f));
  } else if constexpr (F32) {
    bits |= (uint32_t)dpp_i32<0xB1>((int)bits);
    bits |= (uint32_t)dpp_i32<0x4E>((int)bits);
    bits |= (uint32_t)dpp_i32<0x141>((int)bits);
    bits |= (uint32_t)dpp_i32<0x140>((int)bits);
    whole = __ballot((bits & 0xFFFFu) != 0) == 0;  // of all four rows
    low = fmaxf(min16(low), ref - 64.f);
    scale = 4294000000.f * __builtin_amdgcn_rcpf(fmaxf(ref - low, 1e-20f));
    offset = 600.f;
    gap = whole ? 0u : 8u;  // l - low, the product and the cut: two steps each, twice
  }
  // A key below this is no expert: -inf, or past the run.  (By the values' own bits: the key of bf16's lowest value, which
  // is an expert like any other; -inf's is the next below, 0x007F0000.)
  const uint32_t none = whole ? 0x00800000u : 512u;

  // ---- keys, sorted; the largest two scores of the lane where groups are ranked ----
  uint32_t key[8];
#pragma unroll
  for (int i = 0; i < 8; i++) key[i] = 0;
  float a = -INFINITY, b = -INFINITY;
  each([&](int p, const RowPiece<F32, 8>& r) {
    // Rows without an infinity or a NaN need not look at each value.
    bool odd;
    if constexpr (F32) {
      uint32_t far = 0;
#pragma unroll
      for (int i = 0; i < 8; i++) far = max(far, f32_abs_bits(r.get(i)));
      bad = bad || far > 0x7F800000u;
      odd = __ballot(far >= 0x7F800000u) != 0;
    } else {
      u16x2_t far = {0, 0};
#pragma unroll
      for (int i = 0; i < 4; i++) far = __builtin_elementwise_max(far, __builtin_bit_cast(u16x2_t, r.w[i] & 0x7FFF7FFFu));
      const uint32_t most = max(far.x, far.y);
      bad = bad || most > 0x7F80u;
      odd = __ballot(most >= 0x7F80u) != 0;
    }
    if (odd) {
#pragma unroll
      for (int i = 0; i < 8; i++) bad = bad || r.get(i) == INFINITY;
    }
    float c[8];
    if (By != kByLogit && (Biased || A.groups > 1)) {
#pragma unroll
      for (int i = 0; i < 8; i++)
        c[i] = By == kBySoftmax ? __builtin_amdgcn_exp2f((r.get(i) - ref) * kLog2) * inv
                                : __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(r.get(i) * -kLog2));
      if constexpr (Biased) {
        // -inf: excluded, or past the run.
        const float4 b0 = s_bias[(p / 4) * 16 + g], b1 = s_bias[(p / 4 + 1) * 16 + g];
        c[0] += b0.x, c[1] += b0.y, c[2] += b0.z, c[3] += b0.w;
        c[4] += b1.x, c[5] += b1.y, c[6] += b1.z, c[7] += b1.w;
      }
      if (odd) {
#pragma unroll
        for (int i = 0; i < 8; i++) c[i] = r.get(i) > -INFINITY ? c[i] : -INFINITY;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) c[i] = r.get(i);
    }
    if (A.groups > 1) {
#pragma unroll
      for (int i = 0; i < 8; i++) {
        b = __builtin_amdgcn_fmed3f(a, b, c[i]);
        a = fmaxf(a, c[i]);
      }
    }
    uint32_t k8[8];
    if (!Biased && (!F32 || whole)) {
#pragma unroll
      for (int i = 0; i < 8; i++) {
        // Bits in the order of the values; + 0: no -0.
        const uint32_t u = __float_as_uint(r.get(i) + 0.f);
        k8[i] = ((u ^ ((uint32_t)((int)u >> 31) | 0x80000000u)) & 0xFFFF0000u) | (uint32_t)(31 - i);
      }
    } else if constexpr (Biased) {
#pragma unroll
      for (int i = 0; i < 8; i++) k8[i] = (to_u32(fmaf(c[i], scale, offset)) & kScore) | (uint32_t)(31 - i);
    } else {
      // Logits below `low` are held at it.
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float l = r.get(i);
        k8[i] = ((l > -INFINITY ? to_u32(fmaf(fmaxf(l - low, 0.f), scale, offset)) : 0u) & kScore) | (uint32_t)(31 - i);
      }
    }
    sort8(k8);
    const uint32_t place = ((uint32_t)(15 - g) << 5) - (uint32_t)p;
#pragma unroll
    for (int i = 0; i < 8; i++) k8[i] += place;
    merge8(key, k8);
  });
  bool open = bad || B.exact;  // left to select_exact
  bool full = false, kept = true;
  uint32_t mine = 0, last = 0;
  // ---- groups ----
  if (A.groups > 1) {
    // The largest two of the group's lanes.
    const int base = lane - L.pos;
    float ta = a, tb = b;
    for (int d = 1; d < L.lanes; d++) {
      const int from = base + (L.pos + d < L.lanes ? L.pos + d : L.pos + d - L.lanes);
      const float ga = __shfl(a, from), gb = __shfl(b, from);
      tb = __builtin_amdgcn_fmed3f(ta, tb, ga);
      ta = fmaxf(ta, ga);
      tb = fmaxf(tb, gb);  // gb <= ga <= ta
    }
    const float score = L.group >= A.groups ? -INFINITY : By != kByLogit && A.best == 2 && tb > -INFINITY ? ta + tb : ta;
    int before = 0;
    for (int d = 1; d < A.groups; d++) {
      const int other = L.group + d < A.groups ? L.group + d : L.group + d - A.groups;
      const float v = __shfl(score, lane - g + other * L.lanes);
      before += v > score || (v == score && other < L.group) ? 1 : 0;
    }
    kept = L.group < A.groups && score > -INFINITY && before < A.top_groups;
    if constexpr (By != kByLogit) {
      const float in = min16(kept ? score : INFINITY), out = max16(kept ? -INFINITY : score);
      // Sums of two scores and their own rounding.
      open = open || (out > -INFINITY && !(in - out > 4.f * err + 2.4e-7f * (fabsf(in) + 1.f)));
    }
  }
  // ---- the k largest ----
#pragma unroll
  for (int j = 0; j < 8; j++) key[j] = kept && key[j] >= none ? key[j] : 0u;
  full = A.run > kSelRuns && key[kSelRuns - 1] != 0;
#pragma unroll 1
  for (int i = 0; i < A.k; i++) {
    last = umax16(key[0]);
    const bool won = key[0] == last;
#pragma unroll
    for (int j = 0; j < kSelRuns - 1; j++) key[j] = won ? key[j + 1] : key[j];
    key[kSelRuns - 1] = won ? 0u : key[kSelRuns - 1];
    mine = g == i ? last : mine;
  }
  // A lane whose sorted keys are used up may have had another one before the last chosen.
  open = open || (full && key[0] == 0);
  const uint32_t next = umax16(key[0]);
  const uint32_t after = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)mine, 0x101, 0xF, 0xF, true);  // lane g + 1's
  const bool chosen = row && mine >= none;
  bool edge = row && last >= none && next >= none && (last >> 9) - (next >> 9) < gap;
  const int from_e0 = __shfl(L.e0, (lane & 48) + 15 - (int)(mine >> 5 & 15u));
  int id = chosen ? from_e0 + 31 - (int)(mine & 31u) : -1;
  float lc = id >= 0 ? logit_at<F32>(A.logits, t * A.E + id) : -INFINITY;
  bool close = chosen && g + 1 < A.k && after >= none && (mine >> 9) - (after >> 9) < gap;
  if (__ballot(close || edge)) {
    const int next_e0 = __shfl(L.e0, (lane & 48) + 15 - (int)(next >> 5 & 15u));
    const int next_id = edge ? next_e0 + 31 - (int)(next & 31u) : -1;
    // The largest of what is left after the first one left out.
    const uint32_t head = key[0] == next ? key[1] : key[0], third = umax16(head);
    const bool third_near = edge && ((third >= none && (last >> 9) - (third >> 9) < gap) || (full && head == 0));
    // A chosen one that is near to the first left out.
    const bool near = edge && chosen && (mine >> 9) - (next >> 9) < gap;
    if constexpr (Biased) {
      // Equal logits with equal biases are the same sum and have the same key: the lower index comes first already.  In
      // bf16 beside a bias that is the same for many they are common (65536 tokens of 256 experts, bias 0, by float64 and
      // by this: softmax 119, 45 us, sigmoid 47, 43; 512 in 8 groups, sigmoid 101, 86).
      const float bc = id >= 0 ? A.bias[id] : 0.f;
      const float l1 = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(lc), 0x101, 0xF, 0xF, true));
      const float b1 = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(bc), 0x101, 0xF, 0xF, true));
      close = close && !(lc == l1 && bc == b1);
      // The last place is settled if all that are near to it are one such sum.
      const float ln = edge ? logit_at<F32>(A.logits, t * A.E + next_id) : 0.f, bn = edge ? A.bias[next_id] : 0.f;
      const uint64_t unlike = __ballot(third_near || (near && !(lc == ln && bc == bn)));
      edge = edge && ((unlike >> (lane & 48)) & 0xFFFFu) != 0;
    }
    if (By == kBySoftmax && Biased) {
      open = open || close || edge;  // the softmax's sum is float32
    } else if (__ballot(close || edge)) {
      // Those next to each other, and the last and the first that was not chosen, by what they are compared by.
      int at = id >= 0 ? id : 0x7FFFFFFF, other = edge ? next_id : -1;
      double v = -INFINITY, w = -INFINITY;
#pragma unroll 1
      for (int pass = 0; pass < 2; pass++) {
        const int e = pass == 0 ? other : id;
        w = v;
        v = -INFINITY;
        if (e >= 0) {
          v = (double)logit_at<F32>(A.logits, t * A.E + e);
          if (Biased) v = 1.0 / (1.0 + exp(-v)) + (double)A.bias[e];
        }
      }
      // w: the other's.  One that is better takes the last one's place.  What comes after it must not be near, nor a second
      // one of the chosen: which of the three goes is for float64 to say.
      if (edge && g == A.k - 1 && (w > v || (w == v && other < at))) v = w, at = other;
      open = open || (edge && (third_near || (near && g + 1 < A.k)));
      swap_pairs(v, at, A.k, false);
      swap_pairs(v, at, A.k, true);
      swap_pairs(v, at, A.k, false);
      w = __shfl(v, (lane & 48) + ((g + 1) & 15));
      const int wat = __shfl(at, (lane & 48) + ((g + 1) & 15));
      open = open || (g + 1 < A.k && wat != 0x7FFFFFFF && !(v > w || (v == w && at < wat)));
      const int now = at != 0x7FFFFFFF ? at : -1;
      if (now != id) {
        id = now;
        lc = id >= 0 ? logit_at<F32>(A.logits, t * A.E + id) : -INFINITY;
      }
    }
  }
  // Bit 16 r + ..: row r is left open, and written by select_one.
  const uint64_t todo = __ballot(row && open);
  if (t < t1 && ((todo >> (lane & 48)) & 0xFFFFu) == 0) {
    const float w = row ? select_weight(A, g < A.k ? lc : -INFINITY, top, total) : 0.f;
    if (g < A.k) {
      A.ids[t * A.k + g] = id;
      A.weights[t * A.k + g] = w;
      if (s_count && id >= 0) atomicAdd(&s_count[id], 1);
      if (s_ids) s_ids[t * A.k + g] = id;
    }
  }
  return todo;
}

// One token a wave: rows that the 16-lane form leaves open or has no lanes for (more than 16 groups, or more than 32 experts a
// lane: 486 experts in 3 groups 370 us for 65536 tokens, 480 in 3 groups 73).
template <bool F32>
__device__ __forceinline__ void select_one(const SelectArgs& A, int64_t t, SelectLds& lds, int* s_count, int* s_ids) {
  const int lane = threadIdx.x & 63;
  int id = -1;
  float w = 0.f;
  if (!A.valid || A.valid[t]) {
    float top = -INFINITY, total = 1.f;
    const bool fine = select_exact<F32>(A, t, lds.c, &id);
    if (A.softmax && !A.renorm) {
      for (int e = lane; e < A.E; e += 64) top = fmaxf(top, logit_at<F32>(A.logits, t * A.E + e));
      top = wave_max_f32(top);
      total = 0.f;
      if (top > -INFINITY)
        for (int e = lane; e < A.E; e += 64) total += __expf(logit_at<F32>(A.logits, t * A.E + e) - top);
      total = wave_sum_f32(total);
    }
    w = select_weight(A, id >= 0 ? logit_at<F32>(A.logits, t * A.E + id) : -INFINITY, top, total);
    if (!fine) w = __builtin_nanf("");
  }
  if (lane < A.k) {
    A.ids[t * A.k + lane] = id;
    A.weights[t * A.k + lane] = w;
    if (s_count && id >= 0) atomicAdd(&s_count[id], 1);
    if (s_ids) s_ids[t * A.k + lane] = id;
  }
}

// Tokens [t0, t1) by `waves` waves; s_ids: a copy of the ids in LDS, or null.
template <bool F32, int By>
__device__ __forceinline__ void select_range(const SelectArgs& A, int64_t t0, int64_t t1, int waves, SelectLds* lds,
                                             float* s_bias, int* s_count, int* s_ids) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if constexpr (By == kByOne) {
    for (int64_t t = t0 + wave; t < t1; t += waves) select_one<F32>(A, t, lds[wave], s_count, s_ids);
  } else {
    const BiasRange B = bias_range(A);
    const SelectLane L = select_lane(A);
    // The lanes' biases, four at a time: number j of lane g at (j / 4 * 16 + g) * 4 + j % 4.
    if (By != kByLogit && A.bias) {
      for (int i = threadIdx.x; i < 16 * kSelMaxRun; i += 64 * waves) {
        const int g = i / 4 % 16, j = i / 64 * 4 + i % 4;
        const int group = g / A.lanes, at = (g - group * A.lanes) * A.run + j;
        s_bias[i] = group < A.groups && j < A.run && at < A.per ? A.bias[group * A.per + at] : -INFINITY;
      }
    }
    __syncthreads();
    const float4* s_b = reinterpret_cast<const float4*>(s_bias);
    auto go = [&](auto biased) {
      // Rows that are left open wait for every 16th turn, so that their code's registers are not the loop's.
      const int64_t step = 4 * waves;
      int64_t t = t0 + 4 * wave;
      while (t < t1) {
        const int64_t from = t;
        uint64_t open = 0;  // four bits a turn
        for (int i = 0; i < 16 && t < t1; i++, t += step) {
          const uint64_t todo = select_four<F32, By, biased.value>(A, t, t1, L, B, s_b, s_count, s_ids);
          if (todo) {
#pragma unroll
            for (int r = 0; r < 4; r++) open |= (uint64_t)(((todo >> (16 * r)) & 0xFFFFu) != 0) << (4 * i + r);
          }
        }
        for (; open; open &= open - 1) {
          const int b = __builtin_ctzll(open);
          select_one<F32>(A, from + (b >> 2) * step + (b & 3), lds[wave], s_count, s_ids);
        }
      }
    };
    // One bias for all decides as well: of sums that are equal in float64, and of groups that have one expert left.
    if (By != kByLogit && A.bias) go(std::integral_constant<bool, By != kByLogit>{});
    else go(std::false_type{});
  }
}

// Part b: tokens b * per_part .. ; its counts by expert go to the workspace.
// Bound by the instructions of select_four, some 1400 for 4 tokens of 512 experts in 8 groups, with few waves a SIMD: there are
// no more parts than compute units, and the registers of select_one's rare turns count for all (the 1024-thread forms with
// scores are held to 128 and spill 28 to 40 bytes a lane).  65536 such tokens (bf16, 16 places) 68 to 71 us, 1.1 TB/s; 4096
// tokens of 256 experts fp32 7.3 us.  A wave a token in float64 (kByOne: 32 groups) takes 386 us for the former, rows that are
// all left open 414.
template <bool F32, int By, int NT>
__global__ __launch_bounds__(NT) void k_select(SelectArgs A) {
  __shared__ SelectLds lds[NT / 64];
  __shared__ __attribute__((aligned(16))) float s_bias[kMaxE];
  __shared__ int s_count[kMaxE];
  for (int e = threadIdx.x; e < A.E; e += NT) s_count[e] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * A.per_part, t1 = min((int64_t)A.T, t0 + A.per_part);
  select_range<F32, By>(A, t0, t1, NT / 64, lds, s_bias, A.part_count ? s_count : nullptr, nullptr);
  if (!A.part_count) return;
  __syncthreads();
  for (int e = threadIdx.x; e < A.E; e += NT) A.part_count[(int64_t)blockIdx.x * A.E + e] = s_count[e];
}

// ---- the order by expert ---------------------------------------------------------

constexpr int kSortThreads = 1024;
constexpr int kSmallThreads = 512;  // where tokens are chosen for as well: two waves a SIMD, with the registers that takes

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

// Counts the lanes' ids; equal ones, as requests of many tokens leave them, in one addition instead of one after another
// (4096 ids in 8 runs 7.5 -> 5.0 us, 2085 in 3 5.0 -> 3.9; ids in no order of 8 experts 4.95 -> 5.05, of 256 6.4 -> 6.6).
__device__ __forceinline__ void count_one(int* cnt, int e, int E) {
  const uint64_t active = __ballot(true);
  if (__ballot(e == __builtin_amdgcn_readfirstlane(e)) == active) {
    if ((unsigned)e < (unsigned)E && (threadIdx.x & 63) == __builtin_ctzll(active)) atomicAdd(&cnt[e], __popcll(active));
  } else if ((unsigned)e < (unsigned)E) {
    atomicAdd(&cnt[e], 1);
  }
}

// Assignments [lo, hi) into the order, stably: a wave has a run of them, 64 at a
// time; lanes with the same expert find each other by ballots.  first(e, n): the
// place of the range's first assignment of expert e, of which it has n (called by
// thread e < 512 of the whole workgroup, n = 0 for e >= E).  NT threads.
template <int NT, class First>
__device__ __forceinline__ void sort_range(const int32_t* __restrict__ ids, int64_t lo, int64_t hi, int E,
                                           int32_t* __restrict__ sorted, int (*s_cnt)[kMaxE], First first) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int nbits = E > 1 ? 32 - __clz(E - 1) : 0;
  const uint64_t below = lane == 0 ? 0ull : ~0ull >> (64 - lane);
  for (int i = tid; i < (NT / 64) * kMaxE; i += NT) s_cnt[0][i] = 0;
  __syncthreads();
  const int64_t run = ((hi - lo + (NT / 64) - 1) / (NT / 64) + 63) & ~(int64_t)63;
  const int64_t a0 = min(hi, lo + wave * run), a1 = min(hi, a0 + run);
  for (int64_t a = a0 + lane; a < a1; a += 64) count_one(s_cnt[wave], ids[a], E);
  __syncthreads();
  int n = 0;
  if (tid < E)
    for (int w = 0; w < (NT / 64); w++) n += s_cnt[w][tid];
  int at = first(tid, n);
  if (tid < E) {
    for (int w = 0; w < (NT / 64); w++) {
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

template <int NT>
__device__ __forceinline__ void sort_all(const SortArgs& A, int (*s_cnt)[kMaxE], int* s_wave) {
  sort_range<NT>(A.ids, 0, A.n, A.E, A.sorted, s_cnt, [&](int e, int n) {
    const int off = sort_offsets(n, s_wave);
    if (e < A.E) {
      A.counts[e] = n;
      A.offsets[e] = off;
      if (e == A.E - 1) A.offsets[A.E] = off + n;
    }
    return off;
  });
}

// A handful of assignments, their ids in LDS: thread e counts those of expert e and of lower ones, thread a those that
// come before its own.  No sums over lanes or waves, one way through LDS, but every id is looked at by every thread: of 256
// experts 8 ids take 1.91 us against 2.72, 16 ids 2.24 against 2.72, 24 ids 2.76 against 2.73, 64 ids 4.81 against 2.74.
constexpr int kSortTiny = 16;

__device__ __forceinline__ void sort_tiny(const SortArgs& A, const int* s_ids) {
  const int tid = threadIdx.x, n = (int)A.n;
  if ((tid & ~63) >= max(n, A.E)) return;  // a wave with neither
  const int mine = tid < n ? s_ids[tid] : -1;
  const int4* four = reinterpret_cast<const int4*>(s_ids);
  int lower = 0, same = 0, before = 0;
#pragma unroll 4
  for (int i = 0; i < n; i += 4) {
    const int4 v = four[i >> 2];
    const int e4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int e = i + j < n && (unsigned)e4[j] < (unsigned)A.E ? e4[j] : kMaxE;  // the last: counted nowhere
      lower += e < tid ? 1 : 0;
      same += e == tid ? 1 : 0;
      before += e < mine || (e == mine && i + j < tid) ? 1 : 0;
    }
  }
  if (tid < A.E) {
    A.counts[tid] = same;
    A.offsets[tid] = lower;
    if (tid == A.E - 1) A.offsets[A.E] = lower + same;
  }
  if ((unsigned)mine < (unsigned)A.E) A.sorted[before] = tid;
}

// Few assignments: one workgroup.
__global__ __launch_bounds__(kSortThreads) void k_sort_small(SortArgs A) {
  __shared__ __attribute__((aligned(16))) int s_cnt[kSortThreads / 64][kMaxE];
  __shared__ int s_wave[kMaxE / 64];
  if (A.n <= kSortTiny) {
    if (threadIdx.x < A.n) s_cnt[0][threadIdx.x] = A.ids[threadIdx.x];
    __syncthreads();
    sort_tiny(A, s_cnt[0]);
    return;
  }
  sort_all<kSortThreads>(A, s_cnt, s_wave);
}

// Few tokens: the choice and the order in one workgroup, bound by its chain of dependent steps (1 token of 256 experts with
// groups 7.4 us, a launch with nothing to do 1.7).
template <bool F32, int By>
__global__ __launch_bounds__(kSmallThreads) void k_select_small(SelectArgs A, SortArgs S) {
  __shared__ SelectLds lds[kSmallThreads / 64];
  __shared__ __attribute__((aligned(16))) float s_bias[kMaxE];
  __shared__ __attribute__((aligned(16))) int s_ids[kSortTiny];
  const bool tiny = S.n <= kSortTiny;
  select_range<F32, By>(A, 0, A.T, kSmallThreads / 64, lds, s_bias, nullptr, tiny ? s_ids : nullptr);
  __syncthreads();
  if (tiny) {
    sort_tiny(S, s_ids);
    return;
  }
  int(*s_cnt)[kMaxE] = reinterpret_cast<int(*)[kMaxE]>(lds);
  static_assert(sizeof(lds) >= sizeof(int) * kSmallThreads / 64 * kMaxE, "the counters take the scores' place");
  __shared__ int s_wave[kMaxE / 64];
  sort_all<kSmallThreads>(S, s_cnt, s_wave);
}

// Counts of a part's assignments.
__global__ __launch_bounds__(kSortThreads) void k_sort_count(SortArgs A) {
  __shared__ int s_count[kMaxE];
  for (int e = threadIdx.x; e < A.E; e += kSortThreads) s_count[e] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * A.per_part, hi = min((int64_t)A.n, lo + A.per_part);
  for (int64_t a = lo + threadIdx.x; a < hi; a += kSortThreads) count_one(s_count, A.ids[a], A.E);
  __syncthreads();
  for (int e = threadIdx.x; e < A.E; e += kSortThreads) A.part_count[(int64_t)blockIdx.x * A.E + e] = s_count[e];
}

// Counts by part to the parts' prefix sums, in place, and to the experts' totals: 16 experts a workgroup, a wave each (2.6 to
// 4.9 us, a launch and one dependent step after another).
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

// 65536 tokens' 2^20 ids 9.4 us: each workgroup goes twice through its 4096 ids, the lanes with equal ids found by ballots.
__global__ __launch_bounds__(kSortThreads) void k_sort_place(SortArgs A) {
  __shared__ int s_cnt[kSortThreads / 64][kMaxE];
  __shared__ int s_wave[kMaxE / 64];
  const int64_t lo = (int64_t)blockIdx.x * A.per_part, hi = min((int64_t)A.n, lo + A.per_part);
  const int e = threadIdx.x;
  const int total = e < A.E ? A.counts[e] : 0;
  const int before = e < A.E ? A.part_count[(int64_t)blockIdx.x * A.E + e] : 0;
  sort_range<kSortThreads>(A.ids, lo, hi, A.E, A.sorted, s_cnt, [&](int, int) {
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
// Bound by the bytes written and read: 65536 tokens of 512 experts bf16 29.5 us (5.9 TB/s), 4096 of 256 fp32 3.8 us.
template <bool F32>
__global__ __launch_bounds__(kSelThreads) void k_select_grad(SelectArgs A) {
  constexpr int V = F32 ? 4 : 8, kSize = F32 ? 4 : 2, kPieces = kMaxE / 64 / V;
  __shared__ float s_row[kSelWaves][kMaxE];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  float* row = s_row[wave];
  for (int i = lane; i < kMaxE; i += 64) row[i] = 0.f;
  const bool dense = A.softmax && !A.renorm, in_place = A.base && A.base == A.dlogits;
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
      d = w * (A.renorm ? dw - D / A.scale : dw);  // a scale's reciprocal may be beyond float32
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

// Assignments that one workgroup orders by itself: 4096 in 5.0 us of 8 experts, 6.6 of 256, three launches of a part each
// take 7 at least.
constexpr int64_t kSortSmall = 4096;
// Tokens that one workgroup chooses for before it orders them (256 experts, k = 8, one workgroup or three launches: 32
// tokens 8.3, 12.1 us; 64 tokens 11.8, 12.6; 128 tokens 19.5, 13.6).
constexpr int kSelectSmall = 64;

int sort_parts(int64_t n) {
  if (n <= kSortSmall) return 1;
  const int64_t parts = (n + kSortThreads - 1) / kSortThreads;
  return (int)(parts < kSortMaxParts ? parts : kSortMaxParts);
}

int select_parts(int T) {
  if (T <= kSelectSmall) return 1;
  const int parts = (T + kSelPart - 1) / kSelPart;
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

// The kernel for these arguments.
template <class F>
static void by_select(const SelectArgs& A, F f) {
  using std::integral_constant;
  auto by = [&](auto f32) {
    if (A.groups > 16 || A.run > kSelMaxRun) f(f32, integral_constant<int, kByOne>{});
    else if (!A.bias && (A.groups == 1 || A.best == 1)) f(f32, integral_constant<int, kByLogit>{});
    else if (A.softmax) f(f32, integral_constant<int, kBySoftmax>{});
    else f(f32, integral_constant<int, kBySigmoid>{});
  };
  if (A.f32) by(std::true_type{});
  else by(std::false_type{});
}

hipError_t launch_select_forward(SelectArgs A, SortArgs S, bool order, hipStream_t s, const KTime& kt) {
  const int parts = select_parts(A.T);
  A.lanes = A.groups > 16 ? 1 : 16 / A.groups;
  A.run = (A.per + A.lanes - 1) / A.lanes;
  A.per_part = (A.T + (int64_t)parts - 1) / parts;
  A.part_count = order ? S.part_count : nullptr;
  const bool small = parts == 1 && order;
  by_select(A, [&](auto f32, auto by) {
    constexpr bool F = f32.value;
    constexpr int B = by.value;
    if (small) {
      MOE_LAUNCH((k_select_small<F, B>), dim3(1), dim3(kSmallThreads), 0, s, kt.start, kt.stop, A, S);
    } else {
      // 256 threads where the parts have tokens for no more; else 1024, as there are no more parts than compute units (8192
      // tokens 16.5 us against 19.0 with 256 threads, 65536 tokens 39 against 68).
      const bool wide = A.per_part > kSelPart;
      auto* f = wide ? k_select<F, B, 1024> : k_select<F, B, kSelThreads>;
      MOE_LAUNCH(f, dim3(parts), dim3(wide ? 1024 : kSelThreads), 0, s, kt.start, order ? nullptr : kt.stop, A);
    }
  });
  if (small || !order) return hipGetLastError();
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
