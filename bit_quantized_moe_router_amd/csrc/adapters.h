// Low-rank adapters beside a projection: what their forward and backward
// kernels share.  For position i of adapter a, with x = x[src(i)]:
//   forward   h = A x            y[dst(i)] = base + s B h
//   backward  dh = s B^T dy      dx[r(i)]  = base + A^T dh
//             dA = sum dh x^T    dB        = s sum dy h^T
// Both directions are one product that shrinks a wide row to `rank` numbers and
// one that widens them again, so one kernel takes both (k_adapters_rows): the
// numbers between never leave the workgroup, but for the copy that the weight
// gradients read (k_adapters_sums).
//
// Matrix instructions 16x16x32 in bf16.  Lane (m, q) = (lane % 16, lane / 16)
// holds of either operand row m and the numbers 8 q .. 8 q + 7 of the summed
// dimension, and of the result row m of the second operand and rows 4 q .. 4 q +
// 3 of the first.  Which numbers stand in which place of the summed dimension,
// or which columns are called row m, is free as long as both operands (or the
// store) agree; so operands are read in runs of 16 bytes wherever the summed
// dimension lies in memory, and where it is the strided one a lane reads a run
// of each of its 8 rows and turns the 8 x 8 numbers around in registers.
//
// fp32 numbers enter the bf16 instructions as three parts of 8 bits each, which
// hold all 24; their products are exact and summed in fp32.
#pragma once

#include "launch.h"
#include "vec.h"

namespace moe {

// The parts of an fp32 number: each the leading 8 bits of the significand of
// what is left, cut off, so that the next rest is exact and no part overflows.
// An infinity or NaN is all in its first part.
constexpr int kParts = 3;
__device__ __forceinline__ void split_parts(float v, uint32_t part[kParts]) {
  const bool finite = f32_abs_bits(v) < 0x7F800000u;
#pragma unroll
  for (int p = 0; p < kParts; p++) {
    part[p] = __float_as_uint(v) >> 16;
    v = finite ? v - __uint_as_float(part[p] << 16) : 0.f;
  }
}

__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// Eight rows of F bf16 numbers each (F / 2 words a row; F = 1: one number in the
// low half) to F operands of eight numbers.
template <int F>
__device__ __forceinline__ bf16x8_t turned(const uint32_t (&row)[8][(F + 1) / 2], int f) {
  uint32_t d[4];
#pragma unroll
  for (int p = 0; p < 4; p++) {
    const uint32_t a = row[2 * p][f / 2], b = row[2 * p + 1][f / 2];
    d[p] = f & 1 ? high_halves(a, b) : low_halves(a, b);
  }
  return as_bf16x8(d[0], d[1], d[2], d[3]);
}

__device__ __forceinline__ f32x4_t mfma_bf16(bf16x8_t a, bf16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Row of x for position i, of src_rows' own numbering before the division
// (`raw`, the row of dx), or -1 for none.
__device__ __forceinline__ int adapter_src(const AdapterArgs& A, int i, int* raw) {
  const int r = A.src_rows ? A.src_rows[i] : i;
  const int s = A.src_div > 1 && r >= 0 ? div_by(r, A.src) : r;
  const bool in = (unsigned)s < (unsigned)A.x_rows;
  *raw = in ? r : -1;
  return in ? s : -1;
}
__device__ __forceinline__ int adapter_dst(const AdapterArgs& A, int i) {
  const int r = A.dst_rows ? A.dst_rows[i] : i;
  return (unsigned)r < (unsigned)A.y_rows ? r : -1;
}

// The weight gradients' thin operands, for 32 positions at a time (from a multiple of 32) and every rank (padded): three
// parts of 32 numbers each, so that a lane reads the 8 positions of an operand at once.
constexpr int kThinRank = kParts * 32;

// Eight numbers of a row that has n of them left (Even: all or none), as the
// parts that enter the matrix instructions.
template <bool F32, bool Even>
__device__ __forceinline__ RowPiece<F32, 8> piece8(const void* row, int64_t at, int n) {
  RowPiece<F32, 8> p;
  if constexpr (Even) {
    // A piece past the end is read from the row's first numbers and cleared.
    p.load(static_cast<const char*>(row) + (n > 0 ? at : 0) * (F32 ? 4 : 2), 8);
    if (n <= 0) p.clear();
  } else {
    p.load(static_cast<const char*>(row) + at * (F32 ? 4 : 2), n);
  }
  return p;
}

// ---------------------------------------------------------------------------
// RT x 16 positions of one adapter a workgroup of W waves; NR x 16 ranks (rank padded).
// Shrink: the waves split the summed columns, 32 at a time, and join
// their sums in LDS in a fixed order; the result goes to LDS in bf16 parts.
// Widen: the waves split the output columns, and so do `splits` workgroups of
// the same positions, each of which shrinks for itself.
// Even: n_in, n_out and rank are multiples of 8 (rank of NR in the backward
// direction), so that a run of 8 is in its row or out of it.
//
// Bound in small calls by the chain offsets -> source rows -> x and A -> sum of the
// waves -> B (one row of rank 16, 2048 -> 2048, 7.5 us); in large ones by the bytes,
// but a workgroup first only reads, then mostly writes, and a compute unit holds too
// few of them to overlap the two throughout: 4096 rows of rank 16, 4096 -> 4096,
// 37 us, 3.2 TB/s; 32768 rows of 256 adapters of rank 16, 2048 -> 1024, 80 us forward
// (4.9 TB/s of what it moves, 325 MB read) and 74 backward (4.6 TB/s).  The third part of
// the numbers between costs 0.3 to 0.6 us of these.  Consecutive
// tiles on one XCD, so that an adapter's factors reach fewer caches, won 1 to 2 %.
// ---------------------------------------------------------------------------
template <bool Back, bool YF32, int RT, int NR, int W, bool Even>
__global__ __launch_bounds__(64 * W) void k_adapters_rows(AdapterArgs A, int splits) {
  constexpr int BT = 16 * RT, R = 16 * NR, H = W / 2;
  constexpr bool kWideF32 = Back && YF32;               // the wide rows read are fp32
  constexpr int kU = RT + NR <= 2 ? 8 : RT + NR <= 5 ? 4 : 2;  // steps of 32 columns in flight
  constexpr int kRow = R + 8;                           // numbers between two rows of a part in LDS
  __shared__ float s_sum[H][BT][R + 1];
  __shared__ __attribute__((aligned(16))) uint16_t s_part[kParts][BT][kRow];

  RowTile t;
  const int tile = blockIdx.x / splits, split = blockIdx.x - tile * splits;
  if (!find_row_tile<BT>(A.offsets, A.n, A.P, tile, &t)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int m = lane & 15, q = lane >> 4;
  const int r = A.r, K = A.K, N = A.N;

  int src[RT], raw[RT], dst[RT];
#pragma unroll
  for (int i = 0; i < RT; i++) {
    const int p = i * 16 + m;
    src[i] = raw[i] = dst[i] = -1;
    if (p < t.rows) {
      src[i] = adapter_src(A, t.row + p, &raw[i]);
      dst[i] = adapter_dst(A, t.row + p);
    }
  }

  // ---- shrink ----
  const int wide = Back ? N : K;
  f32x4_t acc[RT][NR] = {};
  const uint16_t* fa = A.a + (int64_t)t.e * r * K;
  const uint16_t* fb = A.b + (int64_t)t.e * N * r;
  for (int k0 = wave * 32 * kU; k0 < wide; k0 += W * 32 * kU) {
    RowPiece<kWideF32, 8> x[kU][RT];
    RowPiece<false, 8> w[kU][Back ? 1 : NR];
    uint32_t turn[kU][Back ? 8 : 1][(NR + 1) / 2];
#pragma unroll
    for (int u = 0; u < kU; u++) {
      const int k = k0 + 32 * u + 8 * q;
#pragma unroll
      for (int i = 0; i < RT; i++) {
        const int row = Back ? dst[i] : src[i];
        x[u][i] = piece8<kWideF32, Even>(Back ? A.dy : A.x, (int64_t)max(row, 0) * wide + k, row < 0 ? 0 : wide - k);
      }
      if constexpr (!Back) {
        // A rank past the last one repeats it and is cleared below.
#pragma unroll
        for (int f = 0; f < NR; f++)
          w[u][f] = piece8<false, Even>(fa, (int64_t)min(f * 16 + m, r - 1) * K + k, K - k);
      } else {
        // Rows k .. k + 7 of B, ranks NR m .. NR m + NR - 1.  Rows and ranks past the end repeat the last ones: the
        // rows meet zeros of dy, the ranks are cleared below.
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const uint16_t* row = fb + (int64_t)min(k + j, N - 1) * r;
          if constexpr (Even && NR > 1) {
            const uint16_t* p = row + min(NR * m, r - NR);
            if constexpr (NR == 2) turn[u][j][0] = load_any<uint32_t>(p);
            if constexpr (NR == 4) {
              const uint2 v = load_any<uint2>(p);
              turn[u][j][0] = v.x, turn[u][j][1] = v.y;
            }
            if constexpr (NR == 8) {
              const uint4 v = load_any<uint4>(p);
              turn[u][j][0] = v.x, turn[u][j][1] = v.y, turn[u][j][2] = v.z, turn[u][j][3] = v.w;
            }
          } else {
#pragma unroll
            for (int f = 0; f < NR; f++) {
              const uint32_t v = row[min(NR * m + f, r - 1)];
              turn[u][j][f / 2] = f & 1 ? turn[u][j][f / 2] | v << 16 : v;
            }
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kU; u++) {
#pragma unroll
      for (int f = 0; f < NR; f++) {
        bf16x8_t wv;
        if constexpr (Back) wv = turned<NR>(turn[u], f);
        else wv = as_bf16x8(w[u][f].w[0], w[u][f].w[1], w[u][f].w[2], w[u][f].w[3]);
#pragma unroll
        for (int i = 0; i < RT; i++) {
          if constexpr (!kWideF32) {
            const auto& p = x[u][i].w;
            acc[i][f] = mfma_bf16(wv, as_bf16x8(p[0], p[1], p[2], p[3]), acc[i][f]);
          } else {
            uint32_t d[kParts][4];
#pragma unroll
            for (int j = 0; j < 8; j++) {
              uint32_t part[kParts];
              split_parts(x[u][i].get(j), part);
#pragma unroll
              for (int p = 0; p < kParts; p++) d[p][j / 2] = j & 1 ? d[p][j / 2] | part[p] << 16 : part[p];
            }
            // Small parts first.
#pragma unroll
            for (int p = kParts - 1; p >= 0; p--)
              acc[i][f] = mfma_bf16(wv, as_bf16x8(d[p][0], d[p][1], d[p][2], d[p][3]), acc[i][f]);
          }
        }
      }
    }
  }
  // Result: position m, rank 16 f + 4 q + j (backward: NR (4 q + j) + f).  The upper half of the waves hands its sums to
  // the lower one, whose places are summed in order.
  auto at = [&](int i, int f, int j) -> float& {
    return s_sum[wave % H][i * 16 + m][Back ? NR * (4 * q + j) + f : 16 * f + 4 * q + j];
  };
  if (wave >= H) {
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
      for (int f = 0; f < NR; f++)
#pragma unroll
        for (int j = 0; j < 4; j++) at(i, f, j) = acc[i][f][j];
  }
  __syncthreads();
  if (wave < H) {
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
      for (int f = 0; f < NR; f++)
#pragma unroll
        for (int j = 0; j < 4; j++) at(i, f, j) += acc[i][f][j];
  }
  __syncthreads();
  const float scale = A.scales ? A.scales[t.e] : 1.f;
  for (int j = threadIdx.x; j < BT * R; j += 64 * W) {
    const int p = j / R, c = j % R;
    float v = s_sum[0][p][c];
#pragma unroll
    for (int w = 1; w < H; w++) v += s_sum[w][p][c];
    if (c >= r) v = 0.f;
    const float sv = scale * v;
    if (!Back && A.h_out && split == 0 && p < t.rows && c < r) A.h_out[(int64_t)(t.row + p) * r + c] = v;  // without the scale
    uint32_t part[kParts];
    split_parts(sv, part);
#pragma unroll
    for (int s = 0; s < kParts; s++) s_part[s][p][c] = (uint16_t)part[s];
    if constexpr (Back) s_sum[0][p][c] = sv;
  }
  __syncthreads();
  if (Back && A.thin && split == 0) {
    // dh and h in the layout of k_adapters_sums' operands.
    for (int j = threadIdx.x; j < BT * R; j += 64 * W) {
      const int p = j % BT, c = j / BT;
      if (p >= t.rows) continue;
      const int64_t pos = t.row + p;
      uint16_t* to = A.thin + ((pos >> 5) * R + c) * kThinRank + (pos & 31);
      uint32_t part[kParts];
      split_parts(s_sum[0][p][c], part);
#pragma unroll
      for (int s = 0; s < kParts; s++) to[32 * s] = (uint16_t)part[s];
      split_parts(c < r ? A.h[pos * r + c] : 0.f, part);
#pragma unroll
      for (int s = 0; s < kParts; s++) to[A.thin_h + 32 * s] = (uint16_t)part[s];
    }
  }

  // ---- widen ----
  // The operands of the numbers between: with one chunk of 32 ranks or more, a part an instruction; with 16 ranks
  // the halves of an instruction hold two parts.
  constexpr int kChunks = NR == 1 ? 1 : NR / 2, kOps = NR == 1 ? (kParts + 1) / 2 : kParts;
  auto between = [&](int i, int ch, int s) {
    const int part = NR == 1 ? 2 * s + (q >> 1) : s, c = NR == 1 ? 8 * (q & 1) : 32 * ch + 8 * q;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (NR > 1 || part < kParts) v = *reinterpret_cast<const uint4*>(&s_part[NR == 1 ? min(part, kParts - 1) : part][i * 16 + m][c]);
    return __builtin_bit_cast(bf16x8_t, v);
  };
  if constexpr (!Back) {
    // Four fragments of 16 columns: row 4 a + b of fragment f is column 32 (f / 2) + 8 a + 4 (f % 2) + b, so that a lane
    // has runs of 8 columns of its position and four lanes 64 bytes.
    const int groups = (N + 63) >> 6;
    for (int g = split * W + wave; g < groups; g += W * splits) {
      const int n0 = g * 64;
      RowPiece<YF32, 8> base[RT][2];
      if (A.base) {
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
          for (int u = 0; u < 2; u++) {
            const int c = n0 + 32 * u + 8 * q;
            base[i][u].clear();
            if (dst[i] >= 0 && c < N)
              base[i][u].load(static_cast<const char*>(A.base) + ((int64_t)dst[i] * N + c) * (YF32 ? 4 : 2), Even ? 8 : N - c);
          }
      }
      f32x4_t o[RT][4] = {};
#pragma unroll
      for (int ch = 0; ch < kChunks; ch++) {
        const int c = NR == 1 ? 8 * (q & 1) : 32 * ch + 8 * q;
        bf16x8_t w[4];
#pragma unroll
        for (int f = 0; f < 4; f++) {
          const int n = min(n0 + 32 * (f >> 1) + 8 * (m >> 2) + 4 * (f & 1) + (m & 3), N - 1);
          const auto v = piece8<false, Even>(fb, (int64_t)n * r + c, r - c);
          w[f] = as_bf16x8(v.w[0], v.w[1], v.w[2], v.w[3]);
        }
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
          for (int s = kOps - 1; s >= 0; s--) {
            const bf16x8_t hv = between(i, ch, s);
#pragma unroll
            for (int f = 0; f < 4; f++) o[i][f] = mfma_bf16(w[f], hv, o[i][f]);
          }
      }
#pragma unroll
      for (int i = 0; i < RT; i++) {
        if (dst[i] < 0) continue;
#pragma unroll
        for (int u = 0; u < 2; u++) {
          const int c = n0 + 32 * u + 8 * q, n = N - c;
          if (n <= 0) continue;
          const int64_t at = ((int64_t)dst[i] * N + c) * (YF32 ? 4 : 2);
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; j++) {
            v[j] = o[i][2 * u + j / 4][j % 4];
            if (A.base) v[j] += base[i][u].get(j);
          }
          RowPiece<YF32, 8> p;
          p.set(v);
          p.store(static_cast<char*>(A.y) + at, Even ? 8 : n);
        }
      }
    }
  } else {
    if (!A.dx) return;
    // Eight fragments from rows of 8 columns turned around: row 4 a + b of fragment f is column 32 b + 8 a + f, so that a
    // lane has runs of 8 columns of its position and four lanes 64 bytes.
    const int run = 8 * (4 * (m & 3) + (m >> 2));
    const int groups = (K + 127) >> 7;
    for (int g = split * W + wave; g < groups; g += W * splits) {
      const int n0 = g * 128;
      RowPiece<false, 8> base[RT][4];
      if (A.base) {
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
          for (int u = 0; u < 4; u++) {
            const int c = n0 + 32 * u + 8 * q;
            base[i][u].clear();
            if (raw[i] >= 0 && c < K)
              base[i][u].load(static_cast<const char*>(A.base) + ((int64_t)raw[i] * K + c) * 2, Even ? 8 : K - c);
          }
      }
      f32x4_t o[RT][8] = {};
#pragma unroll
      for (int ch = 0; ch < kChunks; ch++) {
        uint32_t rows[8][4];
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const int c = min((NR == 1 ? 8 * (q & 1) : 32 * ch + 8 * q) + j, r - 1);
          const auto v = piece8<false, Even>(fa, (int64_t)c * K + n0 + run, K - n0 - run);
#pragma unroll
          for (int i = 0; i < 4; i++) rows[j][i] = v.w[i];
        }
        bf16x8_t hv[RT][kOps];
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
          for (int s = 0; s < kOps; s++) hv[i][s] = between(i, ch, s);
#pragma unroll
        for (int f = 0; f < 8; f++) {
          const bf16x8_t w = turned<8>(rows, f);
#pragma unroll
          for (int i = 0; i < RT; i++)
#pragma unroll
            for (int s = kOps - 1; s >= 0; s--) o[i][f] = mfma_bf16(w, hv[i][s], o[i][f]);
        }
      }
#pragma unroll
      for (int i = 0; i < RT; i++) {
        if (raw[i] < 0) continue;
#pragma unroll
        for (int u = 0; u < 4; u++) {
          const int c = n0 + 32 * u + 8 * q, n = K - c;
          if (n <= 0) continue;
          const int64_t at = ((int64_t)raw[i] * K + c) * 2;
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; j++) {
            v[j] = o[i][j][u];
            if (A.base) v[j] += base[i][u].get(j);
          }
          RowPiece<false, 8> p;
          p.set(v);
          p.store(static_cast<char*>(A.dx) + at, Even ? 8 : n);
        }
      }
    }
  }
}

// Sixteenths of the rank, rounded up to what the kernels are made for.
inline int adapter_frags(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8; }

template <bool Back, bool YF32, int RT, int NR, int W, bool Even>
hipError_t adapters_rows(const AdapterArgs& A, int cus, hipStream_t s, hipEvent_t ev0, hipEvent_t ev1) {
  constexpr int BT = 16 * RT;
  const int64_t tiles = ((int64_t)A.P + BT - 1) / BT + (A.n < A.P ? A.n : A.P);
  const int groups = Back ? (A.dx ? (A.K + 127) / 128 : 1) : (A.N + 63) / 64;
  int64_t splits = cus / tiles;
  if (splits > (groups + W - 1) / W) splits = (groups + W - 1) / W;
  if (splits < 1) splits = 1;
  MOE_LAUNCH((k_adapters_rows<Back, YF32, RT, NR, W, Even>), dim3((unsigned)(tiles * splits)), dim3(64 * W), 0, s, ev0, ev1, A,
             (int)splits);
  return hipGetLastError();
}

template <bool Back, bool YF32>
hipError_t adapters_rows_any(const AdapterArgs& A, int cus, hipStream_t s, hipEvent_t ev0, hipEvent_t ev1) {
  const int nr = adapter_frags(A.r);
  const bool even = A.K % 8 == 0 && A.N % 8 == 0 && A.r % 8 == 0;
  // Tiles of 32 positions from a tile of 16 a compute unit on, and from rank 17 on (8 adapters, 2048 -> 2048 bf16, forward,
  // us with 16 / 32 positions: rank 64, 2048 rows 27 / 26, 4096 rows 42 / 31, 32768 rows 212 / 163; rank 32, 2048 rows
  // 19 / 21, 4096 rows 27 / 23, 32768 rows 134 / 121; rank 16, 8192 rows 28 / 33, 32768 rows 106 / 106).  16 waves instead
  // of 8 were no faster (rank 16, 16 rows 8.8 against 7.2, 4096 rows 23.1 against 20.3).
  const bool many = even && (int64_t)A.P >= 16 * cus;
  auto* f = !even ? (nr == 1   ? adapters_rows<Back, YF32, 1, 1, 8, false>
                     : nr == 2 ? adapters_rows<Back, YF32, 1, 2, 8, false>
                     : nr == 4 ? adapters_rows<Back, YF32, 1, 4, 8, false>
                               : adapters_rows<Back, YF32, 1, 8, 8, false>)
            : many  ? (nr == 1   ? adapters_rows<Back, YF32, 1, 1, 8, true>
                       : nr == 2 ? adapters_rows<Back, YF32, 2, 2, 8, true>
                       : nr == 4 ? adapters_rows<Back, YF32, 2, 4, 8, true>
                                 : adapters_rows<Back, YF32, 1, 8, 8, true>)
                    : (nr == 1   ? adapters_rows<Back, YF32, 1, 1, 8, true>
                       : nr == 2 ? adapters_rows<Back, YF32, 1, 2, 8, true>
                       : nr == 4 ? adapters_rows<Back, YF32, 1, 4, 8, true>
                                 : adapters_rows<Back, YF32, 1, 8, 8, true>);
  return f(A, cus, s, ev0, ev1);
}

}  // namespace moe
