// Grouped product of routed rows with microscaled 4-bit expert weights
// (format: mx4.h).  Position i of the expert-sorted order, in expert e's range
// [offsets[e], offsets[e+1]), has
//   z_i = W_e x_src(i),   h_i = silu(z_i[:n/2]) * z_i[n/2:] with SwiGLU,
// and goes to row dst(i) of y, times row_scale[dst(i)].
//
// The weights are the matrix instructions' first operand, so that a lane of
// the result holds one row of x and four consecutive columns of y.
#include "launch.h"
#include "mx4.h"

namespace moe {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

constexpr int kE2m1 = 4;  // operand type code of the scaled matrix instructions

struct MxTile {
  int e, row, rows;  // expert, first position, positions (at most BT)
};

// Tile number `tile` of the order (expert, BT positions at a time), found by
// every wave from the offsets alone: lane l sums the tiles of E/64 consecutive
// experts, a scan over the lanes gives each its first tile.  Offsets are held
// inside [0, P] and made increasing, so that whatever they are no position
// outside the arrays is reached.
template <int BT>
__device__ __forceinline__ bool mx4_find_tile(const int32_t* __restrict__ offsets, int E, int P, int tile, MxTile* out) {
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) >> 6;
  const int e0 = lane * per;
  int mine = 0;
  for (int j = 0; j < per; j++) {
    if (e0 + j >= E) break;
    const int lo = min(max(offsets[e0 + j], 0), P), hi = min(max(offsets[e0 + j + 1], lo), P);
    mine += (hi - lo + BT - 1) / BT;
  }
  int end = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(end, d);
    if (lane >= d) end += v;
  }
  int first = end - mine;
  const uint64_t hit = __ballot(tile >= first && tile < end);
  if (hit == 0) return false;
  const int owner = __builtin_ctzll(hit);
  int e = 0, row = 0, rows = 0;
  if (lane == owner) {
    for (int j = 0; j < per; j++) {
      if (e0 + j >= E) break;
      const int lo = min(max(offsets[e0 + j], 0), P), hi = min(max(offsets[e0 + j + 1], lo), P);
      const int n = (hi - lo + BT - 1) / BT;
      if (tile < first + n) {
        e = e0 + j;
        row = lo + (tile - first) * BT;
        rows = min(hi - row, BT);
        break;
      }
      first += n;
    }
  }
  out->e = __builtin_amdgcn_readlane(e, owner);
  out->row = __builtin_amdgcn_readlane(row, owner);
  out->rows = __builtin_amdgcn_readlane(rows, owner);
  return true;
}

// Row of x that position i reads, or -1 for none.
__device__ __forceinline__ int mx4_src(const Mx4ExpertArgs& A, int i) {
  int r = i;
  if (A.src_rows) {
    r = A.src_rows[i];
    if (r >= 0 && A.src_div > 1) r /= A.src_div;
  }
  return (unsigned)r < (unsigned)A.x_rows ? r : -1;
}

// Row of y that position i writes, or -1 for none.
__device__ __forceinline__ int mx4_dst(const Mx4ExpertArgs& A, int i) {
  const int r = A.dst_rows ? A.dst_rows[i] : i;
  return (unsigned)r < (unsigned)A.y_rows ? r : -1;
}

__device__ __forceinline__ i32x8_t mx4_operand(uint4 v) {
  return i32x8_t{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

// ---------------------------------------------------------------------------
// Few rows an expert: a workgroup of four waves takes 32 output columns of one
// tile of 16 positions.  The waves split K (chunks of 128 columns in turn) and
// their sums are joined through LDS in a fixed order.  Weights go straight
// from memory to registers, 16 bytes a lane: lane (r, q) holds block q of row
// r of a chunk, which is the operand layout of the 16x16x128 instruction.
// bf16 rows: the block's 32 weights are converted (exactly) to bf16 and go
// through four 16x16x32 instructions; both operands number the columns of the
// block the same way, so their order inside an instruction does not matter.
// ---------------------------------------------------------------------------
constexpr int kFewCols = 32;

template <bool XMx, bool Swiglu>
__global__ __launch_bounds__(256) void k_mx4_few(Mx4ExpertArgs A) {
  constexpr int kFrag = Swiglu ? 4 : 2;  // 16-row weight fragments: columns (, then the up half's)
  __shared__ float red[4][kFrag * 4][64];
  const int n_out = Swiglu ? A.n >> 1 : A.n;
  const int cols = (n_out + kFewCols - 1) / kFewCols;
  const int tile = blockIdx.x / cols, n0 = (blockIdx.x - tile * cols) * kFewCols;
  MxTile t;
  if (!mx4_find_tile<16>(A.offsets, A.E, A.P, tile, &t)) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int r = lane & 15, q = lane >> 4;
  const int nb = A.k >> 5;  // blocks a row

  const int pos = t.row + r;
  const int src = r < t.rows ? mx4_src(A, pos) : -1;
  const uint8_t* wc[kFrag];
  const uint8_t* ws[kFrag];
  bool live[kFrag];
#pragma unroll
  for (int f = 0; f < kFrag; f++) {
    const int c = n0 + (f & 1) * 16 + r;
    live[f] = c < n_out;
    const int64_t row = (int64_t)t.e * A.n + (f >= 2 ? n_out : 0) + (live[f] ? c : 0);
    wc[f] = A.w_codes + row * nb * kMxBlockBytes;
    ws[f] = A.w_scales + row * nb;
  }
  f32x4_t acc[kFrag] = {};
  for (int c = wave; c * 4 < nb; c += 4) {
    const int b = c * 4 + q;
    const bool in = b < nb;
    uint4 w[kFrag];
    uint32_t s[kFrag];
#pragma unroll
    for (int f = 0; f < kFrag; f++) {
      w[f] = make_uint4(0, 0, 0, 0);
      s[f] = 127;
      if (in && live[f]) {
        w[f] = *reinterpret_cast<const uint4*>(wc[f] + b * kMxBlockBytes);
        s[f] = ws[f][b];
      }
    }
    if constexpr (XMx) {
      uint4 x = make_uint4(0, 0, 0, 0);
      uint32_t xs = 127;
      if (in && src >= 0) {
        x = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(A.x) + ((int64_t)src * nb + b) * kMxBlockBytes);
        xs = A.x_scales[(int64_t)src * nb + b];
      }
#pragma unroll
      for (int f = 0; f < kFrag; f++)
        acc[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx4_operand(w[f]), mx4_operand(x), acc[f], kE2m1,
                                                                  kE2m1, 0, s[f], 0, xs);
    } else {
      uint4 x[4] = {};
      if (in && src >= 0) {
        const uint4* xp = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(A.x) + (int64_t)src * A.k + b * 32);
#pragma unroll
        for (int j = 0; j < 4; j++) x[j] = xp[j];
      }
#pragma unroll
      for (int f = 0; f < kFrag; f++) {
        const uint32_t d[4] = {w[f].x, w[f].y, w[f].z, w[f].w};
#pragma unroll
        for (int j = 0; j < 4; j++)
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8_t, mx4_unpack8_bf16(d[j], mx4_scale_f32(s[f]))),
              __builtin_bit_cast(bf16x8_t, x[j]), acc[f], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int f = 0; f < kFrag; f++)
#pragma unroll
    for (int i = 0; i < 4; i++) red[wave][f * 4 + i][lane] = acc[f][i];
  __syncthreads();

  // Wave 0 joins the sums: lane (r, q) has position r, columns 16 f + 4 q + i.
  if (wave != 0) return;
  float z[kFrag * 4];
#pragma unroll
  for (int i = 0; i < kFrag * 4; i++) z[i] = (red[0][i][lane] + red[1][i][lane]) + (red[2][i][lane] + red[3][i][lane]);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = Swiglu ? silu_mul(z[i], z[i + (kFrag - 2) * 4]) : z[i];
  const int dst = r < t.rows ? mx4_dst(A, pos) : -1;
  if (A.row_scale && dst >= 0) {
    const float w = A.row_scale[dst];
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] *= w;
  }
  if (A.y_type == kMxTypeMx4) {
    // The block's 32 columns are 8 in each of the lanes r, r + 16, r + 32, r + 48.
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) m = max(m, f32_abs_bits(v[i]));
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    const int s = mx4_scale_byte(m);
    const uint32_t d = mx4_pack8(v, mx4_inv_scale(s));
    if (dst < 0) return;
    const int64_t block = (int64_t)dst * (n_out >> 5) + (n0 >> 5);
    uint16_t* out = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(A.y) + block * kMxBlockBytes);
    out[q] = (uint16_t)d;
    out[4 + q] = (uint16_t)(d >> 16);
    if (q == 0) A.y_scales[block] = (uint8_t)s;
    return;
  }
  if (dst < 0) return;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int c = n0 + (i >> 2) * 16 + 4 * q + (i & 3);
    if (c >= n_out) continue;
    const int64_t at = (int64_t)dst * n_out + c;
    if (A.y_type == kMxTypeF32)
      static_cast<float*>(A.y)[at] = v[i];
    else
      static_cast<uint16_t*>(A.y)[at] = (uint16_t)f32_to_bf16_bits(v[i]);
  }
}

// Tiles of BT positions that E experts with P positions in all can have.
static int64_t max_tiles(int64_t P, int64_t E, int64_t bt) { return P / bt + (E < P ? E : P); }

hipError_t launch_mx4_experts(const Mx4ExpertArgs& A, hipStream_t s, const KTime& kt) {
  const int64_t n_out = A.swiglu ? A.n / 2 : A.n;
  const int64_t grid = max_tiles(A.P, A.E, 16) * ((n_out + kFewCols - 1) / kFewCols);
  if (grid > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  auto* f = A.x_mx4 ? (A.swiglu ? k_mx4_few<true, true> : k_mx4_few<true, false>)
                    : (A.swiglu ? k_mx4_few<false, true> : k_mx4_few<false, false>);
  MOE_LAUNCH(f, dim3((unsigned)grid), dim3(256), 0, s, kt.start, kt.stop, A);
  return hipGetLastError();
}

}  // namespace moe
