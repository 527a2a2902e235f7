// Grouped product of routed rows with microscaled 4-bit expert weights
// (format: mx4.h).  Position i of the expert-sorted order, in expert e's range
// [offsets[e], offsets[e+1]), has
//   z_i = W_e x_src(i),   h_i = silu(z_i[:n/2]) * z_i[n/2:] with SwiGLU,
// and goes to row dst(i) of y, times row_scale[dst(i)].
//
// The weights are the matrix instructions' first operand, so that a lane of
// the result holds one row of x and four consecutive columns of y.
#include <type_traits>

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

// ---------------------------------------------------------------------------
// Many rows an expert, 4-bit x: a workgroup of WN x WT waves takes BN weight
// rows x BT positions; a wave takes FN x FT blocks of 32 x 32 with the
// 32x32x64 scaled instruction.  K goes by in tiles of 256 columns (8 blocks,
// 128 bytes a row) through S stages in LDS, filled by direct loads that stay
// in flight across the barriers.
//
// LDS.  A row's 8 blocks of 16 bytes are stored at slot (block ^ row % 8), so
// that the 16-byte reads of 8 consecutive rows touch all banks; the direct
// loads write consecutive lanes to consecutive addresses, so the exchange is
// made on the memory side, inside the row's 128 bytes.  In step s of a tile a
// lane of half h multiplies block 4 h + s: its four scale bytes of the tile are
// then one dword, of which the instruction picks byte s.
//
// Ragged: k is no multiple of 256, or the scale arrays are not dword aligned.
// The scales are then staged a byte a lane, each in a dword of its own, and
// blocks past the row's end, for which the loads bring the last block again,
// are multiplied as zeros.
// ---------------------------------------------------------------------------
constexpr int kKtBlocks = 8;  // blocks of a K tile

// 16, 4 or 1 bytes a lane from memory to lds + lane * max(size, 4), not waited
// for: the compiler's own form of this load makes it wait for every load in
// flight before the next read of LDS.  m0 holds the LDS address; nothing else
// in these kernels uses it.
template <int Size>
__device__ __forceinline__ void load_to_lds(const void* p, uint32_t lds) {
  static_assert(Size == 16 || Size == 4 || Size == 1, "a direct load's size");
  if constexpr (Size == 16)
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "s"(lds) : "memory");
  else if constexpr (Size == 4)
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(p), "s"(lds) : "memory");
  else
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_ubyte %0, off" ::"v"(p), "s"(lds) : "memory");
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "vmcnt");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Source row, target row and factor of a tile's positions, by all threads of NW waves.
template <int BT, int NW>
__device__ __forceinline__ void mx4_tile_rows(const Mx4ExpertArgs& A, const MxTile& t, int* s_src, int* s_dst, float* s_fac) {
  for (int q = threadIdx.x; q < BT; q += 64 * NW) {
    const bool on = q < t.rows;
    const int dst = on ? mx4_dst(A, t.row + q) : -1;
    s_src[q] = on ? mx4_src(A, t.row + q) : -1;
    s_dst[q] = dst;
    s_fac[q] = A.row_scale && dst >= 0 ? A.row_scale[dst] : 1.f;
  }
  __syncthreads();
}

// Weight row of tile row q from column c0 of y on.  With SwiGLU blocks of 32
// gate rows and of the same 32 up rows take turns.  Rows past the last one read
// the last one, and (in the kernels) positions past the tile, or with no row of
// x, row 0: their results are dropped, or zeroed.
template <bool Swiglu>
__device__ __forceinline__ int64_t mx4_w_row(const Mx4ExpertArgs& A, int e, int n_out, int c0, int q) {
  const int c = Swiglu ? c0 + (q >> 6) * 32 + (q & 31) : c0 + q;
  return (int64_t)e * A.n + (Swiglu && (q & 32) ? n_out : 0) + min(c, n_out - 1);
}

// The K loop over S stages: issue(kt, stage) starts a tile's loads (Loads
// instructions a wave), compute(kt, stage) multiplies it.
template <int S, int Loads, class Issue, class Compute>
__device__ __forceinline__ void mx4_k_loop(int nkt, Issue issue, Compute compute) {
#pragma unroll
  for (int i = 0; i < S - 1; i++)
    if (i < nkt) issue(i, i);
  int stage = 0;
  for (int kt = 0; kt < nkt; kt++) {
    // Stage kt's loads have landed when at most those of the later stages in flight are left.
    const int later = min(S - 2, nkt - 1 - kt);
    if (S >= 5 && later >= 3) wait_loads<Loads * (S >= 5 ? 3 : 0)>();
    else if (S >= 4 && later == 2) wait_loads<Loads * (S >= 4 ? 2 : 0)>();
    else if (S >= 3 && later == 1) wait_loads<Loads * (S >= 3 ? 1 : 0)>();
    else wait_loads<0>();
    // Every wave's loads have landed, and every wave is done reading the stage that is filled next.
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (kt + S - 1 < nkt) issue(kt + S - 1, stage == 0 ? S - 1 : stage - 1);
    compute(kt, stage);
    stage = stage == S - 1 ? 0 : stage + 1;
  }
}

// LDS bytes that a wave of mx4_store_tile needs for C columns.
constexpr int mx4_store_bytes(int C) { return 32 * (C * 4 + 16); }

template <int BN, int BT, int WN, int WT, int S, bool Ragged>
struct MxTileShape {
  static constexpr int kWaves = WN * WT;
  static constexpr int kCodeLoads = (BN + BT) / 8 / kWaves;  // of 8 rows each, a wave
  static constexpr int kScaleRows = Ragged ? 8 : 32;         // rows of a scale load
  static constexpr int kScaleLoads = ((BN + BT) / kScaleRows + kWaves - 1) / kWaves;
  static constexpr int kLoads = kCodeLoads + kScaleLoads;
  static constexpr int kScaleRow = Ragged ? 32 : 8;          // LDS bytes of a row's scales
  static constexpr int kStage = (BN + BT) * (128 + kScaleRow);
  static constexpr int kLds = S * kStage + BT * 12;          // and each position's src, dst, factor
  static_assert((BN + BT) / 8 % kWaves == 0, "code loads divide among the waves");
  static_assert(S >= 2 && kLds <= 160 * 1024, "LDS");
  static_assert(kLoads * (S - 2) < 64, "vmcnt");
  static_assert(mx4_store_bytes(BN / WN) * kWaves <= S * kStage, "the results pass through the stages' LDS");
};

// A wave's FN x FT results to y: C columns from c0 on (with SwiGLU gate and up
// blocks take turns), tile positions from q0 on.  A lane holds one position and
// 4 consecutive columns at a time, so its own stores would be 8 or 16 bytes a
// row; 32 positions at a time go through `buf`, LDS of the wave's own, and out
// as whole rows of C columns.  (Element by element from the registers, the
// stores took 210 of 355 us at 4096 x 8192 x 8192 with bf16 results.)
template <int FN, int FT, bool Swiglu>
__device__ __forceinline__ void mx4_store_tile(const Mx4ExpertArgs& A, const f32x16_t (&acc)[FN][FT], int n_out, int c0,
                                               const int* s_src, const int* s_dst, const float* s_fac, int q0,
                                               uint8_t* buf) {
  constexpr int FO = Swiglu ? FN / 2 : FN, C = FO * 32;
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
  // 16-byte stores where every row of y starts at a multiple of 16 bytes.
  const bool f32 = A.y_type == kMxTypeF32;
  const bool wide = n_out % (f32 ? 4 : 8) == 0 && (reinterpret_cast<uintptr_t>(A.y) & 15) == 0;
#pragma unroll
  for (int j = 0; j < FT; j++) {
    const int q = q0 + j * 32 + r;
    const bool zero = s_src[q] < 0;
    const int dst = s_dst[q];
    const float w = s_fac[q];
#pragma unroll
    for (int i = 0; i < FO; i++) {
      float v[16];  // element 4 g + l is column 8 g + 4 h + l of the block
#pragma unroll
      for (int l = 0; l < 16; l++) {
        const float z = acc[Swiglu ? 2 * i : i][j][l];
        v[l] = zero ? 0.f : (Swiglu ? silu_mul(z, acc[Swiglu ? 2 * i + 1 : i][j][l]) : z) * w;
      }
      if (A.y_type == kMxTypeMx4) {
        uint32_t m = 0;
#pragma unroll
        for (int l = 0; l < 16; l++) m = max(m, f32_abs_bits(v[l]));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        const int s = mx4_scale_byte(m);
        const float inv = mx4_inv_scale(s);
        // Half h has the 16-bit pieces h, 2 + h, 4 + h, 6 + h of the block's 8; it keeps those of its
        // own 8 bytes and gets the others from the other half.
        const uint32_t d0 = mx4_pack8(v, inv), d1 = mx4_pack8(v + 8, inv);
        const uint32_t own = h ? d1 : d0, got = (uint32_t)__shfl_xor((int)(h ? d0 : d1), 32);
        const uint32_t lo = h ? got : own, hi = h ? own : got;
        if (dst >= 0 && c0 + i * 32 < n_out) {
          const int64_t block = (int64_t)dst * (n_out >> 5) + ((c0 + i * 32) >> 5);
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(A.y) + block * kMxBlockBytes + 8 * h) =
              make_uint2((lo & 0xFFFFu) | hi << 16, lo >> 16 | (hi & 0xFFFF0000u));
          if (h == 0) A.y_scales[block] = (uint8_t)s;
        }
      } else if (f32) {
#pragma unroll
        for (int g = 0; g < 4; g++)
          *reinterpret_cast<float4*>(buf + r * (C * 4 + 16) + (i * 32 + 8 * g + 4 * h) * 4) =
              make_float4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
      } else {
#pragma unroll
        for (int g = 0; g < 4; g++)
          *reinterpret_cast<uint2*>(buf + r * (C * 2 + 16) + (i * 32 + 8 * g + 4 * h) * 2) =
              make_uint2(f32_to_bf16_bits(v[4 * g]) | f32_to_bf16_bits(v[4 * g + 1]) << 16,
                         f32_to_bf16_bits(v[4 * g + 2]) | f32_to_bf16_bits(v[4 * g + 3]) << 16);
      }
    }
    if (A.y_type == kMxTypeMx4) continue;
    // The wave's lanes exchange through LDS: writes before reads, and reads before the next round's writes.
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    auto rows = [&](auto size_c) {
      constexpr int size = size_c.value, stride = C * size + 16, per = C * size / 16;  // lanes a row
      if (wide) {
#pragma unroll
        for (int p = 0; p < 32 * per / 64; p++) {
          const int row = p * (64 / per) + lane / per, piece = lane % per, c = c0 + piece * (16 / size);
          const uint4 d = *reinterpret_cast<const uint4*>(buf + row * stride + piece * 16);
          const int to = s_dst[q0 + j * 32 + row];
          if (to >= 0 && c < n_out)
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(A.y) + ((int64_t)to * n_out + c) * size) = d;
        }
      } else {
        for (int e = lane; e < 32 * C; e += 64) {
          const int row = e / C, col = e % C, c = c0 + col, to = s_dst[q0 + j * 32 + row];
          if (to < 0 || c >= n_out) continue;
          const int64_t at = (int64_t)to * n_out + c;
          if constexpr (size == 4)
            static_cast<float*>(A.y)[at] = *reinterpret_cast<const float*>(buf + row * stride + col * 4);
          else
            static_cast<uint16_t*>(A.y)[at] = *reinterpret_cast<const uint16_t*>(buf + row * stride + col * 2);
        }
      }
    };
    if (f32) rows(std::integral_constant<int, 4>{});
    else rows(std::integral_constant<int, 2>{});
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

template <int BN, int BT, int WN, int WT, int S, int Occ, bool Swiglu, bool Ragged>
__global__ __launch_bounds__(64 * WN * WT, Occ) void k_mx4_tile(Mx4ExpertArgs A) {
  using Sh = MxTileShape<BN, BT, WN, WT, S, Ragged>;
  constexpr int FN = BN / 32 / WN, FT = BT / 32 / WT, NW = WN * WT;
  constexpr int kCols = Swiglu ? BN / 2 : BN;  // columns of y
  static_assert(!Swiglu || FN % 2 == 0, "gate and up blocks go in pairs");
  extern __shared__ __attribute__((aligned(16))) uint8_t sm[];
  int* s_src = reinterpret_cast<int*>(sm + S * Sh::kStage);
  int* s_dst = s_src + BT;
  float* s_fac = reinterpret_cast<float*>(s_dst + BT);
  const int n_out = Swiglu ? A.n >> 1 : A.n;
  const int cols = (n_out + kCols - 1) / kCols;
  const int tile = blockIdx.x / cols, c0 = (blockIdx.x - tile * cols) * kCols;
  MxTile t;
  if (!mx4_find_tile<BT>(A.offsets, A.E, A.P, tile, &t)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wn = wave % WN, wt = wave / WN;
  const int r = lane & 31, h = lane >> 5;
  const int nb = A.k >> 5, nkt = (nb + kKtBlocks - 1) / kKtBlocks;

  mx4_tile_rows<BT, NW>(A, t, s_src, s_dst, s_fac);

  auto w_row = [&](int q) -> int64_t { return mx4_w_row<Swiglu>(A, t.e, n_out, c0, q); };
  const uint8_t* code_p[Sh::kCodeLoads];
  const uint8_t* scale_p[Sh::kScaleLoads];
#pragma unroll
  for (int j = 0; j < Sh::kCodeLoads; j++) {
    const int q = (wave + NW * j) * 8 + (lane >> 3);
    code_p[j] = (q < BN ? A.w_codes + w_row(q) * nb * kMxBlockBytes
                        : static_cast<const uint8_t*>(A.x) + (int64_t)max(s_src[q - BN], 0) * nb * kMxBlockBytes);
  }
  // Where the scale loads do not divide among the waves, the last ones are made twice.
  auto scale_load = [&](int j) { return min(wave + NW * j, (BN + BT) / Sh::kScaleRows - 1); };
#pragma unroll
  for (int j = 0; j < Sh::kScaleLoads; j++) {
    const int q = scale_load(j) * Sh::kScaleRows + (Ragged ? lane >> 3 : lane >> 1);
    scale_p[j] = q < BN ? A.w_scales + w_row(q) * nb : A.x_scales + (int64_t)max(s_src[q - BN], 0) * nb;
  }
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)sm);
  auto issue = [&](int kt, int stage) {
    const uint32_t base = lds0 + stage * Sh::kStage;
    int cb = kt * kKtBlocks + ((lane & 7) ^ (lane >> 3));
    int so = kt * kKtBlocks + (Ragged ? lane & 7 : (lane & 1) * 4);
    if (Ragged) cb = min(cb, nb - 1), so = min(so, nb - 1);
#pragma unroll
    for (int j = 0; j < Sh::kCodeLoads; j++)
      load_to_lds<16>(code_p[j] + cb * kMxBlockBytes, base + (wave + NW * j) * 1024);
#pragma unroll
    for (int j = 0; j < Sh::kScaleLoads; j++)
      load_to_lds<Ragged ? 1 : 4>(scale_p[j] + so, base + (BN + BT) * 128 + scale_load(j) * 256);
  };

  f32x16_t acc[FN][FT] = {};
  struct Frags {
    uint4 w[FN], x[FT];
    uint32_t ws[FN], xs[FT];
  };
  auto compute = [&](int kt, int stage) {
    const uint8_t* wl = sm + stage * Sh::kStage + (wn * FN * 32 + r) * 128;
    const uint8_t* xl = sm + stage * Sh::kStage + (BN + wt * FT * 32 + r) * 128;
    const uint8_t* ss = sm + stage * Sh::kStage + (BN + BT) * 128;
    const uint8_t* sw = ss + (wn * FN * 32 + r) * Sh::kScaleRow + h * (Sh::kScaleRow / 2);
    const uint8_t* sx = ss + (BN + wt * FT * 32 + r) * Sh::kScaleRow + h * (Sh::kScaleRow / 2);
    Frags a, b;
    auto load = [&](auto sc, Frags& d) {
      constexpr int s = sc.value;
      const int slot = ((4 * h + s) ^ (r & 7)) * 16;
#pragma unroll
      for (int f = 0; f < FN; f++) d.w[f] = *reinterpret_cast<const uint4*>(wl + f * 32 * 128 + slot);
#pragma unroll
      for (int f = 0; f < FT; f++) d.x[f] = *reinterpret_cast<const uint4*>(xl + f * 32 * 128 + slot);
      // The tile's dword of scales is read in step 0; a ragged one's each step.
      if (Ragged || s == 0) {
#pragma unroll
        for (int f = 0; f < FN; f++)
          d.ws[f] = *reinterpret_cast<const uint32_t*>(sw + f * 32 * Sh::kScaleRow + (Ragged ? s * 4 : 0));
#pragma unroll
        for (int f = 0; f < FT; f++)
          d.xs[f] = *reinterpret_cast<const uint32_t*>(sx + f * 32 * Sh::kScaleRow + (Ragged ? s * 4 : 0));
      }
    };
    auto mul = [&](auto sc, Frags& d, const Frags& sd) {
      constexpr int s = sc.value;
      uint32_t ws[FN], xs[FT];
      const bool in = !Ragged || kt * kKtBlocks + 4 * h + s < nb;
#pragma unroll
      for (int f = 0; f < FN; f++) ws[f] = in ? sd.ws[f] : 0x7Fu;
#pragma unroll
      for (int f = 0; f < FT; f++) {
        xs[f] = in ? sd.xs[f] : 0x7Fu;
        if (!in) d.x[f] = make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < FN; i++)
#pragma unroll
        for (int j = 0; j < FT; j++)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx4_operand(d.w[i]), mx4_operand(d.x[j]), acc[i][j],
                                                                      kE2m1, kE2m1, Ragged ? 0 : s, ws[i], Ragged ? 0 : s,
                                                                      xs[j]);
    };
    // The next step's operands are read while the present one's are multiplied.
    const auto s0 = std::integral_constant<int, 0>{};
    const auto s1 = std::integral_constant<int, 1>{};
    const auto s2 = std::integral_constant<int, 2>{};
    const auto s3 = std::integral_constant<int, 3>{};
    load(s0, a);
    load(s1, b);
    mul(s0, a, a);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (Ragged) {
      load(s2, a);
      mul(s1, b, b);
      __builtin_amdgcn_sched_barrier(0);
      load(s3, b);
      mul(s2, a, a);
      __builtin_amdgcn_sched_barrier(0);
      mul(s3, b, b);
    } else {
      load(s2, a);  // leaves the scales
      mul(s1, b, a);
      __builtin_amdgcn_sched_barrier(0);
      load(s3, b);
      mul(s2, a, a);
      __builtin_amdgcn_sched_barrier(0);
      mul(s3, b, a);
    }
  };

  mx4_k_loop<S, Sh::kLoads>(nkt, issue, compute);
  __syncthreads();  // the stages are free
  mx4_store_tile<FN, FT, Swiglu>(A, acc, n_out, c0 + wn * FN * (Swiglu ? 16 : 32), s_src, s_dst, s_fac, wt * FT * 32,
                                 sm + wave * mx4_store_bytes(kCols / WN));
}

// ---------------------------------------------------------------------------
// Many rows an expert, bf16 x: the same tiles with K tiles of 128 columns (64
// bytes of codes and 256 bytes of x a row).  A wave reads its weight codes from
// LDS, converts them to bf16 (exactly, two a conversion) and multiplies with
// the 32x32x16 instruction; each conversion serves FT instructions.
//
// LDS.  x: 16-byte piece c of a row at slot (c ^ row % 8).  Codes: block b at
// slot (b ^ (row / 4) % 4), 4 blocks a row.  In turn p of a tile a lane of half
// h multiplies block 2 p + h, 8 columns at a time.  Ragged (k no multiple of
// 128, or the scales not dword aligned): as above.
// ---------------------------------------------------------------------------
constexpr int kBtBlocks = 4;  // blocks of a K tile

template <int BN, int BT, int WN, int WT, int S, bool Ragged>
struct MxBfShape {
  static constexpr int kWaves = WN * WT;
  static constexpr int kCodeLoads = BN / 16 / kWaves;  // of 16 rows each, a wave
  static constexpr int kXLoads = BT / 4 / kWaves;      // of 4 rows each
  static constexpr int kScaleRows = Ragged ? 16 : 64;  // rows of a scale load
  static constexpr int kScaleLoads = (BN / kScaleRows + kWaves - 1) / kWaves;
  static constexpr int kLoads = kCodeLoads + kXLoads + kScaleLoads;
  static constexpr int kScaleRow = Ragged ? 16 : 4;
  static constexpr int kStage = BN * (64 + kScaleRow) + BT * 256;
  static constexpr int kLds = S * kStage + BT * 12;
  static_assert(BN / 16 % kWaves == 0 && BT / 4 % kWaves == 0, "loads divide among the waves");
  static_assert(S >= 2 && kLds <= 160 * 1024, "LDS");
  static_assert(kLoads * (S - 2) < 64, "vmcnt");
  static_assert(mx4_store_bytes(BN / WN) * kWaves <= S * kStage, "the results pass through the stages' LDS");
};

template <int BN, int BT, int WN, int WT, int S, int Occ, bool Swiglu, bool Ragged>
__global__ __launch_bounds__(64 * WN * WT, Occ) void k_mx4_tile_bf16(Mx4ExpertArgs A) {
  using Sh = MxBfShape<BN, BT, WN, WT, S, Ragged>;
  constexpr int FN = BN / 32 / WN, FT = BT / 32 / WT, NW = WN * WT;
  constexpr int kCols = Swiglu ? BN / 2 : BN;  // columns of y
  static_assert(!Swiglu || FN % 2 == 0, "gate and up blocks go in pairs");
  extern __shared__ __attribute__((aligned(16))) uint8_t sm[];
  int* s_src = reinterpret_cast<int*>(sm + S * Sh::kStage);
  int* s_dst = s_src + BT;
  float* s_fac = reinterpret_cast<float*>(s_dst + BT);
  const int n_out = Swiglu ? A.n >> 1 : A.n;
  const int cols = (n_out + kCols - 1) / kCols;
  const int tile = blockIdx.x / cols, c0 = (blockIdx.x - tile * cols) * kCols;
  MxTile t;
  if (!mx4_find_tile<BT>(A.offsets, A.E, A.P, tile, &t)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wn = wave % WN, wt = wave / WN;
  const int r = lane & 31, h = lane >> 5;
  const int nb = A.k >> 5, nkt = (nb + kBtBlocks - 1) / kBtBlocks;

  mx4_tile_rows<BT, NW>(A, t, s_src, s_dst, s_fac);

  auto w_row = [&](int q) -> int64_t { return mx4_w_row<Swiglu>(A, t.e, n_out, c0, q); };
  const uint8_t *code_p[Sh::kCodeLoads], *x_p[Sh::kXLoads], *scale_p[Sh::kScaleLoads];
#pragma unroll
  for (int j = 0; j < Sh::kCodeLoads; j++)
    code_p[j] = A.w_codes + w_row((wave + NW * j) * 16 + (lane >> 2)) * nb * kMxBlockBytes;
#pragma unroll
  for (int j = 0; j < Sh::kXLoads; j++)
    x_p[j] = static_cast<const uint8_t*>(A.x) + (int64_t)max(s_src[(wave + NW * j) * 4 + (lane >> 4)], 0) * A.k * 2;
  // Where the scale loads do not divide among the waves, the last ones are made twice.
  auto scale_load = [&](int j) { return min(wave + NW * j, BN / Sh::kScaleRows - 1); };
#pragma unroll
  for (int j = 0; j < Sh::kScaleLoads; j++)
    scale_p[j] = A.w_scales + w_row(scale_load(j) * Sh::kScaleRows + (Ragged ? lane >> 2 : lane)) * nb;
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)sm);
  auto issue = [&](int kt, int stage) {
    const uint32_t base = lds0 + stage * Sh::kStage;
    int cb = kt * kBtBlocks + ((lane & 3) ^ ((lane >> 4) & 3));
    // A row of x is row j of 4 in its load, and row (4 (wave + NW j) + lane / 16) % 8 of the swizzle.
    int so = kt * kBtBlocks + (Ragged ? lane & 3 : 0);
    if (Ragged) cb = min(cb, nb - 1), so = min(so, nb - 1);
#pragma unroll
    for (int j = 0; j < Sh::kCodeLoads; j++)
      load_to_lds<16>(code_p[j] + cb * kMxBlockBytes, base + (wave + NW * j) * 1024);
#pragma unroll
    for (int j = 0; j < Sh::kXLoads; j++) {
      int c = (lane & 15) ^ ((4 * (wave + NW * j) + (lane >> 4)) & 7);
      int xb = kt * kBtBlocks * 4 + c;
      if (Ragged) xb = min(xb, nb * 4 - 1);
      load_to_lds<16>(x_p[j] + xb * 16, base + BN * 64 + (wave + NW * j) * 1024);
    }
#pragma unroll
    for (int j = 0; j < Sh::kScaleLoads; j++)
      load_to_lds<Ragged ? 1 : 4>(scale_p[j] + so, base + BN * 64 + BT * 256 + scale_load(j) * 256);
  };

  f32x16_t acc[FN][FT] = {};
  auto compute = [&](int kt, int stage) {
    const uint8_t* wl = sm + stage * Sh::kStage + (wn * FN * 32 + r) * 64;
    const uint8_t* xl = sm + stage * Sh::kStage + BN * 64 + (wt * FT * 32 + r) * 256;
    const uint8_t* sl = sm + stage * Sh::kStage + BN * 64 + BT * 256 + (wn * FN * 32 + r) * Sh::kScaleRow;
    struct Frags {
      uint4 w[FN], x[FT][4];
      float s[FN];
    } a, b;
    auto load = [&](int p, Frags& d) {
      const int blk = 2 * p + h;
      const bool in = !Ragged || kt * kBtBlocks + blk < nb;
#pragma unroll
      for (int f = 0; f < FN; f++) {
        d.w[f] = *reinterpret_cast<const uint4*>(wl + f * 32 * 64 + ((blk ^ ((r >> 2) & 3)) * 16));
        uint32_t sc = *reinterpret_cast<const uint32_t*>(sl + f * 32 * Sh::kScaleRow + (Ragged ? blk * 4 : 0));
        if (!Ragged) sc >>= 8 * blk;
        d.s[f] = mx4_scale_f32(in ? sc & 0xFFu : 127u);
      }
#pragma unroll
      for (int f = 0; f < FT; f++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
          d.x[f][j] = *reinterpret_cast<const uint4*>(xl + f * 32 * 256 + (((4 * blk + j) ^ (r & 7)) * 16));
          if (!in) d.x[f][j] = make_uint4(0, 0, 0, 0);
        }
    };
    auto mul = [&](const Frags& d) {
#pragma unroll
      for (int j = 0; j < 4; j++) {
        bf16x8_t w[FN];
#pragma unroll
        for (int i = 0; i < FN; i++) {
          const uint32_t c = j == 0 ? d.w[i].x : j == 1 ? d.w[i].y : j == 2 ? d.w[i].z : d.w[i].w;
          w[i] = __builtin_bit_cast(bf16x8_t, mx4_unpack8_bf16(c, d.s[i]));
        }
#pragma unroll
        for (int i = 0; i < FN; i++)
#pragma unroll
          for (int f = 0; f < FT; f++)
            acc[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[i], __builtin_bit_cast(bf16x8_t, d.x[f][j]), acc[i][f], 0, 0, 0);
      }
    };
    load(0, a);
    load(1, b);
    mul(a);
    mul(b);
  };
  mx4_k_loop<S, Sh::kLoads>(nkt, issue, compute);
  __syncthreads();  // the stages are free
  mx4_store_tile<FN, FT, Swiglu>(A, acc, n_out, c0 + wn * FN * (Swiglu ? 16 : 32), s_src, s_dst, s_fac, wt * FT * 32,
                                 sm + wave * mx4_store_bytes(kCols / WN));
}

// Tiles of BT positions that E experts with P positions in all can have.
static int64_t max_tiles(int64_t P, int64_t E, int64_t bt) { return P / bt + (E < P ? E : P); }

template <int BN, int BT, int NW, bool Swiglu>
static hipError_t launch_tile(void (*f)(Mx4ExpertArgs), int lds, std::atomic<uint64_t>& done, const Mx4ExpertArgs& A,
                              hipStream_t s, const KTime& kt) {
  hipError_t e = lds_limit_once(reinterpret_cast<const void*>(f), lds, done);
  if (e != hipSuccess) return e;
  const int64_t n_out = Swiglu ? A.n / 2 : A.n, kc = Swiglu ? BN / 2 : BN;
  const int64_t grid = max_tiles(A.P, A.E, BT) * ((n_out + kc - 1) / kc);
  if (grid > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  MOE_LAUNCH(f, dim3((unsigned)grid), dim3(64 * NW), lds, s, kt.start, kt.stop, A);
  return hipGetLastError();
}

// 4-bit x.
template <int BN, int BT, int WN, int WT, int S, int Occ, bool Ragged>
static hipError_t tile_mx4(const Mx4ExpertArgs& A, hipStream_t s, const KTime& kt) {
  static std::atomic<uint64_t> done[2];
  constexpr int lds = MxTileShape<BN, BT, WN, WT, S, Ragged>::kLds;
  return A.swiglu ? launch_tile<BN, BT, WN * WT, true>(k_mx4_tile<BN, BT, WN, WT, S, Occ, true, Ragged>, lds, done[1], A, s, kt)
                  : launch_tile<BN, BT, WN * WT, false>(k_mx4_tile<BN, BT, WN, WT, S, Occ, false, Ragged>, lds, done[0], A, s, kt);
}

// bf16 x.
template <int BN, int BT, int WN, int WT, int S, int Occ, bool Ragged>
static hipError_t tile_bf16(const Mx4ExpertArgs& A, hipStream_t s, const KTime& kt) {
  static std::atomic<uint64_t> done[2];
  constexpr int lds = MxBfShape<BN, BT, WN, WT, S, Ragged>::kLds;
  return A.swiglu ? launch_tile<BN, BT, WN * WT, true>(k_mx4_tile_bf16<BN, BT, WN, WT, S, Occ, true, Ragged>, lds, done[1], A, s, kt)
                  : launch_tile<BN, BT, WN * WT, false>(k_mx4_tile_bf16<BN, BT, WN, WT, S, Occ, false, Ragged>, lds, done[0], A, s, kt);
}

hipError_t launch_mx4_experts(const Mx4ExpertArgs& A, hipStream_t s, const KTime& kt) {
  const int64_t n_out = A.swiglu ? A.n / 2 : A.n, avg = A.P / A.E;
  const bool dwords = ((reinterpret_cast<uintptr_t>(A.w_scales) | reinterpret_cast<uintptr_t>(A.x_mx4 ? A.x_scales : nullptr)) & 3) == 0;
  if (A.x_mx4 && avg >= 64) {
    if (!dwords || A.k % 256) return tile_mx4<256, 128, 2, 2, 2, 1, true>(A, s, kt);
    if (A.P >= 1024 && A.E == 1) return tile_mx4<256, 256, 2, 4, 2, 2, false>(A, s, kt);
    return tile_mx4<256, 128, 2, 2, 3, 1, false>(A, s, kt);
  }
  if (!A.x_mx4 && avg >= 12) {
    const bool ragged = !dwords || A.k % 128;
    if (avg >= 64) return ragged ? tile_bf16<256, 128, 4, 2, 2, 2, true>(A, s, kt) : tile_bf16<256, 128, 4, 2, 3, 2, false>(A, s, kt);
    return ragged ? tile_bf16<256, 32, 4, 1, 3, 2, true>(A, s, kt) : tile_bf16<256, 32, 4, 1, 3, 2, false>(A, s, kt);
  }
  const int64_t grid = max_tiles(A.P, A.E, 16) * ((n_out + kFewCols - 1) / kFewCols);
  if (grid > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  auto* f = A.x_mx4 ? (A.swiglu ? k_mx4_few<true, true> : k_mx4_few<true, false>)
                    : (A.swiglu ? k_mx4_few<false, true> : k_mx4_few<false, false>);
  MOE_LAUNCH(f, dim3((unsigned)grid), dim3(256), 0, s, kt.start, kt.stop, A);
  return hipGetLastError();
}

}  // namespace moe
