// Grouped product of routed rows with microscaled 4-bit expert weights
// (format: mx4.h).  Position i of the expert-sorted order, in expert e's range
// [offsets[e], offsets[e+1]), has
//   z_i = W_e x_src(i),   h_i = silu(z_i[:n/2]) * z_i[n/2:] with SwiGLU,
// and goes to row dst(i) of y, times row_scale[dst(i)].
//
// The weights are the matrix instructions' first operand, so that a lane of
// the result holds one row of x and four consecutive columns of y.
//
// Two kernels: k_mx4_few, for few rows an expert, is bound by the weights'
// bytes; k_mx4_grid goes through tiles of weights and rows in LDS and comes
// to be bound by the matrix instructions.  MxCost chooses.
#include <cmath>
#include <type_traits>

#include "launch.h"
#include "mx4.h"
#include "positions.h"

namespace moe {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

constexpr int kE2m1 = 4;  // operand type code of the scaled matrix instructions

// Row of x for what src_rows says (or the position, where there is none), or -1 for none.
__device__ __forceinline__ int mx4_src_of(const Mx4ExpertArgs& A, int r) {
  if (A.src_rows && r >= 0 && A.src_div > 1) r = div_by(r, A.src);
  return (unsigned)r < (unsigned)A.x_rows ? r : -1;
}
__device__ __forceinline__ int mx4_src(const Mx4ExpertArgs& A, int i) {
  return mx4_src_of(A, A.src_rows ? A.src_rows[i] : i);
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
// Few rows an expert: a wave takes 32 output columns of one tile of 16
// positions.  Weights go straight from memory to registers, 16 bytes a lane:
// lane (r, q) holds block q of row r of a chunk of 128 columns, which is the
// operand layout of the 16x16x128 instruction.  bf16 rows: the block's 32
// weights are converted (exactly) to bf16 and go through four 16x16x32
// instructions; both operands number the columns of the block the same way, so
// their order inside an instruction does not matter.
//
// Split: the four waves of a workgroup share the columns and split K (chunks
// in turn), and their sums are joined through LDS in a fixed order; otherwise
// they take 32 columns each and all of K.  A single token's gate/up has few
// columns: 8 rows, n = 1024 with SwiGLU are 128 workgroups with the split, half
// the number of compute units, and 32 without.  With more tiles the split would
// only pay the way to the tile (offsets, src) four times as often.
//
// Bound by the weights' bytes, in the smallest calls by the chain offsets ->
// src -> x and weights -> sum, and by the compute units that they leave idle:
// 8 rows, n = 1024, K = 2048 bf16 with SwiGLU take 8.6 us (9 MB; 19.6 without
// the split), 64 rows of 58 experts, n = 2048, K = 512 take 12.8 us (33 MB, 2.6
// TB/s; 15.0 with it).  Both with weights that the last-level cache holds; 9.8
// and 14.4 us with copies of them in turn, 512 MB in all.
// ---------------------------------------------------------------------------
constexpr int kFewCols = 32;

template <bool XMx, bool Swiglu, bool Split>
__global__ __launch_bounds__(256) void k_mx4_few(Mx4ExpertArgs A) {
  constexpr int kFrag = Swiglu ? 4 : 2;  // 16-row weight fragments: columns (, then the up half's)
  constexpr int kCols = Split ? kFewCols : 4 * kFewCols, kStep = Split ? 4 : 1;
  __shared__ float red[Split ? 4 : 1][kFrag * 4][64];
  const int n_out = Swiglu ? A.n >> 1 : A.n;
  const int cols = (n_out + kCols - 1) / kCols;
  const int tile = blockIdx.x / cols, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int n0 = (blockIdx.x - tile * cols) * kCols + (Split ? 0 : wave * kFewCols);
  RowTile t;
  if (!find_row_tile<16>(A.offsets, A.E, A.P, tile, &t)) return;
  if (!Split && n0 >= n_out) return;
  const int r = lane & 15, q = lane >> 4;
  const int nb = A.k >> 5;  // blocks a row

  const int pos = t.row + r;
  const int src = r < t.rows ? mx4_src(A, pos) : -1;
  const int dst = r < t.rows ? mx4_dst(A, pos) : -1;
  const float factor = A.row_scale && dst >= 0 ? A.row_scale[dst] : 1.f;
  const uint8_t* wc[kFrag];
  const uint8_t* ws[kFrag];
#pragma unroll
  for (int f = 0; f < kFrag; f++) {
    // A column past the last one reads the last one's weights and is not stored.
    const int c = min(n0 + (f & 1) * 16 + r, n_out - 1);
    const int64_t row = (int64_t)t.e * A.n + (f >= 2 ? n_out : 0) + c;
    wc[f] = A.w_codes + row * nb * kMxBlockBytes;
    ws[f] = A.w_scales + row * nb;
  }
  const int64_t xrow = (int64_t)max(src, 0) * nb;
  f32x4_t acc[kFrag] = {};
  for (int c = Split ? wave : 0; c * 4 < nb; c += kStep) {
    // A block past the row's end is read as the last one and multiplied as zeros.
    const int b = min(c * 4 + q, nb - 1);
    const bool in = c * 4 + q < nb;
    uint4 w[kFrag];
    uint32_t s[kFrag];
#pragma unroll
    for (int f = 0; f < kFrag; f++) {
      w[f] = *reinterpret_cast<const uint4*>(wc[f] + b * kMxBlockBytes);
      s[f] = ws[f][b];
    }
    if constexpr (XMx) {
      uint4 x = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(A.x) + (xrow + b) * kMxBlockBytes);
      uint32_t xs = A.x_scales[xrow + b];
      if (!in) x = make_uint4(0, 0, 0, 0), xs = 127;
#pragma unroll
      for (int f = 0; f < kFrag; f++)
        acc[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx4_operand(w[f]), mx4_operand(x), acc[f], kE2m1,
                                                                  kE2m1, 0, in ? s[f] : 127, 0, xs);
    } else {
      const uint4* xp = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(A.x) + (xrow + b) * 32);
      uint4 x[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        x[j] = xp[j];
        if (!in) x[j] = make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int f = 0; f < kFrag; f++) {
        const uint32_t d[4] = {w[f].x, w[f].y, w[f].z, w[f].w};
#pragma unroll
        for (int j = 0; j < 4; j++)
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8_t, mx4_unpack8_bf16(d[j], mx4_scale_f32(in ? s[f] : 127))),
              __builtin_bit_cast(bf16x8_t, x[j]), acc[f], 0, 0, 0);
      }
    }
  }
  // Lane (r, q) has position r, columns 16 f + 4 q + i.
  float z[kFrag * 4];
  if constexpr (Split) {
#pragma unroll
    for (int f = 0; f < kFrag; f++)
#pragma unroll
      for (int i = 0; i < 4; i++) red[wave][f * 4 + i][lane] = acc[f][i];
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int i = 0; i < kFrag * 4; i++) z[i] = (red[0][i][lane] + red[1][i][lane]) + (red[2][i][lane] + red[3][i][lane]);
  } else {
#pragma unroll
    for (int i = 0; i < kFrag * 4; i++) z[i] = acc[i >> 2][i & 3];
  }
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    v[i] = (Swiglu ? silu_mul(z[i], z[i + (kFrag - 2) * 4]) : z[i]) * factor;
    if (src < 0) v[i] = 0.f;
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
  // Four columns at once where rows of y begin at a multiple of them.
  if (n_out % 4 == 0 && (reinterpret_cast<uintptr_t>(A.y) & 15) == 0) {
#pragma unroll
    for (int g = 0; g < 2; g++) {
      const int c = n0 + g * 16 + 4 * q;
      if (c >= n_out) continue;
      const int64_t at = (int64_t)dst * n_out + c;
      const float* u = v + 4 * g;
      if (A.y_type == kMxTypeF32)
        *reinterpret_cast<float4*>(static_cast<float*>(A.y) + at) = make_float4(u[0], u[1], u[2], u[3]);
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.y) + at) =
            make_uint2(f32_to_bf16_bits(u[0]) | f32_to_bf16_bits(u[1]) << 16, f32_to_bf16_bits(u[2]) | f32_to_bf16_bits(u[3]) << 16);
    }
    return;
  }
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
// LDS.  A row's 8 blocks of 16 bytes are stored at slot (block ^ (row / 2) % 8),
// so that the 16-byte reads of 16 consecutive rows (two share the 256 bytes of
// the banks) touch every bank once; the direct
// loads write consecutive lanes to consecutive addresses, so the exchange is
// made on the memory side, inside the row's 128 bytes.  In step s of a tile a
// lane of half h multiplies block 4 h + s: its four scale bytes of the tile are
// then one dword, of which the instruction picks byte s.
//
// A row's scales are brought 16 blocks, two K tiles, at a time by one 16-byte
// load a row.
//
// Ragged: k is no multiple of 512, or the scale arrays are not 16-byte aligned.
// The scales are then staged a byte a lane, each in a dword of its own, through
// two stages, and blocks past the row's end, for which the loads bring the last
// block again, are multiplied as zeros.  On 162 products that both forms can
// take this one took 1.05 to 1.47 times as long, 1.25 in the middle (bf16 rows:
// 256 x 32 0.92 to 1.46, 1.08; 256 x 128 0.99 to 1.17, 1.06).
//
// The matrix instructions alone reach 6.0 PFLOP/s with random operands (32 x 32
// x 64); 4096 x 8192 x 8192 takes 155 us, 3.5 PFLOP/s, with tiles of 256 x 256
// (in one run 165 us against 196 with 256 x 128).  A workgroup goes through 64 K
// tiles of 2.4 us there, of which 1.4 would be matrix instructions (2048 cycles
// a SIMD); the rest goes to the barrier and to loads and LDS reads beside them.
// ---------------------------------------------------------------------------
// 16, 4 or 1 bytes a lane from memory to lds + lane * max(size, 4), not waited
// for: the compiler's own form of this load makes it wait for every load in
// flight before the next read of LDS.  m0 holds the LDS address.  It is the
// compiler's own (a clobber list does not take it), set by it right before an
// instruction that reads it; in these kernels there is none but these loads.
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

// Weight row of tile row q from column c0 of y on.  With SwiGLU blocks of 32
// gate rows and of the same 32 up rows take turns.  Rows past the last one read
// the last one, and (in the kernels) positions past the tile, or with no row of
// x, row 0: their results are dropped, or zeroed.
template <bool Swiglu>
__device__ __forceinline__ int64_t mx4_w_row(const Mx4ExpertArgs& A, int e, int n_out, int c0, int q) {
  const int c = Swiglu ? c0 + (q >> 6) * 32 + (q & 31) : c0 + q;
  return (int64_t)e * A.n + (Swiglu && (q & 32) ? n_out : 0) + min(c, n_out - 1);
}

// x, of which the compiler knows nothing: what is computed from it inside a
// loop stays there, instead of in registers that the products need.
__device__ __forceinline__ int here(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// The products so far are computed here: without this they sink, being free of
// side effects, below the barriers and into the next step, behind whose loads
// they would have run.
template <int FN, int FT>
__device__ __forceinline__ void computed(f32x16_t (&acc)[FN][FT]) {
#pragma unroll
  for (int i = 0; i < FN; i++)
#pragma unroll
    for (int j = 0; j < FT; j++) asm volatile("" : "+v"(acc[i][j])::"memory");
}

// A tile's positions in LDS: what src_rows and dst_rows say (or nothing, where
// the position itself is meant).
template <int BT>
struct MxRows {
  int src[BT], dst[BT];
};

// A wave's FN x FT results to y: C columns from c0 on (with SwiGLU gate and up
// blocks take turns), tile positions from q0 on of the `rows` from `row` on.  A
// lane holds one position and 4 consecutive columns at a time, so its own
// stores would be 8 or 16 bytes a row; RT positions at a time go through `buf`,
// Store bytes of LDS of the wave's own, and out as whole rows of C columns.
// (Element by element from the registers, the stores took 210 of 355 us at
// 4096 x 8192 x 8192 with bf16 results.)
template <int YT, int FN, int FT, int Store, int BT, bool Swiglu>
__device__ __forceinline__ void mx4_store_tile(const Mx4ExpertArgs& A, f32x16_t (&acc)[FN][FT], int n_out, int c0,
                                               const MxRows<BT>& R, const float* fac, int row, int rows, int q0, uint8_t* buf) {
  constexpr int FO = Swiglu ? FN / 2 : FN, C = FO * 32;
  const int lane = here(threadIdx.x & 63), r = lane & 31, h = lane >> 5;
  auto target = [&](int q) {
    const int d = A.dst_rows ? R.dst[q] : row + q;
    return q < rows && (unsigned)d < (unsigned)A.y_rows ? d : -1;
  };
#pragma unroll
  for (int j = 0; j < FT; j++) {
    const int q = q0 + j * 32 + r;
    const bool zero = mx4_src_of(A, A.src_rows ? R.src[q] : row + q) < 0;
    const float w = A.row_scale ? fac[q] : 1.f;
#pragma unroll
    for (int i = 0; i < FO; i++)
#pragma unroll
      for (int l = 0; l < 16; l++) {
        const float z = acc[Swiglu ? 2 * i : i][j][l];
        acc[i][j][l] = zero ? 0.f : (Swiglu ? silu_mul(z, acc[Swiglu ? 2 * i + 1 : i][j][l]) : z) * w;
      }
  }
  // Element 4 g + l of a block is column 8 g + 4 h + l.
  if constexpr (YT == kMxTypeMx4) {
#pragma unroll
    for (int j = 0; j < FT; j++) {
      const int dst = target(q0 + j * 32 + r);
#pragma unroll
      for (int i = 0; i < FO; i++) {
        float v[16];
        uint32_t m = 0;
#pragma unroll
        for (int l = 0; l < 16; l++) v[l] = acc[i][j][l], m = max(m, f32_abs_bits(v[l]));
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
      }
    }
  } else {
    constexpr int size = YT == kMxTypeF32 ? 4 : 2, stride = C * size + 16;
    constexpr int RT = 32 * stride <= Store ? 32 : 16 * stride <= Store ? 16 : 8;
    static_assert(RT * stride <= Store, "the results pass through a stage");
    constexpr int per = C * size / 16, kPass = RT * per / 64;  // lanes a row; instructions for RT rows
    static_assert(RT * per % 64 == 0, "whole instructions");
    // 16-byte stores where every row of y starts at a multiple of 16 bytes.
    const bool wide = n_out % (16 / size) == 0 && (reinterpret_cast<uintptr_t>(A.y) & 15) == 0;
    const int piece = lane % per, c = c0 + piece * (16 / size);
#pragma unroll
    for (int j = 0; j < FT; j++)
#pragma unroll
      for (int half = 0; half < 32 / RT; half++) {
        const int qr = q0 + j * 32 + half * RT;
        int to[kPass];
#pragma unroll
        for (int p = 0; p < kPass; p++) to[p] = target(qr + p * (64 / per) + lane / per);
        if (RT == 32 || r / RT == half) {  // the lanes whose position passes through buf
#pragma unroll
          for (int i = 0; i < FO; i++)
#pragma unroll
            for (int g = 0; g < 4; g++) {
              const float v0 = acc[i][j][4 * g], v1 = acc[i][j][4 * g + 1], v2 = acc[i][j][4 * g + 2], v3 = acc[i][j][4 * g + 3];
              uint8_t* at = buf + r % RT * stride + (i * 32 + 8 * g + 4 * h) * size;
              if constexpr (size == 4) {
                *reinterpret_cast<float4*>(at) = make_float4(v0, v1, v2, v3);
              } else {
                const bf16x2_t lo = {(__bf16)v0, (__bf16)v1}, hi = {(__bf16)v2, (__bf16)v3};
                *reinterpret_cast<uint2*>(at) = make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
              }
            }
        }
        // The wave's lanes exchange through LDS: writes before reads, and reads before the next round's writes.
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (wide) {
          uint4 d[kPass];
#pragma unroll
          for (int p = 0; p < kPass; p++)
            d[p] = *reinterpret_cast<const uint4*>(buf + (p * (64 / per) + lane / per) * stride + piece * 16);
#pragma unroll
          for (int p = 0; p < kPass; p++)
            if (to[p] >= 0 && c < n_out)
              *reinterpret_cast<uint4*>(static_cast<uint8_t*>(A.y) + ((int64_t)to[p] * n_out + c) * size) = d[p];
        } else {
          for (int e = lane; e < RT * C; e += 64) {
            const int rr = e / C, col = e % C, t = target(qr + rr);
            if (t < 0 || c0 + col >= n_out) continue;
            const int64_t at = (int64_t)t * n_out + c0 + col;
            if constexpr (size == 4)
              static_cast<float*>(A.y)[at] = *reinterpret_cast<const float*>(buf + rr * stride + col * 4);
            else
              static_cast<uint16_t*>(A.y)[at] = *reinterpret_cast<const uint16_t*>(buf + rr * stride + col * 2);
          }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
  }
}

// ---- the operands of a tile, 4-bit x -------------------------------------------
template <int BN_, int BT_, int WN_, int WT_, bool Swiglu_, bool Ragged>
struct MxOp4 {
  static constexpr int BN = BN_, BT = BT_, WN = WN_, WT = WT_;
  static constexpr bool Swiglu = Swiglu_;
  static constexpr int NW = WN * WT, FN = BN / 32 / WN, FT = BT / 32 / WT;
  static constexpr int kBlocks = 8;                          // of a K tile
  static constexpr int kSteps = 4;
  static constexpr int kCodeLoads = (BN + BT) / 8 / NW;      // of 8 rows each, a wave
  static constexpr int kLoads = kCodeLoads;                  // of every K tile, a wave
  static constexpr int kScaleRows = Ragged ? 8 : 64;         // rows of a scale load
  static constexpr int kScaleTiles = Ragged ? 1 : 2;         // K tiles of a scale load: 16 blocks
  static constexpr int kScaleAll = (BN + BT) / kScaleRows, kScaleLoads = (kScaleAll + NW - 1) / NW;
  static constexpr int kScaleRow = Ragged ? 32 : 16;         // LDS bytes of a row's scales
  static constexpr int kStage = (BN + BT) * 128, kPanel = (BN + BT) * kScaleRow;
  static_assert((BN + BT) / 8 % NW == 0 && (BN + BT) % kScaleRows == 0, "code loads divide among the waves");

  const uint8_t* code_p[kCodeLoads];
  const uint8_t* scale_p[kScaleLoads];
  int wave, lane, nb;

  // The last scale loads are not every wave's.
  __device__ __forceinline__ int scale_load(int j) const { return min(wave + NW * j, kScaleAll - 1); }

  __device__ __forceinline__ void set_w(const Mx4ExpertArgs& A, int e, int n_out, int c0) {
    const int lane = here(this->lane);
#pragma unroll
    for (int j = 0; j < kCodeLoads; j++) {
      const int q = (wave + NW * j) * 8 + (lane >> 3);
      if ((wave + NW * j) * 8 < BN) code_p[j] = A.w_codes + mx4_w_row<Swiglu>(A, e, n_out, c0, q) * nb * kMxBlockBytes;
    }
#pragma unroll
    for (int j = 0; j < kScaleLoads; j++) {
      const int q = scale_load(j) * kScaleRows + (Ragged ? lane >> 3 : lane);
      if (scale_load(j) * kScaleRows < BN) scale_p[j] = A.w_scales + mx4_w_row<Swiglu>(A, e, n_out, c0, q) * nb;
    }
  }
  template <class Src>
  __device__ __forceinline__ void set_x(const Mx4ExpertArgs& A, Src src) {
    const int lane = here(this->lane);
#pragma unroll
    for (int j = 0; j < kCodeLoads; j++) {
      const int q = (wave + NW * j) * 8 + (lane >> 3);
      if ((wave + NW * j) * 8 >= BN)
        code_p[j] = static_cast<const uint8_t*>(A.x) + (int64_t)max(src(q - BN), 0) * nb * kMxBlockBytes;
    }
#pragma unroll
    for (int j = 0; j < kScaleLoads; j++) {
      const int q = scale_load(j) * kScaleRows + (Ragged ? lane >> 3 : lane);
      if (scale_load(j) * kScaleRows >= BN) scale_p[j] = A.x_scales + (int64_t)max(src(q - BN), 0) * nb;
    }
  }
  // The scales that begin with K tile kt, to LDS from `panel` on.
  __device__ __forceinline__ void issue_scales(int kt, uint32_t panel) const {
    int so = kt * kBlocks + (Ragged ? lane & 7 : 0);
    if (Ragged) so = min(so, nb - 1);
#pragma unroll
    for (int j = 0; j < kScaleLoads; j++)
      if (wave + NW * j < kScaleAll) load_to_lds<Ragged ? 1 : 16>(scale_p[j] + so, panel + (wave + NW * j) * (Ragged ? 256 : 1024));
  }
  // Part `part` of kSteps of a K tile's loads.
  template <int part>
  __device__ __forceinline__ void issue(int kt, uint32_t base) const {
    // Row 8 (wave + NW j) + lane / 8 has the exchange 4 (wave % 2) + lane / 16, NW being even.
    static_assert(NW % 2 == 0, "the exchange does not depend on j");
    int cb = kt * kBlocks + ((lane & 7) ^ ((wave & 1) * 4 + (lane >> 4)));
    if (Ragged) cb = min(cb, nb - 1);
#pragma unroll
    for (int j = part; j < kCodeLoads; j += kSteps)
      load_to_lds<16>(code_p[j] + cb * kMxBlockBytes, base + (wave + NW * j) * 1024);
  }
  // Step s of a K tile multiplies block 4 h + s.  The scales of a tile are read with its step 0, a ragged
  // tile's with each step.
  struct Frags {
    uint4 w[FN], x[FT];
    uint32_t ws[FN], xs[FT];  // ragged
  };
  struct Scales {
    uint32_t w[FN], x[FT];
  };
  __device__ __forceinline__ void load_scales(int kt, const uint8_t* panel, int wn, int wt, Scales& d) const {
    if constexpr (!Ragged) {
      const int r = lane & 31, h = lane >> 5;
      const uint8_t* s = panel + r * kScaleRow + (kt & 1) * 8 + h * 4;
#pragma unroll
      for (int f = 0; f < FN; f++) d.w[f] = *reinterpret_cast<const uint32_t*>(s + (wn * FN + f) * 32 * kScaleRow);
#pragma unroll
      for (int f = 0; f < FT; f++) d.x[f] = *reinterpret_cast<const uint32_t*>(s + (BN + (wt * FT + f) * 32) * kScaleRow);
    }
  }
  template <int s>
  __device__ __forceinline__ void load_step(const uint8_t* st, const uint8_t* panel, int wn, int wt, Frags& d) const {
    const int r = lane & 31, h = lane >> 5;
    const uint8_t* at = st + r * 128 + ((4 * h + s) ^ ((r >> 1) & 7)) * 16;
    const uint8_t* sc = panel + r * kScaleRow + h * 16 + s * 4;  // ragged
#pragma unroll
    for (int f = 0; f < FN; f++) d.w[f] = *reinterpret_cast<const uint4*>(at + (wn * FN + f) * 32 * 128);
#pragma unroll
    for (int f = 0; f < FT; f++) d.x[f] = *reinterpret_cast<const uint4*>(at + (BN + (wt * FT + f) * 32) * 128);
    if constexpr (Ragged) {
#pragma unroll
      for (int f = 0; f < FN; f++) d.ws[f] = *reinterpret_cast<const uint32_t*>(sc + (wn * FN + f) * 32 * kScaleRow);
#pragma unroll
      for (int f = 0; f < FT; f++) d.xs[f] = *reinterpret_cast<const uint32_t*>(sc + (BN + (wt * FT + f) * 32) * kScaleRow);
    }
  }
  template <int s>
  __device__ __forceinline__ void mul_step(int kt, Frags& d, const Scales& sc, f32x16_t (&acc)[FN][FT]) const {
    const bool in = !Ragged || kt * kBlocks + 4 * (lane >> 5) + s < nb;
    uint32_t ws[FN], xs[FT];
#pragma unroll
    for (int f = 0; f < FN; f++) ws[f] = !Ragged ? sc.w[f] : in ? d.ws[f] : 0x7Fu;
#pragma unroll
    for (int f = 0; f < FT; f++) {
      xs[f] = !Ragged ? sc.x[f] : in ? d.xs[f] : 0x7Fu;
      if (!in) d.x[f] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < FN; i++)
#pragma unroll
      for (int j = 0; j < FT; j++)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx4_operand(d.w[i]), mx4_operand(d.x[j]), acc[i][j],
                                                                    kE2m1, kE2m1, Ragged ? 0 : s, ws[i], Ragged ? 0 : s,
                                                                    xs[j]);
  }
};

// ---- the operands of a tile, bf16 x ----------------------------------------------
// As above with K tiles of 128 columns.  The weights stay codes in LDS and are
// converted, exactly, on their way into the 32x32x16 bf16 instruction: a
// quarter of the LDS and of the reads that converted weights would need, for
// four conversions an operand, which each wave repeats for its own rows.
// 2085 x 4096 x 2048 takes 52 us, 0.67 PFLOP/s (a library's product of bf16
// matrices reaches 1.2 at 8192 x 8192 x 8192), 4096 rows of 256 experts at n =
// 1024, K = 2048, bound by their 285 MB of weights, 64 us, 4.4 TB/s.
// ST: K tiles of a scale load, 4 (16 bytes a row), or 1 (4 bytes) where LDS is short.
template <int BN_, int BT_, int WN_, int WT_, bool Swiglu_, bool Ragged, int ST>
struct MxOp16 {
  static constexpr int BN = BN_, BT = BT_, WN = WN_, WT = WT_;
  static constexpr bool Swiglu = Swiglu_;
  static constexpr int NW = WN * WT, FN = BN / 32 / WN, FT = BT / 32 / WT;
  static constexpr int kBlocks = 4;                   // of a K tile
  static constexpr int kSteps = 2;
  static constexpr int kCodeLoads = BN / 16 / NW;     // of 16 rows each, a wave
  static constexpr int kXLoads = BT / 4 / NW;         // of 4 rows each
  static constexpr int kLoads = kCodeLoads + kXLoads; // of every K tile, a wave
  static constexpr int kScaleRows = Ragged ? 16 : 64; // rows of a scale load
  static constexpr int kScaleTiles = Ragged ? 1 : ST;
  static constexpr int kScaleAll = BN / kScaleRows, kScaleLoads = (kScaleAll + NW - 1) / NW;
  static constexpr int kScaleRow = Ragged ? 16 : 4 * ST;  // LDS bytes of a row's scales
  static constexpr int kStage = BN * 64 + BT * 256, kPanel = BN * kScaleRow;
  static_assert(BN / 16 % NW == 0 && BT / 4 % NW == 0, "loads divide among the waves");

  const uint8_t *code_p[kCodeLoads], *x_p[kXLoads], *scale_p[kScaleLoads];
  int wave, lane, nb;

  __device__ __forceinline__ int scale_load(int j) const { return min(wave + NW * j, kScaleAll - 1); }

  __device__ __forceinline__ void set_w(const Mx4ExpertArgs& A, int e, int n_out, int c0) {
    const int lane = here(this->lane);
#pragma unroll
    for (int j = 0; j < kCodeLoads; j++)
      code_p[j] = A.w_codes + mx4_w_row<Swiglu>(A, e, n_out, c0, (wave + NW * j) * 16 + (lane >> 2)) * nb * kMxBlockBytes;
#pragma unroll
    for (int j = 0; j < kScaleLoads; j++)
      scale_p[j] = A.w_scales + mx4_w_row<Swiglu>(A, e, n_out, c0, scale_load(j) * kScaleRows + (Ragged ? lane >> 2 : lane)) * nb;
  }
  template <class Src>
  __device__ __forceinline__ void set_x(const Mx4ExpertArgs& A, Src src) {
    const int lane = here(this->lane);
#pragma unroll
    for (int j = 0; j < kXLoads; j++)
      x_p[j] = static_cast<const uint8_t*>(A.x) + (int64_t)max(src((wave + NW * j) * 4 + (lane >> 4)), 0) * A.k * 2;
  }
  __device__ __forceinline__ void issue_scales(int kt, uint32_t panel) const {
    int so = kt * kBlocks + (Ragged ? lane & 3 : 0);
    if (Ragged) so = min(so, nb - 1);
#pragma unroll
    for (int j = 0; j < kScaleLoads; j++)
      if (wave + NW * j < kScaleAll) load_to_lds<Ragged ? 1 : 4 * ST>(scale_p[j] + so, panel + (wave + NW * j) * (Ragged ? 256 : 256 * ST));
  }
  template <int part>
  __device__ __forceinline__ void issue(int kt, uint32_t base) const {
    int cb = kt * kBlocks + ((lane & 3) ^ ((lane >> 4) & 3));
    if (Ragged) cb = min(cb, nb - 1);
#pragma unroll
    for (int j = part; j < kCodeLoads; j += kSteps)
      load_to_lds<16>(code_p[j] + cb * kMxBlockBytes, base + (wave + NW * j) * 1024);
#pragma unroll
    for (int j = part; j < kXLoads; j += kSteps) {
      int xb = kt * kBlocks * 4 + ((lane & 15) ^ ((4 * (wave + NW * j) + (lane >> 4)) & 15));
      if (Ragged) xb = min(xb, nb * 4 - 1);
      load_to_lds<16>(x_p[j] + xb * 16, base + BN * 64 + (wave + NW * j) * 1024);
    }
  }
  // Step s of a K tile multiplies block 2 s + h, 8 columns an instruction.
  struct Frags {
    uint4 w[FN], x[FT][4];
    uint32_t s[FN];
  };
  struct Scales {
    uint32_t w[FN];
  };
  __device__ __forceinline__ void load_scales(int kt, const uint8_t* panel, int wn, int, Scales& d) const {
    if constexpr (!Ragged) {
#pragma unroll
      for (int f = 0; f < FN; f++)
        d.w[f] = *reinterpret_cast<const uint32_t*>(panel + ((wn * FN + f) * 32 + (lane & 31)) * kScaleRow + kt % kScaleTiles * 4);
    }
  }
  template <int s>
  __device__ __forceinline__ void load_step(const uint8_t* st, const uint8_t* panel, int wn, int wt, Frags& d) const {
    const int r = lane & 31, h = lane >> 5, blk = 2 * s + h;
    const uint8_t* wl = st + (wn * FN * 32 + r) * 64 + ((blk ^ ((r >> 2) & 3)) * 16);
    const uint8_t* xl = st + BN * 64 + (wt * FT * 32 + r) * 256;
    const uint8_t* sl = panel + (wn * FN * 32 + r) * kScaleRow + blk * 4;  // ragged
#pragma unroll
    for (int f = 0; f < FN; f++) {
      d.w[f] = *reinterpret_cast<const uint4*>(wl + f * 32 * 64);
      if (Ragged) d.s[f] = *reinterpret_cast<const uint32_t*>(sl + f * 32 * kScaleRow);
    }
#pragma unroll
    for (int f = 0; f < FT; f++)
#pragma unroll
      for (int j = 0; j < 4; j++) d.x[f][j] = *reinterpret_cast<const uint4*>(xl + f * 32 * 256 + (((4 * blk + j) ^ (r & 15)) * 16));
  }
  template <int s>
  __device__ __forceinline__ void mul_step(int kt, Frags& d, const Scales& ts, f32x16_t (&acc)[FN][FT]) const {
    const int blk = 2 * s + (lane >> 5);
    const bool in = !Ragged || kt * kBlocks + blk < nb;
    float sc[FN];
#pragma unroll
    for (int f = 0; f < FN; f++) sc[f] = mx4_scale_f32(!in ? 127u : Ragged ? d.s[f] & 0xFFu : (ts.w[f] >> (8 * blk)) & 0xFFu);
#pragma unroll
    for (int f = 0; f < FT; f++)
#pragma unroll
      for (int j = 0; j < 4; j++)
        if (!in) d.x[f][j] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; j++) {
      bf16x8_t w[FN];
#pragma unroll
      for (int i = 0; i < FN; i++) {
        const uint32_t c = j == 0 ? d.w[i].x : j == 1 ? d.w[i].y : j == 2 ? d.w[i].z : d.w[i].w;
        w[i] = __builtin_bit_cast(bf16x8_t, mx4_unpack8_bf16(c, sc[i]));
      }
#pragma unroll
      for (int i = 0; i < FN; i++)
#pragma unroll
        for (int f = 0; f < FT; f++)
          acc[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[i], __builtin_bit_cast(bf16x8_t, d.x[f][j]), acc[i][f], 0, 0, 0);
    }
  }
};

// ---- the kernel ----------------------------------------------------------------------
// A unit is a tile of BT positions of an expert by BN weight rows.  A workgroup
// goes through several, and its loads run through them without a pause: while
// a unit's results are stored, the next unit's first K tiles are on their way,
// and its src, dst and factors are brought by the same direct loads while the
// unit before it is worked on.  (With a workgroup a unit, the chain
// offsets -> src -> x cost about 8 us each time.)
//
// A workgroup has a range of the units in the order (expert, tile, column
// tile), and consecutive ranges share an XCD, whose L2 then keeps an expert's
// weights for its tiles.  4096 tokens' gate/up with 4-bit rows: 90 us, from 116
// with a workgroup a unit.
template <class Op, int S>
struct MxGrid {
  static constexpr int kPanels = S * Op::kStage;                 // where the two scale panels begin,
  // A panel is replaced that many later, when its last K tile is done.
  static constexpr int kPanelSlots = Op::kScaleTiles >= S - 1 ? 2 : S;
  static constexpr int kRows = kPanels + kPanelSlots * Op::kPanel;  // the rows of three units,
  static constexpr int kFac = kRows + 3 * (int)sizeof(MxRows<Op::BT>);  // the factors of two
  static constexpr int kLds = kFac + 2 * Op::BT * 4;
  static_assert(513 * 4 <= Op::kStage, "the offsets, before the first loads");
  static constexpr int kCols = Op::Swiglu ? Op::BN / 2 : Op::BN;
  static constexpr int kStore = Op::kStage / Op::NW;  // a wave's share of a stage
  static_assert(S >= 2 && kLds <= 160 * 1024, "LDS");
  static_assert(Op::kLoads * (S - 2) < 64, "vmcnt");
  static_assert(!Op::Swiglu || Op::FN % 2 == 0, "gate and up blocks go in pairs");
};

template <class Op, int S, int Occ, int YT>
__global__ __launch_bounds__(64 * Op::NW, Occ) void k_mx4_grid(Mx4ExpertArgs A) {
  using G = MxGrid<Op, S>;
  constexpr int BT = Op::BT, NW = Op::NW, kCols = G::kCols;
  extern __shared__ __attribute__((aligned(16))) uint8_t sm[];
  auto* rows3 = reinterpret_cast<MxRows<BT>*>(sm + G::kRows);
  auto* fac2 = reinterpret_cast<float*>(sm + G::kFac);
  int* s_off = reinterpret_cast<int*>(sm);  // before the first loads
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)sm);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int n_out = Op::Swiglu ? A.n >> 1 : A.n, E = A.E;
  const int cols = (n_out + kCols - 1) / kCols;

  for (int i = threadIdx.x; i <= E; i += 64 * NW) s_off[i] = min(max(A.offsets[i], 0), A.P);
  __syncthreads();
  // Tiles: those of E / 64 consecutive experts a lane, summed over the lanes.
  const int per = (E + 63) >> 6, e0 = lane * per;
  auto tiles_of = [&](int e) { return (max(s_off[e + 1] - s_off[e], 0) + BT - 1) / BT; };
  int mine = 0;
  for (int j = 0; j < per; j++)
    if (e0 + j < E) mine += tiles_of(e0 + j);
  int end = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(end, d);
    if (lane >= d) end += v;
  }
  // Rising offsets have no more tiles than that; below 2^28 units, as P <= 2^24 and n <= 2^16.
  const int units = min(__builtin_amdgcn_readlane(end, 63), A.P / BT + min(E, A.P)) * cols;
  // Workgroup b runs on XCD b % 8: consecutive ranges of units to the workgroups of one XCD.
  const int n_wg = gridDim.x, wg = (blockIdx.x & 7) * (n_wg >> 3) + (blockIdx.x >> 3);  // n_wg is a multiple of 8
  auto cut = [&](int x) { return units / n_wg * x + units % n_wg * x / n_wg; };
  const int u0 = cut(wg), u1 = cut(wg + 1), n_unit = u1 - u0;
  if (n_unit <= 0) return;

  // A unit: expert e, its tile's first position, the expert's positions' end, its column tile, its tile's slot.
  struct Unit {
    int e, row, hi, col, slot, turn;
  };
  auto next_tile = [&](Unit w) {
    const auto* off = (const __attribute__((address_space(4))) int*)A.offsets;  // scalar loads
    w.slot = w.slot == 2 ? 0 : w.slot + 1;
    w.turn ^= 1;
    w.row += BT;
    while (w.row >= w.hi && w.e < E - 1) {
      w.e++;
      w.row = min(max(off[w.e], 0), A.P);
      w.hi = min(max(off[w.e + 1], 0), A.P);
    }
    return w;
  };
  Unit in;
  {
    const int t0 = u0 / cols;
    int first = end - mine, e = 0;
    const int owner = __builtin_ctzll(__ballot(t0 >= first && t0 < end));
    if (lane == owner)
      for (e = e0; t0 >= first + tiles_of(e); e++) first += tiles_of(e);
    in.slot = in.turn = 0;
    in.e = __builtin_amdgcn_readlane(e, owner);
    in.row = __builtin_amdgcn_readfirstlane(s_off[in.e]) + (t0 - __builtin_amdgcn_readlane(first, owner)) * BT;
    in.hi = __builtin_amdgcn_readfirstlane(s_off[in.e + 1]);
    in.col = u0 - t0 * cols;
  }
  // The products' tile, the tile after it and the tile after that, as far as known.
  Unit tile0 = in, tile1 = in, tile2 = in;
  int out_col = in.col;

  // Direct loads of what src_rows and dst_rows say about a tile, 64 positions a wave.
  const uint32_t rows_lds = lds0 + G::kRows;
  auto load_rows = [&](const Unit& w) {
    for (int q = wave * 64; q < BT; q += NW * 64) {
      const int64_t at = min(w.row + q + lane, A.P - 1);
      const uint32_t to = rows_lds + w.slot * (int)sizeof(MxRows<BT>) + q * 4;
      if (BT % 64 == 0 || q + lane < BT) {
        if (A.src_rows) load_to_lds<4>(A.src_rows + at, to);
        if (A.dst_rows) load_to_lds<4>(A.dst_rows + at, to + BT * 4);
      }
    }
  };
  // The same for the factors, once the tile's dst are in LDS.
  auto load_factors = [&](const Unit& w) {
    if (!A.row_scale) return;
    for (int q = wave * 64; q < BT; q += NW * 64) {
      if (BT % 64 != 0 && q + lane >= BT) continue;
      const int d = A.dst_rows ? rows3[w.slot].dst[q + lane] : w.row + q + lane;
      load_to_lds<4>(A.row_scale + ((unsigned)d < (unsigned)A.y_rows ? d : 0),
                     lds0 + G::kFac + (w.turn * BT + q) * 4);
    }
  };

  Op op;
  op.wave = wave;
  op.lane = lane;
  op.nb = A.k >> 5;
  const int nkt = (op.nb + Op::kBlocks - 1) / Op::kBlocks;
  const int n_it = n_unit * nkt;  // nkt is at least S - 1 (launch_mx4_experts)
  load_rows(in);
  wait_loads<0>();
  __syncthreads();

  // A K tile's loads: begin() sets the addresses where a unit begins, issue() is called for each part, end_()
  // moves on.  The loads are in the products' tile or the one after it.
  int in_kt = 0, in_stage = 0, in_unit = 0, in_ahead = 0, in_panel = 0;
  bool in_new = true;
  auto begin_unit = [&] {
    if (in_new) {
      in_new = false;
      const MxRows<BT>& R = rows3[in.slot];
      op.set_x(A, [&](int q) { return mx4_src_of(A, A.src_rows ? R.src[q] : min(in.row + q, A.P - 1)); });
      load_factors(in);
      if (in_unit + cols - in.col < n_unit) {  // a unit of the next tile is this workgroup's
        const Unit w = next_tile(in);
        load_rows(w);
        if (in_ahead) tile2 = w;
        else tile1 = w;
      }
    }
    op.set_w(A, in.e, n_out, in.col * kCols);
  };
  auto begin = [&] {
    if (in_kt == 0) begin_unit();
    if (in_kt % Op::kScaleTiles == 0) {
      op.issue_scales(in_kt, lds0 + G::kPanels + in_panel * Op::kPanel);
      in_panel = in_panel == G::kPanelSlots - 1 ? 0 : in_panel + 1;
    }
  };
  auto end_ = [&] {
    in_stage = in_stage == S - 1 ? 0 : in_stage + 1;
    if (++in_kt == nkt) {
      in_kt = 0;
      in_unit++;
      if (++in.col == cols) {
        in = in_ahead ? tile2 : tile1;
        in.col = 0;
        in_new = true;
        in_ahead++;
      }
    }
  };
  auto issue = [&](auto part) { op.template issue<part.value>(in_kt, lds0 + in_stage * Op::kStage); };

  const int wn = wave % Op::WN, wt = wave / Op::WN;
  f32x16_t acc[Op::FN][Op::FT] = {};
  // Operands are read one step ahead, or two where registers allow it: the barrier between K tiles then stands
  // amid the steps, with two steps' products behind it for the next tile's first reads to hide under.
  constexpr bool kTwo = Op::kSteps == 4 && Op::FN * Op::FT <= 4;
  typename Op::Frags frag[kTwo ? 4 : 2];
  typename Op::Scales scale, next_scale;
  auto stage_ptr = [&](int i) { return sm + i * Op::kStage; };
  int panel = 0;
  auto panel_ptr = [&] { return sm + G::kPanels + panel * Op::kPanel; };
  // Waits until at most `later` K tiles' loads are in flight, and for the other waves to have come as far.
  auto arrive = [&](int later) {
    later = min(later, S - 2);  // -1 after the last K tile
    if (S >= 4 && later >= 2) wait_loads<Op::kLoads * (S >= 4 ? 2 : 0)>();
    else if (S >= 3 && later == 1) wait_loads<Op::kLoads * (S >= 3 ? 1 : 0)>();
    else wait_loads<0>();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };
  const auto s0 = std::integral_constant<int, 0>{};
  const auto s1 = std::integral_constant<int, 1>{};
  const auto s2 = std::integral_constant<int, Op::kSteps == 4 ? 2 : 0>{};
  const auto s3 = std::integral_constant<int, Op::kSteps == 4 ? 3 : 0>{};
#pragma unroll 1
  for (int i = 0; i < S - 1 && i < n_it; i++) {
    begin();
    issue(s0);
    issue(s1);
    if constexpr (Op::kSteps == 4) {
      issue(s2);
      issue(s3);
    }
    end_();
  }
  arrive(n_it - 1);
  op.load_scales(0, panel_ptr(), wn, wt, next_scale);
  op.template load_step<0>(stage_ptr(0), panel_ptr(), wn, wt, frag[0]);
  if constexpr (kTwo) op.template load_step<1>(stage_ptr(0), panel_ptr(), wn, wt, frag[1]);
  int stage = 0, kt = 0;
  for (int it = 0; it < n_it; it++) {
    uint8_t* st = stage_ptr(stage);
    stage = stage == S - 1 ? 0 : stage + 1;
    scale = next_scale;
    const bool last = it == n_it - 1, unit = kt == nkt - 1;
    // K tile it + S - 1 goes where K tile it - 1 was, a part with each step, so that the loads queue up behind
    // products and not behind each other.
    const bool more = it + S - 1 < n_it;
    if (more) begin();
    if (S == 2 && more) {  // they have this K tile's time to arrive
      issue(s0);
      issue(s1);
      if constexpr (Op::kSteps == 4) {
        issue(s2);
        issue(s3);
      }
    }
    auto mul = [&](auto sc) {
      __builtin_amdgcn_sched_barrier(0);
      op.template mul_step<sc.value>(kt, frag[kTwo ? sc.value : sc.value & 1], scale, acc);
      computed(acc);
    };
    if constexpr (kTwo) {
      op.template load_step<2>(st, panel_ptr(), wn, wt, frag[2]);
      if (S > 2 && more) issue(s0), issue(s1);
      mul(s0);
      op.template load_step<3>(st, panel_ptr(), wn, wt, frag[3]);
      if (S > 2 && more) issue(s2), issue(s3);
      mul(s1);
    } else {
      auto step = [&](auto sc) {
        constexpr int s = sc.value;
        op.template load_step<s + 1>(st, panel_ptr(), wn, wt, frag[(s + 1) & 1]);
        if (S > 2 && more) issue(sc);
        mul(sc);
      };
      step(s0);
      if constexpr (Op::kSteps == 4) {
        step(s1);
        step(s2);
        if (S > 2 && more) issue(s3);
      } else {
        if (S > 2 && more) issue(s1);
      }
    }
    if (more) end_();
    // The last steps' operands are in registers: when every wave is here, this stage is free and the next
    // one is complete.  Its first operands are read during the last steps; but at a unit's end the results go
    // out through this stage first.
    arrive(n_it - 2 - it);
    if (unit) {
      if constexpr (kTwo) mul(s2);
      mul(std::integral_constant<int, Op::kSteps - 1>{});
      mx4_store_tile<YT, Op::FN, Op::FT, G::kStore, BT, Op::Swiglu>(
          A, acc, n_out, out_col * kCols + wn * (kCols / Op::WN), rows3[tile0.slot], fac2 + tile0.turn * BT, tile0.row,
          min(tile0.hi - tile0.row, BT),
          wt * Op::FT * 32, st + wave * G::kStore);
      if (last) break;
#pragma unroll
      for (int i = 0; i < Op::FN; i++)
#pragma unroll
        for (int j = 0; j < Op::FT; j++) acc[i][j] = f32x16_t{};
      if (++out_col == cols) {
        out_col = 0;
        tile0 = tile1;
        tile1 = tile2;
        in_ahead--;
      }
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }
    const int next_kt = unit ? 0 : kt + 1;
    if (next_kt % Op::kScaleTiles == 0) panel = panel == G::kPanelSlots - 1 ? 0 : panel + 1;
    op.load_scales(next_kt, panel_ptr(), wn, wt, next_scale);
    op.template load_step<0>(stage_ptr(stage), panel_ptr(), wn, wt, frag[0]);
    if constexpr (kTwo) {
      if (!unit) mul(s2);
      op.template load_step<1>(stage_ptr(stage), panel_ptr(), wn, wt, frag[1]);
    }
    if (!unit) mul(std::integral_constant<int, Op::kSteps - 1>{});
    kt = next_kt;
  }
}

// Tiles of BT positions that E experts with P positions in all can have.
static int64_t max_tiles(int64_t P, int64_t E, int64_t bt) { return P / bt + (E < P ? E : P); }

// PerCu workgroups a compute unit, or as many as there may be units.  Tiles of
// 32 positions: twice that many, as their units are few and short: 67 against
// 73 us for 512 tokens' gate/up, where 512 workgroups have 2 or 3 units each.
template <class Op, int S, int PerCu, int YT>
static hipError_t launch_grid_as(const Mx4ExpertArgs& A, int cus, hipStream_t s, const KTime& kt) {
  using G = MxGrid<Op, S>;
  auto* f = k_mx4_grid<Op, S, Op::NW * PerCu / 4, YT>;
  static_assert(G::kLds * PerCu <= 160 * 1024, "LDS");
  static std::atomic<uint64_t> done{0};
  hipError_t e = lds_limit_once(reinterpret_cast<const void*>(f), G::kLds, done);
  if (e != hipSuccess) return e;
  const int64_t n_out = Op::Swiglu ? A.n / 2 : A.n;
  const int64_t units = max_tiles(A.P, A.E, Op::BT) * ((n_out + G::kCols - 1) / G::kCols);
  const int64_t most = ((int64_t)cus * PerCu * (Op::BT == 32 ? 2 : 1) + 7) / 8 * 8, want = (units + 7) / 8 * 8;
  MOE_LAUNCH(f, dim3((unsigned)(want < most ? want : most)), dim3(64 * Op::NW), G::kLds, s, kt.start, kt.stop, A);
  return hipGetLastError();
}

template <class Op, int S, int PerCu>
static hipError_t launch_grid(const Mx4ExpertArgs& A, int cus, hipStream_t s, const KTime& kt) {
  if (A.y_type == kMxTypeF32) return launch_grid_as<Op, S, PerCu, kMxTypeF32>(A, cus, s, kt);
  if (A.y_type == kMxTypeMx4) return launch_grid_as<Op, S, PerCu, kMxTypeMx4>(A, cus, s, kt);
  return launch_grid_as<Op, S, PerCu, kMxTypeBf16>(A, cus, s, kt);
}

// Stages: a unit has to be at least S - 1 K tiles long, so that a tile's rows are in LDS when the loads get to it,
// and are not replaced before its results are out.  With S = 3 k is a multiple of 512: two K tiles, or four, at least.
template <int BN, int BT, int WN, int WT, int S, int PerCu, bool Ragged>
static hipError_t tile_mx4(const Mx4ExpertArgs& A, int cus, hipStream_t s, const KTime& kt) {
  return A.swiglu ? launch_grid<MxOp4<BN, BT, WN, WT, true, Ragged>, S, PerCu>(A, cus, s, kt)
                  : launch_grid<MxOp4<BN, BT, WN, WT, false, Ragged>, S, PerCu>(A, cus, s, kt);
}

template <int BN, int BT, int WN, int WT, int S, int PerCu, bool Ragged>
static hipError_t tile_bf16(const Mx4ExpertArgs& A, int cus, hipStream_t s, const KTime& kt) {
  constexpr int ST = BT == 32 ? 1 : 4;
  return A.swiglu ? launch_grid<MxOp16<BN, BT, WN, WT, true, Ragged, ST>, S, PerCu>(A, cus, s, kt)
                  : launch_grid<MxOp16<BN, BT, WN, WT, false, Ragged, ST>, S, PerCu>(A, cus, s, kt);
}

// The kernels' times in us, from sizes alone, to choose the shortest.  Over 204
// products on 256 compute units (one matrix with 16 to 2048 rows, n = 256 to
// 4096, K = 512 to 8192, and 16 to 256 experts with up to 256 rows each) the
// choice is 1% slower than the best one on average and 25% at most; over 84 with
// K = 768, 1408 and 2880 1% and 40%.  Those are what the factor for a ragged K
// is for (with 1.3 the choice is 3% slower, with 1.7 0.4%); where both forms can
// be taken the ragged one costs less.  The 2 us each for gathered or scattered
// rows and for factors are no fit: over 120 such products, half of them with
// skewed routing, the choice is 4% slower on average and 58% at most; without
// these terms 2% and 43%, but 8 tokens' skewed down product would take 10.0 us
// instead of 8.1.
// Both sides, measured us: 4-bit x, 1024 x 4096 x 2048 few 88, tiles of 128
// positions 17; 256 x 1024 x 2048 few 9, tiles 14; 256 experts with 4 rows each,
// n = 1024, K = 2048: few 77, tiles 58.  bf16 x, 64 experts with 8 rows each,
// n = 1024, K = 2048: few 30, tiles of 32 positions 24, of 128 36; 2048 x 4096 x
// 8192: few 893, 32 positions 203, 128 x 128 156, 256 x 128 132.
struct MxCost {
  double P, E, n, K;
  bool ragged;
  double start;  // a workgroup's way to its first products: offsets, src and dst, factors
  // Tiles of bt positions, for positions spread evenly over the experts.
  double tiles(double bt) const {
    if (E == 1) return std::ceil(P / bt);
    const double active = E * (1.0 - std::exp(-P / E)), avg = P / active;
    return avg <= bt ? active : P / bt + active / 2;
  }
  // 16 x 32 products over 128 columns go by at `rate` a us; one wave's chain takes `chain` us a column.
  double few(double rate, double chain) const {
    return std::fmax(4.0 + K * chain, 2.0 + tiles(16) * std::ceil(n / 32) * std::ceil(K / 128) / rate);
  }
  // A K tile of kt columns takes lo us, or hi where the other compute units are at work too; a unit `own` us more.
  // slots: units under way at one time.
  double grid(double bn, double bt, double kt, double lo, double hi, double own, double slots) const {
    const double units = tiles(bt) * std::ceil(n / bn), full = std::fmin(1.0, units / slots);
    const double tile = (lo + (hi - lo) * full) * (ragged ? 1.5 : 1.0);
    return start + std::ceil(units / slots) * (std::ceil(K / kt) * tile + own);
  }
};

// Columns of few-row tiles go to the waves of a workgroup where that leaves two workgroups a compute unit.
static bool few_by_columns(const Mx4ExpertArgs& A, int cus) {
  const int64_t n_out = A.swiglu ? A.n / 2 : A.n;
  return max_tiles(A.P, A.E, 16) * ((n_out + 4 * kFewCols - 1) / (4 * kFewCols)) >= 2 * cus;
}

MxKernel mx4_experts_kernel(const Mx4ExpertArgs& A, int cus) {
  // Scales by 16 bytes, two or four K tiles at a time, where every row of them allows it.
  const bool odd = A.k % 512 != 0 || ((reinterpret_cast<uintptr_t>(A.w_scales) |
                                       reinterpret_cast<uintptr_t>(A.x_mx4 ? A.x_scales : nullptr)) & 15) != 0;
  const MxCost C{(double)A.P, (double)A.E, (double)A.n, (double)A.k, odd,
                 5.0 + (A.src_rows || A.dst_rows ? 2 : 0) + (A.row_scale ? 2 : 0)};
  if (A.x_mx4) {
    const double few = C.few(1550 / 256.0 * cus, 1.1e-3), mid = C.grid(256, 128, 256, 1.05, 1.4, 1.7, cus);
    const double big = odd ? 1e30 : C.grid(256, 256, 256, 1.7, 2.4, 1.7, cus);
    if (big < few && big < mid) return MxKernel::k4By256;
    if (mid < few) return odd ? MxKernel::k4By128Odd : MxKernel::k4By128;
  } else {
    const double few = C.few(1130 / 256.0 * cus, 1.6e-3), low = C.grid(256, 32, 128, 0.7, 1.6, 1.0, 2 * cus);
    const double mid = odd ? 1e30 : C.grid(128, 128, 128, 0.86, 1.2, 1.0, cus);
    const double big = C.grid(256, 128, 128, 1.4, 2.0, 1.0, cus);
    if (low < few && low <= mid && low <= big) return odd ? MxKernel::k16By32Odd : MxKernel::k16By32;
    if (mid < few && mid <= big) return MxKernel::k16Half;
    if (big < few) return odd ? MxKernel::k16By128Odd : MxKernel::k16By128;
  }
  return few_by_columns(A, cus) ? MxKernel::kFew : MxKernel::kFewSplit;
}

const char* mx4_experts_kernel_name(MxKernel m) {
  switch (m) {
    case MxKernel::kFew: return "few";
    case MxKernel::kFewSplit: return "few split";
    case MxKernel::k4By256: return "4-bit 256x256";
    case MxKernel::k4By128: return "4-bit 256x128";
    case MxKernel::k4By128Odd: return "4-bit 256x128 odd";
    case MxKernel::k16By32: return "bf16 256x32";
    case MxKernel::k16By32Odd: return "bf16 256x32 odd";
    case MxKernel::k16Half: return "bf16 128x128";
    case MxKernel::k16By128: return "bf16 256x128";
    case MxKernel::k16By128Odd: return "bf16 256x128 odd";
  }
  return "";
}

template <bool Split>
static hipError_t launch_few(const Mx4ExpertArgs& A, hipStream_t s, const KTime& kt) {
  constexpr int cols = Split ? kFewCols : 4 * kFewCols;
  const int64_t n_out = A.swiglu ? A.n / 2 : A.n, grid = max_tiles(A.P, A.E, 16) * ((n_out + cols - 1) / cols);
  if (grid > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  auto* f = A.x_mx4 ? (A.swiglu ? k_mx4_few<true, true, Split> : k_mx4_few<true, false, Split>)
                    : (A.swiglu ? k_mx4_few<false, true, Split> : k_mx4_few<false, false, Split>);
  MOE_LAUNCH(f, dim3((unsigned)grid), dim3(256), 0, s, kt.start, kt.stop, A);
  return hipGetLastError();
}

hipError_t launch_mx4_experts(const Mx4ExpertArgs& A, MxKernel m, int cus, hipStream_t s, const KTime& kt) {
  switch (m) {
    case MxKernel::kFew: return launch_few<false>(A, s, kt);
    case MxKernel::kFewSplit: return launch_few<true>(A, s, kt);
    case MxKernel::k4By256: return tile_mx4<256, 256, 2, 4, 2, 1, false>(A, cus, s, kt);
    case MxKernel::k4By128: return tile_mx4<256, 128, 4, 2, 3, 1, false>(A, cus, s, kt);
    case MxKernel::k4By128Odd: return tile_mx4<256, 128, 4, 2, 2, 1, true>(A, cus, s, kt);
    case MxKernel::k16By32: return tile_bf16<256, 32, 4, 1, 3, 2, false>(A, cus, s, kt);
    case MxKernel::k16By32Odd: return tile_bf16<256, 32, 4, 1, 2, 2, true>(A, cus, s, kt);
    case MxKernel::k16Half: return tile_bf16<128, 128, 2, 4, 3, 1, false>(A, cus, s, kt);
    case MxKernel::k16By128: return tile_bf16<256, 128, 4, 2, 3, 1, false>(A, cus, s, kt);
    case MxKernel::k16By128Odd: return tile_bf16<256, 128, 4, 2, 2, 1, true>(A, cus, s, kt);
  }
  return hipErrorInvalidValue;
}

}  // namespace moe
