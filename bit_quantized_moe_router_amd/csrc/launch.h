// Host-side launchers of the MoE kernels (one per kernel family).
#pragma once

#include <hip/hip_ext.h>

#include <atomic>

#include "common.h"
#include "positions.h"

namespace moe {

// Timing of one launcher call: the first kernel it enqueues stamps `start`
// with its own start and the last one stamps `stop` with its own end
// (hipExtLaunchKernel), so the interval holds the kernels and not the
// dispatch gap before them.  Null events: a plain launch.
// A kernel's dynamic-LDS limit (needed above 64 KB), set once per device on
// the current device; `done` holds one bit per device.
inline hipError_t lds_limit_once(const void* fn, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= 64) return hipErrorInvalidDevice;
  const uint64_t bit = 1ull << dev;
  if (done.load(std::memory_order_acquire) & bit) return hipSuccess;
  e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != hipSuccess) return e;
  done.fetch_or(bit, std::memory_order_acq_rel);
  return hipSuccess;
}

// Assignments per segment of the many-token routing metadata.
constexpr int kSegAssign = 1024;

struct KTime {
  hipEvent_t start = nullptr, stop = nullptr;
};

#define MOE_LAUNCH(kernel, grid, block, smem, stream, ev0, ev1, ...)                                 \
  do {                                                                                               \
    if ((ev0) != nullptr || (ev1) != nullptr)                                                        \
      hipExtLaunchKernelGGL(kernel, grid, block, smem, stream, ev0, ev1, 0, __VA_ARGS__);            \
    else                                                                                             \
      kernel<<<grid, block, smem, stream>>>(__VA_ARGS__);                                            \
  } while (0)

struct PackArgs {
  const uint8_t* codes;
  const uint16_t* scales;
  const uint16_t* biases;
  uint8_t* dst;
  int M, N, K;
  int64_t dst_base;
  int64_t stride_m;
  int64_t stride_nb;
  int64_t stride_g;
  int32_t* small_scales;  // the blob trailer's flag, cleared by a scale with |s| >= 2^-4
};

hipError_t launch_pack(const PackArgs& P, hipStream_t s);
// Writes the blob trailer (flag = 1, rest zero) before the matrices are packed.
hipError_t launch_pack_trailer(uint8_t* trailer, hipStream_t s);
// Router logits: exact float64 ones for T <= 8, otherwise bf16-MFMA screened
// partial sums over 4 slices of h (and partial squared router row norms);
// *two_launches tells which.
hipError_t launch_route_logits(const uint16_t* x, int T, int H, const float* wr, const float* bias, int E,
                               int k, float* logits, double* wsq, int32_t* ids, float* tw, float* xsum,
                               uint16_t* x16, int32_t* segcnt, hipStream_t s, bool* two_launches,
                               const KTime& kt = KTime{});
// Top-k selection (exact recomputation of the screened candidates for T > 8).
hipError_t launch_route_select(const uint16_t* x, int T, int H, const float* wr, const float* bias, int E,
                               int k, const float* logits, const double* wsq, int32_t* ids, float* tw,
                               uint16_t* x16, int32_t* segcnt, hipStream_t s, const KTime& kt = KTime{});
// max_long: tiles of more than BM/2 rows that the schedule keeps whole (the
// rest are cut in two); 0 keeps every tile whole.  segcnt: per-segment expert
// counts of the assignments (kSegAssign ids a segment), taken by the exact
// top-k; used when there is more than one segment.
hipError_t launch_meta(const int32_t* ids, int T, int k, int E, int BM, int with_shared, int max_long,
                       int32_t* counts, int32_t* offsets, int32_t* sorted, int32_t* tiles,
                       int32_t* n_tiles, int32_t* active, int32_t* n_active, int32_t* inv,
                       int32_t* sched, const int32_t* segcnt, hipStream_t s, const KTime& kt = KTime{});
// T <= 8: top-k of exact logits and the metadata in one single-workgroup launch.
hipError_t launch_topk_meta(const float* logits, int T, int E, int k, int32_t* ids, float* tw, int BM,
                            int with_shared, int32_t* counts, int32_t* offsets, int32_t* sorted,
                            int32_t* tiles, int32_t* n_tiles, int32_t* active, int32_t* n_active,
                            int32_t* inv, int32_t* sched, hipStream_t s, const KTime& kt = KTime{});
// max_sched: upper bound of the schedule's entry count (sizes the grid).
hipError_t launch_gateup_gemm(const LayerArgs& L, const ChunkArgs& C, int max_sched, hipStream_t s,
                              const KTime& kt = KTime{});
hipError_t launch_down_gemm(const LayerArgs& L, const ChunkArgs& C, int max_sched, hipStream_t s,
                            const KTime& kt = KTime{});
// Separate-dequant measurement: the chunk's active experts (and the shared
// expert) rebuilt as fp16 into L.wdq; the GEMMs then read B from there.
hipError_t launch_dequant_active(const LayerArgs& L, const ChunkArgs& C, hipStream_t s, const KTime& kt = KTime{});
// Gate/up column tiles per row tile (the GEMM grid's second dimension).
int gateup_col_tiles(int I, int Is);
// Grouped-GEMM workgroups resident per compute unit.
int gemm_wgs_per_cu();
// y[t] += sum_j w_tj * routed output of assignment (t, j) (GEMM path).
hipError_t launch_combine(const LayerArgs& L, const ChunkArgs& C, hipStream_t s, const KTime& kt = KTime{});
// Decode GEMV path: top-k, gate/up + SwiGLU and the down projection split
// over the intermediate (partial outputs in `part`), then their fixed-order sum.
hipError_t launch_gemv_experts(const LayerArgs& L, const ChunkArgs& C, const float* logits, float* part,
                               hipStream_t s, const KTime& kt = KTime{});
hipError_t launch_gemv_reduce(const LayerArgs& L, const ChunkArgs& C, const float* part, hipStream_t s,
                              const KTime& kt = KTime{});
// Decode with the grouped-GEMM path's arithmetic: top-k (ranked routing into
// ids/tw), gate/up + SwiGLU into h16 ([T*k + T][Imax] fp16(h / 256)); then the
// down projection of every assignment and the per-token combine into y.
hipError_t launch_gemv_gateup_bi(const LayerArgs& L, const ChunkArgs& C, const float* logits, uint16_t* h16,
                                 int32_t* ids, float* tw, hipStream_t s, const KTime& kt = KTime{});
hipError_t launch_gemv_down_bi(const LayerArgs& L, const ChunkArgs& C, const uint16_t* h16, const int32_t* ids,
                               const float* tw, hipStream_t s, const KTime& kt = KTime{});

// Rows of the microscaled 4-bit format (mx4.h) beside their values.
struct Mx4RowArgs {
  void* wide;       // [rows] of cols fp32 or bf16 values, ld apart (read by quantize, written by dequantize)
  uint8_t* codes;   // [rows][cols / 2]
  uint8_t* scales;  // [rows][cols / 32]
  int64_t rows, cols, ld;
  bool f32;
};
hipError_t launch_mx4_quantize(const Mx4RowArgs& A, hipStream_t s, const KTime& kt = KTime{});
hipError_t launch_mx4_dequantize(const Mx4RowArgs& A, hipStream_t s, const KTime& kt = KTime{});

// Grouped product with microscaled 4-bit expert weights (mx4_experts.hip).
constexpr int kMxTypeF32 = 0, kMxTypeBf16 = 1, kMxTypeMx4 = 2;
struct Mx4ExpertArgs {
  const uint8_t* w_codes;    // [E][n][k / 2]
  const uint8_t* w_scales;   // [E][n][k / 32]
  const void* x;             // [x_rows][k] bf16, or codes [x_rows][k / 2]
  const uint8_t* x_scales;   // [x_rows][k / 32] with x_mx4
  const int32_t* offsets;    // [E + 1]
  const int32_t* src_rows;   // [P] or null
  const int32_t* dst_rows;   // [P] or null
  const float* row_scale;    // [y_rows] or null
  void* y;                   // [y_rows][n_out] of y_type, n_out = swiglu ? n / 2 : n
  uint8_t* y_scales;         // [y_rows][n_out / 32] with y_type = kMxTypeMx4
  int E, n, k, P, x_rows, y_rows, src_div, y_type;
  bool x_mx4, swiglu;
  Divisor src;  // by src_div
};
// The kernels of the product: few rows an expert (kFewSplit: the waves split K); tiles of 256 weight rows (k16Half:
// 128) by 256, 128 or 32 positions for rows of 4 or 16 bits, Odd where the scales' rows are no whole 16-byte pieces.
enum class MxKernel { kFew, kFewSplit, k4By256, k4By128, k4By128Odd, k16By32, k16By32Odd, k16Half, k16By128, k16By128Odd };
// The one to take.  cus: the device's compute units.
MxKernel mx4_experts_kernel(const Mx4ExpertArgs& A, int cus);
const char* mx4_experts_kernel_name(MxKernel m);
hipError_t launch_mx4_experts(const Mx4ExpertArgs& A, MxKernel m, int cus, hipStream_t s, const KTime& kt = KTime{});

// The router's balance loss (balance.hip).
constexpr int kBalMaxParts = 256;  // partial rows of the forward pass
struct BalanceArgs {
  const void* logits;    // [T][E] fp32 or bf16
  const int32_t* ids;    // [T][k]
  const uint8_t* valid;  // [T] or null
  int T, E, k;
  float balance_coef, z_coef;
  bool f32;
  float* losses;         // [3] loss, balance, z
  int32_t* counts;       // [E]
  float* mean_prob;      // [E]
  int32_t* n_valid;      // [1]
  // Workspace of the forward pass.
  int32_t* done;         // [1]
  double* dots;          // [E / 16, rounded up]
  double* part_z;        // [kBalMaxParts]
  int32_t* part_n;       // [kBalMaxParts]
  int32_t* part_count;   // [kBalMaxParts][E]
  float* part_p;         // [kBalMaxParts][E]
  // Backward pass.
  const float* grad;     // [1] or null
  void* dlogits;         // [T][E] of the logits' type
};
// Partial rows of the forward pass over T tokens (1: no second launch).
int balance_parts(int T, int E);
hipError_t launch_balance_forward(const BalanceArgs& A, hipStream_t s, const KTime& kt = KTime{});
hipError_t launch_balance_backward(const BalanceArgs& A, hipStream_t s, const KTime& kt = KTime{});

// Routing from scores and the order of assignments by expert (select.hip).
constexpr int kSortMaxParts = 256;  // parts of the assignments that are counted apart
struct SelectArgs {
  const void* logits;    // [T][E] fp32 or bf16
  const float* bias;     // [E] or null
  const uint8_t* valid;  // [T] or null
  int32_t* ids;          // [T][k]
  float* weights;        // [T][k]
  int T, E, k, groups, per, top_groups, best;  // per: experts a group
  bool f32, softmax, renorm;
  float scale;
  int lanes, run;        // of 16 lanes a token: lanes a group, experts a lane
  int64_t per_part;      // tokens a part
  int32_t* part_count;   // [parts][E] or null
  // Backward pass.
  const float* dweights; // [T][k]
  const void* base;      // [T][E] of the logits' type, or null
  void* dlogits;
};
struct SortArgs {
  const int32_t* ids;    // [n]
  int64_t n;
  int E;
  int32_t* counts;       // [E]
  int32_t* offsets;      // [E + 1]
  int32_t* sorted;       // [n]
  int32_t* part_count;   // [kSortMaxParts][E], then the parts' prefix sums
  int parts;
  int64_t per_part;      // assignments a part
};
// Parts of n assignments, and of T tokens whose experts are to be chosen (1: no partial counts).
int sort_parts(int64_t n);
int select_parts(int T);
hipError_t launch_sort(SortArgs S, hipStream_t s, const KTime& kt = KTime{});
// order: counts, offsets and the sorted assignments too.
hipError_t launch_select_forward(SelectArgs A, SortArgs S, bool order, hipStream_t s, const KTime& kt = KTime{});
hipError_t launch_select_backward(const SelectArgs& A, hipStream_t s, const KTime& kt = KTime{});

// The sum over each token's routed rows (combine.hip).
struct CombineArgs {
  const void* rows;      // [T * k][H] fp32 or bf16
  const int32_t* ids;    // [T][k] or null
  const float* weights;  // [T][k] or null
  const void* base;      // [T][H] of y's type, or null
  void* y;               // [T][H] fp32 or bf16
  int T, k, H;
  bool rows_f32, y_f32;
  // Backward pass.
  const void* dy;        // [T][H] of y's type
  void* drows;           // [T * k][H] of rows' type, or null
  float* dweights;       // [T][k] or null
};
hipError_t launch_combine_forward(const CombineArgs& A, hipStream_t s, const KTime& kt = KTime{});
hipError_t launch_combine_backward(const CombineArgs& A, hipStream_t s, const KTime& kt = KTime{});

// Low-rank adapters (adapters.h).
struct AdapterArgs {
  const uint16_t* a;        // [n][r][K] bf16
  const uint16_t* b;        // [n][N][r] bf16
  const float* scales;      // [n] or null
  const uint16_t* x;        // [x_rows][K] bf16
  const int32_t* offsets;   // [n + 1]
  const int32_t* src_rows;  // [P] or null
  const int32_t* dst_rows;  // [P] or null
  const void* base;         // forward [y_rows][N] of y's type, backward [..][K] bf16; or null
  void* y;                  // [y_rows][N] fp32 or bf16
  float* h_out;             // [P][r]: h of the forward pass, or null
  int n, r, K, N, P, x_rows, y_rows, src_div;
  Divisor src;              // by src_div
  // Backward pass.
  const float* h;           // [P][r]
  uint16_t* thin;           // dh and, thin_h numbers on, h as operands (adapters.h), or null
  int64_t thin_h;
  const void* dy;           // [y_rows][N] of y's type
  void* dx;                 // [x_rows * src_div][K] bf16 or null
  float* da;                // [n][r][K] or null, with db
  float* db;                // [n][N][r]
};
hipError_t launch_adapters_forward(const AdapterArgs& A, bool y_f32, int cus, hipStream_t s, const KTime& kt = KTime{});
size_t adapters_thin_bytes(int r, int64_t rows);
hipError_t launch_adapters_backward(const AdapterArgs& A, bool y_f32, int cus, hipStream_t s, const KTime& kt = KTime{});

// Measurement probes (csrc/probe.hip): a 16-byte-per-lane streaming read of
// `bytes` with at most max_wgs workgroups (sink: max_wgs words), and the
// MFMA-only rate kernel over `wgs` workgroups (clocks: 2 * wgs words or null;
// sink: wgs words).
hipError_t launch_stream_read(const void* src, size_t bytes, uint32_t* sink, int max_wgs, hipStream_t s,
                              const KTime& kt = KTime{});
hipError_t launch_mfma_rate(int iters, int wgs, uint64_t* clocks, uint32_t* sink, hipStream_t s,
                            const KTime& kt = KTime{});

}  // namespace moe
