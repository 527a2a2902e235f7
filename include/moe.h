/*
 * moe.h - C ABI of the MI355X (gfx950) 4-bit group-affine MoE FFN layer.
 *
 * The layer (the "Optimizing on-device inference for Apple Silicon" page):
 *   - a router scores E experts per token and keeps the top k; one shared
 *     expert processes every token (section "Qwen creates three different
 *     workload shapes");
 *   - each expert is a SwiGLU FFN whose weights are 4-bit integer codes, every
 *     64 consecutive weights along the input dimension sharing one bf16 scale
 *     and one bf16 bias that rebuild the weight as w = s*q + b (section
 *     "Dequantise weights during matrix multiplication");
 *   - routing runs on the GPU as top-k, histogram, prefix scan, scatter and a
 *     block map, with no CPU round trip inside the layer (section "Keep
 *     expert routing on the GPU");
 *   - prefill uses a grouped matrix-matrix product over the routed rows;
 *     single-row decode uses a row-parallel matrix-vector product (sections
 *     "Apple silicon provides different paths for different workloads" and
 *     "Optimise the one-row weight path");
 *   - long prompts are processed in bounded chunks (section "Bound temporary
 *     memory with prompt chunking").
 *
 * Conventions shared by every entry point
 *   - All data pointers are DEVICE pointers unless stated otherwise, and are
 *     owned by the caller.  The library allocates no memory in any call and
 *     never reads device memory on the host.
 *   - bf16 values are passed as uint16_t bit patterns.
 *   - `stream` is a hipStream_t (NULL = the default stream).  Every call only
 *     enqueues work on `stream` and returns; no call synchronises.
 *   - Argument and shape errors are reported before anything is enqueued, so a
 *     failed call leaves no partial work.  A failed kernel launch returns
 *     MOE_ERR_HIP; faults during execution surface at the caller's next
 *     synchronisation.  moe_last_error() gives a thread-local message for the
 *     last failure.
 *   - T = 0 is a valid no-op returning MOE_OK.
 *   - Calls on different streams are safe given distinct workspaces and
 *     outputs.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARGUMENT = 1,   /* null pointer, bad count, k > E, ... */
    MOE_ERR_UNSUPPORTED_SHAPE = 2,  /* H or I not a multiple of 64, group != 64, sizes over limits */
    MOE_ERR_WORKSPACE_TOO_SMALL = 3,/* ws_bytes or packed_bytes below the required size */
    MOE_ERR_HIP = 4,                /* a HIP runtime call or kernel launch failed */
    MOE_ERR_DEVICE_UNSUPPORTED = 5  /* the current device is not gfx950 */
} moe_status;

/*
 * Supported activation range.  The grouped-GEMM path feeds its MFMAs fp16(x /
 * 256) and fp16(h / 256) (h = silu(gate) * up) and stores each routed expert
 * output as fp16(o / 256): exact scalings, in range while |x|, |h| and |o|
 * stay below 65504 * 256 (about 1.7e7).  h grows with the square of the
 * activations' scale; for this layer's weights that is activations up to a
 * few hundred times N(0, 1).  Beyond that the path gives inf or NaN in y
 * (with MOE_OK); the decode GEMV path keeps h in bf16 hi/lo parts and reaches
 * further.  Inputs must be finite.
 */

/*
 * Layer description.  Limits: hidden and inter multiples of 64 (the group
 * size; the pages' format cannot quantise a width that is not a multiple of
 * the group, cf. the Laya page's quantisation section), hidden <= 8192,
 * inter <= 4096, shared_inter a multiple of 64 or 0, 1 <= top_k <= 16,
 * top_k <= n_experts <= 512.
 */
typedef struct {
    int32_t hidden;        /* H: model width, the input of gate/up and the output of down */
    int32_t n_experts;     /* E: routed experts */
    int32_t top_k;         /* k: experts kept per token */
    int32_t inter;         /* I: routed expert intermediate width */
    int32_t shared_inter;  /* Is: shared expert intermediate width, 0 = no shared expert */
    int32_t group_size;    /* must be 64 */
    int32_t gemv_max_rows; /* R*: moe_forward_decode uses the row-parallel GEMV path for
                              T <= R* and the grouped GEMM path above; -1 = library default
                              (8, or 4 with batch_invariant = 1); 0 = always GEMM; at most 8 */
    int32_t max_chunk;     /* tokens per prefill chunk (1..8192); routing metadata is per chunk */
    int32_t tile_rows;     /* BM: rows per tile of the block map; 0 = library default (128);
                              one of 16, 32, 64, 128 */
    int32_t host_sync_routing; /* 0 (the normal path): routing never returns to the host.  1: a
                              measurement of the alternative the pages argue against ("Keep expert
                              routing on the GPU"): after each chunk's routing, the grouped-GEMM path
                              copies the schedule's entry count to the host, synchronises the stream
                              and sizes the GEMM launches from it.  Same kernels and results; the
                              call then blocks and cannot be captured in a graph. */
    int32_t dequant_pass;  /* 0 (the normal path): weights are rebuilt inside the grouped GEMMs.  1: a
                              measurement of the alternative the pages compare against ("Dequantise
                              weights during matrix multiplication"): each chunk's active experts and
                              the shared expert are first rebuilt as fp16 into the workspace (a
                              separate pass), then the grouped GEMMs read fp16 weights.  Same rounding,
                              same results; the workspace grows by 4096/1152 x the packed size. */
    int32_t batch_invariant; /* 0: the decode GEMV path folds scale and bias per group and splits the
                              down projection (its own rounding).  1: the GEMV path computes every
                              output element with the grouped-GEMM path's operations in the same order
                              (fp16 weights rebuilt as s*q + b, fp16(x / 256), one MFMA chain over K,
                              fp16(h / 256) and fp16(o / 256) intermediates, ranked routing weights,
                              combine in rank order), so a row's output does not depend on the row
                              threshold or on the other rows of the call (the dothoosh page on Candle,
                              its section on outputs that change with the kernel chosen by row count).
                              Costs time: the chain over K runs in order, so one row takes about 26 us
                              instead of 20; the default R* is then 4, above which the grouped GEMM
                              path (same bits) is faster. */
} moe_layer_desc;

/*
 * One quantised matrix stack in the canonical format (device pointers):
 *   codes  [M][N][K/2]  uint8, two codes per byte, the even k in the low nibble
 *   scales [M][N][K/64] bf16 bits
 *   biases [M][N][K/64] bf16 bits
 * with M = E for routed matrices and M = 1 for the shared expert; gate and up
 * have N = inter (or shared_inter), K = hidden; down has N = hidden, K = inter.
 */
typedef struct {
    const uint8_t *codes;
    const uint16_t *scales;
    const uint16_t *biases;
} moe_qmatrix;

/*
 * Routing outputs for one chunk of T tokens (device pointers, caller-owned):
 *   topk_ids       [T][k]  int32, experts in order of decreasing logit
 *   topk_weights   [T][k]  float, softmax over the k selected logits
 *   expert_counts  [E]     int32, assignments per expert (histogram)
 *   expert_offsets [E+1]   int32, exclusive prefix scan of the counts
 *   sorted_assign  [T*k]   int32, flat assignment ids t*k+j grouped by expert,
 *                          increasing inside each expert (stable scatter)
 *   tile_map       [moe_max_tiles][3] int32, (expert, first row inside the
 *                          expert's segment, rows) per BM-row tile, experts in
 *                          increasing order, then the shared expert's tiles as
 *                          expert E over the tokens
 *   n_tiles        [1]     int32, the number of valid tile_map entries
 */
typedef struct {
    int32_t *topk_ids;
    float *topk_weights;
    int32_t *expert_counts;
    int32_t *expert_offsets;
    int32_t *sorted_assign;
    int32_t *tile_map;
    int32_t *n_tiles;
} moe_routing;

/*
 * Size in bytes of the packed weight blob for `desc` (host output): the
 * canonical 4-bit codes plus one bf16 scale and one bf16 bias per 64 weights,
 * 0.5625 bytes per parameter (the Laya page's quantisation section gives this
 * storage cost of the group-64 4-bit format), plus a 256-byte trailer (a flag
 * the packer writes for the kernels).  Host-only; no device access.
 */
moe_status moe_packed_bytes(const moe_layer_desc *desc, size_t *bytes);

/*
 * Workspace bytes needed by moe_route / moe_forward_* for up to max_tokens per
 * call (host output).  The workspace holds one chunk's routing metadata and
 * intermediates; prefill reuses it chunk after chunk, so its size is bounded
 * by max_chunk whatever T is ("Optimizing on-device inference for Apple
 * Silicon", section "Bound temporary memory with prompt chunking").  For
 * max_tokens > max_chunk the size includes a second routing area (about 18 MB
 * at H=2048, E=256, k=8 and 2048-token chunks), with which the forward calls
 * route the next chunk while the current one's GEMMs run; a workspace of the
 * one-chunk size (moe_workspace_bytes(desc, min(T, max_chunk))) is still
 * valid for any T and runs the chunks one after the other.
 * Host-only; no device access.
 */
moe_status moe_workspace_bytes(const moe_layer_desc *desc, int32_t max_tokens, size_t *bytes);

/*
 * Upper bound of the tile_map entries moe_route writes for a chunk of T tokens
 * (host output): the block map of fixed-size tiles per expert (section "Keep
 * expert routing on the GPU" of the same page).  Host-only.
 */
moe_status moe_max_tiles(const moe_layer_desc *desc, int32_t T, int32_t *n);

/*
 * Repack canonical quantised weights into the library's blob (device, size
 * moe_packed_bytes).  The format is the page's: 4-bit codes, every 64 weights
 * along the input dimension sharing one bf16 scale and one bf16 bias, w = s*q
 * + b ("Optimizing on-device inference for Apple Silicon", section
 * "Dequantise weights during matrix multiplication").  The blob is opaque and valid only for the desc that
 * made it.  It stores exactly the canonical codes (0.5625 bytes per parameter
 * with the scales and biases), rearranged so that one 64-lane wave reads a
 * 32-row x 64-column group with one 16-byte load per lane; the scales and
 * biases are stored converted to fp16 (round to nearest even), the type the
 * kernels rebuild weights in.  The conversion is exact for magnitudes in
 * [2^-14, 65504]; smaller values lose bits as fp16 subnormals and larger
 * ones become infinity, so the supported scale and bias range is fp16's.  The
 * blob's last 256 bytes are a trailer whose first int32 the packer sets to 1
 * when every scale is below 2^-4 in magnitude (0 otherwise); the grouped GEMM
 * then rebuilds weights with fewer instructions, to the same bits.  sh_* are ignored when
 * shared_inter == 0.  One-time preparation; not part of the forward path.
 */
moe_status moe_pack_weights(const moe_layer_desc *desc, moe_qmatrix gate, moe_qmatrix up,
                            moe_qmatrix down, moe_qmatrix sh_gate, moe_qmatrix sh_up,
                            moe_qmatrix sh_down, void *packed, size_t packed_bytes, void *stream);

/*
 * Route one chunk of T <= max_chunk tokens on the GPU, with no return to the
 * host ("Optimizing on-device inference for Apple Silicon", section "Keep
 * expert routing on the GPU": top-k, histogram, prefix scan, scatter, block
 * map; section "Qwen creates three different workload shapes": top-8 of 256
 * routed experts plus one shared expert): router logits
 * fp32(sum_h x[t,h]*Wr[e,h] accumulated in float64) + logit_bias[e], top-k,
 * softmax weights, then histogram, prefix scan, stable scatter and block map,
 * all on the GPU.
 *   x          [T][H] bf16
 *   router_w   [E][H] float
 *   logit_bias [E] float or NULL
 *   ws         workspace of at least moe_workspace_bytes(desc, T) bytes
 */
moe_status moe_route(const moe_layer_desc *desc, const uint16_t *x, int32_t T,
                     const float *router_w, const float *logit_bias, const moe_routing *out,
                     void *ws, size_t ws_bytes, void *stream);

/*
 * Full layer over T tokens with the grouped dequantising GEMM path, chunk by
 * chunk (max_chunk tokens each; "Optimizing on-device inference for Apple
 * Silicon", sections "Dequantise weights during matrix multiplication", "Match
 * tile size to expert load", "Reduce intermediate and state traffic" and
 * "Bound temporary memory with prompt chunking"):
 *   y[t] = sum_j topk_weights[t,j] * FFN_{topk_ids[t,j]}(x[t]) + FFN_shared(x[t])
 * with FFN(x) = Wd (silu(Wg x) * (Wu x)).
 *   packed  blob from moe_pack_weights
 *   y       [T][H] float (written, not accumulated)
 *   ws      at least moe_workspace_bytes(desc, min(T, max_chunk)) bytes
 * With more than one chunk and a workspace of moe_workspace_bytes(desc, T)
 * bytes, two chunks are in flight at once: even chunks run on `stream` and odd
 * chunks on a second stream of the library's (one per device, created on first
 * use, default priority), except that the combine of a last odd chunk runs on
 * `stream`.  Events order the two streams, and the call returns with all of its
 * work joined to `stream`, so stream order holds for the caller as with one
 * stream (also under graph capture of `stream`).  The result is the same bits
 * either way.  The second stream and its events are created by the first such
 * call on a device; make that call outside graph capture, as HIP may refuse to
 * create a stream while one is being captured.
 */
moe_status moe_forward_prefill(const moe_layer_desc *desc, const void *packed,
                               const float *router_w, const float *logit_bias,
                               const uint16_t *x, int32_t T, float *y,
                               void *ws, size_t ws_bytes, void *stream);

/*
 * Same layer for a few rows: the row-parallel GEMV path when T <=
 * gemv_max_rows (at most 8), otherwise the grouped GEMM path of
 * moe_forward_prefill (any T, chunked the same way).  The pages' one-row
 * weight path ("Optimizing on-device inference for Apple Silicon", section
 * "Optimise the one-row weight path") and the choice of kernel by row count
 * (the dothoosh page on Candle's Metal kernels, its kernel-selection and
 * crossover sections).
 * The GEMV path is three launches: exact router logits; top-k, gate/up +
 * SwiGLU and the down projection of each workgroup's 32 intermediate columns
 * (partial output rows in the workspace); the sum of each token's partials in
 * a fixed order.  y is written once per element, with no atomics, so repeated
 * calls give identical bits.  With batch_invariant = 1 the GEMV path is
 * instead: exact router logits; top-k, gate/up + SwiGLU into fp16 rows of h;
 * down projection and combine, with the grouped GEMM path's operations, so
 * its output equals that path's bit for bit at every T.
 */
moe_status moe_forward_decode(const moe_layer_desc *desc, const void *packed,
                              const float *router_w, const float *logit_bias,
                              const uint16_t *x, int32_t T, float *y,
                              void *ws, size_t ws_bytes, void *stream);

/*
 * moe_forward_decode without a workspace argument, for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc.  Same arguments, kernels and results as
 * moe_forward_decode, whose workspace is here a fixed device array of
 * MOE_STATIC_SCRATCH_BYTES inside the library; each GPU the library runs on
 * holds its own copy until the process ends.  The call allocates and frees
 * nothing (its first call on a device looks the array's address up once).
 * Limits and errors:
 *   - MOE_ERR_WORKSPACE_TOO_SMALL when the layer's decode workspace at this T
 *     exceeds MOE_STATIC_SCRATCH_BYTES (moe_workspace_bytes(desc, T) tells);
 *     16 MiB hold T <= 8 at H=2048, E=256, k=8, I=Is=512 (9.2 MiB);
 *   - MOE_ERR_INVALID_ARGUMENT for host_sync_routing or dequant_pass set.
 * Every call on one GPU uses the same array: calls that overlap in time on
 * one GPU (other streams, other threads) race and give undefined results;
 * serialise them.  Stream-ordered calls on one stream are safe.
 */
#define MOE_STATIC_SCRATCH_BYTES ((size_t)16 << 20)
moe_status moe_forward_decode_static(const moe_layer_desc *desc, const void *packed,
                                     const float *router_w, const float *logit_bias,
                                     const uint16_t *x, int32_t T, float *y, void *stream);

/*
 * Element types of the calls below.  MOE_F32 and MOE_BF16 are plain values;
 * MOE_MX4 is the microscaled 4-bit format (MXFP4), held in two arrays:
 *   codes  [rows][cols/2]  uint8, two e2m1 codes per byte, the even column in
 *                          the low nibble; a code is a sign bit and one of the
 *                          magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6
 *   scales [rows][cols/32] uint8, one per 32 consecutive values of a row: s
 *                          stands for 2^(s - 127), and 255 for NaN
 * A value is code * 2^(s - 127); 0.53125 bytes per value.  It is the 4-bit
 * floating format beside the integer one of moe_pack_weights, and the one that
 * the matrix units multiply without rebuilding it.
 */
enum { MOE_F32 = 0, MOE_BF16 = 1, MOE_MX4 = 2 };

/*
 * Quantise rows to MOE_MX4.  For each block of 32 values with the largest
 * magnitude amax, the scale is 2^(floor(log2 amax) - 2), not below 2^-127, and
 * a code is the e2m1 value nearest to x / scale, ties to the one with an even
 * mantissa bit; magnitudes above 6 scales are held at 6 (amax / scale is below 8).
 * Exact in every other respect, subnormal inputs included; -0 keeps its sign.
 * A block of zeros has the scale byte 0.  A block that holds a NaN or an
 * infinity gets the scale byte 255 and zero codes: it reads back as NaN.
 *   x      [rows] of cols values of x_type (MOE_F32 or MOE_BF16), the rows
 *          ldx values apart (ldx >= cols); any alignment of its type, 16-byte
 *          aligned rows are faster
 *   cols   a positive multiple of 32, at most 2^24; rows = 0 is a no-op
 *   codes, scales  as above, contiguous; codes 16-byte aligned; neither may
 *          overlap x
 */
moe_status moe_mx4_quantize(const void *x, int32_t x_type, int64_t rows, int64_t cols, int64_t ldx,
                            uint8_t *codes, uint8_t *scales, void *stream);

/*
 * Read MOE_MX4 rows back as values of y_type (MOE_F32 or MOE_BF16), exactly,
 * but for magnitudes of 2^128 and more (scale bytes 253 and 254 with the large
 * codes, which moe_mx4_quantize never writes): those become infinity.  y as x
 * above; the values between cols and ldy stay as they were.
 */
moe_status moe_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols,
                              void *y, int32_t y_type, int64_t ldy, void *stream);

/*
 * A stack of expert matrices W_e [n][k] in MOE_MX4 and how they are applied.
 */
typedef struct {
    int32_t n_experts; /* E: 1..512; 1 for one dense matrix */
    int32_t n;         /* rows of a matrix, 1..65536; with swiglu even: the gate rows, then the up rows */
    int32_t k;         /* columns: a multiple of 32, at most 65536 */
    int32_t x_type;    /* MOE_BF16 or MOE_MX4 */
    int32_t y_type;    /* MOE_F32, MOE_BF16, or MOE_MX4 (its columns then a multiple of 32) */
    int32_t swiglu;    /* 1: y = silu(z[:n/2]) * z[n/2:], n/2 columns; 0: y = z, n columns */
} moe_mx4_desc;

/*
 * Grouped product of routed rows with their experts' matrices, the form that
 * moe_forward_* have inside for the integer format: position i in
 * [expert_offsets[e], expert_offsets[e+1]) has z = W_e x[src(i)], and
 * y[dst(i)] = row_scale[dst(i)] * (z, or its SwiGLU).  For any number of rows:
 * a single token's positions are products with a vector.
 *   w_codes, w_scales  [E][n][k/2] and [E][n][k/32]: moe_mx4_quantize of E * n
 *                      rows of k values
 *   x, x_scales        [x_rows] rows of k values of x_type (x_scales NULL for
 *                      MOE_BF16)
 *   expert_offsets     [E+1] int32, increasing from 0 to the number of
 *                      positions, as moe_route writes them
 *   rows               the positions' upper bound on the host, at most 2^24:
 *                      expert_offsets[E] is at most rows (offsets are held
 *                      inside [0, rows])
 *   src_rows, src_div  src(i) = src_rows[i] / src_div, or i where src_rows is
 *                      NULL; moe_route's sorted_assign with src_div = k gives
 *                      each assignment its token's row
 *   dst_rows           dst(i) = dst_rows[i], or i where NULL; each row at most
 *                      once; sorted_assign gives each assignment its own row
 *   row_scale          [y_rows] float or NULL: a factor for each row of y
 *                      (moe_route's topk_weights beside dst_rows = sorted_assign)
 *   y, y_scales        [y_rows] rows of n (with swiglu n/2) values of y_type
 *                      (y_scales NULL but for MOE_MX4)
 * w_codes, x and a MOE_MX4 y are 16-byte aligned, another y to its type;
 * k a multiple of 512 with 16-byte aligned scales, and rows of y that are
 * multiples of 16 bytes, are faster.  A src(i) outside x gives a row of
 * zeros and a dst(i) outside y is not written.  Rows of y that no position
 * maps to, those of positions behind expert_offsets[E] among them, stay as
 * they were.  y must not overlap an input.
 * Products are summed in fp32 (bf16 x with the weights' exact bf16 values,
 * infinity for 2^128 and more, which moe_mx4_quantize never writes; MOE_MX4 x
 * in the scaled matrix instructions), SwiGLU and row_scale are
 * applied in fp32, and the result is rounded once to y_type, for MOE_MX4 as
 * moe_mx4_quantize does.  Repeated calls give identical bits.  No workspace.
 * rows = 0 is a no-op.
 */
moe_status moe_mx4_experts(const moe_mx4_desc *desc, const uint8_t *w_codes, const uint8_t *w_scales,
                           const void *x, const uint8_t *x_scales, int32_t x_rows,
                           const int32_t *expert_offsets, int32_t rows, const int32_t *src_rows,
                           int32_t src_div, const int32_t *dst_rows, const float *row_scale, void *y,
                           uint8_t *y_scales, int32_t y_rows, void *stream);

/*
 * The router's balance loss for training, with the per-expert counts.  With
 * p_t the softmax of token t's logits over the E = n_experts experts, lse_t
 * its log-sum-exp, n the valid tokens, counts_e the assignments of valid
 * tokens to expert e, f_e = counts_e / (n k) and P_e = sum_t p_te / n (sums
 * over valid tokens):
 *   balance = E sum_e f_e P_e          (1 where all experts are used alike)
 *   z       = sum_t lse_t^2 / n
 *   loss    = balance_coef * balance + z_coef * z
 *   logits    [T][E] of logits_type (MOE_F32 or MOE_BF16), any alignment of it
 *   topk_ids  [T][k] int32, moe_route's; an id outside 0..E-1 is counted
 *             nowhere, one that stands twice in a row counts twice
 *   valid     [T] uint8, 0 for a padding token, or NULL: all are valid
 *   losses    [3] float: loss, balance, z
 *   counts    [E] int32
 *   mean_prob [E] float: P_e
 *   n_valid   [1] int32: n
 *   ws        moe_balance_loss_workspace_bytes(T, E) bytes, 8-byte aligned
 * Logits are finite or -inf; a row of -inf alone adds nothing to the sums and
 * has a zero gradient, but counts as a token.  A NaN or +inf in a valid row
 * makes the loss and that row's gradient NaN.  With no valid token, T = 0
 * included, the losses, P and counts are 0.  T * top_k < 2^31.
 * Probabilities are fp32, the sums over tokens fp32 within a workgroup's rows
 * and float64 beyond; repeated calls give identical bits.  Two calls that
 * overlap in time need two workspaces, also when replayed from graphs.
 */
moe_status moe_balance_loss_workspace_bytes(int32_t T, int32_t n_experts, size_t *bytes);
moe_status moe_balance_loss_forward(const void *logits, int32_t logits_type, int32_t T, int32_t n_experts,
                                    const int32_t *topk_ids, int32_t top_k, const uint8_t *valid,
                                    float balance_coef, float z_coef, float *losses, int32_t *counts,
                                    float *mean_prob, int32_t *n_valid, void *ws, size_t ws_bytes,
                                    void *stream);

/*
 * Gradient of the loss with respect to the logits, times the float at
 * grad_loss (device; NULL = 1), from what the forward call read and wrote:
 *   dlogits_te = grad p_te (balance_coef E / n (f_e - sum_j f_j p_tj) + 2 z_coef lse_t / n)
 * with zeros for padding tokens.  f, made of counts, has no gradient.
 *   dlogits  [T][E] of logits_type; may be logits itself
 */
moe_status moe_balance_loss_backward(const void *logits, int32_t logits_type, int32_t T, int32_t n_experts,
                                     int32_t top_k, const uint8_t *valid, float balance_coef,
                                     float z_coef, const int32_t *counts, const int32_t *n_valid,
                                     const float *grad_loss, void *dlogits, void *stream);

/* Default R* of the library with batch_invariant = 0 (host output); with
 * batch_invariant = 1 the default is 4. */
int32_t moe_default_gemv_max_rows(void);

const char *moe_status_str(moe_status s);
const char *moe_last_error(void);

/*
 * Kernel timing for measurement tools.  moe_profile_enable(mask) makes every
 * launch of the kernels whose bit is set in `mask` (bit i = kernel id i; 0
 * turns timing off) stamp a HIP event pair on the launch stream: the first
 * kernel of the step stamps its own start and the last its own end
 * (hipExtLaunchKernel).  A stamped launch costs a few microseconds more than
 * a plain one, so time whole steps with timing off.  moe_profile_read
 * synchronises on those events and returns the summed duration (ms) and
 * launch count of kernel `kernel_id` since the last reset.  Never needed on
 * the forward path.  Not thread-safe.
 *   0 = router logits (screen, or exact for T <= 8), 1 = exact top-k
 *   selection (T > 8), 2 = routing metadata (with top-k for T <= 8 outside
 *   the decode GEMV path), 3 = gate/up grouped GEMM, 4 = down grouped GEMM,
 *   5 = top-k + gate/up GEMV + split down GEMV (decode GEMV path), 6 = sum of
 *   the decode path's partial outputs, 7 = per-token combine of the
 *   grouped-GEMM path, 8 = separate dequant pass (dequant_pass = 1), 9 and
 *   10 = the measurement probes, 11 = moe_mx4_quantize, 12 = moe_mx4_dequantize,
 *   13 = moe_mx4_experts, 14 = moe_balance_loss_forward,
 *   15 = moe_balance_loss_backward
 */
moe_status moe_profile_enable(int32_t mask);
moe_status moe_profile_reset(void);
moe_status moe_profile_read(int32_t kernel_id, double *total_ms, int32_t *launches);

/*
 * The kernel that the calling thread's last moe_mx4_experts call took, for
 * measurement tools and tests ("" before the first): "few" (rows an expert;
 * "few split" where the waves split K), or weight rows x positions of a tile,
 * "4-bit 256x256", "4-bit 256x128", "bf16 256x128", "bf16 128x128" or "bf16
 * 256x32", with " odd" where k is no multiple of 512 or a scale array begins at
 * no multiple of 16 bytes.  A static string.
 */
const char *moe_mx4_experts_kernel(void);

#ifdef __cplusplus
}
#endif
#endif /* MOE_H */
