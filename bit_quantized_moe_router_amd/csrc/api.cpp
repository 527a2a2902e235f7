// C ABI of the MoE layer: argument validation, workspace carving, the chunk
// loop and the GEMV/GEMM dispatch.  Host code only; it enqueues kernels on the
// caller's stream and never allocates device memory, synchronises or reads
// device data (the optional kernel-timing mode aside, which only records
// events and synchronises inside moe_profile_read).
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>
#include <vector>

#include "../../include/moe.h"
#include "launch.h"

using namespace moe;

namespace {

thread_local std::string g_last_error;

moe_status fail(moe_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
moe_status fail(moe_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return s;
}

constexpr int kDefaultTileRows = 128;
constexpr int kDefaultGemvMaxRows = 8;  // measured: the GEMV path is faster at every T <= 8 (the decode maximum)
// With batch_invariant = 1 both paths give the same bits, so the threshold only
// picks the faster: measured, the GEMV path with the grouped GEMM's arithmetic
// is faster up to 4 rows (26 us at T = 1 against 47 us) and slower from 5.
constexpr int kDefaultGemvMaxRowsBi = 4;
constexpr int kMaxRowsDecode = 8;

moe_status validate_desc(const moe_layer_desc* d) {
  if (!d) return fail(MOE_ERR_INVALID_ARGUMENT, "desc is null");
  if (d->group_size != 64) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "group_size must be 64 (got %d)", d->group_size);
  if (d->hidden <= 0 || d->hidden % 64 || d->hidden > 8192)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "hidden must be a positive multiple of 64 <= 8192 (got %d)", d->hidden);
  if (d->inter <= 0 || d->inter % 64 || d->inter > 4096)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "inter must be a positive multiple of 64 <= 4096 (got %d)", d->inter);
  if (d->shared_inter < 0 || d->shared_inter % 64 || d->shared_inter > 4096)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "shared_inter must be 0 or a multiple of 64 <= 4096 (got %d)", d->shared_inter);
  if (d->n_experts < 1 || d->n_experts > 512)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "n_experts must be in 1..512 (got %d)", d->n_experts);
  if (d->top_k < 1 || d->top_k > 16) return fail(MOE_ERR_INVALID_ARGUMENT, "top_k must be in 1..16 (got %d)", d->top_k);
  if (d->top_k > d->n_experts)
    return fail(MOE_ERR_INVALID_ARGUMENT, "top_k (%d) exceeds n_experts (%d)", d->top_k, d->n_experts);
  if (d->gemv_max_rows < -1 || d->gemv_max_rows > kMaxRowsDecode)
    return fail(MOE_ERR_INVALID_ARGUMENT, "gemv_max_rows must be in -1..8 (got %d)", d->gemv_max_rows);
  if (d->max_chunk < 1 || d->max_chunk > 8192)
    return fail(MOE_ERR_INVALID_ARGUMENT, "max_chunk must be in 1..8192 (got %d)", d->max_chunk);
  const int bm = d->tile_rows;
  if (!(bm == 0 || bm == 16 || bm == 32 || bm == 64 || bm == 128))
    return fail(MOE_ERR_INVALID_ARGUMENT, "tile_rows must be 0, 16, 32, 64 or 128 (got %d)", bm);
  if (d->host_sync_routing != 0 && d->host_sync_routing != 1)
    return fail(MOE_ERR_INVALID_ARGUMENT, "host_sync_routing must be 0 or 1 (got %d)", d->host_sync_routing);
  if (d->dequant_pass != 0 && d->dequant_pass != 1)
    return fail(MOE_ERR_INVALID_ARGUMENT, "dequant_pass must be 0 or 1 (got %d)", d->dequant_pass);
  if (d->batch_invariant != 0 && d->batch_invariant != 1)
    return fail(MOE_ERR_INVALID_ARGUMENT, "batch_invariant must be 0 or 1 (got %d)", d->batch_invariant);
  return MOE_OK;
}

int tile_rows(const moe_layer_desc* d) { return d->tile_rows ? d->tile_rows : kDefaultTileRows; }
int imax(const moe_layer_desc* d) { return d->inter > d->shared_inter ? d->inter : d->shared_inter; }

int64_t max_tiles_for(const moe_layer_desc* d, int64_t T) {
  if (T <= 0) return 1;
  const int64_t BM = tile_rows(d), k = d->top_k, E = d->n_experts;
  const int64_t tk = T * k;
  return (tk + BM - 1) / BM + (E < tk ? E : tk) + (d->shared_inter > 0 ? (T + BM - 1) / BM : 0);
}

// Schedule entries: the tiles, plus one more for each tile of more than
// BM/2 rows that the schedule may cut in two.
int64_t max_sched_for(const moe_layer_desc* d, int64_t T) {
  const int64_t mt = max_tiles_for(d, T), BM = tile_rows(d);
  if (T <= 0 || BM < 64) return mt;
  return mt + (T * d->top_k + (d->shared_inter > 0 ? T : 0)) / (BM / 2 + 1);
}

struct Blob {
  int64_t expert_bytes, gateup_bytes, shared_base, shared_gateup_bytes, trailer, total;
};

Blob blob_geom(const moe_layer_desc* d) {
  const int64_t H = d->hidden, I = d->inter, Is = d->shared_inter, E = d->n_experts;
  Blob b;
  b.gateup_bytes = (I / 32) * (H / 64) * 2 * kBlockBytes;
  b.expert_bytes = b.gateup_bytes + (H / 32) * (I / 64) * kBlockBytes;
  b.shared_base = E * b.expert_bytes;
  b.shared_gateup_bytes = (Is / 32) * (H / 64) * 2 * kBlockBytes;
  b.trailer = b.shared_base + (Is ? b.shared_gateup_bytes + (H / 32) * (Is / 64) * kBlockBytes : 0);
  b.total = b.trailer + kTrailerBytes;
  return b;
}

struct Ws {
  size_t logits, wnorm, xsum, x16, ids, tw, counts, offsets, sorted, inv, tiles, sched, n_tiles, active, n_active, segs,
      hbuf, obuf, dpart, wdq;
  size_t span;     // bytes of one chunk's area (logits .. obuf)
  int areas;       // 1, or 2: a second chunk area follows the first
  size_t total;
};

size_t al(size_t x) { return (x + 255) & ~size_t(255); }

// Workspace of one chunk: routing outputs, gathered activations and the
// GEMMs' intermediates.  With areas = 2 it is there twice, so two chunks can
// be in flight at once (one per stream).  Offsets are relative to an area's
// base, except wdq's, which is relative to the workspace.
Ws ws_layout(const moe_layer_desc* d, int64_t Tc, int areas = 1) {
  const int64_t E = d->n_experts, k = d->top_k, H = d->hidden, Im = imax(d);
  const int64_t rows = Tc * k + Tc;
  Ws w;
  size_t o = 0;
  w.logits = o; o += al(4 * Tc * E * 4);  // 4 partial slices of the screened logits
  w.wnorm = o; o += al(4 * E * 8);
  w.xsum = o; o += al(Tc * (H / 64) * 4);
  w.x16 = o; o += al(Tc * H * 2);
  w.ids = o; o += al(Tc * k * 4);
  w.tw = o; o += al(Tc * k * 4);
  w.counts = o; o += al(E * 4);
  w.offsets = o; o += al((E + 1) * 4);
  w.sorted = o; o += al(Tc * k * 4);
  w.inv = o; o += al(Tc * k * 4);
  w.tiles = o; o += al(max_tiles_for(d, Tc) * 3 * 4);
  w.sched = o; o += al((1 + max_sched_for(d, Tc)) * 16);  // count, then an int4 descriptor per entry
  w.n_tiles = o; o += al(4);
  w.active = o; o += al(E * 4);
  w.n_active = o; o += al(4);
  w.segs = o; o += al(((Tc * k + kSegAssign - 1) / kSegAssign) * E * 4);  // per-segment expert counts
  w.hbuf = o; o += al(rows * Im * 2);
  // obuf (grouped-GEMM path) and dpart (decode GEMV path: partial outputs
  // [T*k + T][Imax/32][H] fp32, T <= 8) are never live together: one region.
  const int64_t Td = Tc < kMaxRowsDecode ? Tc : kMaxRowsDecode;
  const int64_t dpart_bytes = (Td * k + Td) * (Im / 32) * H * 4;
  w.obuf = o;
  w.dpart = o;
  o += al((Tc * k + Tc) * H * 2 > dpart_bytes ? (Tc * k + Tc) * H * 2 : dpart_bytes);
  w.span = o;
  w.areas = areas;
  o *= areas;
  // Separate-dequant measurement only: an fp16 copy of the blob's blocks.
  w.wdq = o;
  if (d->dequant_pass) o += al(blob_geom(d).total / kBlockBytes * kDqBlockBytes);
  w.total = o;
  return w;
}

template <class T>
T* at(void* base, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(base) + off);
}

// ---- device check -------------------------------------------------------
std::mutex g_dev_mu;
int g_dev_ok[64];   // 0 = unknown, 1 = gfx950, -1 = other
int g_dev_cus[64];  // compute units

moe_status check_device() {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(MOE_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
  if (dev < 0 || dev >= 64) return fail(MOE_ERR_DEVICE_UNSUPPORTED, "device index %d out of range", dev);
  std::lock_guard<std::mutex> lk(g_dev_mu);
  if (g_dev_ok[dev] == 0) {
    hipDeviceProp_t p;
    e = hipGetDeviceProperties(&p, dev);
    if (e != hipSuccess) return fail(MOE_ERR_HIP, "hipGetDeviceProperties: %s", hipGetErrorString(e));
    g_dev_ok[dev] = strncmp(p.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
    g_dev_cus[dev] = p.multiProcessorCount;
  }
  if (g_dev_ok[dev] != 1) return fail(MOE_ERR_DEVICE_UNSUPPORTED, "device %d is not gfx950", dev);
  return MOE_OK;
}

// Compute units of the current device (after check_device on it).
int device_cus() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 1;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  return g_dev_cus[dev];
}

// Long tiles the schedule keeps whole: one round of gate/up workgroups over
// the device (after check_device on the current device).
int max_long_tiles(const moe_layer_desc* d) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  return g_dev_cus[dev] * gemm_wgs_per_cu() / gateup_col_tiles(d->inter, d->shared_inter);
}

// ---- kernel timing (measurement mode) ----------------------------------------
constexpr int kNumKernels = 23;
struct Pending {
  int kid;
  hipEvent_t a, b;
};
std::mutex g_prof_mu;
uint32_t g_prof_mask = 0;  // bit i: time kernel id i
std::vector<Pending> g_pending;
std::vector<hipEvent_t> g_event_pool;
double g_prof_ms[kNumKernels];
int g_prof_n[kNumKernels];

hipEvent_t get_event() {
  if (!g_event_pool.empty()) {
    hipEvent_t e = g_event_pool.back();
    g_event_pool.pop_back();
    return e;
  }
  // No system-scope fence on record: the profiling events must not flush the
  // caches between the kernels they time (device-scope ordering suffices
  // for timestamps read back with hipEventSynchronize).
  hipEvent_t e = nullptr;
  if (hipEventCreateWithFlags(&e, hipEventDisableSystemFence) != hipSuccess) return nullptr;
  return e;
}

// Launch `fn(KTime)` (returning hipError_t).  When timing is on, the events
// go to the launcher, which has its first kernel stamp the start and its last
// kernel the end; both are also recorded just before, so a call that
// enqueues nothing reads 0.
template <class F>
moe_status timed(int kid, hipStream_t s, const char* what, F fn) {
  Pending p{kid, nullptr, nullptr};
  const bool on = kid >= 0 && ((g_prof_mask >> kid) & 1u);
  if (on) {
    std::lock_guard<std::mutex> lk(g_prof_mu);
    p.a = get_event();
    p.b = get_event();
    if (p.a && p.b) {
      (void)hipEventRecord(p.a, s);
      (void)hipEventRecord(p.b, s);
    }
  }
  KTime kt;
  if (on && p.a && p.b) {
    kt.start = p.a;
    kt.stop = p.b;
  }
  hipError_t e = fn(kt);
  if (on && p.a && p.b) {
    std::lock_guard<std::mutex> lk(g_prof_mu);
    g_pending.push_back(p);
  }
  if (e != hipSuccess) return fail(MOE_ERR_HIP, "%s launch failed: %s", what, hipGetErrorString(e));
  return MOE_OK;
}

#define TRY(x)                     \
  do {                             \
    moe_status _s = (x);           \
    if (_s != MOE_OK) return _s;   \
  } while (0)

LayerArgs layer_args(const moe_layer_desc* d, const void* packed) {
  const Blob b = blob_geom(d);
  LayerArgs L;
  L.blob = static_cast<const uint8_t*>(packed);
  L.H = d->hidden;
  L.E = d->n_experts;
  L.k = d->top_k;
  L.I = d->inter;
  L.Is = d->shared_inter;
  L.expert_bytes = b.expert_bytes;
  L.gateup_bytes = b.gateup_bytes;
  L.shared_base = b.shared_base;
  L.shared_gateup_bytes = b.shared_gateup_bytes;
  L.small_scales = reinterpret_cast<const int32_t*>(L.blob + b.trailer);
  L.wdq = nullptr;
  return L;
}

struct RouteOut {
  int32_t *ids, *counts, *offsets, *sorted, *inv, *tiles, *sched, *n_tiles, *active, *n_active, *segs;
  float *tw, *logits, *xsum;
  double* wsq;
  uint16_t* x16;
};

moe_status run_route(const moe_layer_desc* d, const uint16_t* x, int T, const float* wr,
                     const float* bias, const RouteOut& o, hipStream_t s) {
  const int E = d->n_experts, k = d->top_k, H = d->hidden;
  bool two = false;
  TRY(timed(0, s, "router logits", [&](const KTime& kt) {
    return launch_route_logits(x, T, H, wr, bias, E, k, o.logits, o.wsq, o.ids, o.tw, o.xsum, o.x16, o.segs, s,
                               &two, kt);
  }));
  if (!two) {
    // Few tokens: exact logits are already there; top-k + metadata in one launch.
    return timed(2, s, "top-k + routing metadata", [&](const KTime& kt) {
      return launch_topk_meta(o.logits, T, E, k, o.ids, o.tw, tile_rows(d), d->shared_inter > 0 ? 1 : 0,
                              o.counts, o.offsets, o.sorted, o.tiles, o.n_tiles, o.active, o.n_active, o.inv,
                              o.sched, s, kt);
    });
  }
  TRY(timed(1, s, "top-k", [&](const KTime& kt) {
    return launch_route_select(x, T, H, wr, bias, E, k, o.logits, o.wsq, o.ids, o.tw, o.x16, o.segs, s, kt);
  }));
  TRY(timed(2, s, "routing metadata", [&](const KTime& kt) {
    return launch_meta(o.ids, T, k, E, tile_rows(d), d->shared_inter > 0 ? 1 : 0, max_long_tiles(d), o.counts,
                       o.offsets, o.sorted, o.tiles, o.n_tiles, o.active, o.n_active, o.inv, o.sched, o.segs,
                       s, kt);  // segment counts taken by the exact top-k
  }));
  return MOE_OK;
}

void* area_base(void* ws, const Ws& w, int area) { return static_cast<char*>(ws) + (area ? w.span : 0); }

RouteOut ws_route(void* ws, const Ws& w) {
  RouteOut o;
  o.logits = at<float>(ws, w.logits);
  o.wsq = at<double>(ws, w.wnorm);
  o.xsum = at<float>(ws, w.xsum);
  o.x16 = at<uint16_t>(ws, w.x16);
  o.ids = at<int32_t>(ws, w.ids);
  o.tw = at<float>(ws, w.tw);
  o.counts = at<int32_t>(ws, w.counts);
  o.offsets = at<int32_t>(ws, w.offsets);
  o.sorted = at<int32_t>(ws, w.sorted);
  o.inv = at<int32_t>(ws, w.inv);
  o.tiles = at<int32_t>(ws, w.tiles);
  o.sched = at<int32_t>(ws, w.sched);
  o.n_tiles = at<int32_t>(ws, w.n_tiles);
  o.active = at<int32_t>(ws, w.active);
  o.n_active = at<int32_t>(ws, w.n_active);
  o.segs = at<int32_t>(ws, w.segs);
  return o;
}

ChunkArgs chunk_args(const moe_layer_desc* d, const uint16_t* x, int Tc, const RouteOut& o, void* ws,
                     const Ws& w, float* y) {
  ChunkArgs C;
  C.x = x;
  C.x16 = o.x16;
  C.T = Tc;
  C.Tk = Tc * d->top_k;
  C.xsum = o.xsum;
  C.ids = o.ids;
  C.tw = o.tw;
  C.counts = o.counts;
  C.offsets = o.offsets;
  C.sorted = o.sorted;
  C.inv = o.inv;
  C.tiles = o.tiles;
  C.sched = o.sched;
  C.n_tiles = o.n_tiles;
  C.active = o.active;
  C.n_active = o.n_active;
  C.hbuf = at<uint16_t>(ws, w.hbuf);
  C.obuf = at<uint16_t>(ws, w.obuf);
  C.y = y;
  C.Imax = imax(d);
  return C;
}

moe_status forward_checks(const moe_layer_desc* d, const void* packed, const float* wr,
                          const uint16_t* x, int32_t T, const float* y, const void* ws,
                          size_t ws_bytes) {
  TRY(validate_desc(d));
  if (T < 0) return fail(MOE_ERR_INVALID_ARGUMENT, "T must be >= 0 (got %d)", T);
  if (T == 0) return MOE_OK;
  if (!packed || !wr || !x || !y || !ws) return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  const int64_t Tc = T < d->max_chunk ? T : d->max_chunk;
  const size_t need = ws_layout(d, Tc).total;
  if (ws_bytes < need)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < required %zu", ws_bytes, need);
  return MOE_OK;
}

// The GEMMs of one routed chunk, on stream s (chunk_combine follows them).
moe_status chunk_gemms(const moe_layer_desc* d, const LayerArgs& L, const uint16_t* x, int Tc, const RouteOut& o,
                       float* y, void* area, void* ws, const Ws& w, hipStream_t s) {
  const ChunkArgs C = chunk_args(d, x, Tc, o, area, w, y);
  LayerArgs Lc = L;
  if (d->dequant_pass) {
    Lc.wdq = at<uint8_t>(ws, w.wdq);
    TRY(timed(8, s, "separate dequant", [&](const KTime& kt) { return launch_dequant_active(Lc, C, s, kt); }));
  }
  int mt = (int)max_sched_for(d, Tc);
  if (d->host_sync_routing) {
    // Measurement of the host round trip: read the schedule's entry count
    // back, wait for it, and size the GEMM grids from it.
    int32_t hdr[4] = {0, 0, 0, 0};
    hipError_t e = hipMemcpyAsync(hdr, o.sched, sizeof(hdr), hipMemcpyDeviceToHost, s);
    if (e == hipSuccess) e = hipStreamSynchronize(s);
    if (e != hipSuccess) return fail(MOE_ERR_HIP, "routing read-back: %s", hipGetErrorString(e));
    if (hdr[0] < 0 || hdr[0] > mt) return fail(MOE_ERR_HIP, "routing read-back: bad entry count %d", hdr[0]);
    mt = hdr[0];
  }
  TRY(timed(3, s, "gate/up GEMM", [&](const KTime& kt) { return launch_gateup_gemm(Lc, C, mt, s, kt); }));
  TRY(timed(4, s, "down GEMM", [&](const KTime& kt) { return launch_down_gemm(Lc, C, mt, s, kt); }));
  return MOE_OK;
}

// The per-token combine of one chunk whose down GEMM is ordered before it on stream s.
moe_status chunk_combine(const moe_layer_desc* d, const LayerArgs& L, const uint16_t* x, int Tc, const RouteOut& o,
                         float* y, void* area, const Ws& w, hipStream_t s) {
  const ChunkArgs C = chunk_args(d, x, Tc, o, area, w, y);
  TRY(timed(7, s, "combine", [&](const KTime& kt) { return launch_combine(L, C, s, kt); }));
  return MOE_OK;
}

// ---- the second stream ----------------------------------------------------------
// Per device, a second stream (non-blocking, default priority) that runs every
// other chunk beside the caller's stream.  Events without timing order the two
// streams; they come from a per-device pool and go back to it once every wait
// on them is enqueued (a wait takes the event's state at the time it is
// enqueued).
std::mutex g_side_mu;
hipStream_t g_side[64];
std::vector<hipEvent_t> g_sync_pool[64];

struct SyncEvents {
  int dev = 0;
  std::vector<hipEvent_t> used;
  ~SyncEvents() {
    std::lock_guard<std::mutex> lk(g_side_mu);
    for (hipEvent_t e : used) g_sync_pool[dev].push_back(e);
  }
  moe_status get(hipEvent_t* out) {
    {
      std::lock_guard<std::mutex> lk(g_side_mu);
      if (!g_sync_pool[dev].empty()) {
        *out = g_sync_pool[dev].back();
        g_sync_pool[dev].pop_back();
        used.push_back(*out);
        return MOE_OK;
      }
    }
    hipError_t e = hipEventCreateWithFlags(out, hipEventDisableTiming);
    if (e != hipSuccess) return fail(MOE_ERR_HIP, "hipEventCreateWithFlags: %s", hipGetErrorString(e));
    used.push_back(*out);
    return MOE_OK;
  }
  // Stream `waiter` waits for what is enqueued on `src` so far.
  moe_status order(hipStream_t src, hipStream_t waiter) {
    hipEvent_t ev = nullptr;
    TRY(get(&ev));
    hipError_t e = hipEventRecord(ev, src);
    if (e == hipSuccess) e = hipStreamWaitEvent(waiter, ev, 0);
    if (e != hipSuccess) return fail(MOE_ERR_HIP, "stream ordering: %s", hipGetErrorString(e));
    return MOE_OK;
  }
};

moe_status side_stream(int* dev_out, hipStream_t* out) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(MOE_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
  if (dev < 0 || dev >= 64) return fail(MOE_ERR_DEVICE_UNSUPPORTED, "device index %d out of range", dev);
  std::lock_guard<std::mutex> lk(g_side_mu);
  if (!g_side[dev]) {
    hipStream_t st = nullptr;
    e = hipStreamCreateWithFlags(&st, hipStreamNonBlocking);
    if (e != hipSuccess) return fail(MOE_ERR_HIP, "hipStreamCreateWithFlags: %s", hipGetErrorString(e));
    g_side[dev] = st;
  }
  *dev_out = dev;
  *out = g_side[dev];
  return MOE_OK;
}

// ---- decode without allocation (moe_forward_decode_static) -------------------
// The workspace of moe_forward_decode_static: a fixed device array that each
// GPU the library runs on holds until the process ends.  Host code never uses
// the array's name as an address (it is the host-side stand-in); the device
// address is taken once per device with hipGetSymbolAddress, with that device
// current, and kept in g_scratch_ptr.  Every call on one GPU shares the array,
// so calls that overlap on one GPU race.  No decode kernel reads a workspace
// byte it has not written in the same call, so nothing needs clearing.
constexpr size_t kStaticScratchBytes = MOE_STATIC_SCRATCH_BYTES;
static __device__ __align__(256) uint8_t scratch[kStaticScratchBytes];
std::mutex g_scratch_mu;
void* g_scratch_ptr[64];

moe_status static_scratch(void** out) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(MOE_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
  if (dev < 0 || dev >= 64) return fail(MOE_ERR_DEVICE_UNSUPPORTED, "device index %d out of range", dev);
  std::lock_guard<std::mutex> lk(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess || !p)
      return fail(MOE_ERR_HIP, "hipGetSymbolAddress(scratch) on device %d: %s", dev, hipGetErrorString(e));
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return MOE_OK;
}

// The grouped GEMM path over T tokens, max_chunk tokens at a time.  With one
// chunk area in the workspace every chunk is routed and run on the caller's
// stream, one after the other.  With two (and more than one chunk), chunks
// alternate between the caller's stream (even chunks, area 0) and the second
// stream (odd chunks, area 1), so two chunks are in flight at once: the
// routing of one runs beside the other's GEMMs, and the GEMMs of both share
// the device.  The tokens of different chunks are independent, so the only
// orderings are the call's inputs before the second stream's work, each
// stream's own order for the reuse of its area, and the second stream's work
// joined to the caller's stream before the call returns.
moe_status prefill_loop(const moe_layer_desc* d, const void* packed, const float* wr, const float* bias,
                        const uint16_t* x, int T, float* y, void* ws, size_t ws_bytes, bool may_overlap,
                        hipStream_t s) {
  const LayerArgs L = layer_args(d, packed);
  const int chunk = d->max_chunk, H = d->hidden;
  const int nch = (T + chunk - 1) / chunk;
  const int64_t Tc0 = T < chunk ? T : chunk;
  auto rows = [&](int c) { return T - c * chunk < chunk ? T - c * chunk : chunk; };
  const Ws w2 = ws_layout(d, Tc0, 2);
  const bool two = nch > 1 && may_overlap && !d->host_sync_routing && !d->dequant_pass && ws_bytes >= w2.total;
  if (!two) {
    const Ws w = ws_layout(d, Tc0);
    const RouteOut o = ws_route(ws, w);
    for (int c = 0; c < nch; c++) {
      const int64_t off = (int64_t)c * chunk * H;
      TRY(run_route(d, x + off, rows(c), wr, bias, o, s));
      TRY(chunk_gemms(d, L, x + off, rows(c), o, y + off, ws, ws, w, s));
      TRY(chunk_combine(d, L, x + off, rows(c), o, y + off, ws, w, s));
    }
    return MOE_OK;
  }
  int dev = 0;
  hipStream_t side = nullptr;
  TRY(side_stream(&dev, &side));
  SyncEvents ev;
  ev.dev = dev;
  TRY(ev.order(s, side));  // the inputs and the workspace's previous users come first
  // When the last chunk runs on the second stream, its combine runs on the
  // caller's stream after an event that follows that chunk's down GEMM: the
  // wait then overlaps the other chunk's combine, and it orders all of the
  // second stream's work before the call's end on the caller's stream, so no
  // separate join is needed.
  const bool last_on_side = (nch - 1) & 1;
  auto body = [&]() -> moe_status {
    for (int c = 0; c < nch; c++) {
      hipStream_t st = c & 1 ? side : s;
      void* area = area_base(ws, w2, c & 1);
      const RouteOut o = ws_route(area, w2);
      const int64_t off = (int64_t)c * chunk * H;
      TRY(run_route(d, x + off, rows(c), wr, bias, o, st));
      TRY(chunk_gemms(d, L, x + off, rows(c), o, y + off, area, ws, w2, st));
      hipStream_t cs = st;
      if (c == nch - 1 && last_on_side) {
        TRY(ev.order(side, s));
        cs = s;
      }
      TRY(chunk_combine(d, L, x + off, rows(c), o, y + off, area, w2, cs));
    }
    return MOE_OK;
  };
  const moe_status st = body();
  if (st != MOE_OK) {
    // Best effort, keeping the first error: leave nothing of the call unjoined.
    hipEvent_t e = nullptr;
    if (hipEventCreateWithFlags(&e, hipEventDisableTiming) == hipSuccess) {
      if (hipEventRecord(e, side) == hipSuccess) (void)hipStreamWaitEvent(s, e, 0);
      (void)hipEventDestroy(e);
    }
    return st;
  }
  return last_on_side ? MOE_OK : ev.order(side, s);
}

// Decode after the argument checks; may_overlap is false for the
// static-scratch entry point, which must not create the routing stream.
moe_status decode_impl(const moe_layer_desc* desc, const void* packed, const float* router_w,
                       const float* logit_bias, const uint16_t* x, int32_t T, float* y, void* ws, size_t ws_bytes,
                       bool may_overlap, void* stream) {
  // T > R* (and always T > 8, the GEMV's largest row count) takes the grouped-GEMM path.
  const int R = desc->gemv_max_rows >= 0 ? desc->gemv_max_rows
                : desc->batch_invariant ? kDefaultGemvMaxRowsBi : kDefaultGemvMaxRows;
  const bool gemv = T <= R && T <= desc->max_chunk && (int64_t)T * desc->hidden <= 32768;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (!gemv) return prefill_loop(desc, packed, router_w, logit_bias, x, T, y, ws, ws_bytes, may_overlap, s);
  const LayerArgs L = layer_args(desc, packed);
  const Ws w = ws_layout(desc, T);
  const RouteOut o = ws_route(ws, w);
  // Exact logits; then the top-k, gate/up and split down projection; then the
  // fixed-order sum of the partial outputs.
  bool two = false;
  float* part = at<float>(ws, w.dpart);
  TRY(timed(0, s, "router logits", [&](const KTime& kt) {
    return launch_route_logits(x, T, desc->hidden, router_w, logit_bias, desc->n_experts, desc->top_k, o.logits,
                               o.wsq, o.ids, o.tw, nullptr, nullptr, nullptr, s, &two, kt);
  }));
  const ChunkArgs C = chunk_args(desc, x, T, o, ws, w, y);
  if (desc->batch_invariant) {
    // The grouped-GEMM path's arithmetic: gate/up into fp16 h rows, then down + combine.
    TRY(timed(5, s, "top-k + gate/up GEMV (grouped-GEMM arithmetic)", [&](const KTime& kt) {
      return launch_gemv_gateup_bi(L, C, o.logits, C.hbuf, o.ids, o.tw, s, kt);
    }));
    TRY(timed(6, s, "down GEMV + combine (grouped-GEMM arithmetic)", [&](const KTime& kt) {
      return launch_gemv_down_bi(L, C, C.hbuf, o.ids, o.tw, s, kt);
    }));
    return MOE_OK;
  }
  TRY(timed(5, s, "top-k + gate/up + split down GEMV", [&](const KTime& kt) {
    return launch_gemv_experts(L, C, o.logits, part, s, kt);
  }));
  TRY(timed(6, s, "partial-output sum", [&](const KTime& kt) { return launch_gemv_reduce(L, C, part, s, kt); }));
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_packed_bytes(const moe_layer_desc* desc, size_t* bytes) {
  TRY(validate_desc(desc));
  if (!bytes) return fail(MOE_ERR_INVALID_ARGUMENT, "bytes is null");
  *bytes = (size_t)blob_geom(desc).total;
  return MOE_OK;
}

moe_status moe_workspace_bytes(const moe_layer_desc* desc, int32_t max_tokens, size_t* bytes) {
  TRY(validate_desc(desc));
  if (!bytes) return fail(MOE_ERR_INVALID_ARGUMENT, "bytes is null");
  if (max_tokens < 0) return fail(MOE_ERR_INVALID_ARGUMENT, "max_tokens must be >= 0");
  const int64_t Tc = max_tokens < desc->max_chunk ? max_tokens : desc->max_chunk;
  // Beyond one chunk, room for a second chunk area (two chunks in flight).
  *bytes = ws_layout(desc, Tc > 0 ? Tc : 1, max_tokens > desc->max_chunk ? 2 : 1).total;
  return MOE_OK;
}

moe_status moe_max_tiles(const moe_layer_desc* desc, int32_t T, int32_t* n) {
  TRY(validate_desc(desc));
  if (!n) return fail(MOE_ERR_INVALID_ARGUMENT, "n is null");
  if (T < 0) return fail(MOE_ERR_INVALID_ARGUMENT, "T must be >= 0");
  *n = (int32_t)max_tiles_for(desc, T);
  return MOE_OK;
}

int32_t moe_default_gemv_max_rows(void) { return kDefaultGemvMaxRows; }

moe_status moe_pack_weights(const moe_layer_desc* desc, moe_qmatrix gate, moe_qmatrix up,
                            moe_qmatrix down, moe_qmatrix sh_gate, moe_qmatrix sh_up,
                            moe_qmatrix sh_down, void* packed, size_t packed_bytes, void* stream) {
  TRY(validate_desc(desc));
  const Blob b = blob_geom(desc);
  auto bad = [](const moe_qmatrix& m) { return !m.codes || !m.scales || !m.biases; };
  if (!packed || bad(gate) || bad(up) || bad(down))
    return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (desc->shared_inter > 0 && (bad(sh_gate) || bad(sh_up) || bad(sh_down)))
    return fail(MOE_ERR_INVALID_ARGUMENT, "null shared-expert pointer");
  if (packed_bytes < (size_t)b.total)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "packed buffer %zu bytes < required %lld", packed_bytes,
                (long long)b.total);
  TRY(check_device());
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int H = desc->hidden, I = desc->inter, Is = desc->shared_inter, E = desc->n_experts;
  uint8_t* dst = static_cast<uint8_t*>(packed);
  auto pack = [&](const moe_qmatrix& m, int M, int N, int K, int64_t base, int64_t stride_m,
                  int64_t stride_nb, int64_t stride_g) -> moe_status {
    PackArgs P{m.codes, m.scales, m.biases, dst, M, N, K, base, stride_m, stride_nb, stride_g,
               reinterpret_cast<int32_t*>(dst + b.trailer)};
    hipError_t e = launch_pack(P, s);
    if (e != hipSuccess) return fail(MOE_ERR_HIP, "pack launch failed: %s", hipGetErrorString(e));
    return MOE_OK;
  };
  {
    hipError_t e = launch_pack_trailer(dst + b.trailer, s);
    if (e != hipSuccess) return fail(MOE_ERR_HIP, "pack launch failed: %s", hipGetErrorString(e));
  }
  const int64_t gu_nb = (int64_t)(H / 64) * 2 * kBlockBytes, gu_g = 2 * kBlockBytes;
  TRY(pack(gate, E, I, H, 0, b.expert_bytes, gu_nb, gu_g));
  TRY(pack(up, E, I, H, kBlockBytes, b.expert_bytes, gu_nb, gu_g));
  TRY(pack(down, E, H, I, b.gateup_bytes, b.expert_bytes, (int64_t)(I / 64) * kBlockBytes, kBlockBytes));
  if (Is > 0) {
    TRY(pack(sh_gate, 1, Is, H, b.shared_base, 0, gu_nb, gu_g));
    TRY(pack(sh_up, 1, Is, H, b.shared_base + kBlockBytes, 0, gu_nb, gu_g));
    TRY(pack(sh_down, 1, H, Is, b.shared_base + b.shared_gateup_bytes, 0,
             (int64_t)(Is / 64) * kBlockBytes, kBlockBytes));
  }
  return MOE_OK;
}

moe_status moe_route(const moe_layer_desc* desc, const uint16_t* x, int32_t T, const float* router_w,
                     const float* logit_bias, const moe_routing* out, void* ws, size_t ws_bytes,
                     void* stream) {
  TRY(validate_desc(desc));
  if (T < 0 || T > desc->max_chunk)
    return fail(MOE_ERR_INVALID_ARGUMENT, "T must be in 0..max_chunk (got %d)", T);
  if (T == 0) return MOE_OK;
  if (!x || !router_w || !out || !ws) return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (!out->topk_ids || !out->topk_weights || !out->expert_counts || !out->expert_offsets ||
      !out->sorted_assign || !out->tile_map || !out->n_tiles)
    return fail(MOE_ERR_INVALID_ARGUMENT, "null routing output pointer");
  const Ws w = ws_layout(desc, T);
  if (ws_bytes < w.total)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < required %zu", ws_bytes, w.total);
  TRY(check_device());
  RouteOut o = ws_route(ws, w);
  o.ids = out->topk_ids;
  o.tw = out->topk_weights;
  o.counts = out->expert_counts;
  o.offsets = out->expert_offsets;
  o.sorted = out->sorted_assign;
  o.tiles = out->tile_map;
  o.n_tiles = out->n_tiles;
  return run_route(desc, x, T, router_w, logit_bias, o, static_cast<hipStream_t>(stream));
}

moe_status moe_forward_prefill(const moe_layer_desc* desc, const void* packed, const float* router_w,
                               const float* logit_bias, const uint16_t* x, int32_t T, float* y, void* ws,
                               size_t ws_bytes, void* stream) {
  TRY(forward_checks(desc, packed, router_w, x, T, y, ws, ws_bytes));
  if (T == 0) return MOE_OK;
  TRY(check_device());
  return prefill_loop(desc, packed, router_w, logit_bias, x, T, y, ws, ws_bytes, true,
                      static_cast<hipStream_t>(stream));
}

moe_status moe_forward_decode(const moe_layer_desc* desc, const void* packed, const float* router_w,
                              const float* logit_bias, const uint16_t* x, int32_t T, float* y, void* ws,
                              size_t ws_bytes, void* stream) {
  TRY(forward_checks(desc, packed, router_w, x, T, y, ws, ws_bytes));
  if (T == 0) return MOE_OK;
  TRY(check_device());
  return decode_impl(desc, packed, router_w, logit_bias, x, T, y, ws, ws_bytes, true, stream);
}

moe_status moe_forward_decode_static(const moe_layer_desc* desc, const void* packed, const float* router_w,
                                     const float* logit_bias, const uint16_t* x, int32_t T, float* y,
                                     void* stream) {
  TRY(validate_desc(desc));
  if (T < 0) return fail(MOE_ERR_INVALID_ARGUMENT, "T must be >= 0 (got %d)", T);
  if (T == 0) return MOE_OK;
  if (desc->host_sync_routing || desc->dequant_pass)
    return fail(MOE_ERR_INVALID_ARGUMENT, "the static-scratch decode takes neither host_sync_routing nor dequant_pass");
  if (!packed || !router_w || !x || !y) return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  const size_t need = ws_layout(desc, T < desc->max_chunk ? T : desc->max_chunk).total;
  if (need > kStaticScratchBytes)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "this layer needs %zu bytes of scratch at T=%d; the static scratch holds %zu",
                need, T, kStaticScratchBytes);
  TRY(check_device());
  void* ws = nullptr;
  TRY(static_scratch(&ws));
  TRY(forward_checks(desc, packed, router_w, x, T, y, ws, kStaticScratchBytes));
  return decode_impl(desc, packed, router_w, logit_bias, x, T, y, ws, kStaticScratchBytes, false, stream);
}

// The checks that both directions of the 4-bit storage share; `rows` = 0 needs no pointers.
static moe_status mx4_row_args(const void* wide, int32_t type, int64_t rows, int64_t cols, int64_t ld,
                               const uint8_t* codes, const uint8_t* scales, Mx4RowArgs* A) {
  if (type != MOE_F32 && type != MOE_BF16)
    return fail(MOE_ERR_INVALID_ARGUMENT, "the values must be MOE_F32 or MOE_BF16 (got type %d)", type);
  if (rows < 0) return fail(MOE_ERR_INVALID_ARGUMENT, "rows must be >= 0 (got %lld)", (long long)rows);
  if (cols <= 0 || cols % 32 || cols > (int64_t)1 << 24)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "cols must be a positive multiple of 32 <= 2^24 (got %lld)", (long long)cols);
  if (rows > ((int64_t)1 << 46) / cols)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "%lld rows of %lld values are too many", (long long)rows, (long long)cols);
  if (ld < cols || ld > (int64_t)1 << 40)
    return fail(MOE_ERR_INVALID_ARGUMENT, "the row stride (%lld) is less than cols (%lld), or over 2^40", (long long)ld,
                (long long)cols);
  if (rows && (!wide || !codes || !scales)) return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (reinterpret_cast<uintptr_t>(codes) & 15)
    return fail(MOE_ERR_INVALID_ARGUMENT, "codes must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(wide) & (type == MOE_F32 ? 3 : 1))
    return fail(MOE_ERR_INVALID_ARGUMENT, "the values are not aligned to their type");
  *A = Mx4RowArgs{const_cast<void*>(wide), const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales), rows, cols, ld,
                  type == MOE_F32};
  return MOE_OK;
}

moe_status moe_mx4_quantize(const void* x, int32_t x_type, int64_t rows, int64_t cols, int64_t ldx, uint8_t* codes,
                            uint8_t* scales, void* stream) {
  Mx4RowArgs A;
  TRY(mx4_row_args(x, x_type, rows, cols, ldx, codes, scales, &A));
  if (rows == 0) return MOE_OK;
  TRY(check_device());
  hipStream_t s = static_cast<hipStream_t>(stream);
  return timed(11, s, "4-bit quantisation", [&](const KTime& kt) { return launch_mx4_quantize(A, s, kt); });
}

moe_status moe_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* y,
                              int32_t y_type, int64_t ldy, void* stream) {
  Mx4RowArgs A;
  TRY(mx4_row_args(y, y_type, rows, cols, ldy, codes, scales, &A));
  if (rows == 0) return MOE_OK;
  TRY(check_device());
  hipStream_t s = static_cast<hipStream_t>(stream);
  return timed(12, s, "4-bit read-back", [&](const KTime& kt) { return launch_mx4_dequantize(A, s, kt); });
}

static thread_local const char* g_experts_kernel = "";  // of the last product

moe_status moe_mx4_experts(const moe_mx4_desc* d, const uint8_t* w_codes, const uint8_t* w_scales, const void* x,
                           const uint8_t* x_scales, int32_t x_rows, const int32_t* expert_offsets, int32_t rows,
                           const int32_t* src_rows, int32_t src_div, const int32_t* dst_rows, const float* row_scale,
                           void* y, uint8_t* y_scales, int32_t y_rows, void* stream) {
  if (!d) return fail(MOE_ERR_INVALID_ARGUMENT, "desc is null");
  if (d->n_experts < 1 || d->n_experts > 512)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "n_experts must be in 1..512 (got %d)", d->n_experts);
  if (d->k <= 0 || d->k % 32 || d->k > 65536)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "k must be a positive multiple of 32 <= 65536 (got %d)", d->k);
  if (d->n <= 0 || d->n > 65536) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "n must be in 1..65536 (got %d)", d->n);
  if (d->x_type != MOE_BF16 && d->x_type != MOE_MX4)
    return fail(MOE_ERR_INVALID_ARGUMENT, "x_type must be MOE_BF16 or MOE_MX4 (got %d)", d->x_type);
  if (d->y_type < MOE_F32 || d->y_type > MOE_MX4)
    return fail(MOE_ERR_INVALID_ARGUMENT, "y_type must be MOE_F32, MOE_BF16 or MOE_MX4 (got %d)", d->y_type);
  if (d->swiglu != 0 && d->swiglu != 1)
    return fail(MOE_ERR_INVALID_ARGUMENT, "swiglu must be 0 or 1 (got %d)", d->swiglu);
  if (d->swiglu && d->n % 2) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "n must be even with swiglu (got %d)", d->n);
  const int n_out = d->swiglu ? d->n / 2 : d->n;
  if (d->y_type == MOE_MX4 && n_out % 32)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "a MOE_MX4 y needs a multiple of 32 columns (got %d)", n_out);
  if (rows < 0 || rows > 1 << 24) return fail(MOE_ERR_INVALID_ARGUMENT, "rows must be in 0..2^24 (got %d)", rows);
  if (rows == 0) return MOE_OK;
  if (x_rows < 1 || y_rows < 1)
    return fail(MOE_ERR_INVALID_ARGUMENT, "x_rows and y_rows must be positive (got %d, %d)", x_rows, y_rows);
  if (src_div < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "src_div must be positive (got %d)", src_div);
  if (!w_codes || !w_scales || !x || !expert_offsets || !y || (d->x_type == MOE_MX4 && !x_scales) ||
      (d->y_type == MOE_MX4 && !y_scales))
    return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (!src_rows && rows > x_rows)
    return fail(MOE_ERR_INVALID_ARGUMENT, "without src_rows x needs a row per position (%d < %d)", x_rows, rows);
  if (!dst_rows && rows > y_rows)
    return fail(MOE_ERR_INVALID_ARGUMENT, "without dst_rows y needs a row per position (%d < %d)", y_rows, rows);
  if ((reinterpret_cast<uintptr_t>(w_codes) | reinterpret_cast<uintptr_t>(x)) & 15)
    return fail(MOE_ERR_INVALID_ARGUMENT, "w_codes and x must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(y) & (d->y_type == MOE_MX4 ? 15 : d->y_type == MOE_F32 ? 3 : 1))
    return fail(MOE_ERR_INVALID_ARGUMENT, "y must be aligned to its type, codes to 16 bytes");
  TRY(check_device());
  Mx4ExpertArgs A{w_codes,   w_scales, x,        x_scales,  expert_offsets, src_rows, dst_rows,
                  row_scale, y,        y_scales, d->n_experts, d->n,        d->k,     rows,
                  x_rows,    y_rows,   src_div,  d->y_type, d->x_type == MOE_MX4, d->swiglu == 1, divisor(src_div)};
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int cus = device_cus();
  const MxKernel m = mx4_experts_kernel(A, cus);
  g_experts_kernel = mx4_experts_kernel_name(m);
  return timed(13, s, "4-bit expert product", [&](const KTime& kt) { return launch_mx4_experts(A, m, cus, s, kt); });
}

const char* moe_mx4_experts_kernel(void) { return g_experts_kernel; }

static moe_status balance_shape(int32_t T, int32_t E, int32_t k) {
  if (T < 0) return fail(MOE_ERR_INVALID_ARGUMENT, "T must be >= 0 (got %d)", T);
  if (E < 1 || E > 512) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "n_experts must be in 1..512 (got %d)", E);
  if (k < 1 || k > 16) return fail(MOE_ERR_INVALID_ARGUMENT, "top_k must be in 1..16 (got %d)", k);
  if ((int64_t)T * k > 0x7FFFFFFF)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "T * top_k must be below 2^31 (got %d * %d)", T, k);
  return MOE_OK;
}

static moe_status balance_logits(const void* logits, int32_t type) {
  if (type != MOE_F32 && type != MOE_BF16)
    return fail(MOE_ERR_INVALID_ARGUMENT, "the logits must be MOE_F32 or MOE_BF16 (got type %d)", type);
  if (reinterpret_cast<uintptr_t>(logits) & (type == MOE_F32 ? 3 : 1))
    return fail(MOE_ERR_INVALID_ARGUMENT, "the logits are not aligned to their type");
  return MOE_OK;
}

// Carves the forward pass's workspace (base may be null for its size alone).
static size_t balance_ws(int32_t T, int32_t E, void* base, BalanceArgs* A) {
  const int64_t parts = balance_parts(T, E);
  size_t o = 0;
  const size_t done = o; o += al(4);
  const size_t dots = o; o += al((E + 15) / 16 * 8);
  const size_t pz = o; o += al(parts * 8);
  const size_t pn = o; o += al(parts * 4);
  const size_t pc = o; o += al(parts * E * 4);
  const size_t pp = o; o += al(parts * E * 4);
  if (A) {
    A->done = at<int32_t>(base, done);
    A->dots = at<double>(base, dots);
    A->part_z = at<double>(base, pz);
    A->part_n = at<int32_t>(base, pn);
    A->part_count = at<int32_t>(base, pc);
    A->part_p = at<float>(base, pp);
  }
  return o;
}

moe_status moe_balance_loss_workspace_bytes(int32_t T, int32_t n_experts, size_t* bytes) {
  TRY(balance_shape(T, n_experts, 1));
  if (!bytes) return fail(MOE_ERR_INVALID_ARGUMENT, "bytes is null");
  *bytes = balance_ws(T, n_experts, nullptr, nullptr);
  return MOE_OK;
}

moe_status moe_balance_loss_forward(const void* logits, int32_t logits_type, int32_t T, int32_t n_experts,
                                    const int32_t* topk_ids, int32_t top_k, const uint8_t* valid, float balance_coef,
                                    float z_coef, float* losses, int32_t* counts, float* mean_prob, int32_t* n_valid,
                                    void* ws, size_t ws_bytes, void* stream) {
  TRY(balance_shape(T, n_experts, top_k));
  TRY(balance_logits(logits, logits_type));
  if (!losses || !counts || !mean_prob || !n_valid || !ws || (T > 0 && (!logits || !topk_ids)))
    return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  BalanceArgs A{};
  const size_t need = balance_ws(T, n_experts, ws, &A);
  if (ws_bytes < need)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < required %zu", ws_bytes, need);
  if (reinterpret_cast<uintptr_t>(ws) & 7) return fail(MOE_ERR_INVALID_ARGUMENT, "ws must be 8-byte aligned");
  TRY(check_device());
  A.logits = logits;
  A.ids = topk_ids;
  A.valid = valid;
  A.T = T;
  A.E = n_experts;
  A.k = top_k;
  A.balance_coef = balance_coef;
  A.z_coef = z_coef;
  A.f32 = logits_type == MOE_F32;
  A.losses = losses;
  A.counts = counts;
  A.mean_prob = mean_prob;
  A.n_valid = n_valid;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return timed(14, s, "balance loss", [&](const KTime& kt) { return launch_balance_forward(A, s, kt); });
}

moe_status moe_balance_loss_backward(const void* logits, int32_t logits_type, int32_t T, int32_t n_experts,
                                     int32_t top_k, const uint8_t* valid, float balance_coef, float z_coef,
                                     const int32_t* counts, const int32_t* n_valid, const float* grad_loss,
                                     void* dlogits, void* stream) {
  TRY(balance_shape(T, n_experts, top_k));
  TRY(balance_logits(logits, logits_type));
  TRY(balance_logits(dlogits, logits_type));
  if (T == 0) return MOE_OK;
  if (!logits || !counts || !n_valid || !dlogits) return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  TRY(check_device());
  BalanceArgs A{};
  A.logits = logits;
  A.valid = valid;
  A.T = T;
  A.E = n_experts;
  A.k = top_k;
  A.balance_coef = balance_coef;
  A.z_coef = z_coef;
  A.f32 = logits_type == MOE_F32;
  A.counts = const_cast<int32_t*>(counts);
  A.n_valid = const_cast<int32_t*>(n_valid);
  A.grad = grad_loss;
  A.dlogits = dlogits;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return timed(15, s, "balance loss gradient", [&](const KTime& kt) { return launch_balance_backward(A, s, kt); });
}

static moe_status value_type(const void* p, int32_t type, const char* name) {
  if (type != MOE_F32 && type != MOE_BF16)
    return fail(MOE_ERR_INVALID_ARGUMENT, "%s must be MOE_F32 or MOE_BF16 (got type %d)", name, type);
  if (reinterpret_cast<uintptr_t>(p) & (type == MOE_F32 ? 3 : 1))
    return fail(MOE_ERR_INVALID_ARGUMENT, "%s is not aligned to its type", name);
  return MOE_OK;
}

static moe_status select_shape(const moe_select_desc* d, int32_t T) {
  if (!d) return fail(MOE_ERR_INVALID_ARGUMENT, "desc is null");
  TRY(balance_shape(T, d->n_experts, d->top_k));
  if (d->scores != MOE_SOFTMAX && d->scores != MOE_SIGMOID)
    return fail(MOE_ERR_INVALID_ARGUMENT, "scores must be MOE_SOFTMAX or MOE_SIGMOID (got %d)", d->scores);
  if (d->n_groups < 1 || d->n_groups > 64 || d->n_experts % d->n_groups)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "n_groups must be in 1..64 and divide n_experts (got %d of %d)", d->n_groups,
                d->n_experts);
  if (d->top_groups < 1 || d->top_groups > d->n_groups)
    return fail(MOE_ERR_INVALID_ARGUMENT, "top_groups must be in 1..n_groups (got %d of %d)", d->top_groups, d->n_groups);
  if (d->group_best != 1 && d->group_best != 2)
    return fail(MOE_ERR_INVALID_ARGUMENT, "group_best must be 1 or 2 (got %d)", d->group_best);
  if (d->top_k > d->top_groups * (d->n_experts / d->n_groups))
    return fail(MOE_ERR_INVALID_ARGUMENT, "top_k (%d) exceeds the %d experts of top_groups groups", d->top_k,
                d->top_groups * (d->n_experts / d->n_groups));
  if (d->renormalise != 0 && d->renormalise != 1)
    return fail(MOE_ERR_INVALID_ARGUMENT, "renormalise must be 0 or 1 (got %d)", d->renormalise);
  if (!(d->scale - d->scale == 0.f) || d->scale == 0.f)
    return fail(MOE_ERR_INVALID_ARGUMENT, "scale must be finite and not zero");
  return MOE_OK;
}

static SelectArgs select_args(const moe_select_desc* d, const void* logits, int32_t type, int32_t T) {
  SelectArgs A{};
  A.logits = logits;
  A.T = T;
  A.E = d->n_experts;
  A.k = d->top_k;
  // Groups that all stay leave every expert to choose from.
  A.groups = d->top_groups == d->n_groups ? 1 : d->n_groups;
  A.per = d->n_experts / A.groups;
  A.top_groups = d->top_groups;
  A.best = d->group_best;
  A.f32 = type == MOE_F32;
  A.softmax = d->scores == MOE_SOFTMAX;
  A.renorm = d->renormalise == 1;
  A.scale = d->scale;
  return A;
}

static moe_status sort_ws(size_t need, void* ws, size_t ws_bytes) {
  if (ws_bytes < need) return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < required %zu", ws_bytes, need);
  if (need && !ws) return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (reinterpret_cast<uintptr_t>(ws) & 15) return fail(MOE_ERR_INVALID_ARGUMENT, "ws must be 16-byte aligned");
  return MOE_OK;
}

static size_t sort_bytes(int parts, int32_t E) { return al((size_t)parts * E * 4); }

moe_status moe_select_workspace_bytes(int32_t T, int32_t n_experts, int32_t top_k, size_t* bytes) {
  TRY(balance_shape(T, n_experts, top_k));
  if (!bytes) return fail(MOE_ERR_INVALID_ARGUMENT, "bytes is null");
  *bytes = sort_bytes(select_parts(T), n_experts);
  return MOE_OK;
}

moe_status moe_select_forward(const moe_select_desc* d, const void* logits, int32_t logits_type, int32_t T,
                              const float* bias, const uint8_t* valid, int32_t* topk_ids, float* topk_weights,
                              int32_t* expert_counts, int32_t* expert_offsets, int32_t* sorted_assign, void* ws,
                              size_t ws_bytes, void* stream) {
  TRY(select_shape(d, T));
  TRY(value_type(logits, logits_type, "logits"));
  const bool order = expert_counts || expert_offsets || sorted_assign;
  if (T > 0 && (!logits || !topk_ids || !topk_weights)) return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (order && (!expert_counts || !expert_offsets || (T > 0 && !sorted_assign)))
    return fail(MOE_ERR_INVALID_ARGUMENT, "expert_counts, expert_offsets and sorted_assign go together");
  if (order) TRY(sort_ws(sort_bytes(select_parts(T), d->n_experts), ws, ws_bytes));
  if (T == 0 && !order) return MOE_OK;
  TRY(check_device());
  SelectArgs A = select_args(d, logits, logits_type, T);
  A.bias = bias;
  A.valid = valid;
  A.ids = topk_ids;
  A.weights = topk_weights;
  SortArgs S{};
  if (order) {
    S.ids = topk_ids;
    S.n = (int64_t)T * d->top_k;
    S.E = d->n_experts;
    S.counts = expert_counts;
    S.offsets = expert_offsets;
    S.sorted = sorted_assign;
    S.part_count = static_cast<int32_t*>(ws);
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  return timed(16, s, "routing from scores", [&](const KTime& kt) { return launch_select_forward(A, S, order, s, kt); });
}

moe_status moe_select_backward(const moe_select_desc* d, const void* logits, int32_t logits_type, int32_t T,
                               const int32_t* topk_ids, const float* topk_weights, const float* dweights,
                               const void* base, void* dlogits, void* stream) {
  TRY(select_shape(d, T));
  TRY(value_type(logits, logits_type, "logits"));
  TRY(value_type(base, logits_type, "base"));
  TRY(value_type(dlogits, logits_type, "dlogits"));
  if (T == 0) return MOE_OK;
  if (!logits || !topk_ids || !topk_weights || !dweights || !dlogits)
    return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (base == logits) return fail(MOE_ERR_INVALID_ARGUMENT, "base must not be the logits");
  TRY(check_device());
  SelectArgs A = select_args(d, logits, logits_type, T);
  A.ids = const_cast<int32_t*>(topk_ids);
  A.weights = const_cast<float*>(topk_weights);
  A.dweights = dweights;
  A.base = base;
  A.dlogits = dlogits;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return timed(17, s, "routing gradient", [&](const KTime& kt) { return launch_select_backward(A, s, kt); });
}

static moe_status sort_shape(int32_t n, int32_t E) {
  if (n < 0) return fail(MOE_ERR_INVALID_ARGUMENT, "n must be >= 0 (got %d)", n);
  if (E < 1 || E > 512) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "n_experts must be in 1..512 (got %d)", E);
  return MOE_OK;
}

moe_status moe_sort_workspace_bytes(int32_t n, int32_t n_experts, size_t* bytes) {
  TRY(sort_shape(n, n_experts));
  if (!bytes) return fail(MOE_ERR_INVALID_ARGUMENT, "bytes is null");
  *bytes = sort_bytes(sort_parts(n), n_experts);
  return MOE_OK;
}

moe_status moe_sort_assignments(const int32_t* ids, int32_t n, int32_t n_experts, int32_t* expert_counts,
                                int32_t* expert_offsets, int32_t* sorted_assign, void* ws, size_t ws_bytes,
                                void* stream) {
  TRY(sort_shape(n, n_experts));
  if (!expert_counts || !expert_offsets || (n > 0 && (!ids || !sorted_assign)))
    return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  TRY(sort_ws(sort_bytes(sort_parts(n), n_experts), ws, ws_bytes));
  TRY(check_device());
  SortArgs S{};
  S.ids = ids;
  S.n = n;
  S.E = n_experts;
  S.counts = expert_counts;
  S.offsets = expert_offsets;
  S.sorted = sorted_assign;
  S.part_count = static_cast<int32_t*>(ws);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return timed(18, s, "order by expert", [&](const KTime& kt) { return launch_sort(S, s, kt); });
}

static moe_status combine_shape(int32_t T, int32_t k, int32_t width) {
  if (T < 0) return fail(MOE_ERR_INVALID_ARGUMENT, "T must be >= 0 (got %d)", T);
  if (k < 1 || k > 16) return fail(MOE_ERR_INVALID_ARGUMENT, "k must be in 1..16 (got %d)", k);
  if (width < 1 || width > 1 << 24)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "width must be in 1..2^24 (got %d)", width);
  if ((int64_t)T * k > 0x7FFFFFFF)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "T * k must be below 2^31 (got %d * %d)", T, k);
  return MOE_OK;
}

moe_status moe_combine_forward(const void* rows, int32_t rows_type, int32_t T, int32_t k, int32_t width,
                               const int32_t* topk_ids, const float* weights, const void* base, void* y, int32_t y_type,
                               void* stream) {
  TRY(combine_shape(T, k, width));
  TRY(value_type(rows, rows_type, "rows"));
  TRY(value_type(base, y_type, "base"));
  TRY(value_type(y, y_type, "y"));
  if (T == 0) return MOE_OK;
  if (!rows || !y) return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  TRY(check_device());
  CombineArgs A{};
  A.rows = rows;
  A.ids = topk_ids;
  A.weights = weights;
  A.base = base;
  A.y = y;
  A.T = T;
  A.k = k;
  A.H = width;
  A.rows_f32 = rows_type == MOE_F32;
  A.y_f32 = y_type == MOE_F32;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return timed(19, s, "combine", [&](const KTime& kt) { return launch_combine_forward(A, s, kt); });
}

moe_status moe_combine_backward(const void* dy, int32_t y_type, const void* rows, int32_t rows_type, int32_t T, int32_t k,
                                int32_t width, const int32_t* topk_ids, const float* weights, void* drows, float* dweights,
                                void* stream) {
  TRY(combine_shape(T, k, width));
  TRY(value_type(dy, y_type, "dy"));
  TRY(value_type(rows, rows_type, "rows"));
  TRY(value_type(drows, rows_type, "drows"));
  if (T == 0 || (!drows && !dweights)) return MOE_OK;
  if (!dy || (dweights && !rows)) return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  TRY(check_device());
  CombineArgs A{};
  A.rows = rows;
  A.ids = topk_ids;
  A.weights = weights;
  A.T = T;
  A.k = k;
  A.H = width;
  A.rows_f32 = rows_type == MOE_F32;
  A.y_f32 = y_type == MOE_F32;
  A.dy = dy;
  A.drows = drows;
  A.dweights = dweights;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return timed(20, s, "combine gradient", [&](const KTime& kt) { return launch_combine_backward(A, s, kt); });
}

static moe_status adapter_shape(const moe_adapter_desc* d, int32_t rows) {
  if (!d) return fail(MOE_ERR_INVALID_ARGUMENT, "desc is null");
  if (d->n_adapters < 1 || d->n_adapters > 512)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "n_adapters must be in 1..512 (got %d)", d->n_adapters);
  if (d->rank < 1 || d->rank > 128) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "rank must be in 1..128 (got %d)", d->rank);
  if (d->n_in < 1 || d->n_in > 65536 || d->n_out < 1 || d->n_out > 65536)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "n_in and n_out must be in 1..65536 (got %d, %d)", d->n_in, d->n_out);
  if (d->y_type != MOE_F32 && d->y_type != MOE_BF16)
    return fail(MOE_ERR_INVALID_ARGUMENT, "y_type must be MOE_F32 or MOE_BF16 (got %d)", d->y_type);
  if (rows < 0 || rows > 1 << 24) return fail(MOE_ERR_INVALID_ARGUMENT, "rows must be in 0..2^24 (got %d)", rows);
  return MOE_OK;
}

// What both directions check of the positions and their rows (rows > 0).
static moe_status adapter_args(const moe_adapter_desc* d, const uint16_t* a, const uint16_t* b, const float* scales,
                               const uint16_t* x, int32_t x_rows, const int32_t* offsets, int32_t rows,
                               const int32_t* src_rows, int32_t src_div, const int32_t* dst_rows, int32_t y_rows,
                               AdapterArgs* A) {
  if (x_rows < 1 || y_rows < 1)
    return fail(MOE_ERR_INVALID_ARGUMENT, "x_rows and y_rows must be positive (got %d, %d)", x_rows, y_rows);
  if (src_div < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "src_div must be positive (got %d)", src_div);
  if (!a || !b || !x || !offsets) return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  if ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(x)) & 1)
    return fail(MOE_ERR_INVALID_ARGUMENT, "a, b and x must be aligned to their type");
  if (!src_rows && rows > x_rows)
    return fail(MOE_ERR_INVALID_ARGUMENT, "without src_rows x needs a row per position (%d < %d)", x_rows, rows);
  if (!dst_rows && rows > y_rows)
    return fail(MOE_ERR_INVALID_ARGUMENT, "without dst_rows y needs a row per position (%d < %d)", y_rows, rows);
  A->a = a;
  A->b = b;
  A->scales = scales;
  A->x = x;
  A->offsets = offsets;
  A->src_rows = src_rows;
  A->dst_rows = dst_rows;
  A->n = d->n_adapters;
  A->r = d->rank;
  A->K = d->n_in;
  A->N = d->n_out;
  A->P = rows;
  A->x_rows = x_rows;
  A->y_rows = y_rows;
  A->src_div = src_rows ? src_div : 1;
  A->src = divisor(src_div);
  return MOE_OK;
}

moe_status moe_adapters_forward(const moe_adapter_desc* d, const uint16_t* a, const uint16_t* b, const float* scales,
                                const uint16_t* x, int32_t x_rows, const int32_t* offsets, int32_t rows,
                                const int32_t* src_rows, int32_t src_div, const int32_t* dst_rows, const void* base, void* y,
                                int32_t y_rows, float* h, void* stream) {
  TRY(adapter_shape(d, rows));
  if (rows == 0) return MOE_OK;
  AdapterArgs A{};
  TRY(adapter_args(d, a, b, scales, x, x_rows, offsets, rows, src_rows, src_div, dst_rows, y_rows, &A));
  TRY(value_type(y, d->y_type, "y"));
  TRY(value_type(base, d->y_type, "base"));
  if (!y) return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  TRY(check_device());
  A.base = base;
  A.y = y;
  A.h_out = h;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int cus = device_cus();
  return timed(21, s, "adapters", [&](const KTime& kt) {
    return launch_adapters_forward(A, d->y_type == MOE_F32, cus, s, kt);
  });
}

moe_status moe_adapters_workspace_bytes(const moe_adapter_desc* d, int32_t rows, size_t* bytes) {
  TRY(adapter_shape(d, rows));
  if (!bytes) return fail(MOE_ERR_INVALID_ARGUMENT, "bytes is null");
  *bytes = adapters_thin_bytes(d->rank, rows);
  return MOE_OK;
}

static bool overlap(const void* p, int64_t p_bytes, const void* q, int64_t q_bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + (uint64_t)q_bytes && b < a + (uint64_t)p_bytes;
}

moe_status moe_adapters_backward(const moe_adapter_desc* d, const uint16_t* a, const uint16_t* b, const float* scales,
                                 const uint16_t* x, int32_t x_rows, const float* h, const void* dy, int32_t y_rows,
                                 const int32_t* offsets, int32_t rows, const int32_t* src_rows, int32_t src_div,
                                 const int32_t* dst_rows, const void* base, void* dx, float* da, float* db, void* ws,
                                 size_t ws_bytes, void* stream) {
  TRY(adapter_shape(d, rows));
  if ((da == nullptr) != (db == nullptr)) return fail(MOE_ERR_INVALID_ARGUMENT, "da and db go together");
  if (!dx && base) return fail(MOE_ERR_INVALID_ARGUMENT, "base goes with dx");
  if (!dx && !da) return MOE_OK;
  AdapterArgs A{};
  if (rows > 0) {
    TRY(adapter_args(d, a, b, scales, x, x_rows, offsets, rows, src_rows, src_div, dst_rows, y_rows, &A));
    TRY(value_type(dy, d->y_type, "dy"));
    TRY(value_type(base, MOE_BF16, "base"));
    TRY(value_type(dx, MOE_BF16, "dx"));
    if (!dy || (da && !h)) return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
    size_t need = 0;
    TRY(moe_adapters_workspace_bytes(d, rows, &need));
    if (da) TRY(sort_ws(need, ws, ws_bytes));
    // dx is written while other workgroups still read dy, and before the factors' gradients read x and dy.
    const int64_t row = (int64_t)d->n_in * 2;
    if (dx) {
      const int64_t dx_rows = (int64_t)x_rows * A.src_div, y_size = d->y_type == MOE_F32 ? 4 : 2;
      const int64_t dx_bytes = (dx_rows < 0x7FFFFFFF ? dx_rows : 0x7FFFFFFF) * row;  // rows that an int32 names
      if (overlap(dx, dx_bytes, dy, (int64_t)y_rows * d->n_out * y_size))
        return fail(MOE_ERR_INVALID_ARGUMENT, "dx must not overlap dy");
      if (da && overlap(dx, dx_bytes, x, x_rows * row))
        return fail(MOE_ERR_INVALID_ARGUMENT, "dx must not overlap x where da and db are asked for");
    }
  } else {
    if (!da) return MOE_OK;
    if (!offsets) return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
    A.offsets = offsets;
    A.n = d->n_adapters;
    A.r = d->rank;
    A.K = d->n_in;
    A.N = d->n_out;
  }
  TRY(check_device());
  A.h = h;
  A.dy = dy;
  A.base = base;
  A.dx = dx;
  A.da = da;
  A.db = db;
  A.thin = da ? static_cast<uint16_t*>(ws) : nullptr;
  A.thin_h = adapters_thin_bytes(d->rank, rows) / 4;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int cus = device_cus();
  return timed(22, s, "adapters gradient", [&](const KTime& kt) {
    return launch_adapters_backward(A, d->y_type == MOE_F32, cus, s, kt);
  });
}

const char* moe_status_str(moe_status s) {
  switch (s) {
    case MOE_OK: return "MOE_OK";
    case MOE_ERR_INVALID_ARGUMENT: return "MOE_ERR_INVALID_ARGUMENT";
    case MOE_ERR_UNSUPPORTED_SHAPE: return "MOE_ERR_UNSUPPORTED_SHAPE";
    case MOE_ERR_WORKSPACE_TOO_SMALL: return "MOE_ERR_WORKSPACE_TOO_SMALL";
    case MOE_ERR_HIP: return "MOE_ERR_HIP";
    case MOE_ERR_DEVICE_UNSUPPORTED: return "MOE_ERR_DEVICE_UNSUPPORTED";
  }
  return "MOE_ERR_UNKNOWN";
}

const char* moe_last_error(void) { return g_last_error.c_str(); }

moe_status moe_probe_stream_read(const void* src, size_t bytes, uint32_t* sink, int32_t max_workgroups,
                                 void* stream) {
  if (!src || !sink || max_workgroups < 1 || (reinterpret_cast<uintptr_t>(src) & 15) || (bytes & 15))
    return fail(MOE_ERR_INVALID_ARGUMENT, "probe: null pointer, max_workgroups < 1, or src/bytes not 16-byte aligned");
  TRY(check_device());
  hipStream_t s = static_cast<hipStream_t>(stream);
  return timed(9, s, "stream-read probe",
               [&](const KTime& kt) { return launch_stream_read(src, bytes, sink, max_workgroups, s, kt); });
}

moe_status moe_probe_mfma_rate(int32_t iters, int32_t workgroups, uint64_t* clocks, uint32_t* sink, void* stream) {
  if (iters < 1 || workgroups < 1 || !sink) return fail(MOE_ERR_INVALID_ARGUMENT, "probe: iters, workgroups or sink");
  TRY(check_device());
  hipStream_t s = static_cast<hipStream_t>(stream);
  return timed(10, s, "MFMA-rate probe",
               [&](const KTime& kt) { return launch_mfma_rate(iters, workgroups, clocks, sink, s, kt); });
}

moe_status moe_profile_enable(int32_t mask) {
  g_prof_mask = (uint32_t)mask;
  return MOE_OK;
}

moe_status moe_profile_reset(void) {
  std::lock_guard<std::mutex> lk(g_prof_mu);
  for (auto& p : g_pending) {
    (void)hipEventSynchronize(p.b);
    g_event_pool.push_back(p.a);
    g_event_pool.push_back(p.b);
  }
  g_pending.clear();
  for (int i = 0; i < kNumKernels; i++) {
    g_prof_ms[i] = 0.0;
    g_prof_n[i] = 0;
  }
  return MOE_OK;
}

moe_status moe_profile_read(int32_t kernel_id, double* total_ms, int32_t* launches) {
  if (kernel_id < 0 || kernel_id >= kNumKernels || !total_ms || !launches)
    return fail(MOE_ERR_INVALID_ARGUMENT, "bad profile query");
  std::lock_guard<std::mutex> lk(g_prof_mu);
  for (auto& p : g_pending) {
    hipError_t e = hipEventSynchronize(p.b);
    if (e != hipSuccess) return fail(MOE_ERR_HIP, "hipEventSynchronize: %s", hipGetErrorString(e));
    float ms = 0.f;
    (void)hipEventElapsedTime(&ms, p.a, p.b);
    g_prof_ms[p.kid] += ms;
    g_prof_n[p.kid] += 1;
    g_event_pool.push_back(p.a);
    g_event_pool.push_back(p.b);
  }
  g_pending.clear();
  *total_ms = g_prof_ms[kernel_id];
  *launches = g_prof_n[kernel_id];
  return MOE_OK;
}

}  // extern "C"
