// C ABI of libssd.so: argument validation (before any HIP call) and dispatch
// to the gfx950 kernels.  See include/ssd.h for the contract of every call.
#include "ssd.h"

#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <mutex>

#include "block.h"
#include "bwd.h"
#include "launch.h"

namespace {

thread_local char g_err[512] = {0};
thread_local hipEvent_t* g_events = nullptr;
thread_local int g_n_events = 0;
thread_local int g_timed = 0;

// Records the next timing event (if a registration is active) on `stream`.
struct Timer {
  hipEvent_t* ev;
  int n, i = 0;
  hipStream_t stream;
  Timer(hipStream_t s) : ev(g_events), n(g_n_events), stream(s) {
    g_events = nullptr;
    g_n_events = 0;
    g_timed = 0;
    mark();
  }
  void mark() {
    if (ev && i < n) {
      (void)hipEventRecord(ev[i], stream);
      g_timed = i;
      ++i;
    }
  }
};

ssd_status fail(ssd_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return s;
}

void clear_err() { g_err[0] = 0; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// product of positive sizes with overflow detection (limit 2^62)
// a * b for sizes >= 0 (0 allowed: an empty input), false on a negative size
// or an overflow past 2^62
bool mul_ok(int64_t a, int64_t b, int64_t* out) {
  if (a < 0 || b < 0) return false;
  if (a && b > ((int64_t)1 << 62) / a) return false;
  *out = a * b;
  return true;
}

// A launch holds less than 2^32 threads.  HIP does not refuse a larger one: it
// starts what is left of the threads beyond a multiple of 2^32, without an error.
bool fits(int64_t workgroups, int64_t threads) { return workgroups <= (int64_t)0xffffffff / threads; }

// Workgroups of a prep call, of 256 threads: a wave takes a chunk, or as many as its lanes hold at 4 tokens a
// lane where launch_prep takes them so (N a multiple of 4 and 32-bit sizes).
int64_t prep_workgroups(int64_t BH, int64_t N, int64_t chunk) {
  const int64_t total = BH * ((N + chunk - 1) / chunk);
  const bool by_four = N % 4 == 0 && total < ((int64_t)1 << 31) && BH * N < ((int64_t)1 << 32);
  const int64_t each = 4 * (by_four ? 64 / (chunk / 4) : 1);
  return (total + each - 1) / each;
}

struct Range {
  const char* name;
  const void* p;
  size_t bytes;
};

bool overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

ssd_status check_alias(const Range* outs, int n_out, const Range* ins, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlap(outs[i], ins[j]))
        return fail(SSD_ERR_ALIAS, "output %s overlaps input %s", outs[i].name, ins[j].name);
    for (int j = i + 1; j < n_out; ++j)
      if (overlap(outs[i], outs[j]))
        return fail(SSD_ERR_ALIAS, "outputs %s and %s overlap", outs[i].name, outs[j].name);
  }
  return SSD_OK;
}

ssd_status check_aligned(const Range* rs, int n) {
  for (int i = 0; i < n; ++i)
    if (rs[i].p && !aligned16(rs[i].p))
      return fail(SSD_ERR_ALIGN, "%s is not 16-byte aligned", rs[i].name);
  return SSD_OK;
}

ssd_status hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return SSD_OK;
  return fail(SSD_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// Shared validation of the forward arguments; fills element counts.
ssd_status validate_forward_sizes(int64_t B, int64_t H, int64_t N, int64_t d_h, int order,
                                  int64_t chunk, int dtype, int64_t* BH, int64_t* BHN,
                                  int64_t* BHNd) {
  if (!mul_ok(B, H, BH) || !mul_ok(*BH, N, BHN) || !mul_ok(*BHN, d_h, BHNd))
    return fail(SSD_ERR_SHAPE, "B, H, N must be >= 0, d_h >= 1, and their product must not overflow");
  if (dtype != SSD_F32 && dtype != SSD_BF16) return fail(SSD_ERR_UNSUPPORTED, "dtype %d", dtype);
  if (order != 1 && order != 2) return fail(SSD_ERR_UNSUPPORTED, "order %d (1 or 2)", order);
  if (chunk != 64 && chunk != 128) return fail(SSD_ERR_UNSUPPORTED, "chunk %lld (64 or 128)", (long long)chunk);
  if (order == 1 && d_h != 32 && d_h != 64)
    return fail(SSD_ERR_UNSUPPORTED, "d_h %lld at order 1 (32 or 64)", (long long)d_h);
  if (order == 2 && d_h != 64) return fail(SSD_ERR_UNSUPPORTED, "d_h %lld at order 2 (64)", (long long)d_h);
  if (order == 2 && dtype != SSD_BF16) return fail(SSD_ERR_UNSUPPORTED, "order 2 requires bf16 inputs");
  if (*BH * ((N + 63) / 64) > (int64_t)0x7fffffff) return fail(SSD_ERR_SHAPE, "grid too large");
  return SSD_OK;
}

}  // namespace

extern "C" {

int ssd_abi_version(void) { return SSD_ABI_VERSION; }

const char* ssd_status_str(int s) {
  switch (s) {
    case SSD_OK: return "SSD_OK";
    case SSD_ERR_NULL: return "SSD_ERR_NULL";
    case SSD_ERR_SHAPE: return "SSD_ERR_SHAPE";
    case SSD_ERR_UNSUPPORTED: return "SSD_ERR_UNSUPPORTED";
    case SSD_ERR_ALIGN: return "SSD_ERR_ALIGN";
    case SSD_ERR_ALIAS: return "SSD_ERR_ALIAS";
    case SSD_ERR_WORKSPACE: return "SSD_ERR_WORKSPACE";
    case SSD_ERR_HIP: return "SSD_ERR_HIP";
    default: return "SSD_ERR_UNKNOWN";
  }
}

const char* ssd_last_error(void) { return g_err; }

ssd_status ssd_prep(const float* dt_proj, const float* dt_bias, const float* A_log, int64_t B,
                    int64_t H, int64_t N, int64_t chunk, float* dt, float* a_cs, float* a_chunk,
                    hipStream_t stream) {
  try {
    clear_err();
    int64_t BH, BHN;
    if (!mul_ok(B, H, &BH) || !mul_ok(BH, N, &BHN))
      return fail(SSD_ERR_SHAPE, "ssd_prep: B, H, N must be >= 0 and must not overflow");
    if (chunk != 64 && chunk != 128)
      return fail(SSD_ERR_UNSUPPORTED, "ssd_prep: chunk %lld (64 or 128)", (long long)chunk);
    if (BHN == 0) return SSD_OK;  // empty input: nothing to compute
    if (!dt_proj || !dt_bias || !A_log || !dt || !a_cs || !a_chunk)
      return fail(SSD_ERR_NULL, "ssd_prep: a required pointer is NULL");
    const int64_t nc = (N + chunk - 1) / chunk;
    if (!fits(prep_workgroups(BH, N, chunk), 256)) return fail(SSD_ERR_SHAPE, "ssd_prep: grid too large");
    const Range ins[] = {{"dt_proj", dt_proj, (size_t)BHN * 4},
                         {"dt_bias", dt_bias, (size_t)H * 4},
                         {"A_log", A_log, (size_t)H * 4}};
    const Range outs[] = {{"dt", dt, (size_t)BHN * 4},
                          {"a_cs", a_cs, (size_t)BHN * 4},
                          {"a_chunk", a_chunk, (size_t)(BH * nc) * 4}};
    ssd_status s;
    if ((s = check_aligned(ins, 3)) != SSD_OK || (s = check_aligned(outs, 3)) != SSD_OK) return s;
    if ((s = check_alias(outs, 3, ins, 3)) != SSD_OK) return s;
    return hip_status(ssd::launch_prep(dt_proj, dt_bias, A_log, B, H, N, chunk, dt, a_cs, a_chunk, stream),
                      "ssd_prep launch");
  } catch (...) {
    return fail(SSD_ERR_HIP, "ssd_prep: unexpected exception");
  }
}

ssd_status ssd_prep_amask(const float* A_proj, const float* dt_proj, int64_t B, int64_t H,
                          int64_t N, int64_t chunk, float* dt, float* a_cs, float* a_chunk,
                          hipStream_t stream) {
  try {
    clear_err();
    int64_t BH, BHN;
    if (!mul_ok(B, H, &BH) || !mul_ok(BH, N, &BHN))
      return fail(SSD_ERR_SHAPE, "ssd_prep_amask: B, H, N must be >= 0 and must not overflow");
    if (chunk != 64 && chunk != 128)
      return fail(SSD_ERR_UNSUPPORTED, "ssd_prep_amask: chunk %lld (64 or 128)", (long long)chunk);
    if (BHN == 0) return SSD_OK;  // empty input: nothing to compute
    if (!A_proj || !a_cs || !a_chunk)
      return fail(SSD_ERR_NULL, "ssd_prep_amask: a required pointer is NULL");
    if ((dt_proj == nullptr) != (dt == nullptr))
      return fail(SSD_ERR_NULL, "ssd_prep_amask: dt_proj and dt must both be given or both be NULL");
    const int64_t nc = (N + chunk - 1) / chunk;
    if (!fits(prep_workgroups(BH, N, chunk), 256))
      return fail(SSD_ERR_SHAPE, "ssd_prep_amask: grid too large");
    const Range ins[] = {{"A_proj", A_proj, (size_t)BHN * 4}, {"dt_proj", dt_proj, (size_t)BHN * 4}};
    const Range outs[] = {{"dt", dt, (size_t)BHN * 4},
                          {"a_cs", a_cs, (size_t)BHN * 4},
                          {"a_chunk", a_chunk, (size_t)(BH * nc) * 4}};
    ssd_status s;
    if ((s = check_aligned(ins, 2)) != SSD_OK || (s = check_aligned(outs, 3)) != SSD_OK) return s;
    if ((s = check_alias(outs, 3, ins, 2)) != SSD_OK) return s;
    return hip_status(ssd::launch_prep_amask(A_proj, dt_proj, B, H, N, chunk, dt, a_cs, a_chunk, stream),
                      "ssd_prep_amask launch");
  } catch (...) {
    return fail(SSD_ERR_HIP, "ssd_prep_amask: unexpected exception");
  }
}

size_t ssd_forward_workspace_size(int64_t B, int64_t H, int64_t N, int64_t d_h, int order,
                                  int64_t chunk, int dtype) {
  int64_t BH, BHN, BHNd;
  if (validate_forward_sizes(B, H, N, d_h, order, chunk, dtype, &BH, &BHN, &BHNd) != SSD_OK) return 0;
  if (BHN == 0) return 0;  // an empty input needs no workspace
  return ssd::ws_layout(B, H, N, d_h, order).total_floats * sizeof(float);
}

}  // extern "C"

namespace {

// Scratch memory of ssd_forward_noalloc: a file-scope device array (each GPU
// the library runs on holds its own copy until the process ends).  Host code
// never uses the array's name as an address: the device address comes from
// hipGetSymbolAddress, taken once per device on that device's first call.
static __device__ __align__(256) unsigned char scratch[SSD_NOALLOC_SCRATCH_BYTES];

constexpr int MAX_DEVICES = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[MAX_DEVICES] = {};

ssd_status scratch_of_current_device(void** out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_status(e, "ssd_forward_noalloc: hipGetDevice");
  if (dev < 0 || dev >= MAX_DEVICES)
    return fail(SSD_ERR_HIP, "ssd_forward_noalloc: device %d beyond the %d supported", dev, MAX_DEVICES);
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return hip_status(e, "ssd_forward_noalloc: hipGetSymbolAddress(scratch)");
    if (!p) return fail(SSD_ERR_HIP, "ssd_forward_noalloc: hipGetSymbolAddress returned NULL");
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return SSD_OK;
}

// ssd_forward and ssd_forward_noalloc: every argument check, then (noalloc)
// the device's scratch array in place of the caller's workspace, then the
// launches.
ssd_status forward_core(const char* fn, bool noalloc, const void* q, const void* k, const void* v,
                        const float* dt, const float* a_cs, const float* initial_state,
                        const float* initial_norm, int64_t B, int64_t H, int64_t N, int64_t d_h,
                        int order, int64_t chunk, int dtype, float* y, float* den,
                        float* final_state, float* final_norm, void* workspace,
                        size_t workspace_bytes, hipStream_t stream) {
  int64_t BH, BHN, BHNd;
  ssd_status s = validate_forward_sizes(B, H, N, d_h, order, chunk, dtype, &BH, &BHN, &BHNd);
  if (s != SSD_OK) return s;
  if (BH == 0) return SSD_OK;  // no heads: nothing to compute
  if ((final_state == nullptr) != (final_norm == nullptr))
    return fail(SSD_ERR_NULL, "%s: final_state and final_norm must be given together", fn);
  if ((initial_state == nullptr) != (initial_norm == nullptr))
    return fail(SSD_ERR_NULL, "%s: initial_state and initial_norm must be given together", fn);
  const size_t es = dtype == SSD_BF16 ? 2 : 4;
  const int64_t D = order == 1 ? d_h : d_h * d_h;
  if (BHN == 0) {
    // an empty segment (N = 0): the final states are the initial ones (or zero)
    if (!final_state) return SSD_OK;
    const Range ins0[] = {{"initial_state", initial_state, (size_t)(BH * D * d_h) * 4},
                          {"initial_norm", initial_norm, (size_t)(BH * D) * 4}};
    const Range outs0[] = {{"final_state", final_state, (size_t)(BH * D * d_h) * 4},
                           {"final_norm", final_norm, (size_t)(BH * D) * 4}};
    if ((s = check_aligned(ins0, 2)) != SSD_OK || (s = check_aligned(outs0, 2)) != SSD_OK) return s;
    if ((s = check_alias(outs0, 2, ins0, 2)) != SSD_OK) return s;
    hipError_t e = ssd::launch_copy_or_zero(final_state, initial_state, BH * D * d_h, stream);
    if (e == hipSuccess) e = ssd::launch_copy_or_zero(final_norm, initial_norm, BH * D, stream);
    return hip_status(e, "final-state copy launch");
  }
  // the largest grids, of workgroups of 256: the scan's a head (segments only with few heads); else one a
  // block, at order 1 also one for 256 values of a state, at order 2 16 a head (8 of 512)
  const int64_t nb = (N + 63) / 64;
  int64_t grid = BH * nb;
  if (order == 1 && dtype == SSD_BF16 && ssd::o1_scan_supported(BH, d_h, N)) {
    grid = BH;
  } else {
    const int64_t heads = BH * (order == 1 ? (d_h * d_h + d_h + 255) / 256 : initial_state ? ssd::O2_INIT_PARTS : 16);
    if (order == 2) grid = 16 * ((BH * ((nb + 1) / 2) + 7) / 8);  // the output kernel's, >= BH nb
    if (heads > grid) grid = heads;
  }
  if (!fits(grid, 256)) return fail(SSD_ERR_SHAPE, "%s: grid too large", fn);
  if (!q || !k || !v || !a_cs || !y) return fail(SSD_ERR_NULL, "%s: a required pointer is NULL", fn);
  const size_t need = ssd::ws_layout(B, H, N, d_h, order).total_floats * sizeof(float);
  if (noalloc) {
    if (need > (size_t)SSD_NOALLOC_SCRATCH_BYTES)
      return fail(SSD_ERR_WORKSPACE,
                  "%s: these sizes need %zu bytes of scratch, more than the %zu bytes this entry point "
                  "holds per device; call ssd_forward with a workspace instead",
                  fn, need, (size_t)SSD_NOALLOC_SCRATCH_BYTES);
  } else if (workspace_bytes < need || (need && !workspace)) {
    return fail(SSD_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                workspace ? workspace_bytes : (size_t)0);
  }
  const Range ins[] = {{"q", q, (size_t)BHNd * es},  {"k", k, (size_t)BHNd * es},
                       {"v", v, (size_t)BHNd * es},  {"dt", dt, (size_t)BHN * 4},
                       {"a_cs", a_cs, (size_t)BHN * 4},
                       {"initial_state", initial_state, (size_t)(BH * D * d_h) * 4},
                       {"initial_norm", initial_norm, (size_t)(BH * D) * 4}};
  const Range outs[] = {{"y", y, (size_t)BHNd * 4},
                        {"den", den, (size_t)BHN * 4},
                        {"final_state", final_state, (size_t)(BH * D * d_h) * 4},
                        {"final_norm", final_norm, (size_t)(BH * D) * 4},
                        {"workspace", noalloc ? nullptr : workspace, need}};
  if ((s = check_aligned(ins, 7)) != SSD_OK || (s = check_aligned(outs, 5)) != SSD_OK) return s;
  if ((s = check_alias(outs, 5, ins, 7)) != SSD_OK) return s;
  // every check done: only now the first HIP call
  if (noalloc && (s = scratch_of_current_device(&workspace)) != SSD_OK) return s;

  const bool bf = dtype == SSD_BF16;
  Timer tm(stream);
  const ssd::WsLayout L = ssd::ws_layout(B, H, N, d_h, order);
  float* ws = static_cast<float*>(workspace);
  float* tb = ws + L.tb;
  float* st = ws + L.state;
  hipError_t e;
  if (order == 1 && bf && ssd::o1_scan_supported(BH, d_h, N)) {
    // bf16 inputs: the sequential scan per (head, segment); the segment
    // aggregates and their prefixes (when the sequence is cut into segments)
    // go to the state region of the workspace
    float* agg = st;
    const size_t na = (ssd::o1_scan_agg_floats(BH, d_h, N) + 63) & ~(size_t)63;
    float* sink = st + na;
    if (na + 64 > L.part - L.state)
      return fail(SSD_ERR_WORKSPACE, "%s: internal: segment aggregates exceed the workspace", fn);
    if ((e = ssd::launch_o1_scan(true, d_h, q, k, v, dt, a_cs, BH, N, chunk, initial_state, initial_norm,
                                 agg, nullptr, nullptr, nullptr, nullptr, sink, stream)) != hipSuccess)
      return hip_status(e, "o1_scan aggregate launch");
    tm.mark();
    e = ssd::launch_o1_scan(false, d_h, q, k, v, dt, a_cs, BH, N, chunk, initial_state, initial_norm,
                            agg, y, den, final_state, final_norm, sink, stream);
    tm.mark();
    return hip_status(e, "o1_scan launch");
  }
  if (order == 1) {
    if ((e = ssd::launch_chunk_state(bf, d_h, k, v, dt, a_cs, BH, N, chunk, tb, st, stream)) != hipSuccess)
      return hip_status(e, "chunk_state launch");
    tm.mark();
    if ((e = ssd::launch_state_pass(d_h, BH, N, tb, st, final_state, final_norm, initial_state,
                                    initial_norm, stream)) != hipSuccess)
      return hip_status(e, "state_pass launch");
    tm.mark();
    e = ssd::launch_output(bf, d_h, 1, q, k, v, dt, a_cs, BH, N, chunk, st, nullptr, y, den, stream);
    tm.mark();
    return hip_status(e, "output launch");
  }
  // order 2: per-block preparation (normaliser contributions Z_blk and the
  // numerator operand records), the scale scan, the on-chip numerator scan
  // (which also scans Z), and the output kernel.
  float* part = ws + L.part;
  void* rec = ws + L.rec;
  if ((e = ssd::launch_o2_blockprep(q, k, v, dt, a_cs, BH, N, chunk, tb, st, rec, stream)) != hipSuccess)
    return hip_status(e, "o2_blockprep launch");
  tm.mark();
  float* initmax = nullptr;
  if (initial_state) {
    initmax = ws + L.initmax;
    if ((e = ssd::launch_o2_initmax(initial_state, BH, initmax, stream)) != hipSuccess)
      return hip_status(e, "o2_initmax launch");
  }
  if ((e = ssd::launch_o2_scale_scan(rec, BH, N, initmax, stream)) != hipSuccess)
    return hip_status(e, "o2_scale_scan launch");
  tm.mark();
  if ((e = ssd::launch_o2_state(rec, BH, N, part, final_state, st, final_norm, initial_state,
                                initial_norm, stream)) != hipSuccess)
    return hip_status(e, "o2_state launch");
  tm.mark();
  e = ssd::launch_output(true, 64, 2, q, k, v, dt, a_cs, BH, N, chunk, st, part, y, den, stream);
  tm.mark();
  return hip_status(e, "output launch");
}

}  // namespace

extern "C" {

ssd_status ssd_forward(const void* q, const void* k, const void* v, const float* dt,
                       const float* a_cs, const float* initial_state, const float* initial_norm,
                       int64_t B, int64_t H, int64_t N, int64_t d_h, int order,
                       int64_t chunk, int dtype, float* y, float* den, float* final_state,
                       float* final_norm, void* workspace, size_t workspace_bytes,
                       hipStream_t stream) {
  try {
    clear_err();
    return forward_core("ssd_forward", false, q, k, v, dt, a_cs, initial_state, initial_norm, B, H, N,
                        d_h, order, chunk, dtype, y, den, final_state, final_norm, workspace,
                        workspace_bytes, stream);
  } catch (...) {
    return fail(SSD_ERR_HIP, "ssd_forward: unexpected exception");
  }
}

ssd_status ssd_forward_noalloc(const void* q, const void* k, const void* v, const float* dt,
                               const float* a_cs, const float* initial_state,
                               const float* initial_norm, int64_t B, int64_t H, int64_t N,
                               int64_t d_h, int order, int64_t chunk, int dtype, float* y,
                               float* den, float* final_state, float* final_norm,
                               hipStream_t stream) {
  try {
    clear_err();
    return forward_core("ssd_forward_noalloc", true, q, k, v, dt, a_cs, initial_state, initial_norm, B,
                        H, N, d_h, order, chunk, dtype, y, den, final_state, final_norm, nullptr, 0,
                        stream);
  } catch (...) {
    return fail(SSD_ERR_HIP, "ssd_forward_noalloc: unexpected exception");
  }
}

ssd_status ssd_set_timing_events(hipEvent_t* events, int n) {
  clear_err();
  if (events && n < 5) return fail(SSD_ERR_SHAPE, "ssd_set_timing_events: n must be >= 5");
  g_events = events;
  g_n_events = events ? n : 0;
  return SSD_OK;
}

int ssd_timing_count(void) { return g_timed; }

// Shared by both decode entry points: sizes, parameters, pointers, alignment
// and overlap; `params` are the per-token / per-head decay inputs.
static ssd_status decode_common(const char* fn, const void* q, const void* k, const void* v,
                         const Range* params, int n_params, int64_t S, int64_t H, int64_t d_h,
                         int order, int dtype, int layout, float* state, float* norm_state,
                         float* y, bool* empty) {
  int64_t SH, SHd;
  *empty = false;
  if (!mul_ok(S, H, &SH) || !mul_ok(SH, d_h, &SHd))
    return fail(SSD_ERR_SHAPE, "%s: S, H must be >= 0 and must not overflow", fn);
  if (dtype != SSD_F32 && dtype != SSD_BF16) return fail(SSD_ERR_UNSUPPORTED, "dtype %d", dtype);
  if (order != 1 && order != 2) return fail(SSD_ERR_UNSUPPORTED, "order %d (1 or 2)", order);
  if (d_h != 32 && d_h != 64) return fail(SSD_ERR_UNSUPPORTED, "d_h %lld (32 or 64)", (long long)d_h);
  if (layout != SSD_STATE_FULL && layout != SSD_STATE_PACKED)
    return fail(SSD_ERR_UNSUPPORTED, "%s: layout %d", fn, layout);
  if (layout == SSD_STATE_PACKED && order != 2)
    return fail(SSD_ERR_UNSUPPORTED, "%s: the packed layout is for order 2", fn);
  if (SH == 0) {  // no sequences or heads: nothing to compute
    *empty = true;
    return SSD_OK;
  }
  if (!q || !k || !v || !state || !norm_state || !y)
    return fail(SSD_ERR_NULL, "%s: a required pointer is NULL", fn);
  if (!fits(SH, order == 1 ? 256 : layout == SSD_STATE_PACKED ? 512 : 1024))
    return fail(SSD_ERR_SHAPE, "%s: grid too large", fn);
  const int64_t D = order == 1 ? d_h : (layout == SSD_STATE_PACKED ? d_h * (d_h + 1) / 2 : d_h * d_h);
  int64_t nstate;
  if (!mul_ok(SH, D * d_h, &nstate)) return fail(SSD_ERR_SHAPE, "%s: state too large", fn);
  const size_t es = dtype == SSD_BF16 ? 2 : 4;
  constexpr int MAX_PARAMS = 8;
  if (n_params > MAX_PARAMS) return fail(SSD_ERR_HIP, "%s: internal: too many parameter ranges", fn);
  Range ins[3 + MAX_PARAMS] = {{"q", q, (size_t)SHd * es}, {"k", k, (size_t)SHd * es},
                               {"v", v, (size_t)SHd * es}};
  for (int i = 0; i < n_params; ++i) ins[3 + i] = params[i];
  const Range outs[] = {{"state", state, (size_t)nstate * 4},
                        {"norm_state", norm_state, (size_t)(SH * D) * 4},
                        {"y", y, (size_t)SHd * 4}};
  ssd_status s;
  if ((s = check_aligned(ins, 3 + n_params)) != SSD_OK || (s = check_aligned(outs, 3)) != SSD_OK)
    return s;
  return check_alias(outs, 3, ins, 3 + n_params);
}

ssd_status ssd_decode_step(const void* q, const void* k, const void* v, const float* dt_proj,
                           const float* dt_bias, const float* A_log, int64_t S, int64_t H,
                           int64_t d_h, int order, int dtype, int layout, float* state,
                           float* norm_state, float* y, hipStream_t stream) {
  try {
    clear_err();
    int64_t SH = 0;
    (void)mul_ok(S, H, &SH);
    const Range params[] = {{"dt_proj", dt_proj, (size_t)SH * 4},
                            {"dt_bias", dt_bias, (size_t)(H > 0 ? H : 0) * 4},
                            {"A_log", A_log, (size_t)(H > 0 ? H : 0) * 4}};
    bool empty;
    ssd_status s = decode_common("ssd_decode_step", q, k, v, params, 3, S, H, d_h, order, dtype,
                                 layout, state, norm_state, y, &empty);
    if (s != SSD_OK || empty) return s;
    if (!dt_proj || !dt_bias || !A_log)
      return fail(SSD_ERR_NULL, "ssd_decode_step: a required pointer is NULL");
    return hip_status(ssd::launch_decode(dtype == SSD_BF16, d_h, order, layout == SSD_STATE_PACKED, q, k,
                                         v, dt_proj, dt_bias, A_log, nullptr, S, H, state, norm_state,
                                         y, stream),
                      "decode launch");
  } catch (...) {
    return fail(SSD_ERR_HIP, "ssd_decode_step: unexpected exception");
  }
}

ssd_status ssd_decode_step_amask(const void* q, const void* k, const void* v, const float* A_proj,
                                 const float* dt_proj, int64_t S, int64_t H, int64_t d_h,
                                 int order, int dtype, int layout, float* state,
                                 float* norm_state, float* y, hipStream_t stream) {
  try {
    clear_err();
    int64_t SH = 0;
    (void)mul_ok(S, H, &SH);
    const Range params[] = {{"A_proj", A_proj, (size_t)SH * 4}, {"dt_proj", dt_proj, (size_t)SH * 4}};
    bool empty;
    ssd_status s = decode_common("ssd_decode_step_amask", q, k, v, params, 2, S, H, d_h, order, dtype,
                                 layout, state, norm_state, y, &empty);
    if (s != SSD_OK || empty) return s;
    if (!A_proj) return fail(SSD_ERR_NULL, "ssd_decode_step_amask: A_proj is NULL");
    return hip_status(ssd::launch_decode(dtype == SSD_BF16, d_h, order, layout == SSD_STATE_PACKED, q, k,
                                         v, dt_proj, nullptr, nullptr, A_proj, S, H, state,
                                         norm_state, y, stream),
                      "decode launch");
  } catch (...) {
    return fail(SSD_ERR_HIP, "ssd_decode_step_amask: unexpected exception");
  }
}

ssd_status ssd_decode_step_conv(const void* q, const void* k, const void* v, const float* conv_w,
                                const float* conv_b, int conv_act, void* conv_state,
                                const float* A_proj, const float* dt_proj, const float* dt_bias,
                                const float* A_log, int64_t S, int64_t H, int64_t d_h, int order,
                                int dtype, int layout, float* state, float* norm_state, float* y,
                                hipStream_t stream) {
  try {
    clear_err();
    const char* fn = "ssd_decode_step_conv";
    int64_t SH = 0, SHd = 0;
    (void)mul_ok(S, H, &SH);
    (void)mul_ok(SH, d_h, &SHd);
    const int64_t Hd = (H > 0 ? H : 0) * (d_h > 0 ? d_h : 0);
    const size_t es = dtype == SSD_BF16 ? 2 : 4;
    const Range params[] = {{"A_proj", A_proj, (size_t)SH * 4},
                            {"dt_proj", dt_proj, (size_t)SH * 4},
                            {"dt_bias", dt_bias, (size_t)(H > 0 ? H : 0) * 4},
                            {"A_log", A_log, (size_t)(H > 0 ? H : 0) * 4},
                            {"conv_w", conv_w, (size_t)(3 * Hd * 2) * 4},
                            {"conv_b", conv_b, (size_t)(3 * Hd) * 4}};
    bool empty;
    ssd_status s = decode_common(fn, q, k, v, params, 6, S, H, d_h, order, dtype, layout, state,
                                 norm_state, y, &empty);
    if (s != SSD_OK || empty) return s;
    if (conv_act != 0 && conv_act != 1) return fail(SSD_ERR_UNSUPPORTED, "%s: conv_act %d (0 or 1)", fn, conv_act);
    if (!conv_w || !conv_state) return fail(SSD_ERR_NULL, "%s: conv_w and conv_state are required", fn);
    if (A_proj) {
      if (dt_bias || A_log)
        return fail(SSD_ERR_UNSUPPORTED, "%s: with A_proj (the A-mask) dt_bias and A_log must be NULL", fn);
    } else if (!dt_proj || !dt_bias || !A_log) {
      return fail(SSD_ERR_NULL, "%s: without A_proj, dt_proj, dt_bias and A_log are required", fn);
    }
    // the conv state is read and written in place: it must not overlap any
    // other argument
    const Range cs{"conv_state", conv_state, (size_t)(3 * SHd) * es};
    if (!aligned16(conv_state)) return fail(SSD_ERR_ALIGN, "%s: conv_state is not 16-byte aligned", fn);
    const Range others[] = {{"q", q, (size_t)SHd * es}, {"k", k, (size_t)SHd * es},
                            {"v", v, (size_t)SHd * es}, params[0], params[1], params[2], params[3],
                            params[4], params[5]};
    if ((s = check_alias(&cs, 1, others, 9)) != SSD_OK) return s;
    int64_t D = order == 1 ? d_h : (layout == SSD_STATE_PACKED ? d_h * (d_h + 1) / 2 : d_h * d_h);
    const Range outs[] = {{"state", state, (size_t)(SH * D * d_h) * 4},
                          {"norm_state", norm_state, (size_t)(SH * D) * 4}, {"y", y, (size_t)SHd * 4}};
    if ((s = check_alias(outs, 3, &cs, 1)) != SSD_OK) return s;
    return hip_status(ssd::launch_decode(dtype == SSD_BF16, d_h, order, layout == SSD_STATE_PACKED, q, k, v,
                                         dt_proj, dt_bias, A_log, A_proj, S, H, state, norm_state, y, stream,
                                         ssd::DecodeConv{conv_w, conv_b, conv_state, conv_act}),
                      "decode launch");
  } catch (...) {
    return fail(SSD_ERR_HIP, "ssd_decode_step_conv: unexpected exception");
  }
}

// ssd_state_pack / ssd_state_unpack
static ssd_status state_layout(const char* fn, bool to_packed, const float* src_S, const float* src_z,
                               int64_t BH, int64_t d_h, float* dst_S, float* dst_z,
                               hipStream_t stream) {
  clear_err();
  if (BH < 0) return fail(SSD_ERR_SHAPE, "%s: BH must be >= 0", fn);
  if (d_h != 32 && d_h != 64) return fail(SSD_ERR_UNSUPPORTED, "d_h %lld (32 or 64)", (long long)d_h);
  if (BH == 0) return SSD_OK;
  if (!src_S || !src_z || !dst_S || !dst_z) return fail(SSD_ERR_NULL, "%s: a required pointer is NULL", fn);
  const int64_t Df = d_h * d_h, Dp = d_h * (d_h + 1) / 2;
  int64_t nf, np_;
  if (!mul_ok(BH, Df * d_h, &nf) || !mul_ok(BH, Dp * d_h, &np_) || !fits(BH * d_h, 256))
    return fail(SSD_ERR_SHAPE, "%s: state too large", fn);
  const int64_t ns = to_packed ? nf : np_, nd = to_packed ? np_ : nf;
  const int64_t zs = (to_packed ? Df : Dp) * BH, zd = (to_packed ? Dp : Df) * BH;
  const Range ins[] = {{"source state", src_S, (size_t)ns * 4}, {"source norm", src_z, (size_t)zs * 4}};
  const Range outs[] = {{"state", dst_S, (size_t)nd * 4}, {"norm", dst_z, (size_t)zd * 4}};
  ssd_status s;
  if ((s = check_aligned(ins, 2)) != SSD_OK || (s = check_aligned(outs, 2)) != SSD_OK) return s;
  if ((s = check_alias(outs, 2, ins, 2)) != SSD_OK) return s;
  return hip_status(ssd::launch_state_layout(to_packed, d_h, BH, src_S, src_z, dst_S, dst_z, stream),
                    "state layout launch");
}

ssd_status ssd_state_pack(const float* state, const float* norm_state, int64_t BH, int64_t d_h,
                          float* state_p, float* norm_p, hipStream_t stream) {
  try {
    return state_layout("ssd_state_pack", true, state, norm_state, BH, d_h, state_p, norm_p, stream);
  } catch (...) {
    return fail(SSD_ERR_HIP, "ssd_state_pack: unexpected exception");
  }
}

ssd_status ssd_state_unpack(const float* state_p, const float* norm_p, int64_t BH, int64_t d_h,
                            float* state, float* norm_state, hipStream_t stream) {
  try {
    return state_layout("ssd_state_unpack", false, state_p, norm_p, BH, d_h, state, norm_state, stream);
  } catch (...) {
    return fail(SSD_ERR_HIP, "ssd_state_unpack: unexpected exception");
  }
}

size_t ssd_backward_workspace_size(int64_t B, int64_t H, int64_t N, int64_t d_h, int order,
                                   int64_t chunk, int dtype) {
  int64_t BH, BHN, BHNd;
  if (validate_forward_sizes(B, H, N, d_h, order, chunk, dtype, &BH, &BHN, &BHNd) != SSD_OK) return 0;
  if (BHN == 0) return 0;
  return ssd::bwd_layout(BH, N, d_h, order).total_floats * sizeof(float);
}

ssd_status ssd_backward(const void* q, const void* k, const void* v, const float* dt,
                        const float* a_cs, const float* y, const float* den, const float* dy,
                        int64_t B, int64_t H, int64_t N, int64_t d_h, int order, int64_t chunk,
                        int dtype, float* dq, float* dk, float* dv, float* ddt, float* da,
                        void* workspace, size_t workspace_bytes, hipStream_t stream) {
  try {
    clear_err();
    int64_t BH, BHN, BHNd;
    ssd_status s = validate_forward_sizes(B, H, N, d_h, order, chunk, dtype, &BH, &BHN, &BHNd);
    if (s != SSD_OK) return s;
    if (BHN == 0) return SSD_OK;  // nothing to differentiate
    // workgroups of 256: one a block, and for 256 values of a state (order 1) or for each feature (order 2)
    if (!fits(BH * ((N + 63) / 64), 256) ||
        !fits(BH * (order == 1 ? (d_h * d_h + d_h + 255) / 256 : d_h), 256))
      return fail(SSD_ERR_SHAPE, "ssd_backward: grid too large");
    if (!q || !k || !v || !a_cs || !y || !den || !dy || !dq || !dk || !dv || !da)
      return fail(SSD_ERR_NULL, "ssd_backward: a required pointer is NULL");
    if ((dt == nullptr) != (ddt == nullptr))
      return fail(SSD_ERR_NULL, "ssd_backward: dt and ddt must be given together");
    const size_t need = ssd::bwd_layout(BH, N, d_h, order).total_floats * sizeof(float);
    if (workspace_bytes < need || !workspace)
      return fail(SSD_ERR_WORKSPACE, "ssd_backward: workspace of %zu bytes needed, %zu given", need,
                  workspace ? workspace_bytes : (size_t)0);
    const size_t es = dtype == SSD_BF16 ? 2 : 4;
    const Range ins[] = {{"q", q, (size_t)BHNd * es},  {"k", k, (size_t)BHNd * es},
                         {"v", v, (size_t)BHNd * es},  {"dt", dt, (size_t)BHN * 4},
                         {"a_cs", a_cs, (size_t)BHN * 4}, {"y", y, (size_t)BHNd * 4},
                         {"den", den, (size_t)BHN * 4}, {"dy", dy, (size_t)BHNd * 4}};
    const Range outs[] = {{"dq", dq, (size_t)BHNd * 4}, {"dk", dk, (size_t)BHNd * 4},
                          {"dv", dv, (size_t)BHNd * 4}, {"ddt", ddt, (size_t)BHN * 4},
                          {"da", da, (size_t)BHN * 4},  {"workspace", workspace, need}};
    if ((s = check_aligned(ins, 8)) != SSD_OK || (s = check_aligned(outs, 6)) != SSD_OK) return s;
    if ((s = check_alias(outs, 6, ins, 8)) != SSD_OK) return s;
    return hip_status(ssd::launch_backward(order, dtype == SSD_BF16, d_h, q, k, v, dt, a_cs, y, den, dy, BH,
                                           N, chunk, dq, dk, dv, ddt, da, static_cast<float*>(workspace),
                                           stream),
                      "backward launch");
  } catch (...) {
    return fail(SSD_ERR_HIP, "ssd_backward: unexpected exception");
  }
}

// shared size validation of the two discretisation backward calls
static ssd_status prep_bwd_sizes(const char* fn, int64_t B, int64_t H, int64_t N, int64_t* BHN) {
  int64_t BH;
  if (!mul_ok(B, H, &BH) || !mul_ok(BH, N, BHN))
    return fail(SSD_ERR_SHAPE, "%s: B, H, N must be >= 0 and must not overflow", fn);
  if (!fits(H, 1024)) return fail(SSD_ERR_SHAPE, "%s: H too large", fn);  // a workgroup of 1024 a head
  return SSD_OK;
}

ssd_status ssd_prep_backward(const float* dt_proj, const float* dt_bias, const float* A_log,
                             const float* da, const float* ddt, int64_t B, int64_t H, int64_t N,
                             float* d_dt_proj, float* d_dt_bias, float* d_A_log, hipStream_t stream) {
  try {
    clear_err();
    int64_t BHN;
    ssd_status s = prep_bwd_sizes("ssd_prep_backward", B, H, N, &BHN);
    if (s != SSD_OK) return s;
    if (H == 0) return SSD_OK;
    if (!dt_bias || !A_log || !d_dt_bias || !d_A_log || (BHN && (!dt_proj || !da || !d_dt_proj)))
      return fail(SSD_ERR_NULL, "ssd_prep_backward: a required pointer is NULL");
    const Range ins[] = {{"dt_proj", dt_proj, (size_t)BHN * 4}, {"dt_bias", dt_bias, (size_t)H * 4},
                         {"A_log", A_log, (size_t)H * 4},       {"da", da, (size_t)BHN * 4},
                         {"ddt", ddt, (size_t)BHN * 4}};
    const Range outs[] = {{"d_dt_proj", d_dt_proj, (size_t)BHN * 4},
                          {"d_dt_bias", d_dt_bias, (size_t)H * 4},
                          {"d_A_log", d_A_log, (size_t)H * 4}};
    if ((s = check_aligned(ins, 5)) != SSD_OK || (s = check_aligned(outs, 3)) != SSD_OK) return s;
    if ((s = check_alias(outs, 3, ins, 5)) != SSD_OK) return s;
    return hip_status(ssd::launch_prep_backward(dt_proj, dt_bias, A_log, da, ddt, B, H, N, d_dt_proj,
                                                d_dt_bias, d_A_log, stream),
                      "prep backward launch");
  } catch (...) {
    return fail(SSD_ERR_HIP, "ssd_prep_backward: unexpected exception");
  }
}

ssd_status ssd_prep_amask_backward(const float* A_proj, const float* dt_proj, const float* da,
                                   const float* ddt, int64_t B, int64_t H, int64_t N,
                                   float* d_A_proj, float* d_dt_proj, hipStream_t stream) {
  try {
    clear_err();
    int64_t BHN;
    ssd_status s = prep_bwd_sizes("ssd_prep_amask_backward", B, H, N, &BHN);
    if (s != SSD_OK) return s;
    if (BHN == 0) return SSD_OK;
    if (!A_proj || !da || !d_A_proj)
      return fail(SSD_ERR_NULL, "ssd_prep_amask_backward: a required pointer is NULL");
    if ((dt_proj == nullptr) != (ddt == nullptr) || (dt_proj == nullptr) != (d_dt_proj == nullptr))
      return fail(SSD_ERR_NULL, "ssd_prep_amask_backward: dt_proj, ddt and d_dt_proj go together");
    const Range ins[] = {{"A_proj", A_proj, (size_t)BHN * 4}, {"dt_proj", dt_proj, (size_t)BHN * 4},
                         {"da", da, (size_t)BHN * 4},         {"ddt", ddt, (size_t)BHN * 4}};
    const Range outs[] = {{"d_A_proj", d_A_proj, (size_t)BHN * 4},
                          {"d_dt_proj", d_dt_proj, (size_t)BHN * 4}};
    if ((s = check_aligned(ins, 4)) != SSD_OK || (s = check_aligned(outs, 2)) != SSD_OK) return s;
    if ((s = check_alias(outs, 2, ins, 4)) != SSD_OK) return s;
    return hip_status(ssd::launch_prep_amask_backward(A_proj, dt_proj, da, ddt, B, H, N, d_A_proj,
                                                      d_dt_proj, stream),
                      "prep amask backward launch");
  } catch (...) {
    return fail(SSD_ERR_HIP, "ssd_prep_amask_backward: unexpected exception");
  }
}

// ---- the gated linear recurrence ----

// shared size validation; count = S H d_h or B H N d_h
static ssd_status gated_sizes(const char* fn, int64_t B, int64_t H, int64_t N, int64_t d_h,
                              int64_t* BH, int64_t* count) {
  int64_t BHN;
  if (d_h < 1 || !mul_ok(B, H, BH) || !mul_ok(*BH, N, &BHN) || !mul_ok(BHN, d_h, count))
    return fail(SSD_ERR_SHAPE, "%s: sizes must be >= 0, d_h >= 1, and their product must not overflow", fn);
  if (d_h > SSD_GATED_MAX)
    return fail(SSD_ERR_UNSUPPORTED, "%s: d_h %lld (at most %d)", fn, (long long)d_h, SSD_GATED_MAX);
  int64_t wide, slabs;  // workgroups, were there one to a head, 16 channels and 64 tokens: less than 2^31
  if (!mul_ok(*BH, (d_h + 15) / 16, &slabs) || !mul_ok(slabs, (N + 63) / 64 + 1, &wide) ||
      wide > (int64_t)0x7fffffff)
    return fail(SSD_ERR_SHAPE, "%s: grid too large", fn);
  return SSD_OK;
}

static ssd_status gated_kinds(const char* fn, int input_scale, int dtype) {
  if (input_scale != SSD_INPUT_PLAIN && input_scale != SSD_INPUT_CONVEX && input_scale != SSD_INPUT_UNIT)
    return fail(SSD_ERR_UNSUPPORTED, "%s: input_scale %d (0, 1 or 2)", fn, input_scale);
  if (dtype != SSD_F32 && dtype != SSD_BF16) return fail(SSD_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
  return SSD_OK;
}

static ssd_status check_workspace(const char* fn, const void* workspace, size_t given, size_t need) {
  if (given < need || (need && !workspace))
    return fail(SSD_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                workspace ? given : (size_t)0);
  return SSD_OK;
}

size_t ssd_gated_scan_workspace_size(int64_t B, int64_t H, int64_t N, int64_t d_h) {
  int64_t BH, n;
  if (gated_sizes("ssd_gated_scan_workspace_size", B, H, N, d_h, &BH, &n) != SSD_OK || n == 0) return 0;
  return ssd::gated_scan_floats(BH, N, d_h) * sizeof(float);
}

ssd_status ssd_gated_scan(const void* x, const void* A_proj, const void* I_proj,
                          const float* initial_state, int64_t B, int64_t H, int64_t N, int64_t d_h,
                          int input_scale, int dtype, float* y, float* final_state,
                          void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const char* fn = "ssd_gated_scan";
  try {
    clear_err();
    int64_t BH, n;
    ssd_status s = gated_sizes(fn, B, H, N, d_h, &BH, &n);
    if (s != SSD_OK || (s = gated_kinds(fn, input_scale, dtype)) != SSD_OK) return s;
    if (BH == 0) return SSD_OK;  // no heads: nothing to compute
    const Range h0{"initial_state", initial_state, (size_t)(BH * d_h) * 4};
    const Range hf{"final_state", final_state, (size_t)(BH * d_h) * 4};
    if (n == 0) {  // no tokens: the final state is the initial one (or zero)
      if (!final_state) return SSD_OK;
      if ((s = check_aligned(&h0, 1)) != SSD_OK || (s = check_aligned(&hf, 1)) != SSD_OK) return s;
      if ((s = check_alias(&hf, 1, &h0, 1)) != SSD_OK) return s;
      return hip_status(ssd::launch_copy_or_zero(final_state, initial_state, BH * d_h, stream),
                        "final-state copy launch");
    }
    if (!ssd::gated_scan_fits(dtype == SSD_BF16, BH, N, d_h)) return fail(SSD_ERR_SHAPE, "%s: grid too large", fn);
    if (!x || !A_proj || !y) return fail(SSD_ERR_NULL, "%s: a required pointer is NULL", fn);
    const size_t need = ssd::gated_scan_floats(BH, N, d_h) * sizeof(float);
    if ((s = check_workspace(fn, workspace, workspace_bytes, need)) != SSD_OK) return s;
    const size_t bytes = (size_t)n * (dtype == SSD_BF16 ? 2 : 4);
    const Range ins[] = {{"x", x, bytes}, {"A_proj", A_proj, bytes}, {"I_proj", I_proj, bytes}, h0};
    const Range outs[] = {{"y", y, (size_t)n * 4}, hf, {"workspace", workspace, need}};
    if ((s = check_aligned(ins, 4)) != SSD_OK || (s = check_aligned(outs, 3)) != SSD_OK) return s;
    if ((s = check_alias(outs, 3, ins, 4)) != SSD_OK) return s;
    return hip_status(ssd::launch_gated_scan(dtype == SSD_BF16, input_scale, x, A_proj, I_proj,
                                             initial_state, BH, N, d_h, y, final_state,
                                             static_cast<float*>(workspace), stream),
                      "gated_scan launch");
  } catch (...) {
    return fail(SSD_ERR_HIP, "%s: unexpected exception", fn);
  }
}

ssd_status ssd_gated_scan_step(const void* x, const void* A_proj, const void* I_proj,
                               const float* state, int64_t S, int64_t H, int64_t d_h,
                               int input_scale, int dtype, float* new_state, hipStream_t stream) {
  const char* fn = "ssd_gated_scan_step";
  try {
    clear_err();
    int64_t SH, n;
    ssd_status s = gated_sizes(fn, S, H, 1, d_h, &SH, &n);
    if (s != SSD_OK || (s = gated_kinds(fn, input_scale, dtype)) != SSD_OK) return s;
    if (n == 0) return SSD_OK;  // no sequences or heads: nothing to compute
    if (!fits((n + 1023) / 1024, 256))  // 256 threads to 1024 channels
      return fail(SSD_ERR_SHAPE, "%s: grid too large", fn);
    if (!x || !A_proj || !state || !new_state) return fail(SSD_ERR_NULL, "%s: a required pointer is NULL", fn);
    const size_t bytes = (size_t)n * (dtype == SSD_BF16 ? 2 : 4);
    const Range ins[] = {{"x", x, bytes}, {"A_proj", A_proj, bytes}, {"I_proj", I_proj, bytes},
                         {"state", state, (size_t)n * 4}};
    const Range out{"new_state", new_state, (size_t)n * 4};
    if ((s = check_aligned(ins, 4)) != SSD_OK || (s = check_aligned(&out, 1)) != SSD_OK) return s;
    // in place: state itself is the one input that the output may be
    if ((s = check_alias(&out, 1, ins, state == new_state ? 3 : 4)) != SSD_OK) return s;
    return hip_status(ssd::launch_gated_scan_step(dtype == SSD_BF16, input_scale, x, A_proj, I_proj, state,
                                                  n, new_state, stream),
                      "gated_scan_step launch");
  } catch (...) {
    return fail(SSD_ERR_HIP, "%s: unexpected exception", fn);
  }
}

size_t ssd_gated_scan_backward_workspace_size(int64_t B, int64_t H, int64_t N, int64_t d_h) {
  int64_t BH, n;
  if (gated_sizes("ssd_gated_scan_backward_workspace_size", B, H, N, d_h, &BH, &n) != SSD_OK || n == 0)
    return 0;
  return ssd::gated_scan_backward_floats(BH, N, d_h) * sizeof(float);
}

ssd_status ssd_gated_scan_backward(const void* x, const void* A_proj, const void* I_proj,
                                   const float* initial_state, const float* y, const float* dy,
                                   const float* d_final_state, int64_t B, int64_t H, int64_t N,
                                   int64_t d_h, int input_scale, int dtype, float* dx,
                                   float* dA_proj, float* dI_proj, float* d_initial_state,
                                   void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const char* fn = "ssd_gated_scan_backward";
  try {
    clear_err();
    int64_t BH, n;
    ssd_status s = gated_sizes(fn, B, H, N, d_h, &BH, &n);
    if (s != SSD_OK || (s = gated_kinds(fn, input_scale, dtype)) != SSD_OK) return s;
    if (BH == 0) return SSD_OK;
    const size_t st = (size_t)(BH * d_h) * 4;
    const Range df{"d_final_state", d_final_state, st}, d0{"d_initial_state", d_initial_state, st};
    if (n == 0) {  // no tokens: the state passes through
      if (!d_initial_state) return SSD_OK;
      if ((s = check_aligned(&df, 1)) != SSD_OK || (s = check_aligned(&d0, 1)) != SSD_OK) return s;
      if ((s = check_alias(&d0, 1, &df, 1)) != SSD_OK) return s;
      return hip_status(ssd::launch_copy_or_zero(d_initial_state, d_final_state, BH * d_h, stream),
                        "initial-state gradient copy launch");
    }
    if (!ssd::gated_scan_backward_fits(BH, N, d_h)) return fail(SSD_ERR_SHAPE, "%s: grid too large", fn);
    if (!x || !A_proj || !y || !dy || !dx || !dA_proj)
      return fail(SSD_ERR_NULL, "%s: a required pointer is NULL", fn);
    if ((I_proj == nullptr) != (dI_proj == nullptr))
      return fail(SSD_ERR_NULL, "%s: I_proj and dI_proj must be given together", fn);
    const size_t need = ssd::gated_scan_backward_floats(BH, N, d_h) * sizeof(float);
    if ((s = check_workspace(fn, workspace, workspace_bytes, need)) != SSD_OK) return s;
    const size_t bytes = (size_t)n * (dtype == SSD_BF16 ? 2 : 4), full = (size_t)n * 4;
    const Range ins[] = {{"x", x, bytes},   {"A_proj", A_proj, bytes}, {"I_proj", I_proj, bytes},
                         {"initial_state", initial_state, st},         {"y", y, full},
                         {"dy", dy, full},  df};
    const Range outs[] = {{"dx", dx, full}, {"dA_proj", dA_proj, full}, {"dI_proj", dI_proj, full}, d0,
                          {"workspace", workspace, need}};
    if ((s = check_aligned(ins, 7)) != SSD_OK || (s = check_aligned(outs, 5)) != SSD_OK) return s;
    if ((s = check_alias(outs, 5, ins, 7)) != SSD_OK) return s;
    return hip_status(ssd::launch_gated_scan_backward(dtype == SSD_BF16, input_scale, x, A_proj, I_proj,
                                                      initial_state, y, dy, d_final_state, BH, N, d_h, dx,
                                                      dA_proj, dI_proj, d_initial_state,
                                                      static_cast<float*>(workspace), stream),
                      "gated_scan_backward launch");
  } catch (...) {
    return fail(SSD_ERR_HIP, "%s: unexpected exception", fn);
  }
}

// ---- the norms around a mixer block ----

static ssd_status norm_kinds(const char* fn, int64_t E, float eps, int dtype) {
  if (E < 1) return fail(SSD_ERR_SHAPE, "%s: a norm over %lld channels", fn, (long long)E);
  if (E > SSD_NORM_MAX)
    return fail(SSD_ERR_UNSUPPORTED, "%s: a norm over %lld channels (at most %d)", fn, (long long)E, SSD_NORM_MAX);
  if (!(eps >= 0.f) || eps > 3.4028235e38f)
    return fail(SSD_ERR_UNSUPPORTED, "%s: eps must be finite and >= 0", fn);
  if (dtype != SSD_F32 && dtype != SSD_BF16) return fail(SSD_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
  return SSD_OK;
}

static ssd_status norm_in_sizes(const char* fn, int64_t rows, int64_t E, int64_t* n) {
  if (!mul_ok(rows, E, n)) return fail(SSD_ERR_SHAPE, "%s: rows must be >= 0 and rows E must not overflow", fn);
  return SSD_OK;
}

ssd_status ssd_norm_in(const float* residual, const void* branch, const float* branch_scale,
                       const float* weight, int64_t rows, int64_t E, float eps, int dtype,
                       float* residual_out, void* out, hipStream_t stream) {
  const char* fn = "ssd_norm_in";
  try {
    clear_err();
    int64_t n;
    ssd_status s = norm_kinds(fn, E, eps, dtype);
    if (s != SSD_OK || (s = norm_in_sizes(fn, rows, E, &n)) != SSD_OK) return s;
    if (n == 0) return SSD_OK;
    if (!residual || !weight || !out) return fail(SSD_ERR_NULL, "%s: a required pointer is NULL", fn);
    if ((branch == nullptr) != (residual_out == nullptr))
      return fail(SSD_ERR_NULL, "%s: branch and residual_out must be given together", fn);
    if (branch_scale && !branch) return fail(SSD_ERR_NULL, "%s: branch_scale without branch", fn);
    const size_t bytes = (size_t)n * (dtype == SSD_BF16 ? 2 : 4);
    const Range ins[] = {{"residual", residual, (size_t)n * 4}, {"branch", branch, bytes},
                         {"branch_scale", branch_scale, (size_t)E * 4}, {"weight", weight, (size_t)E * 4}};
    const Range outs[] = {{"residual_out", residual_out, (size_t)n * 4}, {"out", out, bytes}};
    if ((s = check_aligned(ins, 4)) != SSD_OK || (s = check_aligned(outs, 2)) != SSD_OK) return s;
    if ((s = check_alias(outs, 2, ins, 4)) != SSD_OK) return s;
    return hip_status(ssd::launch_norm_in(dtype == SSD_BF16, residual, branch, branch_scale, weight, rows, E,
                                          eps, residual_out, out, stream),
                      "norm_in launch");
  } catch (...) {
    return fail(SSD_ERR_HIP, "%s: unexpected exception", fn);
  }
}

size_t ssd_norm_in_backward_workspace_size(int64_t rows, int64_t E) {
  int64_t n;
  if (E < 1 || E > SSD_NORM_MAX ||
      norm_in_sizes("ssd_norm_in_backward_workspace_size", rows, E, &n) != SSD_OK || n == 0)
    return 0;
  return ssd::norm_in_backward_floats(rows, E) * sizeof(float);
}

ssd_status ssd_norm_in_backward(const void* d_out, const float* d_residual_out,
                                const float* residual_out, const void* branch,
                                const float* branch_scale, const float* weight, int64_t rows,
                                int64_t E, float eps, int dtype, float* d_residual,
                                float* d_branch, float* d_weight, float* d_branch_scale,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const char* fn = "ssd_norm_in_backward";
  try {
    clear_err();
    int64_t n;
    ssd_status s = norm_kinds(fn, E, eps, dtype);
    if (s != SSD_OK || (s = norm_in_sizes(fn, rows, E, &n)) != SSD_OK) return s;
    if (!weight || !d_weight || (n && (!d_out || !residual_out || !d_residual)))
      return fail(SSD_ERR_NULL, "%s: a required pointer is NULL", fn);
    if ((branch_scale == nullptr) != (d_branch_scale == nullptr) ||
        (n && ((branch_scale == nullptr) != (branch == nullptr) ||
               (branch_scale == nullptr) != (d_branch == nullptr))))
      return fail(SSD_ERR_NULL, "%s: branch, branch_scale, d_branch and d_branch_scale go together", fn);
    const size_t need = n ? ssd::norm_in_backward_floats(rows, E) * sizeof(float) : 0;
    if ((s = check_workspace(fn, workspace, workspace_bytes, need)) != SSD_OK) return s;
    const size_t bytes = (size_t)n * (dtype == SSD_BF16 ? 2 : 4), full = (size_t)n * 4, ch = (size_t)E * 4;
    const Range ins[] = {{"d_out", d_out, bytes},   {"d_residual_out", d_residual_out, full},
                         {"residual_out", residual_out, full},      {"branch", branch, bytes},
                         {"branch_scale", branch_scale, ch},        {"weight", weight, ch}};
    const Range outs[] = {{"d_residual", d_residual, full}, {"d_branch", d_branch, full},
                          {"d_weight", d_weight, ch},       {"d_branch_scale", d_branch_scale, ch},
                          {"workspace", workspace, need}};
    if ((s = check_aligned(ins, 6)) != SSD_OK || (s = check_aligned(outs, 5)) != SSD_OK) return s;
    if ((s = check_alias(outs, 5, ins, 6)) != SSD_OK) return s;
    return hip_status(ssd::launch_norm_in_backward(dtype == SSD_BF16, d_out, d_residual_out, residual_out,
                                                   branch, branch_scale, weight, rows, E, eps, d_residual,
                                                   d_branch, d_weight, d_branch_scale,
                                                   static_cast<float*>(workspace), stream),
                      "norm_in_backward launch");
  } catch (...) {
    return fail(SSD_ERR_HIP, "%s: unexpected exception", fn);
  }
}

// sizes of both norm_out calls; n = B H N d_h, E = H d_h
static ssd_status norm_out_sizes(const char* fn, int64_t B, int64_t H, int64_t N, int64_t d_h,
                                 int64_t groups, int64_t* n, int64_t* E) {
  int64_t BN, units;
  if (H < 1 || d_h < 1 || groups < 1 || H % groups != 0)
    return fail(SSD_ERR_SHAPE, "%s: H, d_h and groups must be >= 1 and groups must divide H", fn);
  if (!mul_ok(B, N, &BN) || !mul_ok(H, d_h, E) || !mul_ok(BN, *E, n) || !mul_ok(BN, groups, &units))
    return fail(SSD_ERR_SHAPE, "%s: B, N must be >= 0 and the product of the sizes must not overflow", fn);
  if (BN > (int64_t)0x7fffffff || *E > (int64_t)0x7fffffff)
    return fail(SSD_ERR_SHAPE, "%s: more than 2^31 - 1 tokens or channels", fn);
  // a launch has less than 2^32 threads: up to 32 groups share a workgroup of 512 (fewer where groups are
  // of more channels, of which 2^31 hold fewer groups)
  if (groups > ((int64_t)1 << 28) - 32) return fail(SSD_ERR_SHAPE, "%s: grid too large", fn);
  return SSD_OK;
}

ssd_status ssd_norm_out(const float* y, const void* z, const float* weight, int64_t B, int64_t H,
                        int64_t N, int64_t d_h, int64_t groups, int gate_first, float eps,
                        int dtype, void* out, hipStream_t stream) {
  const char* fn = "ssd_norm_out";
  try {
    clear_err();
    int64_t n, E;
    ssd_status s = norm_out_sizes(fn, B, H, N, d_h, groups, &n, &E);
    if (s != SSD_OK || (s = norm_kinds(fn, E / groups, eps, dtype)) != SSD_OK) return s;
    if (gate_first != 0 && gate_first != 1)
      return fail(SSD_ERR_UNSUPPORTED, "%s: gate_first %d (0 or 1)", fn, gate_first);
    if (n == 0) return SSD_OK;
    if (!y || !z || !weight || !out) return fail(SSD_ERR_NULL, "%s: a required pointer is NULL", fn);
    const size_t bytes = (size_t)n * (dtype == SSD_BF16 ? 2 : 4);
    const Range ins[] = {{"y", y, (size_t)n * 4}, {"z", z, bytes}, {"weight", weight, (size_t)E * 4}};
    const Range o{"out", out, bytes};
    if ((s = check_aligned(ins, 3)) != SSD_OK || (s = check_aligned(&o, 1)) != SSD_OK) return s;
    if ((s = check_alias(&o, 1, ins, 3)) != SSD_OK) return s;
    return hip_status(ssd::launch_norm_out(dtype == SSD_BF16, gate_first != 0, y, z, weight, B, H, N, d_h,
                                           groups, eps, out, stream),
                      "norm_out launch");
  } catch (...) {
    return fail(SSD_ERR_HIP, "%s: unexpected exception", fn);
  }
}

size_t ssd_norm_out_backward_workspace_size(int64_t B, int64_t H, int64_t N, int64_t d_h,
                                            int64_t groups) {
  int64_t n, E;
  if (norm_out_sizes("ssd_norm_out_backward_workspace_size", B, H, N, d_h, groups, &n, &E) != SSD_OK ||
      E / groups > SSD_NORM_MAX || n == 0)
    return 0;
  return ssd::norm_out_backward_floats(B, H, N, d_h, groups) * sizeof(float);
}

ssd_status ssd_norm_out_backward(const void* d_out, const float* y, const void* z,
                                 const float* weight, int64_t B, int64_t H, int64_t N, int64_t d_h,
                                 int64_t groups, int gate_first, float eps, int dtype, float* dy,
                                 float* dz, float* d_weight, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
  const char* fn = "ssd_norm_out_backward";
  try {
    clear_err();
    int64_t n, E;
    ssd_status s = norm_out_sizes(fn, B, H, N, d_h, groups, &n, &E);
    if (s != SSD_OK || (s = norm_kinds(fn, E / groups, eps, dtype)) != SSD_OK) return s;
    if (gate_first != 0 && gate_first != 1)
      return fail(SSD_ERR_UNSUPPORTED, "%s: gate_first %d (0 or 1)", fn, gate_first);
    if (E > ((int64_t)1 << 27) - 32)  // the weight gradients' sum has 32 threads a channel
      return fail(SSD_ERR_SHAPE, "%s: grid too large", fn);
    if (!weight || !d_weight || (n && (!d_out || !y || !z || !dy || !dz)))
      return fail(SSD_ERR_NULL, "%s: a required pointer is NULL", fn);
    const size_t need = n ? ssd::norm_out_backward_floats(B, H, N, d_h, groups) * sizeof(float) : 0;
    if ((s = check_workspace(fn, workspace, workspace_bytes, need)) != SSD_OK) return s;
    const size_t bytes = (size_t)n * (dtype == SSD_BF16 ? 2 : 4), full = (size_t)n * 4, ch = (size_t)E * 4;
    const Range ins[] = {{"d_out", d_out, bytes}, {"y", y, full}, {"z", z, bytes}, {"weight", weight, ch}};
    const Range outs[] = {{"dy", dy, full}, {"dz", dz, full}, {"d_weight", d_weight, ch},
                          {"workspace", workspace, need}};
    if ((s = check_aligned(ins, 4)) != SSD_OK || (s = check_aligned(outs, 4)) != SSD_OK) return s;
    if ((s = check_alias(outs, 4, ins, 4)) != SSD_OK) return s;
    return hip_status(ssd::launch_norm_out_backward(dtype == SSD_BF16, gate_first != 0, d_out, y, z, weight, B,
                                                    H, N, d_h, groups, eps, dy, dz, d_weight,
                                                    static_cast<float*>(workspace), stream),
                      "norm_out_backward launch");
  } catch (...) {
    return fail(SSD_ERR_HIP, "%s: unexpected exception", fn);
  }
}

}  // extern "C"
