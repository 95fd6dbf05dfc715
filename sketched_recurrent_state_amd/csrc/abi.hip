// abi.hip -- the extern "C" entry points of libsketchssm.so: argument checks
// on the host, then one asynchronous launch on the caller's stream. Nothing
// here allocates, frees or synchronises. See include/sketchssm.h.
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <string>

#include "abi_checks.hpp"
#include "launch.hpp"
#include "scan.hpp"
#include "sketchssm.h"

namespace ssm {

namespace {
thread_local std::string g_last_error;
}

ssm_status fail(ssm_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return st;
}

ssm_status ok() {
  g_last_error.clear();
  return SSM_OK;
}

ssm_status launched(hipError_t e, const char* fn) {
  if (e != hipSuccess) return fail(SSM_E_LAUNCH, "%s: launch failed: %s", fn, hipGetErrorString(e));
  return ok();
}

ssm_status check_workspace(const void* workspace, int64_t bytes, size_t need, const char* fn) {
  if (need > 0 && workspace == nullptr) return fail(SSM_E_NULL, "%s: workspace is NULL", fn);
  if (bytes < 0 || (size_t)bytes < need)
    return fail(SSM_E_RANGE, "%s: workspace of %lld bytes, %zu needed", fn, (long long)bytes, need);
  return SSM_OK;
}

const char* last_error() { return g_last_error.c_str(); }

// Whether two arrays share a byte. Rows with one stride are compared column range by column range.
static bool overlap(const Arr& a, const Arr& b) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t a1 = a0 + (a.rows - 1) * a.stride + a.bytes;
  const uintptr_t b1 = b0 + (b.rows - 1) * b.stride + b.bytes;
  if (a1 <= b0 || b1 <= a0) return false;
  if (a.stride != b.stride || a.stride == 0) return true;
  // b's columns begin r bytes into a row that begins with a's
  const size_t r = b0 >= a0 ? (b0 - a0) % a.stride : (a.stride - (a0 - b0) % a.stride) % a.stride;
  return r < a.bytes || r + b.bytes > a.stride;
}

ssm_status check_arrays(const char* fn, const Arr* arrs, size_t n) {
  for (size_t i = 0; i < n; ++i) {
    const Arr& a = arrs[i];
    if (a.p != nullptr && (reinterpret_cast<uintptr_t>(a.p) & (a.align - 1)) != 0)
      return fail(SSM_E_ALIGN, "%s: %s (%p) is not %u-byte aligned", fn, a.name, a.p, a.align);
  }
  for (size_t i = 0; i < n; ++i) {
    const Arr& a = arrs[i];
    if (a.p == nullptr || a.bytes == 0 || a.rows == 0) continue;
    for (size_t j = 0; j < n; ++j) {
      const Arr& b = arrs[j];
      if (i == j || b.p == nullptr || b.bytes == 0 || b.rows == 0) continue;
      if (!a.output && !b.output) continue;
      if (overlap(a, b)) return fail(SSM_E_ALIAS, "%s: %s overlaps %s", fn, a.name, b.name);
    }
  }
  return SSM_OK;
}

}  // namespace ssm

namespace {

using ssm::Arr;
using ssm::check_arrays;
using ssm::check_workspace;
using ssm::fail;
using ssm::launched;
using ssm::ok;

constexpr long long kMaxUnits = 1LL << 24;  // keeps every grid below 2^32 threads

bool in_set(int x, std::initializer_list<int> s) {
  for (int v : s)
    if (v == x) return true;
  return false;
}

ssm_status check_dims(const ssm_dims* d, const char* fn) {
  if (d == nullptr) return fail(SSM_E_NULL, "%s: dims is NULL", fn);
  if (d->rule < SSM_MAMBA2 || d->rule > SSM_KDA)
    return fail(SSM_E_RANGE, "%s: rule %d is not 0 (Mamba-2), 1 (GDN) or 2 (KDA)", fn, d->rule);
  if (d->in_dtype != SSM_IN_BF16 && d->in_dtype != SSM_IN_F32)
    return fail(SSM_E_RANGE, "%s: in_dtype %d is not 0 (bf16) or 1 (fp32)", fn, d->in_dtype);
  if (d->sketch_dtype != SSM_SKETCH_F32 && d->sketch_dtype != SSM_SKETCH_BF16)
    return fail(SSM_E_RANGE, "%s: sketch_dtype %d is not 0 (fp32) or 1 (bf16)", fn,
                d->sketch_dtype);
  if (d->batch < 0) return fail(SSM_E_SHAPE, "%s: batch %d < 0", fn, d->batch);
  if (d->heads < 1) return fail(SSM_E_SHAPE, "%s: heads %d < 1", fn, d->heads);
  if (!in_set(d->d_k, {16, 32, 64, 128}))
    return fail(SSM_E_SHAPE, "%s: d_k %d not in {16, 32, 64, 128}", fn, d->d_k);
  if (!in_set(d->d_v, {16, 32, 64, 128}))
    return fail(SSM_E_SHAPE, "%s: d_v %d not in {16, 32, 64, 128}", fn, d->d_v);
  if (d->window < 1 || d->window > 16)
    return fail(SSM_E_SHAPE, "%s: window %d not in [1, 16]", fn, d->window);
  const int rmax = d->d_k < 32 ? d->d_k : 32;
  if (d->rank < 1 || d->rank > rmax)
    return fail(SSM_E_SHAPE, "%s: rank %d not in [1, %d]", fn, d->rank, rmax);
  if ((long long)d->batch * d->heads >= kMaxUnits)
    return fail(SSM_E_SHAPE, "%s: batch*heads = %lld >= %lld", fn,
                (long long)d->batch * d->heads, kMaxUnits);
  return SSM_OK;
}

struct Sizes {
  size_t units, elem, sk_elem, state, sketch, basis, kbuf, vbuf, dbuf, bbuf, qk, v, dtok, btok, y;
};

Sizes sizes_of(const ssm_dims& d) {
  Sizes z;
  z.units = (size_t)d.batch * (size_t)d.heads;
  z.elem = d.in_dtype == SSM_IN_BF16 ? 2 : 4;
  z.sk_elem = d.sketch_dtype == SSM_SKETCH_BF16 ? 2 : 4;
  const size_t dstr = d.rule == SSM_KDA ? (size_t)d.d_k : 1;
  const size_t W = (size_t)d.window;
  z.state = z.units * d.d_k * d.d_v * 4;
  z.sketch = z.units * d.rank * d.d_v * z.sk_elem;
  z.basis = (size_t)d.heads * d.rank * d.d_k * 4;
  z.kbuf = z.units * W * d.d_k * z.elem;
  z.vbuf = z.units * W * d.d_v * z.elem;
  z.dbuf = z.units * W * dstr * 4;
  z.bbuf = z.units * W * 4;
  z.qk = z.units * d.d_k * z.elem;
  z.v = z.units * d.d_v * z.elem;
  z.dtok = z.units * dstr * 4;
  z.btok = z.units * 4;
  z.y = z.units * d.d_v * 4;
  return z;
}

ssm_status check_beta(const ssm_dims& d, const void* beta, const char* what, const char* fn) {
  if (d.rule == SSM_MAMBA2 && beta != nullptr)
    return fail(SSM_E_RANGE, "%s: %s must be NULL for Mamba-2", fn, what);
  if (d.rule != SSM_MAMBA2 && beta == nullptr)
    return fail(SSM_E_NULL, "%s: %s is NULL (required by the delta rules)", fn, what);
  return SSM_OK;
}

// The current-token pointers of a fused append: all present or all absent.
ssm_status check_token(const ssm_dims& d, const void* k_t, const void* v_t, const void* d_t,
                       const void* b_t, const char* fn) {
  if (k_t == nullptr) {
    if (v_t != nullptr || d_t != nullptr || b_t != nullptr)
      return fail(SSM_E_RANGE, "%s: k_t is NULL but v_t/decay_t/beta_t are not", fn);
    return SSM_OK;
  }
  if (v_t == nullptr) return fail(SSM_E_NULL, "%s: v_t is NULL", fn);
  if (d_t == nullptr) return fail(SSM_E_NULL, "%s: decay_t is NULL", fn);
  return check_beta(d, b_t, "beta_t", fn);
}

ssm_status check_buffers(const ssm_dims& d, const void* k_buf, const void* v_buf,
                         const void* decay_buf, const void* beta_buf, const char* fn) {
  if (k_buf == nullptr) return fail(SSM_E_NULL, "%s: k_buf is NULL", fn);
  if (v_buf == nullptr) return fail(SSM_E_NULL, "%s: v_buf is NULL", fn);
  if (decay_buf == nullptr) return fail(SSM_E_NULL, "%s: decay_buf is NULL", fn);
  return check_beta(d, beta_buf, "beta_buf", fn);
}

// Per-head rank table (host array of heads + 1 prefix offsets).
ssm_status check_rank_offsets(const ssm_dims& d, const int32_t* off, const char* fn) {
  if (off == nullptr) return fail(SSM_E_NULL, "%s: rank_offsets is NULL", fn);
  if (d.heads > ssm::kMaxRankedHeads)
    return fail(SSM_E_SHAPE, "%s: %d heads > %d supported with per-head ranks", fn, d.heads,
                ssm::kMaxRankedHeads);
  if (off[0] != 0) return fail(SSM_E_RANGE, "%s: rank_offsets[0] = %d, not 0", fn, off[0]);
  const int rmax = d.d_k < 32 ? d.d_k : 32;
  for (int h = 0; h < d.heads; ++h) {
    const long long r = (long long)off[h + 1] - off[h];
    if (r < 1 || r > rmax)
      return fail(SSM_E_RANGE, "%s: head %d has rank %lld, not in [1, %d]", fn, h, r, rmax);
  }
  return SSM_OK;
}

// Sketch and basis bytes for a per-head rank table (or the uniform rank when off is NULL).
void apply_ranks(const ssm_dims& d, const int32_t* off, Sizes& z) {
  if (off == nullptr) return;
  const size_t R = (size_t)off[d.heads];
  z.sketch = z.units / (size_t)d.heads * R * d.d_v * z.sk_elem;
  z.basis = R * d.d_k * 4;
}

// A variable-length call: `batch` rows mapped onto a pool of num_slots persistent slots.
ssm_status check_pool(const ssm_dims& d, int32_t num_slots, const int32_t* slot,
                      const int32_t* counts, const char* what, const char* fn) {
  if (num_slots < 1) return fail(SSM_E_SHAPE, "%s: num_slots %d < 1", fn, num_slots);
  if ((long long)num_slots * d.heads >= kMaxUnits)
    return fail(SSM_E_SHAPE, "%s: num_slots*heads = %lld >= %lld", fn,
                (long long)num_slots * d.heads, kMaxUnits);
  if (slot == nullptr && d.batch > num_slots)
    return fail(SSM_E_SHAPE, "%s: %d rows but %d slots and no slot map", fn, d.batch, num_slots);
  if (counts == nullptr) return fail(SSM_E_NULL, "%s: %s is NULL", fn, what);
  return SSM_OK;
}

// Sizes of the persistent arrays (state, sketch, window buffer) for a pool of slots.
Sizes pool_sizes(const ssm_dims& d, int32_t num_slots) {
  ssm_dims p = d;
  p.batch = num_slots;
  const Sizes zp = sizes_of(p);
  Sizes z = sizes_of(d);
  z.state = zp.state;
  z.sketch = zp.sketch;
  z.kbuf = zp.kbuf;
  z.vbuf = zp.vbuf;
  z.dbuf = zp.dbuf;
  z.bbuf = zp.bbuf;
  return z;
}

// Whole-sequence calls: the cells (chunk, head) of a packed batch bound every grid of the scan
// (at most 1,024 threads a cell), so this keeps them below 2^32 threads.
constexpr long long kMaxCells = 1LL << 22;
constexpr int kMaxScanHeads = 1 << 16;

ssm_status check_scan(const ssm_dims* d, int32_t total_tokens, const char* fn) {
  ssm_status st = check_dims(d, fn);
  if (st != SSM_OK) return st;
  if (total_tokens < 0) return fail(SSM_E_SHAPE, "%s: total_tokens %d < 0", fn, total_tokens);
  if (d->heads > kMaxScanHeads)  // a block's 16 tokens within 32-bit byte offsets
    return fail(SSM_E_SHAPE, "%s: %d heads > %d", fn, d->heads, kMaxScanHeads);
  const long long cells =
      ((long long)total_tokens / ssm::CT + d->batch) * d->heads;
  if (cells >= kMaxCells)
    return fail(SSM_E_SHAPE, "%s: (total_tokens/64 + batch)*heads = %lld >= %lld", fn, cells,
                kMaxCells);
  return SSM_OK;
}

// The token arrays of a packed batch; they may be NULL when it holds no token.
ssm_status check_packed(const ssm_dims& d, int32_t total_tokens, const int32_t* plan,
                        const void* q, const void* k, const void* v, const void* decay,
                        const void* beta, const char* fn) {
  if (plan == nullptr) return fail(SSM_E_NULL, "%s: plan is NULL", fn);
  if (total_tokens == 0) return SSM_OK;
  if (q == nullptr) return fail(SSM_E_NULL, "%s: q is NULL", fn);
  if (k == nullptr) return fail(SSM_E_NULL, "%s: k is NULL", fn);
  if (v == nullptr) return fail(SSM_E_NULL, "%s: v is NULL", fn);
  if (decay == nullptr) return fail(SSM_E_NULL, "%s: decay is NULL", fn);
  return check_beta(d, beta, "beta", fn);
}

struct PackedSizes {
  size_t plan, qk, v, gate, beta, y;
  unsigned gate_align;  // one value per token is read alone, KDA's channels four at a time
};

PackedSizes packed_sizes(const ssm_dims& d, int32_t total_tokens) {
  const size_t rows = (size_t)total_tokens * d.heads, e = d.in_dtype == SSM_IN_BF16 ? 2 : 4;
  PackedSizes z;
  z.plan = (2 * ((size_t)d.batch + 1) + ssm::scan_capacity(total_tokens, d.batch)) * 4;
  z.qk = rows * d.d_k * e;
  z.v = rows * d.d_v * e;
  z.gate = rows * (d.rule == SSM_KDA ? d.d_k : 1) * 4;
  z.gate_align = d.rule == SSM_KDA ? 16 : 4;
  z.beta = rows * 4;
  z.y = rows * d.d_v * 4;
  return z;
}

hipError_t launch_scan(const ssm_dims& d, const ssm::ScanArgs& a, bool backward, void* stream) {
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  switch (d.rule) {
    case SSM_MAMBA2: return ssm::launch_scan_rule<ssm::MAMBA2>(d, a, backward, s);
    case SSM_GDN: return ssm::launch_scan_rule<ssm::GDN>(d, a, backward, s);
  }
  return ssm::launch_scan_rule<ssm::KDA>(d, a, backward, s);
}

}  // namespace

extern "C" {

int32_t ssm_abi_version(void) { return SSM_ABI_VERSION; }

const char* ssm_status_string(int32_t status) {
  switch (status) {
    case SSM_OK: return "ok";
    case SSM_E_NULL: return "a required pointer is NULL";
    case SSM_E_SHAPE: return "unsupported or inconsistent dimensions";
    case SSM_E_ALIGN: return "a pointer is not 16-byte aligned";
    case SSM_E_RANGE: return "an argument is out of range";
    case SSM_E_ALIAS: return "an output overlaps an input";
    case SSM_E_LAUNCH: return "kernel launch failed";
  }
  return "unknown status";
}

const char* ssm_last_error(void) { return ssm::last_error(); }

ssm_status ssm_buffer_append(const ssm_dims* d, const void* k_t, const void* v_t,
                             const float* decay_t, const float* beta_t, void* k_buf, void* v_buf,
                             float* decay_buf, float* beta_buf, int32_t slot, void* stream) {
  static const char* fn = "ssm_buffer_append";
  ssm_status st = check_dims(d, fn);
  if (st != SSM_OK) return st;
  if (slot < 0 || slot >= d->window)
    return fail(SSM_E_RANGE, "%s: slot %d not in [0, %d)", fn, slot, d->window);
  if (d->batch == 0) return ok();
  if (k_t == nullptr) return fail(SSM_E_NULL, "%s: k_t is NULL", fn);
  if ((st = check_token(*d, k_t, v_t, decay_t, beta_t, fn)) != SSM_OK) return st;
  if ((st = check_buffers(*d, k_buf, v_buf, decay_buf, beta_buf, fn)) != SSM_OK) return st;
  const Sizes z = sizes_of(*d);
  st = check_arrays(fn, {{k_t, z.qk, false, "k_t"}, {v_t, z.v, false, "v_t"},
                         {decay_t, z.dtok, false, "decay_t"}, {beta_t, z.btok, false, "beta_t"},
                         {k_buf, z.kbuf, true, "k_buf"}, {v_buf, z.vbuf, true, "v_buf"},
                         {decay_buf, z.dbuf, true, "decay_buf"},
                         {beta_buf, z.bbuf, true, "beta_buf"}});
  if (st != SSM_OK) return st;
  (void)hipGetLastError();
  return launched(ssm::launch_buffer_append(*d, k_t, v_t, decay_t, beta_t, k_buf, v_buf,
                                            decay_buf, beta_buf, slot,
                                            reinterpret_cast<hipStream_t>(stream)),
                  fn);
}

static ssm_status update_refresh_impl(const char* fn, const ssm_dims* d, const int32_t* rank_offsets,
                               float* state, void* sketch, const float* basis, const void* k_buf,
                               const void* v_buf, const float* decay_buf, const float* beta_buf,
                               int32_t n_tokens, void* stream, bool ranked,
                               float* read_map = nullptr, bool ls = false) {
  ssm_status st = check_dims(d, fn);
  if (st != SSM_OK) return st;
  if (ranked && (st = check_rank_offsets(*d, rank_offsets, fn)) != SSM_OK) return st;
  if (n_tokens < 0 || n_tokens > d->window)
    return fail(SSM_E_RANGE, "%s: n_tokens %d not in [0, %d]", fn, n_tokens, d->window);
  if (d->batch == 0) return ok();
  if (state == nullptr) return fail(SSM_E_NULL, "%s: state is NULL", fn);
  if (ls) {
    if (d->sketch_dtype != SSM_SKETCH_F32)
      return fail(SSM_E_RANGE, "%s: least-squares coefficients need an fp32 sketch", fn);
    if (sketch == nullptr) return fail(SSM_E_NULL, "%s: sketch_q is NULL", fn);
    if (read_map == nullptr) return fail(SSM_E_NULL, "%s: read_map is NULL", fn);
  }
  if (sketch != nullptr && basis == nullptr)
    return fail(SSM_E_NULL, "%s: basis is NULL but a sketch is requested", fn);
  if (n_tokens > 0) {
    if ((st = check_buffers(*d, k_buf, v_buf, decay_buf, beta_buf, fn)) != SSM_OK) return st;
  }
  if (n_tokens == 0 && sketch == nullptr) return ok();  // nothing to apply, nothing to store
  Sizes z = sizes_of(*d);
  apply_ranks(*d, rank_offsets, z);
  const bool tok = n_tokens > 0;
  const size_t map_bytes = z.units * d->rank * d->d_k * 4;
  st = check_arrays(fn, {{state, z.state, true, "state"}, {sketch, z.sketch, true, ls ? "sketch_q" : "sketch"},
                         {read_map, map_bytes, true, "read_map"},
                         {basis, z.basis, false, "basis"},
                         {tok ? k_buf : nullptr, z.kbuf, false, "k_buf"},
                         {tok ? v_buf : nullptr, z.vbuf, false, "v_buf"},
                         {tok ? decay_buf : nullptr, z.dbuf, false, "decay_buf"},
                         {tok ? beta_buf : nullptr, z.bbuf, false, "beta_buf"}});
  if (st != SSM_OK) return st;
  (void)hipGetLastError();
  return launched(ssm::launch_update_refresh(*d, rank_offsets, state, sketch, basis, k_buf, v_buf, decay_buf,
                                             beta_buf, n_tokens,
                                             reinterpret_cast<hipStream_t>(stream), nullptr,
                                             read_map),
                  fn);
}

static ssm_status sketch_decode_impl(const char* fn, const ssm_dims* d, const int32_t* rank_offsets,
                              const void* sketch, const float* basis, const void* q,
                              const void* k_t, const void* v_t, const float* decay_t,
                              const float* beta_t, void* k_buf, void* v_buf, float* decay_buf,
                              float* beta_buf, int32_t tau, float* y, void* stream, bool ranked,
                              bool ls = false) {
  ssm_status st = check_dims(d, fn);
  if (st != SSM_OK) return st;
  if (ranked && (st = check_rank_offsets(*d, rank_offsets, fn)) != SSM_OK) return st;
  if (tau < 1 || tau > d->window)
    return fail(SSM_E_RANGE, "%s: tau %d not in [1, %d]", fn, tau, d->window);
  if (d->batch == 0) return ok();
  if (ls && d->sketch_dtype != SSM_SKETCH_F32)
    return fail(SSM_E_RANGE, "%s: least-squares coefficients need an fp32 sketch", fn);
  if (sketch == nullptr) return fail(SSM_E_NULL, "%s: %s is NULL", fn, ls ? "sketch_q" : "sketch");
  if (basis == nullptr) return fail(SSM_E_NULL, "%s: %s is NULL", fn, ls ? "read_map" : "basis");
  if (q == nullptr) return fail(SSM_E_NULL, "%s: q is NULL", fn);
  if (y == nullptr) return fail(SSM_E_NULL, "%s: y is NULL", fn);
  if ((st = check_token(*d, k_t, v_t, decay_t, beta_t, fn)) != SSM_OK) return st;
  if ((st = check_buffers(*d, k_buf, v_buf, decay_buf, beta_buf, fn)) != SSM_OK) return st;
  Sizes z = sizes_of(*d);
  apply_ranks(*d, rank_offsets, z);
  if (ls) z.basis = z.units * d->rank * d->d_k * 4;  // the per-unit read map
  const bool fused = k_t != nullptr;
  st = check_arrays(fn, {{sketch, z.sketch, false, ls ? "sketch_q" : "sketch"},
                         {basis, z.basis, false, ls ? "read_map" : "basis"},
                         {q, z.qk, false, "q"}, {k_t, z.qk, false, "k_t"}, {v_t, z.v, false, "v_t"},
                         {decay_t, z.dtok, false, "decay_t"}, {beta_t, z.btok, false, "beta_t"},
                         {k_buf, z.kbuf, fused, "k_buf"}, {v_buf, z.vbuf, fused, "v_buf"},
                         {decay_buf, z.dbuf, fused, "decay_buf"},
                         {beta_buf, z.bbuf, fused, "beta_buf"}, {y, z.y, true, "y"}});
  if (st != SSM_OK) return st;
  (void)hipGetLastError();
  return launched(ssm::launch_sketch_decode(*d, rank_offsets, sketch, basis, q, k_t, v_t, decay_t, beta_t,
                                            k_buf, v_buf, decay_buf, beta_buf, tau, y,
                                            reinterpret_cast<hipStream_t>(stream), nullptr, ls),
                  fn);
}

ssm_status ssm_full_read_decode_step(const ssm_dims* d, const float* state, const void* q,
                                     const void* k_t, const void* v_t, const float* decay_t,
                                     const float* beta_t, void* k_buf, void* v_buf,
                                     float* decay_buf, float* beta_buf, int32_t tau, float* y,
                                     void* stream) {
  static const char* fn = "ssm_full_read_decode_step";
  ssm_status st = check_dims(d, fn);
  if (st != SSM_OK) return st;
  if (tau < 1 || tau > d->window)
    return fail(SSM_E_RANGE, "%s: tau %d not in [1, %d]", fn, tau, d->window);
  if (d->batch == 0) return ok();
  if (state == nullptr) return fail(SSM_E_NULL, "%s: state is NULL", fn);
  if (q == nullptr) return fail(SSM_E_NULL, "%s: q is NULL", fn);
  if (y == nullptr) return fail(SSM_E_NULL, "%s: y is NULL", fn);
  if ((st = check_token(*d, k_t, v_t, decay_t, beta_t, fn)) != SSM_OK) return st;
  if ((st = check_buffers(*d, k_buf, v_buf, decay_buf, beta_buf, fn)) != SSM_OK) return st;
  const Sizes z = sizes_of(*d);
  const bool fused = k_t != nullptr;
  st = check_arrays(fn, {{state, z.state, false, "state"}, {q, z.qk, false, "q"},
                         {k_t, z.qk, false, "k_t"}, {v_t, z.v, false, "v_t"},
                         {decay_t, z.dtok, false, "decay_t"}, {beta_t, z.btok, false, "beta_t"},
                         {k_buf, z.kbuf, fused, "k_buf"}, {v_buf, z.vbuf, fused, "v_buf"},
                         {decay_buf, z.dbuf, fused, "decay_buf"},
                         {beta_buf, z.bbuf, fused, "beta_buf"}, {y, z.y, true, "y"}});
  if (st != SSM_OK) return st;
  (void)hipGetLastError();
  return launched(ssm::launch_full_read_decode(*d, state, q, k_t, v_t, decay_t, beta_t, k_buf,
                                               v_buf, decay_buf, beta_buf, tau, y,
                                               reinterpret_cast<hipStream_t>(stream)),
                  fn);
}

ssm_status ssm_recurrent_decode_step(const ssm_dims* d, float* state, const void* q,
                                     const void* k_t, const void* v_t, const float* decay_t,
                                     const float* beta_t, float* y, void* stream) {
  static const char* fn = "ssm_recurrent_decode_step";
  ssm_status st = check_dims(d, fn);
  if (st != SSM_OK) return st;
  if (d->batch == 0) return ok();
  if (state == nullptr) return fail(SSM_E_NULL, "%s: state is NULL", fn);
  if (q == nullptr) return fail(SSM_E_NULL, "%s: q is NULL", fn);
  if (y == nullptr) return fail(SSM_E_NULL, "%s: y is NULL", fn);
  if (k_t == nullptr) return fail(SSM_E_NULL, "%s: k_t is NULL", fn);
  if ((st = check_token(*d, k_t, v_t, decay_t, beta_t, fn)) != SSM_OK) return st;
  const Sizes z = sizes_of(*d);
  st = check_arrays(fn, {{state, z.state, true, "state"}, {q, z.qk, false, "q"},
                         {k_t, z.qk, false, "k_t"}, {v_t, z.v, false, "v_t"},
                         {decay_t, z.dtok, false, "decay_t"}, {beta_t, z.btok, false, "beta_t"},
                         {y, z.y, true, "y"}});
  if (st != SSM_OK) return st;
  (void)hipGetLastError();
  return launched(ssm::launch_recurrent_step(*d, state, q, k_t, v_t, decay_t, beta_t, y,
                                             reinterpret_cast<hipStream_t>(stream)),
                  fn);
}

ssm_status ssm_fit_basis(const ssm_dims* d, const void* samples, int32_t n_samples,
                         float* basis, void* stream) {
  static const char* fn = "ssm_fit_basis";
  ssm_status st = check_dims(d, fn);
  if (st != SSM_OK) return st;
  if (samples == nullptr) return fail(SSM_E_NULL, "%s: samples is NULL", fn);
  if (basis == nullptr) return fail(SSM_E_NULL, "%s: basis is NULL", fn);
  if (n_samples < 1 || n_samples > (1 << 24))
    return fail(SSM_E_SHAPE, "%s: n_samples %d not in [1, 2^24]", fn, n_samples);
  const Sizes z = sizes_of(*d);
  const size_t sample_bytes = (size_t)d->heads * (size_t)n_samples * d->d_k * z.elem;
  st = check_arrays(fn, {{samples, sample_bytes, false, "samples"}, {basis, z.basis, true, "basis"}});
  if (st != SSM_OK) return st;
  (void)hipGetLastError();
  return launched(ssm::launch_fit_basis(*d, samples, n_samples, basis,
                                        reinterpret_cast<hipStream_t>(stream)),
                  fn);
}

ssm_status ssm_stream_probe(float* buf, int64_t n_tiles, int32_t shape, void* stream) {
  static const char* fn = "ssm_stream_probe";
  if (buf == nullptr) return fail(SSM_E_NULL, "%s: buf is NULL", fn);
  if (shape != 0 && shape != 1) return fail(SSM_E_RANGE, "%s: shape %d is not 0 or 1", fn, shape);
  if (n_tiles < 1 || n_tiles >= kMaxUnits)
    return fail(SSM_E_SHAPE, "%s: n_tiles %lld not in [1, 2^24)", fn, (long long)n_tiles);
  if (shape == 1 && (n_tiles & 1))
    return fail(SSM_E_SHAPE, "%s: shape 1 needs an even n_tiles (got %lld)", fn, (long long)n_tiles);
  ssm_status st = check_arrays(fn, {{buf, (size_t)n_tiles * 65536, true, "buf"}});
  if (st != SSM_OK) return st;
  (void)hipGetLastError();
  return launched(ssm::launch_stream_probe(buf, (long long)n_tiles, shape,
                                           reinterpret_cast<hipStream_t>(stream)),
                  fn);
}

ssm_status ssm_window_update_refresh(const ssm_dims* d, float* state, void* sketch,
                                     const float* basis, const void* k_buf, const void* v_buf,
                                     const float* decay_buf, const float* beta_buf,
                                     int32_t n_tokens, void* stream) {
  return update_refresh_impl("ssm_window_update_refresh", d, nullptr, state, sketch, basis, k_buf,
                             v_buf, decay_buf, beta_buf, n_tokens, stream, false);
}

ssm_status ssm_window_update_refresh_ranked(const ssm_dims* d, const int32_t* rank_offsets,
                                            float* state, void* sketch, const float* basis,
                                            const void* k_buf, const void* v_buf,
                                            const float* decay_buf, const float* beta_buf,
                                            int32_t n_tokens, void* stream) {
  return update_refresh_impl("ssm_window_update_refresh_ranked", d, rank_offsets, state, sketch,
                             basis, k_buf, v_buf, decay_buf, beta_buf, n_tokens, stream, true);
}

ssm_status ssm_sketch_decode_step(const ssm_dims* d, const void* sketch, const float* basis,
                                  const void* q, const void* k_t, const void* v_t,
                                  const float* decay_t, const float* beta_t, void* k_buf,
                                  void* v_buf, float* decay_buf, float* beta_buf, int32_t tau,
                                  float* y, void* stream) {
  return sketch_decode_impl("ssm_sketch_decode_step", d, nullptr, sketch, basis, q, k_t, v_t,
                            decay_t, beta_t, k_buf, v_buf, decay_buf, beta_buf, tau, y, stream,
                            false);
}

ssm_status ssm_sketch_decode_step_ranked(const ssm_dims* d, const int32_t* rank_offsets,
                                         const void* sketch, const float* basis, const void* q,
                                         const void* k_t, const void* v_t, const float* decay_t,
                                         const float* beta_t, void* k_buf, void* v_buf,
                                         float* decay_buf, float* beta_buf, int32_t tau, float* y,
                                         void* stream) {
  return sketch_decode_impl("ssm_sketch_decode_step_ranked", d, rank_offsets, sketch, basis, q,
                            k_t, v_t, decay_t, beta_t, k_buf, v_buf, decay_buf, beta_buf, tau, y,
                            stream, true);
}

ssm_status ssm_window_update_refresh_ls(const ssm_dims* d, float* state, float* sketch_q,
                                        float* read_map, const float* basis, const void* k_buf,
                                        const void* v_buf, const float* decay_buf,
                                        const float* beta_buf, int32_t n_tokens, void* stream) {
  return update_refresh_impl("ssm_window_update_refresh_ls", d, nullptr, state, sketch_q, basis,
                             k_buf, v_buf, decay_buf, beta_buf, n_tokens, stream, false, read_map,
                             true);
}

ssm_status ssm_sketch_decode_step_ls(const ssm_dims* d, const float* sketch_q,
                                     const float* read_map, const void* q, const void* k_t,
                                     const void* v_t, const float* decay_t,
                                     const float* beta_t, void* k_buf, void* v_buf,
                                     float* decay_buf, float* beta_buf, int32_t tau, float* y,
                                     void* stream) {
  return sketch_decode_impl("ssm_sketch_decode_step_ls", d, nullptr, sketch_q, read_map, q, k_t,
                            v_t, decay_t, beta_t, k_buf, v_buf, decay_buf, beta_buf, tau, y,
                            stream, false, true);
}

ssm_status ssm_window_update_refresh_varlen(const ssm_dims* d, int32_t num_slots,
                                            const int32_t* slot, const int32_t* n_tokens,
                                            float* state, void* sketch, const float* basis,
                                            const void* k_buf, const void* v_buf,
                                            const float* decay_buf, const float* beta_buf,
                                            void* stream) {
  static const char* fn = "ssm_window_update_refresh_varlen";
  ssm_status st = check_dims(d, fn);
  if (st != SSM_OK) return st;
  if (d->batch == 0) return ok();
  if ((st = check_pool(*d, num_slots, slot, n_tokens, "n_tokens", fn)) != SSM_OK) return st;
  if (state == nullptr) return fail(SSM_E_NULL, "%s: state is NULL", fn);
  if (sketch != nullptr && basis == nullptr)
    return fail(SSM_E_NULL, "%s: basis is NULL but a sketch is requested", fn);
  if ((st = check_buffers(*d, k_buf, v_buf, decay_buf, beta_buf, fn)) != SSM_OK) return st;
  const Sizes z = pool_sizes(*d, num_slots);
  const size_t rows = (size_t)d->batch * 4;
  st = check_arrays(fn, {{state, z.state, true, "state"}, {sketch, z.sketch, true, "sketch"},
                         {basis, z.basis, false, "basis"}, {k_buf, z.kbuf, false, "k_buf"},
                         {v_buf, z.vbuf, false, "v_buf"}, {decay_buf, z.dbuf, false, "decay_buf"},
                         {beta_buf, z.bbuf, false, "beta_buf"},
                         {slot, rows, false, "slot", 4}, {n_tokens, rows, false, "n_tokens", 4}});
  if (st != SSM_OK) return st;
  const ssm::Varlen vl{slot, n_tokens, num_slots, 0, d->window};
  (void)hipGetLastError();
  return launched(ssm::launch_update_refresh(*d, nullptr, state, sketch, basis, k_buf, v_buf,
                                             decay_buf, beta_buf, 0,
                                             reinterpret_cast<hipStream_t>(stream), &vl),
                  fn);
}

ssm_status ssm_sketch_decode_step_varlen(const ssm_dims* d, int32_t num_slots,
                                         const int32_t* slot, const int32_t* tau,
                                         const void* sketch, const float* basis, const void* q,
                                         const void* k_t, const void* v_t, const float* decay_t,
                                         const float* beta_t, void* k_buf, void* v_buf,
                                         float* decay_buf, float* beta_buf, float* y,
                                         void* stream) {
  static const char* fn = "ssm_sketch_decode_step_varlen";
  ssm_status st = check_dims(d, fn);
  if (st != SSM_OK) return st;
  if (d->batch == 0) return ok();
  if ((st = check_pool(*d, num_slots, slot, tau, "tau", fn)) != SSM_OK) return st;
  if (sketch == nullptr) return fail(SSM_E_NULL, "%s: sketch is NULL", fn);
  if (basis == nullptr) return fail(SSM_E_NULL, "%s: basis is NULL", fn);
  if (q == nullptr) return fail(SSM_E_NULL, "%s: q is NULL", fn);
  if (y == nullptr) return fail(SSM_E_NULL, "%s: y is NULL", fn);
  if ((st = check_token(*d, k_t, v_t, decay_t, beta_t, fn)) != SSM_OK) return st;
  if ((st = check_buffers(*d, k_buf, v_buf, decay_buf, beta_buf, fn)) != SSM_OK) return st;
  const Sizes z = pool_sizes(*d, num_slots);
  const size_t rows = (size_t)d->batch * 4;
  const bool fused = k_t != nullptr;
  st = check_arrays(fn, {{sketch, z.sketch, false, "sketch"}, {basis, z.basis, false, "basis"},
                         {q, z.qk, false, "q"}, {k_t, z.qk, false, "k_t"}, {v_t, z.v, false, "v_t"},
                         {decay_t, z.dtok, false, "decay_t"}, {beta_t, z.btok, false, "beta_t"},
                         {k_buf, z.kbuf, fused, "k_buf"}, {v_buf, z.vbuf, fused, "v_buf"},
                         {decay_buf, z.dbuf, fused, "decay_buf"},
                         {beta_buf, z.bbuf, fused, "beta_buf"}, {y, z.y, true, "y"},
                         {slot, rows, false, "slot", 4}, {tau, rows, false, "tau", 4}});
  if (st != SSM_OK) return st;
  const ssm::Varlen vl{slot, tau, num_slots, 1, d->window};
  (void)hipGetLastError();
  return launched(ssm::launch_sketch_decode(*d, nullptr, sketch, basis, q, k_t, v_t, decay_t,
                                            beta_t, k_buf, v_buf, decay_buf, beta_buf, 0, y,
                                            reinterpret_cast<hipStream_t>(stream), &vl),
                  fn);
}

ssm_status ssm_decode_step_varlen(const ssm_dims* d, int32_t num_slots, const int32_t* slot,
                                  const int32_t* tau, const int32_t* parity, int32_t n_update,
                                  const int32_t* update_rows, float* state, void* sketch0,
                                  void* sketch1, const float* basis, const void* q,
                                  const void* k_t, const void* v_t, const float* decay_t,
                                  const float* beta_t, void* k_buf, void* v_buf,
                                  float* decay_buf, float* beta_buf, float* y, void* stream) {
  static const char* fn = "ssm_decode_step_varlen";
  ssm_status st = check_dims(d, fn);
  if (st != SSM_OK) return st;
  if (n_update < 0 || n_update > d->batch)
    return fail(SSM_E_RANGE, "%s: n_update %d not in [0, batch = %d]", fn, n_update, d->batch);
  if (d->batch == 0) return ok();
  if ((st = check_pool(*d, num_slots, slot, tau, "tau", fn)) != SSM_OK) return st;
  if (parity == nullptr) return fail(SSM_E_NULL, "%s: parity is NULL", fn);
  if (n_update > 0 && update_rows == nullptr)
    return fail(SSM_E_NULL, "%s: update_rows is NULL with n_update = %d", fn, n_update);
  if (state == nullptr) return fail(SSM_E_NULL, "%s: state is NULL", fn);
  if (sketch0 == nullptr) return fail(SSM_E_NULL, "%s: sketch0 is NULL", fn);
  if (sketch1 == nullptr) return fail(SSM_E_NULL, "%s: sketch1 is NULL", fn);
  if (basis == nullptr) return fail(SSM_E_NULL, "%s: basis is NULL", fn);
  if (q == nullptr) return fail(SSM_E_NULL, "%s: q is NULL", fn);
  if (y == nullptr) return fail(SSM_E_NULL, "%s: y is NULL", fn);
  if (k_t == nullptr)
    return fail(SSM_E_NULL, "%s: k_t is NULL (the step appends the current token)", fn);
  if ((st = check_token(*d, k_t, v_t, decay_t, beta_t, fn)) != SSM_OK) return st;
  if ((st = check_buffers(*d, k_buf, v_buf, decay_buf, beta_buf, fn)) != SSM_OK) return st;
  const Sizes z = pool_sizes(*d, num_slots);
  const size_t rows = (size_t)d->batch * 4;
  st = check_arrays(fn, {{state, z.state, true, "state"}, {sketch0, z.sketch, true, "sketch0"},
                         {sketch1, z.sketch, true, "sketch1"}, {basis, z.basis, false, "basis"},
                         {q, z.qk, false, "q"}, {k_t, z.qk, false, "k_t"}, {v_t, z.v, false, "v_t"},
                         {decay_t, z.dtok, false, "decay_t"}, {beta_t, z.btok, false, "beta_t"},
                         {k_buf, z.kbuf, true, "k_buf"}, {v_buf, z.vbuf, true, "v_buf"},
                         {decay_buf, z.dbuf, true, "decay_buf"},
                         {beta_buf, z.bbuf, true, "beta_buf"}, {y, z.y, true, "y"},
                         {slot, rows, false, "slot", 4}, {tau, rows, false, "tau", 4},
                         {parity, rows, false, "parity", 4},
                         {update_rows, (size_t)n_update * 4, false, "update_rows", 4}});
  if (st != SSM_OK) return st;
  (void)hipGetLastError();
  return launched(ssm::launch_decode_step(*d, num_slots, slot, tau, parity, n_update,
                                          update_rows, state, sketch0, sketch1, basis, q, k_t,
                                          v_t, decay_t, beta_t, k_buf, v_buf, decay_buf,
                                          beta_buf, y, reinterpret_cast<hipStream_t>(stream)),
                  fn);
}

ssm_status ssm_scan_sizes(const ssm_dims* d, int32_t total_tokens, int64_t* plan_ints,
                          int64_t* forward_bytes, int64_t* backward_bytes) {
  static const char* fn = "ssm_scan_sizes";
  const ssm_status st = check_scan(d, total_tokens, fn);
  if (st != SSM_OK) return st;
  if (plan_ints != nullptr) *plan_ints = (int64_t)(packed_sizes(*d, total_tokens).plan / 4);
  if (forward_bytes != nullptr)
    *forward_bytes = (int64_t)ssm::scan_work(*d, total_tokens, false, nullptr).bytes;
  if (backward_bytes != nullptr)
    *backward_bytes = (int64_t)ssm::scan_work(*d, total_tokens, true, nullptr).bytes;
  return ok();
}

ssm_status ssm_scan_plan(const int32_t* lengths, int32_t n_seqs, int32_t total_tokens,
                         int32_t* plan, void* stream) {
  static const char* fn = "ssm_scan_plan";
  if (n_seqs < 0 || n_seqs >= kMaxUnits)
    return fail(SSM_E_SHAPE, "%s: n_seqs %d not in [0, 2^24)", fn, n_seqs);
  if (total_tokens < 0) return fail(SSM_E_SHAPE, "%s: total_tokens %d < 0", fn, total_tokens);
  if (n_seqs == 0) return ok();
  if (lengths == nullptr) return fail(SSM_E_NULL, "%s: lengths is NULL", fn);
  if (plan == nullptr) return fail(SSM_E_NULL, "%s: plan is NULL", fn);
  const size_t ints = 2 * ((size_t)n_seqs + 1) + ssm::scan_capacity(total_tokens, n_seqs);
  const ssm_status st = check_arrays(fn, {{lengths, (size_t)n_seqs * 4, false, "lengths", 4},
                                          {plan, ints * 4, true, "plan", 4}});
  if (st != SSM_OK) return st;
  (void)hipGetLastError();
  return launched(ssm::launch_scan_plan(lengths, n_seqs, total_tokens, plan,
                                        reinterpret_cast<hipStream_t>(stream)),
                  fn);
}

ssm_status ssm_window_plan(const ssm_dims* d, const int32_t* lengths, int32_t* tau,
                           int32_t* parity, int32_t* update_rows, int32_t* n_update,
                           void* stream) {
  static const char* fn = "ssm_window_plan";
  ssm_status st = check_dims(d, fn);
  if (st != SSM_OK) return st;
  if (d->batch == 0) return ok();
  if (lengths == nullptr) return fail(SSM_E_NULL, "%s: lengths is NULL", fn);
  if (tau == nullptr) return fail(SSM_E_NULL, "%s: tau is NULL", fn);
  if (parity == nullptr) return fail(SSM_E_NULL, "%s: parity is NULL", fn);
  if (update_rows == nullptr) return fail(SSM_E_NULL, "%s: update_rows is NULL", fn);
  if (n_update == nullptr) return fail(SSM_E_NULL, "%s: n_update is NULL", fn);
  const size_t rows = (size_t)d->batch * 4;
  st = check_arrays(fn, {{lengths, rows, false, "lengths", 4}, {tau, rows, true, "tau", 4},
                         {parity, rows, true, "parity", 4},
                         {update_rows, rows, true, "update_rows", 4},
                         {n_update, 4, true, "n_update", 4}});
  if (st != SSM_OK) return st;
  (void)hipGetLastError();
  return launched(ssm::launch_window_plan(lengths, d->batch, d->window, tau, parity, update_rows,
                                          n_update, reinterpret_cast<hipStream_t>(stream)),
                  fn);
}

ssm_status ssm_scan_forward(const ssm_dims* d, int32_t total_tokens, const int32_t* plan,
                            int32_t num_slots, const int32_t* slot, const float* state_in,
                            const void* q, const void* k, const void* v, const float* decay,
                            const float* beta, float* state, float* y, void* workspace,
                            int64_t workspace_bytes, void* stream) {
  static const char* fn = "ssm_scan_forward";
  ssm_status st = check_scan(d, total_tokens, fn);
  if (st != SSM_OK) return st;
  if (d->batch == 0) return ok();
  if ((st = check_packed(*d, total_tokens, plan, q, k, v, decay, beta, fn)) != SSM_OK) return st;
  if ((st = check_pool(*d, num_slots, slot, plan, "plan", fn)) != SSM_OK) return st;
  if (state == nullptr) return fail(SSM_E_NULL, "%s: state is NULL", fn);
  if (y == nullptr && total_tokens > 0) return fail(SSM_E_NULL, "%s: y is NULL", fn);
  const ssm::ScanWork w = ssm::scan_work(*d, total_tokens, false, workspace);
  if ((st = check_workspace(workspace, workspace_bytes, w.bytes, fn)) != SSM_OK) return st;
  const PackedSizes z = packed_sizes(*d, total_tokens);
  const size_t states = pool_sizes(*d, num_slots).state;
  st = check_arrays(
      fn, {{plan, z.plan, false, "plan", 4}, {slot, (size_t)d->batch * 4, false, "slot", 4},
           {state_in == state ? nullptr : state_in, states, false, "state_in"},
           {q, z.qk, false, "q"}, {k, z.qk, false, "k"}, {v, z.v, false, "v"},
           {decay, z.gate, false, "decay", z.gate_align}, {beta, z.beta, false, "beta", 4},
           {state, states, true, "state"}, {y, z.y, true, "y"},
           {workspace, w.bytes, true, "workspace"}});
  if (st != SSM_OK) return st;
  ssm::ScanArgs a{};
  a.plan = ssm::ScanPlan{plan, d->batch, total_tokens, ssm::scan_capacity(total_tokens, d->batch)};
  a.heads = d->heads;
  a.d_v = d->d_v;
  a.num_slots = num_slots;
  a.slot = slot;
  a.state_in = state_in;
  a.q = q;
  a.k = k;
  a.v = v;
  a.decay = decay;
  a.beta = beta;
  a.state = state;
  a.y = y;
  a.w = w;
  (void)hipGetLastError();
  return launched(launch_scan(*d, a, false, stream), fn);
}

ssm_status ssm_scan_backward(const ssm_dims* d, int32_t total_tokens, const int32_t* plan,
                             const float* state_in, const void* q, const void* k, const void* v,
                             const float* decay, const float* beta, const float* dy,
                             const float* dstate, void* dq, void* dk, void* dv,
                             float* dlog_decay, float* dbeta, float* dstate_in, void* workspace,
                             int64_t workspace_bytes, void* stream) {
  static const char* fn = "ssm_scan_backward";
  ssm_status st = check_scan(d, total_tokens, fn);
  if (st != SSM_OK) return st;
  if (d->batch == 0) return ok();
  if ((st = check_packed(*d, total_tokens, plan, q, k, v, decay, beta, fn)) != SSM_OK) return st;
  if (total_tokens > 0) {
    if (dy == nullptr) return fail(SSM_E_NULL, "%s: dy is NULL", fn);
    if (dq == nullptr) return fail(SSM_E_NULL, "%s: dq is NULL", fn);
    if (dk == nullptr) return fail(SSM_E_NULL, "%s: dk is NULL", fn);
    if (dv == nullptr) return fail(SSM_E_NULL, "%s: dv is NULL", fn);
    if (dlog_decay == nullptr) return fail(SSM_E_NULL, "%s: dlog_decay is NULL", fn);
    if ((st = check_beta(*d, dbeta, "dbeta", fn)) != SSM_OK) return st;
  }
  const ssm::ScanWork w = ssm::scan_work(*d, total_tokens, true, workspace);
  if ((st = check_workspace(workspace, workspace_bytes, w.bytes, fn)) != SSM_OK) return st;
  const PackedSizes z = packed_sizes(*d, total_tokens);
  const size_t states = sizes_of(*d).state;
  st = check_arrays(
      fn, {{plan, z.plan, false, "plan", 4}, {state_in, states, false, "state_in"},
           {q, z.qk, false, "q"}, {k, z.qk, false, "k"}, {v, z.v, false, "v"},
           {decay, z.gate, false, "decay", z.gate_align}, {beta, z.beta, false, "beta", 4},
           {dy, z.y, false, "dy"},
           {dstate, states, false, "dstate"}, {dq, z.qk, true, "dq"}, {dk, z.qk, true, "dk"},
           {dv, z.v, true, "dv"}, {dlog_decay, z.gate, true, "dlog_decay", z.gate_align},
           {dbeta, z.beta, true, "dbeta", 4}, {dstate_in, states, true, "dstate_in"},
           {workspace, w.bytes, true, "workspace"}});
  if (st != SSM_OK) return st;
  ssm::ScanArgs a{};
  a.plan = ssm::ScanPlan{plan, d->batch, total_tokens, ssm::scan_capacity(total_tokens, d->batch)};
  a.heads = d->heads;
  a.d_v = d->d_v;
  a.num_slots = d->batch;
  a.state_in = state_in;
  a.q = q;
  a.k = k;
  a.v = v;
  a.decay = decay;
  a.beta = beta;
  a.dy = dy;
  a.dstate = dstate;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.dlog = dlog_decay;
  a.dbeta = dbeta;
  a.dstate_in = dstate_in;
  a.w = w;
  (void)hipGetLastError();
  return launched(launch_scan(*d, a, true, stream), fn);
}

}  // extern "C"
