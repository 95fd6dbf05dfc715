// layer_abi.hip -- the extern "C" entry points of the short convolution, the selective recurrence and the
// output norm: argument checks on the host, then the launches on the caller's stream. Nothing here
// allocates, frees or synchronises. See include/sketchssm.h.
#include <float.h>

#include "abi_checks.hpp"
#include "layer.hpp"

namespace {

using ssm::Arr;
using ssm::check_arrays;
using ssm::check_workspace;
using ssm::fail;
using ssm::launched;
using ssm::ok;

constexpr int kMaxBatch = 1 << 24, kMaxChannels = 1 << 20;

// The arrays of one call.
struct Arrays {
  Arr list[48];
  size_t n = 0;
  void add(const void* p, size_t bytes, bool output, const char* name, unsigned align = 16) {
    list[n++] = Arr{p, bytes, output, name, align};
  }
  void rows(const ssm_rows& r, long long rows, size_t width, size_t elem, bool output,
            const char* name) {
    list[n++] = Arr{r.data, width * elem, output, name, 16, (size_t)rows, (size_t)r.stride * elem};
  }
  ssm_status check(const char* fn) const { return check_arrays(fn, list, n); }
};

size_t elem_of(int in_dtype) { return in_dtype == SSM_IN_BF16 ? 2 : 4; }

ssm_status check_dtype(int t, const char* what, const char* fn) {
  if (t != SSM_IN_BF16 && t != SSM_IN_F32)
    return fail(SSM_E_RANGE, "%s: %s %d is not 0 (bf16) or 1 (fp32)", fn, what, t);
  return SSM_OK;
}

// Rows that hold `rows` > 0 rows of `width`.
ssm_status check_rows(const ssm_rows& r, size_t width, const char* name, const char* fn) {
  if (r.data == nullptr) return fail(SSM_E_NULL, "%s: %s is NULL", fn, name);
  if (r.stride < (int64_t)width || r.stride % 8 != 0 || r.stride >= (1LL << 26))
    return fail(SSM_E_SHAPE, "%s: %s has a stride of %lld, not a multiple of 8 in [%zu, 2^26)", fn,
                name, (long long)r.stride, width);
  return SSM_OK;
}

ssm_status check_batch(int batch, int total, const char* fn) {
  if (batch < 0 || batch >= kMaxBatch)
    return fail(SSM_E_SHAPE, "%s: batch %d not in [0, 2^24)", fn, batch);
  if (total < 0) return fail(SSM_E_SHAPE, "%s: total_tokens %d < 0", fn, total);
  return SSM_OK;
}

// The reciprocal root takes a smaller eps for 0, which would make NaN of a run of zeros.
ssm_status check_eps(float eps, const char* fn) {
  if (!(eps >= FLT_MIN))
    return fail(SSM_E_RANGE, "%s: eps %g is not at least 2^-126", fn, (double)eps);
  return SSM_OK;
}

ssm_status check_slots(int batch, int num_slots, const int32_t* slot, const char* fn) {
  if (num_slots < 1) return fail(SSM_E_SHAPE, "%s: num_slots %d < 1", fn, num_slots);
  if (slot == nullptr && batch > num_slots)
    return fail(SSM_E_SHAPE, "%s: %d rows but %d slots and no slot map", fn, batch, num_slots);
  return SSM_OK;
}

ssm::ScanPlan plan_of(const int32_t* plan, int batch, int total) {
  if (batch == 0) return ssm::ScanPlan{nullptr, 0, 0, 0};
  return ssm::ScanPlan{plan, batch, total, ssm::scan_capacity(total, batch)};
}
size_t plan_bytes(int batch, int total) {
  return (2 * ((size_t)batch + 1) + ssm::scan_capacity(total, batch)) * 4;
}

// ---------------------------------------------------------------------------
// convolution
// ---------------------------------------------------------------------------
const char* const kX[] = {"x[0]", "x[1]", "x[2]", "x[3]"};
const char* const kY[] = {"y[0]", "y[1]", "y[2]", "y[3]"};
const char* const kDy[] = {"dy[0]", "dy[1]", "dy[2]", "dy[3]"};
const char* const kDx[] = {"dx[0]", "dx[1]", "dx[2]", "dx[3]"};

ssm_status check_conv(const ssm_conv_dims* d, int total, const char* fn, int& C) {
  if (d == nullptr) return fail(SSM_E_NULL, "%s: dims is NULL", fn);
  ssm_status st = check_dtype(d->in_dtype, "in_dtype", fn);
  if (st != SSM_OK) return st;
  if ((st = check_batch(d->batch, total, fn)) != SSM_OK) return st;
  if (d->taps < 2 || d->taps > 4) return fail(SSM_E_SHAPE, "%s: taps %d not in [2, 4]", fn, d->taps);
  if (d->activation != SSM_ACT_NONE && d->activation != SSM_ACT_SILU)
    return fail(SSM_E_RANGE, "%s: activation %d is not 0 (none) or 1 (silu)", fn, d->activation);
  if (d->parts < 1 || d->parts > SSM_CONV_PARTS)
    return fail(SSM_E_SHAPE, "%s: parts %d not in [1, %d]", fn, d->parts, SSM_CONV_PARTS);
  long long sum = 0;
  bool normed = false;
  for (int p = 0; p < d->parts; ++p) {
    const int c = d->channels[p], n = d->norm[p];
    if (c < 8 || c % 8 != 0 || c > kMaxChannels)
      return fail(SSM_E_SHAPE, "%s: channels[%d] = %d is not a multiple of 8 in [8, 2^20]", fn, p, c);
    if (n != 0 && n != 16 && n != 32 && n != 64 && n != 128)
      return fail(SSM_E_SHAPE, "%s: norm[%d] = %d not in {0, 16, 32, 64, 128}", fn, p, n);
    if (n != 0 && c % n != 0)
      return fail(SSM_E_SHAPE, "%s: channels[%d] = %d is not a multiple of norm[%d] = %d", fn, p, c, p,
                  n);
    normed |= n != 0;
    sum += c;
  }
  if (sum > kMaxChannels) return fail(SSM_E_SHAPE, "%s: %lld channels > 2^20", fn, sum);
  if (normed && (st = check_eps(d->eps, fn)) != SSM_OK) return st;
  const long long tiles = (sum + 511) / 512;
  if (((long long)total / ssm::CT + d->batch) * tiles >= (1LL << 24))
    return fail(SSM_E_SHAPE, "%s: (total_tokens/64 + batch) * ceil(channels/512) >= 2^24", fn);
  C = (int)sum;
  return SSM_OK;
}

ssm_status check_parts(const ssm_conv_dims& d, const ssm_rows* r, long long rows, bool output,
                       const char* const* names, const char* what, Arrays& arrs, const char* fn) {
  if (rows == 0) return SSM_OK;
  if (r == nullptr) return fail(SSM_E_NULL, "%s: %s is NULL", fn, what);
  for (int p = 0; p < d.parts; ++p) {
    const ssm_status st = check_rows(r[p], (size_t)d.channels[p], names[p], fn);
    if (st != SSM_OK) return st;
    arrs.rows(r[p], rows, (size_t)d.channels[p], elem_of(d.in_dtype), output, names[p]);
  }
  return SSM_OK;
}

ssm::ConvArgs conv_args(const ssm_conv_dims& d, int C, const ssm_rows* x, const ssm_rows* y,
                        const ssm_rows* dy, const ssm_rows* dx, const float* weight,
                        const float* bias) {
  ssm::ConvArgs a{};
  a.parts = d.parts;
  a.C = C;
  a.silu = d.activation == SSM_ACT_SILU;
  a.eps = d.eps;
  a.weight = weight;
  a.bias = bias;
  int offset = 0;
  for (int p = 0; p < d.parts; ++p) {
    ssm::ConvPart& P = a.part[p];
    P.channels = d.channels[p];
    P.offset = offset;
    P.norm = d.norm[p];
    P.scale = d.norm[p] ? d.scale[p] : 1.f;
    if (x) P.x = ssm::rows_of(x[p]);
    if (y) P.y = ssm::rows_of(y[p]);
    if (dy) P.dy = ssm::rows_of(dy[p]);
    if (dx) P.dx = ssm::rows_of(dx[p]);
    offset += P.channels;
  }
  return a;
}

size_t conv_state_bytes(const ssm_conv_dims& d, int C, long long slots) {
  return (size_t)slots * (d.taps - 1) * C * elem_of(d.in_dtype);
}

// ---------------------------------------------------------------------------
// selective recurrence
// ---------------------------------------------------------------------------
ssm_status check_selective(const ssm_selective_dims* d, int total, const char* fn) {
  if (d == nullptr) return fail(SSM_E_NULL, "%s: dims is NULL", fn);
  ssm_status st = check_dtype(d->in_dtype, "in_dtype", fn);
  if (st != SSM_OK) return st;
  if ((st = check_batch(d->batch, total, fn)) != SSM_OK) return st;
  if (d->d_state != 8 && d->d_state != 16 && d->d_state != 32 && d->d_state != 64)
    return fail(SSM_E_SHAPE, "%s: d_state %d not in {8, 16, 32, 64}", fn, d->d_state);
  if (d->groups < 1) return fail(SSM_E_SHAPE, "%s: groups %d < 1", fn, d->groups);
  if (d->channels < 1 || d->channels > kMaxChannels || d->channels % d->groups != 0 ||
      d->channels / d->groups % 16 != 0)
    return fail(SSM_E_SHAPE, "%s: channels %d is not a multiple of 16 * groups (%d) up to 2^20", fn,
                d->channels, d->groups);
  if (d->softplus != 0 && d->softplus != 1)
    return fail(SSM_E_RANGE, "%s: softplus %d is not 0 or 1", fn, d->softplus);
  if (((long long)total / ssm::CT + d->batch) * (d->channels / 16) >= (1LL << 31))
    return fail(SSM_E_SHAPE, "%s: (total_tokens/64 + batch) * channels/16 >= 2^31", fn);
  return SSM_OK;
}

ssm_status check_selective_in(const ssm_selective_dims& d, const ssm_selective_inputs* in,
                              long long rows, Arrays& arrs, const char* fn) {
  if (in == nullptr) return fail(SSM_E_NULL, "%s: inputs is NULL", fn);
  const size_t D = (size_t)d.channels, N = (size_t)d.d_state, e = elem_of(d.in_dtype);
  if (in->A == nullptr) return fail(SSM_E_NULL, "%s: A is NULL", fn);
  arrs.add(in->A, D * N * 4, false, "A");
  arrs.add(in->D, D * 4, false, "D");
  arrs.add(in->dt_bias, D * 4, false, "dt_bias");
  if (rows == 0) return SSM_OK;
  const struct {
    const ssm_rows& r;
    size_t width;
    const char* name;
  } all[] = {{in->x, D, "x"}, {in->dt, D, "dt"}, {in->z, D, "z"},
             {in->B, d.groups * N, "B"}, {in->C, d.groups * N, "C"}};
  for (const auto& v : all) {
    if (&v.r == &in->z && v.r.data == nullptr) continue;
    const ssm_status st = check_rows(v.r, v.width, v.name, fn);
    if (st != SSM_OK) return st;
    arrs.rows(v.r, rows, v.width, e, false, v.name);
  }
  return SSM_OK;
}

ssm_status check_row_output(const ssm_rows* r, long long rows, size_t width, size_t e, bool output,
                            const char* name, Arrays& arrs, const char* fn) {
  if (rows == 0) return SSM_OK;
  if (r == nullptr) return fail(SSM_E_NULL, "%s: %s is NULL", fn, name);
  const ssm_status st = check_rows(*r, width, name, fn);
  if (st != SSM_OK) return st;
  arrs.rows(*r, rows, width, e, output, name);
  return SSM_OK;
}

ssm::SelectiveArgs selective_args(const ssm_selective_dims& d, const ssm_selective_inputs& in) {
  ssm::SelectiveArgs a{};
  a.x = ssm::rows_of(in.x);
  a.dt = ssm::rows_of(in.dt);
  a.gated = in.z.data != nullptr;
  a.z = ssm::rows_of(a.gated ? in.z : in.x);
  a.B = ssm::rows_of(in.B);
  a.C = ssm::rows_of(in.C);
  a.A = in.A;
  a.D = in.D;
  a.dt_bias = in.dt_bias;
  a.channels = d.channels;
  a.groups = d.groups;
  a.softplus = d.softplus;
  return a;
}

// ---------------------------------------------------------------------------
// norm
// ---------------------------------------------------------------------------
ssm_status check_norm(const ssm_norm_dims* d, int rows, const char* fn) {
  if (d == nullptr) return fail(SSM_E_NULL, "%s: dims is NULL", fn);
  ssm_status st = check_dtype(d->x_dtype, "x_dtype", fn);
  if (st != SSM_OK) return st;
  if ((st = check_dtype(d->in_dtype, "in_dtype", fn)) != SSM_OK) return st;
  if (rows < 0) return fail(SSM_E_SHAPE, "%s: rows %d < 0", fn, rows);
  if (d->groups < 1) return fail(SSM_E_SHAPE, "%s: groups %d < 1", fn, d->groups);
  if (d->width < 8 || d->width > 8192 || d->width % 8 != 0)
    return fail(SSM_E_SHAPE, "%s: width %d is not a multiple of 8 in [8, 8192]", fn, d->width);
  if ((long long)d->groups * d->width > kMaxChannels)
    return fail(SSM_E_SHAPE, "%s: groups * width = %lld > 2^20", fn, (long long)d->groups * d->width);
  if ((long long)rows * d->groups >= (1LL << 31))
    return fail(SSM_E_SHAPE, "%s: rows * groups = %lld >= 2^31", fn, (long long)rows * d->groups);
  if (d->gate < SSM_GATE_NONE || d->gate > SSM_GATE_BEFORE)
    return fail(SSM_E_RANGE, "%s: gate %d is not 0 (none), 1 (after) or 2 (before)", fn, d->gate);
  if (d->gate != SSM_GATE_NONE && d->activation != SSM_ACT_SILU && d->activation != SSM_ACT_SIGMOID)
    return fail(SSM_E_RANGE, "%s: activation %d is not 1 (silu) or 2 (sigmoid)", fn, d->activation);
  if ((d->shared != 0 && d->shared != 1) || (d->centred != 0 && d->centred != 1))
    return fail(SSM_E_RANGE, "%s: shared %d and centred %d are 0 or 1", fn, d->shared, d->centred);
  return check_eps(d->eps, fn);
}

// The arrays of both directions.
ssm_status check_norm_in(const ssm_norm_dims& d, int rows, const ssm_rows* x, const ssm_rows* z,
                         const float* weight, const float* bias, Arrays& arrs, const char* fn) {
  const size_t width = (size_t)d.groups * d.width, wide = d.shared ? (size_t)d.width : width;
  ssm_status st = check_row_output(x, rows, width, elem_of(d.x_dtype), false, "x", arrs, fn);
  if (st != SSM_OK) return st;
  if (d.gate == SSM_GATE_NONE) {
    if (z != nullptr && z->data != nullptr)
      return fail(SSM_E_RANGE, "%s: z must be NULL without a gate", fn);
  } else {
    st = check_row_output(z, rows, width, elem_of(d.in_dtype), false, "z", arrs, fn);
    if (st != SSM_OK) return st;
  }
  if (weight == nullptr) return fail(SSM_E_NULL, "%s: weight is NULL", fn);
  arrs.add(weight, wide * 4, false, "weight");
  arrs.add(bias, wide * 4, false, "bias");
  return SSM_OK;
}

ssm::NormArgs norm_args(const ssm_norm_dims& d, int rows, const ssm_rows* x, const ssm_rows* z,
                        const float* weight, const float* bias) {
  ssm::NormArgs a{};
  if (x) a.x = ssm::rows_of(*x);
  if (z) a.z = ssm::rows_of(*z);
  a.rows = rows;
  a.groups = d.groups;
  a.width = d.width;
  a.gate = d.gate;
  a.sigmoid = d.activation == SSM_ACT_SIGMOID;
  a.shared = d.shared || d.groups == 1;
  a.centred = d.centred;
  a.eps = d.eps;
  a.weight = weight;
  a.bias = bias;
  return a;
}

// One group's weights are shared by all of its rows either way.
ssm_norm_dims norm_dims(const ssm_norm_dims& d) {
  ssm_norm_dims n = d;
  n.shared = d.shared || d.groups == 1;
  return n;
}

hipStream_t stream_of(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

ssm_status ssm_conv_sizes(const ssm_conv_dims* d, int32_t total_tokens, int64_t* backward_bytes) {
  int C;
  const ssm_status st = check_conv(d, total_tokens, "ssm_conv_sizes", C);
  if (st != SSM_OK) return st;
  if (backward_bytes != nullptr) *backward_bytes = (int64_t)ssm::conv_workspace(*d, total_tokens);
  return ok();
}

ssm_status ssm_conv_forward(const ssm_conv_dims* d, int32_t total_tokens, const int32_t* plan,
                            int32_t num_slots, const int32_t* slot, const void* state_in,
                            const ssm_rows* x, const float* weight, const float* bias, void* state,
                            const ssm_rows* y, void* stream) {
  static const char* fn = "ssm_conv_forward";
  int C;
  ssm_status st = check_conv(d, total_tokens, fn, C);
  if (st != SSM_OK) return st;
  if (d->batch == 0) return ok();
  if (plan == nullptr) return fail(SSM_E_NULL, "%s: plan is NULL", fn);
  if (weight == nullptr) return fail(SSM_E_NULL, "%s: weight is NULL", fn);
  const bool states = state != nullptr || state_in != nullptr;
  if (states && (st = check_slots(d->batch, num_slots, slot, fn)) != SSM_OK) return st;
  Arrays arrs;
  arrs.add(plan, plan_bytes(d->batch, total_tokens), false, "plan", 4);
  arrs.add(weight, (size_t)C * d->taps * 4, false, "weight");
  arrs.add(bias, (size_t)C * 4, false, "bias");
  if (states) {
    const size_t bytes = conv_state_bytes(*d, C, num_slots);
    arrs.add(slot, (size_t)d->batch * 4, false, "slot", 4);
    arrs.add(state_in == state ? nullptr : state_in, bytes, false, "state_in");
    arrs.add(state, bytes, true, "state");
  }
  if ((st = check_parts(*d, x, total_tokens, false, kX, "x", arrs, fn)) != SSM_OK) return st;
  if ((st = check_parts(*d, y, total_tokens, true, kY, "y", arrs, fn)) != SSM_OK) return st;
  if ((st = arrs.check(fn)) != SSM_OK) return st;
  ssm::ConvArgs a = conv_args(*d, C, total_tokens ? x : nullptr, total_tokens ? y : nullptr, nullptr,
                              nullptr, weight, bias);
  a.plan = plan_of(plan, d->batch, total_tokens);
  a.num_slots = states ? num_slots : d->batch;
  a.slot = states ? slot : nullptr;
  a.state_in = state_in;
  a.state = state;
  (void)hipGetLastError();
  return launched(ssm::launch_conv_forward(*d, a, stream_of(stream)), fn);
}

ssm_status ssm_conv_backward(const ssm_conv_dims* d, int32_t total_tokens, const int32_t* plan,
                             const void* state_in, const ssm_rows* x, const float* weight,
                             const float* bias, const ssm_rows* dy, const void* dstate,
                             const ssm_rows* dx, float* dweight, float* dbias, void* dstate_in,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  static const char* fn = "ssm_conv_backward";
  int C;
  ssm_status st = check_conv(d, total_tokens, fn, C);
  if (st != SSM_OK) return st;
  if (d->batch > 0 && plan == nullptr) return fail(SSM_E_NULL, "%s: plan is NULL", fn);
  if (weight == nullptr) return fail(SSM_E_NULL, "%s: weight is NULL", fn);
  if (dweight == nullptr) return fail(SSM_E_NULL, "%s: dweight is NULL", fn);
  const size_t need = ssm::conv_workspace(*d, total_tokens);
  if ((st = check_workspace(workspace, workspace_bytes, need, fn)) != SSM_OK) return st;
  const size_t states = conv_state_bytes(*d, C, d->batch);
  const long long rows = d->batch > 0 ? total_tokens : 0;
  Arrays arrs;
  if (d->batch > 0) arrs.add(plan, plan_bytes(d->batch, total_tokens), false, "plan", 4);
  arrs.add(weight, (size_t)C * d->taps * 4, false, "weight");
  arrs.add(bias, (size_t)C * 4, false, "bias");
  arrs.add(state_in, states, false, "state_in");
  arrs.add(dstate, states, false, "dstate");
  arrs.add(dweight, (size_t)C * d->taps * 4, true, "dweight");
  arrs.add(dbias, (size_t)C * 4, true, "dbias");
  arrs.add(dstate_in, states, true, "dstate_in");
  arrs.add(workspace, need, true, "workspace");
  if ((st = check_parts(*d, x, rows, false, kX, "x", arrs, fn)) != SSM_OK) return st;
  if ((st = check_parts(*d, dy, rows, false, kDy, "dy", arrs, fn)) != SSM_OK) return st;
  if ((st = check_parts(*d, dx, rows, true, kDx, "dx", arrs, fn)) != SSM_OK) return st;
  if ((st = arrs.check(fn)) != SSM_OK) return st;
  ssm::ConvArgs a = conv_args(*d, C, rows ? x : nullptr, nullptr, rows ? dy : nullptr,
                              rows ? dx : nullptr, weight, bias);
  a.plan = plan_of(plan, d->batch, total_tokens);
  a.num_slots = d->batch;
  a.state_in = state_in;
  a.dstate = dstate;
  a.dstate_in = dstate_in;
  a.partial = static_cast<float*>(workspace);
  a.dweight = dweight;
  a.dbias = dbias;
  (void)hipGetLastError();
  return launched(ssm::launch_conv_backward(*d, a, stream_of(stream)), fn);
}

ssm_status ssm_conv_step(const ssm_conv_dims* d, int32_t num_slots, const int32_t* slot,
                         const ssm_rows* x, const float* weight, const float* bias, void* state,
                         const ssm_rows* y, void* stream) {
  static const char* fn = "ssm_conv_step";
  int C;
  ssm_status st = check_conv(d, 0, fn, C);
  if (st != SSM_OK) return st;
  if (d->batch == 0) return ok();
  if (weight == nullptr) return fail(SSM_E_NULL, "%s: weight is NULL", fn);
  if (state == nullptr) return fail(SSM_E_NULL, "%s: state is NULL", fn);
  if ((st = check_slots(d->batch, num_slots, slot, fn)) != SSM_OK) return st;
  Arrays arrs;
  arrs.add(slot, (size_t)d->batch * 4, false, "slot", 4);
  arrs.add(weight, (size_t)C * d->taps * 4, false, "weight");
  arrs.add(bias, (size_t)C * 4, false, "bias");
  arrs.add(state, conv_state_bytes(*d, C, num_slots), true, "state");
  if ((st = check_parts(*d, x, d->batch, false, kX, "x", arrs, fn)) != SSM_OK) return st;
  if ((st = check_parts(*d, y, d->batch, true, kY, "y", arrs, fn)) != SSM_OK) return st;
  if ((st = arrs.check(fn)) != SSM_OK) return st;
  ssm::ConvArgs a = conv_args(*d, C, x, y, nullptr, nullptr, weight, bias);
  a.num_slots = num_slots;
  a.slot = slot;
  a.state = state;
  (void)hipGetLastError();
  return launched(ssm::launch_conv_step(*d, a, stream_of(stream)), fn);
}

ssm_status ssm_selective_sizes(const ssm_selective_dims* d, int32_t total_tokens,
                               int64_t* forward_bytes, int64_t* backward_bytes) {
  const ssm_status st = check_selective(d, total_tokens, "ssm_selective_sizes");
  if (st != SSM_OK) return st;
  if (forward_bytes != nullptr)
    *forward_bytes = (int64_t)ssm::selective_work(*d, total_tokens, false, nullptr).bytes;
  if (backward_bytes != nullptr)
    *backward_bytes = (int64_t)ssm::selective_work(*d, total_tokens, true, nullptr).bytes;
  return ok();
}

ssm_status ssm_selective_forward(const ssm_selective_dims* d, int32_t total_tokens,
                                 const int32_t* plan, int32_t num_slots, const int32_t* slot,
                                 const float* state_in, const ssm_selective_inputs* in, float* state,
                                 const ssm_rows* out, void* workspace, int64_t workspace_bytes,
                                 void* stream) {
  static const char* fn = "ssm_selective_forward";
  ssm_status st = check_selective(d, total_tokens, fn);
  if (st != SSM_OK) return st;
  if (d->batch == 0) return ok();
  if (plan == nullptr) return fail(SSM_E_NULL, "%s: plan is NULL", fn);
  if (state == nullptr) return fail(SSM_E_NULL, "%s: state is NULL", fn);
  if ((st = check_slots(d->batch, num_slots, slot, fn)) != SSM_OK) return st;
  const ssm::SelectiveWork w = ssm::selective_work(*d, total_tokens, false, workspace);
  if ((st = check_workspace(workspace, workspace_bytes, w.bytes, fn)) != SSM_OK) return st;
  const size_t states = (size_t)num_slots * d->channels * d->d_state * 4;
  Arrays arrs;
  arrs.add(plan, plan_bytes(d->batch, total_tokens), false, "plan", 4);
  arrs.add(slot, (size_t)d->batch * 4, false, "slot", 4);
  arrs.add(state_in == state ? nullptr : state_in, states, false, "state_in");
  arrs.add(state, states, true, "state");
  arrs.add(workspace, w.bytes, true, "workspace");
  if ((st = check_selective_in(*d, in, total_tokens, arrs, fn)) != SSM_OK) return st;
  st = check_row_output(out, total_tokens, (size_t)d->channels, elem_of(d->in_dtype), true, "out", arrs,
                        fn);
  if (st != SSM_OK) return st;
  if ((st = arrs.check(fn)) != SSM_OK) return st;
  ssm::SelectiveArgs a = selective_args(*d, *in);
  a.plan = plan_of(plan, d->batch, total_tokens);
  a.num_slots = num_slots;
  a.slot = slot;
  a.state_in = state_in;
  a.state = state;
  if (out) a.out = ssm::rows_of(*out);
  a.w = w;
  (void)hipGetLastError();
  return launched(ssm::launch_selective_forward(*d, a, stream_of(stream)), fn);
}

ssm_status ssm_selective_backward(const ssm_selective_dims* d, int32_t total_tokens,
                                  const int32_t* plan, const float* state_in,
                                  const ssm_selective_inputs* in, const ssm_rows* dout,
                                  const float* dstate, const ssm_selective_grads* grads,
                                  float* dstate_in, void* workspace, int64_t workspace_bytes,
                                  void* stream) {
  static const char* fn = "ssm_selective_backward";
  ssm_status st = check_selective(d, total_tokens, fn);
  if (st != SSM_OK) return st;
  if ((long long)total_tokens * d->groups * d->d_state > (1LL << 31) - 128)  // twice that: threads of a grid
    return fail(SSM_E_SHAPE, "%s: total_tokens * groups * d_state > 2^31 - 128", fn);
  if (d->batch > 0 && plan == nullptr) return fail(SSM_E_NULL, "%s: plan is NULL", fn);
  if (grads == nullptr) return fail(SSM_E_NULL, "%s: grads is NULL", fn);
  const ssm::SelectiveWork w = ssm::selective_work(*d, total_tokens, true, workspace);
  if ((st = check_workspace(workspace, workspace_bytes, w.bytes, fn)) != SSM_OK) return st;
  const size_t D = (size_t)d->channels, N = (size_t)d->d_state, e = elem_of(d->in_dtype);
  const size_t states = (size_t)d->batch * D * N * 4;
  const long long rows = d->batch > 0 ? total_tokens : 0;
  Arrays arrs;
  if (d->batch > 0) arrs.add(plan, plan_bytes(d->batch, total_tokens), false, "plan", 4);
  arrs.add(state_in, states, false, "state_in");
  arrs.add(dstate, states, false, "dstate");
  arrs.add(dstate_in, states, true, "dstate_in");
  arrs.add(workspace, w.bytes, true, "workspace");
  if ((st = check_selective_in(*d, in, rows, arrs, fn)) != SSM_OK) return st;
  if ((st = check_row_output(dout, rows, D, e, false, "dout", arrs, fn)) != SSM_OK) return st;
  const bool gated = rows > 0 && in->z.data != nullptr;
  const struct {
    const ssm_rows& r;
    size_t width;
    const char* name;
    bool given;
  } all[] = {{grads->dx, D, "dx", true},
             {grads->ddt, D, "ddt", true},
             {grads->dz, D, "dz", gated},
             {grads->dB, d->groups * N, "dB", true},
             {grads->dC, d->groups * N, "dC", true}};
  for (const auto& v : all) {
    if (rows == 0) break;
    if (!v.given) {
      if (v.r.data != nullptr) return fail(SSM_E_RANGE, "%s: %s is given without its input", fn, v.name);
      continue;
    }
    if ((st = check_row_output(&v.r, rows, v.width, e, true, v.name, arrs, fn)) != SSM_OK) return st;
  }
  if (grads->dA == nullptr) return fail(SSM_E_NULL, "%s: dA is NULL", fn);
  if ((grads->dD != nullptr) != (in->D != nullptr))
    return fail(grads->dD ? SSM_E_RANGE : SSM_E_NULL, "%s: dD goes with D", fn);
  if ((grads->ddt_bias != nullptr) != (in->dt_bias != nullptr))
    return fail(grads->ddt_bias ? SSM_E_RANGE : SSM_E_NULL, "%s: ddt_bias goes with dt_bias", fn);
  arrs.add(grads->dA, D * N * 4, true, "dA");
  arrs.add(grads->dD, D * 4, true, "dD");
  arrs.add(grads->ddt_bias, D * 4, true, "ddt_bias");
  if ((st = arrs.check(fn)) != SSM_OK) return st;
  ssm::SelectiveArgs a = selective_args(*d, *in);
  a.plan = plan_of(plan, d->batch, total_tokens);
  a.num_slots = d->batch;
  a.state_in = state_in;
  a.dstate = dstate;
  a.dstate_in = dstate_in;
  if (dout) a.dout = ssm::rows_of(*dout);
  a.dx = ssm::rows_of(grads->dx);
  a.ddt = ssm::rows_of(grads->ddt);
  a.dz = ssm::rows_of(grads->dz);
  a.dB = ssm::rows_of(grads->dB);
  a.dC = ssm::rows_of(grads->dC);
  a.dA = grads->dA;
  a.dD = grads->dD;
  a.ddt_bias = grads->ddt_bias;
  a.w = w;
  (void)hipGetLastError();
  return launched(ssm::launch_selective_backward(*d, a, stream_of(stream)), fn);
}

ssm_status ssm_selective_step(const ssm_selective_dims* d, int32_t num_slots, const int32_t* slot,
                              const ssm_selective_inputs* in, float* state, const ssm_rows* out,
                              void* stream) {
  static const char* fn = "ssm_selective_step";
  ssm_status st = check_selective(d, 0, fn);
  if (st != SSM_OK) return st;
  if (d->batch == 0) return ok();
  if ((long long)d->batch * d->channels * (d->d_state > 16 ? d->d_state : 16) >= (1LL << 34))
    return fail(SSM_E_SHAPE, "%s: batch * channels * max(d_state, 16) >= 2^34", fn);
  if (state == nullptr) return fail(SSM_E_NULL, "%s: state is NULL", fn);
  if ((st = check_slots(d->batch, num_slots, slot, fn)) != SSM_OK) return st;
  Arrays arrs;
  arrs.add(slot, (size_t)d->batch * 4, false, "slot", 4);
  arrs.add(state, (size_t)num_slots * d->channels * d->d_state * 4, true, "state");
  if ((st = check_selective_in(*d, in, d->batch, arrs, fn)) != SSM_OK) return st;
  st = check_row_output(out, d->batch, (size_t)d->channels, elem_of(d->in_dtype), true, "out", arrs, fn);
  if (st != SSM_OK) return st;
  if ((st = arrs.check(fn)) != SSM_OK) return st;
  ssm::SelectiveArgs a = selective_args(*d, *in);
  a.num_slots = num_slots;
  a.slot = slot;
  a.state = state;
  a.out = ssm::rows_of(*out);
  (void)hipGetLastError();
  return launched(ssm::launch_selective_step(*d, a, stream_of(stream)), fn);
}

ssm_status ssm_gated_norm(const ssm_norm_dims* d, int32_t rows, const ssm_rows* x, const ssm_rows* z,
                          const float* weight, const float* bias, const ssm_rows* out, void* stream) {
  static const char* fn = "ssm_gated_norm";
  ssm_status st = check_norm(d, rows, fn);
  if (st != SSM_OK) return st;
  if (rows == 0) return ok();
  Arrays arrs;
  if ((st = check_norm_in(*d, rows, x, z, weight, bias, arrs, fn)) != SSM_OK) return st;
  st = check_row_output(out, rows, (size_t)d->groups * d->width, elem_of(d->in_dtype), true, "out", arrs,
                        fn);
  if (st != SSM_OK) return st;
  if ((st = arrs.check(fn)) != SSM_OK) return st;
  ssm::NormArgs a = norm_args(*d, rows, x, z, weight, bias);
  a.out = ssm::rows_of(*out);
  (void)hipGetLastError();
  return launched(ssm::launch_norm(norm_dims(*d), a, stream_of(stream)), fn);
}

ssm_status ssm_gated_norm_sizes(const ssm_norm_dims* d, int32_t rows, int64_t* backward_bytes) {
  const ssm_status st = check_norm(d, rows, "ssm_gated_norm_sizes");
  if (st != SSM_OK) return st;
  if (backward_bytes != nullptr) *backward_bytes = (int64_t)ssm::norm_workspace(norm_dims(*d), rows);
  return ok();
}

ssm_status ssm_gated_norm_backward(const ssm_norm_dims* d, int32_t rows, const ssm_rows* x,
                                   const ssm_rows* z, const float* weight, const float* bias,
                                   const ssm_rows* dout, const ssm_rows* dx, const ssm_rows* dz,
                                   float* dweight, float* dbias, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
  static const char* fn = "ssm_gated_norm_backward";
  ssm_status st = check_norm(d, rows, fn);
  if (st != SSM_OK) return st;
  if (dweight == nullptr) return fail(SSM_E_NULL, "%s: dweight is NULL", fn);
  const size_t need = ssm::norm_workspace(norm_dims(*d), rows);
  if ((st = check_workspace(workspace, workspace_bytes, need, fn)) != SSM_OK) return st;
  const size_t width = (size_t)d->groups * d->width, wide = d->shared ? (size_t)d->width : width;
  Arrays arrs;
  if ((st = check_norm_in(*d, rows, x, z, weight, bias, arrs, fn)) != SSM_OK) return st;
  st = check_row_output(dout, rows, width, elem_of(d->in_dtype), false, "dout", arrs, fn);
  if (st != SSM_OK) return st;
  st = check_row_output(dx, rows, width, elem_of(d->x_dtype), true, "dx", arrs, fn);
  if (st != SSM_OK) return st;
  if (d->gate == SSM_GATE_NONE) {
    if (dz != nullptr && dz->data != nullptr)
      return fail(SSM_E_RANGE, "%s: dz must be NULL without a gate", fn);
  } else {
    st = check_row_output(dz, rows, width, elem_of(d->in_dtype), true, "dz", arrs, fn);
    if (st != SSM_OK) return st;
  }
  arrs.add(dweight, wide * 4, true, "dweight");
  arrs.add(dbias, wide * 4, true, "dbias");
  arrs.add(workspace, need, true, "workspace");
  if ((st = arrs.check(fn)) != SSM_OK) return st;
  ssm::NormArgs a = norm_args(*d, rows, rows ? x : nullptr, rows ? z : nullptr, weight, bias);
  if (rows) {
    a.dout = ssm::rows_of(*dout);
    a.dx = ssm::rows_of(*dx);
    if (d->gate != SSM_GATE_NONE) a.dz = ssm::rows_of(*dz);
  }
  a.partial = static_cast<float*>(workspace);
  a.dweight = dweight;
  a.dbias = dbias;
  (void)hipGetLastError();
  return launched(ssm::launch_norm_backward(norm_dims(*d), a, stream_of(stream)), fn);
}

}  // extern "C"
