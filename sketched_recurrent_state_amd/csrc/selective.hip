// selective.hip -- the selective recurrence over packed prompts and for single tokens.
#include "selective.hpp"

namespace ssm {

namespace {

// The main pass over a group: outputs and final states.
template <int S, int NS, typename T>
__global__ void __launch_bounds__(64 * WAVES) selective_scan_kernel(const SelectiveArgs a) {
  using SH = SelShape<S, NS>;
  using Block = SelBlock<T, S, NS, true, true, false>;
  constexpr int N = SH::N, CH = SH::CH, EC = SH::EC, EN = SH::EN;
  __shared__ __align__(16) float2 sv[WAVES][TB][CH + 1];  // delta, delta x; a row of 16 channels more would
                                                          // start in the same bank again
  __shared__ __align__(16) float sb[WAVES][TB][N], sc[WAVES][TB][N];
  __shared__ float sy[WAVES][TB][CH];
  __shared__ __align__(16) float sbias[WAVES][CH], sskip[WAVES][CH];
  const int wave = scalar(threadIdx.x >> 6), tiles = a.channels / CH;
  const int tile_blocks = (tiles + WAVES - 1) / WAVES;
  const int tile = blockIdx.x % tile_blocks * WAVES + wave;
  if (tile >= tiles) return;
  const SelTile w = sel_tile<S>(a, tile);
  const SelGroup grp = sel_group(a, blockIdx.x / tile_blocks);
  const int my = w.c0 + w.ch, n0 = w.sg * NS;
  float A[NS], h[NS];
  Vec<float, NS>::load(a.A + (size_t)my * N + n0, A);
#pragma unroll
  for (int i = 0; i < NS; ++i) A[i] *= kLog2e;
  stage_channels(sbias[wave], a.dt_bias, w);
  stage_channels(sskip[wave], a.D, w);
  wave_lds_sync();
  if (a.state != a.state_in)
    for_empty_sequences(a, grp, [&](int, int slot) {
      const size_t at = ((size_t)slot * a.channels + my) * N + n0;
      float v[NS];
      zero(v);
      if (a.state_in) Vec<float, NS>::load(a.state_in + at, v);
      Vec<float, NS>::store(a.state + at, v);
    });
  SelCell c, ahead;
  if (!next_cell(a, grp.e0, grp.e1, c)) return;
  zero(h);
  if (!c.starts()) carry_in<N>(a, grp, c, my, n0, A, h);
  Block next;
  next.load(a, w, c, 0);
  for (bool more = true; more; c = ahead) {
    more = next_cell(a, c.entry + 1, grp.e1, ahead);
    const size_t at = (size_t)c.slot * a.channels * N + (uint32_t)(my * N + n0);
    if (c.starts()) {
      zero(h);
      // in place, the group where the sequence ends may have written its state by now
      const bool copied = a.state == a.state_in && goes_on(c.entry, c.len, grp.e1, a.plan.cap);
      const float* from = copied ? a.w.start + (size_t)grp.g * a.channels * N : a.state_in + (size_t)c.slot * a.channels * N;
      if (a.state_in) Vec<float, NS>::load(from + (uint32_t)(my * N + n0), h);
    }
    for (int t0 = 0; t0 < c.count; t0 += TB) {
      const Block now = next;
      const bool on = t0 + w.t < c.count;
      const int tok0 = c.first + c.pos + t0;
      if (t0 + TB < c.count) next.load(a, w, c, t0 + TB);
      else if (more) next.load(a, w, ahead, 0);
      float x[EC], dt[EC], delta[EC], bias[EC], b[EN], cc[EN];
      now.x.unpack(x);
      now.dt.unpack(dt);
      now.b.unpack(b);
      Vec<float, EC>::load(&sbias[wave][w.q * EC], bias);
#pragma unroll
      for (int i = 0; i < EC; ++i) dt[i] += bias[i];
      steps(a, dt, t0 + TB <= c.count, on, delta);
#pragma unroll
      for (int i = 0; i < EC; ++i) sv[wave][w.t][w.q * EC + i] = make_float2(delta[i], delta[i] * x[i]);
      Vec<float, EN>::store(&sb[wave][w.t][w.q * EN], b);
      now.c.unpack(cc);
      Vec<float, EN>::store(&sc[wave][w.t][w.q * EN], cc);
      wave_lds_sync();
      float y[(TB + S - 1) / S];  // lane sg keeps the tokens that are sg modulo S
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const float2 v = sv[wave][t][w.ch];
        float bb[NS], ct[NS], yt = 0.f;
        Vec<float, NS>::load(&sb[wave][t][n0], bb);
        Vec<float, NS>::load(&sc[wave][t][n0], ct);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          h[i] = fmaf(__builtin_amdgcn_exp2f(v.x * A[i]), h[i], v.y * bb[i]);
          yt = fmaf(ct[i], h[i], yt);
        }
        yt = state_sum<S>(yt);
        y[t / S] = t % S == 0 ? yt : w.sg == t % S ? yt : y[t / S];
      }
#pragma unroll
      for (int i = 0; i < TB / S; ++i) sy[wave][i * S + w.sg][w.ch] = y[i];
      wave_lds_sync();
      if (on) {
        float z[EC], o[EC], skip[EC];
        now.z.unpack(z);
        Vec<float, EC>::load(&sskip[wave][w.q * EC], skip);
#pragma unroll
        for (int i = 0; i < EC; ++i) o[i] = fmaf(skip[i], x[i], sy[wave][w.t][w.q * EC + i]);
        apply_gate(a, z, o);
        store_row<T, EC>(row_at<T>(a.out, tok0, w.t, w.c0 + w.q * EC), o);
      }
      wave_lds_sync();
    }
    if (c.ends()) Vec<float, NS>::store(a.state + at, h);
  }
}

// The local pass: the state that the group's last sequence leaves, if it goes on behind the group. Where states are
// continued in place it also copies the one that such a sequence begins with: the main pass reads it in this group
// and writes the final state in a later one, in no order.
template <int S, int NS, typename T>
__global__ void __launch_bounds__(64 * WAVES) selective_local_kernel(const SelectiveArgs a) {
  using SH = SelShape<S, NS>;
  using Block = SelBlock<T, S, NS, false, false, false>;
  constexpr int N = SH::N, CH = SH::CH, EC = SH::EC, EN = SH::EN;
  __shared__ __align__(16) float2 sv[WAVES][TB][CH + 1];  // delta, delta x
  __shared__ __align__(16) float sb[WAVES][TB][N];
  __shared__ __align__(16) float sbias[WAVES][CH];
  const int wave = scalar(threadIdx.x >> 6), tiles = a.channels / CH;
  const int tile_blocks = (tiles + WAVES - 1) / WAVES;
  const int tile = blockIdx.x % tile_blocks * WAVES + wave;
  if (tile >= tiles) return;
  const SelTile w = sel_tile<S>(a, tile);
  const SelGroup grp = sel_group(a, blockIdx.x / tile_blocks);
  SelCell c, last;
  if (!prev_cell(a, grp.e1 - 1, grp.e0 - 1, last) || last.ends()) return;
  if (!next_cell(a, max(seq_entry(a, last.seq), grp.e0), grp.e1, c) || c.seq != last.seq) return;
  const int my = w.c0 + w.ch, n0 = w.sg * NS;
  float A[NS], h[NS], sum = 0.f;
  Vec<float, NS>::load(a.A + (size_t)my * N + n0, A);
#pragma unroll
  for (int i = 0; i < NS; ++i) A[i] *= kLog2e;
  stage_channels(sbias[wave], a.dt_bias, w);
  wave_lds_sync();
  zero(h);
  if (c.starts() && a.state_in) {
    Vec<float, NS>::load(a.state_in + (size_t)c.slot * a.channels * N + (uint32_t)(my * N + n0), h);
    if (a.state == a.state_in)
      Vec<float, NS>::store(a.w.start + ((size_t)grp.g * a.channels + my) * N + n0, h);
  }
  Block next;
  next.load(a, w, c, 0);
  SelCell ahead;
  for (bool more = true; more; c = ahead) {
    more = next_cell(a, c.entry + 1, grp.e1, ahead);
    for (int t0 = 0; t0 < c.count; t0 += TB) {
      const Block now = next;
      const bool on = t0 + w.t < c.count;
      if (t0 + TB < c.count) next.load(a, w, c, t0 + TB);
      else if (more) next.load(a, w, ahead, 0);
      float x[EC], dt[EC], delta[EC], bias[EC], b[EN];
      now.x.unpack(x);
      now.dt.unpack(dt);
      now.b.unpack(b);
      Vec<float, EC>::load(&sbias[wave][w.q * EC], bias);
#pragma unroll
      for (int i = 0; i < EC; ++i) dt[i] += bias[i];
      steps(a, dt, t0 + TB <= c.count, on, delta);
#pragma unroll
      for (int i = 0; i < EC; ++i) sv[wave][w.t][w.q * EC + i] = make_float2(delta[i], delta[i] * x[i]);
      Vec<float, EN>::store(&sb[wave][w.t][w.q * EN], b);
      wave_lds_sync();
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const float2 v = sv[wave][t][w.ch];
        float bb[NS];
        Vec<float, NS>::load(&sb[wave][t][n0], bb);
        sum += v.x;
#pragma unroll
        for (int i = 0; i < NS; ++i) h[i] = fmaf(__builtin_amdgcn_exp2f(v.x * A[i]), h[i], v.y * bb[i]);
      }
      wave_lds_sync();
    }
  }
  Vec<float, NS>::store(a.w.local + ((size_t)grp.g * a.channels + my) * N + n0, h);
  if (w.sg == 0) a.w.sums[(size_t)grp.g * a.channels + my] = sum;
}

// Single tokens: a lane holds 4 states of a channel (2 where d_state = 8), so that a wave's state is
// one run of memory, for R rows of the batch at a time. Bound by HBM: the state read and written, past the
// caches, which the next step's state would not find it in anyway.
template <int NS>
__device__ __forceinline__ void load_state(const float* p, float (&h)[NS]) {
  typedef float vec __attribute__((ext_vector_type(NS)));
  const vec v = __builtin_nontemporal_load(reinterpret_cast<const vec*>(p));
#pragma unroll
  for (int i = 0; i < NS; ++i) h[i] = v[i];
}
template <int NS>
__device__ __forceinline__ void store_state(float* p, const float (&h)[NS]) {
  typedef float vec __attribute__((ext_vector_type(NS)));
  vec v;
#pragma unroll
  for (int i = 0; i < NS; ++i) v[i] = h[i];
  __builtin_nontemporal_store(v, reinterpret_cast<vec*>(p));
}

constexpr int SR = 2;  // rows of a lane: 256 rows of 5,120 channels x 16 states 39 us, with 1 row 42, with 4 39.5; 53 us
                       // through the caches, a row a lane

template <int S, int NS, typename T>
__global__ void __launch_bounds__(256) selective_step_kernel(const SelectiveArgs a, int rows) {
  constexpr int N = S * NS;
  const long long item = ((long long)blockIdx.x * 256 + threadIdx.x) / S;
  const int sg = threadIdx.x % S, c = (int)(item % a.channels), row0 = (int)(item / a.channels) * SR;
  if (row0 >= rows) return;
  const int g = c / (a.channels / a.groups);
  float h[SR][NS], b[SR][NS], cc[SR][NS], x[SR], dt[SR], z[SR], A[NS];
  float* state[SR];
#pragma unroll
  for (int r = 0; r < SR; ++r) {
    const int row = min(row0 + r, rows - 1), slot = a.slot ? a.slot[row] : row;
    const bool on = row0 + r < rows && slot >= 0 && slot < a.num_slots;
    state[r] = on ? a.state + ((size_t)slot * a.channels + c) * N + sg * NS : nullptr;
    zero(h[r]);
    if (on) load_state(state[r], h[r]);
    Vec<T, NS>::load(a.B.row<T>(row) + g * N + sg * NS, b[r]);
    Vec<T, NS>::load(a.C.row<T>(row) + g * N + sg * NS, cc[r]);
    Vec<T, 1>::load(a.x.row<T>(row) + c, &x[r]);
    Vec<T, 1>::load(a.dt.row<T>(row) + c, &dt[r]);
    Vec<T, 1>::load(a.z.row<T>(row) + c, &z[r]);  // x where there is no gate
  }
  Vec<float, NS>::load(a.A + (size_t)c * N + sg * NS, A);
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, skip = a.D ? a.D[c] : 0.f;
#pragma unroll
  for (int r = 0; r < SR; ++r) {
    const float raw = dt[r] + bias;
    const float delta = a.softplus ? softplus(raw) : raw;
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      h[r][i] = fmaf(__builtin_amdgcn_exp2f(delta * (kLog2e * A[i])), h[r][i], delta * x[r] * b[r][i]);
      y = fmaf(cc[r][i], h[r][i], y);
    }
    y = fmaf(skip, x[r], state_sum<S>(y));
    if (a.gated) y *= z[r] * sigmoid(z[r]);
    if (state[r]) {
      store_state(state[r], h[r]);
      if (sg == 0) store_row<T, 1>(a.out.out<T>(row0 + r) + c, &y);
    }
  }
}

}  // namespace

// Ten waves a SIMD of the whole GPU in all (6 of the forward pass's and 3 of the gradients' are resident at
// a time): with fewer, longer groups the last ones leave SIMDs without work. By chunks of a group, on a busy GPU, the
// rule's choice in brackets: a prompt of 8192 tokens x 5120 channels 3: 305 us, 4: 292, [5]: 295, 6: 311, 8: 310, 11: 351,
// 16: 413; 41 unlike prompts of 8003 tokens 3: 263, 4: 248, 5: 264, [6]: 271, 8: 260, 11: 269, 16: 330; gradients of
// 2 x 2048 tokens 1: 501, 2: 458, [3]: 464, 5: 484, 9: 549, 17: 654. Joining the groups before costs a
// group about a fiftieth of a chunk each, so long prompts of few channels get longer groups.
constexpr int kWaves = 10240;
SelGroups selective_groups(const ssm_selective_dims& d, int cap) {
  if (cap < 1) return SelGroups{1, 1};
  const int tiles = selective_tiles(d);
  int groups = (kWaves + tiles - 1) / tiles;
  if (groups > cap) groups = cap;
  int chunks = (cap + groups - 1) / groups;
  while ((long long)chunks * chunks * 50 < cap) ++chunks;
  return SelGroups{chunks, (cap + chunks - 1) / chunks};
}

SelectiveWork selective_work(const ssm_selective_dims& d, int total, bool backward, void* base) {
  SelectiveWork w{};
  const SelGroups g = selective_groups(d, d.batch > 0 ? scan_capacity(total, d.batch) : 0);
  const size_t states = (size_t)d.channels * d.d_state;
  size_t at = 0;
  auto take = [&](size_t floats) {
    float* p = reinterpret_cast<float*>(static_cast<char*>(base) + at);
    at += floats * sizeof(float);  // channels are a multiple of 16, so every part is one of 64 bytes
    return p;
  };
  if (g.groups > 1 || backward) {  // backwards a wrong plan's only group may claim to go on
    w.local = take(g.groups * states);
    w.sums = take((size_t)g.groups * d.channels);
  }
  if (g.groups > 1 && !backward) w.start = take(g.groups * states);
  if (backward) {
    w.back = take(g.groups * states);
    w.states = take((size_t)kept_places(total) * states);
    w.until = take((size_t)kept_places(total) * d.channels);
    w.dbc = take(((size_t)total + 1) * selective_tiles(d) * 2 * d.d_state);
    w.partial = take((size_t)g.groups * d.channels * (d.d_state + 2));
  }
  w.bytes = at;
  return w;
}

hipError_t launch_selective_forward(const ssm_selective_dims& d, SelectiveArgs& a, hipStream_t stream) {
  const SelGroups g = selective_groups(d, a.plan.cap);
  a.time_groups = g.groups;
  a.group_chunks = g.chunks;
  return over_groups(d, a, [&](auto S, auto NS, auto T, dim3 grid) {
    constexpr int s = decltype(S)::value, ns = decltype(NS)::value;
    using TI = typename decltype(T)::type;
    if (g.groups > 1)
      hipLaunchKernelGGL((selective_local_kernel<s, ns, TI>), grid, dim3(64 * WAVES), 0, stream, a);
    hipLaunchKernelGGL((selective_scan_kernel<s, ns, TI>), grid, dim3(64 * WAVES), 0, stream, a);
  });
}

hipError_t launch_selective_step(const ssm_selective_dims& d, const SelectiveArgs& a,
                                 hipStream_t stream) {
  const long long items = (long long)((d.batch + SR - 1) / SR) * d.channels;
  return selective_dispatch(d, [&](auto S, auto NS, auto T) {
    constexpr int s = decltype(S)::value;
    hipLaunchKernelGGL((selective_step_kernel<s, decltype(NS)::value, typename decltype(T)::type>),
                       dim3((unsigned)((items * s + 255) / 256)), dim3(256), 0, stream, a, d.batch);
    return hipGetLastError();
  });
}

}  // namespace ssm
