// selective.hip -- the selective recurrence over packed prompts and for single tokens.
#include "selective.hpp"

namespace ssm {

namespace {

// One block of a sequence: raw inputs of the lane's token.
template <typename T, int S, int NS, bool OUT>
struct SelBlock {
  using SH = SelShape<S, NS>;
  Packed<T, SH::EC> x, dt, z;
  Packed<T, SH::EN> b, c;
  __device__ __forceinline__ void load(const SelectiveArgs& a, const SelTile& w, int64_t tok, bool on) {
    const int c0 = w.c0 + w.q * SH::EC, n0 = w.group * SH::N + w.q * SH::EN;
    load_or_zero(x, a.x.row<T>(tok) + c0, on);
    load_or_zero(dt, a.dt.row<T>(tok) + c0, on);
    load_or_zero(b, a.B.row<T>(tok) + n0, on);
    if constexpr (OUT) {
      load_or_zero(z, a.z.p ? a.z.row<T>(tok) + c0 : nullptr, on && a.z.p);
      load_or_zero(c, a.C.row<T>(tok) + n0, on);
    }
  }
};

// OUT: outputs and final states. Otherwise (the backward pass's first kernel): the state before every
// block but the sequence's first.
template <int S, int NS, typename T, bool OUT>
__global__ void __launch_bounds__(64 * WAVES) selective_scan_kernel(const SelectiveArgs a) {
  using SH = SelShape<S, NS>;
  constexpr int N = SH::N, CH = SH::CH, EC = SH::EC, EN = SH::EN;
  __shared__ __align__(16) float2 sv[WAVES][TB][CH];
  __shared__ __align__(16) float sb[WAVES][TB][N], sc[WAVES][OUT ? TB : 1][N];
  __shared__ float sy[WAVES][OUT ? TB : 1][CH];
  const int wave = threadIdx.x >> 6, tiles = a.channels / CH;
  const int tile_blocks = (tiles + WAVES - 1) / WAVES;
  const int tile = blockIdx.x % tile_blocks * WAVES + wave;
  if (tile >= tiles) return;
  const SelTile w = sel_tile<S>(a, tile);
  const int my = w.c0 + w.ch, n0 = w.sg * NS;
  float A[NS], bias[EC], skip[EC];
  Vec<float, NS>::load(a.A + (size_t)my * N + n0, A);
#pragma unroll
  for (int i = 0; i < NS; ++i) A[i] *= kLog2e;
#pragma unroll
  for (int i = 0; i < EC; ++i) {
    bias[i] = a.dt_bias ? a.dt_bias[w.c0 + w.q * EC + i] : 0.f;
    skip[i] = a.D ? a.D[w.c0 + w.q * EC + i] : 0.f;
  }
  for (int s = blockIdx.x / tile_blocks; s < a.plan.seqs; s += a.walkers) {
    SelSeq q;
    if (!sel_sequence(a, s, q)) continue;
    const size_t at = ((size_t)q.slot * a.channels + my) * N + n0;
    float h[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) h[i] = 0.f;
    if (a.state_in) Vec<float, NS>::load(a.state_in + at, h);
    SelBlock<T, S, NS, OUT> next;
    next.load(a, w, (int64_t)q.tok + w.t, w.t < q.len);
    for (int t0 = 0; t0 < q.len; t0 += TB) {
      const SelBlock<T, S, NS, OUT> now = next;
      const bool on = t0 + w.t < q.len;
      next.load(a, w, (int64_t)q.tok + t0 + TB + w.t, t0 + TB + w.t < q.len);
      if constexpr (!OUT) {
        if (t0 > 0) {
          const size_t block = (size_t)(q.tok / TB + t0 / TB - 1);
          Vec<float, NS>::store(a.w.states + (block * a.channels + my) * N + n0, h);
        }
      }
      float x[EC], dt[EC], b[EN], c[EN];
      now.x.unpack(x);
      now.dt.unpack(dt);
      now.b.unpack(b);
#pragma unroll
      for (int i = 0; i < EC; ++i) {
        const float raw = dt[i] + bias[i];
        const float delta = on ? (a.softplus ? softplus(raw) : raw) : 0.f;
        sv[wave][w.t][w.q * EC + i] = make_float2(delta, delta * x[i]);
      }
      Vec<float, EN>::store(&sb[wave][w.t][w.q * EN], b);
      if constexpr (OUT) {
        now.c.unpack(c);
        Vec<float, EN>::store(&sc[wave][w.t][w.q * EN], c);
      }
      wave_lds_sync();
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const float2 v = sv[wave][t][w.ch];
        float bb[NS], cc[NS], y = 0.f;
        Vec<float, NS>::load(&sb[wave][t][n0], bb);
        if constexpr (OUT) Vec<float, NS>::load(&sc[wave][t][n0], cc);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          h[i] = fmaf(__builtin_amdgcn_exp2f(v.x * A[i]), h[i], v.y * bb[i]);
          if constexpr (OUT) y = fmaf(cc[i], h[i], y);
        }
        if constexpr (OUT) {
          y = state_sum<S>(y);
          if (w.sg == 0) sy[wave][t][w.ch] = y;
        }
      }
      wave_lds_sync();
      if constexpr (OUT) {
        if (on) {
          float z[EC], y[EC];
          now.z.unpack(z);
#pragma unroll
          for (int i = 0; i < EC; ++i) {
            y[i] = fmaf(skip[i], x[i], sy[wave][w.t][w.q * EC + i]);
            if (a.z.p) y[i] *= z[i] * sigmoid(z[i]);
          }
          store_row<T, EC>(a.out.out<T>((int64_t)q.tok + t0 + w.t) + w.c0 + w.q * EC, y);
        }
        wave_lds_sync();
      }
    }
    if constexpr (OUT) Vec<float, NS>::store(a.state + at, h);
  }
}

// Single tokens: a lane holds 4 states of a channel (2 where d_state = 8), so that a wave's state is
// one run of memory. Bound by HBM: the state read and written.
template <int S, int NS, typename T>
__global__ void __launch_bounds__(256) selective_step_kernel(const SelectiveArgs a, long long items) {
  constexpr int N = S * NS;
  const long long item = ((long long)blockIdx.x * 256 + threadIdx.x) / S;
  const int sg = threadIdx.x % S;
  if (item >= items) return;
  const int row = (int)(item / a.channels), c = (int)(item % a.channels);
  const int slot = a.slot ? a.slot[row] : row;
  if (slot < 0 || slot >= a.num_slots) return;
  float* state = a.state + ((size_t)slot * a.channels + c) * N + sg * NS;
  const int g = c / (a.channels / a.groups);
  float h[NS], A[NS], b[NS], cc[NS], x, dt, z = 0.f;
  Vec<float, NS>::load(state, h);
  Vec<float, NS>::load(a.A + (size_t)c * N + sg * NS, A);
  Vec<T, NS>::load(a.B.row<T>(row) + g * N + sg * NS, b);
  Vec<T, NS>::load(a.C.row<T>(row) + g * N + sg * NS, cc);
  Vec<T, 1>::load(a.x.row<T>(row) + c, &x);
  Vec<T, 1>::load(a.dt.row<T>(row) + c, &dt);
  if (a.z.p) Vec<T, 1>::load(a.z.row<T>(row) + c, &z);
  const float raw = dt + (a.dt_bias ? a.dt_bias[c] : 0.f);
  const float delta = a.softplus ? softplus(raw) : raw;
  float y = 0.f;
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    h[i] = fmaf(__builtin_amdgcn_exp2f(delta * (kLog2e * A[i])), h[i], delta * x * b[i]);
    y = fmaf(cc[i], h[i], y);
  }
  Vec<float, NS>::store(state, h);
  y = state_sum<S>(y);
  if (sg == 0) {
    if (a.D) y = fmaf(a.D[c], x, y);
    if (a.z.p) y *= z * sigmoid(z);
    store_row<T, 1>(a.out.out<T>(row) + c, &y);
  }
}

int walkers_of(const ssm_selective_dims& d, int tile_blocks) {
  const int most = 4096 / tile_blocks > 1 ? 4096 / tile_blocks : 1;
  return d.batch < most ? (d.batch > 0 ? d.batch : 1) : most;
}

int tiles_of(const ssm_selective_dims& d) {  // of the mapping of selective_dispatch
  const int S = d.d_state <= 16 ? 4 : d.d_state / 4;
  return d.channels * S / 64;
}
int tile_blocks_of(const ssm_selective_dims& d) { return (tiles_of(d) + WAVES - 1) / WAVES; }

template <bool OUT>
hipError_t launch_scan_pass(const ssm_selective_dims& d, SelectiveArgs& a, hipStream_t stream) {
  const int tb = tile_blocks_of(d);
  a.walkers = walkers_of(d, tb);
  return selective_dispatch(d, [&](auto S, auto NS, auto T) {
    hipLaunchKernelGGL((selective_scan_kernel<decltype(S)::value, decltype(NS)::value,
                                              typename decltype(T)::type, OUT>),
                       dim3((unsigned)tb * (unsigned)a.walkers), dim3(64 * WAVES), 0, stream, a);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_selective_states(const ssm_selective_dims& d, SelectiveArgs& a, hipStream_t stream) {
  return launch_scan_pass<false>(d, a, stream);
}

SelectiveWork selective_work(const ssm_selective_dims& d, int total, bool backward, void* base) {
  SelectiveWork w{};
  if (!backward) return w;
  const int tb = tile_blocks_of(d);
  size_t at = 0;
  auto take = [&](size_t floats) {
    float* p = reinterpret_cast<float*>(static_cast<char*>(base) + at);
    at += floats * sizeof(float);
    return p;
  };
  w.states = take(((size_t)total / TB + 1) * d.channels * d.d_state);
  w.dbc = take((size_t)total * tiles_of(d) * 2 * d.d_state);
  w.partial = take((size_t)walkers_of(d, tb) * d.channels * (d.d_state + 2));
  w.bytes = at;
  return w;
}

hipError_t launch_selective_forward(const ssm_selective_dims& d, SelectiveArgs& a, hipStream_t stream) {
  return launch_scan_pass<true>(d, a, stream);
}

hipError_t launch_selective_step(const ssm_selective_dims& d, const SelectiveArgs& a,
                                 hipStream_t stream) {
  const long long items = (long long)d.batch * d.channels;
  return selective_dispatch(d, [&](auto S, auto NS, auto T) {
    constexpr int s = decltype(S)::value;
    hipLaunchKernelGGL((selective_step_kernel<s, decltype(NS)::value, typename decltype(T)::type>),
                       dim3((unsigned)((items * s + 255) / 256)), dim3(256), 0, stream, a, items);
    return hipGetLastError();
  });
}

}  // namespace ssm
