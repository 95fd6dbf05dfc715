// selective_grads.hip -- gradients of the selective recurrence.
//
// Backwards over a sequence, with G = dL/dh of a token (all later ones included):
//   G_t = C_t dy_t + a_{t+1} G_{t+1},  a = exp(delta A)
//   dC = sum_channels dy h,  dB = sum_channels G delta x,
//   e = sum_n G B,  dx = delta e + D dy,  ddelta = x e + sum_n G a h_{t-1} A,
//   dA = sum_t delta G a h_{t-1},  dstate_in = a_0 G_0.
// The states are computed again, a block of 16 tokens at a time, from those that a forward pass left
// before every block. A wave's sums over channels are stored for each token and added up
// afterwards in a fixed order; those over tokens stay in registers.
#include "selective.hpp"

namespace ssm {

namespace {

template <typename T, int S, int NS>
struct GradBlock {
  using SH = SelShape<S, NS>;
  Packed<T, SH::EC> x, dt, z, dy;
  Packed<T, SH::EN> b, c;
  float h0[NS];  // the state before the block
  __device__ __forceinline__ void load(const SelectiveArgs& a, const SelTile& w, const SelCell& cell, int t0,
                                       int my, int n) {
    const bool on = t0 + w.t < cell.count;
    const int64_t tok = (int64_t)cell.first + cell.pos + t0 + w.t;
    const int c0 = w.c0 + w.q * SH::EC, n0 = w.group * SH::N + w.q * SH::EN;
    load_or_zero(x, a.x.row<T>(tok) + c0, on);
    load_or_zero(dt, a.dt.row<T>(tok) + c0, on);
    load_or_zero(dy, a.dout.row<T>(tok) + c0, on);
    load_or_zero(z, a.z.p ? a.z.row<T>(tok) + c0 : nullptr, on && a.z.p);
    load_or_zero(b, a.B.row<T>(tok) + n0, on);
    load_or_zero(c, a.C.row<T>(tok) + n0, on);
    if (cell.pos + t0 > 0) {
      const size_t block = (size_t)(cell.first / TB + (cell.pos + t0) / TB - 1);
      Vec<float, NS>::load(a.w.states + (block * a.channels + my) * SH::N + n, h0);
    } else if (a.state_in) {
      Vec<float, NS>::load(a.state_in + ((size_t)cell.slot * a.channels + my) * SH::N + n, h0);
    } else {
      zero(h0);
    }
  }
};

template <int S, int NS, typename T>
__global__ void __launch_bounds__(64 * WAVES) selective_grads_kernel(const SelectiveArgs a) {
  using SH = SelShape<S, NS>;
  constexpr int N = SH::N, CH = SH::CH, EC = SH::EC, EN = SH::EN;
  __shared__ __align__(16) float4 sv[WAVES][TB][CH];  // delta, delta x, dL/dy, -
  __shared__ __align__(16) float sb[WAVES][TB][N], sc[WAVES][TB][N];
  __shared__ __align__(16) float4 so[WAVES][TB][CH];  // sum G B, sum G a h A, y
  const int wave = threadIdx.x >> 6, tiles = a.channels / CH;
  const int tile_blocks = (tiles + WAVES - 1) / WAVES;
  const int tile = blockIdx.x % tile_blocks * WAVES + wave;
  if (tile >= tiles) return;
  const SelTile w = sel_tile<S>(a, tile);
  const SelGroup grp = sel_group(a, blockIdx.x / tile_blocks);
  const int my = w.c0 + w.ch, n0 = w.sg * NS;
  float A[NS], A2[NS], dA[NS], bias[EC], skip[EC], dD[EC], dbias[EC];
  Vec<float, NS>::load(a.A + (size_t)my * N + n0, A);
  zero(dA);
  zero(dD);
  zero(dbias);
#pragma unroll
  for (int i = 0; i < NS; ++i) A2[i] = kLog2e * A[i];
#pragma unroll
  for (int i = 0; i < EC; ++i) {
    bias[i] = a.dt_bias ? a.dt_bias[w.c0 + w.q * EC + i] : 0.f;
    skip[i] = a.D ? a.D[w.c0 + w.q * EC + i] : 0.f;
  }
  if (a.dstate_in)
    for_empty_sequences(a, grp, [&](int, int slot) {
      const size_t at = ((size_t)slot * a.channels + my) * N + n0;
      float v[NS];
      zero(v);
      if (a.dstate) Vec<float, NS>::load(a.dstate + at, v);
      Vec<float, NS>::store(a.dstate_in + at, v);
    });
  SelCell cell, ahead;
  bool more = prev_cell(a, grp.e1 - 1, grp.e0 - 1, cell);
  float g[NS];
  zero(g);
  if (more && !cell.ends()) carry_back<N>(a, grp, cell, my, n0, A2, g);
  for (; more; cell = ahead) {
    more = prev_cell(a, cell.entry - 1, grp.e0 - 1, ahead);
    const size_t at = ((size_t)cell.slot * a.channels + my) * N + n0;
    if (cell.ends()) {
      zero(g);
      if (a.dstate) Vec<float, NS>::load(a.dstate + at, g);
    }
    for (int t0 = (cell.count - 1) / TB * TB; t0 >= 0; t0 -= TB) {
      GradBlock<T, S, NS> now;
      now.load(a, w, cell, t0, my, n0);
      const bool on = t0 + w.t < cell.count;
      const int64_t tok = (int64_t)cell.first + cell.pos + t0 + w.t;
      const float(&h0)[NS] = now.h0;
      float x[EC], raw[EC], z[EC], dy[EC], dout[EC], b[EN], c[EN];
      now.x.unpack(x);
      now.dt.unpack(raw);
      now.z.unpack(z);
      now.dy.unpack(dout);
      now.b.unpack(b);
      now.c.unpack(c);
#pragma unroll
      for (int i = 0; i < EC; ++i) {
        raw[i] += bias[i];
        const float delta = on ? (a.softplus ? softplus(raw[i]) : raw[i]) : 0.f;
        dy[i] = a.z.p ? dout[i] * (z[i] * sigmoid(z[i])) : dout[i];
        sv[wave][w.t][w.q * EC + i] = make_float4(delta, delta * x[i], dy[i], 0.f);
      }
      Vec<float, EN>::store(&sb[wave][w.t][w.q * EN], b);
      Vec<float, EN>::store(&sc[wave][w.t][w.q * EN], c);
      wave_lds_sync();
      float h[TB][NS], d[TB][NS];  // states after, decays
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const float4 v = sv[wave][t][w.ch];
        float bb[NS];
        Vec<float, NS>::load(&sb[wave][t][n0], bb);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          d[t][i] = __builtin_amdgcn_exp2f(v.x * A2[i]);
          h[t][i] = fmaf(d[t][i], t ? h[t ? t - 1 : 0][i] : h0[i], v.y * bb[i]);
        }
      }
#pragma unroll
      for (int t = TB - 1; t >= 0; --t) {
        const float4 v = sv[wave][t][w.ch];
        float bb[NS], cc[NS], dB[NS], dC[NS];
        Vec<float, NS>::load(&sb[wave][t][n0], bb);
        Vec<float, NS>::load(&sc[wave][t][n0], cc);
        float e = 0.f, f = 0.f, y = 0.f;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          g[i] = fmaf(cc[i], v.z, g[i]);
          dC[i] = v.z * h[t][i];
          dB[i] = v.y * g[i];
          y = fmaf(cc[i], h[t][i], y);
          e = fmaf(bb[i], g[i], e);
          const float p = g[i] * (d[t][i] * (t ? h[t ? t - 1 : 0][i] : h0[i]));
          dA[i] = fmaf(v.x, p, dA[i]);
          f = fmaf(A[i], p, f);
          g[i] *= d[t][i];
        }
        e = state_sum<S>(e);
        f = state_sum<S>(f);
        y = state_sum<S>(y);
        if (w.sg == 0) so[wave][t][w.ch] = make_float4(e, f, y, 0.f);
        // every lane has read this token's B and C: the sums over channels take their place
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          dB[i] = channel_sum<S>(dB[i]);
          dC[i] = channel_sum<S>(dC[i]);
        }
        wave_lds_sync();
        if (w.ch == 0) {
          Vec<float, NS>::store(&sb[wave][t][n0], dB);
          Vec<float, NS>::store(&sc[wave][t][n0], dC);
        }
      }
      wave_lds_sync();
      if (on) {
        float dx[EC], ddt[EC], dz[EC];
#pragma unroll
        for (int i = 0; i < EC; ++i) {
          const float4 o = so[wave][w.t][w.q * EC + i];
          const float delta = a.softplus ? softplus(raw[i]) : raw[i];
          dx[i] = fmaf(delta, o.x, skip[i] * dy[i]);
          ddt[i] = fmaf(x[i], o.x, o.y) * (a.softplus ? sigmoid(raw[i]) : 1.f);
          dbias[i] += ddt[i];
          dD[i] = fmaf(dy[i], x[i], dD[i]);
          const float s = sigmoid(z[i]);
          dz[i] = dout[i] * fmaf(skip[i], x[i], o.z) * (s * fmaf(z[i], 1.f - s, 1.f));
        }
        const int c0 = w.c0 + w.q * EC;
        store_row<T, EC>(a.dx.out<T>(tok) + c0, dx);
        store_row<T, EC>(a.ddt.out<T>(tok) + c0, ddt);
        if (a.z.p) store_row<T, EC>(a.dz.out<T>(tok) + c0, dz);
        float* to = a.w.dbc + ((size_t)tok * tiles + tile) * 2 * N + w.q * EN;
        Vec<float, EN>::load(&sb[wave][w.t][w.q * EN], b);
        Vec<float, EN>::load(&sc[wave][w.t][w.q * EN], c);
        Vec<float, EN>::store(to, b);
        Vec<float, EN>::store(to + N, c);
      }
      wave_lds_sync();
    }
    if (a.dstate_in && cell.starts()) Vec<float, NS>::store(a.dstate_in + at, g);
  }
  // this group's sums over tokens: dA, then dD and ddt_bias
  float* sums = a.w.partial + (size_t)grp.g * a.channels * (N + 2);
  Vec<float, NS>::store(sums + (size_t)my * N + n0, dA);
#pragma unroll
  for (int i = 0; i < EC; ++i) {
    dD[i] = channel_sum<4>(dD[i]);  // over the 16 tokens of a block: lanes with the same quarter
    dbias[i] = channel_sum<4>(dbias[i]);
  }
  if (w.t == 0) {
    float* p = sums + (size_t)a.channels * N + w.c0 + w.q * EC;
    Vec<float, EC>::store(p, dD);
    Vec<float, EC>::store(p + a.channels, dbias);
  }
}

// dB and dC: the sums over the tiles of a group.
template <int N, typename T>
__global__ void __launch_bounds__(256) selective_sum_tiles_kernel(const SelectiveArgs a, int tiles) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int n = (int)(i % (2 * N)), g = (int)(i / (2 * N) % a.groups);
  const long long tok = i / (2 * N) / a.groups;
  // tokens behind the last sequence have no sums
  if (tok >= a.plan.total || tok >= a.plan.start(a.plan.seqs)) return;
  const int per = tiles / a.groups;
  const float* p = a.w.dbc + ((size_t)tok * tiles + (size_t)g * per) * 2 * N + n;
  float s = 0.f;
#pragma unroll 8
  for (int k = 0; k < per; ++k) s += p[(size_t)k * 2 * N];
  T* to = n < N ? a.dB.out<T>(tok) + g * N + n : a.dC.out<T>(tok) + g * N + n - N;
  store_row<T, 1>(to, &s);
}

// dA, dD and ddt_bias: the sums over the groups of chunks.
__global__ void __launch_bounds__(256)
selective_sum_groups_kernel(const SelectiveArgs a, int N) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  const int cols = a.channels * (N + 2);
  if (i >= cols) return;
  float s = 0.f;
#pragma unroll 8
  for (int k = 0; k < a.time_groups; ++k) s += a.w.partial[(size_t)k * cols + i];
  const int dA = a.channels * N;
  if (i < dA) a.dA[i] = s;
  else if (i < dA + a.channels) {
    if (a.dD) a.dD[i - dA] = s;
  } else if (a.ddt_bias) {
    a.ddt_bias[i - dA - a.channels] = s;
  }
}

}  // namespace

hipError_t launch_selective_backward(const ssm_selective_dims& d, SelectiveArgs& a, hipStream_t stream) {
  hipError_t e = launch_selective_local(d, a, true, stream);
  if (e == hipSuccess) e = launch_selective_states(d, a, stream);
  if (e != hipSuccess) return e;
  return selective_dispatch(d, [&](auto S, auto NS, auto T) {
    constexpr int s = decltype(S)::value, ns = decltype(NS)::value;
    using TI = typename decltype(T)::type;
    const int tiles = d.channels * s / 64, tb = (tiles + WAVES - 1) / WAVES;
    hipLaunchKernelGGL((selective_grads_kernel<s, ns, TI>), dim3((unsigned)tb * (unsigned)a.time_groups),
                       dim3(64 * WAVES), 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const long long sums = (long long)a.plan.total * a.groups * 2 * s * ns;
    if (sums > 0) {
      hipLaunchKernelGGL((selective_sum_tiles_kernel<s * ns, TI>), dim3((unsigned)((sums + 255) / 256)),
                         dim3(256), 0, stream, a, tiles);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const int cols = d.channels * (d.d_state + 2);
    hipLaunchKernelGGL(selective_sum_groups_kernel, dim3((cols + 255) / 256), dim3(256), 0, stream, a,
                       d.d_state);
    return hipGetLastError();
  });
}

}  // namespace ssm
