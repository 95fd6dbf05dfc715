// conv.hip -- the short causal convolution of a layer's inputs, its activation and the l2 norm of
// queries and keys, forward, backward and for single tokens (formulas in include/sketchssm.h).
//
// One pass over the tokens: every lane holds E channels, its taps and the last K - 1 inputs in registers
// and walks a run of tokens, so that an input is read once (and K - 1 more at the start of a run)
// and nothing goes through LDS. Bound by HBM. A norm's run of channels is 2 to 32 neighbouring lanes: its
// sums are DPP steps. E = 8 forward (16 bytes of bf16 a load) and 4 backward, whose sums for the weights
// would otherwise take 256 registers and leave one wave a SIMD (327 us instead of 158 for the case below).
//
// 8192 tokens of 12,288 channels in bf16, queries and keys normalised: forward 86 us for 403 MB, 4.7 TB/s, the rate
// of a large copy on this card; backward 140 us for 604 MB, 4.3 TB/s, its vector units issuing in 86 % of the cycles
// (39 instructions a value). A run is a chunk's 64 tokens; shorter where that leaves fewer than 2,048 waves. One token of
// 256 rows: 13.5 us for 50 MB.
#include "layer.hpp"
#include "launch.hpp"

namespace ssm {

namespace {

constexpr int NT = 256;  // threads of a workgroup: four waves, each on runs of its own

constexpr int EF = 8, EB = 4;  // channels of a lane, forward and backward

// This lane's part, tile and run.
struct ConvLane {
  int part, run, c;  // c: first of the lane's channels in the part
  bool active;
};
template <int E>
__device__ __forceinline__ ConvLane conv_lane(const ConvArgs& a) {
  int p = 0;
#pragma unroll
  for (int i = 1; i < CP; ++i)
    if (i < a.parts && (int)blockIdx.x >= a.part[i].first_block) p = i;
  const ConvPart& P = a.part[p];
  const int b = blockIdx.x - P.first_block, log = P.log_lanes;
  const int tile = b % P.tiles, lane = threadIdx.x & 63;
  ConvLane l;
  l.part = p;
  l.run = (b / P.tiles * (NT >> 6) + (threadIdx.x >> 6)) * (64 >> log) + (lane >> log);
  l.c = ((tile << log) + (lane & ((1 << log) - 1))) * E;
  l.active = l.c < P.channels;
  return l;
}

// Sum over an aligned run of 2, 4, .. 32 lanes (all of them active).
__device__ __forceinline__ float run_sum(float x, int lanes) {
  x += dpp<DPP_QUAD_1032>(x);
  if (lanes >= 4) x += dpp<DPP_QUAD_2301>(x);
  if (lanes >= 8) x += dpp<DPP_HALF_MIRROR>(x);
  if (lanes >= 16) x += dpp<DPP_ROR8>(x);
  if (lanes >= 32) x = xsum16(x);
  return x;
}
// The same of two values: as in the sum of one, but each test is made once.
__device__ __forceinline__ void run_sums(float& x, float& y, int lanes) {
  const auto both = [&](auto f) { x += f(x); y += f(y); };
  both([](float v) { return dpp<DPP_QUAD_1032>(v); });
  if (lanes >= 4) both([](float v) { return dpp<DPP_QUAD_2301>(v); });
  if (lanes >= 8) both([](float v) { return dpp<DPP_HALF_MIRROR>(v); });
  if (lanes >= 16) both([](float v) { return dpp<DPP_ROR8>(v); });
  if (lanes >= 32) {
    x = xsum16(x);
    y = xsum16(y);
  }
}

template <int K, int E>
struct Taps {
  float w[E * K], b[E];
  __device__ __forceinline__ void load(const ConvArgs& a, int c) {
    Vec<float, E * K>::load(a.weight + (size_t)c * K, w);
    if (a.bias) {
      Vec<float, E>::load(a.bias + c, b);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) b[i] = 0.f;
    }
  }
  // u of the token whose inputs are x[K - 1], the ones before it x[0 .. K - 2]
  __device__ __forceinline__ float at(const float (*x)[E], int i) const {
    float u = b[i];
#pragma unroll
    for (int j = 0; j < K; ++j) u = fmaf(w[i * K + j], x[j][i], u);
    return u;
  }
};

template <typename T, int E>
__device__ __forceinline__ void store_channels(T* p, const float (&v)[E]) {
  if constexpr (E == 8) store8(p, v);
  else store4(p, make_float4(v[0], v[1], v[2], v[3]));
}
template <int E>
__device__ __forceinline__ void clear(float (&v)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] = 0.f;
}

// y of a token from its window of inputs
template <int K, int E>
__device__ __forceinline__ void conv_token(const ConvArgs& a, const ConvPart& P, const Taps<K, E>& taps,
                                           const float (*x)[E], float (&y)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) y[i] = taps.at(x, i);
  if (a.silu) {
#pragma unroll
    for (int i = 0; i < E; ++i) y[i] *= sigmoid(y[i]);
  }
  if (P.norm_lanes) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(y[i], y[i], s);
    const float r = P.scale * __builtin_amdgcn_rsqf(run_sum(s, P.norm_lanes) + a.eps);
#pragma unroll
    for (int i = 0; i < E; ++i) y[i] *= r;
  }
}

// A run of tokens of one sequence.
struct Run {
  int seq, slot, first, len;  // the sequence: its number, state, first token and length
  int pos, count;             // the run's first token in the sequence, and its tokens
};
__device__ __forceinline__ bool slot_of(const ConvArgs& a, int seq, int& slot) {
  slot = a.slot ? a.slot[seq] : seq;
  return slot >= 0 && slot < a.num_slots;
}
// Run r of the chunks; false where it holds no token.
__device__ __forceinline__ bool conv_run(const ConvArgs& a, int r, Run& run) {
  const int per = 6 - a.log_run;  // log2 of a chunk's runs
  if (r >= a.runs || !a.plan.locate(r >> per, run.seq, run.first, run.len, run.pos)) return false;
  const int skip = (r & ((1 << per) - 1)) << a.log_run, left = run.len - run.pos;
  run.count = min(min(left, CT) - skip, 1 << a.log_run);
  run.pos += skip;
  return run.count > 0 && slot_of(a, run.seq, run.slot);
}

// The sequence whose state run r has to carry over because it holds no token: sequence e without
// tokens is dealt with by the first run of table entry e (the table has an entry for every sequence).
__device__ __forceinline__ bool empty_sequence(const ConvArgs& a, int r, int& slot) {
  const int per = 6 - a.log_run, e = r >> per;
  if (r >= a.runs || (r & ((1 << per) - 1)) != 0 || e >= a.plan.seqs) return false;
  int tok, len, first;
  return a.plan.sequence(e, tok, len, first) && len == 0 && slot_of(a, e, slot);
}

// The K - 1 inputs before the run, oldest first: tokens of the sequence, or its kept state.
template <int K, int E, typename T>
__device__ __forceinline__ void history(const ConvArgs& a, const ConvPart& P, const Run& run, int c,
                                        float (*x)[E]) {
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    const int p = run.pos - (K - 1) + j;
    if (p >= 0) {
      Vec<T, E>::load(P.x.row<T>(run.first + p) + c, x[j]);
    } else if (a.state_in) {
      Vec<T, E>::load(static_cast<const T*>(a.state_in) +
                          ((size_t)run.slot * (K - 1) + (K - 1 + p)) * a.C + P.offset + c,
                      x[j]);
    } else {
      clear(x[j]);
    }
  }
}

template <int K, typename T>
__global__ void __launch_bounds__(NT) conv_forward_kernel(const ConvArgs a) {
  constexpr int E = EF;
  const ConvLane l = conv_lane<E>(a);
  if (!l.active) return;
  const ConvPart& P = a.part[l.part];
  const int c = l.c;
  constexpr int U = 8;  // tokens fetched at once
  int slot;
  if (a.state && a.state != a.state_in && empty_sequence(a, l.run, slot)) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const size_t at = ((size_t)slot * (K - 1) + j) * a.C + P.offset + c;
      float v[E];
      clear(v);
      if (a.state_in) Vec<T, E>::load(static_cast<const T*>(a.state_in) + at, v);
      store_channels(static_cast<T*>(a.state) + at, v);
    }
  }
  Run run;
  if (!conv_run(a, l.run, run)) return;
  Taps<K, E> taps;
  taps.load(a, P.offset + c);
  float x[K - 1 + U][E];
  history<K, E, T>(a, P, run, c, x);
  if (run.pos == 0 && a.state) {
    // the last K - 1 of the kept inputs and the sequence's; read before they are written, since
    // both may be the same memory: only this lane touches them
    const int len = run.len;
    float end[K - 1][E];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int p = len - (K - 1) + j;
      if (p >= 0) {
        Vec<T, E>::load(P.x.row<T>(run.first + p) + c, end[j]);
      } else {
#pragma unroll
        for (int h = 0; h < K - 1; ++h)
          if (K - 1 + p == h)
#pragma unroll
            for (int i = 0; i < E; ++i) end[j][i] = x[h][i];
      }
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
      store_channels(static_cast<T*>(a.state) + ((size_t)run.slot * (K - 1) + j) * a.C + P.offset + c, end[j]);
  }
  const T* in = P.x.row<T>(run.first + run.pos) + c;
  T* out = P.y.out<T>(run.first + run.pos) + c;
  for (int t = 0; t < run.count; t += U) {
    Packed<T, E> raw[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (t + i < run.count) raw[i].load(in + (int64_t)(t + i) * P.x.stride);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (t + i < run.count) {
        raw[i].unpack(x[K - 1 + i]);
        float y[E];
        conv_token(a, P, taps, x + i, y);
        store_channels(out + (int64_t)(t + i) * P.y.stride, y);
      }
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
#pragma unroll
      for (int i = 0; i < E; ++i) x[j][i] = x[U + j][i];
  }
}

// Gradients. With g = dL/du, dx of a token is sum_j w_j g of the token K-1-j after it, so a run goes
// on for K - 1 tokens behind its end (their g once more), and the first run of a sequence
// makes the gradient of the kept inputs on the way.
// The next four tokens' rows are on their way; a row's registers are filled again as soon as it is unpacked, and its
// address is one step on from the row before (140 us for 8192 tokens of 12,288 channels; 152 with four rows unpacked,
// then four fetched at products of their numbers). Three waves a SIMD: four would put 25 registers into memory
// (190 us); eight tokens ahead 150 us.
template <int K, typename T>
__global__ void __launch_bounds__(NT, 3) conv_backward_kernel(const ConvArgs a) {
  constexpr int E = EB, U = 4;
  const ConvLane l = conv_lane<E>(a);
  if (!l.active || l.run >= a.rows) return;
  const ConvPart& P = a.part[l.part];
  const int c = l.c;
  Taps<K, E> taps;
  taps.load(a, P.offset + c);
  float dw[E * K], db[E];
  clear(dw);
  clear(db);
  for (int r = l.run; r < a.runs; r += a.rows) {
    int slot;
    if (a.dstate_in && empty_sequence(a, r, slot)) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        const size_t at = ((size_t)slot * (K - 1) + j) * a.C + P.offset + c;
        float v[E];
        clear(v);
        if (a.dstate) Vec<T, E>::load(static_cast<const T*>(a.dstate) + at, v);
        store_channels(static_cast<T*>(a.dstate_in) + at, v);
      }
    }
    Run run;
    if (!conv_run(a, r, run)) continue;
    float x[K - 1 + U][E], g[K - 1 + U][E];  // [K - 1 + i]: of token t + i
    history<K, E, T>(a, P, run, c, x);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) clear(g[j]);
    const int left = run.len - run.pos;           // tokens up to the sequence's end
    const int steps = run.count + K - 1, with_g = min(steps, left);
    const int64_t t0 = (int64_t)run.first + run.pos;
    Packed<T, E> rx[U], ry[U];
    const T *nx = P.x.row<T>(t0) + c, *ny = P.dy.row<T>(t0) + c;  // the row to be read next
#pragma unroll
    for (int i = 0; i < U; ++i) {  // rows behind the last are read again, and not used
      rx[i].load(nx);
      ry[i].load(ny);
      nx += i + 1 < with_g ? P.x.stride : 0;
      ny += i + 1 < with_g ? P.dy.stride : 0;
    }
    T* px = P.dx.out<T>(t0) + c - (K - 1) * P.dx.stride;  // where dx of token t - (K - 1) goes
    for (int t = 0; t < steps; t += U) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float(&gt)[E] = g[K - 1 + i];
        float dy[E];
        rx[i].unpack(x[K - 1 + i]);
        ry[i].unpack(dy);
        rx[i].load(nx);
        ry[i].load(ny);
        const bool more = t + i + U + 1 < with_g;
        nx += more ? P.x.stride : 0;
        ny += more ? P.dy.stride : 0;
        float act[E], slope[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          act[e] = taps.at(x + i, e);
          slope[e] = 1.f;
        }
        if (a.silu) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float s = sigmoid(act[e]);
            act[e] *= s;
            slope[e] = fmaf(act[e], 1.f - s, s);
          }
        }
        if (P.norm_lanes) {
          float s = 0.f, d = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            s = fmaf(act[e], act[e], s);
            d = fmaf(act[e], dy[e], d);
          }
          run_sums(s, d, P.norm_lanes);
          const float r1 = __builtin_amdgcn_rsqf(s + a.eps), f = P.scale * r1;
          d *= -r1 * r1;
#pragma unroll
          for (int e = 0; e < E; ++e) dy[e] = f * fmaf(act[e], d, dy[e]);
        }
        const bool here = t + i < with_g;
#pragma unroll
        for (int e = 0; e < E; ++e) gt[e] = here ? dy[e] * slope[e] : 0.f;
        if (t + i < run.count) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            db[e] += gt[e];
#pragma unroll
            for (int j = 0; j < K; ++j) dw[e * K + j] = fmaf(gt[e], x[i + j][e], dw[e * K + j]);
          }
        }
        // dx of the token K - 1 back
        const int s = t + i - (K - 1);
        if ((t + i < steps && (s >= 0 || (run.pos == 0 && a.dstate_in)))) {
          float dx[E];
          const int end = t + i - left;  // its row in the final state, if any
          if (a.dstate && end >= 0 && end < K - 1) {
            Vec<T, E>::load(static_cast<const T*>(a.dstate) +
                                ((size_t)run.slot * (K - 1) + end) * a.C + P.offset + c,
                            dx);
          } else {
            clear(dx);
          }
#pragma unroll
          for (int j = 0; j < K; ++j)
#pragma unroll
            for (int e = 0; e < E; ++e) dx[e] = fmaf(taps.w[e * K + j], g[K - 1 + i - j][e], dx[e]);
          if (s >= 0) {
            store_channels(px + i * P.dx.stride, dx);
          } else {
            store_channels(static_cast<T*>(a.dstate_in) + ((size_t)run.slot * (K - 1) + t + i) * a.C +
                               P.offset + c,
                           dx);
          }
        }
      }
      px += U * P.dx.stride;
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          x[j][e] = x[U + j][e];
          g[j][e] = g[U + j][e];
        }
    }
  }
  float* row = a.partial + (size_t)l.run * (K + 1) * a.C + P.offset + c;
#pragma unroll
  for (int j = 0; j < K; ++j) {
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = dw[e * K + j];
    store_channels(row + (size_t)j * a.C, v);
  }
  store_channels(row + (size_t)K * a.C, db);
}

// The sums over the rows of partial sums, in a fixed order: 64 columns by 16 runs of rows a workgroup.
constexpr int RY = 16;
__global__ void __launch_bounds__(64 * RY)
conv_sum_kernel(const float* __restrict__ partial, int rows, int K, int C, float* __restrict__ dweight,
                float* __restrict__ dbias) {
  __shared__ float part[RY][64];
  const int x = threadIdx.x & 63, y = threadIdx.x >> 6, cols = (K + 1) * C;
  const int col = blockIdx.x * 64 + x;
  float s = 0.f;
  if (col < cols) {
#pragma unroll 8
    for (int r = y; r < rows; r += RY) s += partial[(size_t)r * cols + col];
  }
  part[y][x] = s;
  __syncthreads();
  if (y > 0 || col >= cols) return;
#pragma unroll
  for (int i = 1; i < RY; ++i) s += part[i][x];
  const int j = col / C, c = col % C;
  if (j < K) dweight[(size_t)c * K + j] = s;
  else if (dbias) dbias[c] = s;
}

template <int K, typename T>
__global__ void __launch_bounds__(NT) conv_step_kernel(const ConvArgs a) {
  constexpr int E = EF;
  const ConvLane l = conv_lane<E>(a);
  int slot;
  if (!l.active || l.run >= a.runs || !slot_of(a, l.run, slot)) return;
  const ConvPart& P = a.part[l.part];
  T* state = static_cast<T*>(a.state) + (size_t)slot * (K - 1) * a.C + P.offset + l.c;
  Packed<T, E> raw[K];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) raw[j].load(state + (size_t)j * a.C);
  raw[K - 1].load(P.x.row<T>(l.run) + l.c);
  Taps<K, E> taps;
  taps.load(a, P.offset + l.c);
  float x[K][E], y[E];
#pragma unroll
  for (int j = 0; j < K; ++j) raw[j].unpack(x[j]);
  conv_token(a, P, taps, x, y);
  store_channels(P.y.out<T>(l.run) + l.c, y);
#pragma unroll
  for (int j = 0; j < K - 1; ++j) raw[j + 1].store(state + (size_t)j * a.C);
}

// Calls f(taps, input type) with compile-time constants.
template <typename F>
hipError_t conv_dispatch(const ssm_conv_dims& d, F&& f) {
  auto with = [&](auto K) -> hipError_t {
    if (d.in_dtype == SSM_IN_BF16) return f(K, type_tag<uint16_t>{});
    return f(K, type_tag<float>{});
  };
  switch (d.taps) {
    case 2: return with(std::integral_constant<int, 2>{});
    case 3: return with(std::integral_constant<int, 3>{});
    case 4: return with(std::integral_constant<int, 4>{});
  }
  return hipErrorInvalidValue;
}

// Tiles of the parts, with E channels a lane; returns the grid for `runs` runs of a tile.
template <int E>
unsigned conv_grid(ConvArgs& a, int runs) {
  unsigned blocks = 0;
  for (int p = 0; p < a.parts; ++p) {
    ConvPart& P = a.part[p];
    int log = 1;
    while (log < 6 && (E << log) < P.channels) ++log;
    P.norm_lanes = P.norm / E;
    while ((1 << log) < P.norm_lanes) ++log;  // a norm's run stays inside a tile
    P.log_lanes = log;
    P.tiles = (P.channels + (E << log) - 1) / (E << log);
    P.first_block = (int)blocks;
    const int at_once = (NT >> 6) * (64 >> log);
    blocks += (unsigned)P.tiles * (unsigned)((runs + at_once - 1) / at_once);
  }
  return blocks;
}

constexpr int kWaves = 2048;  // of the whole GPU, two a SIMD, below which runs are made shorter

// log2 of the tokens of a run, for waves of `wide` channels
int run_log(int cap, int C, int wide) {
  int log = 6;
  while (log > 3 && ((long long)cap << (6 - log)) * ((C + wide - 1) / wide) < kWaves) --log;
  return log;
}

constexpr int kMostRows = 1024;  // of partial sums: a row is (taps + 1) C floats, written and read once
int partial_rows(int runs) { return runs < kMostRows ? runs : kMostRows; }

int channels_of(const ssm_conv_dims& d) {
  int C = 0;
  for (int p = 0; p < d.parts; ++p) C += d.channels[p];
  return C;
}

}  // namespace

size_t conv_workspace(const ssm_conv_dims& d, int total) {
  const int C = channels_of(d), cap = scan_capacity(total, d.batch);
  const int log = run_log(cap, C, 64 * EB);
  return (size_t)partial_rows(cap << (6 - log)) * (d.taps + 1) * C * sizeof(float);
}

hipError_t launch_conv_forward(const ssm_conv_dims& d, ConvArgs& a, hipStream_t stream) {
  a.log_run = run_log(a.plan.cap, a.C, 64 * EF);
  a.runs = a.plan.cap << (6 - a.log_run);
  const unsigned grid = conv_grid<EF>(a, a.runs);
  return conv_dispatch(d, [&](auto K, auto T) {
    hipLaunchKernelGGL((conv_forward_kernel<decltype(K)::value, typename decltype(T)::type>),
                       dim3(grid), dim3(NT), 0, stream, a);
    return hipGetLastError();
  });
}

hipError_t launch_conv_backward(const ssm_conv_dims& d, ConvArgs& a, hipStream_t stream) {
  a.log_run = run_log(a.plan.cap, a.C, 64 * EB);
  a.runs = a.plan.cap << (6 - a.log_run);
  a.rows = partial_rows(a.runs);
  const unsigned grid = conv_grid<EB>(a, a.rows);
  return conv_dispatch(d, [&](auto K, auto T) {
    constexpr int k = decltype(K)::value;
    if (a.rows > 0) {  // no sequences: the sums of nothing are still written
      hipLaunchKernelGGL((conv_backward_kernel<k, typename decltype(T)::type>), dim3(grid), dim3(NT),
                         0, stream, a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    const int cols = (k + 1) * a.C;
    hipLaunchKernelGGL(conv_sum_kernel, dim3((cols + 63) / 64), dim3(64 * RY), 0, stream, a.partial,
                       a.rows, k, a.C, a.dweight, a.dbias);
    return hipGetLastError();
  });
}

hipError_t launch_conv_step(const ssm_conv_dims& d, ConvArgs& a, hipStream_t stream) {
  a.runs = d.batch;
  const unsigned grid = conv_grid<EF>(a, a.runs);
  return conv_dispatch(d, [&](auto K, auto T) {
    hipLaunchKernelGGL((conv_step_kernel<decltype(K)::value, typename decltype(T)::type>),
                       dim3(grid), dim3(NT), 0, stream, a);
    return hipGetLastError();
  });
}

}  // namespace ssm
