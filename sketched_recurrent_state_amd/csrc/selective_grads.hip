// selective_grads.hip -- gradients of the selective recurrence.
//
// Backwards over a sequence, with G = dL/dh of a token (all later ones included):
//   G_t = C_t dy_t + a_{t+1} G_{t+1},  a = exp(delta A)
//   dC = sum_channels dy h,  dB = sum_channels G delta x,
//   e = sum_n G B,  dx = delta e + D dy,  ddelta = x e + sum_n G a h_{t-1} A,
//   dA = sum_t delta G a h_{t-1},  dstate_in = a_0 G_0.
// The first pass keeps the state before every 8 tokens as it is from the group's zero, so it need not know the groups
// before; the walk back adds to each exp(A sum delta) h of the group's start (4 exps a lane for 8 tokens, where a pass of its
// own for the true states took 79 us), and computes the states between from it. A wave's sums over channels are stored for each
// token and added up afterwards in a fixed order; those over tokens stay in registers.
//
// Bound by the vector ALU: 2 x 2048 tokens, 5120 channels x 16 states, bf16, on a busy GPU 292 us of 461 in all, 20
// instructions a state and token in the walk (4 to compute a state again, 10 for its gradients, 2 for the sums over a
// channel's lanes, 4 for those over channels) and 4 around it; the vector ALU is busy nine tenths of the time at the clock it
// keeps. The first pass 127 us, the sums over channels 36, over groups 5 (the first passes after a pause: 337, 145, 36, 5).
// Eight lanes a channel with two states each (168 registers without the parts) took 530 us at the time, against 370.
// With 32 and 64 states a wave has 8 and 4 channels, and the sums over them that it stores for every token are 4 and 16 times
// as many a channel as with 16: 64 prompts of 100 tokens, 5120 channels x 64 states, 3.8 ms.
#include "selective.hpp"

namespace ssm {

namespace {

template <typename T, int S, int NS>
using GradBlock = SelBlock<T, S, NS, true, true, true>;

// The first pass over a group: of every sequence the state before each HB tokens but its first, from zero (or the
// sequence's start), with the sum of delta since the group's start where the sequence began before it; the state
// that the last sequence leaves, if it goes on behind the group; the gradient that the first sequence leaves
// at the group's start, if it began before.
template <int S, int NS, typename T>
__global__ void __launch_bounds__(64 * WAVES) selective_states_kernel(const SelectiveArgs a) {
  using SH = SelShape<S, NS>;
  using Block = SelBlock<T, S, NS, true, true, true>;
  constexpr int N = SH::N, CH = SH::CH, EC = SH::EC, EN = SH::EN;
  __shared__ __align__(16) float4 sv[WAVES][TB][CH + 1];  // delta, delta x, dL/dy
  __shared__ __align__(16) float sb[WAVES][TB][N], sc[WAVES][TB][N];
  __shared__ __align__(16) float sbias[WAVES][CH];
  const int wave = scalar(threadIdx.x >> 6), tiles = a.channels / CH;
  const int tile_blocks = (tiles + WAVES - 1) / WAVES;
  const int tile = blockIdx.x % tile_blocks * WAVES + wave;
  if (tile >= tiles) return;
  const SelTile w = sel_tile<S>(a, tile);
  const SelGroup grp = sel_group(a, blockIdx.x / tile_blocks);
  SelCell c, ahead;
  if (!next_cell(a, grp.e0, grp.e1, c)) return;
  const int began = c.starts() ? -1 : c.seq;  // the sequence that began before the group
  const int my = w.c0 + w.ch, n0 = w.sg * NS;
  const size_t at = ((size_t)grp.g * a.channels + my) * N + n0;
  float A[NS], h[NS], g[NS], p[NS], sum = 0.f;
  Vec<float, NS>::load(a.A + (size_t)my * N + n0, A);
  zero(h);
  zero(g);
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    A[i] *= kLog2e;
    p[i] = 1.f;
  }
  stage_channels(sbias[wave], a.dt_bias, w);
  wave_lds_sync();
  Block next{};
  const auto fetch = [&](const SelCell& c, int t0) {
    next.load_state(a, w, c, t0);
    if (c.seq == began) next.load_more(a, w, c, t0);
  };
  fetch(c, 0);
  for (bool more = true; more; c = ahead) {
    more = next_cell(a, c.entry + 1, grp.e1, ahead);
    const bool leaves = c.seq == began;
    if (c.starts()) {
      zero(h);
      sum = 0.f;
      if (a.state_in)
        Vec<float, NS>::load(a.state_in + (size_t)c.slot * a.channels * N + (uint32_t)(my * N + n0), h);
    }
    for (int t0 = 0; t0 < c.count; t0 += TB) {
      const Block now = next;
      const bool on = t0 + w.t < c.count;
      if (t0 + TB < c.count) fetch(c, t0 + TB);
      else if (more) fetch(ahead, 0);
      const auto keep_state = [&](int t) {
        const size_t part = (size_t)kept_place(c.first, c.pos + t0 + t) * a.channels;
        Vec<float, NS>::store(a.w.states + part * N + (uint32_t)(my * N + n0), h);
        if (leaves && w.sg == 0) a.w.until[part + my] = sum;
      };
      float x[EC], dt[EC], delta[EC], bias[EC], b[EN], dy[EC];
      now.x.unpack(x);
      now.dt.unpack(dt);
      now.b.unpack(b);
      zero(dy);
      if (leaves) {
        float z[EC], cc[EN];
        now.z.unpack(z);
        now.dy.unpack(dy);
        now.c.unpack(cc);
        apply_gate(a, z, dy);
        Vec<float, EN>::store(&sc[wave][w.t][w.q * EN], cc);
      }
      Vec<float, EC>::load(&sbias[wave][w.q * EC], bias);
#pragma unroll
      for (int i = 0; i < EC; ++i) dt[i] += bias[i];
      steps(a, dt, t0 + TB <= c.count, on, delta);
#pragma unroll
      for (int i = 0; i < EC; ++i)
        sv[wave][w.t][w.q * EC + i] = make_float4(delta[i], delta[i] * x[i], dy[i], 0.f);
      Vec<float, EN>::store(&sb[wave][w.t][w.q * EN], b);
      wave_lds_sync();
      if (c.pos + t0 > 0) keep_state(0);
      const auto tokens = [&](auto with) {
#pragma unroll
        for (int t = 0; t < TB; ++t) {
          if (t == HB && t0 + HB < c.count) keep_state(HB);
          const float4 v = sv[wave][t][w.ch];
          float bb[NS], ct[NS];
          Vec<float, NS>::load(&sb[wave][t][n0], bb);
          if constexpr (with) Vec<float, NS>::load(&sc[wave][t][n0], ct);
          sum += v.x;
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            const float decay = __builtin_amdgcn_exp2f(v.x * A[i]);
            h[i] = fmaf(decay, h[i], v.y * bb[i]);
            if constexpr (with) {
              p[i] *= decay;
              g[i] = fmaf(p[i], ct[i] * v.z, g[i]);
            }
          }
          // keeps the additions here: moved behind the block, their operands took 155 registers instead of 103
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            asm volatile("" : "+v"(h[i]));
            if constexpr (with) asm volatile("" : "+v"(g[i]));
          }
        }
      };
      if (leaves) tokens(std::true_type{});
      else tokens(std::false_type{});
      wave_lds_sync();
    }
    if (leaves && !(more && ahead.seq == began)) {
      if (c.ends() && a.dstate) {
        float l[NS];
        Vec<float, NS>::load(a.dstate + ((size_t)c.slot * a.channels + my) * N + n0, l);
#pragma unroll
        for (int i = 0; i < NS; ++i) g[i] = fmaf(p[i], l[i], g[i]);
      }
      Vec<float, NS>::store(a.w.back + at, g);
    }
    if (!more && !c.ends()) {
      Vec<float, NS>::store(a.w.local + at, h);
      if (w.sg == 0) a.w.sums[(size_t)grp.g * a.channels + my] = sum;
    }
  }
}

// What was kept of the states before a block's two parts (of the later one, if it holds a token), and the sums of
// delta until there where the sequence began before the group.
template <int N, int NS>
__device__ __forceinline__ void part_states(const SelectiveArgs& a, const SelCell& cell, int t0, int my, int n0,
                                            bool began, float (&h)[TB / HB][NS], float (&until)[TB / HB]) {
  static_assert(TB / HB == 2, "two parts");
  const uint32_t at = (uint32_t)(my * N + n0);
  const size_t step = (size_t)a.channels * N, part = (size_t)(kept_place(cell.first, cell.pos + t0) + 1);
  const float* kept = a.w.states + part * step;
  until[0] = until[1] = 0.f;
  if (began) {
    const float* u = a.w.until + part * a.channels + my;
    until[0] = *(u - a.channels);
    if (t0 + HB < cell.count) until[1] = *u;
  }
  zero(h[0]);
  zero(h[1]);
  if (t0 + HB < cell.count) Vec<float, NS>::load(kept + at, h[1]);
  if (cell.pos + t0 > 0) Vec<float, NS>::load(kept - step + at, h[0]);
  else if (a.state_in) Vec<float, NS>::load(a.state_in + (size_t)cell.slot * step + at, h[0]);
}

// Sums of v[0 .. V) over the lanes that share lane % S, by halving: every step adds two lanes' values
// and gives each half of the lanes half of the values. Afterwards v[0 .. kHalved) of a lane are
// v[halved_at ..) of all lanes. V = 2 NS values take 16 instructions instead of 48 (S = 4).
template <int S, int V>
__device__ __forceinline__ void channel_halve(float (&v)[V], int lane) {
  constexpr int V1 = V / 2, V2 = V / 4, V3 = V / 8;
#pragma unroll
  for (int i = 0; i < V1; ++i) halve32(v[i], v[i + V1]);
#pragma unroll
  for (int i = 0; i < V2; ++i) halve16(v[i], v[i + V2]);
  if constexpr (S <= 8) {
    if constexpr (V3 > 0) {
#pragma unroll
      for (int i = 0; i < V3; ++i) v[i] = halve8(v[i], v[i + V3], lane & 8);
    } else {
      v[0] += dpp<DPP_ROR8>(v[0]);
    }
  }
  if constexpr (S <= 4) v[0] += dpp<DPP_ROR4>(v[0]);
}
template <int S, int V>
__device__ __forceinline__ int halved_at(int lane) {
  return (lane & 32 ? V / 2 : 0) + (lane & 16 ? V / 4 : 0) + (S <= 8 && (lane & 8) ? V / 8 : 0);
}
template <int S, int V>
constexpr int kHalved = S == 16 ? V / 4 : V >= 8 ? V / 8 : 1;  // values a lane is left with

__device__ __forceinline__ void store3(float4* p, const float (&v)[3]) {
  *reinterpret_cast<float3*>(p) = make_float3(v[0], v[1], v[2]);
}

// A block's states are computed in two parts of HB tokens, the later first, each from the state kept before it:
// 16 tokens' states and decays would take 128 registers and leave two waves a SIMD.
template <int S, int NS, typename T>
__global__ void __launch_bounds__(64 * WAVES, 3) selective_grads_kernel(const SelectiveArgs a) {
  using SH = SelShape<S, NS>;
  constexpr int N = SH::N, CH = SH::CH, EC = SH::EC, EN = SH::EN, KEEP = (HB + S - 1) / S;
  // rows of CH + 1: one of 16 channels would start in the same bank as the last
  __shared__ __align__(16) float4 sv[WAVES][TB][CH + 1];  // delta, delta x, dL/dy, x
  __shared__ __align__(16) float4 so[WAVES][TB][CH + 1];  // sum G B, sum G a h A / ln 2, y, d delta / d dt
  __shared__ __align__(16) float sb[WAVES][TB][N], sc[WAVES][TB][N];
  __shared__ __align__(16) float sz[WAVES][TB][CH];       // dL/dout times the gate's derivative
  __shared__ __align__(16) float sbias[WAVES][CH], sskip[WAVES][CH];
  const int wave = scalar(threadIdx.x >> 6), tiles = a.channels / CH;
  const int tile_blocks = (tiles + WAVES - 1) / WAVES;
  const int tile = blockIdx.x % tile_blocks * WAVES + wave;
  if (tile >= tiles) return;
  const SelTile w = sel_tile<S>(a, tile);
  const SelGroup grp = sel_group(a, blockIdx.x / tile_blocks);
  const int my = w.c0 + w.ch, n0 = w.sg * NS;
  float A2[NS], dA[NS], dD[EC], dbias[EC];
  Vec<float, NS>::load(a.A + (size_t)my * N + n0, A2);
  zero(dA);
  zero(dD);
  zero(dbias);
#pragma unroll
  for (int i = 0; i < NS; ++i) A2[i] *= kLog2e;
  stage_channels(sbias[wave], a.dt_bias, w);
  stage_channels(sskip[wave], a.D, w);
  wave_lds_sync();
  if (a.dstate_in)
    for_empty_sequences(a, grp, [&](int, int slot) {
      const size_t at = ((size_t)slot * a.channels + my) * N + n0;
      float v[NS];
      zero(v);
      if (a.dstate) Vec<float, NS>::load(a.dstate + at, v);
      Vec<float, NS>::store(a.dstate_in + at, v);
    });
  // the lane's place among dB and dC of a token and tile: its values are dB of its NS states, then dC
  const int kept = halved_at<S, 2 * NS>(w.lane);
  const uint32_t dbc_at = 4 * (uint32_t)((kept < NS ? 0 : N - NS) + n0 + kept);
  const uint32_t dbc_pitch = (uint32_t)tiles * (8 * N);  // bytes from token to token: tiles < 2^18
  char* const dbc_tile = reinterpret_cast<char*>(a.w.dbc) + (uint32_t)tile * (8 * N);
  char* const dbc_none = dbc_tile + (uint64_t)(uint32_t)a.plan.total * dbc_pitch;
  // the state that the group's first sequence had before the group
  __shared__ __align__(16) float sh[WAVES][64][NS];
  SelCell cell, ahead;
  int began = -1;
  if (next_cell(a, grp.e0, grp.e1, cell) && !cell.starts()) {
    float h[NS];
    carry_in<N>(a, grp, cell, my, n0, A2, h);
    Vec<float, NS>::store(sh[wave][w.lane], h);
    began = cell.seq;
  }
  bool more = prev_cell(a, grp.e1 - 1, grp.e0 - 1, cell);
  float g[NS];
  zero(g);
  GradBlock<T, S, NS> next;
  if (more) {
    if (!cell.ends()) carry_back<N>(a, grp, cell, my, n0, A2, g);
    next.load(a, w, cell, (cell.count - 1) / TB * TB);
  }
  for (; more; cell = ahead) {
    more = prev_cell(a, cell.entry - 1, grp.e0 - 1, ahead);
    const size_t at = (size_t)cell.slot * a.channels * N + (uint32_t)(my * N + n0);
    if (cell.ends()) {
      zero(g);
      if (a.dstate) Vec<float, NS>::load(a.dstate + at, g);
    }
    for (int t0 = (cell.count - 1) / TB * TB; t0 >= 0; t0 -= TB) {
      const GradBlock<T, S, NS> now = next;
      float h[TB / HB][NS], until[TB / HB];
      part_states<N>(a, cell, t0, my, n0, cell.seq == began, h, until);
      if (t0 > 0) next.load(a, w, cell, t0 - TB);
      else if (more) next.load(a, w, ahead, (ahead.count - 1) / TB * TB);
      const bool on = t0 + w.t < cell.count;
      const int tok0 = cell.first + cell.pos + t0;
      {
        float x[EC], raw[EC], delta[EC], bias[EC], z[EC], dy[EC], b[EN], c[EN];
        now.x.unpack(x);
        now.dt.unpack(raw);
        now.z.unpack(z);
        now.dy.unpack(dy);
        now.b.unpack(b);
        now.c.unpack(c);
        Vec<float, EC>::load(&sbias[wave][w.q * EC], bias);
#pragma unroll
        for (int i = 0; i < EC; ++i) raw[i] += bias[i];
        steps(a, raw, t0 + TB <= cell.count, on, delta);
        if (a.gated) {
          float dz[EC];
#pragma unroll
          for (int i = 0; i < EC; ++i) {
            const float s = sigmoid(z[i]);
            dz[i] = dy[i] * (s * fmaf(z[i], 1.f - s, 1.f));
            dy[i] *= z[i] * s;
          }
          Vec<float, EC>::store(&sz[wave][w.t][w.q * EC], dz);
        }
#pragma unroll
        for (int i = 0; i < EC; ++i) {
          sv[wave][w.t][w.q * EC + i] = make_float4(delta[i], delta[i] * x[i], dy[i], x[i]);
          so[wave][w.t][w.q * EC + i].w = a.softplus ? sigmoid(raw[i]) : 1.f;
        }
        Vec<float, EN>::store(&sb[wave][w.t][w.q * EN], b);
        Vec<float, EN>::store(&sc[wave][w.t][w.q * EN], c);
      }
      wave_lds_sync();
      char* const dbc = dbc_tile + (uint64_t)(uint32_t)tok0 * dbc_pitch;
#pragma unroll
      for (int part = TB / HB - 1; part >= 0; --part) {
        float keep[KEEP][3];  // lane sg keeps the tokens that are sg modulo S
        float hs[HB + 1][NS], d[HB][NS];  // states before each token and after the last, decays
#pragma unroll
        for (int i = 0; i < NS; ++i) hs[0][i] = h[part][i];
        if (cell.seq == began) {
          float h0[NS];
          Vec<float, NS>::load(sh[wave][w.lane], h0);
#pragma unroll
          for (int i = 0; i < NS; ++i)
            hs[0][i] = fmaf(__builtin_amdgcn_exp2f(A2[i] * until[part]), h0[i], hs[0][i]);
        }
#pragma unroll
        for (int t = 0; t < HB; ++t) {
          const float2 v = *reinterpret_cast<const float2*>(&sv[wave][part * HB + t][w.ch]);
          float bb[NS];
          Vec<float, NS>::load(&sb[wave][part * HB + t][n0], bb);
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            d[t][i] = __builtin_amdgcn_exp2f(v.x * A2[i]);
            hs[t + 1][i] = fmaf(d[t][i], hs[t][i], v.y * bb[i]);
          }
        }
#pragma unroll
        for (int t = HB - 1; t >= 0; --t) {
          const int tb = part * HB + t;
          const float4 v = sv[wave][tb][w.ch];
          float bb[NS], cc[NS], sums[2 * NS];
          Vec<float, NS>::load(&sb[wave][tb][n0], bb);
          Vec<float, NS>::load(&sc[wave][tb][n0], cc);
          float e = 0.f, f = 0.f, y = 0.f;
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            g[i] = fmaf(cc[i], v.z, g[i]);
            sums[i] = v.y * g[i];
            sums[NS + i] = v.z * hs[t + 1][i];
            y = fmaf(cc[i], hs[t + 1][i], y);
            e = fmaf(bb[i], g[i], e);
            g[i] *= d[t][i];
            const float p = g[i] * hs[t][i];
            dA[i] = fmaf(v.x, p, dA[i]);
            f = fmaf(A2[i], p, f);
          }
          // dA is not used before the walk's end, so the compiler would add to it behind the whole block and keep
          // its 16 tokens' products in registers until then (241 instead of 164)
#pragma unroll
          for (int i = 0; i < NS; ++i) asm volatile("" : "+v"(dA[i]));
          e = state_sum<S>(e);
          f = state_sum<S>(f);
          y = state_sum<S>(y);
          float(&k)[3] = keep[t / S];
          const bool mine = w.sg == t % S;
          const bool first = t == HB - 1 || t % S == S - 1;  // of the tokens that share the registers
          k[0] = first || mine ? e : k[0];
          k[1] = first || mine ? f : k[1];
          k[2] = first || mine ? y : k[2];
          // each sum is stored as it is made, by every lane that has it; rows without a token (whose sums are
          // zero) go to a row behind the last
          channel_halve<S>(sums, w.lane);
          char* row = t0 + tb < cell.count ? dbc + (uint32_t)tb * dbc_pitch : dbc_none;
#pragma unroll
          for (int i = 0; i < kHalved<S, 2 * NS>; ++i)
            *reinterpret_cast<float*>(row + (dbc_at + 4 * (uint32_t)i)) = sums[i];
        }
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
          if (S <= HB || w.sg < HB)
            store3(&so[wave][part * HB + i * S + w.sg][w.ch], keep[i]);
        wave_lds_sync();
      }
      if (on) {
        float dx[EC], ddt[EC], skip[EC];
        Vec<float, EC>::load(&sskip[wave][w.q * EC], skip);
        const int c0 = w.c0 + w.q * EC;
        float ypre[EC];
#pragma unroll
        for (int i = 0; i < EC; ++i) {
          const float4 v = sv[wave][w.t][w.q * EC + i], o = so[wave][w.t][w.q * EC + i];
          dx[i] = fmaf(v.x, o.x, skip[i] * v.z);
          ddt[i] = fmaf(v.w, o.x, kLn2 * o.y) * o.w;
          dbias[i] += ddt[i];
          dD[i] = fmaf(v.z, v.w, dD[i]);
          ypre[i] = fmaf(skip[i], v.w, o.z);
        }
        if (a.gated) {
          float dz[EC];
          Vec<float, EC>::load(&sz[wave][w.t][w.q * EC], dz);
#pragma unroll
          for (int i = 0; i < EC; ++i) dz[i] *= ypre[i];
          store_row<T, EC>(row_at<T>(a.dz, tok0, w.t, c0), dz);
        }
        store_row<T, EC>(row_at<T>(a.dx, tok0, w.t, c0), dx);
        store_row<T, EC>(row_at<T>(a.ddt, tok0, w.t, c0), ddt);
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
    dD[i] = token_sum(dD[i]);  // over the 16 tokens of a block: lanes with the same quarter
    dbias[i] = token_sum(dbias[i]);
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
  const SelGroups g = selective_groups(d, a.plan.cap);
  a.time_groups = g.groups;
  a.group_chunks = g.chunks;
  hipError_t e = over_groups(d, a, [&](auto S, auto NS, auto T, dim3 grid) {
    constexpr int s = decltype(S)::value, ns = decltype(NS)::value;
    using TI = typename decltype(T)::type;
    hipLaunchKernelGGL((selective_states_kernel<s, ns, TI>), grid, dim3(64 * WAVES), 0, stream, a);
    hipLaunchKernelGGL((selective_grads_kernel<s, ns, TI>), grid, dim3(64 * WAVES), 0, stream, a);
  });
  if (e != hipSuccess) return e;
  return selective_dispatch(d, [&](auto S, auto NS, auto T) {
    constexpr int s = decltype(S)::value, ns = decltype(NS)::value;
    using TI = typename decltype(T)::type;
    const int tiles = selective_tiles(d);
    hipError_t e = hipSuccess;
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
