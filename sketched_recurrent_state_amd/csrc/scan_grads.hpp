// scan_grads.hpp -- the gradients of q, k, the gates and beta of one chunk (64 tokens) of
// one head, all chunks at once, from the state S at the chunk's start, its gradient G at the
// chunk's end, and every token's r and e (notation in scan.hpp).
//
// The blocks of a chunk meet through decays across whole blocks: with F_a the decay of the
// blocks before block a and B_b that of the blocks after block b,
//   dq_a        = F_a I_a (dy_a S) + sum_{b <= a} (dP_ab G_ab) k_b
//   dk_a reader = -F_a I_a (dr_a S) + sum_{b <= a} (dK_ab G_ab) k_b
//   dk_b writer = B_b O_b (w_b G) + sum_{a >= b} (dP_ab G_ab)^T q_a + (dK_ab G_ab)^T k_a
// so S and G are read and split once a chunk and never carried from block to block. A scalar
// gate's G_ab goes into dP and dK. KDA's, one for each channel, goes into the keys and queries:
// a product over the gates between two tokens is taken in two factors that meet at the boundary
// between their blocks, halves of a block or runs of four tokens, and term by term within a run,
// so that all but the last are matrix products (2 x 4096 tokens x 32 heads of 128 x 128, bf16:
// 2,412 -> 564 us against the whole 16-token diagonal term by term). And
//   rowsum(S_end * G) = F rowsum(S * G) + sum_j k_j (state part of the writer's dk_j)
// starts the sums of the gates' gradients without the state at the chunk's end. What passes a
// gate is so the difference of sums over the chunk's tokens: its rounding is relative to their
// terms, not to itself, and it is written as 0 where the gate is exactly 0.
//
// A wave owns 16 or 32 key channels, so the contractions over d_v stay in its
// registers; dy, e and r pass through LDS 32 values of d_v at a time, split there once for all
// waves. The 20 tiles of dP and dK are dealt over the waves.
//
// A GDN cell of 128 x 128 reads 128 KB of S and G, 96 KB of dy, r and e and 32 KB of keys and
// queries and writes 33 KB: 0.6 GB for the 2,048 cells of 4096 tokens x 32 heads, in 266 us. Its
// eight waves fill a CU's registers: vector ALU 99 us, matrix cores 52 us, and half of every wave's
// time waiting at barriers and for memory. (S and G fetched a step ahead: within 1 %; rows of LDS
// without padding: the same.)
#pragma once

#include "scan.hpp"

namespace ssm {

// The value of x summed over the lanes above this one of the four that differ in bits 4 and 5,
// and over all four.
__device__ __forceinline__ void above(float x, int lane, int g, float& after, float& total) {
  after = total = 0.f;
#pragma unroll
  for (int o = 0; o < 4; ++o) {
    const float y = __shfl(x, (lane & 15) + 16 * o);
    total += y;
    if (o > g) after += y;
  }
}

struct Split8 {  // eight values, the operand of a 32-deep product
  uint4 h, m, l;
};
__device__ __forceinline__ Split8 split8(f32x4 x, f32x4 y) {
  const Split4 a = split4(x), b = split4(y);
  return Split8{make_uint4(a.h.x, a.h.y, b.h.x, b.h.y), make_uint4(a.m.x, a.m.y, b.m.x, b.m.y),
                make_uint4(a.l.x, a.l.y, b.l.x, b.l.y)};
}
// c + a b, of which a has PA parts and b PB (1: exact values)
template <int PA, int PB>
__device__ __forceinline__ f32x4 mfma_parts(const Split8& a, const Split8& b, f32x4 c) {
  if constexpr (PA == 3) c = mfma32(a.l, b.h, c);
  if constexpr (PB == 3) c = mfma32(a.h, b.l, c);
  if constexpr (PA == 3 && PB == 3) c = mfma32(a.m, b.m, c);
  if constexpr (PA == 3) c = mfma32(a.m, b.h, c);
  if constexpr (PB == 3) c = mfma32(a.h, b.m, c);
  return mfma32(a.h, b.h, c);
}

// Channel tiles of a wave: two with Mamba-2's two products; the delta rules' three leave no
// registers for a second tile (GDN, 2,048 cells of 128 x 128: two 301 us, 367 us held to half the registers, one 269 us).
template <int RULE, int DK>
constexpr int kGradTiles = RULE == MAMBA2 && DK >= 32 ? 2 : 1;
template <int RULE, int DK>
constexpr int kGradThreads = 64 * (DK / 16 / kGradTiles<RULE, DK>);

template <int RULE, int DK, int DV, typename TIN>
__global__ void __launch_bounds__((kGradThreads<RULE, DK>),
                                  (DK == 128 || (RULE == MAMBA2 && DK == 64) ? 2 : 1))
scan_grads_kernel(const ScanArgs a) {
  constexpr bool DELTA = RULE != MAMBA2, CH = RULE == KDA, BF = sizeof(TIN) == 2;
  constexpr bool EXACT = BF && !CH;                  // keys and queries
  constexpr int RP = !DELTA && BF ? 1 : 3;           // parts of w / r (Mamba-2: the values)
  constexpr int TD = kGradTiles<RULE, DK>, NT = kGradThreads<RULE, DK>, W = NT / 64;
  constexpr int NS = DV >= 32 ? DV / 32 : 1;         // steps of 32 values of d_v
  constexpr int PAIRS = NB * (NB + 1) / 2, TILES = DELTA ? 2 * PAIRS : PAIRS;
  constexpr int TW = (TILES + W - 1) / W;            // dP and dK tiles of a wave
  constexpr int RS = 80, PART = CT * RS;             // row of 32 bf16 and its padding, a part
  constexpr int NY = 0, NR = 3 * PART, NE = NR + RP * PART;  // dy, r, e in LDS
  constexpr int ROWS = NE + (DELTA ? 3 : 0) * PART;
  // afterwards, in the same memory: the tiles in three parts, row-major 16 x 16 bf16, and for
  // KDA the diagonal ones in fp32
  constexpr int MAT = 3 * 512, LP = 20, DIAG = TILES * MAT;
  static_assert(DIAG + (CH ? 2 * NB * SB * LP * 4 : 0) <= ROWS, "the tiles fit");
  __shared__ __align__(16) char rows[ROWS];
  __shared__ float sx[W][CT], send[W];
  const int h = blockIdx.x % a.heads, chunk = blockIdx.x / a.heads;
  const size_t cell = a.cell(chunk, h);
  int tok, count;
  if (!a.plan.cell(chunk, tok, count)) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63, m = lane & 15, g = lane >> 4;
  const int d0 = wave * 16 * TD + m;  // channel of tile u: d0 + 16 u
  const int nb = (count + SB - 1) / SB;
  const size_t H = a.heads;
  const TIN* q = static_cast<const TIN*>(a.q);
  const TIN* k = static_cast<const TIN*>(a.k);
  const TIN* v = static_cast<const TIN*>(a.v);
  const float* row = a.w.row + cell * NB * ROW;  // block x: + ROW * x
  const size_t base = (size_t)tok * H + h;  // token i: base + i * H

  // ---- products with S and G, and dP and dK, over d_v
  constexpr int PIECES = CT * (DV >= 32 ? 8 : 4);    // of four values, a step and an array
  constexpr int NP = (PIECES + NT - 1) / NT, PR = PIECES / CT;
  struct Stage {
    f32x4 y[NP], r[NP], e[DELTA ? NP : 1];
  };
  auto fetch = [&](Stage& s, int step) {
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const int i = min(tid + n * NT, PIECES - 1), t = i / PR, c = 32 * step + i % PR * 4;
      const size_t at = (base + (size_t)min(t, count - 1) * H) * DV + c;
      const size_t wr = (cell * CT + min(t, count - 1)) * DV + c;
      s.y[n] = *reinterpret_cast<const f32x4*>(a.dy + at);
      if constexpr (DELTA) {
        s.r[n] = *reinterpret_cast<const f32x4*>(a.w.r + wr);
        s.e[n] = *reinterpret_cast<const f32x4*>(a.w.e + wr);
      } else {
        Quad<TIN> x;
        x.load(v + at);
#pragma unroll
        for (int j = 0; j < 4; ++j) s.r[n][j] = x[j];
      }
    }
  };
  float db[DELTA ? NP : 1] = {};
  auto put = [&](const Stage& s) {
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const int i = tid + n * NT, t = i / PR;
      if (PIECES % NT != 0 && i >= PIECES) break;
      char* to = rows + t * RS + i % PR * 8;
      const uint32_t ok = row_mask(t < count);  // tokens behind the end: zero
      auto one = [&](f32x4 x, int at, int parts) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = masked(x[j], ok);
        const Split4 p = split4(x);
        *reinterpret_cast<uint2*>(to + at) = p.h;
        if (parts == 3) {
          *reinterpret_cast<uint2*>(to + at + PART) = p.m;
          *reinterpret_cast<uint2*>(to + at + 2 * PART) = p.l;
        }
      };
      one(s.y[n], NY, 3);
      one(s.r[n], NR, RP);
      if constexpr (DELTA) {
        one(s.e[n], NE, 3);
#pragma unroll
        for (int j = 0; j < 4; ++j) db[n] += s.e[n][j] * s.r[n][j];
      }
    }
  };
  auto operand = [&](int at, int parts, int blk) {  // lane (m, g): token 16 blk + m, values 8g ..
    const char* p = rows + at + (SB * blk + m) * RS + 16 * g;
    Split8 s;
    s.h = *reinterpret_cast<const uint4*>(p);
    if (parts == 3) {
      s.m = *reinterpret_cast<const uint4*>(p + PART);
      s.l = *reinterpret_cast<const uint4*>(p + 2 * PART);
    }
    return s;
  };

  f32x4 dq[NB][TD] = {}, dkr[DELTA ? NB : 1][TD] = {}, dkw[NB][TD] = {}, tile[TW] = {};
  float end[TD] = {};  // rowsum(S * G)
  const float* S0 = a.w.S + cell * DK * DV;
  const float* G0 = a.w.G + cell * DK * DV;
  if constexpr (DV < 32) {  // the upper half of the only step
    for (int i = tid; i < ROWS / 4; i += NT) reinterpret_cast<uint32_t*>(rows)[i] = 0;
  }
  Stage st;
  fetch(st, 0);
#pragma unroll 1
  for (int step = 0; step < NS; ++step) {
    __syncthreads();  // the step before has been read
    put(st);
    fetch(st, min(step + 1, NS - 1));
    Split8 S[TD], G[TD];
#pragma unroll
    for (int u = 0; u < TD; ++u) {
      const size_t at = (size_t)(d0 + 16 * u) * DV + 32 * step + (DV >= 32 ? 8 * g : 8 * (g & 1));
      f32x4 s0 = *reinterpret_cast<const f32x4*>(S0 + at), s1 = *reinterpret_cast<const f32x4*>(S0 + at + 4);
      f32x4 g0 = *reinterpret_cast<const f32x4*>(G0 + at), g1 = *reinterpret_cast<const f32x4*>(G0 + at + 4);
      if constexpr (DV < 32) {
        if (g >= 2) s0 = s1 = g0 = g1 = f32x4{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) end[u] += s0[i] * g0[i] + s1[i] * g1[i];
      S[u] = split8(s0, s1);
      G[u] = split8(g0, g1);
    }
    __syncthreads();
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      if (blk >= nb) break;
      const Split8 y = operand(NY, 3, blk), r = operand(NR, RP, blk);
#pragma unroll
      for (int u = 0; u < TD; ++u) {
        dq[blk][u] = mfma_parts<3, 3>(y, S[u], dq[blk][u]);
        dkw[blk][u] = mfma_parts<RP, 3>(r, G[u], dkw[blk][u]);
      }
      if constexpr (DELTA) {
        const Split8 e = operand(NE, 3, blk);
#pragma unroll
        for (int u = 0; u < TD; ++u) dkr[blk][u] = mfma_parts<3, 3>(e, S[u], dkr[blk][u]);
      }
    }
    // dP_ab and dK_ab transposed (rows: block b's tokens), so that a lane holds four columns
    // of a row of the tile itself
    int pair = 0;
#pragma unroll
    for (int x = 0; x < NB; ++x)
#pragma unroll
      for (int y = 0; y <= x; ++y, ++pair)
#pragma unroll
        for (int kind = 0; kind < (DELTA ? 2 : 1); ++kind) {
          const int n = pair + kind * PAIRS;
          if (n % W == wave && x < nb)
            tile[n / W] = mfma_parts<RP, 3>(operand(NR, RP, y), operand(kind ? NE : NY, 3, x), tile[n / W]);
        }
  }
  if constexpr (DELTA) {
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const int t = (tid + n * NT) / PR;
      float s = db[n] + dpp<DPP_QUAD_1032>(db[n]);
      s += dpp<DPP_QUAD_2301>(s);
      if constexpr (PR == 8) s += xor4(s);
      if ((PIECES % NT == 0 || tid + n * NT < PIECES) && tid % PR == 0 && t < count)
        a.dbeta[base + (size_t)t * H] = s;
    }
  }

  // ---- dP and dK: the triangles, beta, and a scalar gate's decay
  __syncthreads();
  float whole[NB];  // scalar gates: a block's decay
#pragma unroll
  for (int c = 0; c < NB; ++c) whole[c] = !CH && c < nb ? row[ROW * c + SB - 1] : 1.f;
  {
    int pair = 0;
#pragma unroll
    for (int x = 0; x < NB; ++x)
#pragma unroll
      for (int y = 0; y <= x; ++y, ++pair) {
        float between = 1.f;
#pragma unroll
        for (int c = y + 1; c < x; ++c) between *= whole[c];
#pragma unroll
        for (int kind = 0; kind < (DELTA ? 2 : 1); ++kind) {
          const int n = pair + kind * PAIRS;
          if (n % W != wave || x >= nb) continue;
          // lane (m, g): row (reader) m of block x, columns (writers) 4g + i of block y
          f32x4 t = tile[n / W];
          if constexpr (DELTA) {
            t *= *reinterpret_cast<const f32x4*>(row + ROW * y + 2 * SB + 4 * g);
            if (kind) t *= -row[ROW * x + 2 * SB + m];
          }
          if constexpr (!CH) {
            if (x != y) {
              t *= *reinterpret_cast<const f32x4*>(row + ROW * y + SB + 4 * g);
              t *= row[ROW * x + m] * between;
            } else {
              const float gate = SB * x + m < count ? a.decay[base + (size_t)(SB * x + m) * H] : 1.f;
              float ratio[4] = {1.f, 1.f, 1.f, 1.f};
#pragma unroll
              for (int l = 1; l < SB; ++l) {
                const float al = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(gate), l));
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (l > 4 * g + i && l <= m) ratio[i] *= al;
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) t[i] *= ratio[i];
            }
          }
          if (x == y) {
#pragma unroll
            for (int i = 0; i < 4; ++i) t[i] = 4 * g + i + kind <= m ? t[i] : 0.f;
            if constexpr (CH)
              *reinterpret_cast<f32x4*>(rows + DIAG + ((kind * NB + x) * SB + m) * LP * 4 + 16 * g) = t;
          }
          const Split4 p = split4(t);
          char* to = rows + n * MAT + m * 32 + g * 8;
          *reinterpret_cast<uint2*>(to) = p.h;
          *reinterpret_cast<uint2*>(to + 512) = p.m;
          *reinterpret_cast<uint2*>(to + 1024) = p.l;
        }
      }
  }
  __syncthreads();
  auto tile_rows = [&](int n) {  // lane (m, g): row m, columns 4g ..
    const char* p = rows + n * MAT + m * 32 + g * 8;
    return Split4{*reinterpret_cast<const uint2*>(p), *reinterpret_cast<const uint2*>(p + 512),
                  *reinterpret_cast<const uint2*>(p + 1024)};
  };
  auto tile_cols = [&](int n) {  // lane (m, g): column m, rows 4g ..
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const char* p = rows + n * MAT + (4 * g + (m >> 2)) * 32 + (m & 3) * 8;
    Split4 s;
    s.h = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
    s.m = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 512)));
    s.l = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 1024)));
    return s;
  };

  // ---- a block's keys and queries: rows 4g + i of channel d0 + 16 u
  auto load_rows = [&](const TIN* p, int blk, int u) {
    f32x4 x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = SB * blk + 4 * g + i;
      x[i] = to_f32(masked(p[(base + (size_t)min(t, count - 1) * H) * DK + d0 + 16 * u],
                           row_mask(t < count)));
    }
    return x;
  };
  // c + a x, x the rows of a block (exact or not)
  auto times = [&](const Split4& t, f32x4 x, f32x4 c) {
    if constexpr (EXACT) {
      const uint2 e = make_uint2(heads(x[0], x[1]), heads(x[2], x[3])), none = make_uint2(0u, 0u);
      c = mfma_two(t.l, e, none, none, c);
      return mfma_two(t.h, e, t.m, e, c);
    } else {
      return mfma_split(t, split4(x), c);
    }
  };
  auto store = [&](void* p, int blk, int u, f32x4 x) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (SB * blk + 4 * g + i < count)
        ssm::put(static_cast<TIN*>(p) + (base + (size_t)(SB * blk + 4 * g + i) * H) * DK + d0 + 16 * u, x[i]);
  };

  if constexpr (!CH) {
    f32x4 kx[NB][TD], qx[NB][TD];
    float all = 1.f, before = 1.f;
#pragma unroll
    for (int c = 0; c < NB; ++c) all *= whole[c];
#pragma unroll
    for (int u = 0; u < TD; ++u) end[u] *= all;
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      if (blk >= nb) break;
      float after = 1.f;
#pragma unroll
      for (int c = blk + 1; c < NB; ++c) after *= whole[c];
      const f32x4 in = *reinterpret_cast<const f32x4*>(row + ROW * blk + 4 * g) * before;
      f32x4 out = *reinterpret_cast<const f32x4*>(row + ROW * blk + SB + 4 * g) * after, beta;
      if constexpr (DELTA) {
        beta = *reinterpret_cast<const f32x4*>(row + ROW * blk + 2 * SB + 4 * g);
        out *= beta;
      }
#pragma unroll
      for (int u = 0; u < TD; ++u) {
        kx[blk][u] = load_rows(k, blk, u);
        qx[blk][u] = load_rows(q, blk, u);
        dq[blk][u] *= in;
        if constexpr (DELTA) dkr[blk][u] *= -in * beta;
        dkw[blk][u] *= out;
#pragma unroll
        for (int i = 0; i < 4; ++i) end[u] += kx[blk][u][i] * dkw[blk][u][i];
      }
      before *= whole[blk];
    }
    int pair = 0;
#pragma unroll
    for (int x = 0; x < NB; ++x)
#pragma unroll
      for (int y = 0; y <= x; ++y, ++pair) {
        if (x >= nb) continue;
        const Split4 P = tile_rows(pair), Pt = tile_cols(pair);
#pragma unroll
        for (int u = 0; u < TD; ++u) {
          dq[x][u] = times(P, kx[y][u], dq[x][u]);
          dkw[y][u] = times(Pt, qx[x][u], dkw[y][u]);
        }
        if constexpr (DELTA) {
          const Split4 K = tile_rows(PAIRS + pair), Kt = tile_cols(PAIRS + pair);
#pragma unroll
          for (int u = 0; u < TD; ++u) {
            dkr[x][u] = times(K, kx[y][u], dkr[x][u]);
            dkw[y][u] = times(Kt, kx[x][u], dkw[y][u]);
          }
        }
      }
    float e = 0.f;
#pragma unroll
    for (int u = 0; u < TD; ++u) e += end[u];
    e = row_allreduce(xsum32(xsum16(e)));
    if (lane == 0) send[wave] = e;
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      if (blk >= nb) break;
      f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < TD; ++u) {
        f32x4 dk = dkw[blk][u];
        s += qx[blk][u] * dq[blk][u] - kx[blk][u] * dkw[blk][u];
        if constexpr (DELTA) {
          s += kx[blk][u] * dkr[blk][u];
          dk += dkr[blk][u];
        }
        store(a.dq, blk, u, dq[blk][u]);
        store(a.dk, blk, u, dk);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float t = row_allreduce(s[i]);
        if (m == 0) sx[wave][SB * blk + 4 * g + i] = t;
      }
    }
    __syncthreads();
    if (wave == 0) {  // suffix sums over the chunk's tokens, lane = token
      float s = 0.f, last = 0.f;
      for (int w = 0; w < W; ++w) {
        s += lane < SB * nb ? sx[w][lane] : 0.f;
        last += send[w];
      }
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const float t = __shfl_down(s, o);
        if (lane + o < 64) s += t;
      }
      if (lane < count) {  // a gate of 0 lets nothing through: what the sums leave is rounding
        const size_t t = base + (size_t)lane * H;
        a.dlog[t] = a.decay[t] == 0.f ? 0.f : last + s;
      }
    }
  } else {
    static_assert(!CH || TD == 1, "a channel tile a wave");
    const float* diagP = reinterpret_cast<const float*>(rows + DIAG);
    const float* diagK = diagP + NB * SB * LP;
    // Rows 4g + i of every block, and their gates in runs of four tokens: the run's decay into
    // token i (in4) and out of it (out4), of runs 1 and 2 (w1, w2), and of the runs before and
    // after this lane's.
    f32x4 kx[NB], qx[NB], ax[NB], in4[NB], out4[NB];
    float w1[NB], w2[NB], pre[NB], post[NB], blocks[NB];
#pragma unroll
    for (int x = 0; x < NB; ++x) {
      kx[x] = load_rows(k, x, 0);
      qx[x] = load_rows(q, x, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = SB * x + 4 * g + i;
        const float gate = a.decay[(base + (size_t)min(t, count - 1) * H) * DK + d0];
        ax[x][i] = t < count ? gate : 1.f;
      }
    }
#pragma unroll
    for (int x = 0; x < NB; ++x) {
      in4[x][0] = ax[x][0];
      out4[x][3] = 1.f;
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        in4[x][i] = in4[x][i - 1] * ax[x][i];
        out4[x][3 - i] = out4[x][4 - i] * ax[x][4 - i];
      }
      const float w = in4[x][3], w0 = __shfl(w, m), w3 = __shfl(w, m + 48);
      w1[x] = __shfl(w, m + 16);
      w2[x] = __shfl(w, m + 32);
      pre[x] = (g > 0 ? w0 : 1.f) * (g > 1 ? w1[x] : 1.f) * (g > 2 ? w2[x] : 1.f);
      post[x] = (g < 3 ? w3 : 1.f) * (g < 2 ? w2[x] : 1.f) * (g < 1 ? w1[x] : 1.f);
      blocks[x] = w0 * w1[x] * w2[x] * w3;
    }
    float after = 1.f;
#pragma unroll
    for (int x = 0; x < NB; ++x) end[0] *= blocks[x];
#pragma unroll
    for (int x = NB - 1; x >= 0; --x) {  // end: rowsum(S_end * G), the last token's sum
      if (x < nb) {
        const f32x4 beta = *reinterpret_cast<const f32x4*>(row + ROW * x + 2 * SB + 4 * g);
        dkr[x][0] *= -beta;
        dkw[x][0] *= beta;
        const f32x4 out = out4[x] * (post[x] * after);
#pragma unroll
        for (int i = 0; i < 4; ++i) end[0] += dkw[x][0][i] * out[i] * kx[x][i];
      }
      after *= blocks[x];
    }
    // across blocks, from the ends of the writers' blocks to the starts of the readers'
#pragma unroll
    for (int y = 0; y < NB - 1; ++y) {
      const Split4 t = split4(kx[y] * (out4[y] * post[y]));
#pragma unroll
      for (int x = y + 1; x < NB; ++x) {
        if (x >= nb) continue;
        dq[x][0] = mfma_split(tile_rows(x * (x + 1) / 2 + y), t, dq[x][0] * blocks[y]);
        dkr[x][0] = mfma_split(tile_rows(PAIRS + x * (x + 1) / 2 + y), t, dkr[x][0] * blocks[y]);
      }
    }
#pragma unroll
    for (int x = NB - 1; x > 0; --x) {
      if (x >= nb) continue;
      const f32x4 in = in4[x] * pre[x];
      const Split4 tq = split4(qx[x] * in), tk = split4(kx[x] * in);
#pragma unroll
      for (int y = 0; y < x; ++y) {
        dkw[y][0] = mfma_split(tile_cols(x * (x + 1) / 2 + y), tq, dkw[y][0] * blocks[x]);
        dkw[y][0] = mfma_split(tile_cols(PAIRS + x * (x + 1) / 2 + y), tk, dkw[y][0]);
      }
    }
    // within a block, from the last block to the first: between its halves, between the runs of
    // a half (tiles with all else masked), and within the lane's run term by term
    const int run = m >> 2;
    const uint32_t half = row_mask(run >= 2 && g < 2), runs = row_mask((run & 1) && g == run - 1);
    const uint32_t halfT = row_mask(run < 2 && g >= 2), runsT = row_mask(!(run & 1) && g == run + 1);
    auto only = [](const Split4& t, uint32_t mask) {
      return Split4{make_uint2(t.h.x & mask, t.h.y & mask), make_uint2(t.m.x & mask, t.m.y & mask),
                    make_uint2(t.l.x & mask, t.l.y & mask)};
    };
    const f32x4 none = {0.f, 0.f, 0.f, 0.f};
    float carry = xsum32(xsum16(end[0]));
#pragma unroll
    for (int x = NB - 1; x >= 0; --x) {
      if (x >= nb) continue;
      const int n = x * (x + 1) / 2 + x;
      const float far1 = g == 0 ? w1[x] : 1.f, far2 = g == 3 ? w2[x] : 1.f;
      const f32x4 kw = kx[x] * out4[x], qr = qx[x] * in4[x], kr = kx[x] * in4[x];
      const Split4 kw4 = split4(kw), kw8 = split4(kw * far1);
      const Split4 qr4 = split4(qr), qr8 = split4(qr * far2);
      const Split4 kr4 = split4(kr), kr8 = split4(kr * far2);
      const Split4 P = tile_rows(n), K = tile_rows(PAIRS + n), Pt = tile_cols(n), Kt = tile_cols(PAIRS + n);
      f32x4 xq = dq[x][0] * pre[x], xr = dkr[x][0] * pre[x], xw = dkw[x][0] * post[x];
      xq += mfma_split(only(P, runs), kw4, mfma_split(only(P, half), kw8, none) * far2);
      xr += mfma_split(only(K, runs), kw4, mfma_split(only(K, half), kw8, none) * far2);
      const f32x4 w = mfma_split(only(Kt, halfT), kr8, mfma_split(only(Pt, halfT), qr8, none)) * far1;
      xw += mfma_split(only(Kt, runsT), kr4, mfma_split(only(Pt, runsT), qr4, w));
      xq *= in4[x];
      xr *= in4[x];
      xw *= out4[x];
      f32x4 dP[4], dK[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dP[i] = *reinterpret_cast<const f32x4*>(diagP + (x * SB + 4 * g + i) * LP + 4 * g);
        dK[i] = *reinterpret_cast<const f32x4*>(diagK + (x * SB + 4 * g + i) * LP + 4 * g);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float p = 1.f;
#pragma unroll
        for (int i = j; i < 4; ++i) {
          if (i > j) p *= ax[x][i];
          const float t = p * kx[x][j];
          xq[i] += dP[i][j] * t;
          float s = dP[i][j] * qx[x][i];
          if (i > j) {
            xr[i] += dK[i][j] * t;
            s += dK[i][j] * kx[x][i];
          }
          xw[j] += p * s;
        }
      }
      store(a.dq, x, 0, xq);
      store(a.dk, x, 0, xr + xw);
      f32x4 s = qx[x] * xq + kx[x] * (xr - xw);
#pragma unroll
      for (int i = 2; i >= 0; --i) s[i] += s[i + 1];
      float later, total;
      above(s[0], lane, g, later, total);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (SB * x + 4 * g + i < count)
          a.dlog[(base + (size_t)(SB * x + 4 * g + i) * H) * DK + d0] =
              ax[x][i] == 0.f ? 0.f : carry + later + s[i];
      carry += total;
    }
  }
}

}  // namespace ssm
