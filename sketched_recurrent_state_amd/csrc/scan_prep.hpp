// scan_prep.hpp -- what a block of 16 tokens needs before the state is known: the
// decayed products K and P, the inverse of the unit lower triangular I + K diag(b),
// and the gate products (notation in scan.hpp). One wave per block, all blocks at once.
//
// KDA also writes three decayed copies of its keys and queries in fp32 (the passes would
// otherwise decay them once for each column block): 80 us for 131,072 token rows of 128, 360 MB
// read and written; a wave a block took 107 us. With scalar gates the 16 dependent steps of the substitution take most of the
// time: 40 us for 262,144 rows (GDN, bf16).
#pragma once

#include "scan.hpp"

namespace ssm {

// Waves of a block: KDA's channels are divided over them (the block's keys, queries and gates in
// LDS leave room for 5 workgroups on a CU, too few waves if each has one).
template <int RULE, int DK>
constexpr int kPrepWaves = RULE == KDA && DK >= 64 ? DK / 32 : 1;

// LDS written by this wave's other lanes
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup", "local");
  __builtin_amdgcn_wave_barrier();
}

template <int RULE, int DK, typename TIN, bool BWD>
__global__ void __launch_bounds__((64 * kPrepWaves<RULE, DK>)) scan_prep_kernel(const ScanArgs a) {
  constexpr bool DELTA = RULE != MAMBA2, CH = RULE == KDA;
  constexpr bool EXACT = kExact<RULE, TIN> && DK >= 32;
  constexpr int T = DK / 16, LD = DK + 4, LK = 20;
  constexpr int W = kPrepWaves<RULE, DK>, TW = T / W;  // waves, and channel tiles of a wave
  __shared__ __align__(16) float sq[CH ? SB * LD : 1], sk[CH ? SB * LD : 1], sa[CH ? SB * LD : 1];
  __shared__ __align__(16) float sl[2 * SB * LK];
  const int blk = blockIdx.x % NB, h = blockIdx.x / NB % a.heads, c = blockIdx.x / NB / a.heads;
  const size_t cell = a.cell(c, h), block = cell * NB + blk;
  int tok, count;
  if (!a.plan.cell(c, tok, count) || SB * blk >= count) return;
  tok += SB * blk;
  count -= SB * blk;  // valid rows: min(count, 16)
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, m = lane & 15, g = lane >> 4;
  const bool valid = m < count;
  const uint32_t rm = row_mask(valid);
  const size_t at = (size_t)(tok + (valid ? m : 0)) * a.heads + h;  // lane's token row
  const TIN* q = static_cast<const TIN*>(a.q);
  const TIN* k = static_cast<const TIN*>(a.k);

  float b = 0.f;
  if constexpr (DELTA) b = valid ? a.beta[at] : 0.f;
  f32x4 P = {0.f, 0.f, 0.f, 0.f}, K = P;
  if constexpr (!CH) {
    const float gate = valid ? a.decay[at] : 1.f;
    float in, out, ratio[4];
    gate_products(gate, m, g, in, out, ratio);
    float* row = a.w.row + block * ROW;
    if (g == 0) {
      row[m] = in;
      row[SB + m] = out;
      row[2 * SB + m] = b;
    }
    if constexpr (EXACT) {
#pragma unroll
      for (int t = 0; t < T / 2; ++t) {
        uint4 qa = *reinterpret_cast<const uint4*>(q + at * DK + 32 * t + 8 * g);
        uint4 ka = *reinterpret_cast<const uint4*>(k + at * DK + 32 * t + 8 * g);
        qa = masked(qa, rm);
        ka = masked(ka, rm);
        P = mfma32(qa, ka, P);
        if constexpr (DELTA) K = mfma32(ka, ka, K);
      }
    }
    // q k^T and k k^T: slot g of product (t, i) is channel 16 t + 4 g + i
#pragma unroll
    for (int t = 0; t < (EXACT ? 0 : T); ++t) {
      Quad<TIN> qa, ka;
      qa.load(q + at * DK + 16 * t + 4 * g);
      ka.load(k + at * DK + 16 * t + 4 * g);
      qa.mask(rm);
      ka.mask(rm);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        P = mfma4(qa[i], ka[i], P);
        if constexpr (DELTA) K = mfma4(ka[i], ka[i], K);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      P[i] = m <= 4 * g + i ? P[i] * ratio[i] : 0.f;
      K[i] = m < 4 * g + i ? K[i] * ratio[i] : 0.f;
    }
  } else {
    // stage the block; lane (m, g) takes token m, channels 16 t + 4 g + i of the wave's tiles
    const int c0 = 16 * TW * wave + 4 * g;
#pragma unroll
    for (int t = 0; t < TW; ++t) {
      Quad<TIN> qa, ka;
      Quad<float> aa;
      const size_t o = at * DK + 16 * t + c0;
      qa.load(q + o);
      ka.load(k + o);
      aa.load(a.decay + o);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int s = m * LD + 16 * t + c0 + i;
        sq[s] = masked(qa[i], rm);
        sk[s] = masked(ka[i], rm);
        sa[s] = valid ? aa[i] : 1.f;
      }
    }
    if (tid < SB) a.w.row[block * ROW + 2 * SB + m] = b;
    __syncthreads();
    // I q, I k and the whole block's decay, and O k, one channel at a time
    static_assert(64 * W >= 2 * DK || !CH, "two threads a channel");
    const int ch = tid % DK;
    const size_t o = block * SB * DK;
    if (tid < DK) {
      float p = 1.f;
#pragma unroll
      for (int l = 0; l < SB; ++l) {
        p *= sa[l * LD + ch];
        a.w.qh[o + l * DK + ch] = p * sq[l * LD + ch];
        a.w.kh[o + l * DK + ch] = p * sk[l * LD + ch];
      }
      a.w.all[block * DK + ch] = p;
    } else if (tid < 2 * DK) {
      float p = 1.f;
#pragma unroll
      for (int l = SB - 1; l >= 0; --l) {
        a.w.kt[o + l * DK + ch] = p * sk[l * LD + ch];
        p *= sa[l * LD + ch];
      }
    }
    // column m of K and P, the wave's channels of them: the key decays from row to row
    float p[4 * TW];
#pragma unroll
    for (int t = 0; t < TW; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) p[4 * t + i] = sk[m * LD + 16 * t + c0 + i];
#pragma unroll
    for (int r = 0; r < SB; ++r) {
      float sp = 0.f, sK = 0.f;
#pragma unroll
      for (int t = 0; t < TW; ++t) {
        const f32x4 qr = *reinterpret_cast<const f32x4*>(sq + r * LD + 16 * t + c0);
        const f32x4 kr = *reinterpret_cast<const f32x4*>(sk + r * LD + 16 * t + c0);
        const f32x4 ar = *reinterpret_cast<const f32x4*>(sa + r * LD + 16 * t + c0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float& x = p[4 * t + i];
          x *= r > m ? ar[i] : 1.f;
          sp += qr[i] * x;
          sK += kr[i] * x;
        }
      }
      sp = xsum32(xsum16(sp));
      sK = xsum32(xsum16(sK));
      if (r >> 2 == g) {  // lane (m, g) keeps rows 4 g + i
        P[r & 3] = m <= r ? sp : 0.f;
        K[r & 3] = m < r ? sK : 0.f;
      }
    }
    if constexpr (W > 1) {  // the sums over the waves, by the first, which goes on alone
      __syncthreads();
      f32x4* sums = reinterpret_cast<f32x4*>(sq);
      if (wave > 0) {
        sums[2 * tid] = P;
        sums[2 * tid + 1] = K;
      }
      __syncthreads();
      if (wave > 0) return;
#pragma unroll
      for (int w = 1; w < W; ++w) {
        P += sums[2 * (tid + 64 * w)];
        K += sums[2 * (tid + 64 * w) + 1];
      }
    }
  }
  if constexpr (BWD) {  // lane (m, g) holds the transpose's row m, columns 4g + i
    store_split(a.w.P, block, lane, split4(P));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) sl[(4 * g + i) * LK + m] = P[i];
    wave_sync();
    store_split(a.w.P, block, lane, split4(*reinterpret_cast<const f32x4*>(sl + m * LK + 4 * g)));
    wave_sync();
  }
  if constexpr (DELTA) {
    // (I + L)^-1 by forward substitution, column m: lanes of g = 0 take L = K diag(b), of
    // g = 1 L = diag(b) K. In fp32 throughout: later rows inherit the earlier rows' errors.
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sl[(4 * g + i) * LK + m] = K[i] * b;
      sl[SB * LK + (4 * g + i) * LK + m] = K[i] * __shfl(b, 4 * g + i);
    }
    wave_sync();
    const float* L = sl + (g & 1) * SB * LK;
    float x[SB];
#pragma unroll
    for (int r = 0; r < SB; ++r) {
      float s = r == m ? 1.f : 0.f;
#pragma unroll
      for (int l = 0; l < r; ++l) s -= L[r * LK + l] * x[l];
      x[r] = s;
    }
    wave_sync();  // L has been read
    if (g < 2) {
#pragma unroll
      for (int r = 0; r < SB; ++r) sl[g * SB * LK + r * LK + m] = x[r];
    }
    wave_sync();
    store_split(a.w.A, block, lane, split4(*reinterpret_cast<const f32x4*>(sl + m * LK + 4 * g)));
    if constexpr (BWD) {
      f32x4 t;
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = sl[SB * LK + (4 * g + i) * LK + m];
      store_split(a.w.A2, block, lane, split4(t));
    }
  }
}

}  // namespace ssm
