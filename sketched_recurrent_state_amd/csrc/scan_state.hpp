// scan_state.hpp -- the two passes along a sequence: the state forwards
// (scan_state_kernel) and its gradient backwards (scan_gradient_kernel). Notation in
// scan.hpp. The recurrence acts on the d_k side only, so columns of the state never meet:
// a wave holds 16 of them in registers from the first block to the last. The state is kept
// in fp32; once per block it is split into three bf16 parts and multiplied by the keys and
// queries, which are exact (bf16 inputs with scalar gates) or split too.
//
// Two shapes. Wide: each of a workgroup's waves holds a column block of its own. Narrow, for
// few units (scan_rule.hpp says when): the rows of one column block are divided over DS
// waves, which add up their parts of k S through LDS, and one more wave works out y a block
// behind, off the recurrence's path.
//
// The waves of a workgroup share the block's operands: they are loaded into registers two
// blocks ahead, put into LDS when the block before is under way, and read from there.
//
// Rows of the state's tiles: tile 2s + h holds channel 32 s + 8 g + 4 h + i in row 4g + i, so
// that the two tiles' registers are the 32-deep B operand whose slot 8g + j is channel
// 32 s + 8 g + j: the A operand is then 16 consecutive bytes of a key. The update needs the
// keys the other way round (four tokens of one channel): ds_read_b64_tr_b16 transposes them.
// With d_k = 16 the upper half of the only 32 channels is zero.
//
// Bounds. Narrow (a GDN prompt of 8192 tokens, 32 heads, 128 x 128, bf16: 437 us of 477): the
// chain of 512 dependent blocks, 0.85 us each, of which a wave issues instructions for half and
// waits for LDS, barriers and products for the rest. Wide (16 unlike prompts, 8192 tokens, 32
// heads: 172 us): the vector ALU, 464 instructions a block and wave, most of them the split of
// the state; busy 91 % of the time while all sequences run, and the longest one's tail after.
// Thirty-two tokens a step would halve the splits, but its registers leave two waves a SIMD:
// 521 us and 239 us.
//
// Rows behind the sequence's end are given the last token's keys and queries (the plan of a
// partial block has b = 0 and no P or K there), and values and dy of zero: they write nothing.
#pragma once

#include "scan.hpp"

namespace ssm {

template <int DK>
constexpr int kPadded = DK < 32 ? 32 : DK;

template <int DK>
struct KeyTile {
  // Row stride in bytes: rows 16 dwords apart modulo the 64 banks, so that the 4 rows x 4
  // pieces of 8 bytes that 16 lanes read together fall on different banks.
  static constexpr int STRIDE = DK >= 128 ? 2 * DK + 64 : DK == 64 ? 192 : 64;
  static constexpr int BYTES = SB * STRIDE;
  // Channels 32 s + 8 g .. + 7 of token m.
  static __device__ __forceinline__ uint4 row(const char* lds, int m, int g, int s) {
    return *reinterpret_cast<const uint4*>(lds + m * STRIDE + 64 * s + 16 * g);
  }
  // Tokens 4g .. 4g + 3 of the channel in row m of tile t = 2s + h. Sixteen lanes transpose
  // four rows of 16 values: lane p + 4 r names values 4p .. 4p + 3 of row r and receives column
  // p + 4 r of the four.
  static __device__ __forceinline__ uint2 column(const char* lds, int m, int g, int t) {
    const char* p = lds + (4 * g + (m >> 2)) * STRIDE + 64 * (t >> 1) + 16 * (m & 3) + 8 * (t & 1);
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
  }
};

// Channel of row i (of this lane's four) of tile t.
__device__ __forceinline__ int split_channel(int t, int g, int i) {
  return 32 * (t >> 1) + 8 * g + 4 * (t & 1) + i;
}

__device__ __forceinline__ f32x4 vec(float4 x) { return f32x4{x.x, x.y, x.z, x.w}; }

// Keys and queries of a block in LDS. `rows`: the operand of the product with the state;
// `cols`: that of the update. One array serves both where the gates are scalars.
template <int RULE, int DK, typename TIN>
struct SplitBlock {
  static constexpr bool EXACT = kExact<RULE, TIN>;
  static constexpr int DP = kPadded<DK>, PARTS = EXACT ? 1 : 3, ARRAYS = RULE == KDA ? 3 : 2;
  static constexpr int COLS = RULE == KDA ? 2 : 0;  // rows are array 0, queries array 1
  using KT = KeyTile<DP>;
  __align__(16) char key[ARRAYS][PARTS][KT::BYTES];
  uint2 P[192], A[192];             // split operands, 3 x 64 lanes
  __align__(16) float row[3 * SB];  // decay in, decay out, b
  __align__(16) float all[RULE == KDA ? DK : 4];

  __device__ __forceinline__ Split4 split(const uint2* p, int lane) const {
    return Split4{p[lane], p[64 + lane], p[128 + lane]};
  }
  __device__ __forceinline__ f32x4 rows(int which, int g) const {
    return vec(*reinterpret_cast<const float4*>(row + SB * which + 4 * g));
  }
  // The whole block's decay of tile t's four rows of this lane.
  __device__ __forceinline__ f32x4 whole(int t, int g) const {
    if constexpr (RULE == KDA) {
      const int c = split_channel(t, g, 0);
      return c < DK ? vec(*reinterpret_cast<const float4*>(all + c)) : f32x4{0.f, 0.f, 0.f, 0.f};
    } else {
      const float a = row[SB - 1];
      return f32x4{a, a, a, a};
    }
  }
  // c + (array's rows) S for 32 channels s, S split
  __device__ __forceinline__ f32x4 product(int array, int m, int g, int s, uint4 sh, uint4 sm,
                                           uint4 sl, f32x4 c) const {
    const uint4 h = KT::row(key[array][0], m, g, s);
    if constexpr (EXACT) {
      c = mfma32(h, sl, c);
      c = mfma32(h, sm, c);
    } else {
      const uint4 mid = KT::row(key[array][1], m, g, s), l = KT::row(key[array][2], m, g, s);
      c = mfma32(l, sh, c);
      c = mfma32(h, sl, c);
      c = mfma32(mid, sm, c);
      c = mfma32(mid, sh, c);
      c = mfma32(h, sm, c);
    }
    return mfma32(h, sh, c);
  }
  // The array's columns of tile t, and c + their transpose times w.
  __device__ __forceinline__ Split4 columns(int array, int m, int g, int t) const {
    Split4 s;
    s.h = KT::column(key[array][0], m, g, t);
    if constexpr (!EXACT) {
      s.m = KT::column(key[array][1], m, g, t);
      s.l = KT::column(key[array][2], m, g, t);
    }
    return s;
  }
  static __device__ __forceinline__ f32x4 update(const Split4& k, const Split4& w, f32x4 c) {
    if constexpr (EXACT) return mfma_exact(k.h, w, c);
    else return mfma_split(k, w, c);
  }
};

// A thread's share of a block, in registers between the load and the LDS write.
template <int RULE, int DK, typename TIN, int NT, bool Q, bool P>
struct SplitShare {
  using Block = SplitBlock<RULE, DK, TIN>;
  static constexpr bool EXACT = Block::EXACT, DELTA = RULE != MAMBA2;
  static constexpr int E = EXACT ? 8 : 4;  // values of a 16-byte piece
  static constexpr int KP = SB * DK / E, NK = (KP + NT - 1) / NT, NP = (192 + NT - 1) / NT;
  uint4 k[NK], q[Q ? NK : 1], c[RULE == KDA ? NK : 1];
  uint2 p[P ? NP : 1], a[DELTA ? NP : 1];
  float row, all[RULE == KDA ? (DK + NT - 1) / NT : 1];

  // Where a thread's pieces are: byte offsets from the block's first token, in two parts, of
  // which the first (the token's) is cut at the sequence's last token.
  struct Place {
    uint32_t token[NK], column[NK];
    __device__ __forceinline__ Place(const ScanArgs& s, int tid) {
#pragma unroll
      for (int n = 0; n < NK; ++n) {
        const int piece = min(tid + n * NT, KP - 1);  // the surplus threads load the last one again
        token[n] = piece / (DK / E) * token_bytes(s);
        column[n] = piece % (DK / E) * 16;
      }
    }
    static __device__ __forceinline__ uint32_t token_bytes(const ScanArgs& s) {
      return (uint32_t)(s.heads * DK * sizeof(TIN));
    }
  };
  // Block j of a unit whose first token is row `at` of the inputs and whose first block is
  // `block0` of the workspace; `count` tokens from the block's first to the sequence's end.
  // rows, cols: KDA's decayed keys in the workspace; A: the pass's inverse.
  __device__ __forceinline__ void load(const ScanArgs& s, const Place& place, const float* rows,
                                       const float* cols, const float* A, size_t at, size_t block0,
                                       int j, int count, int tid) {
    const size_t block = block0 + j;
    if constexpr (RULE == KDA) {
#pragma unroll
      for (int n = 0; n < NK; ++n) {
        const uint32_t piece = min(tid + n * NT, KP - 1);
        k[n] = reinterpret_cast<const uint4*>(rows + block * SB * DK)[piece];
        c[n] = reinterpret_cast<const uint4*>(cols + block * SB * DK)[piece];
        if constexpr (Q) q[n] = reinterpret_cast<const uint4*>(s.w.qh + block * SB * DK)[piece];
      }
    } else {
      const size_t first = (at + (size_t)(SB * j) * s.heads) * DK * sizeof(TIN);
      const char* pk = static_cast<const char*>(s.k) + first;
      const char* pq = static_cast<const char*>(s.q) + first;
      const uint32_t last = (uint32_t)(min(count, SB) - 1) * Place::token_bytes(s);
#pragma unroll
      for (int n = 0; n < NK; ++n) {
        const uint32_t o = min(place.token[n], last) + place.column[n];
        k[n] = *reinterpret_cast<const uint4*>(pk + o);
        if constexpr (Q) q[n] = *reinterpret_cast<const uint4*>(pq + o);
      }
    }
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const uint32_t i = min(tid + n * NT, 191);
      if constexpr (P) p[n] = (reinterpret_cast<const uint2*>(s.w.P) + block * 192)[i];
      if constexpr (DELTA) a[n] = (reinterpret_cast<const uint2*>(A) + block * 192)[i];
    }
    row = (s.w.row + block * ROW)[(uint32_t)min(tid, ROW - 1)];
    if constexpr (RULE == KDA) {
#pragma unroll
      for (int n = 0; n < (DK + NT - 1) / NT; ++n)
        all[n] = (s.w.all + block * DK)[(uint32_t)min(tid + n * NT, DK - 1)];
    }
  }
  static __device__ __forceinline__ void put_piece(Block& b, int array, int piece, uint4 x) {
    char* to = b.key[array][0] + piece / (DK / E) * Block::KT::STRIDE + piece % (DK / E) * (2 * E);
    if constexpr (EXACT) {
      *reinterpret_cast<uint4*>(to) = x;
    } else {
      const Split4 s = split4(__builtin_bit_cast(f32x4, x));
      *reinterpret_cast<uint2*>(to) = s.h;
      *reinterpret_cast<uint2*>(to + Block::KT::BYTES) = s.m;
      *reinterpret_cast<uint2*>(to + 2 * Block::KT::BYTES) = s.l;
    }
  }
  __device__ __forceinline__ void put(Block& b, int tid) const {
#pragma unroll
    for (int n = 0; n < NK; ++n) {
      const int piece = tid + n * NT;
      if (KP % NT == 0 || piece < KP) {
        put_piece(b, 0, piece, k[n]);
        if constexpr (Q) put_piece(b, 1, piece, q[n]);
        if constexpr (RULE == KDA) put_piece(b, 2, piece, c[n]);
      }
    }
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const int i = tid + n * NT;
      if (192 % NT == 0 || i < 192) {
        if constexpr (P) b.P[i] = p[n];
        if constexpr (DELTA) b.A[i] = a[n];
      }
    }
    if (tid < 3 * SB) b.row[tid] = row;
    if constexpr (RULE == KDA) {
#pragma unroll
      for (int n = 0; n < (DK + NT - 1) / NT; ++n)
        if (tid + n * NT < DK) b.all[tid + n * NT] = all[n];
    }
  }
};

// A lane's four values of a block's tokens 4g + i (one column), cut at the sequence's last token.
template <typename T>
struct ColumnPlace {
  uint32_t token[4], bytes;
  __device__ __forceinline__ ColumnPlace(size_t stride, int g) : bytes((uint32_t)(stride * sizeof(T))) {
#pragma unroll
    for (int i = 0; i < 4; ++i) token[i] = (4 * g + i) * bytes;
  }
  __device__ __forceinline__ void load(const T* p, int j, int len, T (&x)[4]) const {
    const char* first = reinterpret_cast<const char*>(p) + (size_t)(SB * j) * bytes;
    const uint32_t last = (uint32_t)(min(len - SB * j, SB) - 1) * bytes;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const T*>(first + min(token[i], last));
  }
};

// Zero for the channels of the blocks that d_k = 16 leaves empty.
template <int RULE, int DK, typename TIN, int N>
__device__ __forceinline__ void clear_padding(SplitBlock<RULE, DK, TIN> (&buf)[N], int tid, int nt) {
  if constexpr (DK < kPadded<DK>) {
    uint32_t* p = reinterpret_cast<uint32_t*>(buf);
    for (int i = tid; i < (int)(sizeof(buf) / 4); i += nt) p[i] = 0;
    __syncthreads();
  }
}

// The state's tiles of this wave times the block's rows, and times its queries.
template <int TL>
struct StateParts {
  uint4 h[TL / 2], m[TL / 2], l[TL / 2];
  __device__ __forceinline__ explicit StateParts(const f32x4 (&S)[TL]) {
#pragma unroll
    for (int c = 0; c < TL / 2; ++c) {
      const Split4 x = split4(S[2 * c]), y = split4(S[2 * c + 1]);
      h[c] = make_uint4(x.h.x, x.h.y, y.h.x, y.h.y);
      m[c] = make_uint4(x.m.x, x.m.y, y.m.x, y.m.y);
      l[c] = make_uint4(x.l.x, x.l.y, y.l.x, y.l.y);
    }
  }
  template <typename B>
  __device__ __forceinline__ f32x4 times(const B& b, int array, int s0, int lm, int lg) const {
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < TL / 2; ++c) s = b.product(array, lm, lg, s0 + c, h[c], m[c], l[c], s);
    return s;
  }
};

// The sum of x over the first DS waves.
template <int DS>
__device__ __forceinline__ f32x4 wave_sum(const f32x4* x, int lane) {
  f32x4 s = x[lane];
#pragma unroll
  for (int i = 1; i < DS; ++i) s += x[64 * i + lane];
  return s;
}

// A wave's part of the state in memory: tile t's row i at element `offset(t, i)`.
template <int DK, int TL, typename F>
__device__ __forceinline__ void each_row(int s0, int g, F&& f) {
#pragma unroll
  for (int t = 0; t < TL; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = 32 * s0 + split_channel(t, g, i);
      if (DK == kPadded<DK> || c < DK) f(t, i, (size_t)c);
    }
}

// Shape of a pass: NW waves that hold state, NARROW or not, and whether a wave more makes y.
template <int DK, int NW, bool NARROW>
struct SplitShape {
  static constexpr int DS = NARROW ? NW : 1;            // waves of a column block
  static constexpr int TL = kPadded<DK> / 16 / DS;      // tiles of a wave
  static constexpr int CB = NW / DS;                    // column blocks of the workgroup
};

template <int RULE, int DK, typename TIN, bool NARROW>
constexpr int split_buffers() {
  // two blocks in LDS, or one where two would leave room for a single workgroup on a CU
  return NARROW || 2 * sizeof(SplitBlock<RULE, DK, TIN>) <= 80 * 1024 ? 2 : 1;
}

template <int RULE, typename TIN>
__device__ __forceinline__ f32x4 y_part(const Split4& P, f32x4 w, f32x4 o) {
  if constexpr (RULE == MAMBA2 && sizeof(TIN) == 2) {  // the values are exact
    const uint2 x = make_uint2(heads(w[0], w[1]), heads(w[2], w[3])), none = make_uint2(0u, 0u);
    o = mfma_two(P.l, x, none, none, o);
    return mfma_two(P.h, x, P.m, x, o);
  } else {
    return mfma_split(P, split4(w), o);
  }
}

// Forwards. Writes y and the final state, or for the backward pass (BWD) r of every token and
// the state at each chunk's start.
template <int RULE, int DK, typename TIN, int NW, bool NARROW, bool BWD>
__global__ void __launch_bounds__(64 * (NW + (NARROW && !BWD)), 2) scan_state_kernel(const ScanArgs a) {
  constexpr bool DELTA = RULE != MAMBA2, SCALAR = RULE != KDA;
  using Shape = SplitShape<DK, NW, NARROW>;
  constexpr int TL = Shape::TL, DS = Shape::DS, NT = 64 * NW;
  constexpr bool YWAVE = NARROW && !BWD;
  constexpr int NBUF = split_buffers<RULE, DK, TIN, NARROW>();
  using Block = SplitBlock<RULE, DK, TIN>;
  using Share = SplitShare<RULE, DK, TIN, NT, !BWD, !BWD>;
  __shared__ Block buf[NBUF];
  __shared__ f32x4 xk[DS > 1 && DELTA ? NT : 1], xq[2][YWAVE ? NT : 1], xw[2][YWAVE ? 64 : 1];
  int unit, part;
  unit_of(blockIdx.x, a.d_v / (16 * Shape::CB), unit, part);
  const int seq = unit / a.heads, h = unit % a.heads;
  if (seq >= a.plan.seqs) return;
  int tok, len, first;
  if (!a.plan.sequence(seq, tok, len, first)) return;
  const int srow = a.slot ? a.slot[seq] : seq;
  if (srow < 0 || srow >= a.num_slots) return;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, m = lane & 15, g = lane >> 4;
  const int col = 16 * (part * Shape::CB + wave / DS) + m, dpart = wave % DS, s0 = dpart * TL / 2;
  const size_t stride = (size_t)a.heads * a.d_v;
  const size_t ro = ((size_t)tok * a.heads + h) * a.d_v;  // the unit's first row of v and y
  const int blocks = (len + SB - 1) / SB;
  clear_padding(buf, tid, 64 * (NW + YWAVE));

  if constexpr (YWAVE) {
    if (wave == NW) {  // y of block j - 1, while the others are at block j
      float* y = a.y + ro + 16 * part + m;
      Split4 P;
      f32x4 in = {1.f, 1.f, 1.f, 1.f}, o;
      for (int j = 0; j <= blocks; ++j) {
        __syncthreads();
        // half of it on either side of the others' second barrier
        f32x4 w;
        if (j > 0) {
          o = wave_sum<DS>(xq[(j - 1) & 1], lane) * in;
          w = xw[(j - 1) & 1][lane];
        }
        if constexpr (DS > 1 && DELTA) {
          if (j < blocks) __syncthreads();
        }
        if (j > 0) {
          o = y_part<RULE, TIN>(P, w, o);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (SB * (j - 1) + 4 * g + i < len) y[(size_t)(SB * (j - 1) + 4 * g + i) * stride] = o[i];
        }
        if (j == blocks) return;
        P = buf[j & 1].split(buf[j & 1].P, lane);
        if constexpr (SCALAR) in = buf[j & 1].rows(0, g);
      }
    }
  }

  const size_t so = ((size_t)srow * a.heads + h) * DK * a.d_v + col;
  const TIN* v = static_cast<const TIN*>(a.v) + ro + col;
  f32x4 S[TL] = {};
  if (a.state_in)
    each_row<DK, TL>(s0, g, [&](int t, int i, size_t c) { S[t][i] = a.state_in[so + c * a.d_v]; });

  struct Ahead {
    Share s;
    TIN v[4];
  };
  const size_t cell0 = a.cell(first, h);
  const typename Share::Place place(a, tid);
  const ColumnPlace<TIN> vplace(stride, g);
  auto fetch = [&](Ahead& x, int j) {
    x.s.load(a, place, a.w.kh, a.w.kt, a.w.A, (size_t)tok * a.heads + h, cell0 * NB, j, len - SB * j, tid);
    vplace.load(v, j, len, x.v);
  };
  auto run = [&](const Block& b, const TIN (&vr)[4], int j) {
    const size_t cell = cell0 + j / NB;
    if constexpr (BWD) {
      if (j % NB == 0) {
        float* p = a.w.S + cell * DK * a.d_v + col;
        each_row<DK, TL>(s0, g, [&](int t, int i, size_t c) { p[c * a.d_v] = S[t][i]; });
      }
    }
    // what follows the sum over waves is read before it
    f32x4 ks, o, w;
    const f32x4 in = b.rows(0, g), out = b.rows(1, g), beta = b.rows(2, g);
    Split4 A, kt[NARROW ? TL : 1];
    if constexpr (DELTA) A = b.split(b.A, lane);
    if constexpr (NARROW) {
#pragma unroll
      for (int t = 0; t < TL; ++t) kt[t] = b.columns(Block::COLS, m, g, 2 * s0 + t);
    }
    if constexpr (DELTA || !BWD) {
      const StateParts<TL> x(S);
      if constexpr (DELTA) ks = x.times(b, 0, s0, m, g);
      if constexpr (DS > 1 && DELTA) {
        xk[tid] = ks;
        __syncthreads();
        ks = wave_sum<DS>(xk, lane);
      }
      if constexpr (!BWD) o = x.times(b, 1, s0, m, g);
    }
    f32x4 vf;
#pragma unroll
    for (int i = 0; i < 4; ++i) vf[i] = SB * j + 4 * g + i < len ? to_f32(vr[i]) : 0.f;
    if constexpr (DELTA) {
      if constexpr (SCALAR) ks *= in;
      const f32x4 r = mfma_split(A, split4(vf - ks), f32x4{0.f, 0.f, 0.f, 0.f});
      if constexpr (BWD) {
        if (dpart == 0) {
          float* p = a.w.r + (cell * CT + SB * (j % NB) + 4 * g) * a.d_v + col;
#pragma unroll
          for (int i = 0; i < 4; ++i) p[i * a.d_v] = r[i];
        }
      }
      w = beta * r;
    } else {
      w = vf;
    }
    if constexpr (YWAVE) {
      if (dpart == 0) xw[j & 1][lane] = w;
    }
    // S <- a_1..a_16 S + (O k)^T w
    const Split4 ow = split4(SCALAR ? out * w : w);
#pragma unroll
    for (int t = 0; t < TL; ++t)
      S[t] = Block::update(NARROW ? kt[NARROW ? t : 0] : b.columns(Block::COLS, m, g, t), ow,
                           S[t] * b.whole(2 * s0 + t, g));
    if constexpr (YWAVE) xq[j & 1][tid] = o;
    if constexpr (!BWD && !YWAVE) {
      if constexpr (SCALAR) o *= in;
      o = y_part<RULE, TIN>(b.split(b.P, lane), w, o);
      float* y = a.y + ro + col + (size_t)(SB * j + 4 * g) * stride;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (SB * j + 4 * g + i < len) y[i * stride] = o[i];
    }
  };
  if (blocks > 0) {
    // Past the end the last block is fetched and put again: a fetch behind a branch would make
    // every wait for the one before it a wait for all loads.
    Ahead x0, x1;
    fetch(x0, 0);
    fetch(x1, min(1, blocks - 1));
    x0.s.put(buf[0], tid);
    auto step = [&](Ahead& now, const Ahead& next, int b, int j) {
      TIN vr[4] = {now.v[0], now.v[1], now.v[2], now.v[3]};
      fetch(now, min(j + 2, blocks - 1));
      __syncthreads();  // block j is in its buffer, and nobody reads the other one any more
      run(buf[b % NBUF], vr, j);
      if constexpr (NBUF == 1) __syncthreads();
      next.s.put(buf[(b + 1) % NBUF], tid);
    };
    for (int j = 0;;) {
      step(x0, x1, 0, j);
      if (++j == blocks) break;
      step(x1, x0, 1, j);
      if (++j == blocks) break;
    }
  }
  if constexpr (YWAVE) __syncthreads();  // the last block's w and q S
  if constexpr (!BWD)
    each_row<DK, TL>(s0, g, [&](int t, int i, size_t c) { a.state[so + c * a.d_v] = S[t][i]; });
}

// Backwards. Writes dv, e of every token, dL/dS at each chunk's end and dL/d(initial state).
template <int RULE, int DK, typename TIN, int NW, bool NARROW>
__global__ void __launch_bounds__(64 * NW, 2) scan_gradient_kernel(const ScanArgs a) {
  constexpr bool DELTA = RULE != MAMBA2, SCALAR = RULE != KDA;
  using Shape = SplitShape<DK, NW, NARROW>;
  constexpr int TL = Shape::TL, DS = Shape::DS, NT = 64 * NW;
  constexpr int NBUF = split_buffers<RULE, DK, TIN, NARROW>();
  using Block = SplitBlock<RULE, DK, TIN>;
  using Share = SplitShare<RULE, DK, TIN, NT, true, true>;
  __shared__ Block buf[NBUF];
  __shared__ f32x4 xk[DS > 1 ? NT : 1];
  int unit, part;
  unit_of(blockIdx.x, a.d_v / (16 * Shape::CB), unit, part);
  const int seq = unit / a.heads, h = unit % a.heads;
  if (seq >= a.plan.seqs) return;
  int tok, len, first;
  if (!a.plan.sequence(seq, tok, len, first)) return;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, m = lane & 15, g = lane >> 4;
  const int col = 16 * (part * Shape::CB + wave / DS) + m, dpart = wave % DS, s0 = dpart * TL / 2;
  const size_t so = ((size_t)seq * a.heads + h) * DK * a.d_v + col;
  const size_t stride = (size_t)a.heads * a.d_v;
  const size_t ro = ((size_t)tok * a.heads + h) * a.d_v + col;
  const float* dy = a.dy + ro;
  const int blocks = (len + SB - 1) / SB;
  clear_padding(buf, tid, NT);

  f32x4 G[TL] = {};
  if (a.dstate)
    each_row<DK, TL>(s0, g, [&](int t, int i, size_t c) { G[t][i] = a.dstate[so + c * a.d_v]; });

  struct Ahead {
    Share s;
    float dy[4];
  };
  const size_t cell0 = a.cell(first, h);
  const typename Share::Place place(a, tid);
  const ColumnPlace<float> yplace(stride, g);
  auto fetch = [&](Ahead& x, int j) {
    x.s.load(a, place, a.w.kt, a.w.kh, a.w.A2, (size_t)tok * a.heads + h, cell0 * NB, j, len - SB * j,
             tid);
    yplace.load(dy, j, len, x.dy);
  };
  auto run = [&](const Block& b, const float (&yr)[4], int j) {
    const size_t cell = cell0 + j / NB;
    if (j % NB == NB - 1 || j == blocks - 1) {
      float* p = a.w.G + cell * DK * a.d_v + col;
      each_row<DK, TL>(s0, g, [&](int t, int i, size_t c) { p[c * a.d_v] = G[t][i]; });
    }
    const f32x4 in = b.rows(0, g), out = b.rows(1, g), beta = b.rows(2, g);
    f32x4 y, iy;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = SB * j + 4 * g + i < len ? yr[i] : 0.f;
    iy = SCALAR ? in * y : y;
    Split4 A, P, q[NARROW ? TL : 1], k[NARROW ? TL : 1];
    if constexpr (NARROW) {  // what follows the sum over waves is read before it
      P = b.split(b.P, lane);
      if constexpr (DELTA) A = b.split(b.A, lane);
#pragma unroll
      for (int t = 0; t < TL; ++t) {
        q[t] = b.columns(1, m, g, 2 * s0 + t);
        if constexpr (DELTA) k[t] = b.columns(Block::COLS, m, g, 2 * s0 + t);
      }
    }
    f32x4 w = StateParts<TL>(G).times(b, 0, s0, m, g);
    if constexpr (DS > 1) xk[tid] = w;
    if constexpr (!NARROW) P = b.split(b.P, lane);
    const f32x4 pdy = mfma_split(P, split4(y), f32x4{0.f, 0.f, 0.f, 0.f});
    const Split4 iys = split4(iy);
#pragma unroll
    for (int t = 0; t < TL; ++t)
      G[t] = Block::update(NARROW ? q[NARROW ? t : 0] : b.columns(1, m, g, t), iys,
                           G[t] * b.whole(2 * s0 + t, g));
    if constexpr (DS > 1) {
      __syncthreads();
      w = wave_sum<DS>(xk, lane);
    }
    w = (SCALAR ? out * w : w) + pdy;
    f32x4 dr = w;
    if constexpr (DELTA) {
      if constexpr (!NARROW) A = b.split(b.A, lane);
      const f32x4 e = mfma_split(A, split4(w), f32x4{0.f, 0.f, 0.f, 0.f});
      if (dpart == 0) {
        float* p = a.w.e + (cell * CT + SB * (j % NB) + 4 * g) * a.d_v + col;
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i * a.d_v] = e[i];
      }
      dr = beta * e;
      const Split4 ir = split4(SCALAR ? -(in * dr) : -dr);
#pragma unroll
      for (int t = 0; t < TL; ++t)
        G[t] = Block::update(NARROW ? k[NARROW ? t : 0] : b.columns(Block::COLS, m, g, t), ir, G[t]);
    }
    if (dpart == 0) {
      TIN* dv = static_cast<TIN*>(a.dv) + ro + (size_t)(SB * j + 4 * g) * stride;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (SB * j + 4 * g + i < len) put(dv + i * stride, dr[i]);
    }
  };
  if (blocks > 0) {
    Ahead x0, x1;
    fetch(x0, blocks - 1);
    fetch(x1, max(blocks - 2, 0));
    x0.s.put(buf[0], tid);
    auto step = [&](Ahead& now, const Ahead& next, int b, int j) {
      float yr[4] = {now.dy[0], now.dy[1], now.dy[2], now.dy[3]};
      fetch(now, max(j - 2, 0));
      __syncthreads();
      run(buf[b % NBUF], yr, j);
      if constexpr (NBUF == 1) __syncthreads();
      next.s.put(buf[(b + 1) % NBUF], tid);
    };
    for (int j = blocks - 1;;) {
      step(x0, x1, 0, j);
      if (--j < 0) break;
      step(x1, x0, 1, j);
      if (--j < 0) break;
    }
  }
  if (a.dstate_in)
    each_row<DK, TL>(s0, g, [&](int t, int i, size_t c) { a.dstate_in[so + c * a.d_v] = G[t][i]; });
}

}  // namespace ssm
