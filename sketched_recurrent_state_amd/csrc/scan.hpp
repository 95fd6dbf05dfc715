// scan.hpp -- the layer's recurrence over whole sequences (prompt processing and
// training): shared definitions of the scan kernels.
//
// Per (sequence, head), with D_t = a_t I (Mamba-2, GDN) or Diag(a_t) (KDA):
//   S_t = D_t S_{t-1} + k_t w_t^T,   y_t = S_t^T q_t,
//   w_t = v_t (Mamba-2)  or  b_t r_t,  r_t = v_t - (D_t S_{t-1})^T k_t (delta rules),
// which is the update S <- M S + b k v^T of the decode entry points with the rank-one
// part of M moved into the write.
//
// Sixteen tokens ("a block") at a time. With S the state before the block and, inside
// it, I_i = a_1 .. a_i (decay into the block), O_j = a_{j+1} .. a_16 (decay out of it)
// and G_ij = a_{j+1} .. a_i, all products of gates taken directly (no logarithms and no
// quotients, so a gate of zero is exact):
//   K_ij = k_i^T G_ij k_j  (j < i),     P_ij = q_i^T G_ij k_j  (j <= i)
//   r = (I + K diag(b))^-1 (v - (I k) S),  w = b r
//   y = (I q) S + P w,       S' = a_1..a_16 S + (O k)^T w
// and backwards, with G = dL/dS after the block and e = dL/dw:
//   e = (I + diag(b) K)^-T (P^T dy + (O k) G),  dr = b e = dv,  db_i = e_i . r_i
//   G' = a_1..a_16 G + (I q)^T dy - (I k)^T dr
//   dP = dy w^T, dK = -dr w^T (same triangles);
//   dq_i = I_i S dy_i + sum_j dP_ij G_ij k_j
//   dk_i = -I_i S dr_i + sum_j dK_ij G_ij k_j                       (its part as a reader)
//        + O_i G w_i + sum_j G_ji (dP_ji q_j + dK_ji k_j)           (its part as a writer)
//   d ln a_t = rowsum(S_end * G_end) + sum_{i >= t} (q_i dq_i + k_i dk_i^reader - k_i dk_i^writer),
// the last summed over the channels when the gate is a scalar.
//
// Matrix-core layouts. A result tile holds row 4g + i (g = lane / 16) and column lane % 16
// in its i-th register. In fp32 (v_mfma_f32_16x16x4_f32) that register is the B operand of
// the i-th product of a 16-deep contraction whose slot g stands for row 4g + i; split in
// bf16 (below) two tiles' registers, or one tile's in two parts, are the B operand of one
// 32-deep product. So states and right-hand sides stay in registers from
// one product to the next.
#pragma once

#include "common.hpp"
#include "launch.hpp"
#include "scan_table.hpp"

namespace ssm {

constexpr int SB = 16;          // tokens of a block
constexpr int NB = CT / SB;     // blocks of a chunk

typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mfma4(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

// fp32 -> the input type (bf16: to nearest, ties to even)
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(uint16_t* p, float x) { *p = (uint16_t)pack_bf16x2(x, x); }

// x where the row holds a token, else 0. A mask on the bits, not a select: a select lets the
// compiler put every load of a partial block behind a branch of its own.
__device__ __forceinline__ uint32_t row_mask(bool ok) { return ok ? 0xFFFFFFFFu : 0u; }
__device__ __forceinline__ float masked(float x, uint32_t mask) {
  return __uint_as_float(__float_as_uint(x) & mask);
}
__device__ __forceinline__ uint16_t masked(uint16_t x, uint32_t mask) { return (uint16_t)(x & mask); }
__device__ __forceinline__ uint4 masked(uint4 x, uint32_t mask) {
  return make_uint4(x.x & mask, x.y & mask, x.z & mask, x.w & mask);
}

// Four consecutive elements, raw until unpacked.
template <typename T>
struct Quad;
template <>
struct Quad<float> {
  float4 x;
  __device__ __forceinline__ void load(const float* p) { x = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void mask(uint32_t m) {
    x = make_float4(masked(x.x, m), masked(x.y, m), masked(x.z, m), masked(x.w, m));
  }
  __device__ __forceinline__ float operator[](int i) const {
    return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w;
  }
};
template <>
struct Quad<uint16_t> {
  uint2 x;
  __device__ __forceinline__ void load(const uint16_t* p) { x = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void mask(uint32_t m) { x = make_uint2(x.x & m, x.y & m); }
  __device__ __forceinline__ float operator[](int i) const {
    const uint32_t w = i < 2 ? x.x : x.y;
    return (i & 1) ? bf16_hi(w) : bf16_lo(w);
  }
};

// ---------------------------------------------------------------------------
// fp32 products on the bf16 matrix cores
// ---------------------------------------------------------------------------
// x = h + m + l: three bf16 values of 8 bits each. A product with
// an exact bf16 operand takes three matrix products, one with another split operand six
// (hh, hm, mh, hl, lh, mm), with fp32 sums. The dropped ones are below 2^-21 of the product
// (m < 2^-7 and l < 2^-15 of the value's power of two, which they share a sign with): 0.6 * 2^-24
// of it in the mean, always toward zero, where an fp32 product is off by up to 2^-24 either way.
// bf16 products run 16 times faster than fp32 ones, so three cost a fifth and six three eighths.
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

struct Split4 {
  uint2 h, m, l;  // four values each
};

// Each part is the leading 16 bits of what the parts before it leave (cut, not rounded), so
// the three hold all 24 bits. (Rounded parts with the differences from v_dot2_f32_bf16 take 7
// instructions a pair instead of 11, but ran slower: 1057 us against 1015 us for a GDN prompt
// of 8192 tokens x 32 heads.)
__device__ __forceinline__ float without_head(float x) {
  return x - __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t heads(float a, float b) {  // their leading 16 bits, a's low
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ void split2(float a, float b, uint32_t& h, uint32_t& m, uint32_t& l) {
  h = heads(a, b);
  a = without_head(a);
  b = without_head(b);
  m = heads(a, b);
  l = heads(without_head(a), without_head(b));
}
__device__ __forceinline__ Split4 split4(f32x4 x) {
  Split4 s;
  split2(x[0], x[1], s.h.x, s.m.x, s.l.x);
  split2(x[2], x[3], s.h.y, s.m.y, s.l.y);
  return s;
}

__device__ __forceinline__ f32x4 mfma32(uint4 a, uint4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
// Two 16-deep contractions in one 32-deep product: of its slots 8g + j, j < 4 take the
// first pair's rows 4g + j and j >= 4 the second pair's.
__device__ __forceinline__ f32x4 mfma_two(uint2 a0, uint2 b0, uint2 a1, uint2 b1, f32x4 c) {
  return mfma32(make_uint4(a0.x, a0.y, a1.x, a1.y), make_uint4(b0.x, b0.y, b1.x, b1.y), c);
}
// c + a b, both split (16-deep)
__device__ __forceinline__ f32x4 mfma_split(const Split4& a, const Split4& b, f32x4 c) {
  c = mfma_two(a.l, b.h, a.h, b.l, c);
  c = mfma_two(a.m, b.h, a.m, b.m, c);
  return mfma_two(a.h, b.h, a.h, b.m, c);
}
// c + a b, a exact. The last part takes a 32-deep product with an empty half, for products that add
// to one result keep to one instruction: behind a 16-deep one (v_mfma_f32_16x16x16_bf16) the compiler
// issues the 32-deep one that adds to its result without a wait, and that one's rows 2 and 3 then lack
// the first one's (in a loop of such pairs of whole numbers 93 % of the elements of these rows, none
// with 16 wait states in between; no memory and no other wave takes part).
__device__ __forceinline__ f32x4 mfma_exact(uint2 a, const Split4& b, f32x4 c) {
  const uint2 none = make_uint2(0u, 0u);
  c = mfma_two(a, b.l, none, none, c);
  return mfma_two(a, b.h, a, b.m, c);
}

// Whether the keys and queries are exact bf16 operands: KDA's, decayed channel by channel, and
// fp32 ones are split.
template <int RULE, typename TIN>
constexpr bool kExact = RULE != KDA && sizeof(TIN) == 2;

// Workspace: fp32 arrays with one part per cell (head, chunk), cell = head * cap + chunk, so that
// a unit's blocks follow one another.
struct ScanWork {
  // A operands in three bf16 parts, [cells][NB][3][64 lanes][4]:
  float* P;      // P                              (backward: its transpose)
  float* A;      // (I + K diag(b))^-1             (delta rules)
  float* A2;     // the transpose of (I + diag(b) K)^-1  (backward, delta rules)
  float* row;    // [cells][NB][3][SB]   decay in, decay out (scalar gates), b
  float* qh;     // [cells][CT][d_k]     I q                          (KDA)
  float* kh;     // [cells][CT][d_k]     I k
  float* kt;     // [cells][CT][d_k]     O k
  float* all;    // [cells][NB][d_k]     a_1 .. a_16
  float* r;      // [cells][CT][d_v]     r                            (backward, delta rules)
  float* e;      // [cells][CT][d_v]     e
  float* S;      // [cells][d_k][d_v]    state at the chunk's start   (backward)
  float* G;      // [cells][d_k][d_v]    dL/dS at the chunk's end
  size_t bytes;
};

inline ScanWork scan_work(const ssm_dims& d, int total, bool backward, void* base) {
  const size_t cells = (size_t)scan_capacity(total, d.batch) * d.heads;
  const bool delta = d.rule != SSM_MAMBA2, kda = d.rule == SSM_KDA;
  const size_t block = 3 * 64 * 4 / 2;
  ScanWork w{};
  size_t at = 0;
  auto take = [&](bool used, size_t per_cell) -> float* {
    if (!used) return nullptr;
    float* p = reinterpret_cast<float*>(static_cast<char*>(base) + at);
    at += cells * per_cell * sizeof(float);  // every part is a multiple of 16 bytes
    return p;
  };
  w.P = take(true, NB * block);
  w.A = take(delta, NB * block);
  w.A2 = take(delta && backward, NB * block);
  w.row = take(true, 3 * CT);
  w.qh = take(kda, (size_t)CT * d.d_k);
  w.kh = take(kda, (size_t)CT * d.d_k);
  w.kt = take(kda, (size_t)CT * d.d_k);
  w.all = take(kda, (size_t)NB * d.d_k);
  w.r = take(delta && backward, (size_t)CT * d.d_v);
  w.e = take(delta && backward, (size_t)CT * d.d_v);
  w.S = take(backward, (size_t)d.d_k * d.d_v);
  w.G = take(backward, (size_t)d.d_k * d.d_v);
  w.bytes = at;
  return w;
}

// A split 16 x 16 operand in the workspace: three 512-byte runs of 8 bytes per lane.
__device__ __forceinline__ void store_split(float* base, size_t block, int lane, const Split4& s) {
  uint2* p = reinterpret_cast<uint2*>(base) + block * 192 + lane;
  p[0] = s.h;
  p[64] = s.m;
  p[128] = s.l;
}
constexpr int ROW = 3 * SB;  // a block's part of ScanWork::row

struct ScanArgs {
  ScanPlan plan;
  int heads, d_v, num_slots;
  const int32_t* slot;
  const float* state_in;
  const void *q, *k, *v;
  const float *decay, *beta;
  float* state;  // forward: final states
  float* y;
  const float *dy, *dstate;
  void *dq, *dk, *dv;
  float *dlog, *dbeta, *dstate_in;
  ScanWork w;
  __device__ __forceinline__ size_t cell(int chunk, int head) const {
    return (size_t)head * plan.cap + chunk;
  }
};

// Products of the block's scalar gates for lane (m = lane % 16, g = lane / 16), whose own
// gate is a: in = a_0..a_m, out = a_{m+1}..a_15, and ratio[i] = a_{m+1}..a_{4g+i} (row
// 4g + i, column m; 1 on and above the diagonal).
__device__ __forceinline__ void gate_products(float a, int m, int g, float& in, float& out,
                                              float (&ratio)[4]) {
  in = out = 1.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) ratio[i] = 1.f;
#pragma unroll
  for (int l = 0; l < SB; ++l) {
    const float al = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(a), l));
    if (l <= m) in *= al;
    if (l > m) {
      out *= al;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (l <= 4 * g + i) ratio[i] *= al;
    }
  }
}

// Units to workgroups: the `parts` workgroups of a unit on one XCD (block b runs on XCD
// b % 8), so that its keys and queries are fetched into one L2.
__device__ __forceinline__ void unit_of(int b, int parts, int& unit, int& part) {
  unit = (b & 7) + 8 * (b / (8 * parts));
  part = (b >> 3) % parts;
}
inline unsigned unit_grid(long long units, int parts) {
  return (unsigned)((units + 7) / 8 * 8 * parts);
}

}  // namespace ssm
