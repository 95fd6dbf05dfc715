// scan_table.hpp -- what the scan kernels read from a packed batch's plan, and the checks that keep
// every access within the arrays whatever the plan holds. Plain C++ but for the attributes, so that
// the checks can be run without a device.
#pragma once

#include <stdint.h>

namespace ssm {

constexpr int CT = 64;  // tokens of a chunk (an entry of the chunk table)

// The plan of ssm_scan_plan: [seq_start (n + 1) | chunk_start (n + 1) | chunk_seq (cap)].
struct ScanPlan {
  const int32_t* p;
  int seqs, total, cap;
  __host__ __device__ __forceinline__ int start(int s) const { return p[s]; }
  __host__ __device__ __forceinline__ int chunk(int s) const { return p[seqs + 1 + s]; }
  // Chunk c's first token and token count; false where c holds none. Whatever the
  // table holds, the tokens named are inside [0, total).
  __host__ __device__ __forceinline__ bool cell(int c, int& tok, int& count) const {
    const int s = p[2 * (seqs + 1) + c];
    if (s < 0 || s >= seqs) return false;
    const long long k = (long long)c - chunk(s);
    const long long b = start(s) + CT * k, e = start(s + 1);
    if (k < 0 || b < 0 || b >= e || e > total || start(s) < 0) return false;
    tok = (int)b;
    count = (int)(e - b < CT ? e - b : CT);
    return true;
  }
  // Chunk c's sequence, that sequence's first token and length, and the chunk's place in it; false
  // where cell() is.
  __host__ __device__ __forceinline__ bool locate(int c, int& s, int& first, int& len, int& pos) const {
    int tok, count;
    if (!cell(c, tok, count)) return false;
    s = p[2 * (seqs + 1) + c];
    first = start(s);
    len = start(s + 1) - first;
    pos = tok - first;
    return true;
  }
  // Sequence s's first token, length and first chunk; false where the table is not a plan's.
  __host__ __device__ __forceinline__ bool sequence(int s, int& tok, int& len, int& first) const {
    const int b = start(s), e = start(s + 1);
    first = chunk(s);
    if (b < 0 || e < b || e > total || first < 0) return false;
    tok = b;
    len = e - b;
    return (long long)first + (len + CT - 1) / CT <= cap;
  }
};

// Whether a sequence of len > 0 tokens whose first chunk is entry c goes on behind its group, the entries before e1.
__host__ __device__ __forceinline__ bool goes_on(int c, int len, int e1, int cap) {
  return e1 < cap && c + (len - 1) / CT >= e1;
}

// The gradients of the selective recurrence keep the state before every KT tokens of a sequence but its first. The
// place of that before token pos (a multiple of KT, not 0) of the sequence whose first token is `first`: no two
// sequences' meet, whatever their lengths, and all are below kept_places(tokens of the batch).
constexpr int KT = 8;
__host__ __device__ __forceinline__ int kept_place(int first, int pos) { return first / KT + pos / KT - 1; }
inline int kept_places(int total) { return total / KT + 1; }

inline int scan_capacity(int total, int seqs) { return total / CT + seqs; }

}  // namespace ssm
