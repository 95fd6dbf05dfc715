// plan.hip -- index arrays built on the device from request lengths: the chunk table of
// a packed batch of sequences (for the scan kernels) and the window positions of a
// serving step (for ssm_decode_step_varlen).
//
// Both are a few hundred kilobytes at most, so a launch costs more than the bytes. Each
// is one launch: instead of passing prefix sums from workgroup to workgroup (which
// would need a second launch or a wait), every workgroup sums what lies before its part
// again: 8 us for a batch of hundreds of sequences and 16 us for 20,000 (8 us is a launch's own
// time in a queue), 18 us for 200,000 rows of a window plan. The repeated sums grow with the
// square of the number: 180 us for 200,000 sequences (a plan serves every layer's passes, which
// take milliseconds then), 88 us for a million rows.
#include "common.hpp"
#include "launch.hpp"
#include "scan.hpp"

namespace ssm {

namespace {

constexpr int PT = 1024;  // threads of a workgroup, and entries of the chunk table it fills
constexpr int PW = PT / 64;

// Exclusive sum over the workgroup's threads; `total` is the sum of all. sw: PW values.
template <typename I>
__device__ __forceinline__ I wave_inclusive(I x, int lanes) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < lanes; o <<= 1) {
    const I y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  return x;
}
template <typename I>
__device__ __forceinline__ I before_wave(const I* sw, I& total) {  // the waves' sums, by every wave
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const I w = wave_inclusive(lane < PW ? sw[lane] : I(0), PW);
  total = __shfl(w, PW - 1);
  const I before = __shfl(w, wave > 0 ? wave - 1 : 0);
  return wave > 0 ? before : I(0);
}
template <typename I>
__device__ __forceinline__ I block_exclusive(I x, I* sw, I& total) {
  const I s = wave_inclusive(x, 64);
  __syncthreads();  // the last call's reads of sw are done
  if ((threadIdx.x & 63) == 63) sw[threadIdx.x >> 6] = s;
  __syncthreads();
  return before_wave(sw, total) + s - x;
}
// The same for two values at once.
__device__ __forceinline__ void block_exclusive(int64_t& t, int& c, int64_t* sw64, int* sw32,
                                                int64_t& all_t, int& all_c) {
  const int64_t st = wave_inclusive(t, 64);
  const int sc = wave_inclusive(c, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) {
    sw64[threadIdx.x >> 6] = st;
    sw32[threadIdx.x >> 6] = sc;
  }
  __syncthreads();
  t = before_wave(sw64, all_t) + st - t;
  c = before_wave(sw32, all_c) + sc - c;
}

constexpr int PS = 4;            // sequences of a thread
constexpr int TILE = PT * PS;    // sequences of a tile

// Workgroup b fills the chunk table's entries [b * PT, (b + 1) * PT) and the starts of the
// tiles b, b + gridDim.x, .. of the sequences. A thread holds PS consecutive sequences.
__global__ void __launch_bounds__(PT)
scan_plan_kernel(const int32_t* __restrict__ lengths, int n, int total, int cap,
                 int32_t* __restrict__ plan) {
  __shared__ int64_t sw64[PW];
  __shared__ int32_t sw32[PW], owner[PT];
  const int tid = threadIdx.x, e0 = blockIdx.x * PT;
  int32_t* seq_start = plan;
  int32_t* chunk_start = plan + n + 1;
  int32_t* chunk_seq = plan + 2 * (n + 1);
  owner[tid] = -1;
  int64_t tokens = 0;  // of the tiles before
  int chunks = 0;
  const int grid = gridDim.x, tiles = (n + TILE - 1) / TILE;
  for (int tile = 0; tile < tiles; ++tile) {
    // done: the table's part is full, and no tile's starts are left to write
    const int left = tiles - 1 - (int)blockIdx.x;
    if (chunks >= e0 + PT && (left < 0 || tile > (int)blockIdx.x + left / grid * grid)) break;
    const int s0 = tile * TILE + tid * PS;
    int len[PS];
    int64_t sum = 0;
    int mine = 0;
#pragma unroll
    for (int i = 0; i < PS; ++i) {
      const int l = s0 + i < n ? lengths[s0 + i] : 0;
      len[i] = l > 0 ? l : 0;
      sum += len[i];
      mine += (int)(((int64_t)len[i] + CT - 1) / CT);
    }
    int64_t at = sum, all;
    int c = mine, all_chunks;
    block_exclusive(at, c, sw64, sw32, all, all_chunks);
    at += tokens;
    tokens += all;
    // lengths past the arrays' end are cut
    int start[PS], nc[PS], kept = 0;
#pragma unroll
    for (int i = 0; i < PS; ++i) {
      const int64_t end = at + len[i];
      start[i] = (int)(at < total ? at : total);
      nc[i] = (int)(((end < total ? end : total) - start[i] + CT - 1) / CT);
      kept += nc[i];
      at = end;
    }
    if (tokens > total) c = block_exclusive(kept, sw32, all_chunks);
    c += chunks;
    chunks += all_chunks;
    const bool writes = tile % grid == (int)blockIdx.x;
#pragma unroll
    for (int i = 0; i < PS; ++i) {
      const int s = s0 + i;
      if (s >= n) break;
      if (writes) {
        seq_start[s] = start[i];
        chunk_start[s] = c;
        if (s == n - 1) {
          seq_start[n] = (int)(at < total ? at : total);
          chunk_start[n] = c + nc[i];
        }
      }
      // the sequence's first entry of this workgroup's part
      const int first = c > e0 ? c : e0;
      if (nc[i] > 0 && c + nc[i] > e0 && first < e0 + PT) owner[first - e0] = s;
      c += nc[i];
    }
  }
  __syncthreads();
  // an entry belongs to the last sequence that starts at or before it
  const int lane = tid & 63, wave = tid >> 6;
  int s = owner[tid];
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(s, o);
    if (lane >= o) s = max(s, y);
  }
  if (lane == 63) sw32[wave] = s;
  __syncthreads();
  for (int w = 0; w < wave; ++w) s = max(s, sw32[w]);
  const int entry = e0 + tid;
  if (entry < cap) chunk_seq[entry] = entry < chunks ? s : -1;
}

// L / W and "L is the last of its window" for any int32 L and W <= 16.
// Quotient of L >= 0: magic = ceil(2^(31 + s) / W) with 2^s >= W exceeds the quotient's multiple
// by less than W / 2^(31 + s) per unit of L, too little to reach the next integer.
// Last (W divides x = L + 1): with W = 2^k odd, x times the inverse of the odd part modulo 2^32,
// rotated right by k, is x / W for the multiples of W and at least 2^32 / W for the others. The
// window's last L >= 0 are those with 1 <= x / W <= 2^31 / W. Half the instructions of a quotient.
struct WindowDiv {
  uint32_t magic, inverse, limit;
  int shift, rotate, window;
  __device__ __forceinline__ int div(int x) const {
    return window == 1 ? x : (int)(__umulhi((uint32_t)x, magic) >> shift);
  }
  __device__ __forceinline__ bool last(int l) const {
    const uint32_t x = ((uint32_t)l + 1u) * inverse;
    return __builtin_amdgcn_alignbit(x, x, rotate) - 1u < limit;
  }
};

// Workgroup b plans rows [b * PT * PS, ..): the listed rows before them are counted from
// the lengths again.
__global__ void __launch_bounds__(PT)
window_plan_kernel(const int32_t* __restrict__ lengths, int n, WindowDiv w,
                   int32_t* __restrict__ tau, int32_t* __restrict__ parity,
                   int32_t* __restrict__ rows, int32_t* __restrict__ count) {
  __shared__ int sw[PW];
  const int tid = threadIdx.x, r0 = blockIdx.x * TILE;
  int before = 0, total;
#pragma unroll 8
  for (int r = tid; r < r0; r += PT) before += w.last(lengths[r]);
  block_exclusive(before, sw, total);
  const int listed = total;
  int l[PS], mine = 0;
#pragma unroll
  for (int i = 0; i < PS; ++i) {
    const int r = r0 + tid * PS + i;
    l[i] = r < n ? lengths[r] : -1;
    mine += w.last(l[i]);
  }
  int at = listed + block_exclusive(mine, sw, total);
  // the rows not listed fill the list's tail with -1: this part's have the places that
  // follow when the list's places are counted from its end
  int tail = n - 1 - (r0 + tid * PS - at);
#pragma unroll
  for (int i = 0; i < PS; ++i) {
    const int r = r0 + tid * PS + i;
    if (r >= n) break;
    const int q = l[i] >= 0 ? w.div(l[i]) : 0;
    tau[r] = l[i] >= 0 ? l[i] - q * w.window + 1 : 0;
    parity[r] = q & 1;
    if (w.last(l[i])) rows[at++] = r;
    else rows[tail--] = -1;
    if (r == n - 1) *count = at;
  }
}

}  // namespace

hipError_t launch_scan_plan(const int32_t* lengths, int n, int total, int32_t* plan,
                            hipStream_t stream) {
  const int cap = scan_capacity(total, n);
  hipLaunchKernelGGL(scan_plan_kernel, dim3((cap + PT - 1) / PT), dim3(PT), 0, stream, lengths, n,
                     total, cap, plan);
  return hipGetLastError();
}

hipError_t launch_window_plan(const int32_t* lengths, int n, int window, int32_t* tau,
                              int32_t* parity, int32_t* rows, int32_t* count, hipStream_t stream) {
  WindowDiv w{};
  w.window = window;
  uint32_t odd = (uint32_t)window;
  for (; !(odd & 1); odd >>= 1) ++w.rotate;
  w.inverse = 1;
  for (int i = 0; i < 5; ++i) w.inverse *= 2 - odd * w.inverse;  // Newton: correct bits double
  w.limit = (1u << 31) / (uint32_t)window;
  int s = 0;
  while ((1 << s) < window) ++s;
  if (window > 1) {
    w.magic = (uint32_t)(((1ull << (31 + s)) + window - 1) / window);
    w.shift = s - 1;
  }
  hipLaunchKernelGGL(window_plan_kernel, dim3((n + TILE - 1) / TILE), dim3(PT), 0, stream, lengths,
                     n, w, tau, parity, rows, count);
  return hipGetLastError();
}

}  // namespace ssm
