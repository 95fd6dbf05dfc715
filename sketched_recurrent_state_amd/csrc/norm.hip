// norm.hip -- the norm of a layer's outputs in groups of channels with a gate, forward and backward
// (formulas in include/sketchssm.h).
//
// One pass: a lane holds 8 channels of a group, which stay in registers between the group's statistics
// and its result. A group of up to 512 channels is an aligned run of lanes of one wave, a wider one a
// workgroup of as many waves as it needs. Bound by HBM: 8192 rows of 32 groups of 128, fp32 in, bf16 gate and
// result, 44 us for 268 MB (6.1 TB/s, half of it reads of what a caller has just written); backward of 4096 rows of
// one group of 5,120 58 us for 294 MB (5.1 TB/s).
#include "layer.hpp"
#include "launch.hpp"

namespace ssm {

namespace {

constexpr int NT = 256;     // threads of a workgroup of narrow groups
constexpr int SMALL = 512;  // the widest group of one wave
constexpr int MOST = 1024;  // threads of a workgroup of one wide group (8192 channels)
constexpr long long kMostBlocks = 1 << 21;  // keeps a grid below 2^32 threads; then a workgroup takes several

// Lanes of a group: a power of two of them in a wave, or (0) a workgroup.
inline int group_lanes(int width) {
  if (width > SMALL) return 0;
  int l = 2;
  while (8 * l < width) l *= 2;
  return l;
}
inline int threads_of(int width) { return width > SMALL ? (width + SMALL - 1) / SMALL * 64 : NT; }

// Sum over the lanes of a group (L >= 2 aligned lanes of a wave), or over the workgroup (L = 0;
// all threads call it). N values at once.
template <int L, int N>
__device__ __forceinline__ void group_sum(float (&x)[N], float (*sw)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] += dpp<DPP_QUAD_1032>(x[i]);
    if constexpr (L == 0 || L >= 4) x[i] += dpp<DPP_QUAD_2301>(x[i]);
    if constexpr (L == 0 || L >= 8) x[i] += dpp<DPP_HALF_MIRROR>(x[i]);
    if constexpr (L == 0 || L >= 16) x[i] += dpp<DPP_ROR8>(x[i]);
    if constexpr (L == 0 || L >= 32) x[i] = xsum16(x[i]);
    if constexpr (L == 0 || L >= 64) x[i] = xsum32(x[i]);
  }
  if constexpr (L == 0) {
    __syncthreads();  // the last call's reads are done
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) sw[threadIdx.x >> 6][i] = x[i];
    __syncthreads();
    const int waves = blockDim.x >> 6;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = sw[0][i];
    for (int w = 1; w < waves; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] += sw[w][i];
  }
}

__device__ __forceinline__ float gate_of(float z, bool sig) {
  const float s = sigmoid(z);
  return sig ? s : z * s;
}
// the gate and its derivative
__device__ __forceinline__ float gate_of(float z, bool sig, float& slope) {
  const float s = sigmoid(z);
  slope = sig ? s * (1.f - s) : s * fmaf(z, 1.f - s, 1.f);
  return sig ? s : z * s;
}

// Mean (0 where not centred) and 1 / sqrt(var + eps) of a group's u, which is 0 in lanes without channels.
template <int L>
__device__ __forceinline__ void group_stats(const NormArgs& a, bool on, const float (&u)[8], float (*sw)[1],
                                            float& mean, float& r) {
  const float inv = 1.f / (float)a.width;
  mean = 0.f;
  if (a.centred) {
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < 8; ++i) s[0] += u[i];
    group_sum<L>(s, sw);
    mean = s[0] * inv;
  }
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < 8; ++i) s[0] = fmaf(u[i] - mean, u[i] - mean, s[0]);
  s[0] = on ? s[0] : 0.f;
  group_sum<L>(s, sw);
  r = __builtin_amdgcn_rsqf(fmaf(s[0], inv, a.eps));
}

__device__ __forceinline__ void load_weights(const float* p, size_t at, float otherwise, float (&w)[8]) {
  if (p) {
    Vec<float, 8>::load(p + at, w);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = otherwise;
  }
}

// A lane's place: its group's number in the workgroup and its first channel.
template <int L>
struct Place {
  static constexpr int PER = L == 0 ? 1 : NT / (L == 0 ? 1 : L);  // groups of a workgroup
  int group, c;
  bool on;  // lanes past the group's width read its first channels, and do not count
  __device__ __forceinline__ Place(int width) {
    const int lane = L == 0 ? threadIdx.x : threadIdx.x % (L == 0 ? 1 : L);
    group = L == 0 ? 0 : threadIdx.x / (L == 0 ? 1 : L);
    on = 8 * lane < width;
    c = on ? 8 * lane : 0;
  }
};

template <typename T>
__device__ __forceinline__ void unpack_on(const Packed<T, 8>& raw, bool on, float (&x)[8]) {
  raw.unpack(x);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = on ? x[i] : 0.f;
}

template <int L, int GATE, typename TX, typename T>
__global__ void __launch_bounds__(L == 0 ? MOST : NT) norm_kernel(const NormArgs a) {
  __shared__ float sw[MOST / 64][1];
  const Place<L> k(a.width);
  long long item = (long long)blockIdx.x * k.PER + k.group;
  for (; item < (long long)a.rows * a.groups; item += (long long)gridDim.x * k.PER) {
    const int row = (int)(item / a.groups), g = (int)(item % a.groups);
    const size_t at = (size_t)g * a.width + k.c, wat = a.shared ? k.c : at;
    Packed<TX, 8> rx;
    Packed<T, 8> rz;
    rx.load(a.x.row<TX>(row) + at);
    if constexpr (GATE != SSM_GATE_NONE) rz.load(a.z.row<T>(row) + at);
    float x[8], gate[8], w[8], b[8], o[8];
    load_weights(a.weight, wat, 1.f, w);
    load_weights(a.bias, wat, 0.f, b);
    unpack_on(rx, k.on, x);
    if constexpr (GATE != SSM_GATE_NONE) {
      unpack_on(rz, k.on, gate);
#pragma unroll
      for (int i = 0; i < 8; ++i) gate[i] = gate_of(gate[i], a.sigmoid);
    }
    if constexpr (GATE == SSM_GATE_BEFORE) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= gate[i];
    }
    float mean, r;
    group_stats<L>(a, k.on, x, sw, mean, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      o[i] = fmaf((x[i] - mean) * r, w[i], b[i]);
      if constexpr (GATE == SSM_GATE_AFTER) o[i] *= gate[i];
    }
    if (k.on) store8(a.out.out<T>(row) + at, o);
  }
}

// Backward: a lane keeps its channels (of one group, or of every group where weights are shared) over
// the rows that its workgroup takes, with their sums for the weights in registers. The next row is read
// while this one's sums go through the lanes.
template <int L, int GATE, typename TX, typename T>
__global__ void __launch_bounds__(L == 0 ? MOST : NT) norm_backward_kernel(const NormArgs a) {
  __shared__ float sw[MOST / 64][1], sw2[MOST / 64][2];
  const Place<L> k(a.width);
  constexpr int PER = Place<L>::PER;
  // items: (row, group) where weights are shared, else the rows of one group
  const int g0 = a.shared ? 0 : (int)blockIdx.x * PER + k.group;
  const long long items = a.shared ? (long long)a.rows * a.groups : (g0 < a.groups ? a.rows : 0);
  const int first = a.shared ? (int)blockIdx.y * PER + k.group : blockIdx.y;
  const int stride = a.shared ? a.parts * PER : a.parts;
  const size_t wat = (size_t)(a.shared || g0 >= a.groups ? 0 : g0) * a.width + k.c;
  float w[8], b[8], dw[8], db[8];
  load_weights(a.weight, wat, 1.f, w);
  if constexpr (GATE == SSM_GATE_AFTER) load_weights(a.bias, wat, 0.f, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = db[i] = 0.f;
  const float inv = 1.f / (float)a.width;
  Packed<TX, 8> rx;
  Packed<T, 8> rz, rd;
  const auto place = [&](long long item, int& row, size_t& at) {
    row = a.shared ? (int)(item / a.groups) : (int)item;
    at = a.shared ? (size_t)(item % a.groups) * a.width + k.c : wat;
  };
  const auto fetch = [&](long long item) {
    int row;
    size_t at;
    place(item, row, at);
    rx.load(a.x.row<TX>(row) + at);
    rd.load(a.dout.row<T>(row) + at);
    if constexpr (GATE != SSM_GATE_NONE) rz.load(a.z.row<T>(row) + at);
  };
  if (first < items) fetch(first);
  for (long long item = first; item < items; item += stride) {
    int row;
    size_t at;
    place(item, row, at);
    float x[8], u[8], gate[8], slope[8], d[8], dz[8];
    unpack_on(rx, k.on, x);
    unpack_on(rd, k.on, d);
    if constexpr (GATE != SSM_GATE_NONE) {
      unpack_on(rz, k.on, gate);
#pragma unroll
      for (int i = 0; i < 8; ++i) gate[i] = gate_of(gate[i], a.sigmoid, slope[i]);
    }
    if (item + stride < items) fetch(item + stride);
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = GATE == SSM_GATE_BEFORE ? x[i] * gate[i] : x[i];
    float mean, r;
    group_stats<L>(a, k.on, u, sw, mean, r);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = (u[i] - mean) * r;
      float o = d[i];
      if constexpr (GATE == SSM_GATE_AFTER) {
        dz[i] = o * fmaf(n, w[i], b[i]) * slope[i];
        o *= gate[i];
      }
      u[i] = n;
      dw[i] = fmaf(o, n, dw[i]);  // d is 0 in lanes without channels
      db[i] += o;
      d[i] = o * w[i];
      s[0] = fmaf(d[i], n, s[0]);
      s[1] += d[i];
    }
    group_sum<L>(s, sw2);
    const float sn = s[0] * inv, s1 = a.centred ? s[1] * inv : 0.f;
    float dx[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float du = r * (d[i] - u[i] * sn - s1);
      if constexpr (GATE == SSM_GATE_BEFORE) {
        dz[i] = du * x[i] * slope[i];
        dx[i] = du * gate[i];
      } else {
        dx[i] = du;
      }
    }
    if (k.on) {
      store8(a.dx.out<TX>(row) + at, dx);
      if constexpr (GATE != SSM_GATE_NONE) store8(a.dz.out<T>(row) + at, dz);
    }
  }
  // the workgroup's sums: those of its other places join the first's where weights are shared
  const size_t cols = (size_t)(a.shared ? 1 : a.groups) * a.width;
  float* out = a.partial + (size_t)blockIdx.y * 2 * cols;
  if constexpr (L != 0) {
    if (a.shared) {
      __shared__ float sums[2][SMALL];
      for (int p = 0; p < PER; ++p) {
        if (k.group == p && k.on)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            sums[0][k.c + i] = dw[i] + (p ? sums[0][k.c + i] : 0.f);
            sums[1][k.c + i] = db[i] + (p ? sums[1][k.c + i] : 0.f);
          }
        __syncthreads();
      }
      for (int c = threadIdx.x; c < a.width; c += NT) {
        out[c] = sums[0][c];
        out[cols + c] = sums[1][c];
      }
      return;
    }
  }
  if (!k.on || g0 >= a.groups) return;
  store8(out + wat, dw);
  store8(out + cols + wat, db);
}

// The sums over the rows of partial sums, in a fixed order.
constexpr int RY = 16;
__global__ void __launch_bounds__(64 * RY)
norm_sum_kernel(const float* __restrict__ partial, int rows, int cols, float* __restrict__ dweight,
                float* __restrict__ dbias) {
  __shared__ float part[RY][64];
  const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + x, n = dbias ? 2 * cols : cols;
  float s = 0.f;
  if (col < n) {
#pragma unroll 8
    for (int r = y; r < rows; r += RY) s += partial[(size_t)r * 2 * cols + col];
  }
  part[y][x] = s;
  __syncthreads();
  if (y > 0 || col >= n) return;
#pragma unroll
  for (int i = 1; i < RY; ++i) s += part[i][x];
  if (col < cols) dweight[col] = s;
  else dbias[col - cols] = s;
}

// Calls f(lanes of a group (0: a workgroup), gate, x type, in type).
template <typename F>
hipError_t norm_dispatch(const ssm_norm_dims& d, F&& f) {
  auto types = [&](auto L, auto G) -> hipError_t {
    if (d.x_dtype == SSM_IN_BF16) {
      if (d.in_dtype == SSM_IN_BF16) return f(L, G, type_tag<uint16_t>{}, type_tag<uint16_t>{});
      return f(L, G, type_tag<uint16_t>{}, type_tag<float>{});
    }
    if (d.in_dtype == SSM_IN_BF16) return f(L, G, type_tag<float>{}, type_tag<uint16_t>{});
    return f(L, G, type_tag<float>{}, type_tag<float>{});
  };
  auto gates = [&](auto L) -> hipError_t {
    switch (d.gate) {
      case SSM_GATE_NONE: return types(L, std::integral_constant<int, SSM_GATE_NONE>{});
      case SSM_GATE_AFTER: return types(L, std::integral_constant<int, SSM_GATE_AFTER>{});
      case SSM_GATE_BEFORE: return types(L, std::integral_constant<int, SSM_GATE_BEFORE>{});
    }
    return hipErrorInvalidValue;
  };
  switch (group_lanes(d.width)) {
    case 0: return gates(std::integral_constant<int, 0>{});
    case 2: return gates(std::integral_constant<int, 2>{});
    case 4: return gates(std::integral_constant<int, 4>{});
    case 8: return gates(std::integral_constant<int, 8>{});
    case 16: return gates(std::integral_constant<int, 16>{});
    case 32: return gates(std::integral_constant<int, 32>{});
    case 64: return gates(std::integral_constant<int, 64>{});
  }
  return hipErrorInvalidValue;
}

// Workgroups over the groups of a row, and over the rows: as many as the GPU holds at once, so that each
// keeps its sums for as many rows as it can and all end together. 4096 rows, fp32 x, bf16 gate: of 5,120
// channels (10 waves a workgroup) 256 of them 55 us, 512: 59, 768: 62, 1024: 68; of 32 groups of 128 (4 waves)
// 256: 50, 512: 36, 768: 34.
struct BackwardGrid {
  int tiles, parts;
};
BackwardGrid backward_grid(const ssm_norm_dims& d, int rows) {
  const int lanes = group_lanes(d.width), per = lanes ? NT / lanes : 1;
  BackwardGrid b;
  b.tiles = d.shared ? 1 : (d.groups + per - 1) / per;
  const long long items = d.shared ? ((long long)rows * d.groups + per - 1) / per : rows;
  const int waves = threads_of(d.width) / 64;
  long long parts = 256 * ((lanes ? 12 : 16) / waves) / b.tiles;  // registers: 3 and 4 waves a SIMD
  if (parts > items) parts = items;
  b.parts = parts < 1 ? 1 : (int)parts;
  return b;
}

}  // namespace

size_t norm_workspace(const ssm_norm_dims& d, int rows) {
  return (size_t)backward_grid(d, rows).parts * 2 * (d.shared ? 1 : d.groups) * d.width * sizeof(float);
}

hipError_t launch_norm(const ssm_norm_dims& d, const NormArgs& a, hipStream_t stream) {
  return norm_dispatch(d, [&](auto L, auto G, auto TX, auto T) {
    constexpr int l = decltype(L)::value, per = Place<l>::PER;
    const long long blocks = ((long long)a.rows * a.groups + per - 1) / per;
    hipLaunchKernelGGL((norm_kernel<l, decltype(G)::value, typename decltype(TX)::type,
                                    typename decltype(T)::type>),
                       dim3((unsigned)(blocks < kMostBlocks ? blocks : kMostBlocks)),
                       dim3(threads_of(d.width)), 0, stream, a);
    return hipGetLastError();
  });
}

hipError_t launch_norm_backward(const ssm_norm_dims& d, NormArgs& a, hipStream_t stream) {
  const BackwardGrid b = backward_grid(d, a.rows);
  a.parts = b.parts;
  return norm_dispatch(d, [&](auto L, auto G, auto TX, auto T) {
    hipLaunchKernelGGL((norm_backward_kernel<decltype(L)::value, decltype(G)::value,
                                             typename decltype(TX)::type, typename decltype(T)::type>),
                       dim3((unsigned)b.tiles, (unsigned)b.parts), dim3(threads_of(d.width)), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int cols = (a.shared ? 1 : a.groups) * a.width;
    hipLaunchKernelGGL(norm_sum_kernel, dim3((2 * cols + 63) / 64), dim3(64 * RY), 0, stream,
                       a.partial, a.parts, cols, a.dweight, a.dbias);
    return hipGetLastError();
  });
}

}  // namespace ssm
