// norm.hip -- the norm of a layer's outputs in groups of channels with a gate, forward and backward
// (formulas in include/sketchssm.h).
//
// One pass: a group's values stay in registers between its statistics and its result. A group of
// up to 512 channels is an aligned run of lanes of one wave (8 channels a lane), a wider one a
// workgroup. Bound by HBM.
#include "layer.hpp"
#include "launch.hpp"

namespace ssm {

namespace {

constexpr int NT = 256;
constexpr int SMALL = 512;  // the widest group of one wave
constexpr long long kMostBlocks = 1 << 23;  // keeps a grid below 2^32 threads; then a workgroup takes several

// Lanes of a group of the first kind.
inline int group_lanes(int width) {
  int l = 2;
  while (8 * l < width) l *= 2;
  return l;
}

// Sum over the lanes of a group (L >= 2 aligned lanes of a wave), or over the workgroup (L = 0;
// all threads call it).
template <int L>
__device__ __forceinline__ float group_sum(float x, float* sw) {
  x += dpp<DPP_QUAD_1032>(x);
  if constexpr (L == 0 || L >= 4) x += dpp<DPP_QUAD_2301>(x);
  if constexpr (L == 0 || L >= 8) x += dpp<DPP_HALF_MIRROR>(x);
  if constexpr (L == 0 || L >= 16) x += dpp<DPP_ROR8>(x);
  if constexpr (L == 0 || L >= 32) x = xsum16(x);
  if constexpr (L == 0 || L >= 64) x = xsum32(x);
  if constexpr (L == 0) {
    __syncthreads();  // the last call's reads are done
    if ((threadIdx.x & 63) == 0) sw[threadIdx.x >> 6] = x;
    __syncthreads();
    x = sw[0];
#pragma unroll
    for (int i = 1; i < NT / 64; ++i) x += sw[i];
  }
  return x;
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

// A lane's channels of a group: V runs of 8. The first is at 8 * lane, the next a workgroup's
// channels further.
template <int V>
struct Cols {
  int c[V];
  bool on[V];
  __device__ __forceinline__ Cols(int lane, int width) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      c[v] = 8 * (lane + v * NT);
      on[v] = c[v] < width;
      if (!on[v]) c[v] = 0;
    }
  }
};

// Mean (0 where not centred) and 1 / sqrt(var + eps) of a group's u, 0 in lanes without channels.
template <int L, int V>
__device__ __forceinline__ void group_stats(const NormArgs& a, const Cols<V>& k, const float (&u)[V][8],
                                            float* sw, float& mean, float& r) {
  const float inv = 1.f / (float)a.width;
  mean = 0.f;
  if (a.centred) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += u[v][i];
    mean = group_sum<L>(s, sw) * inv;
  }
  float s = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (k.on[v])
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(u[v][i] - mean, u[v][i] - mean, s);
  r = __builtin_amdgcn_rsqf(fmaf(group_sum<L>(s, sw), inv, a.eps));
}

template <int V>
__device__ __forceinline__ void load_weights(const float* p, const Cols<V>& k, size_t at, float otherwise,
                                             float (&w)[V][8]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (p) {
      Vec<float, 8>::load(p + at + k.c[v], w[v]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[v][i] = otherwise;
    }
  }
}

// Loads x (and z): 0 in lanes without channels.
template <typename T, int V>
__device__ __forceinline__ void load_cols(const T* p, const Cols<V>& k, float (&x)[V][8]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    Packed<T, 8> raw = {};
    if (k.on[v]) raw.load(p + k.c[v]);
    raw.unpack(x[v]);
  }
}

template <int L, int V, typename TX, typename T>
__global__ void __launch_bounds__(NT) norm_kernel(const NormArgs a) {
  __shared__ float sw[NT / 64];
  constexpr int PER = L == 0 ? 1 : NT / (L == 0 ? 1 : L);  // groups of a workgroup
  const int lane = L == 0 ? threadIdx.x : threadIdx.x % (L == 0 ? 1 : L);
  const Cols<V> k(lane, a.width);
  long long item = (long long)blockIdx.x * PER + (L == 0 ? 0 : threadIdx.x / (L == 0 ? 1 : L));
  for (; item < (long long)a.rows * a.groups; item += (long long)gridDim.x * PER) {
    const int row = (int)(item / a.groups), g = (int)(item % a.groups);
    const size_t at = (size_t)g * a.width, wat = a.shared ? 0 : at;
    float x[V][8], gate[V][8], w[V][8], b[V][8];
    load_cols<TX, V>(a.x.row<TX>(row) + at, k, x);
    if (a.gate != SSM_GATE_NONE) {
      load_cols<T, V>(a.z.row<T>(row) + at, k, gate);
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) gate[v][i] = gate_of(gate[v][i], a.sigmoid);
    }
    load_weights<V>(a.weight, k, wat, 1.f, w);
    load_weights<V>(a.bias, k, wat, 0.f, b);
    if (a.gate == SSM_GATE_BEFORE) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[v][i] *= gate[v][i];
    }
    float mean, r;
    group_stats<L, V>(a, k, x, sw, mean, r);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!k.on[v]) continue;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[i] = fmaf((x[v][i] - mean) * r, w[v][i], b[v][i]);
        if (a.gate == SSM_GATE_AFTER) o[i] *= gate[v][i];
      }
      store8(a.out.out<T>(row) + at + k.c[v], o);
    }
  }
}

// Backward: a lane keeps its channels (of one group, or of every group where weights are shared) over
// the rows that its workgroup takes, with their sums for the weights in registers.
template <int L, int V, typename TX, typename T>
__global__ void __launch_bounds__(NT) norm_backward_kernel(const NormArgs a) {
  __shared__ float sw[NT / 64];
  constexpr int PER = L == 0 ? 1 : NT / (L == 0 ? 1 : L);
  const int lane = L == 0 ? threadIdx.x : threadIdx.x % (L == 0 ? 1 : L);
  const int place = L == 0 ? 0 : threadIdx.x / (L == 0 ? 1 : L);
  const Cols<V> k(lane, a.width);
  // items: (row, group) where weights are shared, else the rows of one group
  const int wgroups = a.shared ? 1 : a.groups;
  const int tile = blockIdx.x, g0 = a.shared ? 0 : tile * PER + place;
  const long long items = a.shared ? (long long)a.rows * a.groups : (g0 < a.groups ? a.rows : 0);
  const int first = a.shared ? (int)blockIdx.y * PER + place : blockIdx.y;
  const int stride = a.shared ? a.parts * PER : a.parts;
  const size_t wat = a.shared ? 0 : (size_t)(g0 < a.groups ? g0 : 0) * a.width;
  float w[V][8], b[V][8], dw[V][8], db[V][8];
  load_weights<V>(a.weight, k, wat, 1.f, w);
  load_weights<V>(a.bias, k, wat, 0.f, b);
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[v][i] = db[v][i] = 0.f;
  const float inv = 1.f / (float)a.width;
  for (long long item = first; item < items; item += stride) {
    const int row = a.shared ? (int)(item / a.groups) : (int)item;
    const size_t at = a.shared ? (size_t)(item % a.groups) * a.width : wat;
    float x[V][8], u[V][8], gate[V][8], slope[V][8], d[V][8];
    load_cols<TX, V>(a.x.row<TX>(row) + at, k, x);
    load_cols<T, V>(a.dout.row<T>(row) + at, k, d);
    if (a.gate != SSM_GATE_NONE) {
      load_cols<T, V>(a.z.row<T>(row) + at, k, gate);
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) gate[v][i] = gate_of(gate[v][i], a.sigmoid, slope[v][i]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        u[v][i] = a.gate == SSM_GATE_BEFORE ? x[v][i] * gate[v][i] : x[v][i];
    float mean, r;
    group_stats<L, V>(a, k, u, sw, mean, r);
    float dz[V][8], sn = 0.f, s1 = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = (u[v][i] - mean) * r;
        float o = d[v][i];
        if (a.gate == SSM_GATE_AFTER) {
          dz[v][i] = o * fmaf(n, w[v][i], b[v][i]) * slope[v][i];
          o *= gate[v][i];
        }
        u[v][i] = n;
        if (k.on[v]) {
          dw[v][i] = fmaf(o, n, dw[v][i]);
          db[v][i] += o;
        }
        d[v][i] = o * w[v][i];
        if (k.on[v]) {
          sn = fmaf(d[v][i], n, sn);
          s1 += d[v][i];
        }
      }
    sn = group_sum<L>(sn, sw) * inv;
    s1 = a.centred ? group_sum<L>(s1, sw) * inv : 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!k.on[v]) continue;
      float dx[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float du = r * (d[v][i] - u[v][i] * sn - s1);
        if (a.gate == SSM_GATE_BEFORE) {
          dz[v][i] = du * x[v][i] * slope[v][i];
          dx[i] = du * gate[v][i];
        } else {
          dx[i] = du;
        }
      }
      store8(a.dx.out<TX>(row) + at + k.c[v], dx);
      if (a.gate != SSM_GATE_NONE) store8(a.dz.out<T>(row) + at + k.c[v], dz[v]);
    }
  }
  // the workgroup's sums: those of its other places join the first's where weights are shared
  const size_t cols = (size_t)wgroups * a.width;
  float* out = a.partial + (size_t)blockIdx.y * 2 * cols;
  if constexpr (L != 0) {
    if (a.shared) {
      __shared__ float sums[2][SMALL];
      for (int p = 0; p < PER; ++p) {
        if (place == p && k.on[0])
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            sums[0][k.c[0] + i] = dw[0][i] + (p ? sums[0][k.c[0] + i] : 0.f);
            sums[1][k.c[0] + i] = db[0][i] + (p ? sums[1][k.c[0] + i] : 0.f);
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
  if (!a.shared && g0 >= a.groups) return;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (k.on[v]) {
      store8(out + wat + k.c[v], dw[v]);
      store8(out + cols + wat + k.c[v], db[v]);
    }
}

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

// Calls f(L, V, x type, in type): lanes of a group (0: a workgroup) and runs of 8 channels a lane.
template <typename F>
hipError_t norm_dispatch(const ssm_norm_dims& d, F&& f) {
  auto types = [&](auto L, auto V) -> hipError_t {
    if (d.x_dtype == SSM_IN_BF16) {
      if (d.in_dtype == SSM_IN_BF16) return f(L, V, type_tag<uint16_t>{}, type_tag<uint16_t>{});
      return f(L, V, type_tag<uint16_t>{}, type_tag<float>{});
    }
    if (d.in_dtype == SSM_IN_BF16) return f(L, V, type_tag<float>{}, type_tag<uint16_t>{});
    return f(L, V, type_tag<float>{}, type_tag<float>{});
  };
#define SSM_CASE(l, v) return types(std::integral_constant<int, l>{}, std::integral_constant<int, v>{})
  if (d.width <= SMALL) {
    switch (group_lanes(d.width)) {
      case 2: SSM_CASE(2, 1);
      case 4: SSM_CASE(4, 1);
      case 8: SSM_CASE(8, 1);
      case 16: SSM_CASE(16, 1);
      case 32: SSM_CASE(32, 1);
      case 64: SSM_CASE(64, 1);
    }
  }
  switch ((d.width + 8 * NT - 1) / (8 * NT)) {
    case 1: SSM_CASE(0, 1);
    case 2: SSM_CASE(0, 2);
    case 3: SSM_CASE(0, 3);
    case 4: SSM_CASE(0, 4);
  }
#undef SSM_CASE
  return hipErrorInvalidValue;
}

// Workgroups over the groups of a row, and over the rows.
struct BackwardGrid {
  int tiles, parts;
};
BackwardGrid backward_grid(const ssm_norm_dims& d, int rows) {
  const int per = d.width <= SMALL ? NT / group_lanes(d.width) : 1;
  BackwardGrid b;
  b.tiles = d.shared ? 1 : (d.groups + per - 1) / per;
  const long long items = d.shared ? ((long long)rows * d.groups + per - 1) / per : rows;
  long long parts = 1024 / b.tiles;
  if (parts > items) parts = items;
  b.parts = parts < 1 ? 1 : (int)parts;
  return b;
}

}  // namespace

size_t norm_workspace(const ssm_norm_dims& d, int rows) {
  return (size_t)backward_grid(d, rows).parts * 2 * (d.shared ? 1 : d.groups) * d.width * sizeof(float);
}

hipError_t launch_norm(const ssm_norm_dims& d, const NormArgs& a, hipStream_t stream) {
  return norm_dispatch(d, [&](auto L, auto V, auto TX, auto T) {
    constexpr int l = decltype(L)::value, per = l == 0 ? 1 : NT / (l == 0 ? 1 : l);
    const long long blocks = ((long long)a.rows * a.groups + per - 1) / per;
    hipLaunchKernelGGL((norm_kernel<l, decltype(V)::value, typename decltype(TX)::type,
                                    typename decltype(T)::type>),
                       dim3((unsigned)(blocks < kMostBlocks ? blocks : kMostBlocks)), dim3(NT), 0, stream, a);
    return hipGetLastError();
  });
}

hipError_t launch_norm_backward(const ssm_norm_dims& d, NormArgs& a, hipStream_t stream) {
  const BackwardGrid b = backward_grid(d, a.rows);
  a.parts = b.parts;
  return norm_dispatch(d, [&](auto L, auto V, auto TX, auto T) {
    hipLaunchKernelGGL((norm_backward_kernel<decltype(L)::value, decltype(V)::value,
                                             typename decltype(TX)::type, typename decltype(T)::type>),
                       dim3((unsigned)b.tiles, (unsigned)b.parts), dim3(NT), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int cols = (a.shared ? 1 : a.groups) * a.width;
    hipLaunchKernelGGL(norm_sum_kernel, dim3((2 * cols + 63) / 64), dim3(64 * RY), 0, stream,
                       a.partial, a.parts, cols, a.dweight, a.dbias);
    return hipGetLastError();
  });
}

}  // namespace ssm
