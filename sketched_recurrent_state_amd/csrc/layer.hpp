// layer.hpp -- what a layer does around its recurrence (short convolution, selective recurrence, output
// norm): arguments of the launches and device helpers the kernels share. Arguments are validated
// in layer_abi.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"
#include "scan_table.hpp"
#include "sketchssm.h"

namespace ssm {

constexpr int CP = SSM_CONV_PARTS;

// Rows of one array: row t from p + t * stride elements on.
struct Rows {
  const void* p;
  int64_t stride;
  template <typename T>
  __device__ __forceinline__ const T* row(int64_t t) const {
    return static_cast<const T*>(p) + t * stride;
  }
  template <typename T>
  __device__ __forceinline__ T* out(int64_t t) const {
    return static_cast<T*>(const_cast<void*>(p)) + t * stride;
  }
};
inline Rows rows_of(const ssm_rows& r) { return Rows{r.data, r.stride}; }

// ---------------------------------------------------------------------------
// convolution
// ---------------------------------------------------------------------------
// A part's channels over lanes: 2^log_lanes lanes a tile (64, fewer where the part is narrower), the
// wave's other lanes on other runs of tokens. The last three and norm_lanes are set by the launch.
struct ConvPart {
  Rows x, y, dy, dx;
  int channels, offset;  // its channels, and those of the parts before
  int norm;              // channels of a norm's run, 0: no norm
  float scale;
  int norm_lanes;        // its lanes
  int log_lanes, tiles, first_block;
};

struct ConvArgs {
  ScanPlan plan;
  ConvPart part[CP];
  int parts, C, silu, num_slots;
  int log_run;  // log2 of the tokens of a run (8 .. 64)
  int runs;     // runs of all chunks (a step: rows)
  int rows;     // backward: rows of partial sums, each of every rows-th run
  float eps;
  const float *weight, *bias;
  const int32_t* slot;
  const void *state_in, *dstate;
  void *state, *dstate_in;
  float* partial;  // [rows][taps + 1][C]
  float *dweight, *dbias;
};

size_t conv_workspace(const ssm_conv_dims& d, int total_tokens);
hipError_t launch_conv_forward(const ssm_conv_dims& d, ConvArgs& a, hipStream_t stream);
hipError_t launch_conv_backward(const ssm_conv_dims& d, ConvArgs& a, hipStream_t stream);
hipError_t launch_conv_step(const ssm_conv_dims& d, ConvArgs& a, hipStream_t stream);

// ---------------------------------------------------------------------------
// selective recurrence
// ---------------------------------------------------------------------------
struct SelectiveWork {
  // for every group of chunks, of the sequences that go on behind it:
  float* local;    // [groups][channels][d_state]  the state it leaves, from zero (or the sequence's start)
  float* sums;     // [groups][channels]           the sum of its deltas
  float* back;     // backward: [groups][channels][d_state]  the gradient that leaves it at its start
  float* states;   // backward: the state before every 8 tokens of a sequence but its first, from the group's zero
  float* until;    // backward: [those places][channels]  the sum of delta from the group's start
  float* dbc;      // [tokens + 1][tiles][2][d_state]  dB and dC of a wave's channels
  float* partial;  // [groups][channels][d_state + 2]  dA, dD, ddt_bias of a group's tokens
  float* start;    // forward: [groups][channels][d_state]  the kept state such a sequence begins with in the group
                   // (behind what the gradients read: among it, their calls took 1 % longer)
  size_t bytes;
};

struct SelectiveArgs {
  ScanPlan plan;
  Rows x, dt, z, B, C, out, dout;
  Rows dx, ddt, dz, dB, dC;
  const float *A, *D, *dt_bias;
  int channels, groups, softplus, num_slots;
  int gated;  // without a gate z is x
  int time_groups, group_chunks;  // groups of the plan's chunks, and chunks of one
  const int32_t* slot;
  const float *state_in, *dstate;
  float *state, *dstate_in;
  float *dA, *dD, *ddt_bias;
  SelectiveWork w;
};

SelectiveWork selective_work(const ssm_selective_dims& d, int total_tokens, bool backward, void* base);
hipError_t launch_selective_forward(const ssm_selective_dims& d, SelectiveArgs& a, hipStream_t stream);
hipError_t launch_selective_backward(const ssm_selective_dims& d, SelectiveArgs& a, hipStream_t stream);
hipError_t launch_selective_step(const ssm_selective_dims& d, const SelectiveArgs& a, hipStream_t stream);

// ---------------------------------------------------------------------------
// norm
// ---------------------------------------------------------------------------
struct NormArgs {
  Rows x, z, out, dout, dx, dz;
  int rows, groups, width;
  int gate, sigmoid, shared, centred;
  float eps;
  const float *weight, *bias;
  int parts;       // backward: rows of partial sums
  float* partial;  // [parts][2][groups or 1][width]
  float *dweight, *dbias;
};

size_t norm_workspace(const ssm_norm_dims& d, int rows);
hipError_t launch_norm(const ssm_norm_dims& d, const NormArgs& a, hipStream_t stream);
hipError_t launch_norm_backward(const ssm_norm_dims& d, NormArgs& a, hipStream_t stream);

// ---------------------------------------------------------------------------
// device helpers
// ---------------------------------------------------------------------------
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

// 1 / (1 + e^-x): the exponent's rounding gives |x| 2^-24 of the value, the other steps 4 ulp.
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                 pack_bf16x2(v[6], v[7]));
}

// LDS written by this wave's other lanes
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup", "local");
  __builtin_amdgcn_wave_barrier();
}

}  // namespace ssm
