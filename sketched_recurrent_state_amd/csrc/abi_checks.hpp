// abi_checks.hpp -- what the C entry points share: the calling thread's last error and the checks
// of pointers before anything is enqueued. Defined in abi.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "sketchssm.h"

namespace ssm {

ssm_status fail(ssm_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
ssm_status ok();
ssm_status launched(hipError_t e, const char* fn);
const char* last_error();

// An array argument. Rows of `bytes` each, `stride` bytes apart (rows = 1: one run).
struct Arr {
  const void* p;
  size_t bytes;
  bool output;
  const char* name;
  unsigned align = 16;
  size_t rows = 1, stride = 0;
};

// Alignment, and no output over an input or another output. Arrays of rows with one stride may
// interleave: column ranges of one matrix.
ssm_status check_arrays(const char* fn, const Arr* arrs, size_t n);
inline ssm_status check_arrays(const char* fn, std::initializer_list<Arr> arrs) {
  return check_arrays(fn, arrs.begin(), arrs.size());
}

ssm_status check_workspace(const void* workspace, int64_t bytes, size_t need, const char* fn);

}  // namespace ssm
