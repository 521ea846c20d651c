// Host-side argument checks and launch timing shared by the entry points
// (defined in api.hip).  Every check runs before any GPU call; a failing
// one records the message that tp_last_error() returns.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/tpmlp.h"

namespace tpmlp {

struct Buf {
  const void* p;
  size_t bytes;
  const char* name;
};

int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int ok();
int hip_fail(hipError_t e, const char* what);
bool aligned16(const void* p);
bool overlap(const Buf& a, const Buf& b);
// every output against every input and every other output
int check_alias(const Buf* ins, int nin, const Buf* outs, int nout);
// 16-byte alignment, and presence where `required`
int check_ptrs(const Buf* bufs, int n, bool required);
// buffers that are required only when they hold something: 16-byte alignment
int check_sized(const Buf* bufs, int n);
// the same for tables of int32 or fp32 elements: 4-byte alignment
int check_tables(const Buf* bufs, int n);
// the current device is a gfx950
int check_device();

constexpr int64_t kMaxDim = (int64_t)1 << 30;
// Largest leading dimension (H, and the Z_save width 2 F_shard): the bf16
// kernels address one 256-row tile through 32-bit buffer offsets, so
// 256 rows x ld x 2 bytes must stay below 2^31.
constexpr int64_t kMaxLd = (int64_t)1 << 21;

// Launch timing (tp_launch_events): whether this thread's caller-owned
// events still have room for a unit, and recording its begin and end.
bool timing_armed();
hipError_t timing_mark(hipStream_t st, bool end);

template <typename F>
hipError_t timed(hipStream_t st, F&& launch) {
  if (!timing_armed()) return launch();
  hipError_t he = timing_mark(st, false);
  if (he != hipSuccess) return he;
  he = launch();
  if (he != hipSuccess) return he;
  return timing_mark(st, true);
}

}  // namespace tpmlp
