// Host helpers shared by the C-ABI layers (attn_api.cu, scored_api.cu,
// rope.cu): per-device facts, tensor maps, pointer and overlap checks.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <mutex>

#include "attn.h"

namespace attn {

struct DeviceInfo {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
  int num_sms = 0;
  int l2_bytes = 0;
  uint32_t* status = nullptr;   // the device status word
};

// Records e as this thread's last CUDA error; ATTN_ERR_CUDA.
attn_status_t cuda_fail(cudaError_t e);

// Facts of the current device, resolved once per device.
attn_status_t device_info(DeviceInfo** out);

// 3-D map over a [planes, rows, inner] array with 128-byte swizzled boxes of
// box_rows rows x (128 bytes of elements).
attn_status_t make_map(CUtensorMap* m, const void* base, int inner, int rows, int planes, bool f32 = false,
                       unsigned box_rows = 128);

// Key splits for `units` work units of nkb key tiles each on `slots` SMs.
int wave_splits(long long units, int nkb, int slots);

inline size_t elem_size(attn_dtype_t dt) { return dt == ATTN_BF16 ? 2 : 4; }
inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

struct Range {
  uintptr_t lo, hi;
};
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }
inline Range range(const void* p, size_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + bytes};
}

inline attn_status_t check_ptr(const void* p, size_t bytes, size_t align) {
  if (bytes == 0) return ATTN_OK;  // empty tensors may be NULL
  if (p == nullptr) return ATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(p) % align) return ATTN_ERR_MISALIGNED;
  return ATTN_OK;
}

}  // namespace attn
