// pages.h - what the full-attention layers' kernels share: limits, argument checks and the
// launchers behind the rkv_page_* and rkv_prompt_* entry points.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/rkv.h"

namespace rkv {

constexpr int kMaxBatch = 8192;        // sequences of a page table or of packed prompts
constexpr int kPageMaxGroup = 16;      // query heads per key/value head of a page read

// Records a formatted message for rkv_last_error and returns s (rkv_api.cu).
rkv_status fail_with(rkv_status s, const char* fmt, ...);

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

inline bool is_aligned(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// Row r, head h of a strided [rows, heads, D] tensor.
struct Strides {
  int64_t row, head;
};

// Host checks of the structures every entry point takes; RKV_OK or an error.
rkv_status check_pages(const rkv_pages* pg);
rkv_status check_table(const rkv_page_table* t, int block_tokens);

__device__ __forceinline__ void raise_flag(int32_t* flags, int32_t bit) {
  if (flags) atomicOr(flags, bit);
}

}  // namespace rkv
