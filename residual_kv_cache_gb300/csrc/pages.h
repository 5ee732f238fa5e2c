// pages.h - what the full-attention layers' kernels share: limits, argument checks and the
// launchers behind the rkv_page_* and rkv_prompt_* entry points.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

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

// Whether scores times the scale stay numbers: one that fp32 cannot hold makes NaN of a masked
// score (0 times infinity).
inline bool scale_ok(double scale) { return scale >= 1e-30 && scale < 1e30; }

// Row r, head h of a strided [rows, heads, D] tensor.
struct Strides {
  int64_t row, head;
};

// Host checks of the structures every entry point takes; RKV_OK or an error.
rkv_status check_pages(const rkv_pages* pg);
rkv_status check_table(const rkv_page_table* t, int block_tokens);

// 2-D tensor map of byte rows of `inner` (64 or 128) bytes, swizzled by their width, box =
// {inner, box_rows}; false where the driver's encoder is missing or refuses (rkv_api.cu).
bool encode_map_bytes(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint32_t box_rows);
// 3-D tensor map of a strided bf16 [rows, heads, D] tensor, 128-byte swizzle, box =
// {64 elements, 1 head, box_rows}.
bool encode_map_heads(CUtensorMap* m, const void* base, uint64_t D, uint64_t heads, uint64_t rows,
                      const int64_t strides[2], uint32_t box_rows);

// The current device and its number of SMs (looked up once a device); false without one.
inline bool current_device(int& dev, int& sms) {
  static std::atomic<int> known[64];
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return true;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) return false;
  if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  return true;
}

// Opts a kernel into `smem` bytes of dynamic shared memory on the current device, once per
// device (the attribute belongs to the device's copy of the function).  One instance per
// kernel; concurrent first calls set the same value twice.
class SmemOptIn {
 public:
  template <typename F>
  cudaError_t operator()(F* fn, size_t smem, int dev) {
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (done_.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && dev < 64) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

__device__ __forceinline__ void raise_flag(int32_t* flags, int32_t bit) {
  if (flags) atomicOr(flags, bit);
}

// Inclusive prefix sums of (a, b) over the block, and the block's totals.
template <int kThreads>
__device__ __forceinline__ void block_scan(int64_t& a, int& b, int64_t& total_a, int& total_b) {
  __shared__ int64_t wa[kThreads / 32];
  __shared__ int wb[kThreads / 32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t xa = __shfl_up_sync(0xffffffffu, a, o);
    const int xb = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) a += xa, b += xb;
  }
  __syncthreads();                    // an earlier scan's totals have been read
  if (lane == 31) wa[w] = a, wb[w] = b;
  __syncthreads();
  total_a = 0, total_b = 0;
  int64_t pa = 0;
  int pb = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i == w) pa = total_a, pb = total_b;
    total_a += wa[i], total_b += wb[i];
  }
  a += pa, b += pb;
}

}  // namespace rkv
