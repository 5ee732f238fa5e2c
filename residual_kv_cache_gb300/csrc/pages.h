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

inline bool block_ok(int b) { return b == 16 || b == 32 || b == 64 || b == 128; }

inline int log2_block(int block_tokens) {
  int s = 0;
  while ((1 << s) < block_tokens) ++s;
  return s;
}

// Whether the rows of D of a strided [rows, heads, D] tensor are apart, in one order of the
// strides or the other (in binary64: exact where it matters, and no product overflows).
inline bool rows_apart(int rows, int heads, int D, const int64_t strides[2]) {
  const double row = (double)strides[0], head = (double)strides[1], Dl = D;
  const bool rows1 = rows == 1, heads1 = heads == 1;
  return (heads1 || head >= Dl) && (rows1 || row >= Dl) &&
         (rows1 || heads1 || row >= (heads - 1) * head + Dl || head >= (rows - 1) * row + Dl);
}

// Whether two int32 arrays share memory, and whether they do without being the same one.
inline bool shared(const int32_t* p, int64_t np, const int32_t* q, int64_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + 4 * (uint64_t)nq && b < a + 4 * (uint64_t)np;
}
inline bool half_shared(const int32_t* p, int64_t np, const int32_t* q, int64_t nq) {
  return p != q && shared(p, np, q, nq);
}

// The bytes of a strided [rows, heads, D] tensor: n_outer blocks of n_inner runs of `width` bytes.
// (Strides that are never used are 0.)
struct RowBytes {
  int64_t base, outer, inner, n_outer, n_inner, width;
  int64_t block() const { return (n_inner - 1) * inner + width; }
  int64_t end() const { return base + (n_outer - 1) * outer + block(); }
  bool operator==(const RowBytes& o) const {
    return base == o.base && outer == o.outer && inner == o.inner && n_outer == o.n_outer && n_inner == o.n_inner &&
           width == o.width;
  }
};

// false: the tensor does not fit an address space.
inline bool row_bytes(const void* p, int rows, int heads, int D, const int64_t strides[2], int size, RowBytes& r) {
  const double extent = ((double)(rows - 1) * (double)strides[0] + (double)(heads - 1) * (double)strides[1] + D) * size;
  if (!(extent < 4611686018427387904.0)) return false;                // 2^62
  int64_t s[2] = {rows > 1 ? strides[0] * size : 0, heads > 1 ? strides[1] * size : 0};
  const int big = s[1] > s[0];
  r.base = (int64_t)reinterpret_cast<uintptr_t>(p);
  r.outer = s[big], r.inner = s[!big];
  r.n_outer = r.outer ? (big ? heads : rows) : 1, r.n_inner = r.inner ? (big ? rows : heads) : 1;
  r.width = (int64_t)D * size;
  return true;
}

inline int64_t gcd_of(int64_t a, int64_t b) {
  while (b) {
    const int64_t t = a % b;
    a = b, b = t;
  }
  return a;
}
inline int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }

// Whether bytes [x, x + w) meet a run of b, whose runs are apart (rows_apart).
inline bool run_meets(const RowBytes& b, int64_t x, int64_t w) {
  x -= b.base;
  int64_t lo = 0, hi = 0;                        // blocks that begin before x + w and end after x
  if (b.n_outer > 1) {
    lo = floor_div(x - b.block(), b.outer) + 1, hi = floor_div(x + w - 1, b.outer);
    lo = lo < 0 ? 0 : lo, hi = hi > b.n_outer - 1 ? b.n_outer - 1 : hi;
  }
  for (int64_t i = lo; i <= hi; ++i) {
    const int64_t y = x - i * b.outer;
    int64_t first = 0, last = 0;                 // the same of the block's runs
    if (b.n_inner > 1) {
      first = floor_div(y - b.width, b.inner) + 1, last = floor_div(y + w - 1, b.inner);
      first = first < 0 ? 0 : first, last = last > b.n_inner - 1 ? b.n_inner - 1 : last;
    } else if (y + w <= 0 || y >= b.width) {
      continue;
    }
    if (first <= last) return true;
  }
  return false;
}

// Whether a and b share a byte; b's runs are apart.  Most pairs are apart as a whole, or lie side
// by side in each row (parts of one projection): a division then.  Others are looked through run
// by run; of more than 2^20 runs without an answer it is yes.
inline bool rows_meet(const RowBytes& a, const RowBytes& b) {
  if (a.end() <= b.base || b.end() <= a.base) return false;
  // places within a period of both: blocks of the outer strides, runs of all strides
  const int64_t outer = gcd_of(a.outer, b.outer), all = gcd_of(outer, gcd_of(a.inner, b.inner));
  if (outer) {
    const int64_t at = b.base - a.base - floor_div(b.base - a.base, outer) * outer;
    if (at >= a.block() && at + b.block() <= outer) return false;
  }
  if (all) {
    const int64_t at = b.base - a.base - floor_div(b.base - a.base, all) * all;
    if (at >= a.width && at + b.width <= all) return false;
  }
  RowBytes to = b;
  int64_t blocks = a.n_outer;
  if (a.outer == b.outer) {                      // only the distance of two blocks matters
    to.base -= (a.n_outer - 1) * a.outer;
    to.n_outer += a.n_outer - 1;
    blocks = 1;
  }
  int64_t left = 1 << 20;
  for (int64_t i = 0; i < blocks; ++i)
    for (int64_t j = 0; j < a.n_inner; ++j)
      if (left-- == 0 || run_meets(to, a.base + i * a.outer + j * a.inner, a.width)) return true;
  return false;
}

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
// device (the attribute belongs to the device's copy of the function), and where asked into
// clusters of 16 CTAs.  One instance per kernel; concurrent first calls set the same value twice.
class SmemOptIn {
 public:
  template <typename F>
  cudaError_t operator()(F* fn, size_t smem, int dev, bool wide_clusters = false) {
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (done_.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && wide_clusters) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && dev < 64) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

// Launches a kernel of one argument whose blocks may be set up while the stream's previous kernel
// ends: it has to begin with pdl_wait_previous_grid(), before it reads or writes global memory
// (calls in a stream then follow one another 1 to 3 us sooner: a beam step's forks 10.2 -> 7.4 us).  `cluster` CTAs make a cluster.
template <typename Args>
cudaError_t launch_behind(void (*kernel)(Args), const Args& a, unsigned grid, unsigned threads, size_t smem,
                          cudaStream_t s, unsigned cluster = 1) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {cluster, 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

__device__ __forceinline__ void raise_flag(int32_t* flags, int32_t bit) {
  if (flags) atomicOr(flags, bit);
}

// Largest index i in [0, n) with v[i] <= x (v non-decreasing, v[0] <= x).
__device__ __forceinline__ int last_not_above(const int* v, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
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
