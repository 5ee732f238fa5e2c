// k_pages.cu - pages of the full-attention layers' 8-bit K/V: the plan of a step's pages
// and rows from the requests' lengths, their release, and the append of new rows.
//
// Plan.  With len and new the stored and appended positions, P the page size,
//   have = ceil(len / P), need = ceil((len + new) / P) - have,
//   first = exclusive prefix sum of need, cu = exclusive prefix sum of new:
// page have + i of a sequence is free[n_free - 1 - (first + i)], and packed row r lies in
// the sequence with cu_b <= r < cu_{b+1}, at position len_b + r - cu_b.  Every CTA scans the
// lengths itself (they fit in shared memory), so pages and rows are independent items found
// by bisection, and no CTA waits for another's prefix.  Nothing a CTA reads may change
// before all have read it (lengths and the free count can be updated in place): the CTAs
// form one cluster and meet once after their scans.  The call is a handful of dependent
// loads: latency bounds it up to some 10^4 rows, the row maps' stores beyond.
//
// Append.  One CTA takes the rows that a step brings to one (page, head) of K or of V: it
// holds them in registers between finding their largest magnitude and storing their codes,
// so each row is read once, and no other CTA touches the page's scale.  Bandwidth bounds
// long appends, latency single tokens.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "pages.h"

namespace rkv {
namespace cg = cooperative_groups;
namespace {

constexpr int kPlanThreads = 512;
constexpr int kMaxPlanCtas = 8;      // portable cluster size

// Largest index i in [0, n) with v[i] <= x (v non-decreasing, v[0] <= x).
__device__ __forceinline__ int last_not_above(const int* v, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

struct PlanArgs {
  const int32_t* new_tokens;
  const int32_t* seq_len;
  int32_t* table;
  const int32_t* free_blocks;
  const int32_t* n_free;
  int32_t* seq_len_out;
  int32_t* n_free_out;
  int32_t* cu_rows;
  int32_t* row_seq;
  int32_t* row_pos;
  int32_t* row_slot;
  int32_t* flags;
  int batch, max_blocks, num_blocks, shift, max_rows;   // page size = 1 << shift
};

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(PlanArgs p) {
  extern __shared__ int psm[];
  int* s_cu = psm;                   // [batch] first row of each sequence
  int* s_first = s_cu + p.batch;     // [batch] first taken page of each sequence
  int* s_len = s_first + p.batch;    // [batch] stored positions
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x;
  const int P1 = (1 << p.shift) - 1;
  const int64_t cap = (int64_t)p.max_blocks << p.shift;
  const int n_free = *p.n_free;

  int64_t rows = 0;
  int pages = 0;                     // at most `rows`: exact wherever the rows fit
  bool bad = n_free < 0 || n_free > p.num_blocks;
  for (int b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int len = 0, nw = 0;
    if (b < p.batch) len = p.seq_len[b], nw = p.new_tokens[b];
    if (len < 0 || nw < 0 || (int64_t)len + nw > cap) bad = true, len = 0, nw = 0;
    const int need = (int)(((int64_t)len + nw + P1) >> p.shift) - (int)(((int64_t)len + P1) >> p.shift);
    int64_t a = nw, ta;
    int c = need, tc;
    block_scan<kPlanThreads>(a, c, ta, tc);
    if (b < p.batch) {
      s_cu[b] = (int)min(rows + a - nw, (int64_t)INT32_MAX);
      s_first[b] = pages + c - need;
      s_len[b] = len;
    }
    rows += ta;
    pages += tc;
  }
  bad = __syncthreads_or(bad);
  const bool full = !bad && (rows > p.max_rows || pages > n_free);
  const bool ok = !bad && !full;
  const int total = ok ? (int)rows : 0;
  // The old lengths of a refused step are still to be copied: read them before the barrier.
  cluster.sync();                    // every CTA has read the lengths and the free count

  const int step = gridDim.x * kPlanThreads, first = blockIdx.x * kPlanThreads + tid;
  for (int r = first; r < p.max_rows; r += step) {
    int seq = -1, pos = -1, slot = -1;
    if (r < total) {
      // empty sequences share their first row with the next: the last one is the owner
      seq = last_not_above(s_cu, p.batch, r);
      pos = s_len[seq] + r - s_cu[seq];
      const int page = pos >> p.shift, have = (s_len[seq] + P1) >> p.shift;
      const int64_t at = (int64_t)seq * p.max_blocks + page;
      const int id = page < have ? p.table[at]
                                 : p.free_blocks[n_free - 1 - (s_first[seq] + page - have)];
      if (id >= 0 && id < p.num_blocks)
        slot = (id << p.shift) + (pos & P1);
      else
        raise_flag(p.flags, RKV_FLAG_BAD_INDEX);
    }
    p.row_seq[r] = seq;
    p.row_pos[r] = pos;
    p.row_slot[r] = slot;
  }
  if (ok) {
    for (int i = first; i < pages; i += step) {
      const int seq = last_not_above(s_first, p.batch, i);
      const int have = (s_len[seq] + P1) >> p.shift;
      p.table[(int64_t)seq * p.max_blocks + have + i - s_first[seq]] = p.free_blocks[n_free - 1 - i];
    }
  }
  for (int b = first; b < p.batch; b += step) {
    p.cu_rows[b] = ok ? s_cu[b] : 0;
    const int next = b + 1 < p.batch ? s_cu[b + 1] : total;
    if (ok)
      p.seq_len_out[b] = s_len[b] + next - s_cu[b];
    else if (p.seq_len_out != p.seq_len)
      p.seq_len_out[b] = p.seq_len[b];
  }
  if (first == 0) {
    p.cu_rows[p.batch] = total;
    *p.n_free_out = ok ? n_free - pages : n_free;
    if (bad) raise_flag(p.flags, RKV_FLAG_BAD_INDEX);
    if (full) raise_flag(p.flags, RKV_FLAG_NO_SPACE);
  }
}

// One CTA: a release moves a few thousand ids at a request's end.
__global__ void __launch_bounds__(kPlanThreads)
    page_release_kernel(int32_t* table, int32_t* seq_len, const int32_t* finished,
                        int32_t* free_blocks, int32_t* n_free_p, int batch, int max_blocks,
                        int num_blocks, int shift, int32_t* flags) {
  extern __shared__ int psm[];
  int* s_first = psm;                // [batch] first released page of each sequence
  const int tid = threadIdx.x;
  const int64_t cap = (int64_t)max_blocks << shift;
  const int n_free = *n_free_p;
  int64_t pages = 0;
  bool bad = n_free < 0 || n_free > num_blocks;
  for (int b0 = 0; b0 < batch; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int len = 0;
    if (b < batch && finished[b] != 0) len = seq_len[b];
    if (len < 0 || len > cap) bad = true, len = 0;
    const int gives = (int)(((int64_t)len + (1 << shift) - 1) >> shift);
    int64_t a = gives, ta;
    int c = 0, tc;
    block_scan<kPlanThreads>(a, c, ta, tc);
    if (b < batch) s_first[b] = (int)min(pages + a - gives, (int64_t)INT32_MAX);
    pages += ta;
  }
  bad = __syncthreads_or(bad);
  if (bad || pages > num_blocks - n_free) {
    if (tid == 0) raise_flag(flags, bad ? RKV_FLAG_BAD_INDEX : RKV_FLAG_NO_SPACE);
    return;
  }
  for (int i = tid; i < (int)pages; i += kPlanThreads) {
    const int seq = last_not_above(s_first, batch, i);
    int32_t* e = table + (int64_t)seq * max_blocks + (i - s_first[seq]);
    free_blocks[n_free + i] = *e;
    *e = -1;
  }
  for (int b = tid; b < batch; b += kPlanThreads)
    if (finished[b] != 0) seq_len[b] = 0;
  if (tid == 0) *n_free_p = n_free + (int)pages;
}

// ------------------------------------------------------------------------------ append
constexpr int kAppendThreads = 256;

struct AppendArgs {
  const void* x[2];                  // k, v
  Strides st[2];
  uint8_t* codes[2];
  float* scale[2];
  const int32_t* table;
  const int32_t* seq_len;
  const int32_t* cu;
  int32_t* flags;
  int batch, max_blocks, num_blocks, N, shift, n_rows;
};

// Exponent e of the smallest scale 2^e with amax <= 448 2^e (448 = 1.75 2^8), in [-64, 120].
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(-64, min(120, e));      // zero and subnormals: exponent field 0
}

__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Eight consecutive values of a row as floats.
__device__ __forceinline__ void load_row8(const __nv_bfloat16* p, float* f) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load_row8(const float* p, float* f) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// Two floats to E4M3, nearest even, saturating (NaN stays NaN).
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// Grid (units, N, 2): unit u = the u-th (sequence, page) that the step touches, in order;
// z: K or V.  D / 8 threads share a row; a thread holds kHold chunks of eight values.
template <typename T, int D, int kPage>
__global__ void __launch_bounds__(kAppendThreads) page_append_kernel(AppendArgs p) {
  constexpr int kLanes = D / 8;                              // threads of one row
  constexpr int kRows = kAppendThreads / kLanes;             // rows of one pass
  constexpr int kHold = (kPage + kRows - 1) / kRows;         // passes over a page
  __shared__ int s_seq, s_page, s_lo, s_hi, s_row0;
  __shared__ float s_max[kAppendThreads / 32];
  const int tid = threadIdx.x, u = blockIdx.x, h = blockIdx.y, z = blockIdx.z;

  // the unit's sequence and page
  if (tid == 0) s_seq = -1;
  int64_t base = 0;
  for (int b0 = 0; b0 < p.batch && base <= u; b0 += kAppendThreads) {
    const int b = b0 + tid;
    int lo = 0, hi = 0, r0 = 0;      // the step's positions [lo, hi) of sequence b
    if (b < p.batch) {
      r0 = p.cu[b];
      const int64_t rows = (int64_t)p.cu[b + 1] - r0, len = p.seq_len[b];
      if (rows != 0) {
        if (rows > 0 && r0 >= 0 && rows <= len && len <= (int64_t)p.max_blocks << p.shift) {
          lo = (int)(len - rows);
          hi = lo + (int)max((int64_t)0, min(rows, (int64_t)p.n_rows - r0));
        } else if (u == 0 && h == 0 && z == 0) {
          raise_flag(p.flags, RKV_FLAG_BAD_INDEX);
        }
      }
    }
    const int P1 = (1 << p.shift) - 1;
    const int touched = hi > lo ? ((hi + P1) >> p.shift) - (lo >> p.shift) : 0;
    int64_t a = touched, ta;
    int c = 0, tc;
    block_scan<kAppendThreads>(a, c, ta, tc);
    const int64_t mine = base + a - touched;
    if (u >= mine && u < base + a) {
      s_seq = b;
      s_page = (lo >> p.shift) + (int)(u - mine);
      s_lo = lo, s_hi = hi, s_row0 = r0;
    }
    base += ta;
  }
  __syncthreads();
  const int seq = s_seq;
  if (seq < 0) return;               // fewer pages than the grid's bound
  const int page = s_page, P = 1 << p.shift;
  const int lo = max(s_lo, page << p.shift), hi = min(s_hi, (page + 1) << p.shift);
  const int off0 = lo & (P - 1), n = hi - lo;                // rows of the page, from off0
  const int row0 = s_row0 + (lo - s_lo);
  const int id = p.table[(int64_t)seq * p.max_blocks + page];
  if (id < 0 || id >= p.num_blocks) {
    if (tid == 0) raise_flag(p.flags, RKV_FLAG_BAD_INDEX);
    return;
  }
  const int64_t head = (int64_t)id * p.N + h;
  float* scale_p = p.scale[z] + head;
  uint8_t* codes = p.codes[z] + (head << p.shift) * D;
  const T* x = static_cast<const T*>(p.x[z]) + (int64_t)row0 * p.st[z].row + (int64_t)h * p.st[z].head;
  const int lane = tid % kLanes, r_in = tid / kLanes;
  const float held = off0 > 0 ? *scale_p : 0.f;

  float f[kHold][8];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    const int r = i * kRows + r_in;
    if (r < n) {
      load_row8(x + (int64_t)r * p.st[z].row + lane * 8, f[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float m = fabsf(f[i][e]);
        if (m < INFINITY) amax = fmaxf(amax, m);             // finite values only
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((tid & 31) == 0) s_max[tid >> 5] = amax;
  __syncthreads();                   // every thread has read the held scale
#pragma unroll
  for (int i = 0; i < kAppendThreads / 32; ++i) amax = fmaxf(amax, s_max[i]);
  const float need = pow2i(scale_exponent(amax));
  const float s = held > need ? held : need;
  const float inv = 1.f / s;         // a power of two: exact
  if (tid == 0) *scale_p = s;
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    const int r = i * kRows + r_in;
    if (r < n) {
      uint32_t w[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        w[e] = to_e4m3x2(f[i][4 * e] * inv, f[i][4 * e + 1] * inv) |
               to_e4m3x2(f[i][4 * e + 2] * inv, f[i][4 * e + 3] * inv) << 16;
      *reinterpret_cast<uint2*>(codes + (int64_t)(off0 + r) * D + lane * 8) = make_uint2(w[0], w[1]);
    }
  }
  if (held > 0.f && held < s) {      // the page's earlier rows at the grown scale
    const float ratio = held / s;    // a power of two: exact
    for (int r = r_in; r < off0; r += kRows) {
      uint2* q = reinterpret_cast<uint2*>(codes + (int64_t)r * D + lane * 8);
      const uint2 c = *q;
      const uint32_t in[2] = {c.x, c.y};
      uint32_t w[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t half[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((uint16_t)(in[e] >> (16 * j)), __NV_E4M3);
          const float2 v = __half22float2(__half2(hr));
          half[j] = to_e4m3x2(v.x * ratio, v.y * ratio);
        }
        w[e] = half[0] | half[1] << 16;
      }
      *q = make_uint2(w[0], w[1]);
    }
  }
}

int log2_block(int block_tokens) {
  int s = 0;
  while ((1 << s) < block_tokens) ++s;
  return s;
}

bool block_ok(int b) { return b == 16 || b == 32 || b == 64 || b == 128; }

// The kernels' shared memory beyond 48 KB is opted into on every call that needs it: the
// attribute belongs to the current device's copy of the function.
template <typename F>
bool opt_in(F* fn, size_t smem) {
  return smem <= 48 * 1024 ||
         cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess;
}

template <typename T, int D>
void launch_append(const AppendArgs& a, int block_tokens, dim3 grid, cudaStream_t s) {
  switch (block_tokens) {
    case 16: page_append_kernel<T, D, 16><<<grid, kAppendThreads, 0, s>>>(a); break;
    case 32: page_append_kernel<T, D, 32><<<grid, kAppendThreads, 0, s>>>(a); break;
    case 64: page_append_kernel<T, D, 64><<<grid, kAppendThreads, 0, s>>>(a); break;
    default: page_append_kernel<T, D, 128><<<grid, kAppendThreads, 0, s>>>(a); break;
  }
}

}  // namespace

rkv_status check_pages(const rkv_pages* pg) {
  if (!pg) return fail_with(RKV_EINVAL, "pages is NULL");
  if (!pg->k || !pg->v || !pg->k_scale || !pg->v_scale) return fail_with(RKV_EINVAL, "NULL page storage");
  if (!is_aligned(pg->k, 16) || !is_aligned(pg->v, 16) || !is_aligned(pg->k_scale, 4) || !is_aligned(pg->v_scale, 4))
    return fail_with(RKV_EALIGN, "page storage must be 16-byte aligned (scales 4-byte)");
  if (pg->n_kv_heads < 1 || pg->n_kv_heads > 65535) return fail_with(RKV_EINVAL, "n_kv_heads must be in 1..65535");
  if (pg->head_dim != 64 && pg->head_dim != 128) return fail_with(RKV_EINVAL, "head_dim must be 64 or 128");
  if (!block_ok(pg->block_tokens)) return fail_with(RKV_EINVAL, "block_tokens must be 16, 32, 64 or 128");
  if (pg->num_blocks < 1 || (int64_t)pg->num_blocks * pg->n_kv_heads * pg->block_tokens > INT32_MAX)
    return fail_with(RKV_EINVAL, "num_blocks must be >= 1 and num_blocks * N * block_tokens below 2^31");
  return RKV_OK;
}

rkv_status check_table(const rkv_page_table* t, int block_tokens) {
  if (!t) return fail_with(RKV_EINVAL, "table is NULL");
  if (!t->block_table || !t->seq_len) return fail_with(RKV_EINVAL, "NULL block_table or seq_len");
  if (t->batch < 1 || t->batch > kMaxBatch) return fail_with(RKV_EINVAL, "batch must be in 1..%d", kMaxBatch);
  if (t->max_blocks < 1 || (int64_t)t->max_blocks * block_tokens > INT32_MAX)
    return fail_with(RKV_EINVAL, "max_blocks must be >= 1 and max_blocks * block_tokens below 2^31");
  return RKV_OK;
}

}  // namespace rkv

using namespace rkv;

extern "C" rkv_status rkv_page_plan(const rkv_page_table* table, const int32_t* new_tokens,
                                    const int32_t* free_blocks, const int32_t* n_free,
                                    int32_t num_blocks, int32_t block_tokens, int32_t max_rows,
                                    int32_t* seq_len_out, int32_t* n_free_out, int32_t* cu_rows,
                                    int32_t* row_seq, int32_t* row_pos, int32_t* row_slot,
                                    int32_t* flags, void* stream) {
  if (!block_ok(block_tokens)) return fail_with(RKV_EINVAL, "block_tokens must be 16, 32, 64 or 128");
  if (rkv_status st = check_table(table, block_tokens)) return st;
  if (num_blocks < 1 || (int64_t)num_blocks * block_tokens > INT32_MAX)
    return fail_with(RKV_EINVAL, "num_blocks must be >= 1 and num_blocks * block_tokens below 2^31");
  if (max_rows < 0) return fail_with(RKV_EINVAL, "max_rows must be >= 0");
  if (!new_tokens || !free_blocks || !n_free || !seq_len_out || !n_free_out || !cu_rows ||
      (max_rows > 0 && (!row_seq || !row_pos || !row_slot)))
    return fail_with(RKV_EINVAL, "NULL pointer");
  PlanArgs a;
  a.new_tokens = new_tokens;
  a.seq_len = table->seq_len;
  a.table = table->block_table;
  a.free_blocks = free_blocks;
  a.n_free = n_free;
  a.seq_len_out = seq_len_out;
  a.n_free_out = n_free_out;
  a.cu_rows = cu_rows;
  a.row_seq = row_seq;
  a.row_pos = row_pos;
  a.row_slot = row_slot;
  a.flags = flags;
  a.batch = table->batch;
  a.max_blocks = table->max_blocks;
  a.num_blocks = num_blocks;
  a.shift = log2_block(block_tokens);
  a.max_rows = max_rows;
  // CTAs of one cluster, doubled while each still has a few thousand rows to fill
  int ctas = 1;
  while (ctas < kMaxPlanCtas && max_rows > ctas * 4 * kPlanThreads) ctas *= 2;
  const size_t smem = sizeof(int) * 3 * (size_t)a.batch;
  if (!opt_in(page_plan_kernel, smem)) return fail_with(RKV_ECUDA, "cudaFuncSetAttribute failed");
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(ctas);
  lc.blockDim = dim3(kPlanThreads);
  lc.dynamicSmemBytes = smem;
  lc.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&lc, page_plan_kernel, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? RKV_OK : fail_with(RKV_ECUDA, "page plan launch failed: %s", cudaGetErrorString(e));
}

extern "C" rkv_status rkv_page_release(const rkv_page_table* table, const int32_t* finished,
                                       int32_t* free_blocks, int32_t* n_free, int32_t num_blocks,
                                       int32_t block_tokens, int32_t* flags, void* stream) {
  if (!block_ok(block_tokens)) return fail_with(RKV_EINVAL, "block_tokens must be 16, 32, 64 or 128");
  if (rkv_status st = check_table(table, block_tokens)) return st;
  if (num_blocks < 1 || (int64_t)num_blocks * block_tokens > INT32_MAX)
    return fail_with(RKV_EINVAL, "num_blocks must be >= 1 and num_blocks * block_tokens below 2^31");
  if (!finished || !free_blocks || !n_free) return fail_with(RKV_EINVAL, "NULL pointer");
  page_release_kernel<<<1, kPlanThreads, sizeof(int) * (size_t)table->batch,
                        static_cast<cudaStream_t>(stream)>>>(
      table->block_table, table->seq_len, finished, free_blocks, n_free, table->batch,
      table->max_blocks, num_blocks, log2_block(block_tokens), flags);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? RKV_OK : fail_with(RKV_ECUDA, "page release launch failed: %s", cudaGetErrorString(e));
}

extern "C" rkv_status rkv_page_append(const rkv_pages* pages, const rkv_page_table* table,
                                      const void* k, const int64_t k_strides[2], const void* v,
                                      const int64_t v_strides[2], int32_t dtype, int32_t n_rows,
                                      const int32_t* cu_rows, int32_t* flags, void* stream) {
  if (rkv_status st = check_pages(pages)) return st;
  if (rkv_status st = check_table(table, pages->block_tokens)) return st;
  if (dtype != RKV_F32 && dtype != RKV_BF16) return fail_with(RKV_EINVAL, "dtype must be RKV_F32 or RKV_BF16");
  if (n_rows < 0) return fail_with(RKV_EINVAL, "n_rows < 0");
  if (n_rows == 0) return RKV_OK;
  if (!k || !v || !k_strides || !v_strides || !cu_rows) return fail_with(RKV_EINVAL, "NULL pointer");
  const int per16 = dtype == RKV_F32 ? 4 : 8;
  for (int i = 0; i < 2; ++i)
    if (k_strides[i] < 0 || v_strides[i] < 0 || k_strides[i] % per16 || v_strides[i] % per16)
      return fail_with(RKV_EALIGN, "strides must be >= 0 and multiples of 16 bytes");
  if (!is_aligned(k, 16) || !is_aligned(v, 16)) return fail_with(RKV_EALIGN, "k and v must be 16-byte aligned");
  AppendArgs a;
  a.x[0] = k, a.x[1] = v;
  a.st[0] = {k_strides[0], k_strides[1]};
  a.st[1] = {v_strides[0], v_strides[1]};
  a.codes[0] = static_cast<uint8_t*>(pages->k), a.codes[1] = static_cast<uint8_t*>(pages->v);
  a.scale[0] = pages->k_scale, a.scale[1] = pages->v_scale;
  a.table = table->block_table;
  a.seq_len = table->seq_len;
  a.cu = cu_rows;
  a.flags = flags;
  a.batch = table->batch;
  a.max_blocks = table->max_blocks;
  a.num_blocks = pages->num_blocks;
  a.N = pages->n_kv_heads;
  a.shift = log2_block(pages->block_tokens);
  a.n_rows = n_rows;
  // pages a step can touch: a sequence's rows touch at most (rows - 2) / P + 2, and no more
  // than its rows
  const int64_t bound = (int64_t)n_rows / pages->block_tokens + 2 * (int64_t)a.batch;
  const dim3 grid((unsigned)(bound < n_rows ? bound : n_rows), a.N, 2);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == RKV_F32)
    pages->head_dim == 128 ? launch_append<float, 128>(a, pages->block_tokens, grid, s)
                           : launch_append<float, 64>(a, pages->block_tokens, grid, s);
  else
    pages->head_dim == 128 ? launch_append<__nv_bfloat16, 128>(a, pages->block_tokens, grid, s)
                           : launch_append<__nv_bfloat16, 64>(a, pages->block_tokens, grid, s);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? RKV_OK : fail_with(RKV_ECUDA, "page append launch failed: %s", cudaGetErrorString(e));
}
