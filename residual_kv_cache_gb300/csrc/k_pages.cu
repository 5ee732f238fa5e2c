// k_pages.cu - pages of the full-attention layers' 8-bit K/V: the plan of a step's pages
// and rows from the requests' lengths, their release, and the append of new rows.
//
// Plan.  With len and new the stored and appended positions, P the page size,
//   have = ceil(len / P), need = ceil((len + new) / P) - have,
//   first = exclusive prefix sum of need, cu = exclusive prefix sum of new:
// page have + i of a sequence is free[n_free - 1 - (first + i)], and packed row r lies in
// the sequence with cu_b <= r < cu_{b+1}, at position len_b + r - cu_b.  Every CTA scans the
// lengths itself (they fit in shared memory), so pages and rows are independent items found
// by bisection, and no CTA waits for another's prefix.  No CTA may change what another still
// reads: where several CTAs share the rows and the lengths or the free count are updated in
// place, a second kernel does that from the offsets.  The call is a handful of dependent
// loads and latency bounds it: a thread takes kPlanRows rows whose loads overlap (up to
// 512 new tokens for each of 256 sequences: 14.6 us on one cluster of 8 CTAs, one row at a
// time, 5.2 us so; one token for each of 16 3.2 us).
//
// Append.  A CTA takes the rows that a step brings to a run of 64 positions (whole pages; one
// page of 128), of K or of V, and one or more heads in turn: it holds a head's rows in
// registers between finding their pages' largest magnitudes and storing their codes, so each
// row is read once, and no other CTA touches the pages' scales.  Bandwidth bounds long
// appends, latency single tokens: finding the run takes about as long as a head's rows, so a
// CTA takes several heads where there are CTAs enough (32768 rows of 8 heads of 128: 64 us
// with a head a CTA, 36 us so, 5.6 TB/s, as fp32 55 us, 6.1 TB/s; on pages of 16 62 us with a
// page a CTA, 43 us so; one row for each of 16 sequences 2.9 us).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "pages.h"

namespace rkv {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanRows = 4;         // rows of one thread at a time
constexpr int kPlanMaxCtas = 512;

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
  int state;                         // this kernel also writes the new lengths and free count
};

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(PlanArgs p) {
  extern __shared__ int psm[];
  int* s_cu = psm;                   // [batch] first row of each sequence
  int* s_first = s_cu + p.batch;     // [batch] first taken page of each sequence
  int* s_len = s_first + p.batch;    // [batch] stored positions
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
  bad = __syncthreads_or(bad);     // and: everyone's sums are in shared memory
  const bool full = !bad && (rows > p.max_rows || pages > n_free);
  const bool ok = !bad && !full;
  const int total = ok ? (int)rows : 0;
  const int step = gridDim.x * kPlanThreads, first = blockIdx.x * kPlanThreads + tid;
  // rows without a sign: up to 2^20 past a max_rows of up to 2^31 - 1
  static_assert((int64_t)kPlanMaxCtas * kPlanThreads * kPlanRows <= 1 << 20);
  const uint32_t max_rows = p.max_rows;
  for (uint32_t r0 = first; r0 < max_rows; r0 += step * kPlanRows) {
    int seq[kPlanRows], pos[kPlanRows], id[kPlanRows];
#pragma unroll
    for (int i = 0; i < kPlanRows; ++i) {
      const uint32_t r = r0 + i * step;
      seq[i] = pos[i] = id[i] = -1;
      if (r < (uint32_t)total) {
        // empty sequences share their first row with the next: the last one is the owner
        const int b = last_not_above(s_cu, p.batch, (int)r);
        seq[i] = b;
        pos[i] = s_len[b] + ((int)r - s_cu[b]);
        const int page = pos[i] >> p.shift, have = (s_len[b] + P1) >> p.shift;
        const int32_t* at = page < have ? p.table + (int64_t)b * p.max_blocks + page
                                        : p.free_blocks + (n_free - 1 - (s_first[b] + page - have));
        id[i] = *at;
      }
    }
#pragma unroll
    for (int i = 0; i < kPlanRows; ++i) {
      const uint32_t r = r0 + i * step;
      if (r < max_rows) {
        const bool fine = id[i] >= 0 && id[i] < p.num_blocks;
        if (r < (uint32_t)total && !fine) raise_flag(p.flags, RKV_FLAG_BAD_INDEX);
        p.row_seq[r] = seq[i];
        p.row_pos[r] = pos[i];
        p.row_slot[r] = fine ? (id[i] << p.shift) + (pos[i] & P1) : -1;
      }
    }
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
    if (p.state) {
      const int next = b + 1 < p.batch ? s_cu[b + 1] : total;
      p.seq_len_out[b] = ok ? s_len[b] + next - s_cu[b] : p.seq_len[b];
    }
  }
  if (first == 0) {
    p.cu_rows[p.batch] = total;
    if (p.state) *p.n_free_out = ok ? n_free - pages : n_free;
    if (bad) raise_flag(p.flags, RKV_FLAG_BAD_INDEX);
    if (full) raise_flag(p.flags, RKV_FLAG_NO_SPACE);
  }
}

// The lengths and the free count after a planned step, from its offsets (all 0 where it was
// refused).  One CTA.
__global__ void __launch_bounds__(kPlanThreads) page_plan_state_kernel(PlanArgs p) {
  const int tid = threadIdx.x;
  const int64_t P1 = (1 << p.shift) - 1;
  const int n_free = *p.n_free;
  int taken = 0;
  for (int b = tid; b < p.batch; b += kPlanThreads) {
    const int len = p.seq_len[b], nw = p.cu_rows[b + 1] - p.cu_rows[b];
    if (nw > 0) taken += (int)((len + nw + P1) >> p.shift) - (int)((len + P1) >> p.shift);
    p.seq_len_out[b] = len + nw;
  }
  int64_t none = 0, total_none;
  int total;
  block_scan<kPlanThreads>(none, taken, total_none, total);
  if (tid == 0) *p.n_free_out = n_free - total;
}

// Release: the pages of the marked sequences, in order, of which those that are there (an entry
// of the table may be out of range) go to the end of the free list.  One CTA: a release moves
// a few thousand ids at a request's end.  Where all of them fit they go to the places that they
// have if all are pages (2048 of one sequence 8.8 us, 256 of each of 16 10.9 us, 12.9 us with
// their places scanned); where some are not, the others are moved up by a second pass.
constexpr int kReleasePages = 4;     // neighbouring entries of a thread in that pass

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
  const int room = num_blocks - n_free;
  // (s_first is exact where the pages fit its type)
  if (bad || pages > INT32_MAX) {
    if (tid == 0) raise_flag(flags, bad ? RKV_FLAG_BAD_INDEX : RKV_FLAG_NO_SPACE);
    return;
  }
  // of entry i: its place in the table
  auto entry = [&](int i) {
    const int seq = last_not_above(s_first, batch, i);
    return table + (int64_t)seq * max_blocks + (i - s_first[seq]);
  };
  auto is_page = [&](int id) { return id >= 0 && id < num_blocks; };
  if (pages > room) {                // fewer may be there
    int64_t here = 0, good;
    int c = 0, tc;
    for (int64_t i = tid; i < pages; i += kPlanThreads) here += is_page(*entry((int)i));
    block_scan<kPlanThreads>(here, c, good, tc);
    if (good > room) {
      if (tid == 0) raise_flag(flags, RKV_FLAG_NO_SPACE);
      return;
    }
  }
  const bool fit = pages <= room;
  bool stray = false;
  if (fit) {
    for (int64_t i = tid; i < pages; i += kPlanThreads) {
      int32_t* e = entry((int)i);
      const int id = *e;
      stray |= !is_page(id);
      free_blocks[n_free + i] = id;
      *e = -1;
    }
  }
  int placed = (int)pages;
  if (__syncthreads_or(stray) || !fit) {
    // (a pass reads its entries before it writes, and never behind them)
    placed = 0;
    stray = false;
    for (int64_t i0 = 0; i0 < pages; i0 += kPlanThreads * kReleasePages) {
      int id[kReleasePages];
      int here = 0, total;
      int64_t none = 0, total_none;
#pragma unroll
      for (int k = 0; k < kReleasePages; ++k) {
        const int64_t i = i0 + tid * kReleasePages + k;
        id[k] = -1;
        if (i < pages) {
          int32_t* e = fit ? free_blocks + n_free + i : entry((int)i);
          id[k] = *e;
          if (!fit) *e = -1;
          stray |= !is_page(id[k]);
        }
        here += is_page(id[k]);
      }
      const int mine = here;
      block_scan<kPlanThreads>(none, here, total_none, total);
      int at = n_free + placed + here - mine;
#pragma unroll
      for (int k = 0; k < kReleasePages; ++k)
        if (is_page(id[k])) free_blocks[at++] = id[k];
      placed += total;
    }
    if (stray) raise_flag(flags, RKV_FLAG_BAD_INDEX);
  }
  for (int b = tid; b < batch; b += kPlanThreads)
    if (finished[b] != 0) seq_len[b] = 0;
  if (tid == 0) *n_free_p = n_free + placed;
}

// ------------------------------------------------------------------------------ append
constexpr int kAppendThreads = 256;
constexpr int kAppendCtas = 10;

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

// Exponent e of the smallest scale 2^e with amax <= 448 2^e (448 = 1.75 2^8), in [-64, 120],
// from amax's bits.
__device__ __forceinline__ int scale_exponent(uint32_t u) {
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(-64, min(120, e));      // zero and subnormals: exponent field 0
}

__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Two floats to E4M3, nearest even, saturating (NaN stays NaN).
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// Eight codes of a stored row, rounded again at a scale grown by 1 / ratio (powers of two:
// the products are exact).
__device__ __forceinline__ void rescale8(uint8_t* codes, float ratio) {
  uint2* q = reinterpret_cast<uint2*>(codes);
  const uint2 old = *q;
  const uint32_t in[2] = {old.x, old.y};
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

// Bits of the largest finite magnitude of eight values (of floats of one sign, larger values
// have larger bits).
__device__ __forceinline__ uint32_t finite_max8(const float* f) {
  uint32_t a = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t m = __float_as_uint(f[e]) & 0x7FFFFFFFu;
    if (m < 0x7F800000u) a = max(a, m);
  }
  return a;
}
__device__ __forceinline__ uint2 codes8(const float* f, float inv) {
  uint32_t w[2];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    w[e] = to_e4m3x2(f[4 * e] * inv, f[4 * e + 1] * inv) |
           to_e4m3x2(f[4 * e + 2] * inv, f[4 * e + 3] * inv) << 16;
  return make_uint2(w[0], w[1]);
}

// Eight consecutive values of a row, as loaded and as floats.
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ uint32_t finite_max() const {
    const uint32_t m2 = __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu),
                                 __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
    const uint32_t m = max(m2 << 16, m2 & 0xFFFF0000u);
    if (m < 0x7F800000u) return m;
    float f[8];                      // an infinity or NaN among them
    get(f);
    return finite_max8(f);
  }
  __device__ __forceinline__ uint2 codes(float inv) const {
    float f[8];
    get(f);
    return codes8(f, inv);
  }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Chunk<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ uint32_t finite_max() const {
    float f[8];
    get(f);
    return finite_max8(f);
  }
  __device__ __forceinline__ uint2 codes(float inv) const {
    float f[8];
    get(f);
    return codes8(f, inv);
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
};

// The rows that a step brings to one run of 2^shift positions of a sequence.
struct Run {
  int seq, run;                      // positions run 2^shift ..
  int lo, hi;                        // rows [lo, hi) of the run are new
  int row;                           // packed row of the first
};

// Unit blockIdx.x: the u-th (sequence, run) that the step touches, in order.  False for units
// past the last.
__device__ __forceinline__ bool find_run(const AppendArgs& p, int shift, Run& out) {
  __shared__ Run s_run;
  const int tid = threadIdx.x, u = blockIdx.x, P1 = (1 << shift) - 1;
  const bool checks = u == 0 && blockIdx.y == 0 && blockIdx.z == 0;    // looks at every sequence
  if (tid == 0) s_run.seq = -1;
  int64_t base = 0;
  for (int b0 = 0; b0 < p.batch && (base <= u || checks); b0 += kAppendThreads) {
    const int b = b0 + tid;
    int lo = 0, hi = 0, r0 = 0;      // the step's positions [lo, hi) of sequence b
    if (b < p.batch) {
      r0 = p.cu[b];
      const int64_t rows = (int64_t)p.cu[b + 1] - r0, len = p.seq_len[b];
      if (rows != 0) {
        if (rows > 0 && r0 >= 0 && rows <= len && len <= (int64_t)p.max_blocks << p.shift) {
          lo = (int)(len - rows);
          hi = lo + (int)max((int64_t)0, min(rows, (int64_t)p.n_rows - r0));
          if (checks && hi - lo < rows) raise_flag(p.flags, RKV_FLAG_BAD_INDEX);
        } else if (checks) {
          raise_flag(p.flags, RKV_FLAG_BAD_INDEX);
        }
      }
    }
    const int touched = hi > lo ? (int)(((int64_t)hi + P1) >> shift) - (lo >> shift) : 0;
    int64_t a = touched, ta;
    int c = 0, tc;
    block_scan<kAppendThreads>(a, c, ta, tc);
    const int64_t mine = base + a - touched;
    if (u >= mine && u < base + a) {
      Run r;
      r.seq = b;
      r.run = (lo >> shift) + (int)(u - mine);
      const int64_t at = (int64_t)r.run << shift;
      r.lo = (int)max((int64_t)0, lo - at);
      r.hi = (int)min((int64_t)P1 + 1, hi - at);
      r.row = r0 + (int)(at + r.lo - lo);
      s_run = r;
    }
    base += ta;
  }
  __syncthreads();
  out = s_run;
  return out.seq >= 0;
}

// Id of page `page` of a sequence, -1 (and a flag) where it is out of range.
__device__ __forceinline__ int page_id(const AppendArgs& p, int seq, int page) {
  const int id = p.table[(int64_t)seq * p.max_blocks + page];
  if (id >= 0 && id < p.num_blocks) return id;
  raise_flag(p.flags, RKV_FLAG_BAD_INDEX);
  return -1;
}

constexpr int kRunTokens = 64;       // positions of a run, or a page where that is longer

// Grid (units, head groups, 2): unit u = the u-th (sequence, run) that the step touches, in
// order; kPar heads at a time, every gridDim.y-th such set; z: K or V.  D / 8 threads share a
// row; a thread holds kHold chunks of eight values of each head: those of rows r_in,
// r_in + kRows, ... of the run.  A warp's rows of one chunk lie in one page.
template <typename T, int D, int kPage>
__global__ void __launch_bounds__(kAppendThreads) page_append_kernel(AppendArgs p) {
  constexpr int kRun = kPage > kRunTokens ? kPage : kRunTokens;
  constexpr int kLanes = D / 8;                              // threads of one row
  constexpr int kRows = kAppendThreads / kLanes;             // rows of one pass: 16 or 32
  constexpr int kHold = kRun / kRows;                        // passes over a run
  constexpr int kPar = kHold >= 4 ? 1 : 4 / kHold;           // heads held at a time
  constexpr int kMerge = kPage > kRows ? kPage / kRows : 1;  // passes of one page
  constexpr int kMax = kHold / kMerge;                       // maxima of a thread
  constexpr int kWarps = kPage < kRows ? kAppendThreads / 32 * kPage / kRows : kAppendThreads / 32;   // of a page
  __shared__ __align__(16) uint32_t s_max[kPar][kMax][kAppendThreads / 32];
  __shared__ int s_id[kRun / kPage];
  const int tid = threadIdx.x, z = blockIdx.z, warp = tid >> 5;
  Run u;
  if (!find_run(p, __builtin_ctz(kRun), u)) return;
  if (tid < kRun / kPage) {
    const bool touched = tid * kPage < u.hi && (tid + 1) * kPage > u.lo;
    s_id[tid] = touched ? page_id(p, u.seq, u.run * (kRun / kPage) + tid) : -1;
  }
  __syncthreads();
  const int lane = tid % kLanes, r_in = tid / kLanes;
  // of chunk i: its row of the run, its page of the run, whether it is new and its page there
  auto row_of = [&](int i) { return i * kRows + r_in; };
  auto page_of = [&](int i) { return row_of(i) / kPage; };
  int id[kHold];
#pragma unroll
  for (int i = 0; i < kHold; ++i) id[i] = row_of(i) >= u.lo && row_of(i) < u.hi ? s_id[page_of(i)] : -1;
  // only the first page can hold earlier rows
  const int first = u.lo / kPage, before = u.lo % kPage, first_id = s_id[first];
  const T* rows = static_cast<const T*>(p.x[z]) + ((int64_t)u.row - u.lo) * p.st[z].row + lane * 8;
  for (int h0 = blockIdx.y * kPar; h0 < p.N; h0 += gridDim.y * kPar) {
    float held[kPar];
    uint32_t amax[kPar][kMax];
    Chunk<T> c[kPar][kHold];
#pragma unroll
    for (int g = 0; g < kPar; ++g) {
      held[g] = before > 0 && first_id >= 0 && h0 + g < p.N ? p.scale[z][(int64_t)first_id * p.N + h0 + g] : 0.f;
      const T* x = rows + (int64_t)(h0 + g) * p.st[z].head;
#pragma unroll
      for (int i = 0; i < kHold; ++i)
        if (h0 + g < p.N && id[i] >= 0) c[g][i].load(x + (int64_t)row_of(i) * p.st[z].row);
    }
#pragma unroll
    for (int g = 0; g < kPar; ++g) {
#pragma unroll
      for (int m = 0; m < kMax; ++m) {
        uint32_t x = 0;
#pragma unroll
        for (int i = m * kMerge; i < (m + 1) * kMerge; ++i)
          if (h0 + g < p.N && id[i] >= 0) x = max(x, c[g][i].finite_max());
        amax[g][m] = __reduce_max_sync(0xffffffffu, x);
      }
    }
    __syncthreads();                 // the last heads' maxima have been read
    if ((tid & 31) == 0) {
#pragma unroll
      for (int g = 0; g < kPar; ++g)
#pragma unroll
        for (int m = 0; m < kMax; ++m) s_max[g][m][warp] = amax[g][m];
    }
    __syncthreads();                 // every thread has read the held scales
#pragma unroll
    for (int g = 0; g < kPar; ++g) {
      if (h0 + g >= p.N) break;
#pragma unroll
      for (int m = 0; m < kMax; ++m) {
        uint32_t x = 0;
#pragma unroll
        for (int w = 0; w < kWarps; w += 4) {
          const uint4 y = *reinterpret_cast<const uint4*>(&s_max[g][m][warp / kWarps * kWarps + w]);
          x = max(max(max(x, y.x), max(y.y, y.z)), y.w);
        }
        const int page = page_of(m * kMerge), pid = s_id[page];
        if (pid < 0) continue;
        const bool grows = page == first && before > 0;
        const float need = pow2i(scale_exponent(x));
        const float s = grows && held[g] > need ? held[g] : need;
        const float inv = 1.f / s;   // a power of two: exact
        const int64_t head = (int64_t)pid * p.N + h0 + g;
        uint8_t* codes = p.codes[z] + (head * kPage) * D + lane * 8;
        if (row_of(m * kMerge) % kPage == 0 && lane == 0) p.scale[z][head] = s;
#pragma unroll
        for (int i = m * kMerge; i < (m + 1) * kMerge; ++i)
          if (id[i] >= 0)
            *reinterpret_cast<uint2*>(codes + (int64_t)(row_of(i) % kPage) * D) = c[g][i].codes(inv);
        if (grows && held[g] > 0.f && held[g] < s)
          for (int r = row_of(m * kMerge) % kPage; r < before; r += kRows < kPage ? kRows : kPage)
            rescale8(codes + (int64_t)r * D, held[g] / s);
      }
    }
  }
}

// The same for calls of few rows a sequence: a warp takes one head of a page, D / 32 values a
// lane, and reads its rows twice where there are several.  Grid (units, ceil(N / 8), 2).
template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads) page_append_narrow_kernel(AppendArgs p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;         // rows of one pass of a warp
  const int tid = threadIdx.x, z = blockIdx.z, h = blockIdx.y * (kAppendThreads / 32) + (tid >> 5);
  Run u;
  if (!find_run(p, p.shift, u) || h >= p.N) return;
  const int id = page_id(p, u.seq, u.run);
  if (id < 0) return;
  const int lane = tid % kLanes, r_in = (tid & 31) / kLanes, n = u.hi - u.lo;
  const int64_t head = (int64_t)id * p.N + h;
  const T* x = static_cast<const T*>(p.x[z]) + (int64_t)u.row * p.st[z].row + (int64_t)h * p.st[z].head + lane * 8;
  const float held = u.lo > 0 ? p.scale[z][head] : 0.f;
  Chunk<T> c;
  uint32_t amax = 0;
  for (int r = r_in; r < n; r += kRows) {
    c.load(x + (int64_t)r * p.st[z].row);
    amax = max(amax, c.finite_max());
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  const float need = pow2i(scale_exponent(amax));
  const float s = held > need ? held : need;
  const float inv = 1.f / s;
  uint8_t* codes = p.codes[z] + (head << p.shift) * D + lane * 8;
  __syncwarp();                      // every lane has read the held scale
  if ((tid & 31) == 0) p.scale[z][head] = s;
  for (int r = r_in; r < n; r += kRows) {
    if (n > kRows) c.load(x + (int64_t)r * p.st[z].row);   // else still held
    *reinterpret_cast<uint2*>(codes + (int64_t)(u.lo + r) * D) = c.codes(inv);
  }
  if (held > 0.f && held < s)
    for (int r = r_in; r < u.lo; r += kRows) rescale8(codes + (int64_t)r * D, held / s);
}

int log2_block(int block_tokens) {
  int s = 0;
  while ((1 << s) < block_tokens) ++s;
  return s;
}

bool block_ok(int b) { return b == 16 || b == 32 || b == 64 || b == 128; }

// Runs that a step can touch: a sequence's rows touch at most (rows - 2) / length + 2, and no
// more than its rows.
int64_t touched_runs(const AppendArgs& a, int length) {
  const int64_t bound = (int64_t)a.n_rows / length + 2 * (int64_t)a.batch;
  return bound < a.n_rows ? bound : a.n_rows;
}

template <typename T, int D, int kPage>
void launch_page(const AppendArgs& a, int sms, cudaStream_t s) {
  constexpr int kRun = kPage > kRunTokens ? kPage : kRunTokens;
  constexpr int kHold = kRun * D / 8 / kAppendThreads, kPar = kHold >= 4 ? 1 : 4 / kHold;
  const int64_t units = touched_runs(a, kRun);
  // head groups: as few heads a CTA as make kAppendCtas CTAs an SM
  const int64_t groups = (int64_t)kAppendCtas * sms / (2 * units) + 1, most = ceil_div(a.N, kPar);
  page_append_kernel<T, D, kPage><<<dim3((unsigned)units, (unsigned)(groups < most ? groups : most), 2),
                                    kAppendThreads, 0, s>>>(a);
}

template <typename T, int D>
void launch_append(const AppendArgs& a, int block_tokens, int sms, cudaStream_t s) {
  // Up to two rows a sequence on average: a warp a head (8 heads of 128, pages of 64: one row
  // for each of 256 sequences 3.9 us, 11.8 with the other kernel, two for each of 64 3.0 and
  // 6.8.  512 rows of one sequence of 256: 8.8 and 8.2, on pages of 16 4.5 and 10.7).
  if (a.n_rows <= 2 * a.batch) {
    const dim3 grid((unsigned)touched_runs(a, block_tokens), (unsigned)ceil_div(a.N, kAppendThreads / 32), 2);
    page_append_narrow_kernel<T, D><<<grid, kAppendThreads, 0, s>>>(a);
    return;
  }
  switch (block_tokens) {
    case 16: launch_page<T, D, 16>(a, sms, s); break;
    case 32: launch_page<T, D, 32>(a, sms, s); break;
    case 64: launch_page<T, D, 64>(a, sms, s); break;
    default: launch_page<T, D, 128>(a, sms, s); break;
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
  // (the reads count positions up to the end of a tile of 128)
  if (t->max_blocks < 1 || (int64_t)t->max_blocks * block_tokens > INT32_MAX - 127)
    return fail_with(RKV_EINVAL, "max_blocks must be >= 1 and max_blocks * block_tokens at most 2^31 - 128");
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
  // one CTA for up to four rows a thread twice over; then as many as that takes
  int ctas = 1;
  if (max_rows > 2 * kPlanRows * kPlanThreads) ctas = (max_rows - 1) / (kPlanRows * kPlanThreads) + 1;
  ctas = ctas < kPlanMaxCtas ? ctas : kPlanMaxCtas;
  const bool in_place = seq_len_out == a.seq_len || n_free_out == n_free;
  a.state = ctas == 1 || !in_place;
  const size_t smem = sizeof(int) * 3 * (size_t)a.batch;
  static SmemOptIn opt_in;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      opt_in(page_plan_kernel, sizeof(int) * 3 * (size_t)kMaxBatch, dev) != cudaSuccess)
    return fail_with(RKV_ECUDA, "no usable current device");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  page_plan_kernel<<<ctas, kPlanThreads, smem, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && !a.state) {
    page_plan_state_kernel<<<1, kPlanThreads, 0, s>>>(a);
    e = cudaGetLastError();
  }
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
  int dev = 0, sms = 0;
  if (!current_device(dev, sms)) return fail_with(RKV_ECUDA, "no usable current device");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int P = pages->block_tokens;
  if (dtype == RKV_F32)
    pages->head_dim == 128 ? launch_append<float, 128>(a, P, sms, s)
                           : launch_append<float, 64>(a, P, sms, s);
  else
    pages->head_dim == 128 ? launch_append<__nv_bfloat16, 128>(a, P, sms, s)
                           : launch_append<__nv_bfloat16, 64>(a, P, sms, s);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? RKV_OK : fail_with(RKV_ECUDA, "page append launch failed: %s", cudaGetErrorString(e));
}
