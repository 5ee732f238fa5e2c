// k_page_share.cu - pages that several sequences hold: rows of the table forked, cut and freed,
// pages compacted, pages copied in the caches, stored rows gathered.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "pages.h"

namespace rkv {
namespace {

// ------------------------------------------------------------------- table operations
// One cluster does a call, so that its phases can wait for one another; a warp takes a run of
// tasks (128 neighbouring entries of a row of the table), the same ones in every phase.
constexpr int kTableThreads = 1024;
constexpr int kTableWarps = kTableThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kTaskEntries = 128;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Every thread's earlier writes are seen by every thread of the cluster afterwards.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct Tasks {
  int first, last, per_row;          // this warp's [first, last)
  __device__ __forceinline__ Tasks(int batch, int width) {
    per_row = (width + kTaskEntries - 1) / kTaskEntries;
    const int64_t n = (int64_t)batch * per_row;
    const int64_t warps = (int64_t)cluster_size() * kTableWarps;
    const int64_t w = (int64_t)cluster_rank() * kTableWarps + threadIdx.x / 32;
    first = (int)(n * w / warps), last = (int)(n * (w + 1) / warps);
  }
};

struct ForkArgs {
  const int32_t* source;
  const int32_t* length;
  const int32_t* finished;
  const int32_t* table;
  const int32_t* seq_len;
  int32_t* table_out;
  int32_t* seq_len_out;
  int32_t* free_blocks;
  const int32_t* n_free;
  int32_t* n_free_out;
  int32_t* copy_src;
  int32_t* copy_dst;
  int32_t* copy_rows;
  int32_t* held;                     // [num_blocks] -1: held whole; the first row that has begun it; kNone
  int32_t* first;                    // [num_blocks] first entry of the old table that may give it up
  int32_t* counts;                   // [warps] pages that a warp's tasks free
  int32_t* stage;                    // [batch, max_blocks] new rows, for a table changed in place
  int32_t* flags;
  int batch, max_blocks, num_blocks, shift;
};

constexpr int kNone = INT32_MAX;

// The table, lengths and count as they were, and no copies.
__device__ __forceinline__ void fork_refused(const ForkArgs& p, int32_t flag, int n_free) {
  const int64_t step = (int64_t)cluster_size() * kTableThreads, at = (int64_t)cluster_rank() * kTableThreads + threadIdx.x;
  if (p.table_out != p.table)
    for (int64_t i = at; i < (int64_t)p.batch * p.max_blocks; i += step) p.table_out[i] = p.table[i];
  for (int64_t b = at; b < p.batch; b += step) {
    if (p.seq_len_out != p.seq_len) p.seq_len_out[b] = p.seq_len[b];
    p.copy_src[b] = p.copy_dst[b] = -1;
    p.copy_rows[b] = 0;
  }
  if (at == 0) {
    if (p.n_free_out != p.n_free) *p.n_free_out = n_free;
    raise_flag(p.flags, flag);
  }
}

__global__ void __launch_bounds__(kTableThreads) page_fork_kernel(const __grid_constant__ ForkArgs p) {
  extern __shared__ int fsm[];
  int* s_src = fsm;                  // [batch] source row, -1: none
  int* s_new = s_src + p.batch;      // [batch] positions after the call
  int* s_have = s_new + p.batch;     // [batch] pages before it
  int* s_copy = s_have + p.batch;    // [batch] place among the copies, -1: none
  int* s_from = s_copy + p.batch;    // [batch] page that is copied
  __shared__ int s_width, s_base[kTableWarps];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  const int P1 = (1 << p.shift) - 1, M = p.max_blocks;
  const int64_t cap = (int64_t)M << p.shift;
  const bool in_place = p.table_out == p.table;
  const int n_free = *p.n_free;
  auto is_page = [&](int id) { return id >= 0 && id < p.num_blocks; };
  auto pages = [&](int n) { return (int)(((int64_t)n + P1) >> p.shift); };

  for (int i = rank * kTableThreads + tid; i < p.num_blocks; i += ctas * kTableThreads) p.held[i] = p.first[i] = kNone;
  if (tid == 0) s_width = 0;
  bool bad = n_free < 0 || n_free > p.num_blocks;
  int width = 0;
  for (int b = tid; b < p.batch; b += kTableThreads) {
    int len = p.seq_len[b], s = p.source ? p.source[b] : b, n = 0;
    if (p.finished && p.finished[b] != 0) s = -1;
    if (len < 0 || len > cap) bad = true, len = 0;
    if (s >= p.batch) bad = true, s = -1;
    if (s >= 0) {
      const int all = p.seq_len[s];
      n = p.length && p.length[b] >= 0 ? p.length[b] : all;
      if (n < 0 || n > all || all > cap) bad = true, n = 0;
    }
    s_src[b] = max(s, -1);
    s_new[b] = n;
    s_have[b] = pages(len);
    width = max(width, max(s_have[b], pages(n)));
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    fork_refused(p, RKV_FLAG_BAD_INDEX, n_free);
    return;
  }
  atomicMax(&s_width, width);
  cluster_sync();
  const Tasks tasks(p.batch, in_place ? s_width : M);

  // who holds what: rows after the call, and the entries that go
  bool stray = false;
  for (int t = tasks.first; t < tasks.last; ++t) {
    const int b = t / tasks.per_row, j0 = (t - b * tasks.per_row) * kTaskEntries;
    const int s = s_src[b], n = s_new[b], m = pages(n), have = s_have[b];
#pragma unroll
    for (int k = 0; k < kTaskEntries / 32; ++k) {
      const int j = j0 + k * 32 + lane;
      if (j < m) {
        const int id = p.table[(int64_t)s * M + j];
        if (in_place && s != b) p.stage[(int64_t)b * M + j] = id;
        if (is_page(id)) atomicMin(p.held + id, j == m - 1 && (n & P1) ? b : -1);
        else stray = true;
      }
      if (j < have && (s != b || j >= m)) {
        const int id = p.table[(int64_t)b * M + j];
        if (is_page(id)) atomicMin(p.first + id, b * M + j);
        else stray = true;
      }
    }
  }
  if (stray) raise_flag(p.flags, RKV_FLAG_BAD_INDEX);
  cluster_sync();

  // pages that go, in the order of the entries; copies, in that of the rows
  auto freed = [&](int b, int j, int& id) {
    const int s = s_src[b];
    if (j >= s_have[b] || (s == b && j < pages(s_new[b]))) return false;
    id = p.table[(int64_t)b * M + j];
    return is_page(id) && __ldcg(p.held + id) == kNone && __ldcg(p.first + id) == b * M + j;
  };
  int gone = 0;
  for (int t = tasks.first; t < tasks.last; ++t) {
    const int b = t / tasks.per_row, j0 = (t - b * tasks.per_row) * kTaskEntries;
#pragma unroll
    for (int k = 0; k < kTaskEntries / 32; ++k) {
      int id;
      gone += __popc(__ballot_sync(0xffffffffu, freed(b, j0 + k * 32 + lane, id)));
    }
  }
  if (lane == 0) p.counts[rank * kTableWarps + wid] = gone;
  int copies = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kTableThreads) {
    const int b = b0 + tid;
    int id = -1;
    if (b < p.batch && (s_new[b] & P1)) {
      id = p.table[(int64_t)s_src[b] * M + pages(s_new[b]) - 1];
      if (!is_page(id) || __ldcg(p.held + id) == b) id = -1;
    }
    int64_t none = 0, total_none;
    int c = id >= 0, total;
    block_scan<kTableThreads>(none, c, total_none, total);
    if (b < p.batch) {
      s_copy[b] = id >= 0 ? copies + c - 1 : -1;
      s_from[b] = id;
    }
    copies += total;
  }
  cluster_sync();

  int64_t none = 0, total_none;
  const int warps = ctas * kTableWarps;
  const int mine = tid < warps ? __ldcg(p.counts + tid) : 0;
  int before = mine, total;
  static_assert(kMaxCluster * kTableWarps <= kTableThreads);
  block_scan<kTableThreads>(none, before, total_none, total);
  if (tid / kTableWarps == rank) s_base[tid % kTableWarps] = before - mine;
  __syncthreads();
  const int64_t end = (int64_t)n_free + total;
  if (end > p.num_blocks || end < copies) {
    fork_refused(p, RKV_FLAG_NO_SPACE, n_free);
    return;
  }
  int at = n_free + s_base[wid];
  for (int t = tasks.first; t < tasks.last; ++t) {
    const int b = t / tasks.per_row, j0 = (t - b * tasks.per_row) * kTaskEntries;
#pragma unroll
    for (int k = 0; k < kTaskEntries / 32; ++k) {
      int id;
      const bool goes = freed(b, j0 + k * 32 + lane, id);
      const uint32_t all = __ballot_sync(0xffffffffu, goes);
      if (goes) p.free_blocks[at + __popc(all & ((1u << lane) - 1))] = id;
      at += __popc(all);
    }
  }
  cluster_sync();

  for (int t = tasks.first; t < tasks.last; ++t) {
    const int b = t / tasks.per_row, j0 = (t - b * tasks.per_row) * kTaskEntries;
    const int s = s_src[b], m = pages(s_new[b]);
#pragma unroll
    for (int k = 0; k < kTaskEntries / 32; ++k) {
      const int j = j0 + k * 32 + lane;
      int32_t* out = p.table_out + (int64_t)b * M + j;
      if (j < m) {
        if (j == m - 1 && s_copy[b] >= 0) *out = __ldcg(p.free_blocks + (end - 1 - s_copy[b]));
        else if (!in_place) *out = p.table[(int64_t)s * M + j];
        else if (s != b) *out = p.stage[(int64_t)b * M + j];
      } else if (j < (in_place ? s_have[b] : M)) {
        *out = -1;
      }
    }
  }
  for (int b = rank * kTableThreads + tid; b < p.batch; b += ctas * kTableThreads) {
    const int c = s_copy[b];
    p.seq_len_out[b] = s_new[b];
    p.copy_src[b] = s_from[b];
    p.copy_dst[b] = c >= 0 ? __ldcg(p.free_blocks + (end - 1 - c)) : -1;
    p.copy_rows[b] = c >= 0 ? s_new[b] & P1 : 0;
  }
  if (rank == 0 && tid == 0) *p.n_free_out = (int)(end - copies);
}

struct CompactArgs {
  const int32_t* table;
  const int32_t* seq_len;
  int32_t* table_out;
  int32_t* free_blocks;
  int32_t* n_free;
  int32_t* src;
  int32_t* dst;
  int32_t* count;
  uint32_t* bits;                    // [words] held pages
  int32_t* before;                   // [words] held pages before a word's
  int32_t* totals;                   // [CTAs] held pages of a CTA's words
  int32_t* flags;
  int batch, max_blocks, num_blocks, shift;
};

__global__ void __launch_bounds__(kTableThreads) page_compact_kernel(const __grid_constant__ CompactArgs p) {
  extern __shared__ int fsm[];
  int* s_have = fsm;                 // [batch] pages
  __shared__ int s_width, s_low;
  const int tid = threadIdx.x, lane = tid & 31;
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  const int step = ctas * kTableThreads, me = rank * kTableThreads + tid;
  const int P1 = (1 << p.shift) - 1, M = p.max_blocks, num = p.num_blocks;
  const int words = (int)(((int64_t)num + 31) / 32), places = num / 2;
  const bool in_place = p.table_out == p.table;
  auto is_page = [&](int id) { return id >= 0 && id < num; };

  for (int i = me; i < words; i += step) p.bits[i] = 0;
  if (tid == 0) s_width = s_low = 0;
  bool bad = false;
  int width = 0;
  for (int b = tid; b < p.batch; b += kTableThreads) {
    int len = p.seq_len[b];
    if (len < 0 || len > (int64_t)M << p.shift) bad = true, len = 0;
    s_have[b] = (int)(((int64_t)len + P1) >> p.shift);
    width = max(width, s_have[b]);
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (!in_place)
      for (int64_t i = me; i < (int64_t)p.batch * M; i += step) p.table_out[i] = p.table[i];
    for (int i = me; i < places; i += step) p.src[i] = p.dst[i] = -1;
    if (me == 0) *p.count = 0, raise_flag(p.flags, RKV_FLAG_BAD_INDEX);
    return;
  }
  atomicMax(&s_width, width);
  cluster_sync();
  const Tasks tasks(p.batch, in_place ? s_width : M);

  bool stray = false;
  for (int t = tasks.first; t < tasks.last; ++t) {
    const int b = t / tasks.per_row, j0 = (t - b * tasks.per_row) * kTaskEntries;
#pragma unroll
    for (int k = 0; k < kTaskEntries / 32; ++k) {
      const int j = j0 + k * 32 + lane;
      if (j < s_have[b]) {
        const int id = p.table[(int64_t)b * M + j];
        if (is_page(id)) atomicOr(p.bits + (id >> 5), 1u << (id & 31));
        else stray = true;
      }
    }
  }
  if (stray) raise_flag(p.flags, RKV_FLAG_BAD_INDEX);
  cluster_sync();

  // this CTA's words, neighbouring ones to a thread
  const int w0 = (int)((int64_t)words * rank / ctas), w1 = (int)((int64_t)words * (rank + 1) / ctas);
  const int each = (w1 - w0 + kTableThreads - 1) / kTableThreads;
  const int from = min(w1, w0 + tid * each), to = min(w1, from + each);
  int mine = 0;
  for (int w = from; w < to; ++w) mine += __popc(__ldcg(p.bits + w));
  int64_t none = 0, total_none;
  int sum = mine, total;
  block_scan<kTableThreads>(none, sum, total_none, total);
  if (tid == 0) p.totals[rank] = total;
  cluster_sync();
  int n_live = 0, base = 0, low = 0;
  uint32_t owner = 0;                // of the word of page n_live
  for (uint32_t c = 0; c < ctas; ++c) {
    if (c == rank) base = n_live;
    n_live += __ldcg(p.totals + c);
  }
  // held pages below n_live: those of the CTAs before that word's, and of its own words
  for (uint32_t c = 0, sofar = 0; c < ctas; ++c) {
    if ((int)((int64_t)words * c / ctas) <= n_live >> 5) owner = c, low = sofar;
    sofar += __ldcg(p.totals + c);
  }
  int part = 0;
  for (int w = (int)((int64_t)words * owner / ctas) + tid; w <= n_live >> 5 && w < words; w += kTableThreads) {
    const uint32_t x = __ldcg(p.bits + w);
    part += __popc(w == n_live >> 5 ? x & ((1u << (n_live & 31)) - 1) : x);
  }
  part = __reduce_add_sync(0xffffffffu, part);
  if (lane == 0 && part) atomicAdd(&s_low, part);
  __syncthreads();
  low += s_low;
  const int moves = n_live - low;
  int at = base + sum - mine;
  for (int w = from; w < to; ++w) {
    const uint32_t x = __ldcg(p.bits + w);
    p.before[w] = at;
    int live = at;
    for (int i = 0; i < 32 && w * 32 + i < num; ++i) {
      const int id = w * 32 + i;
      if (x >> i & 1) {
        if (id >= n_live) p.src[live - low] = id;
        ++live;
      } else if (id < n_live) {
        p.dst[id - live] = id;
      }
    }
    at += __popc(x);
  }
  cluster_sync();

  for (int t = tasks.first; t < tasks.last; ++t) {
    const int b = t / tasks.per_row, j0 = (t - b * tasks.per_row) * kTaskEntries;
#pragma unroll
    for (int k = 0; k < kTaskEntries / 32; ++k) {
      const int j = j0 + k * 32 + lane;
      const int64_t e = (int64_t)b * M + j;
      if (j < s_have[b]) {
        const int id = p.table[e];
        if (is_page(id) && id >= n_live) {
          const int r = __ldcg(p.before + (id >> 5)) + __popc(__ldcg(p.bits + (id >> 5)) & ((1u << (id & 31)) - 1));
          p.table_out[e] = __ldcg(p.dst + (r - low));
        } else if (!in_place) {
          p.table_out[e] = id;
        }
      } else if (!in_place && j < M) {
        p.table_out[e] = -1;
      }
    }
  }
  for (int i = me; i < num - n_live; i += step) p.free_blocks[i] = num - 1 - i;
  for (int i = moves + me; i < places; i += step) p.src[i] = p.dst[i] = -1;
  if (me == 0) *p.n_free = num - n_live, *p.count = moves;
}

// Launches a table kernel as one cluster of as many CTAs as its entries fill.
template <typename Args>
cudaError_t launch_table(void (*kernel)(Args), const Args& a, int batch, int max_blocks, size_t smem, cudaStream_t s) {
  const int64_t warps = (int64_t)batch * ceil_div(max_blocks, kTaskEntries);
  unsigned ctas = 1;
  while (ctas < kMaxCluster && (int64_t)ctas * kTableWarps < warps) ctas *= 2;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {ctas, 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kTableThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// ------------------------------------------------------------------------- page copies
constexpr int kCopyThreads = 256;
constexpr int kCopyLayers = 128;
constexpr int kCopyLoads = 8;        // 16-byte loads of a lane in flight

struct CopyLayer {
  uint8_t* codes[2];
  float* scale[2];
};
struct CopyArgs {
  CopyLayer layer[kCopyLayers];
  const int32_t* src;
  const int32_t* dst;
  const int32_t* rows;
  const int32_t* count;
  int32_t* flags;
  int layers, n, N, num_blocks, block_tokens, head_dim;
};

// A warp copies the rows of one (pair, layer, K or V, head), which lie side by side.
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const __grid_constant__ CopyArgs p) {
  const int lane = threadIdx.x & 31;
  const int n = p.count ? max(0, min(p.n, *p.count)) : p.n;
  const int64_t items = (int64_t)n * p.layers * 2 * p.N;
  const int64_t head_bytes = (int64_t)p.block_tokens * p.head_dim;
  for (int64_t it = (int64_t)blockIdx.x * (kCopyThreads / 32) + threadIdx.x / 32; it < items;
       it += (int64_t)gridDim.x * (kCopyThreads / 32)) {
    const int h = (int)(it % p.N);
    const int64_t rest = it / p.N;
    const int kv = (int)(rest & 1), layer = (int)((rest >> 1) % p.layers), i = (int)((rest >> 1) / p.layers);
    const int from = p.src[i], to = p.dst[i];
    int rows = p.rows ? p.rows[i] : p.block_tokens;
    if (from < 0 && to < 0) continue;
    if (from < 0 || to < 0 || from >= p.num_blocks || to >= p.num_blocks || rows < 0 || rows > p.block_tokens) {
      if (lane == 0) raise_flag(p.flags, RKV_FLAG_BAD_INDEX);
      continue;
    }
    const CopyLayer& c = p.layer[layer];
    const int64_t sh = (int64_t)from * p.N + h, dh = (int64_t)to * p.N + h;
    const uint4* a = reinterpret_cast<const uint4*>(c.codes[kv] + sh * head_bytes);
    uint4* b = reinterpret_cast<uint4*>(c.codes[kv] + dh * head_bytes);
    const int chunks = rows * p.head_dim / 16;
    for (int x0 = lane; x0 < chunks; x0 += 32 * kCopyLoads) {
      uint4 u[kCopyLoads];
#pragma unroll
      for (int k = 0; k < kCopyLoads; ++k)
        if (x0 + 32 * k < chunks) u[k] = a[x0 + 32 * k];
#pragma unroll
      for (int k = 0; k < kCopyLoads; ++k)
        if (x0 + 32 * k < chunks) b[x0 + 32 * k] = u[k];
    }
    if (lane == 0) c.scale[kv][dh] = c.scale[kv][sh];
  }
}

// ------------------------------------------------------------------------------ gather
constexpr int kGatherThreads = 256;
constexpr int kGatherRows = 16;      // positions of a chunk: never in two pages
constexpr int kGatherCtas = 4;       // CTAs an SM

struct GatherArgs {
  const uint8_t* codes[2];
  const float* scale[2];
  const int32_t* table;
  const int32_t* seq_len;
  const int32_t* length;
  __nv_bfloat16* out[2];
  Strides st[2];
  int32_t* cu;
  int32_t* flags;
  int batch, max_blocks, num_blocks, N, shift, max_rows, shares;
};

// A warp takes a share of the heads of one chunk.
template <int D>
__global__ void __launch_bounds__(kGatherThreads) page_gather_kernel(const __grid_constant__ GatherArgs p) {
  constexpr int kLanes = D / 16;                 // lanes of one row
  constexpr int kRows = 32 / kLanes;             // rows of one load
  constexpr int kLoads = kGatherRows / kRows;
  extern __shared__ int fsm[];
  int* s_cu = fsm;                   // [batch] first row of each sequence
  int* s_chunk = s_cu + p.batch;     // [batch] first chunk of each
  const int tid = threadIdx.x, lane = tid & 31;
  int64_t rows = 0;
  int chunks = 0;                    // exact wherever the rows fit
  bool bad = false;
  for (int b0 = 0; b0 < p.batch; b0 += kGatherThreads) {
    const int b = b0 + tid;
    int len = 0;
    if (b < p.batch) {
      const int all = p.seq_len[b];
      len = p.length ? p.length[b] : all;
      if (len < 0 || len > all || all > (int64_t)p.max_blocks << p.shift) bad = true, len = 0;
    }
    const int mine = (int)(((int64_t)len + kGatherRows - 1) / kGatherRows);
    int64_t a = len, ta;
    int c = mine, tc;
    block_scan<kGatherThreads>(a, c, ta, tc);
    if (b < p.batch) {
      s_cu[b] = (int)min(rows + a - len, (int64_t)INT32_MAX);
      s_chunk[b] = chunks + c - mine;
    }
    rows += ta;
    chunks += tc;
  }
  bad = __syncthreads_or(bad);
  const bool full = !bad && rows > p.max_rows, ok = !bad && !full;
  const int total = ok ? (int)rows : 0;
  if (blockIdx.x == 0) {
    for (int b = tid; b < p.batch; b += kGatherThreads) p.cu[b] = ok ? s_cu[b] : 0;
    if (tid == 0) {
      p.cu[p.batch] = total;
      if (bad) raise_flag(p.flags, RKV_FLAG_BAD_INDEX);
      if (full) raise_flag(p.flags, RKV_FLAG_NO_SPACE);
    }
  }
  if (!ok) return;
  const int64_t tasks = (int64_t)chunks * p.shares;
  const int r_in = lane / kLanes, x = (lane % kLanes) * 16;
  for (int64_t task = (int64_t)blockIdx.x * (kGatherThreads / 32) + tid / 32; task < tasks;
       task += (int64_t)gridDim.x * (kGatherThreads / 32)) {
    const int chunk = (int)(task / p.shares), share = (int)(task - (int64_t)chunk * p.shares);
    const int b = last_not_above(s_chunk, p.batch, chunk);
    const int j0 = (chunk - s_chunk[b]) * kGatherRows, row0 = s_cu[b] + j0;
    const int left = (b + 1 < p.batch ? s_cu[b + 1] : total) - row0;           // rows of the chunk, or more
    const int id = p.table[(int64_t)b * p.max_blocks + (j0 >> p.shift)];
    const bool there = id >= 0 && id < p.num_blocks;
    if (!there && lane == 0) raise_flag(p.flags, RKV_FLAG_BAD_INDEX);
    const int lo = (int)((int64_t)p.N * share / p.shares), hi = (int)((int64_t)p.N * (share + 1) / p.shares);
    for (int h = lo; h < hi; ++h) {
      const int64_t head = (int64_t)id * p.N + h;
      uint4 u[2][kLoads];
      float s[2];
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint8_t* src = p.codes[kv] + ((head << p.shift) + (j0 & ((1 << p.shift) - 1))) * D + x;
        s[kv] = there ? p.scale[kv][head] : 0.0f;
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int r = k * kRows + r_in;
          u[kv][k] = make_uint4(0, 0, 0, 0);
          if (there && r < left) u[kv][k] = *reinterpret_cast<const uint4*>(src + r * D);
        }
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int r = k * kRows + r_in;
          if (r >= left) continue;
          const uint32_t in[4] = {u[kv][k].x, u[kv][k].y, u[kv][k].z, u[kv][k].w};
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((uint16_t)(in[e / 2] >> (16 * (e & 1))), __NV_E4M3);
            const float2 v = __half22float2(__half2(hr));
            const __nv_bfloat162 t = __floats2bfloat162_rn(v.x * s[kv], v.y * s[kv]);
            w[e] = *reinterpret_cast<const uint32_t*>(&t);
          }
          uint4* dst = reinterpret_cast<uint4*>(p.out[kv] + (int64_t)(row0 + r) * p.st[kv].row + (int64_t)h * p.st[kv].head + x);
          dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
          dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
    }
  }
}

rkv_status check_fork_table(const rkv_page_table* table, int32_t num_blocks, int32_t block_tokens) {
  if (!block_ok(block_tokens)) return fail_with(RKV_EINVAL, "block_tokens must be 16, 32, 64 or 128");
  if (rkv_status st = check_table(table, block_tokens)) return st;
  if (num_blocks < 1 || (int64_t)num_blocks * block_tokens > INT32_MAX)
    return fail_with(RKV_EINVAL, "num_blocks must be >= 1 and num_blocks * block_tokens below 2^31");
  if ((int64_t)table->batch * table->max_blocks > INT32_MAX)
    return fail_with(RKV_EINVAL, "batch * max_blocks must be below 2^31");
  return RKV_OK;
}

size_t round16(size_t n) { return (n + 15) & ~(size_t)15; }

size_t fork_bytes(const rkv_page_table* t, int num_blocks) {
  return 4 * (2 * round16(num_blocks) + kMaxCluster * kTableWarps + (size_t)t->batch * t->max_blocks);
}
size_t compact_bytes(int num_blocks) { return 4 * (2 * round16(((size_t)num_blocks + 31) / 32) + kMaxCluster); }

rkv_status check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (!workspace || bytes < need)
    return fail_with(RKV_ECAPACITY, "workspace has %zu of %zu bytes", workspace ? bytes : (size_t)0, need);
  if (!is_aligned(workspace, 16)) return fail_with(RKV_EALIGN, "workspace must be 16-byte aligned");
  return RKV_OK;
}

}  // namespace
}  // namespace rkv

using namespace rkv;

extern "C" rkv_status rkv_page_fork_workspace(const rkv_page_table* table, int32_t num_blocks,
                                              int32_t block_tokens, size_t* bytes) {
  if (!bytes) return fail_with(RKV_EINVAL, "bytes is NULL");
  if (rkv_status st = check_fork_table(table, num_blocks, block_tokens)) return st;
  *bytes = fork_bytes(table, num_blocks);
  return RKV_OK;
}

extern "C" rkv_status rkv_page_fork(const rkv_page_table* table, const int32_t* source, const int32_t* length,
                                    const int32_t* finished, int32_t* free_blocks, const int32_t* n_free,
                                    int32_t num_blocks, int32_t block_tokens, int32_t* block_table_out,
                                    int32_t* seq_len_out, int32_t* n_free_out, int32_t* copy_src,
                                    int32_t* copy_dst, int32_t* copy_rows, void* workspace,
                                    size_t workspace_bytes, int32_t* flags, void* stream) {
  if (rkv_status st = check_fork_table(table, num_blocks, block_tokens)) return st;
  if (!free_blocks || !n_free || !block_table_out || !seq_len_out || !n_free_out || !copy_src || !copy_dst || !copy_rows)
    return fail_with(RKV_EINVAL, "NULL pointer");
  if (rkv_status st = check_workspace(workspace, workspace_bytes, fork_bytes(table, num_blocks))) return st;
  ForkArgs a;
  a.source = source, a.length = length, a.finished = finished;
  a.table = table->block_table, a.seq_len = table->seq_len;
  a.table_out = block_table_out, a.seq_len_out = seq_len_out;
  a.free_blocks = free_blocks, a.n_free = n_free, a.n_free_out = n_free_out;
  a.copy_src = copy_src, a.copy_dst = copy_dst, a.copy_rows = copy_rows;
  a.held = static_cast<int32_t*>(workspace);
  a.first = a.held + round16(num_blocks);
  a.counts = a.first + round16(num_blocks);
  a.stage = a.counts + kMaxCluster * kTableWarps;
  a.flags = flags;
  a.batch = table->batch, a.max_blocks = table->max_blocks, a.num_blocks = num_blocks;
  a.shift = log2_block(block_tokens);
  static SmemOptIn opt_in;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || opt_in(page_fork_kernel, sizeof(int) * 5 * (size_t)kMaxBatch, dev) != cudaSuccess)
    return fail_with(RKV_ECUDA, "no usable current device");
  const cudaError_t e = launch_table(page_fork_kernel, a, a.batch, a.max_blocks, sizeof(int) * 5 * (size_t)a.batch,
                                     static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RKV_OK : fail_with(RKV_ECUDA, "page fork launch failed: %s", cudaGetErrorString(e));
}

extern "C" rkv_status rkv_page_compact_workspace(int32_t num_blocks, size_t* bytes) {
  if (!bytes) return fail_with(RKV_EINVAL, "bytes is NULL");
  if (num_blocks < 1) return fail_with(RKV_EINVAL, "num_blocks must be >= 1");
  *bytes = compact_bytes(num_blocks);
  return RKV_OK;
}

extern "C" rkv_status rkv_page_compact(const rkv_page_table* table, int32_t* free_blocks, int32_t* n_free,
                                       int32_t num_blocks, int32_t block_tokens, int32_t* block_table_out,
                                       int32_t* src, int32_t* dst, int32_t* count, void* workspace,
                                       size_t workspace_bytes, int32_t* flags, void* stream) {
  if (rkv_status st = check_fork_table(table, num_blocks, block_tokens)) return st;
  if (!free_blocks || !n_free || !block_table_out || !count || (num_blocks > 1 && (!src || !dst)))
    return fail_with(RKV_EINVAL, "NULL pointer");
  if (rkv_status st = check_workspace(workspace, workspace_bytes, compact_bytes(num_blocks))) return st;
  const size_t words = round16(((size_t)num_blocks + 31) / 32);
  CompactArgs a;
  a.table = table->block_table, a.seq_len = table->seq_len, a.table_out = block_table_out;
  a.free_blocks = free_blocks, a.n_free = n_free;
  a.src = src, a.dst = dst, a.count = count;
  a.bits = static_cast<uint32_t*>(workspace);
  a.before = static_cast<int32_t*>(workspace) + words;
  a.totals = a.before + words;
  a.flags = flags;
  a.batch = table->batch, a.max_blocks = table->max_blocks, a.num_blocks = num_blocks;
  a.shift = log2_block(block_tokens);
  const cudaError_t e = launch_table(page_compact_kernel, a, a.batch, a.max_blocks, sizeof(int) * (size_t)a.batch,
                                     static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RKV_OK : fail_with(RKV_ECUDA, "page compact launch failed: %s", cudaGetErrorString(e));
}

extern "C" rkv_status rkv_page_copy(const rkv_pages* layers, int32_t n_layers, const int32_t* src,
                                    const int32_t* dst, const int32_t* rows, const int32_t* count, int32_t n,
                                    int32_t* flags, void* stream) {
  if (n_layers < 1 || n_layers > kCopyLayers || !layers)
    return fail_with(RKV_EINVAL, "layers must be 1..%d", kCopyLayers);
  CopyArgs a;
  for (int l = 0; l < n_layers; ++l) {
    const rkv_pages& pg = layers[l];
    if (rkv_status st = check_pages(&pg)) return st;
    if (pg.n_kv_heads != layers->n_kv_heads || pg.head_dim != layers->head_dim ||
        pg.block_tokens != layers->block_tokens || pg.num_blocks != layers->num_blocks)
      return fail_with(RKV_EINVAL, "layers' pages differ in shape");
    a.layer[l].codes[0] = static_cast<uint8_t*>(pg.k), a.layer[l].codes[1] = static_cast<uint8_t*>(pg.v);
    a.layer[l].scale[0] = pg.k_scale, a.layer[l].scale[1] = pg.v_scale;
  }
  if (n < 0) return fail_with(RKV_EINVAL, "n < 0");
  if (n == 0) return RKV_OK;
  if (!src || !dst) return fail_with(RKV_EINVAL, "NULL pointer");
  a.src = src, a.dst = dst, a.rows = rows, a.count = count, a.flags = flags;
  a.layers = n_layers, a.n = n, a.N = layers->n_kv_heads;
  a.num_blocks = layers->num_blocks, a.block_tokens = layers->block_tokens, a.head_dim = layers->head_dim;
  int dev = 0, sms = 0;
  if (!current_device(dev, sms)) return fail_with(RKV_ECUDA, "no usable current device");
  const int64_t items = (int64_t)n * n_layers * 2 * a.N, ctas = (items + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
  const int64_t most = 4 * (int64_t)sms;
  page_copy_kernel<<<(unsigned)(ctas < most ? ctas : most), kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? RKV_OK : fail_with(RKV_ECUDA, "page copy launch failed: %s", cudaGetErrorString(e));
}

extern "C" rkv_status rkv_page_gather(const rkv_pages* pages, const rkv_page_table* table, const int32_t* length,
                                      void* k, const int64_t k_strides[2], void* v, const int64_t v_strides[2],
                                      int32_t max_rows, int32_t* cu_rows, int32_t* flags, void* stream) {
  if (rkv_status st = check_pages(pages)) return st;
  if (rkv_status st = check_table(table, pages->block_tokens)) return st;
  if (max_rows < 0) return fail_with(RKV_EINVAL, "max_rows must be >= 0");
  if (!cu_rows || !k_strides || !v_strides || (max_rows > 0 && (!k || !v))) return fail_with(RKV_EINVAL, "NULL pointer");
  for (int i = 0; i < 2; ++i)
    if (k_strides[i] < 0 || v_strides[i] < 0 || k_strides[i] % 8 || v_strides[i] % 8)
      return fail_with(RKV_EALIGN, "strides must be >= 0 and multiples of 16 bytes");
  if (!is_aligned(k, 16) || !is_aligned(v, 16)) return fail_with(RKV_EALIGN, "k and v must be 16-byte aligned");
  if (max_rows > 0 && (!rows_apart(max_rows, pages->n_kv_heads, pages->head_dim, k_strides) ||
                       !rows_apart(max_rows, pages->n_kv_heads, pages->head_dim, v_strides)))
    return fail_with(RKV_EINVAL, "rows of k or v overlap");
  GatherArgs a;
  a.codes[0] = static_cast<const uint8_t*>(pages->k), a.codes[1] = static_cast<const uint8_t*>(pages->v);
  a.scale[0] = pages->k_scale, a.scale[1] = pages->v_scale;
  a.table = table->block_table, a.seq_len = table->seq_len, a.length = length;
  a.out[0] = static_cast<__nv_bfloat16*>(k), a.out[1] = static_cast<__nv_bfloat16*>(v);
  a.st[0] = {k_strides[0], k_strides[1]}, a.st[1] = {v_strides[0], v_strides[1]};
  a.cu = cu_rows, a.flags = flags;
  a.batch = table->batch, a.max_blocks = table->max_blocks, a.num_blocks = pages->num_blocks;
  a.N = pages->n_kv_heads, a.shift = log2_block(pages->block_tokens), a.max_rows = max_rows;
  static SmemOptIn opt_in[2];
  int dev = 0, sms = 0;
  const bool wide = pages->head_dim == 128;
  void (*kernel)(GatherArgs) = wide ? page_gather_kernel<128> : page_gather_kernel<64>;
  if (!current_device(dev, sms) || opt_in[wide](kernel, sizeof(int) * 2 * (size_t)kMaxBatch, dev) != cudaSuccess)
    return fail_with(RKV_ECUDA, "no usable current device");
  // as many warps as the GPU holds; few rows are shared by warps, some heads each
  const int64_t warps = (int64_t)sms * kGatherCtas * (kGatherThreads / 32);
  const int64_t chunks = (int64_t)max_rows / kGatherRows + a.batch;            // at most
  const int64_t shares = warps / chunks;
  a.shares = (int)(shares < 1 ? 1 : shares < a.N ? shares : a.N);
  const int64_t ctas = (chunks * a.shares + kGatherThreads / 32 - 1) / (kGatherThreads / 32);
  const int64_t most = (int64_t)sms * kGatherCtas;
  kernel<<<(unsigned)(ctas < most ? ctas : most), kGatherThreads, sizeof(int) * 2 * (size_t)a.batch,
           static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? RKV_OK : fail_with(RKV_ECUDA, "page gather launch failed: %s", cudaGetErrorString(e));
}
