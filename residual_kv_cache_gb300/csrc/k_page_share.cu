// k_page_share.cu - pages that several sequences hold: rows of the table forked, cut and freed,
// pages compacted, pages copied in the caches, stored rows gathered.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "pages.h"
#include "ptx.cuh"

namespace rkv {
namespace {

// ------------------------------------------------------------------- table operations
// A call is a few phases that wait for one another, each a load or two long, and latency bounds
// it: one CTA does it, or a cluster of up to 16.  A warp takes a run of tasks (128 neighbouring
// entries of a row of the table), the same ones in every phase, and holds the entries of the
// first of them in registers from the first phase to the last.  (Not
// built: several launches, or a whole grid with barriers of its own, put at a microsecond or two
// for each boundary.)
//
// Fork.  With R the rows after the call, a page is held whole where some R has it as one of its
// full pages, else begun by the rows that have it last.  One word a page says which (-1, or the
// lowest row that has begun it), another the first entry of the old table that lets go of it;
// both are minima, so the order of the threads does not matter.  A page goes where nobody holds
// it, and its first entry gives it its place in the list.  16 beams of up to 16384 tokens (one
// CTA, the words in its shared memory) 7.5 us, 256 slots of 4100 tokens on pages of 16 (16 CTAs,
// the words in L2) 11.7.  Words in the cluster's shared memory instead: 20.8 on eight CTAs, where
// words in L2 took 24 and on 16 CTAs 15 (random atomics on another CTA's memory pass no faster).
// Of the 12 some 2.5 are the launch, the barriers and the writes that they wait for 4, the rest
// nine dependent loads and the code itself.
//
// Compact.  A bit a page says whether a row holds it.  Each CTA marks its own entries' pages in
// a map of its own; the maps are joined a part a CTA, counted, and taken over by all, so that a
// page's rank is one look-up.  16 requests of up to 2000 tokens 4.8 us, 256 of up to 8000 on
// pages of 16 (78 000 entries, 104 000 pages) 12.3; with one map in L2 marked and read by all 24,
// with one spread over the cluster's shared memory 30 (of eight CTAs 52).
constexpr int kTableThreads = 1024;
constexpr int kTableWarps = kTableThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kTaskEntries = 128;
constexpr int kLaneEntries = kTaskEntries / 32;
constexpr size_t kTableSmem = 220 * 1024;      // dynamic shared memory of a CTA at most

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
__device__ __forceinline__ void cluster_sync(uint32_t ctas) {
  if (ctas == 1) __syncthreads();
  else asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
// The same variable of another CTA of the cluster.
template <typename T>
__device__ __forceinline__ T* in_cta(T* p, uint32_t rank) {
  uint64_t r;
  asm("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
  return reinterpret_cast<T*>(r);
}
// Tasks of a warp.  These kernels run their code once, and much of what a phase costs beside its
// loads is the fetching of its instructions: with two tasks held and not three or four, the others'
// loop not unrolled, and no divisions, 16 beams went from 9.1 to 7.8 us, the compaction of 16
// requests from 6.0 to 4.8.
struct Tasks {
  int first, last, per_row;          // this warp's [first, last)
  int row, part;                     // row of the first, and its place in it
  __device__ __forceinline__ Tasks(int batch, int width, uint32_t rank, uint32_t ctas) {
    per_row = (width + kTaskEntries - 1) / kTaskEntries;
    const int64_t n = (int64_t)batch * per_row;
    const int lg = __popc(ctas * kTableWarps - 1), w = (int)rank * kTableWarps + threadIdx.x / 32;     // a power of two of warps
    first = (int)(n * w >> lg), last = (int)(n * (w + 1) >> lg);
    row = per_row ? first / per_row : 0;
    part = first - row * per_row;
  }
  // f(i, row, entry of the row) for the entries of this lane: i counts those of the first kHold
  // tasks and is -1 in the others.  Every lane of the warp makes the same calls.
  template <int kHold, typename F>
  __device__ __forceinline__ void each(F f) const {
    const int lane = threadIdx.x & 31;
    int b = row, c = part;
#pragma unroll
    for (int h = 0; h < kHold; ++h) {
      if (first + h < last) {
#pragma unroll
        for (int k = 0; k < kLaneEntries; ++k) f(h * kLaneEntries + k, b, c * kTaskEntries + lane + 32 * k);
        if (++c == per_row) c = 0, ++b;
      }
    }
    for (int t = first + kHold; t < last; ++t) {
#pragma unroll 1
      for (int k = 0; k < kLaneEntries; ++k) f(-1, b, c * kTaskEntries + lane + 32 * k);
      if (++c == per_row) c = 0, ++b;
    }
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
  int2* state;                       // [num_blocks], of calls whose CTA does not hold it
  int32_t* stage;                    // [batch, max_blocks] new rows, for a table changed in place
  int32_t* flags;
  int batch, max_blocks, num_blocks, shift;
};

// What is known of a page: x: -1 where a row holds it whole, else the first row that has begun
// it, kNone without one; y: the first entry of the old table that lets go of it.
constexpr int kNone = INT32_MAX;
constexpr int kForkHold = 2;

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

// kLocal: one CTA, with the pages' state in its shared memory.
template <bool kLocal>
__global__ void __launch_bounds__(kTableThreads) page_fork_kernel(const __grid_constant__ ForkArgs p) {
  extern __shared__ int fsm[];
  int* s_src = fsm;                  // [batch] source row, -1: none
  int* s_new = s_src + p.batch;      // [batch] positions after the call
  int* s_have = s_new + p.batch;     // [batch] pages before it
  int* s_copy = s_have + p.batch;    // [batch] place among the copies, -1: none
  int* s_from = s_copy + p.batch;    // [batch] page that is copied, -1: none
  int2* s_state = reinterpret_cast<int2*>(fsm + (5 * p.batch + 1) / 2 * 2);
  __shared__ int s_width, s_count[kTableWarps], s_total[kMaxCluster], s_copies[kMaxBatch / kTableThreads][kTableWarps];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const uint32_t rank = kLocal ? 0 : cluster_rank(), ctas = kLocal ? 1 : cluster_size();
  const int step = ctas * kTableThreads, me = rank * kTableThreads + tid;
  const int P1 = (1 << p.shift) - 1, M = p.max_blocks, num = p.num_blocks;
  const int64_t cap = (int64_t)M << p.shift;
  const bool in_place = p.table_out == p.table;
  auto is_page = [&](int id) { return id >= 0 && id < num; };
  auto pages = [&](int n) { return (int)(((uint32_t)n + P1) >> p.shift); };      // (n + 127 < 2^31: check_table)
  auto state = [&](int id) {
    if constexpr (kLocal) return s_state + id;
    else return p.state + id;
  };
  auto read_state = [&](int id) {
    if constexpr (kLocal) return s_state[id];
    else return __ldcg(p.state + id);
  };

  if (kLocal)
    for (int i = tid; i < num; i += kTableThreads) s_state[i] = make_int2(kNone, kNone);
  if (tid == 0) s_width = 0;
  pdl_wait_previous_grid();
  const int n_free = *p.n_free;
  // as given, at first: positions before the call in s_have, those asked for in s_new
  for (int b = tid; b < p.batch; b += kTableThreads) {
    s_have[b] = p.seq_len[b];
    const int s = p.source ? p.source[b] : b, n = p.length ? p.length[b] : -1;
    const bool ends = p.finished && p.finished[b] != 0;
    s_src[b] = ends ? -1 : s;
    s_new[b] = n;
  }
  if (!kLocal)
    for (int i = me; i < num; i += step) p.state[i] = make_int2(kNone, kNone);
  __syncthreads();
  bool bad = n_free < 0 || n_free > num;
  int width = 0;
  for (int b = tid; b < p.batch; b += kTableThreads) {
    int s = s_src[b], n = 0;
    const int want = s_new[b], len = s_have[b];
    if (len < 0 || len > cap) bad = true;
    if (s >= p.batch) bad = true, s = -1;
    if (s >= 0) {
      const int all = s_have[s];
      n = want >= 0 ? want : all;
      if (n < 0 || n > all || all > cap) bad = true, n = 0;
    }
    s_src[b] = max(s, -1);
    s_new[b] = n;
    if (kLocal) s_from[b] = -1;
    width = max(width, max(pages(len), pages(n)));
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    // every CTA has read source and length before one writes seq_len_out, which may be one of
    // them: all see the same call and refuse it (one that went on would wait for CTAs that ended)
    cluster_sync(ctas);
    fork_refused(p, RKV_FLAG_BAD_INDEX, n_free);
    return;
  }
  for (int b = tid; b < p.batch; b += kTableThreads) s_have[b] = pages(s_have[b]);
  width = __reduce_max_sync(0xffffffffu, width);
  if (lane == 0) atomicMax(&s_width, width);
  cluster_sync(ctas);
  const Tasks tasks(p.batch, in_place ? s_width : M, rank, ctas);

  // who holds what: rows after the call, and the entries that go
  int to[kForkHold * kLaneEntries], gone[kForkHold * kLaneEntries];      // -1: none
  auto load = [&](int b, int j, int& t, int& g) {
    const int s = s_src[b], m = pages(s_new[b]);
    t = j < m ? p.table[(int64_t)s * M + j] : -1;
    g = j < s_have[b] && (s != b || j >= m) ? p.table[(int64_t)b * M + j] : -1;
  };
  tasks.each<kForkHold>([&](int i, int b, int j) {
    if (i >= 0) load(b, j, to[i], gone[i]);
  });
  for (int b = tid; b < p.batch && !kLocal; b += kTableThreads) {        // last pages that are begun
    const int n = s_new[b];
    s_from[b] = n & P1 ? p.table[(int64_t)s_src[b] * M + pages(n) - 1] : -1;
  }
  bool stray = false;
  tasks.each<kForkHold>([&](int i, int b, int j) {
    int t, g;
    if (i >= 0) t = to[i], g = gone[i];
    else load(b, j, t, g);
    const int s = s_src[b], n = s_new[b], m = pages(n);
    if (j < m) {
      // (-1 is the least: a store of it and another row's minimum end the same)
      if (!is_page(t)) stray = true;
      else if (j == m - 1 && (n & P1)) atomicMin(&state(t)->x, b);
      else *const_cast<volatile int*>(&state(t)->x) = -1;
      if (kLocal && j == m - 1 && (n & P1)) s_from[b] = t;
      if (i < 0 && in_place && s != b) p.stage[(int64_t)b * M + j] = t;
    }
    if (j < s_have[b] && (s != b || j >= m)) {
      if (is_page(g)) atomicMin(&state(g)->y, b * M + j);
      else stray = true;
    }
  });
  if (stray) raise_flag(p.flags, RKV_FLAG_BAD_INDEX);
  cluster_sync(ctas);

  // pages that go, in the order of the entries; copies, in that of the rows
  auto goes = [&](int b, int j, int g) {
    if (!is_page(g)) return false;
    const int2 s = read_state(g);
    return s.x == kNone && s.y == b * M + j;
  };
  int count = 0;
  tasks.each<kForkHold>([&](int i, int b, int j) {
    int t, g;
    if (i >= 0) g = gone[i];
    else load(b, j, t, g);
    const bool go = goes(b, j, g);
    if (i >= 0) gone[i] = go ? g : -1;
    count += __popc(__ballot_sync(0xffffffffu, go));
  });
  if (lane == 0) s_count[wid] = count;
  for (int r = 0, b = tid; r * kTableThreads < p.batch; ++r, b += kTableThreads) {
    int id = b < p.batch ? s_from[b] : -1;
    if (!is_page(id) || read_state(id).x == b) id = -1;
    const uint32_t these = __ballot_sync(0xffffffffu, id >= 0);
    if (lane == 0) s_copies[r][wid] = __popc(these);
    if (b < p.batch) {
      s_copy[b] = id >= 0 ? __popc(these & ((1u << lane) - 1)) : -1;     // of the warp's, at first
      s_from[b] = id;
    }
  }
  __syncthreads();
  int copies = 0;
  for (int r = 0, b = tid; r * kTableThreads < p.batch; ++r, b += kTableThreads) {
    const int n = s_copies[r][lane];
    const int earlier = copies + __reduce_add_sync(0xffffffffu, lane < wid ? n : 0);
    if (b < p.batch && s_copy[b] >= 0) s_copy[b] += earlier;
    copies += __reduce_add_sync(0xffffffffu, n);
  }
  int before = lane < wid ? s_count[lane] : 0, all = s_count[lane];
  before = __reduce_add_sync(0xffffffffu, before);
  all = __reduce_add_sync(0xffffffffu, all);
  if (tid < ctas) *in_cta(&s_total[rank], tid) = all;
  cluster_sync(ctas);

  int total = 0;
  for (uint32_t c = 0; c < ctas; ++c) {
    if (c < rank) before += s_total[c];
    total += s_total[c];
  }
  const int64_t end = (int64_t)n_free + total;
  if (end > num || end < copies) {
    fork_refused(p, RKV_FLAG_NO_SPACE, n_free);
    return;
  }
  int at = n_free + before;
  tasks.each<kForkHold>([&](int i, int b, int j) {
    int t, g;
    bool go;
    if (i >= 0) {
      g = gone[i], go = g >= 0;
    } else {
      load(b, j, t, g);
      go = goes(b, j, g);
    }
    const uint32_t these = __ballot_sync(0xffffffffu, go);
    if (go) p.free_blocks[at + __popc(these & ((1u << lane) - 1))] = g;
    at += __popc(these);
  });
  cluster_sync(ctas);

  tasks.each<kForkHold>([&](int i, int b, int j) {
    const int s = s_src[b], m = pages(s_new[b]);
    int32_t* out = p.table_out + (int64_t)b * M + j;
    if (j < m) {
      if (j == m - 1 && s_copy[b] >= 0) *out = __ldcg(p.free_blocks + (end - 1 - s_copy[b]));
      else if (!in_place) *out = i >= 0 ? to[i] : p.table[(int64_t)s * M + j];
      else if (s != b) *out = i >= 0 ? to[i] : p.stage[(int64_t)b * M + j];
    } else if (j < (in_place ? s_have[b] : M)) {
      *out = -1;
    }
  });
  for (int b = me; b < p.batch; b += step) {
    const int c = s_copy[b];
    p.seq_len_out[b] = s_new[b];
    p.copy_src[b] = s_from[b];
    const int page = c >= 0 ? __ldcg(p.free_blocks + (end - 1 - c)) : -1;
    if (c >= 0 && !is_page(page)) raise_flag(p.flags, RKV_FLAG_BAD_INDEX);
    p.copy_dst[b] = page;
    p.copy_rows[b] = c >= 0 ? s_new[b] & P1 : 0;
  }
  if (me == 0) *p.n_free_out = (int)(end - copies);
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
  int2* state;                       // [CTAs, words], of pools that shared memory does not take
  int32_t* flags;
  int batch, max_blocks, num_blocks, shift, words;   // words of a CTA: a power of two
};

constexpr int kCompactHold = 2;

// Of each 32 pages, x: which of them rows hold (a bit each); y: how many of the CTA's pages are
// held before them.  kLocal: each CTA marks the pages of its own entries in its shared memory,
// joins its words of all CTAs' marks, and takes the others' joined words over, so that every
// look-up is its own; else all is in the workspace.
template <bool kLocal>
__global__ void __launch_bounds__(kTableThreads) page_compact_kernel(const __grid_constant__ CompactArgs p) {
  extern __shared__ int fsm[];
  int* s_have = fsm;                 // [batch] pages
  int2* s_state = reinterpret_cast<int2*>(fsm + (p.batch + 1) / 2 * 2);
  __shared__ int s_width, s_count[kTableWarps], s_total[kMaxCluster], s_base[kMaxCluster + 1];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  const int step = ctas * kTableThreads, me = rank * kTableThreads + tid;
  const int P1 = (1 << p.shift) - 1, M = p.max_blocks, num = p.num_blocks, places = num / 2;
  const int lg = __popc(p.words - 1), words = ctas << lg, first = rank << lg;
  const bool in_place = p.table_out == p.table;
  int* s_mark = reinterpret_cast<int*>(s_state + words);       // [words], where there are several CTAs
  auto is_page = [&](int id) { return id >= 0 && id < num; };
  auto state = [&](int w) {
    if constexpr (kLocal) return s_state + w;
    else return p.state + w;
  };
  auto read_state = [&](int w) {
    if constexpr (kLocal) return s_state[w];
    else return __ldcg(p.state + w);
  };

  if constexpr (kLocal) {
    for (int i = tid; i < words; i += kTableThreads) {
      s_state[i].x = 0;
      if (ctas > 1) s_mark[i] = 0;
    }
  }
  if (tid == 0) s_width = 0;
  pdl_wait_previous_grid();
  if constexpr (!kLocal)
    for (int i = me; i < words; i += step) p.state[i].x = 0;
  bool bad = false;
  int width = 0;
  for (int b = tid; b < p.batch; b += kTableThreads) {
    int len = p.seq_len[b];
    if (len < 0 || len > (int64_t)M << p.shift) bad = true, len = 0;
    s_have[b] = (int)(((uint32_t)len + P1) >> p.shift);
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
  width = __reduce_max_sync(0xffffffffu, width);
  if (lane == 0) atomicMax(&s_width, width);
  if constexpr (kLocal) __syncthreads();
  else cluster_sync(ctas);
  const Tasks tasks(p.batch, in_place ? s_width : M, rank, ctas);

  int held[kCompactHold * kLaneEntries];
  tasks.each<kCompactHold>([&](int i, int b, int j) {
    if (i >= 0) held[i] = j < s_have[b] ? p.table[(int64_t)b * M + j] : -1;
  });
  bool stray = false;
  tasks.each<kCompactHold>([&](int i, int b, int j) {
    if (j >= s_have[b]) return;
    const int id = i >= 0 ? held[i] : p.table[(int64_t)b * M + j];
    if (!is_page(id)) stray = true;
    else if (kLocal && ctas > 1) atomicOr(s_mark + (id >> 5), 1 << (id & 31));
    else atomicOr(&state(id >> 5)->x, 1 << (id & 31));
  });
  if (stray) raise_flag(p.flags, RKV_FLAG_BAD_INDEX);
  cluster_sync(ctas);

  // held pages before each of this CTA's words
  int total = 0;
  for (int w0 = 0; w0 < p.words; w0 += kTableThreads) {
    const int w = w0 + tid;
    int x = 0;
    if (w < p.words) {
      x = read_state(first + w).x;
      if (kLocal && ctas > 1) {
        int part[kMaxCluster];
#pragma unroll
        for (uint32_t c = 0; c < kMaxCluster; ++c) part[c] = c < ctas ? *in_cta(s_mark + first + w, c) : 0;
#pragma unroll
        for (uint32_t c = 0; c < kMaxCluster; ++c) x |= part[c];
      }
    }
    const int n = __popc(x);
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (w0) __syncthreads();         // the last round's counts have been read
    if (lane == 31) s_count[wid] = sum;
    __syncthreads();
    const int counted = s_count[lane];
    sum += total + __reduce_add_sync(0xffffffffu, lane < wid ? counted : 0);
    if (w < p.words) *state(first + w) = make_int2(x, sum - n);
    total += __reduce_add_sync(0xffffffffu, counted);
  }
  if (tid < ctas) *in_cta(&s_total[rank], tid) = total;
  cluster_sync(ctas);
  if (tid <= ctas) {
    int n = 0;
    for (uint32_t c = 0; c < tid; ++c) n += s_total[c];
    s_base[tid] = n;
  }
  if (kLocal && ctas > 1) {
    constexpr int kAhead = 4;
    const int used = (num >> 5) + 1;
    for (int w0 = tid; w0 < used; w0 += kAhead * kTableThreads) {
      int2 v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int w = w0 + k * kTableThreads;
        if (w < used && w < words) v[k] = *in_cta(s_state + w, w >> lg);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int w = w0 + k * kTableThreads;
        if (w < used && w < words && w >> lg != rank) s_state[w] = v[k];
      }
    }
  }
  __syncthreads();
  const int n_live = s_base[ctas];
  auto below = [&](int id) {         // held pages before page id
    const int2 s = read_state(id >> 5);
    return s_base[id >> 5 >> lg] + s.y + __popc(s.x & ((1u << (id & 31)) - 1));
  };
  // those below n_live stay; each of the others goes to the next hole
  const int stay = n_live < num ? below(n_live) : n_live, moves = n_live - stay;
  for (int w = wid; w < p.words; w += kTableWarps) {
    const int word = first + w;
    if ((int64_t)word * 32 >= num) break;
    const int2 s = read_state(word);
    const int id = word * 32 + lane, live = s_base[rank] + s.y + __popc(s.x & ((1u << lane) - 1));
    if (s.x >> lane & 1) {
      if (id >= n_live) p.src[live - stay] = id;
    } else if (id < n_live) {
      p.dst[id - live] = id;
    }
  }
  cluster_sync(ctas);                // (none reads another's shared memory from here on)

  tasks.each<kCompactHold>([&](int i, int b, int j) {
    const int64_t e = (int64_t)b * M + j;
    if (j < s_have[b]) {
      const int id = i >= 0 ? held[i] : p.table[e];
      if (is_page(id) && id >= n_live) p.table_out[e] = __ldcg(p.dst + (below(id) - stay));
      else if (!in_place) p.table_out[e] = id;
    } else if (!in_place && j < M) {
      p.table_out[e] = -1;
    }
  });
  for (int i = me; i < num - n_live; i += step) p.free_blocks[i] = num - 1 - i;
  for (int i = moves + me; i < places; i += step) p.src[i] = p.dst[i] = -1;
  if (me == 0) *p.n_free = num - n_live, *p.count = moves;
}

// CTAs for a table: one for up to `alone` tasks a warp (a cluster's barriers and its state in L2
// cost more), else as many as leave a warp one task.  64 requests of up to 1000 tokens on pages of
// 16, two tasks a warp: a fork on one CTA 9.2 us, on two 9.5, a compaction 9.1 and 8.7 (of up to
// 2000 10.9 and 9.6); 128 of up to 2000, four tasks: a fork 16.4 and on four CTAs 11.0 (before
// the code was shortened).  The pool is not looked at, and one much larger than its table costs: a
// fork clears a word a page of it, a compaction writes its lists.  16 rows of up to 16384 tokens:
// a fork 7.4 us in 3144 pages, 7.6 in 20 000, 22 in 10^5, 131 in 10^6; a compaction 6.4, 11, 26, 223.
unsigned table_ctas(int batch, int max_blocks, int alone) {
  const int64_t tasks = (int64_t)batch * ceil_div(max_blocks, kTaskEntries);
  unsigned ctas = 1;
  if (tasks > alone * kTableWarps)
    while (ctas < kMaxCluster && (int64_t)ctas * kTableWarps < tasks) ctas *= 2;
  return ctas;
}

// ------------------------------------------------------------------------- page copies
constexpr int kCopyThreads = 256;
constexpr int kCopyCtas = 24;        // CTAs an SM at most
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

// A warp copies the rows of one (pair, layer, K or V, head), which lie side by side, eight loads in
// flight a lane.  Bandwidth bounds it: 701 pages of 128 KB in 8 layers 217 us, the rate of a plain
// copy.  One wave of CTAs with the same work to each is 234 us: those that finish early leave
// their SM idle.  (24 CTAs an SM at most, since a list may be mostly empty.)  The 12 begun pages
// of a forked step (a list of 16 with four absent) in 28 layers take 5.0 us, three dependent loads.
// What a list has past its count costs nothing: the 701 pairs in one of 500 000 entries 217.6 us.
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const __grid_constant__ CopyArgs p) {
  const int lane = threadIdx.x & 31;
  pdl_wait_previous_grid();
  const int n = p.count ? max(0, min(p.n, *p.count)) : p.n;
  const int per_pair = p.layers * 2 * p.N;       // below 2^24
  const int64_t items = (int64_t)n * per_pair;
  const int64_t head_bytes = (int64_t)p.block_tokens * p.head_dim;
  for (int64_t it = (int64_t)blockIdx.x * (kCopyThreads / 32) + threadIdx.x / 32; it < items;
       it += (int64_t)gridDim.x * (kCopyThreads / 32)) {
    const int i = (int)(it / per_pair);
    const uint32_t in = (uint32_t)(it - (int64_t)i * per_pair), rest = in / (uint32_t)p.N;
    const int h = (int)(in - rest * (uint32_t)p.N), kv = (int)(rest & 1), layer = (int)(rest >> 1);
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
constexpr int kGatherCtas = 3;       // CTAs an SM
constexpr int kGatherWaves = 4;      // times that many in the grid
constexpr int kGatherHeads = 4;      // heads that a warp takes at most

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

// Sixteen codes, used once.  (Not the read-only path: the blocks may be on their SM while the
// kernel that wrote the codes still runs.)
__device__ __forceinline__ uint4 load_codes(const uint8_t* p) {
  uint4 u;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "l"(p)
               : "memory");
  return u;
}

// Sixteen codes times a scale as bf16.
__device__ __forceinline__ void decode16(const uint4& u, float scale, uint32_t* w) {
  const uint32_t in[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((uint16_t)(in[e / 2] >> (16 * (e & 1))), __NV_E4M3);
    const float2 v = __half22float2(__half2(hr));
    const __nv_bfloat162 t = __floats2bfloat162_rn(v.x * scale, v.y * scale);
    w[e] = *reinterpret_cast<const uint32_t*>(&t);
  }
}
// 32 bytes: one store where they are a sector.
template <bool kWide>
__device__ __forceinline__ void store16(__nv_bfloat16* p, const uint32_t* w) {
  if constexpr (kWide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// A warp takes a share of the heads of one chunk, at most four, so that a row's heads are written
// at about the same time.  Bandwidth bounds long ones (a third reads, two thirds writes): 109 500
// rows of 8 heads of 128 107 us, 6.3 TB/s; 197 000 of 4 heads on pages of 16 96.5 us.  With a sector
// written by two 16-byte stores 144 us, one wave of CTAs 113, the next head's codes loaded ahead no
// gain, codes widened by integer instructions no gain.  1000 rows take 3.6 us.  kWide: the rows of
// k and v start on 32 bytes.
template <int D, bool kWide>
__global__ void __launch_bounds__(kGatherThreads, kGatherCtas) page_gather_kernel(const __grid_constant__ GatherArgs p) {
  constexpr int kLanes = D / 16;                 // lanes of one row
  constexpr int kRows = 32 / kLanes;             // rows of one load
  constexpr int kLoads = kGatherRows / kRows;
  extern __shared__ int fsm[];
  int* s_cu = fsm;                   // [batch] first row of each sequence
  int* s_chunk = s_cu + p.batch;     // [batch] first chunk of each
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_wait_previous_grid();
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
          if (there && r < left) u[kv][k] = load_codes(src + r * D);
        }
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        __nv_bfloat16* dst = p.out[kv] + (int64_t)row0 * p.st[kv].row + (int64_t)h * p.st[kv].head + x;
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int r = k * kRows + r_in;
          if (r >= left) continue;
          uint32_t w[8];
          decode16(u[kv][k], s[kv], w);
          store16<kWide>(dst + r * p.st[kv].row, w);
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

// Workspaces: the pages' state, for tables of more pages than shared memory takes, and a fork's
// new rows.
size_t fork_bytes(const rkv_page_table* t, int num_blocks) {
  return round16(sizeof(int2) * (size_t)num_blocks) + sizeof(int32_t) * (size_t)t->batch * t->max_blocks;
}
// Words of a CTA: a power of two that `ctas` times covers the pages.
int compact_words(int num_blocks, unsigned ctas) {
  int w = 1;
  while ((int64_t)w * ctas * 32 < num_blocks) w *= 2;
  return w;
}
size_t compact_bytes(int num_blocks) { return sizeof(int2) * kMaxCluster * (size_t)compact_words(num_blocks, kMaxCluster); }

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
  const int64_t entries = (int64_t)table->batch * table->max_blocks;
  if (half_shared(block_table_out, entries, table->block_table, entries) ||
      half_shared(seq_len_out, table->batch, table->seq_len, table->batch))
    return fail_with(RKV_EINVAL, "block_table_out or seq_len_out overlaps the table's and is not it");
  if (rkv_status st = check_workspace(workspace, workspace_bytes, fork_bytes(table, num_blocks))) return st;
  ForkArgs a;
  a.source = source, a.length = length, a.finished = finished;
  a.table = table->block_table, a.seq_len = table->seq_len;
  a.table_out = block_table_out, a.seq_len_out = seq_len_out;
  a.free_blocks = free_blocks, a.n_free = n_free, a.n_free_out = n_free_out;
  a.copy_src = copy_src, a.copy_dst = copy_dst, a.copy_rows = copy_rows;
  a.state = static_cast<int2*>(workspace);
  a.stage = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + round16(sizeof(int2) * (size_t)num_blocks));
  a.flags = flags;
  a.batch = table->batch, a.max_blocks = table->max_blocks, a.num_blocks = num_blocks;
  a.shift = log2_block(block_tokens);
  const unsigned ctas = table_ctas(a.batch, a.max_blocks, 2);
  const size_t fixed = sizeof(int) * 5 * (size_t)a.batch + 8, state = sizeof(int2) * (size_t)num_blocks;
  const bool local = ctas == 1 && fixed + state <= kTableSmem;
  void (*kernel)(ForkArgs) = local ? page_fork_kernel<true> : page_fork_kernel<false>;
  static SmemOptIn opt_in[2];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || opt_in[local](kernel, kTableSmem, dev, true) != cudaSuccess)
    return fail_with(RKV_ECUDA, "no usable current device");
  const cudaError_t e = launch_behind(kernel, a, ctas, kTableThreads, fixed + (local ? state : 0),
                                      static_cast<cudaStream_t>(stream), ctas);
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
  const int64_t entries = (int64_t)table->batch * table->max_blocks;
  if (half_shared(block_table_out, entries, table->block_table, entries))
    return fail_with(RKV_EINVAL, "block_table_out overlaps the table's and is not it");
  if (rkv_status st = check_workspace(workspace, workspace_bytes, compact_bytes(num_blocks))) return st;
  CompactArgs a;
  a.table = table->block_table, a.seq_len = table->seq_len, a.table_out = block_table_out;
  a.free_blocks = free_blocks, a.n_free = n_free;
  a.src = src, a.dst = dst, a.count = count;
  a.state = static_cast<int2*>(workspace);
  a.flags = flags;
  a.batch = table->batch, a.max_blocks = table->max_blocks, a.num_blocks = num_blocks;
  a.shift = log2_block(block_tokens);
  const unsigned ctas = table_ctas(a.batch, a.max_blocks, 1);
  a.words = compact_words(num_blocks, ctas);
  const size_t fixed = sizeof(int) * (size_t)a.batch + 8;
  const size_t state = (sizeof(int2) + (ctas > 1 ? sizeof(int) : 0)) * (size_t)a.words * ctas;
  const bool local = fixed + state <= kTableSmem;
  void (*kernel)(CompactArgs) = local ? page_compact_kernel<true> : page_compact_kernel<false>;
  static SmemOptIn opt_in[2];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || opt_in[local](kernel, kTableSmem, dev, true) != cudaSuccess)
    return fail_with(RKV_ECUDA, "no usable current device");
  const cudaError_t e = launch_behind(kernel, a, ctas, kTableThreads, fixed + (local ? state : 0),
                                      static_cast<cudaStream_t>(stream), ctas);
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
  const int64_t most = kCopyCtas * (int64_t)sms;
  const cudaError_t e = launch_behind(page_copy_kernel, a, (unsigned)(ctas < most ? ctas : most), kCopyThreads, 0,
                                      static_cast<cudaStream_t>(stream));
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
  RowBytes kb, vb;
  if (max_rows > 0 && (!row_bytes(k, max_rows, pages->n_kv_heads, pages->head_dim, k_strides, 2, kb) ||
                       !row_bytes(v, max_rows, pages->n_kv_heads, pages->head_dim, v_strides, 2, vb)))
    return fail_with(RKV_EINVAL, "strides pass the address space");
  if (max_rows > 0 && rows_meet(kb, vb)) return fail_with(RKV_EINVAL, "k and v overlap");
  // (every block reads the lengths, one writes cu_rows)
  if (shared(cu_rows, (int64_t)table->batch + 1, table->seq_len, table->batch) ||
      (length && shared(cu_rows, (int64_t)table->batch + 1, length, table->batch)))
    return fail_with(RKV_EINVAL, "cu_rows overlaps seq_len or length");
  GatherArgs a;
  a.codes[0] = static_cast<const uint8_t*>(pages->k), a.codes[1] = static_cast<const uint8_t*>(pages->v);
  a.scale[0] = pages->k_scale, a.scale[1] = pages->v_scale;
  a.table = table->block_table, a.seq_len = table->seq_len, a.length = length;
  a.out[0] = static_cast<__nv_bfloat16*>(k), a.out[1] = static_cast<__nv_bfloat16*>(v);
  a.st[0] = {k_strides[0], k_strides[1]}, a.st[1] = {v_strides[0], v_strides[1]};
  a.cu = cu_rows, a.flags = flags;
  a.batch = table->batch, a.max_blocks = table->max_blocks, a.num_blocks = pages->num_blocks;
  a.N = pages->n_kv_heads, a.shift = log2_block(pages->block_tokens), a.max_rows = max_rows;
  // 32-byte stores need rows that start on them
  bool wide = is_aligned(k, 32) && is_aligned(v, 32);
  for (int i = 0; i < 2; ++i) wide = wide && k_strides[i] % 16 == 0 && v_strides[i] % 16 == 0;
  static SmemOptIn opt_in[2][2];
  int dev = 0, sms = 0;
  const bool d128 = pages->head_dim == 128;
  void (*kernel)(GatherArgs) = d128 ? (wide ? page_gather_kernel<128, true> : page_gather_kernel<128, false>)
                                    : (wide ? page_gather_kernel<64, true> : page_gather_kernel<64, false>);
  if (!current_device(dev, sms) || opt_in[d128][wide](kernel, sizeof(int) * 2 * (size_t)kMaxBatch, dev) != cudaSuccess)
    return fail_with(RKV_ECUDA, "no usable current device");
  // few heads a warp, so that a row's heads are written at about the same time; fewer where the
  // GPU holds more warps than that makes
  const int64_t warps = (int64_t)sms * kGatherCtas * (kGatherThreads / 32);
  const int64_t chunks = (int64_t)max_rows / kGatherRows + a.batch;            // at most
  const int64_t shares = warps / chunks, least = ceil_div(a.N, kGatherHeads);
  a.shares = (int)(shares < least ? least : shares < a.N ? shares : a.N);
  const int64_t ctas = (chunks * a.shares + kGatherThreads / 32 - 1) / (kGatherThreads / 32);
  const int64_t most = (int64_t)sms * kGatherCtas * kGatherWaves;
  const cudaError_t e = launch_behind(kernel, a, (unsigned)(ctas < most ? ctas : most), kGatherThreads,
                                      sizeof(int) * 2 * (size_t)a.batch, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RKV_OK : fail_with(RKV_ECUDA, "page gather launch failed: %s", cudaGetErrorString(e));
}
