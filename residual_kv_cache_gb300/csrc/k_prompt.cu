// k_prompt.cu - causal attention of packed prompts: o = softmax(scale q K^T) V.
//
// Bound by the tensor core: 4 D flops for each visible (query, key) pair and head.  A CTA
// works on two tiles of 128 query rows that read the same key/value head, so that the tensor
// core always has one tile's products while the other tile's softmax runs:
//   S_t = Q_t K^T   [128 rows x 128 keys] in TMEM, thread r of softmax group t owns row r
//   P_t = 2^(c s - m) as bf16 in TMEM, m per row
//   O_t += P_t V    A = P_t from TMEM, V an MN-major B; accumulated in TMEM
// tcgen05 products execute in issue order, and a commit covers everything issued before it:
// with P_t over S_t (D = 128), S_t of key tile j is complete only when P_t V of tile j - 1
// is, so one barrier a tile tells its group both.  With D = 64 there is room for P_t beside
// S_t, and the next S_t is computed as soon as this one has been read.
//
// What bounds the loop is the chain from S_t over P_t to the next S_t (with D = 128: softmax,
// P V, Q K^T and two hand-overs of some 350 cycles, where the two tiles' products take 2048
// cycles a key tile).  So the softmax is short: no reduction crosses threads, and no maximum
// is taken in the usual tile.  m is the maximum over the first 64 keys; a bf16 weight has the
// range of an fp32, and nothing is lost while weights grow past 1.  Only when a row's
// weights of 64 keys sum to more than 2^24 is m raised to the scores' maximum, the sum and the
// accumulator rescaled and the half tile done again.  P_t is handed over in halves of 64
// keys, so that its product starts on the first.  Sums are fp32 over the unrounded weights.
//
// Row tiles of one sequence and key/value head are numbered r = q_tile G + head and taken
// in consecutive pairs, so that both need the same keys (or one tile more): with an even G
// two heads of one query tile, with G = 1 two neighbouring query tiles.  One CTA an SM works
// through pairs:
//   * where there are several for each CTA, it takes every gridDim-th pair of the list, heads
//     fastest, in alternating directions.  Of up to 32 sequences the list is sorted by the
//     keys that the pairs see, most first (eight prompts of 300 to 1900 tokens, 28 heads: the
//     busiest CTA has 6 % more than the mean, where sequence by sequence it had 32 %); of more
//     sequences it goes sequence by sequence, longest rows first.  The CTAs at work read the
//     same keys;
//   * where there are fewer pairs than CTAs, and many keys, all key tiles of all pairs are
//     cut into equal contiguous shares, and a pair that lies in several shares is joined from
//     fp32 partials (m, l, O) by a second kernel, in their order.
//
// Packed rows: a tile's rows behind its sequence are other sequences' rows.  Their queries
// fill lanes whose results are not stored and who have no vote; their keys are masked by
// position; their values are zeroed in shared memory, for 0 times what they hold must be 0.
// Within the sequence that is left to the end: only a NaN or infinity of V that a row does not
// see can reach it so, and the result shows it (hidden_stray).
//
// Measured back to back, one prompt of 16384 tokens, 32 heads on 8: heads of 128 1.38 ms (1.59
// PFLOP/s; a library product of two matrices reaches 1.92), heads of 64 1.24 ms (0.89: the
// chain of waits is the same, for half the flops; without any arithmetic between them it takes
// 0.99 ms); one of 77 tokens 9.1 us, the latency of one tile.
//
// Warps: 0-3 and 4-7 softmax of tiles 0 and 1, 8 TMA, 9 MMA, 10 work list, 11 TMEM.
#include <cuda_bf16.h>

#include "pages.cuh"

namespace rkv {
namespace {

constexpr int kRows = 128;                 // query rows of a tile
constexpr int kKeys = 128;                 // keys of a tile
constexpr int kPrThreads = 384;
// Limit of a wait, some 8 s: a warp that weighs rows again keeps the other roles waiting, 32 rows
// over 10^6 keys for some 4 s.
constexpr long long kPrWait = 8 * kWaitCycles;
constexpr int kItems = 3;                  // work items held ahead
constexpr float kPrRaise = 16777216.f;     // 2^24: a row's weights of 64 keys may sum to it

// Two row tiles of one sequence and key/value head.
struct Item {
  int kvh;                                 // key/value head; -1 ends the list
  int k0, lk;                              // the sequence's first key row, its keys
  int row[2], rows[2];                     // first row of q / out, rows of the tile (0: none)
  int head[2];                             // query head
  int lim[2];                              // keys that the tile's row 0 sees (may be <= 0)
  int j0, n[2];                            // key tiles [j0, n[t]); n[0] <= n[1]
  int slot;                                // partial in the workspace, or -1: all keys
};

constexpr int kPrMaxCtas = 160;            // CTAs of a launch (two partials each)
constexpr int kFewCtas = 152, kFewGain = 10;   // (few_pairs)
constexpr int kMinShare = 8;               // key tiles (of one row tile) that are worth a CTA

// What the joining kernel has to know of a partial.
struct Partial {
  int valid, last;                         // last: it ends its pair
  int row[2], rows[2], head[2], lim[2];
  int k0, lk;
};

struct PrArgs {
  const __nv_bfloat16 *q, *k, *v;          // (where the tensor maps do not serve)
  __nv_bfloat16* out;
  float* lse;
  Strides qst, kst, vst, ost;
  const int32_t *cu_q, *cu_k;
  int32_t* flags;
  int batch, total_q, total_k, Hq, N, G;
  float scale_log2;
  int split;                               // equal shares; else whole pairs
  Partial* info;                           // [2 grid]: a CTA's continued pair, its unfinished one
  float *pm, *pl, *po;                     // [2 grid][2][128], .., [2 grid][2][128][D]
};

// The key tiles of one sequence's row tiles, in closed form.
struct Seq {
  int q0, lq, k0, lk, nq, c, G;
  __device__ __forceinline__ Seq(int q0_, int lq_, int k0_, int lk_, int G_)
      : q0(q0_), lq(lq_), k0(k0_), lk(lk_), G(G_) {
    nq = (lq + kRows - 1) / kRows;
    const int off = lk - lq;               // ceil(off / 128)
    c = off > 0 ? (off + kKeys - 1) / kKeys : -(-off / kKeys);
  }
  __device__ __forceinline__ int tiles() const { return nq * G; }
  __device__ __forceinline__ int pairs() const { return (nq * G + 1) / 2; }
  // key tiles that query tile qt sees
  __device__ __forceinline__ int n(int qt) const {
    return qt == nq - 1 ? (lk + kKeys - 1) / kKeys : max(0, qt + 1 + c);
  }
  // sum of n over the query tiles before q, q < nq
  __device__ __forceinline__ int before(int q) const {
    const int m = c >= 0 ? q : max(0, q + c);
    return m * (m + 1) / 2 + (c >= 0 ? q * c : 0);
  }
  // sum of n over the row tiles before r
  __device__ __forceinline__ int prefix(int r) const {
    if (nq == 0) return 0;
    const int q = min(r / G, nq - 1);
    return G * before(q) + (r - q * G) * n(q);
  }
  // the pair of row tiles r1 - 1 (where it is >= 0) and r1, of key/value head h
  __device__ __forceinline__ void item(Item& it, int r0, int r1, int h) const {
    it.kvh = h;
    it.k0 = k0, it.lk = lk;
    it.j0 = 0, it.slot = -1;
    // query tile and head of r1, and of the row tile before it
    int qt = (int)((uint32_t)r1 / (uint32_t)G), e = r1 - qt * G;
#pragma unroll
    for (int t = 1; t >= 0; --t) {
      const bool is = t == 1 || r0 >= 0;
      it.row[t] = q0 + qt * kRows;
      it.rows[t] = is ? min(kRows, lq - qt * kRows) : 0;
      it.head[t] = h * G + e;
      it.lim[t] = lk - lq + qt * kRows + 1;
      it.n[t] = is ? n(qt) : 0;
      if (is && --e < 0) e = G - 1, --qt;
    }
  }
};

// The sequence of lane i's index (none past the batch): its rows and keys, cut to what there is.
__device__ __forceinline__ void load_seq(const PrArgs& a, int b, int& q0, int& lq, int& k0, int& lk) {
  q0 = lq = k0 = lk = 0;
  if (b >= a.batch) return;
  const int c0 = a.cu_q[b], c1 = a.cu_q[b + 1], d0 = a.cu_k[b], d1 = a.cu_k[b + 1];
  q0 = min(max(c0, 0), a.total_q), k0 = min(max(d0, 0), a.total_k);
  const int q1 = min(max(c1, q0), a.total_q), k1 = min(max(d1, k0), a.total_k);
  lq = q1 - q0, lk = k1 - k0;
  if (blockIdx.x == 0 && (q0 != c0 || q1 != c1 || k0 != d0 || k1 != d1)) raise_flag(a.flags, RKV_FLAG_BAD_INDEX);
}

// The pairs of a sequence (most keys first) whose second tile sees at least n key tiles.
__device__ __forceinline__ int pairs_seeing(const Seq& q, int n) {
  if (q.nq == 0) return 0;
  int qt = max(0, n - 1 - q.c);            // the first query tile that does
  if (n <= 0) qt = 0;
  else if (qt >= q.nq - 1) {
    if (n > q.n(q.nq - 1)) return 0;
    qt = q.nq - 1;
  }
  return (q.tiles() - 1 - qt * q.G) / 2 + 1;
}

// Calls emit(item) for CTA blockIdx.x's items of a list of up to 32 sequences' pairs, sorted by
// their key tiles; lane i: sequence i.
template <typename F>
__device__ __forceinline__ void walk_sorted(const PrArgs& a, const Seq& mine, F emit) {
  const int lane = threadIdx.x & 31;
  const uint32_t total = __reduce_add_sync(0xffffffffu, mine.pairs()) * (uint32_t)a.N;
  int level = __reduce_max_sync(0xffffffffu, mine.nq > 0 ? mine.n(mine.nq - 1) : 0);
  for (uint32_t round = 0;; ++round) {
    const uint32_t i = round * gridDim.x + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    Item it;
    it.kvh = -1;
    if (i < total) {
      int lo = 0;                          // item i's key tiles: the most that more than i pairs see
      while (lo < level) {
        const int at = (lo + level + 1) / 2;
        const bool by = __reduce_add_sync(0xffffffffu, pairs_seeing(mine, at)) * (uint32_t)a.N > i;
        lo = by ? at : lo;
        level = by ? level : at - 1;
      }
      const int above = pairs_seeing(mine, level + 1), upto = pairs_seeing(mine, level);
      const uint32_t before = __reduce_add_sync(0xffffffffu, above) * (uint32_t)a.N;
      uint32_t incl = (uint32_t)(upto - above) * (uint32_t)a.N;
      const uint32_t own = incl;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      const int b = __ffs(__ballot_sync(0xffffffffu, before + incl > i)) - 1;
      const uint32_t rel = i - before - __shfl_sync(0xffffffffu, incl - own, b), p = rel / (uint32_t)a.N;
      const Seq q(__shfl_sync(0xffffffffu, mine.q0, b), __shfl_sync(0xffffffffu, mine.lq, b),
                  __shfl_sync(0xffffffffu, mine.k0, b), __shfl_sync(0xffffffffu, mine.lk, b), a.G);
      const int r1 = q.tiles() - 1 - 2 * (__shfl_sync(0xffffffffu, above, b) + (int)p);
      q.item(it, r1 - 1, r1, (int)(rel - p * a.N));
    }
    if (!emit(it) || it.kvh < 0) return;
  }
}

// Calls emit(item) for CTA blockIdx.x's items in order, until there are no more or it returns
// false; run by a whole warp.  (q0, lq, k0, lk: lane i's sequence i.)
template <typename F>
__device__ __forceinline__ void walk_pairs(const PrArgs& a, int q0, int lq, int k0, int lk, F emit) {
  const int lane = threadIdx.x & 31;
  int64_t base = 0, round = 0;             // items before sequence b
  int b = 0, chunk = 0;                    // lane i: sequence chunk + i
  while (true) {
    const int64_t i = round * gridDim.x + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    Item it;
    it.kvh = -1;
    while (b < a.batch) {
      if (chunk != (b & ~31)) {
        chunk = b & ~31;
        load_seq(a, chunk + lane, q0, lq, k0, lk);
      }
      const int my_pairs = Seq(q0, lq, k0, lk, a.G).pairs();
      if (b == chunk && a.batch > 32) {    // skip the chunk if it ends before i
        int64_t sum = (int64_t)my_pairs * a.N;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (i >= base + sum) {
          base += sum;
          b += 32;
          continue;
        }
      }
      const int64_t here = (int64_t)__shfl_sync(0xffffffffu, my_pairs, b & 31) * a.N;
      if (i >= base + here) {
        base += here;
        ++b;
        continue;
      }
      const Seq q(__shfl_sync(0xffffffffu, q0, b & 31), __shfl_sync(0xffffffffu, lq, b & 31),
                  __shfl_sync(0xffffffffu, k0, b & 31), __shfl_sync(0xffffffffu, lk, b & 31), a.G);
      const uint32_t rel = (uint32_t)(i - base), p = rel / (uint32_t)a.N;
      const int r1 = q.tiles() - 1 - 2 * (int)p;             // longest first
      q.item(it, r1 - 1, r1, (int)(rel - p * a.N));
      break;
    }
    if (!emit(it) || it.kvh < 0) return;
    ++round;
  }
}

// The same of CTA blockIdx.x's equal share.
template <typename F>
__device__ __forceinline__ void walk_shares(const PrArgs& a, int q0, int lq, int k0, int lk, F emit) {
  const int lane = threadIdx.x & 31, cta = blockIdx.x;
  int total = 0;                           // key tiles of all row tiles (few_pairs: in 32 bits)
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    if (b0 > 0) load_seq(a, b0 + lane, q0, lq, k0, lk);
    const Seq q(q0, lq, k0, lk, a.G);
    total += q.prefix(q.tiles()) * a.N;
  }
  total = __reduce_add_sync(0xffffffffu, total);
  const int C = max(1, min((int)gridDim.x, total / kMinShare)), quot = total / C, rest = total % C;
  const int f0 = cta < C ? quot * cta + rest * cta / C : total;
  // pairs without keys have no tiles: they belong to the share they begin in, the last
  // share's end included
  const int f1 = cta + 1 < C ? quot * (cta + 1) + rest * (cta + 1) / C : total + (cta + 1 == C ? 1 : 0);
  Partial part[2];
  part[0].valid = part[1].valid = 0;
  int base = 0;                            // tiles before sequence b
  int b = 0, chunk = a.batch <= 32 ? 0 : -1;
  bool go = f0 < f1;
  while (go && b < a.batch && base < f1) {
    if (chunk != (b & ~31)) {
      chunk = b & ~31;
      load_seq(a, chunk + lane, q0, lq, k0, lk);
    }
    const Seq q(__shfl_sync(0xffffffffu, q0, b & 31), __shfl_sync(0xffffffffu, lq, b & 31),
                __shfl_sync(0xffffffffu, k0, b & 31), __shfl_sync(0xffffffffu, lk, b & 31), a.G);
    const int head = q.prefix(q.tiles());
    // every head's first pair that ends behind f0 or begins at or behind it
    for (int h = 0; h < a.N && go; ++h, base += head) {
      if (base + head < f0 || base >= f1) continue;
      int lo = 0, hi = q.pairs();          // 32 places at a time
      while (lo < hi && base < f0) {
        const int at = lo + (int)((int64_t)(hi - lo) * lane / 32), r = 2 * at;
        const uint32_t found = __ballot_sync(0xffffffffu, base + q.prefix(min(r + 2, q.tiles())) > f0 ||
                                                              base + q.prefix(r) >= f0);
        const int k = found ? __ffs(found) - 1 : 32;
        const int above = k > 0 ? __shfl_sync(0xffffffffu, at, k - 1) + 1 : lo;
        hi = k < 32 ? __shfl_sync(0xffffffffu, at, k & 31) : hi;
        lo = above;
      }
      int e = base + q.prefix(2 * lo);
      for (int p = lo; p < q.pairs() && go; ++p) {
        const bool two = 2 * p + 1 < q.tiles();
        const int s = e;
        e += q.n(2 * p / q.G) + (two ? q.n((2 * p + 1) / q.G) : 0);
        if (s >= f1) break;
        Item it;
        q.item(it, two ? 2 * p : -1, two ? 2 * p + 1 : 2 * p, h);
        const int n1 = it.n[1];
        // tiles [f0, f1) of the pair's as a range of its key tiles
        // (cost = n1 for one tile, else 2 n1 or 2 n1 - 1: x n1 / cost rounded up)
        const int cost = e - s, x0 = max(f0 - s, 0), x1 = min(f1 - s, cost);
        const int j0 = two ? (x0 + 1) / 2 : x0, j1 = two ? (x1 + 1) / 2 : x1;
        if (cost > 0 && j1 <= j0) continue;                  // its few tiles are a neighbour's
        it.j0 = j0;
        it.n[0] = min(it.n[0], j1), it.n[1] = j1;
        if (j0 > 0 || j1 < n1) {
          const int w = j0 > 0 ? 0 : 1;
          it.slot = 2 * cta + w;
          part[w].valid = 1, part[w].last = j1 == n1;
          part[w].k0 = it.k0, part[w].lk = it.lk;
#pragma unroll
          for (int t = 0; t < 2; ++t)
            part[w].row[t] = it.row[t], part[w].rows[t] = it.rows[t], part[w].head[t] = it.head[t],
            part[w].lim[t] = it.lim[t];
        }
        go = emit(it);
      }
    }
    ++b;
  }
  if (lane == 0) {
    a.info[2 * cta] = part[0];
    a.info[2 * cta + 1] = part[1];
  }
  if (go || !(f0 < f1)) {
    Item it;
    it.kvh = -1;
    emit(it);
  }
}

template <int D>
struct PrCfg {
  static constexpr uint32_t kTileB = kKeys * D * 2;          // bytes of a Q, K or V tile
  static constexpr int kSlots = D == 128 ? 4 : 8;            // ring of K and V tiles
  // TMEM columns: S_t at 128 t; O_t at 256 + D t; P_t over S_t, or, where there is room, at
  // 384 + 64 t, so that the next S_t can be computed while P_t is still in use
  static constexpr bool kApart = D == 64;
  static constexpr uint32_t kO = 256, kP = kApart ? 384 : 0, kPStride = kApart ? 64 : 128;
  static constexpr uint32_t kStage = 32 * 128;               // a warp's rows on their way out
  static constexpr uint32_t kSmem = 1024 + (2 + kSlots) * kTileB + 8 * kStage;
};

// A tile of 128 rows x D bf16 as D / 64 blocks of [128 rows x 128 bytes].
template <int D>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int head, int row) {
#pragma unroll
  for (int b = 0; b < D / 64; ++b)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst + b * kKeys * 128)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(b * 64), "r"(head), "r"(row)
        : "memory");
}

// Descriptor of an MN-major operand: 64-element blocks `lbo` bytes apart, groups of 8 rows
// (K) 1024 bytes apart, 128-byte swizzle.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// tmem_ld32, and the largest magnitude of the 32 (NaN if there is one).
__device__ __forceinline__ void tmem_ld32_top(uint32_t taddr, uint32_t* r, uint32_t& top) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.abs.NaN.f32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(top)
      : "r"(taddr));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

// 128 bytes of each of a warp's 32 rows, lane = row, to dst + row stride (`live` rows): through
// the warp's shared memory, so that a store writes whole 128-byte lines (a lane writing its
// own row touches 32 lines a store: an item's results took 5000 cycles so).
__device__ __forceinline__ void store_rows(uint8_t* stage, const uint32_t* w, int live, uint8_t* dst, int64_t stride) {
  const int lane = threadIdx.x & 31;
  __syncwarp();                                              // the last rows have been read
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) =
        make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  __syncwarp();
  const int c = lane & 7;
  dst += (lane >> 3) * stride + c * 16;
#pragma unroll
  for (int k = 0; k < 8; ++k, dst += 4 * stride) {
    const int r = 4 * k + (lane >> 3);
    const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 128 + ((c ^ (r & 7)) << 4));
    if (r < live) *reinterpret_cast<uint4*>(dst) = v;
  }
}

// A NaN or infinity of V makes NaN also of the rows that do not see it, where it shares a tile
// with keys that they see: their weight of 0 times it.  So a row whose result is not finite is
// looked at again, by a warp: do the values from the row's last key on to the end of its tiles
// hold one, in an element that is not NaN among the last values that the row sees?
template <int D>
__device__ __forceinline__ bool hidden_stray(const PrArgs& a, int kvh, int k0, int see, int end) {
  constexpr int kW = D / 64;                                 // words of a lane
  const __nv_bfloat16* v0 = a.v + (int64_t)k0 * a.vst.row + kvh * a.vst.head + (threadIdx.x & 31) * (2 * kW);
  uint32_t nan[kW] = {}, stray = 0;
#pragma unroll 2
  for (int j = max(see - 32, 0); j < see; ++j) {
#pragma unroll
    for (int i = 0; i < kW; ++i)
      nan[i] |= __vcmpgtu2(reinterpret_cast<const uint32_t*>(v0 + j * a.vst.row)[i] & 0x7FFF7FFFu, 0x7F807F80u);
  }
#pragma unroll 2
  for (int j = see; j < end; ++j) {
#pragma unroll
    for (int i = 0; i < kW; ++i)
      stray |= __vcmpgeu2(reinterpret_cast<const uint32_t*>(v0 + j * a.vst.row)[i] & 0x7FFF7FFFu, 0x7F807F80u) & ~nan[i];
  }
  return __any_sync(0xffffffffu, stray != 0);
}

// Then the row (of q, of query head `head`) is weighed again without the tensor core, over the
// keys that it sees and no others: some 20 instructions of a warp a key.  A lane scores a key;
// of the result, relative to m, it holds D / 32 elements.
template <int D>
__device__ __forceinline__ void weigh_visible(const PrArgs& a, int64_t row, int head, int k0, int see, float m,
                                              float* o) {
  constexpr int kW = D / 64, kFlight = 4;                   // values' rows in flight
  const int lane = threadIdx.x & 31, kvh = head / a.G;
  const uint4* q = reinterpret_cast<const uint4*>(a.q + row * a.qst.row + head * a.qst.head);
#pragma unroll
  for (int e = 0; e < 2 * kW; ++e) o[e] = 0.f;
#pragma unroll 1
  for (int j0 = 0; j0 < see; j0 += 32) {
    const int n = min(32, see - j0);
    const uint4* k = reinterpret_cast<const uint4*>(a.k + (int64_t)(k0 + j0 + min(lane, n - 1)) * a.kst.row +
                                                    kvh * a.kst.head);
    float s = 0.f;
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c) {
      const uint4 x = q[c], y = k[c];
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s = fmaf(__uint_as_float(xs[i] << 16), __uint_as_float(ys[i] << 16), s);
        s = fmaf(__uint_as_float(xs[i] & 0xFFFF0000u), __uint_as_float(ys[i] & 0xFFFF0000u), s);
      }
    }
    const float p = ex2_approx(fmaf(s, a.scale_log2, -m));
    const __nv_bfloat16* v = a.v + (int64_t)(k0 + j0) * a.vst.row + kvh * a.vst.head + lane * (2 * kW);
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kFlight) {
      uint32_t x[kFlight][kW];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
#pragma unroll
        for (int e = 0; e < kW; ++e)                         // (none: 0 times 0)
          x[i][e] = i0 + i < n ? reinterpret_cast<const uint32_t*>(v + (i0 + i) * a.vst.row)[e] : 0u;
      }
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const float w = __shfl_sync(0xffffffffu, p, i0 + i);
#pragma unroll
        for (int e = 0; e < kW; ++e) {
          o[2 * e] = fmaf(w, __uint_as_float(x[i][e] << 16), o[2 * e]);
          o[2 * e + 1] = fmaf(w, __uint_as_float(x[i][e] & 0xFFFF0000u), o[2 * e + 1]);
        }
      }
    }
    bool lost = true;                                        // nothing changes any more
#pragma unroll
    for (int e = 0; e < 2 * kW; ++e) lost &= o[e] != o[e];
    if (__all_sync(0xffffffffu, lost)) break;
  }
}

template <int D>
__global__ void __launch_bounds__(kPrThreads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, PrArgs a) {
  using C = PrCfg<D>;
  constexpr int kSlots = C::kSlots;
  extern __shared__ uint8_t raw[];
  uint8_t* s_q = align1024(raw);
  uint8_t* s_kv = s_q + 2 * C::kTileB;
  __shared__ __align__(8) uint64_t kv_full[kSlots], kv_empty[kSlots], q_full, q_empty, s_full[2], s_empty[2],
      p_half[2], p_full[2], p_empty[2], p_mid[2], o_full[2], i_full[kItems], i_empty[kItems], drain;
  __shared__ Item items[kItems];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_status;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = &s_abort;
  int* status = a.flags ? a.flags : &s_status;               // where a wait that gives up reports

  if (tid == 0) {
    tma_prefetch(&tm_q);
    tma_prefetch(&tm_k);
    tma_prefetch(&tm_v);
    for (int i = 0; i < kSlots; ++i) mbar_init(&kv_full[i], 1), mbar_init(&kv_empty[i], 1);
    mbar_init(&q_full, 1), mbar_init(&q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1), mbar_init(&s_empty[i], 4), mbar_init(&p_half[i], 128);
      mbar_init(&p_full[i], 128), mbar_init(&p_empty[i], 1), mbar_init(&p_mid[i], 1);
      mbar_init(&o_full[i], 1);
    }
    for (int i = 0; i < kItems; ++i) mbar_init(&i_full[i], 1), mbar_init(&i_empty[i], 10);
    mbar_init(&drain, 1);
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 11) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 8) {
      // ------------------------------------------------------------------------ TMA
      if (elect_one()) {
        Ring kv;
        int64_t issued = 0;
        uint32_t q_ph = 1;
        bool ok = true;
        for (int s = 0, ph = 0; ok; s == kItems - 1 ? (s = 0, ph ^= 1) : ++s) {
          if (!(ok = wait_one<kPrWait>(&i_full[s], ph, abort, status))) break;
          const Item it = items[s];
          mbar_arrive(&i_empty[s]);
          if (it.kvh < 0) break;
          if (it.n[1] == 0) continue;
          const bool both = it.n[0] > it.j0;
          if (!(ok = wait_one<kPrWait>(&q_empty, q_ph, abort, status))) break;
          q_ph ^= 1u;
          mbar_arrive_expect_tx(&q_full, (both ? 2 : 1) * C::kTileB);
          if (both) load_tile<D>(s_q, &tm_q, &q_full, it.head[0], it.row[0]);
          load_tile<D>(s_q + C::kTileB, &tm_q, &q_full, it.head[1], it.row[1]);
          for (int j = 2 * it.j0; j < 2 * it.n[1]; ++j) {            // K 0, V 0, K 1, V 1, ...
            if (!(ok = wait_one<kPrWait>(&kv_empty[kv.stage], kv.phase ^ 1u, abort, status))) break;
            mbar_arrive_expect_tx(&kv_full[kv.stage], C::kTileB);
            load_tile<D>(s_kv + kv.stage * C::kTileB, (j & 1) ? &tm_v : &tm_k, &kv_full[kv.stage], it.kvh,
                         it.k0 + (j >> 1) * kKeys);
            kv.next(kSlots);
            ++issued;
          }
        }
        if (*abort) {                                        // no copy may outlive the CTA
          for (int i = 0; i < kSlots && i < issued; ++i) {
            kv.stage = kv.stage == 0 ? (kv.phase ^= 1u, kSlots - 1) : kv.stage - 1;
            drain_wait(&kv_full[kv.stage], kv.phase);
          }
          if (issued > 0) drain_wait(&q_full, q_ph);
        }
      }
    } else if (warp == 9) {
      // ------------------------------------------------------------------------ MMA
      // One thread: its branch is known to the compiler to have one, and its waits need no
      // warp-wide agreement (a lane-0 branch issued the same products in 1.5x the time).
      if (elect_one()) {
        constexpr uint32_t id_s = idesc_bf16_f32(128, kKeys);
        constexpr uint32_t id_o = idesc_bf16_f32(128, D) | (1u << 16);
        Ring kv;                                             // the next slot to be used
        uint32_t q_ph = 0, p_ph[2] = {0, 0}, s_ph[2] = {1, 1};
        bool ok = true;
        const uint32_t q_sm = smem_u32(s_q), kv_sm = smem_u32(s_kv);
        // S_t = Q_t K^T
        auto qk = [&](int t, int slot) {
          if (C::kApart) {                                   // the last S_t has been read
            ok = ok && wait_one<kPrWait>(&s_empty[t], s_ph[t], abort, status);
            s_ph[t] ^= 1u;
            if (!ok) return;
            tc_fence_after();
          }
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint32_t off = (uint32_t)(i >> 2) * (kKeys * 128) + (uint32_t)(i & 3) * 32;
            umma_bf16(tmem + t * 128, sdesc_sw128(q_sm + t * C::kTileB + off),
                      sdesc_sw128(kv_sm + slot * C::kTileB + off), id_s, i > 0);
          }
          umma_commit(&s_full[t]);
        };
        // O_t (+)= P_t V, half the keys at a time as P_t comes
        auto pv = [&](int t, int slot, bool acc) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ok = ok && wait_one<kPrWait>(h ? &p_full[t] : &p_half[t], p_ph[t], abort, status);
            if (!ok) return;
            tc_fence_after();
#pragma unroll
            for (int i = 4 * h; i < 4 * h + 4; ++i)
              umma_bf16_ta(tmem + C::kO + t * D, tmem + C::kP + t * C::kPStride + i * 8,
                           sdesc_mn(kv_sm + slot * C::kTileB + i * 2048, kKeys * 128), id_o, acc || i > 0);
            if (h == 0) umma_commit(&p_mid[t]);
          }
          p_ph[t] ^= 1u;
          if (C::kApart) umma_commit(&p_empty[t]);
        };
        for (int s = 0, ph = 0; ok; s == kItems - 1 ? (s = 0, ph ^= 1) : ++s) {
          if (!(ok = wait_one<kPrWait>(&i_full[s], ph, abort, status))) break;
          const int kvh = items[s].kvh, n0 = items[s].n[0], n1 = items[s].n[1], j0 = items[s].j0;
          mbar_arrive(&i_empty[s]);
          if (kvh < 0) break;
          if (n1 == 0) continue;
          if (!(ok = wait_one<kPrWait>(&q_full, q_ph, abort, status))) break;
          q_ph ^= 1u;
          if (!(ok = wait_one<kPrWait>(&kv_full[kv.stage], kv.phase, abort, status))) break;
          tc_fence_after();
          if (n0 > j0) qk(0, kv.stage);
          qk(1, kv.stage);
          umma_commit(&kv_empty[kv.stage]);
          if (n1 == j0 + 1) umma_commit(&q_empty);
          kv.next(kSlots);
          for (int j = j0; j < n1 && ok; ++j) {
            const Ring v = kv;                               // V j, then K j + 1
            kv.next(kSlots);
            // K j + 1 is done with once the second tile's scores are computed
            auto next_qk = [&](int t) {
              if (j + 1 < (t ? n1 : n0)) qk(t, kv.stage);
              if (t == 1 && j + 1 < n1) {
                umma_commit(&kv_empty[kv.stage]);
                if (j + 2 == n1) umma_commit(&q_empty);
              }
            };
            if (C::kApart) {
              if (j + 1 < n1 && !(ok = ok && wait_one<kPrWait>(&kv_full[kv.stage], kv.phase, abort, status))) break;
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                next_qk(t);
                if (t == 0 && !(ok = ok && wait_one<kPrWait>(&kv_full[v.stage], v.phase, abort, status))) break;
                if (j < (t ? n1 : n0)) {
                  pv(t, v.stage, j > j0);
                  if (j + 1 == (t ? n1 : n0)) umma_commit(&o_full[t]);
                }
              }
              umma_commit(&kv_empty[v.stage]);
            } else {
              if (!(ok = ok && wait_one<kPrWait>(&kv_full[v.stage], v.phase, abort, status))) break;
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                if (j < (t ? n1 : n0)) {
                  pv(t, v.stage, j > j0);
                  if (t == 1) umma_commit(&kv_empty[v.stage]);
                  if (t == 0 && j + 1 < n1) ok = ok && wait_one<kPrWait>(&kv_full[kv.stage], kv.phase, abort, status);
                  if (t == 1 && j + 1 < n1 && j >= n0)       // tile 0 has not waited for it
                    ok = ok && wait_one<kPrWait>(&kv_full[kv.stage], kv.phase, abort, status);
                  if (!ok) break;
                  next_qk(t);
                  if (j + 1 == (t ? n1 : n0)) umma_commit(&o_full[t]);
                }
              }
            }
            if (j + 1 < n1) kv.next(kSlots);
          }
        }
        if (*abort) {
          umma_commit(&drain);
          drain_wait(&drain, 0);
        }
      }
    } else if (warp == 10) {
      // ------------------------------------------------------------------ work list
      int s = 0, q0, lq, k0, lk;
      uint32_t ph = 1;
      load_seq(a, lane, q0, lq, k0, lk);
      auto emit = [&](const Item& it) {
        if (!wait_warp<kWaitForWork>(&i_empty[s], ph, abort, status)) return false;
        if (lane == 0) {
          items[s] = it;
          mbar_arrive(&i_full[s]);
        }
        __syncwarp();
        if (++s == kItems) s = 0, ph ^= 1u;
        return true;
      };
      if (a.split) walk_shares(a, q0, lq, k0, lk, emit);
      else if (a.batch <= 32) walk_sorted(a, Seq(q0, lq, k0, lk, a.G), emit);
      else walk_pairs(a, q0, lq, k0, lk, emit);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // -------------------------------------------------------------------------- softmax
    const int t = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_tm = tmem + t * 128 + lanes, o_tm = tmem + C::kO + t * D + lanes;
    const uint32_t p_tm = tmem + C::kP + t * C::kPStride + lanes;
    uint32_t s_ph = 0, o_ph = 0, p_ph = 1, mid_ph = 0;
    Ring kv;                                                 // slot of K j
    const float c = a.scale_log2;
    bool ok = true;
    for (int si = 0, ph = 0; ok; si == kItems - 1 ? (si = 0, ph ^= 1) : ++si) {
      if (!(ok = wait_warp<kPrWait>(&i_full[si], ph, abort, status))) break;
      const int kvh = items[si].kvh, n = items[si].n[t], n1 = items[si].n[1], lk = items[si].lk;
      const int j0 = items[si].j0;
      // keys that this row sees
      const int see = min(items[si].lim[t] + r, lk);
      const int see0 = items[si].lim[t];
      const int rows = items[si].rows[t];
      if (kvh < 0) break;
      // m in base 2.  A lane behind the sequence holds another's query: with an infinite m its
      // weights are 0 or NaN and it never votes for a maximum to be taken.  (Nobody shares the
      // votes of a warp that lies wholly behind; one that ran ahead of the others through its
      // first tile cost a prompt of 77 tokens 0.3 us.)
      float m = r < rows || (r & ~31) >= rows ? -INFINITY : INFINITY, l = 0.f;
      const uint64_t cc = f32x2_pack(c, c);
      for (int j = j0; j < n1; ++j) {
        kv.next(kSlots);                                     // now V j
        if (j < n) {
          if (!(ok = wait_warp<kPrWait>(&s_full[t], s_ph, abort, status))) break;
          s_ph ^= 1u;
          tc_fence_after();
          const bool masked = (j + 1) * kKeys > see0;        // some row does not see every key
          const int vis = see - j * kKeys;
          uint32_t xa[32], xb[32], w[32];
          // scores of keys k .. k + 31 that the row does not see
          auto mask = [&](uint32_t* x, int k) {
            if (masked) {
              const int n_vis = vis - k;
              const uint32_t bits = n_vis >= 32 ? 0xFFFFFFFFu : n_vis <= 0 ? 0u : (1u << n_vis) - 1;
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = bits >> e & 1u ? x[e] : 0xFF800000u;
            }
          };
          auto top_of = [&](const uint32_t* x) {
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
#pragma unroll
              for (int u = 0; u < 4; ++u)
                mx[u] = max3(mx[u], __uint_as_float(x[e + 2 * u]), __uint_as_float(x[e + 2 * u + 1]));
            }
            return max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
          };
          // weights of 32 keys, and their sum added to two pairs
          auto weigh = [&](const uint32_t* x, uint32_t* out, uint64_t* sum) {
            const float z = m == -INFINITY ? 0.f : -m;
            const uint64_t nm = f32x2_pack(z, z);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float y0, y1;
              f32x2_unpack(fma2(f32x2_pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), cc, nm), y0, y1);
              y0 = ex2_approx(y0);
              y1 = ex2_approx(y1);
              sum[i & 1] = f32x2_add(sum[i & 1], f32x2_pack(y0, y1));
              out[i] = bf16x2(y0, y1);
            }
          };
          auto total = [&](const uint64_t* sum) {
            float a0, a1;
            f32x2_unpack(f32x2_add(sum[0], sum[1]), a0, a1);
            return a0 + a1;
          };
          // m becomes the maximum with `top`; what was summed so far is rescaled (`acc`: an
          // accumulator among it, whose products are complete)
          auto raise_to = [&](float top, bool acc) {
            const float mn = fmaxf(m, top * c);
            const float f = m == mn ? 1.f : ex2_approx(m - mn);
            l *= f;
            m = mn;
            if (acc) {
#pragma unroll 1
              for (int i = 0; i < D / 16; ++i) {
                uint32_t o[16];
                tmem_ld16(o_tm + 16 * i, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(o_tm + 16 * i, o);
              }
            }
          };
          float part;
          if (C::kApart) {                                   // P V of tile j - 1 is complete
            if (!(ok = wait_warp<kPrWait>(&p_empty[t], p_ph, abort, status))) break;
            p_ph ^= 1u;
            tc_fence_after();
          }
          bool again = __any_sync(0xffffffffu, m == -INFINITY);   // to begin with
          while (true) {
            if (again) {
              float top = -INFINITY;
#pragma unroll 1
              for (int i = 0; i < 4; ++i) {
                tmem_ld32(s_tm + 32 * i, xa);
                tmem_ld_wait();
                mask(xa, 32 * i);
                top = fmaxf(top, top_of(xa));
                // to begin with, the first 64 keys do
                if (i == 1 && j == j0 && __all_sync(0xffffffffu, top > -INFINITY || m == INFINITY)) break;
              }
              raise_to(top, j > j0);
            }
            uint64_t sum[2] = {0, 0};
            tmem_ld32(s_tm, xa);
            tmem_ld_wait();
            tmem_ld32(s_tm + 32, xb);
            mask(xa, 0);
            weigh(xa, w, sum);
            tmem_ld_wait();
            tmem_ld32(s_tm + 64, xa);
            mask(xb, 32);
            weigh(xb, w + 16, sum);
            part = total(sum);
            if (again || !__any_sync(0xffffffffu, part > kPrRaise)) break;
            again = true;
            tmem_ld_wait();
          }
          l += part;
          if ((j + 1) * kKeys > lk) {                        // values behind the sequence
            if (!(ok = wait_warp<kPrWait>(&kv_full[kv.stage], kv.phase, abort, status))) break;
            if (j * kKeys + r >= lk) {
              uint8_t* v = s_kv + kv.stage * C::kTileB + r * 128;
#pragma unroll
              for (int b = 0; b < D / 64; ++b)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  *reinterpret_cast<uint4*>(v + b * kKeys * 128 + i * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
          tmem_st32(p_tm, w);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&p_half[t]);                           // the product starts on 64 keys
          tmem_ld_wait();
          tmem_ld32(s_tm + 96, xb);
          mask(xa, 64);
          again = false;
          while (true) {
            uint64_t sum[2] = {0, 0};
            weigh(xa, w, sum);
            tmem_ld_wait();
            if (C::kApart && !again) {
              tc_fence_before();
              if (lane == 0) mbar_arrive(&s_empty[t]);       // S_t is in registers
            }
            if (!again) mask(xb, 96);
            weigh(xb, w + 16, sum);
            part = total(sum);
            if (again || !__any_sync(0xffffffffu, part > kPrRaise)) break;
            // the first half's product has to be complete
            if (!(ok = wait_warp<kPrWait>(&p_mid[t], mid_ph, abort, status))) break;
            tc_fence_after();
            raise_to(fmaxf(top_of(xa), top_of(xb)), true);
            again = true;
          }
          if (!ok) break;
          mid_ph ^= 1u;
          l += part;
          tmem_st32(p_tm + 32, w);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&p_full[t]);
        }
        kv.next(kSlots);                                     // now K j + 1
      }
      if (!ok) break;
      // the rows' results
      const int w0 = (warp & 3) * 32, live = items[si].rows[t] - w0;       // of the warp's rows
      const int64_t at = items[si].row[t] + w0;
      const int head = items[si].head[t], slot = items[si].slot, k0 = items[si].k0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&i_empty[si]);
      if (n > j0) {
        if (!(ok = wait_warp<kPrWait>(&o_full[t], o_ph, abort, status))) break;
        o_ph ^= 1u;
        tc_fence_after();
      }
      uint8_t* stage = s_kv + kSlots * C::kTileB + warp * C::kStage;
      if (slot >= 0) {
        // a partial: relative to m
        const int64_t prow = ((int64_t)slot * 2 + t) * kRows + w0;
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          uint32_t x[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = 0;
          if (n > j0) {
            tmem_ld32(o_tm + 32 * i, x);
            tmem_ld_wait();
          }
          store_rows(stage, x, live, reinterpret_cast<uint8_t*>(a.po + prow * D + 32 * i), D * 4);
        }
        if (lane < live) a.pm[prow + lane] = m, a.pl[prow + lane] = l;
      } else {
        const float inv = l != 0.f ? 1.f / l : 0.f;
        uint8_t* dst = reinterpret_cast<uint8_t*>(a.out + at * a.ost.row + head * a.ost.head);
        uint32_t w[D / 2];
        float top = 0.f;                                     // largest magnitude, or NaN
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          uint32_t x[64];
          if (n > j0) {
            uint32_t m0, m1;
            tmem_ld32_top(o_tm + 64 * i, x, m0);
            tmem_ld32_top(o_tm + 64 * i + 32, x + 32, m1);
            tmem_ld_wait();
            top += __uint_as_float(m0) + __uint_as_float(m1);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            w[32 * i + e] =
                l != 0.f ? bf16x2(__uint_as_float(x[2 * e]) * inv, __uint_as_float(x[2 * e + 1]) * inv) : 0u;
          }
        }
        // a row whose result is not finite though its sum is: what it does not see may be why
        // (looked at before the row is stored: out may be q)
        const bool finite = top - top == 0.f || l == 0.f || !(l - l == 0.f) || lane >= live;
        for (uint32_t rest = __ballot_sync(0xffffffffu, !finite); rest != 0; rest &= rest - 1) {
          const int b = __ffs(rest) - 1, see_b = __shfl_sync(0xffffffffu, see, b);
          if (!hidden_stray<D>(a, kvh, k0, see_b, min(lk, n * kKeys))) continue;
          float o[D / 32];
          weigh_visible<D>(a, at + b, head, k0, see_b, __shfl_sync(0xffffffffu, m, b), o);
          const float inv_b = __shfl_sync(0xffffffffu, inv, b);
#pragma unroll
          for (int e = 0; e < D / 64; ++e)
            reinterpret_cast<uint32_t*>(stage)[lane * (D / 64) + e] = bf16x2(o[2 * e] * inv_b, o[2 * e + 1] * inv_b);
          __syncwarp();
          if (lane == b) {
#pragma unroll
            for (int e = 0; e < D / 8; ++e) {
              const uint4 x = reinterpret_cast<const uint4*>(stage)[e];
              w[4 * e] = x.x, w[4 * e + 1] = x.y, w[4 * e + 2] = x.z, w[4 * e + 3] = x.w;
            }
          }
          __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < D / 64; ++i) store_rows(stage, w + 32 * i, live, dst + 128 * i, a.ost.row * 2);
        if (lane < live && a.lse)
          a.lse[(at + lane) * a.Hq + head] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 11) tmem_dealloc(tmem, 512);
}

// Joins the partials of the pair that CTA blockIdx.x began and did not finish: its own, then
// those of the CTAs after it until one that ends the pair.  Grid (grid, 2 tiles, 8), a warp
// two rows.
constexpr int kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) prompt_join_kernel(PrArgs a, int grid) {
  constexpr int kE = D / 32, kAhead = 8;                     // partials' rows in flight
  const int c = blockIdx.x, t = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait_previous_grid();
  const Partial& part = a.info[2 * c + 1];
  if (!part.valid || part.last) return;
  const int row0 = part.row[t], rows = part.rows[t], head = part.head[t];
  int n = 0;                                                 // partials
  for (int e0 = c + 1; n == 0 && e0 < grid; e0 += 32) {
    const int e = e0 + lane;
    const uint32_t at_end = __ballot_sync(0xffffffffu, e < grid && a.info[2 * e].valid && a.info[2 * e].last);
    if (at_end) n = e0 - c + __ffs(at_end);
  }
  if (n == 0) return;                                        // of a call that gave up
  auto slot_of = [&](int i) { return i == 0 ? 2 * c + 1 : 2 * (c + i); };
  for (int r = blockIdx.z * (kJoinThreads / 32) + warp; r < rows; r += gridDim.z * (kJoinThreads / 32)) {
    float m = -INFINITY, l = 0.f, o[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] = 0.f;
    for (int i0 = 0; i0 < n; i0 += 32) {                     // lane i: partial i0 + i
      float pm = -INFINITY, pl = 0.f;
      if (i0 + lane < n) {
        const int64_t at = ((int64_t)slot_of(i0 + lane) * 2 + t) * kRows + r;
        pm = __ldcg(a.pm + at), pl = __ldcg(a.pl + at);
      }
      float top = fmaxf(m, pm);
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
      // a part without keys weighs nothing; NaN stays
      const float f = pm == -INFINITY && pl == 0.f ? 0.f : ex2_approx(pm - top);
      const float fm = m == -INFINITY ? 0.f : ex2_approx(m - top);
      float add = pl * f;
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) add += __shfl_xor_sync(0xffffffffu, add, k);
      l = l * fm + add;
      m = top;
#pragma unroll
      for (int e = 0; e < kE; ++e) o[e] *= fm;
      for (int i1 = i0; i1 < min(n, i0 + 32); i1 += kAhead) {
        float po[kAhead][kE];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
#pragma unroll
          for (int e = 0; e < kE; ++e) po[u][e] = 0.f;
          if (i1 + u >= n) continue;
          const float* src = a.po + (((int64_t)slot_of(i1 + u) * 2 + t) * kRows + r) * D + lane * kE;
          if (kE == 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
            po[u][0] = v.x, po[u][1] = v.y, po[u][kE - 2] = v.z, po[u][kE - 1] = v.w;
          } else {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
            po[u][0] = v.x, po[u][1] = v.y;
          }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const float w = __shfl_sync(0xffffffffu, f, i1 + u - i0);
#pragma unroll
          for (int e = 0; e < kE; ++e) o[e] = fmaf(po[u][e], w, o[e]);
        }
      }
    }
    const int64_t at = row0 + r;
    float none = 0.f;                                        // NaN where the result is not finite
#pragma unroll
    for (int e = 0; e < kE; ++e) none = fmaf(o[e], 0.f, none);
    if (__any_sync(0xffffffffu, none != 0.f) && l != 0.f && l - l == 0.f) {
      const int see = min(part.lim[t] + r, part.lk);         // (a row's tiles end 255 keys behind it at most)
      if (hidden_stray<D>(a, head / a.G, part.k0, see, (int)min((int64_t)part.lk, (int64_t)see + 255)))
        weigh_visible<D>(a, at, head, part.k0, see, m, o);
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    __nv_bfloat16* dst = a.out + at * a.ost.row + head * a.ost.head + lane * kE;
#pragma unroll
    for (int e = 0; e < kE; e += 2)
      *reinterpret_cast<uint32_t*>(dst + e) = l != 0.f ? bf16x2(o[e] * inv, o[e + 1] * inv) : 0u;
    if (a.lse && lane == 0)
      a.lse[at * a.Hq + head] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
  }
}

template <int D>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PrArgs& a, int grid,
                   int dev, cudaStream_t s) {
  static SmemOptIn opt_in;
  cudaError_t e = opt_in(prompt_attention_kernel<D>, PrCfg<D>::kSmem, dev);
  if (e != cudaSuccess) return e;
  prompt_attention_kernel<D><<<grid, kPrThreads, PrCfg<D>::kSmem, s>>>(q, k, v, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || !a.split) return e;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(grid, 2, kRows / (kJoinThreads / 32) / 2);
  lc.blockDim = dim3(kJoinThreads);
  lc.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  e = cudaLaunchKernelEx(&lc, prompt_join_kernel<D>, a, grid);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

// Whether the call's pairs are so few that its key tiles are shared out instead.
// Whole pairs take as long as the longest, shares the mean and a join that costs about
// kFewGain key tiles of a pair (512 queries over 16384 keys, 32 heads: 202 us whole, 107 in
// shares; one query over 8192 keys 101 and 25; 1024 over 1024, 144 pairs, 20 and 32).
bool few_pairs(const rkv_prompt& p) {
  const int64_t pairs = ((int64_t)p.total_q / kRows + p.batch) * p.n_q_heads / 2;   // at most
  const int64_t keys = p.total_k / kKeys / p.batch;                                // key tiles, mean
  return p.total_k <= 1 << 26 && pairs < kFewCtas && (kFewCtas - pairs) * keys > kFewGain * kFewCtas;
}

rkv_status check_prompt(const rkv_prompt* pr) {
  if (!pr) return fail_with(RKV_EINVAL, "prompt is NULL");
  const rkv_prompt& p = *pr;
  if (p.head_dim != 64 && p.head_dim != 128) return fail_with(RKV_EINVAL, "head_dim must be 64 or 128");
  if (p.n_kv_heads < 1 || p.n_q_heads < 1 || p.n_q_heads > 65535 || p.n_q_heads % p.n_kv_heads)
    return fail_with(RKV_EINVAL, "n_q_heads must be a multiple of n_kv_heads, at most 65535");
  if (p.batch < 1 || p.batch > kMaxBatch) return fail_with(RKV_EINVAL, "batch must be in 1..%d", kMaxBatch);
  if (p.total_q < 0 || p.total_k < 0 || p.total_q > 1 << 30 || p.total_k > 1 << 30 ||
      (int64_t)p.total_q * p.n_q_heads > (int64_t)1 << 33)
    return fail_with(RKV_EINVAL, "total_q and total_k must be in 0..2^30, total_q * n_q_heads at most 2^33");
  if (!scale_ok(p.scale)) return fail_with(RKV_EINVAL, "scale must be at least 1e-30 and below 1e30");
  return RKV_OK;
}

}  // namespace
}  // namespace rkv

using namespace rkv;

extern "C" rkv_status rkv_prompt_attention_workspace(const rkv_prompt* prompt, size_t* bytes) {
  if (!bytes) return fail_with(RKV_EINVAL, "bytes is NULL");
  if (rkv_status st = check_prompt(prompt)) return st;
  const size_t slots = 2 * kPrMaxCtas, rows = 2 * kRows;
  *bytes = few_pairs(*prompt)
               ? slots * (sizeof(Partial) + sizeof(float) * rows * (2 + (size_t)prompt->head_dim))
               : 0;
  return RKV_OK;
}

extern "C" rkv_status rkv_prompt_attention(const rkv_prompt* pr, int32_t* flags, void* stream) {
  if (rkv_status st = check_prompt(pr)) return st;
  const rkv_prompt& p = *pr;
  if (p.total_q == 0) return RKV_OK;
  if (!p.q || !p.out || !p.cu_q || !p.cu_k || (p.total_k > 0 && (!p.k || !p.v)))
    return fail_with(RKV_EINVAL, "NULL pointer");
  const int64_t* strides[4] = {p.q_strides, p.k_strides, p.v_strides, p.out_strides};
  for (const int64_t* st : strides)
    if (st[0] < 0 || st[1] < 0 || st[0] % 8 || st[1] % 8)
      return fail_with(RKV_EALIGN, "strides must be >= 0 and multiples of 16 bytes");
  if (!is_aligned(p.q, 16) || !is_aligned(p.k, 16) || !is_aligned(p.v, 16) || !is_aligned(p.out, 16))
    return fail_with(RKV_EALIGN, "q, k, v and out must be 16-byte aligned");
  // out's rows of D: apart, in one order of the strides or the other
  // (in binary64: exact where it matters, and no product overflows)
  const double row = (double)p.out_strides[0], head = (double)p.out_strides[1], Dl = p.head_dim;
  const bool rows1 = p.total_q == 1, heads1 = p.n_q_heads == 1;
  const bool apart = (heads1 || head >= Dl) && (rows1 || row >= Dl) &&
                     (rows1 || heads1 || row >= (p.n_q_heads - 1) * head + Dl || head >= (p.total_q - 1) * row + Dl);
  if (!apart) return fail_with(RKV_EINVAL, "rows of out overlap");
  size_t need = 0;
  if (rkv_status st = rkv_prompt_attention_workspace(pr, &need)) return st;
  if (p.workspace_bytes < need || (need > 0 && !p.workspace))
    return fail_with(RKV_ECAPACITY, "workspace has %zu of %zu bytes", p.workspace ? p.workspace_bytes : (size_t)0, need);
  if (!is_aligned(p.workspace, 16)) return fail_with(RKV_EALIGN, "workspace must be 16-byte aligned");
  int dev = 0, sms = 0;
  if (!current_device(dev, sms)) return fail_with(RKV_ECUDA, "no usable current device");
  // without keys the maps are never read; they still need an extent
  const uint64_t D = p.head_dim;
  const bool keys = p.total_k > 0;
  CUtensorMap mq, mk, mv;
  if (!encode_map_heads(&mq, p.q, D, p.n_q_heads, p.total_q, p.q_strides, kRows) ||
      !encode_map_heads(&mk, keys ? p.k : p.q, D, keys ? p.n_kv_heads : 1, keys ? p.total_k : 1,
                        p.k_strides, kKeys) ||
      !encode_map_heads(&mv, keys ? p.v : p.q, D, keys ? p.n_kv_heads : 1, keys ? p.total_k : 1,
                        p.v_strides, kKeys))
    return fail_with(RKV_ECUDA, "cuTensorMapEncodeTiled is unavailable or rejected q, k or v");
  PrArgs a;
  a.out = static_cast<__nv_bfloat16*>(p.out);
  a.lse = p.lse;
  a.ost = {p.out_strides[0], p.out_strides[1]};
  a.q = static_cast<const __nv_bfloat16*>(p.q), a.qst = {p.q_strides[0], p.q_strides[1]};
  a.k = static_cast<const __nv_bfloat16*>(p.k), a.kst = {p.k_strides[0], p.k_strides[1]};
  a.v = static_cast<const __nv_bfloat16*>(p.v), a.vst = {p.v_strides[0], p.v_strides[1]};
  a.cu_q = p.cu_q, a.cu_k = p.cu_k;
  a.flags = flags;
  a.batch = p.batch, a.total_q = p.total_q, a.total_k = p.total_k;
  a.Hq = p.n_q_heads, a.N = p.n_kv_heads, a.G = a.Hq / a.N;
  a.scale_log2 = (float)(p.scale * 1.4426950408889634);
  a.split = need > 0;
  int grid = sms < kPrMaxCtas ? sms : kPrMaxCtas;
  if (a.split) {
    a.po = static_cast<float*>(p.workspace);
    a.pm = a.po + (size_t)2 * kPrMaxCtas * 2 * kRows * p.head_dim;
    a.pl = a.pm + 2 * kPrMaxCtas * 2 * kRows;
    a.info = reinterpret_cast<Partial*>(a.pl + 2 * kPrMaxCtas * 2 * kRows);
  } else {
    // no more CTAs than row tiles there can be
    const int64_t tiles = ((int64_t)p.total_q / kRows + p.batch) * p.n_q_heads;
    if (tiles < grid) grid = (int)tiles;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = D == 128 ? launch<128>(mq, mk, mv, a, grid, dev, s) : launch<64>(mq, mk, mv, a, grid, dev, s);
  return e == cudaSuccess ? RKV_OK : fail_with(RKV_ECUDA, "prompt attention launch failed: %s", cudaGetErrorString(e));
}
