// k_page_attention.cu - decode attention over 8-bit pages: o = softmax(scale q K^T) V for one
// query row a sequence, K and V as E4M3 codes with a power-of-two scale per page and head.
//
// The read is bound by HBM: every stored byte is needed once, and the G query heads that
// share a key/value head are too few for the work to be more than a few operations a byte.
// So the bytes go from HBM to shared memory by TMA and from there straight into the tensor
// core: no code is ever decoded by a thread.
//
//   Tile = 128 positions of one (sequence, key/value head); its pages are 1 to 8 boxes of
//   [P rows x D bytes], stacked into a K tile and a V tile (rows swizzled by TMA).
//   Scores:   S[token, n]  = K_tile Q^T       M = 128 tokens, N = 16 or 32, K = D
//   Values:   O[d, n]     += V_tile^T P       M = D (128 lanes), N = 32 or 64, K = 128 tokens
//   both tcgen05.mma kind::f8f6f4 with fp32 accumulation in TMEM; V enters as an MN-major A.
//   The operands that are not stored in 8 bits are split into parts, one column each.  A bf16
//   q (scaled to its row's largest) is two E4M3 parts, hi + lo / 16: exact where it is within
//   2^-14 of that largest, and within 2^-21 of it everywhere.  A weight is four E5M2 parts,
//   a + (b + (c + d / 16) / 16) / 2048.  A part takes 4 bits off what is left (three and a
//   sign), and with a head's largest weight at 2^4 or more the last one's step, 2^-16 / 2^19,
//   is 2^-39 of it: a weight is off by 2^-15 of itself down to 2^-18 of the largest, by
//   2^-11 down to 2^-28, and by 2^-40 of the largest at any size.  The range is what long
//   contexts need: beside one key that takes most of the weight, the others have 2^-17 and
//   less each and still are most of the result where that key's value is small.  (Three E4M3
//   parts, with their range of 2^-18, lost them; a fourth E4M3 part would have 2^-28 of the
//   largest as its last step, for more bits than an output of bf16 shows.  The fourth part
//   costs long reads nothing, 256 sequences of 1024 tokens 2 us of 55, and 4 of 49 with 16
//   heads of 64 a key head.)  The products are exact and the parts are joined in fp32.
//   Softmax: two groups of 128 threads take a CTA's tiles in turn, each with its own score
//   buffer, weights, sums and accumulator, so that one group's chain of dependent steps runs
//   beside the other's, across the ends of sequences too.  The group of a segment's last tile
//   joins the other's part to its own.  Of many short segments a group takes each whole: two
//   of them then run side by side, where both groups' turns at one would mostly wait for its
//   ends (1024 sequences of 256 tokens, 8 heads: 162 us by turns, 122 us whole; of three
//   groups 139, of four 158: short segments run all of the code every 2 us, and a fifth of
//   their stalls already wait for instructions).
//   Thread t of a group owns token t (TMEM lane t).  Scores s are kept in base 2, and a page's
//   value scale 2^e is folded into the weights: the second product takes 2^(s + e - m), the
//   sum 2^(s - m).  The reference m of a head is the maximum of s + e over some earlier tiles
//   less 4, so the parts hold the terms that weigh most, whatever the pages' scales.  It is
//   raised (sums and accumulators rescaled) only when an s + e exceeds it by 8, which one vote
//   a tile finds: the usual tile has no reduction across tokens.
//
// Work split: all tiles of the call in the order (sequence, head, tile) are cut into equal
// contiguous shares, one a CTA (one CTA an SM), whatever the lengths.  A (sequence, head)
// that lies inside one share is written to `out` directly; others leave fp32 partials (m, l,
// o), at most two a CTA, which the second kernel joins in tile order: no atomics, the same
// bits on every run.
//
// Measured, 32 query heads on 8 of 128, pages of 64: 16 sequences of up to 131072 tokens, 3.34
// GB, 480-484 us (6.9 TB/s, where a copy reaches 6.8); one of 1000 tokens 9.4 us, the latency
// of one tile's chain, the join's and two launches; between, about 11 us on top of the bytes.
// Heads of 64 are half the bytes and the same chain: the same lengths 305 us (5.5 TB/s), up to
// 16384 tokens 49 us, where heads of 128 take 70.
//
// Warps: 0 TMA producer, 1 MMA issuer, 2 queries and segment list, 3 page scales and the rows
// of empty sequences, 4-7 and 8-11 softmax.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <cfloat>

#include "pages.cuh"

namespace rkv {
namespace {

constexpr int kTile = 128;                 // positions per tile
constexpr int kSoftWarp0 = 4;
constexpr int kNG = 2;                     // softmax groups
constexpr int kPaThreads = 128 + 128 * kNG;
constexpr int kSlots = 4;                  // segments whose queries are held ahead
constexpr int kMaxCtas = 256;              // shares of a call (partials in the workspace)
constexpr int kMaxTilePages = kTile / 16;
constexpr uint32_t kPaTmemCols = 256;
constexpr float kRaise = 8.f;              // weights stay below 2^8: what is left of them after a
                                           // part, 2^-4 of them, times its factor below 2^15
constexpr float kBelow = 4.f;              // a new reference lies so far below the maximum
constexpr int kParts = 4;                  // parts of a weight
// Part i + 1 holds what part i has left, times this.
__host__ __device__ constexpr float part_factor(int i) { return i == 0 ? 2048.f : 16.f; }
constexpr int kSoloTiles = 8, kSoloShare = 4;   // solo: at most so many tiles, 1 / so many of the share

// A run of tiles of one (sequence, head) inside a CTA's share.
struct Segment {
  int b, h, tile0, tiles, len, slot;       // slot: workspace partial, or -1 for the whole
  int solo;                                // one softmax group takes all of it
  // Softmax group of tile t, where the segment begins with group g; group of the next
  // segment's first tile.
  __device__ __forceinline__ int group(int g, int t) const { return solo ? g : (int)((uint32_t)(g + t) % kNG); }
  __device__ __forceinline__ int next_group(int g) const { return (int)((uint32_t)(g + (solo ? 1 : tiles)) % kNG); }
};

// What the joining kernel has to know of a share's partial.
struct PartialOf {
  int row;                                 // b N + h, -1: there is none
  int ends;                                // 1: begins its (b, h), 2: ends it
};

struct PaArgs {
  const float *ks, *vs;
  const int32_t *table, *seq_len;
  const __nv_bfloat16* q;
  Strides qst;
  __nv_bfloat16* out;
  float* lse;
  int32_t* flags;
  PartialOf* info;                         // of partial 2 c + i, the i-th that share c may leave
  float *pm, *pl, *po;                     // partials [2 kMaxCtas][G], [..][G], [..][G][D]
  int batch, N, G, shift, num_blocks, max_blocks;
  float scale_log2;
};

// kH: query heads computed (G rounded up to 2, 4, 6, 8, 12 or 16).
template <int D, int kH>
struct PaCfg {
  static constexpr int kGP = kH <= 8 ? 8 : 16;               // rows of one part
  static constexpr int kNQ = 2 * kGP;                        // score columns: hi, lo
  static constexpr int kNP = kParts * kGP;                   // weight columns
  // TMEM columns: a score buffer for each group, then an accumulator for each
  static constexpr uint32_t kSStride = 32, kOCol = kNG * kSStride, kOStride = kNP;
  static_assert(kOCol + kNG * kOStride <= kPaTmemCols);
  static constexpr uint32_t kHalf = kTile * D;               // bytes of a K or V tile
  static constexpr uint32_t kStage = 2 * kHalf;
  // as many as fit (of up to 8 heads; with 5 against 6, 61 sequences of up to 5000 tokens take
  // 53.4 against 52.3 us)
  static constexpr int kStages = (kH <= 8 ? 6 : 5) * (128 / D);
  static constexpr uint32_t kQBytes = kNQ * D;               // one segment's query tile
  static constexpr uint32_t kPBytes = kNP * kTile;           // one weight tile
  static constexpr uint32_t kPOff = kStages * kStage + kSlots * kQBytes;
  static constexpr uint32_t kMetaOff = kPOff + kNG * kPBytes;
  static constexpr uint32_t kMeta = kStages * kMaxTilePages * 8;   // (k scale, v scale)
  static constexpr uint32_t kJoinOff = kMetaOff + kMeta;           // a group's o, m, l
  static constexpr uint32_t kJoin = kH * (kTile + 2);              // floats
  static constexpr uint32_t kSmem = 1024 + kJoinOff + kNG * kJoin * 4;
};

__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

// The stored length of sequence b, cut to what the table can hold.
__device__ __forceinline__ int length_of(const PaArgs& a, int b, bool& bad) {
  const int len = a.seq_len[b];
  const int64_t cap = (int64_t)a.max_blocks << a.shift;
  bad = len < 0 || len > cap;
  return len < 0 ? 0 : (int)(len > cap ? cap : len);
}

// Equal contiguous shares of `total` tiles: share c begins at start(c).
struct Shares {
  int64_t q;
  int r, C;
  __device__ __forceinline__ Shares(int64_t total, int max_c) {
    C = (int)min((int64_t)max_c, total);
    if (C == 0) {
      q = 0, r = 0;
    } else if (total <= INT32_MAX) {
      q = (int)total / C;
      r = (int)total % C;
    } else {
      q = total / C;
      r = (int)(total % C);
    }
  }
  __device__ __forceinline__ int64_t start(int c) const { return q * c + r * c / C; }
};

// Pages of a segment's sequence that its tiles reach, and the id of one (-1 past them).
__device__ __forceinline__ int page_end(const PaArgs& a, const Segment& g) {
  return min((int)(((int64_t)g.len + (1 << a.shift) - 1) >> a.shift), (g.tile0 + g.tiles) * (kTile >> a.shift));
}
__device__ __forceinline__ int page_at(const PaArgs& a, const Segment& g, int page, int end) {
  return page < end ? __ldg(a.table + (int64_t)g.b * a.max_blocks + page) : -1;
}

// tcgen05.mma kind::f8f6f4, 8-bit operands in shared memory, fp32 accumulation.
__device__ __forceinline__ void umma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
      "}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// Instruction descriptor: fp32 D, E4M3 A, E4M3 or E5M2 B; trans_a: A is MN-major.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, bool b_e5m2, bool trans_a) {
  return (1u << 4) | (b_e5m2 ? 1u << 10 : 0u) | (trans_a ? 1u << 15 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Descriptor of a tile with D-byte rows (128- or 64-byte swizzle, groups of 8 rows).
template <int D>
__device__ __forceinline__ uint64_t sdesc_rows(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)((8 * D) >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)(D == 128 ? 2 : 4) << 61;
}

// Byte offset of 16-byte chunk c of row r in such a tile.
template <int D>
__device__ __forceinline__ uint32_t chunk_off(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ uint32_t e5m2x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}
// (an E5M2 code is the upper byte of an fp16)
__device__ __forceinline__ float2 from_e5m2x2(uint32_t c) {
  const uint32_t h = __byte_perm(c, 0u, 0x1404u);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Whether pred holds in any thread of softmax group g.
__device__ __forceinline__ bool vote_group(int g, bool pred) { return !bar_red_and(1 + g, 128, !pred); }

template <int D, int kH>
__global__ void __launch_bounds__(kPaThreads, 1)
    page_attention_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                          PaArgs a) {
  using C = PaCfg<D, kH>;
  constexpr int kST = C::kStages, kGP = C::kGP, kNQ = C::kNQ, kNP = C::kNP;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = align1024(raw);
  uint8_t* s_q = sm + kST * C::kStage;
  uint8_t* s_p = sm + C::kPOff;
  float2* s_meta = reinterpret_cast<float2*>(sm + C::kMetaOff);
  __shared__ __align__(8) uint64_t full[kST], empty[kST], s_full[kNG], s_empty[kNG], p_full[kNG], p_empty[kNG],
      j_full[kNG], j_empty[kNG], d_full[kSlots], q_full[kSlots], q_empty[kSlots], drain;
  __shared__ Segment seg[kSlots];
  __shared__ float s_qf[kSlots][16];
  __shared__ float s_red[kNG][4][16];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_status, s_b0;
  __shared__ int64_t s_pref;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = &s_abort;
  int* status = a.flags ? a.flags : &s_status;               // where a wait that gives up reports

  // of a small batch every warp reads the lengths at once, ahead of the set-up
  bool any_bad = false;
  int64_t mine = a.batch <= 32 && lane < a.batch ? tiles_of(length_of(a, lane, any_bad)) : 0;
  if (tid == 0) {
    tma_prefetch(&tm_k);
    tma_prefetch(&tm_v);
    for (int i = 0; i < kST; ++i) mbar_init(&full[i], 2), mbar_init(&empty[i], 1);
    for (int i = 0; i < kNG; ++i) {
      mbar_init(&s_full[i], 1), mbar_init(&s_empty[i], 4);
      mbar_init(&p_full[i], 128), mbar_init(&p_empty[i], 1);
      mbar_init(&j_full[i], 128), mbar_init(&j_empty[i], 128);
    }
    for (int i = 0; i < kSlots; ++i) mbar_init(&d_full[i], 1), mbar_init(&q_full[i], 1), mbar_init(&q_empty[i], 3 + 4 * kNG);
    mbar_init(&drain, 1);
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, kPaTmemCols);
    tmem_relinquish();
  }

  // the call's tiles, and the sequence in which this CTA's share begins
  const int cta = blockIdx.x;
  int64_t total = 0, incl = 0, f0 = 0, f1 = 0;
  auto cut = [&]() {                                         // the share
    const Shares shares(total * a.N, gridDim.x);
    f0 = cta < shares.C ? shares.start(cta) : 0;
    f1 = cta < shares.C ? shares.start(cta + 1) : 0;
  };
  if (a.batch <= 32) {
    // up to a warp's width every warp scans by itself
    incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
    cut();
    if (warp == 2 && mine > 0 && (incl - mine) * a.N <= f0 && f0 < incl * a.N) s_b0 = lane, s_pref = incl - mine;
  } else {
    for (int b0 = 0; b0 < a.batch; b0 += kPaThreads) {
      bool bad = false;
      const int b = b0 + tid;
      mine = b < a.batch ? tiles_of(length_of(a, b, bad)) : 0;
      any_bad |= bad;
      int64_t n = mine, t;
      int x = 0, tx;
      block_scan<kPaThreads>(n, x, t, tx);
      incl = total + n;
      total += t;
    }
    cut();
    int64_t pref = incl - mine;
    if (a.batch <= kPaThreads) {
      if (mine > 0 && pref * a.N <= f0 && f0 < incl * a.N) s_b0 = tid, s_pref = pref;
    } else {
      pref = 0;
      for (int b0 = 0; b0 < a.batch && pref * a.N <= f0; b0 += kPaThreads) {
        bool bad;
        const int b = b0 + tid;
        mine = b < a.batch ? tiles_of(length_of(a, b, bad)) : 0;
        int64_t n = mine, t;
        int x = 0, tx;
        block_scan<kPaThreads>(n, x, t, tx);
        if (mine > 0 && (pref + n - mine) * a.N <= f0 && f0 < (pref + n) * a.N) s_b0 = b, s_pref = pref + n - mine;
        pref += t;
      }
    }
  }
  if (any_bad && blockIdx.x == 0) raise_flag(a.flags, RKV_FLAG_BAD_INDEX);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = s_tmem;

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    const int P = 1 << a.shift, ppt = kTile >> a.shift;      // pages per tile
    Ring ring;
    int64_t issued = 0;
    bool ok = true, ahead = false;
    int id_ahead = -1;
    for (int s = 0, ph = 0; ok; s == kSlots - 1 ? (s = 0, ph ^= 1) : ++s) {
      if (!(ok = wait_warp(&d_full[s], ph, abort, status))) break;
      const Segment g = seg[s];
      if (g.b < 0) break;
      const int end = page_end(a, g);
      // lane i holds page p0 + i: 32 pages, a whole number of tiles
      int p0 = g.tile0 * ppt;
      int id = ahead ? id_ahead : page_at(a, g, p0 + lane, end);
      // the next segment's first pages, if it is known yet
      const int sn = s == kSlots - 1 ? 0 : s + 1;
      ahead = __all_sync(0xffffffffu, mbar_test(&d_full[sn], s == kSlots - 1 ? ph ^ 1 : ph));
      if (ahead) {
        const Segment gn = seg[sn];
        id_ahead = gn.b >= 0 ? page_at(a, gn, gn.tile0 * ppt + lane, page_end(a, gn)) : -1;
      }
      for (int t = 0; t < g.tiles && ok; p0 += 32) {
        const bool stored = p0 + lane < end, good = id >= 0 && id < a.num_blocks;
        if (stored && !good) raise_flag(a.flags, RKV_FLAG_BAD_INDEX);
        const int row = (int)(((int64_t)id * a.N + g.h) << a.shift);
        const int id_next = page_at(a, g, p0 + 32 + lane, end);
        for (int i = 0; i < 32 && t < g.tiles; i += ppt, ++t) {
          if (!(ok = wait_warp(&empty[ring.stage], ring.phase ^ 1u, abort, status))) break;
          uint8_t* st = sm + ring.stage * C::kStage;
          const bool here = lane >= i && lane < i + ppt;
          const uint32_t n = __popc(__ballot_sync(0xffffffffu, here && good));
          if (lane == 0) mbar_arrive_expect_tx(&full[ring.stage], n * 2u * (uint32_t)(P * D));
          __syncwarp();
          if (here && good) {
            const uint32_t off = (uint32_t)(lane - i) * (uint32_t)(P * D);
            tma_load_2d(st + off, &tm_v, &full[ring.stage], 0, row);
            tma_load_2d(st + C::kHalf + off, &tm_k, &full[ring.stage], 0, row);
          }
          ring.next(kST);
          ++issued;
        }
        id = id_next;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_empty[s]);
    }
    if (*abort && lane == 0)                                 // no copy may outlive the CTA
      for (int i = 0; i < kST && i < issued; ++i) {
        ring.stage = ring.stage == 0 ? (ring.phase ^= 1u, kST - 1) : ring.stage - 1;
        drain_wait(&full[ring.stage], ring.phase);
      }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    // Whatever is ready is issued: the next tile's scores once its bytes are there and its
    // group has read its last ones, a group's second product once its weights are there.
    // (In a fixed order, a segment's last product waited for the other group's next scores.)
    if (elect_one()) {
      constexpr uint32_t id_s = idesc_f8(128, kNQ, false, false), id_o = idesc_f8(128, kNP, true, true);
      Ring ring;                                             // stage of the next scores
      uint32_t s_ph = 0xFFFFFFFFu, p_ph = 0;                 // bit g: group g's
      // each group's tiles between their two products, oldest lowest: 8 bits of a stage + 1,
      // the top one set where the tile goes on with a sum
      uint64_t queue[kNG] = {};
      int open = 0;                                          // tiles in the queues
      int s = 0, t = 0, begin = 0;
      uint32_t ph = 0;
      bool have = false, ended = false;
      Segment sg;
      long long t0 = clock64();
      while (!(ended && open == 0)) {
        bool moved = false;
        // the tests at once: their latencies overlap
        const int gs = have ? sg.group(begin, t) : 0;
        bool p_ok[kNG];
#pragma unroll
        for (int g = 0; g < kNG; ++g) p_ok[g] = mbar_test(&p_full[g], p_ph >> g & 1u);
        const bool bytes_ok = mbar_test(&full[ring.stage], ring.phase), s_ok = mbar_test(&s_empty[gs], s_ph >> gs & 1u);
        const bool seg_ok = mbar_test(&q_full[s], ph);
#pragma unroll
        for (int g = 0; g < kNG; ++g) {
          if (queue[g] != 0 && p_ok[g]) {
            // O_g (+)= V^T P; M = 128 lanes: for D = 64 the upper 64 read the K tile behind V
            // and are unused
            const uint32_t e = (uint32_t)queue[g] & 0xFFu, stage = (e & 0x7Fu) - 1u;
            queue[g] >>= 8;
            --open;
            p_ph ^= 1u << g;
            tc_fence_after();
            const uint32_t vt = smem_u32(sm + stage * C::kStage);
            const uint32_t pt = smem_u32(s_p + g * C::kPBytes);
#pragma unroll
            for (int i = 0; i < kTile / 32; ++i)
              umma_f8(tmem + C::kOCol + g * C::kOStride, sdesc_rows<D>(vt + i * 32 * D, C::kHalf),
                      sdesc_rows<128>(pt + i * 32, 16), id_o, (e & 0x80u) != 0 || i > 0);
            umma_commit(&empty[stage]);
            umma_commit(&p_empty[g]);
            moved = true;
          }
        }
        if (!have && !ended && seg_ok) {
          sg = seg[s];
          have = sg.b >= 0;
          ended = !have;
          t = 0;
          moved = true;
        } else if (have) {
          const int g = gs;
          if (bytes_ok && s_ok) {
            s_ph ^= 1u << g;
            tc_fence_after();
            const uint32_t kt = smem_u32(sm + ring.stage * C::kStage + C::kHalf);
            const uint32_t qt = smem_u32(s_q + s * C::kQBytes);
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
              umma_f8(tmem + g * C::kSStride, sdesc_rows<D>(kt + i * 32, 16), sdesc_rows<D>(qt + i * 32, 16),
                      id_s, i > 0);
            umma_commit(&s_full[g]);
            const uint64_t e = (uint64_t)(ring.stage + 1) | (t >= (sg.solo ? 1 : kNG) ? 0x80u : 0u);
            // behind the group's older ones (never more than there are stages)
#pragma unroll
            for (int i = 0; i < kNG; ++i)
              if (i == g) queue[i] |= e << (queue[i] == 0 ? 0 : (71 - __clzll((long long)queue[i])) / 8 * 8);
            ++open;
            ring.next(kST);
            if (++t == sg.tiles) {
              umma_commit(&q_empty[s]);
              begin = sg.next_group(begin);
              have = false;
              if (++s == kSlots) s = 0, ph ^= 1u;
            }
            moved = true;
          }
        }
        if (moved) {
          t0 = clock64();
        } else if (*abort || clock64() - t0 > kWaitCycles) {
          if (!*abort) {
            *abort = 1;
            atomicOr(status, RKV_FLAG_TIMEOUT);
          }
          break;
        }
      }
      if (*abort) {
        umma_commit(&drain);
        drain_wait(&drain, 0);
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------- segments and their query tiles
    // eight lanes a head: D / 8 values each, four heads at a time
    constexpr int kW = D / 16, kRounds = (kH + 3) / 4;       // words (2 values) per lane; passes
    const int sub = lane & 7;
    int64_t left = f1 - f0;                                  // tiles of the share still to come
    int b = left > 0 ? s_b0 : a.batch, h = 0, tile = 0, chunk = -1, len_l = 0;    // lane i: length of sequence chunk + i
    bool first = true, ok = true;
    if (lane < 2) a.info[2 * cta + lane] = {-1, 0};
    __syncwarp();
    for (int s = 0, ph = 1; ok; s == kSlots - 1 ? (s = 0, ph ^= 1) : ++s) {
      Segment g{-1, 0, 0, 0, 0, -1, 0};
      while (left > 0 && b < a.batch) {
        if (chunk != (b & ~31)) {
          chunk = b & ~31;
          bool bad;
          len_l = chunk + lane < a.batch ? length_of(a, chunk + lane, bad) : 0;
        }
        g.len = __shfl_sync(0xffffffffu, len_l, b & 31);
        const int nb = tiles_of(g.len);
        if (nb == 0) {
          ++b;
          continue;
        }
        if (first) {                                         // where the share begins
          const int64_t rel = f0 - s_pref * a.N;             // 32 bits spare a long division
          if (rel <= INT32_MAX) h = (int)rel / nb, tile = (int)rel % nb;
          else h = (int)(rel / nb), tile = (int)(rel % nb);
        }
        g.b = b, g.h = h, g.tile0 = tile;
        g.tiles = (int)min((int64_t)(nb - tile), left);
        g.slot = g.tiles == nb ? -1 : 2 * cta + (first ? 0 : 1);
        if (g.slot >= 0 && lane == 0) a.info[g.slot] = {b * a.N + h, (tile == 0 ? 1 : 0) | (tile + g.tiles == nb ? 2 : 0)};
        g.solo = g.tiles <= kSoloTiles && (int64_t)g.tiles * kSoloShare <= f1 - f0;
        left -= g.tiles;
        first = false;
        tile = 0;
        if (++h == a.N) h = 0, ++b;
        break;
      }
      uint32_t raw[kRounds][kW];                             // loaded while the slot is awaited
      if (g.b >= 0) {
        const __nv_bfloat16* q = a.q + g.b * a.qst.row + (int64_t)g.h * a.G * a.qst.head + sub * (2 * kW);
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
          const int head = 4 * i + (lane >> 3);
#pragma unroll
          for (int e = 0; e < kW; e += 4) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (head < a.G) v = __ldg(reinterpret_cast<const uint4*>(q + head * a.qst.head + 2 * e));
            raw[i][e] = v.x, raw[i][e + 1] = v.y, raw[i][e + 2] = v.z, raw[i][e + 3] = v.w;
          }
        }
      }
      if (!(ok = wait_warp<kWaitForWork>(&q_empty[s], ph, abort, status))) break;
      if (lane == 0) {
        seg[s] = g;
        mbar_arrive(&d_full[s]);                             // the copies need no more
      }
      if (g.b >= 0) {
        uint8_t* qt = s_q + s * C::kQBytes;
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
          const int head = 4 * i + (lane >> 3);
          // the largest finite magnitude, on the bits; what is not finite becomes NaN
          uint32_t m2 = 0;
#pragma unroll
          for (int e = 0; e < kW; ++e) {
            const uint32_t mag = raw[i][e] & 0x7FFF7FFFu, over = __vcmpgeu2(mag, 0x7F807F80u);
            m2 = __vmaxu2(m2, mag & ~over);
            raw[i][e] |= over & 0x7FFF7FFFu;
          }
          uint32_t amax = max(m2 >> 16, m2 & 0xFFFFu);       // bf16 bits
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          // 2^7 <= amax 2^-ex < 2^8
          const int ex = max((int)(amax >> 7) - 127, -100) - 7;
          const float mul = __uint_as_float((uint32_t)(127 - ex) << 23);
          uint32_t hi[kW / 2], lo[kW / 2];
#pragma unroll
          for (int e = 0; e < kW; ++e) {
            const float x = __uint_as_float(raw[i][e] << 16) * mul, y = __uint_as_float(raw[i][e] & 0xFFFF0000u) * mul;
            const uint32_t c = e4m3x2(x, y);
            const float2 r = from_e4m3x2(c);
            const uint32_t d = e4m3x2((x - r.x) * 16.f, (y - r.y) * 16.f);
            hi[e / 2] = e & 1 ? hi[e / 2] | c << 16 : c;
            lo[e / 2] = e & 1 ? lo[e / 2] | d << 16 : d;
          }
          if (head < kH) {
            // the lane's D / 8 bytes of the head's rows
            const int col = sub * (D / 8);
            uint8_t* oh = qt + chunk_off<D>(head, col >> 4) + (col & 15);
            uint8_t* ol = qt + chunk_off<D>(kGP + head, col >> 4) + (col & 15);
            if (kW == 8) {
              *reinterpret_cast<uint4*>(oh) = make_uint4(hi[0], hi[1], hi[kW / 2 - 2], hi[kW / 2 - 1]);
              *reinterpret_cast<uint4*>(ol) = make_uint4(lo[0], lo[1], lo[kW / 2 - 2], lo[kW / 2 - 1]);
            } else {
              *reinterpret_cast<uint2*>(oh) = make_uint2(hi[0], hi[1]);
              *reinterpret_cast<uint2*>(ol) = make_uint2(lo[0], lo[1]);
            }
            if (sub == 0) s_qf[s][head] = __uint_as_float((uint32_t)(127 + ex) << 23) * a.scale_log2;
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[s]);
      if (g.b < 0) break;
    }
  } else if (warp == 3) {
    // --------------------------------------------------- page scales, a tile at a time
    const int ppt = kTile >> a.shift;
    Ring ring;
    bool ok = true;
    for (int s = 0, ph = 0; ok; s == kSlots - 1 ? (s = 0, ph ^= 1) : ++s) {
      if (!(ok = wait_warp(&d_full[s], ph, abort, status))) break;
      const Segment g = seg[s];
      if (g.b < 0) break;
      const int end = page_end(a, g);
      int p0 = g.tile0 * ppt, id = page_at(a, g, p0 + lane, end);
      for (int t = 0; t < g.tiles && ok; p0 += 32) {
        // a page that is not there has a negative scale
        const int64_t head = (int64_t)id * a.N + g.h;
        float2 sc = make_float2(0.f, -1.f);
        if (id >= 0 && id < a.num_blocks) sc = make_float2(__ldg(a.ks + head), __ldg(a.vs + head));
        id = page_at(a, g, p0 + 32 + lane, end);
        for (int i = 0; i < 32 && t < g.tiles; i += ppt, ++t) {
          if (!(ok = wait_warp(&empty[ring.stage], ring.phase ^ 1u, abort, status))) break;
          if (lane >= i && lane < i + ppt) s_meta[ring.stage * kMaxTilePages + lane - i] = sc;
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[ring.stage]);
          ring.next(kST);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_empty[s]);
    }
    // the rows of empty sequences, dealt out to the CTAs
    const int chunks = a.N * a.G * (D / 8);
    for (int b0 = cta; b0 < a.batch; b0 += 32 * gridDim.x) {
      bool bad;
      const int b = b0 + lane * gridDim.x;
      uint32_t none = __ballot_sync(0xffffffffu, b < a.batch && length_of(a, b, bad) == 0);
      for (; none != 0; none &= none - 1) {
        const int64_t e = b0 + (__ffs(none) - 1) * gridDim.x;
        uint4* out = reinterpret_cast<uint4*>(a.out) + e * chunks;
        for (int i = lane; i < chunks; i += 32) out[i] = make_uint4(0u, 0u, 0u, 0u);
        for (int i = lane; a.lse && i < a.N * a.G; i += 32) a.lse[e * a.N * a.G + i] = -INFINITY;
      }
    }
  } else if (warp >= kSoftWarp0) {
    // ---------------------------------------------------------------------- softmax
    const int wg = (warp - kSoftWarp0) >> 2, tok = tid & 127, w = warp & 3;
    const uint32_t tm = tmem + ((uint32_t)(w * 32) << 16);
    const uint32_t s_tm = tm + wg * C::kSStride;
    uint8_t* pt = s_p + wg * C::kPBytes;
    float* s_join = reinterpret_cast<float*>(sm + C::kJoinOff);
    Ring ring;                                               // stage of the segment's tile t
    uint32_t s_ph = 0, p_ph = 0, j_ph = 0;                   // j_ph: bit g, group g's parts
    int begin = 0;                                           // group of the segment's first tile
    bool ok = true;
    for (int s = 0, ph = 0; true; s == kSlots - 1 ? (s = 0, ph ^= 1) : ++s) {
      ok = ok && wait_warp(&q_full[s], ph, abort, status);
      if (vote_group(wg, !ok)) break;
      const Segment g = seg[s];
      if (g.b < 0) break;
      if (g.solo && begin != wg) {                           // the other group's
        begin = g.next_group(begin);
        for (int t = 0; t < g.tiles; ++t) ring.next(kST);
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_empty[s]);
        continue;
      }
      float m[kH], l[kH], qf[kH];
#pragma unroll
      for (int h = 0; h < kH; ++h) m[h] = -FLT_MAX, l[h] = 0.f, qf[h] = s_qf[s][h];
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_empty[s]);
      const uint32_t o_tm = tm + C::kOCol + wg * C::kOStride;
      bool first = true;                                     // the group's first tile of the segment
      const int owner = g.group(begin, g.tiles - 1);   // of the last tile
      for (int t = 0; t < g.tiles; ++t) {
        const int stage = ring.stage;
        const uint32_t st_ph = ring.phase;
        ring.next(kST);
        if (g.group(begin, t) != wg) continue;
        ok = ok && wait_warp(&full[stage], st_ph, abort, status) && wait_warp(&s_full[wg], s_ph, abort, status);
        s_ph ^= 1u;
        float x[kH];
        const float2 sc = s_meta[stage * kMaxTilePages + (tok >> a.shift)];
        const bool valid = (g.tile0 + t) * kTile + tok < g.len && !(sc.y < 0.f);
        if (ok) {
          tc_fence_after();
          uint32_t r[kNQ];
          if (kNQ == 16) tmem_ld16(s_tm, r);
          else tmem_ld32(s_tm, r);
          tmem_ld_wait();
          tc_fence_before();
          if (lane == 0) mbar_arrive(&s_empty[wg]);
#pragma unroll
          for (int h = 0; h < kH; ++h) {
            const float d = fmaf(__uint_as_float(r[kGP + h]), 0.0625f, __uint_as_float(r[h]));
            x[h] = valid ? d * (sc.x * qf[h]) : -INFINITY;
          }
        }
        // log2 of the value scale: the weights times it are what has to stay in range
        const float ev = (float)((int)(__float_as_uint(sc.y) >> 23) - 127);
        bool raise = !ok || first;
        if (ok) {
#pragma unroll
          for (int h = 0; h < kH; ++h) raise |= x[h] + ev > m[h] + kRaise;
        }
        // the products of the group's last tile have been added, its weights can go
        if (!first) {
          ok = ok && wait_warp(&p_empty[wg], p_ph, abort, status);
          p_ph ^= 1u;
        }
        if (vote_group(wg, raise || !ok)) {
          if (vote_group(wg, !ok)) {
            ok = false;
            break;
          }
          // the reference becomes the maximum so far, less kBelow
          // (one instruction a warp and head, on integers of the same order; NaN left out)
#pragma unroll
          for (int h = 0; h < kH; ++h) {
            const float y = fmaxf(x[h] + ev, -INFINITY);
            const int i = __float_as_int(y), key = i ^ (i >> 31 & 0x7FFFFFFF);
            const int top = __reduce_max_sync(0xffffffffu, key);
            if (lane == 0) s_red[wg][w][h] = __int_as_float(top ^ (top >> 31 & 0x7FFFFFFF));
          }
          bar_sync(1 + wg, 128);
          float f[kH];
#pragma unroll
          for (int h = 0; h < kH; ++h) {
            const float mn = fmaxf(m[h], fmaxf(fmaxf(s_red[wg][0][h], s_red[wg][1][h]),
                                               fmaxf(s_red[wg][2][h], s_red[wg][3][h])) - kBelow);
            f[h] = ex2_approx(m[h] - mn);
            l[h] *= f[h];
            m[h] = mn;
          }
          if (!first) {
            tc_fence_after();
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
              uint32_t r[kGP];
              if (kGP == 8) tmem_ld8(o_tm + part * kGP, r);
              else tmem_ld16(o_tm + part * kGP, r);
              tmem_ld_wait();
#pragma unroll
              for (int h = 0; h < kH; ++h) r[h] = __float_as_uint(__uint_as_float(r[h]) * f[h]);
              if (kGP == 8) tmem_st8(o_tm + part * kGP, r);
              else tmem_st16(o_tm + part * kGP, r);
            }
            tmem_st_wait();
          }
          bar_sync(1 + wg, 128);                             // s_red has been read
        }
        // the weights, their sum, and their parts for the second product
        const uint32_t c16 = (uint32_t)tok >> 4, c0 = (uint32_t)tok & 15u;
#pragma unroll
        for (int h = 0; h < kH; h += 2) {
          const float p0 = ex2_approx(x[h] - m[h]), p1 = ex2_approx(x[h + 1] - m[h + 1]);
          l[h] += p0;
          l[h + 1] += p1;
          float u0 = valid ? p0 * sc.y : 0.f, u1 = valid ? p1 * sc.y : 0.f;
#pragma unroll
          for (int part = 0; part < kParts; ++part) {
            const uint32_t c = e5m2x2(u0, u1);
            const int n0 = part * kGP + h, n1 = n0 + 1;
            pt[n0 * 128 + ((c16 ^ (n0 & 7)) << 4) + c0] = (uint8_t)c;
            pt[n1 * 128 + ((c16 ^ (n1 & 7)) << 4) + c0] = (uint8_t)(c >> 8);
            if (part + 1 < kParts) {
              const float2 e = from_e5m2x2(c);
              u0 = (u0 - e.x) * part_factor(part);
              u1 = (u1 - e.y) * part_factor(part);
            }
          }
        }
        if (!valid) {                                        // 0 x what the row holds must be 0
          uint8_t* vt = sm + stage * C::kStage + tok * D;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) *reinterpret_cast<uint4*>(vt + i * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&p_full[wg]);
        first = false;
      }
      begin = g.next_group(begin);
      // the groups that hand their part to the last tile's
      const int others = g.solo ? 0 : min(g.tiles, kNG) - 1;
      const uint32_t j_now = j_ph;
#pragma unroll
      for (int i = 1; i < kNG; ++i)
        if (i <= others) j_ph ^= 1u << ((uint32_t)(owner + kNG - i) % kNG);
      if (first && ok) continue;                             // none of the tiles was the group's
      // the group's sums and accumulator
      if (ok && !first) {
        ok = wait_warp(&p_empty[wg], p_ph, abort, status);
        p_ph ^= 1u;
      }
      if (vote_group(wg, !ok)) break;
      tc_fence_after();
      float o[kH];
#pragma unroll
      for (int h = 0; h < kH; ++h) o[h] = 0.f;
#pragma unroll
      for (int part = kParts - 1; part >= 0; --part) {
        uint32_t r[kGP];
        if (kGP == 8) tmem_ld8(o_tm + part * kGP, r);
        else tmem_ld16(o_tm + part * kGP, r);
        tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < kH; ++h) o[h] = fmaf(o[h], 1.f / part_factor(part), __uint_as_float(r[h]));
      }
      tc_fence_before();
#pragma unroll
      for (int h = 0; h < kH; ++h) {
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], i);
      }
      if (lane == 0) {
#pragma unroll
        for (int h = 0; h < kH; ++h) s_red[wg][w][h] = l[h];
      }
      bar_sync(1 + wg, 128);
#pragma unroll
      for (int h = 0; h < kH; ++h)
        l[h] = s_red[wg][0][h] + s_red[wg][1][h] + s_red[wg][2][h] + s_red[wg][3][h];
      if (others > 0 && wg != owner) {
        // its place is free once the last part has been taken
        ok = wait_warp(&j_empty[wg], (j_now >> wg & 1u) ^ 1u, abort, status);
        if (!ok) continue;
        float* part = s_join + wg * C::kJoin;
#pragma unroll
        for (int h = 0; h < kH; ++h) {
          part[h * kTile + tok] = o[h];
          if (tok == 0) part[kH * kTile + h] = m[h], part[kH * kTile + kH + h] = l[h];
        }
        mbar_arrive(&j_full[wg]);
        continue;
      }
      for (int i = 1; i <= others && ok; ++i) {              // the others' parts
        const int other = (int)((uint32_t)(owner + kNG - i) % kNG);
        const float* part = s_join + other * C::kJoin;
        ok = wait_warp(&j_full[other], j_now >> other & 1u, abort, status);
        if (!ok) break;
#pragma unroll
        for (int h = 0; h < kH; ++h) {
          const float m1 = part[kH * kTile + h], mn = fmaxf(m[h], m1);
          const float fa = ex2_approx(m[h] - mn), fb = ex2_approx(m1 - mn);
          o[h] = o[h] * fa + part[h * kTile + tok] * fb;
          l[h] = l[h] * fa + part[kH * kTile + kH + h] * fb;
          m[h] = mn;
        }
        mbar_arrive(&j_empty[other]);
      }
      if (!ok) continue;
      const int64_t row = g.slot < 0 ? ((int64_t)g.b * a.N + g.h) * a.G : (int64_t)g.slot * a.G;
      float mt = 0.f, lt = 0.f;                              // of head tok
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        if (tok == h) mt = m[h], lt = l[h];
        if (h < a.G && tok < D) {
          if (g.slot < 0) a.out[(row + h) * D + tok] = __float2bfloat16(l[h] != 0.f ? __fdividef(o[h], l[h]) : 0.f);
          else a.po[(row + h) * D + tok] = o[h];
        }
      }
      if (tok < a.G) {
        if (g.slot >= 0) a.pm[row + tok] = mt, a.pl[row + tok] = lt;
        else if (a.lse) a.lse[row + tok] = lt != 0.f ? (mt + log2f(lt)) * 0.6931471805599453f : -INFINITY;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kPaTmemCols);
}

// Joins the partials of the (sequence, key/value head) that share blockIdx.x begins and does
// not end: its own, then those of the shares after it up to the one that ends it.  Grid
// (shares, G / 4 rounded up).  A warp takes a query head, or, of fewer than four, a part of its
// partials; a row of D floats is one load of D / 4 lanes, kJoinAhead of them in flight.  (A
// block for each sequence and head, each of which found its shares from the lengths, took 40 us
// longer for 1024 sequences; partials read one after the other 16 us longer for 38 of them.)
constexpr int kJoinThreads = 128, kJoinWarps = kJoinThreads / 32, kJoinAhead = 8;

template <int D>
__global__ void __launch_bounds__(kJoinThreads, 8) page_attention_join_kernel(PaArgs a, int grid) {
  constexpr int kLanes = D / 4, kRows = 32 / kLanes, kChunks = kMaxCtas / 32;
  const int c0 = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ float4 s_o[kJoinWarps][kLanes];
  __shared__ float s_f[kJoinWarps][kMaxCtas];
  pdl_wait_previous_grid();
  // the share's last partial, if it goes on in the next one
  const int4 both = __ldcg(reinterpret_cast<const int4*>(a.info + 2 * c0));
  const PartialOf p0{both.x, both.y}, p1{both.z, both.w};
  const bool second = p1.row >= 0;
  if (!second && (p0.row < 0 || p0.ends != 1)) return;
  const int first = second ? 2 * c0 + 1 : 2 * c0;
  int n = 0;                                 // partials
  for (int i0 = 1; n == 0 && c0 + i0 < grid; i0 += 32) {
    const int c = c0 + i0 + lane;
    const uint32_t at_end = __ballot_sync(0xffffffffu, c < grid && (__ldcg(&a.info[2 * c].ends) & 2));
    if (at_end) n = i0 + __ffs(at_end);
  }
  if (n == 0) return;                        // of a call that gave up
  const int heads = a.G > 2 ? 4 : a.G;       // of this CTA
  const int parts = kJoinWarps / heads, part = warp / heads, g = blockIdx.y * heads + warp % heads;
  const bool live = g < a.G;
  const int64_t row = (int64_t)(second ? p1.row : p0.row) * a.G + g;
  auto slot_of = [&](int i) { return (i == 0 ? first : 2 * (c0 + i)) * a.G + g; };
  float m = -FLT_MAX, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live) {
    float f[kChunks], pl[kChunks];           // lane i: partials i, 32 + i, ..
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int i = 32 * c + lane;
      f[c] = -FLT_MAX, pl[c] = 0.f;
      if (i < n) f[c] = __ldcg(a.pm + slot_of(i)), pl[c] = __ldcg(a.pl + slot_of(i));
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) m = fmaxf(m, f[c]);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      if (32 * c >= n) break;
      const float w = ex2_approx(f[c] - m);
      l += pl[c] * w;
      s_f[warp][32 * c + lane] = w;
    }
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
    __syncwarp();
    const float4* po = reinterpret_cast<const float4*>(a.po) + lane % kLanes;
    const int step = parts * kRows;
    for (int i0 = part * kRows + lane / kLanes; i0 < n; i0 += kJoinAhead * step) {
      float4 x[kJoinAhead];
#pragma unroll
      for (int u = 0; u < kJoinAhead; ++u) {
        x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i0 + u * step < n) x[u] = __ldcg(po + (int64_t)slot_of(i0 + u * step) * kLanes);
      }
#pragma unroll
      for (int u = 0; u < kJoinAhead; ++u) {
        const float w = i0 + u * step < n ? s_f[warp][i0 + u * step] : 0.f;
        o.x = fmaf(x[u].x, w, o.x), o.y = fmaf(x[u].y, w, o.y);
        o.z = fmaf(x[u].z, w, o.z), o.w = fmaf(x[u].w, w, o.w);
      }
    }
    __syncwarp();
    if (kRows == 2) {
      o.x += __shfl_xor_sync(0xffffffffu, o.x, 16), o.y += __shfl_xor_sync(0xffffffffu, o.y, 16);
      o.z += __shfl_xor_sync(0xffffffffu, o.z, 16), o.w += __shfl_xor_sync(0xffffffffu, o.w, 16);
    }
  }
  if (parts > 1) {                           // the parts' sums, in their order
    if (lane < kLanes) s_o[warp][lane] = o;
    __syncthreads();
    for (int k = 1; part == 0 && k < parts; ++k) {
      const float4 x = s_o[warp + k * heads][lane % kLanes];
      o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
    }
  }
  if (!live || part > 0) return;
  const float inv = l != 0.f ? 1.f / l : 0.f;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv), hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  if (lane < kLanes)
    reinterpret_cast<uint2*>(a.out + row * D)[lane] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  if (a.lse && lane == 0) a.lse[row] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

rkv_status check_heads(const rkv_pages* pages, int n_q_heads) {
  if (n_q_heads < 1 || n_q_heads % pages->n_kv_heads || n_q_heads / pages->n_kv_heads > kPageMaxGroup)
    return fail_with(RKV_EINVAL, "n_q_heads must be a multiple of n_kv_heads, at most %d times it", kPageMaxGroup);
  return RKV_OK;
}

template <int D, int kH>
cudaError_t launch_main(const CUtensorMap& mk, const CUtensorMap& mv, const PaArgs& a, int grid, int dev,
                        cudaStream_t s) {
  static SmemOptIn opt_in;
  using C = PaCfg<D, kH>;
  const cudaError_t e = opt_in(page_attention_kernel<D, kH>, C::kSmem, dev);
  if (e != cudaSuccess) return e;
  page_attention_kernel<D, kH><<<grid, kPaThreads, C::kSmem, s>>>(mk, mv, a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_all(const CUtensorMap& mk, const CUtensorMap& mv, const PaArgs& a, int grid, int dev,
                        cudaStream_t s) {
  // As many heads as there are, nearly: short calls pay for the code of every head (12 against
  // 16: 18 sequences of up to 16927 tokens, one key head, 21.4 and 23.8 us, 256 of 1024, two
  // key heads, 48 and 59; 6 against 8: 256 of 1024, four key heads, 57 and 63).
  cudaError_t e = a.G <= 2    ? launch_main<D, 2>(mk, mv, a, grid, dev, s)
                  : a.G <= 4  ? launch_main<D, 4>(mk, mv, a, grid, dev, s)
                  : a.G <= 6  ? launch_main<D, 6>(mk, mv, a, grid, dev, s)
                  : a.G <= 8  ? launch_main<D, 8>(mk, mv, a, grid, dev, s)
                  : a.G <= 12 ? launch_main<D, 12>(mk, mv, a, grid, dev, s)
                              : launch_main<D, 16>(mk, mv, a, grid, dev, s);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(grid, ceil_div(a.G, 4));
  lc.blockDim = dim3(kJoinThreads);
  lc.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  e = cudaLaunchKernelEx(&lc, page_attention_join_kernel<D>, a, grid);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace
}  // namespace rkv

using namespace rkv;

extern "C" rkv_status rkv_page_attention_workspace(const rkv_pages* pages, const rkv_page_table* table,
                                                   int32_t n_q_heads, size_t* bytes) {
  if (!bytes) return fail_with(RKV_EINVAL, "bytes is NULL");
  if (rkv_status st = check_pages(pages)) return st;
  if (rkv_status st = check_table(table, pages->block_tokens)) return st;
  if (rkv_status st = check_heads(pages, n_q_heads)) return st;
  const size_t G = n_q_heads / pages->n_kv_heads;
  *bytes = 2 * kMaxCtas * (sizeof(PartialOf) + sizeof(float) * G * (2 + (size_t)pages->head_dim));
  return RKV_OK;
}

extern "C" rkv_status rkv_page_attention(const rkv_pages* pages, const rkv_page_table* table, const void* q,
                                         const int64_t q_strides[2], int32_t n_q_heads, double scale,
                                         void* out, float* lse, void* workspace, size_t workspace_bytes,
                                         int32_t* flags, void* stream) {
  size_t need = 0;
  if (rkv_status st = rkv_page_attention_workspace(pages, table, n_q_heads, &need)) return st;
  if (!q || !q_strides || !out || !workspace) return fail_with(RKV_EINVAL, "NULL pointer");
  if (!scale_ok(scale)) return fail_with(RKV_EINVAL, "scale must be at least 1e-30 and below 1e30");
  if (workspace_bytes < need) return fail_with(RKV_ECAPACITY, "workspace has %zu of %zu bytes", workspace_bytes, need);
  if (!is_aligned(q, 16) || !is_aligned(out, 16) || !is_aligned(workspace, 16) || q_strides[0] < 0 ||
      q_strides[1] < 0 || q_strides[0] % 8 || q_strides[1] % 8)
    return fail_with(RKV_EALIGN, "q, out, workspace and q's strides must be whole 16 bytes");
  int dev = 0, sms = 0;
  if (!current_device(dev, sms)) return fail_with(RKV_ECUDA, "no usable current device");
  const int D = pages->head_dim;
  const uint64_t rows = (uint64_t)pages->num_blocks * pages->n_kv_heads * pages->block_tokens;
  CUtensorMap mk, mv;
  if (!encode_map_bytes(&mk, pages->k, D, rows, pages->block_tokens) ||
      !encode_map_bytes(&mv, pages->v, D, rows, pages->block_tokens))
    return fail_with(RKV_ECUDA, "cuTensorMapEncodeTiled is unavailable or rejected the pages");
  PaArgs a;
  a.ks = pages->k_scale, a.vs = pages->v_scale;
  a.table = table->block_table, a.seq_len = table->seq_len;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.qst = {q_strides[0], q_strides[1]};
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse, a.flags = flags;
  a.batch = table->batch;
  a.N = pages->n_kv_heads, a.G = n_q_heads / a.N;
  a.info = static_cast<PartialOf*>(workspace);
  a.pm = reinterpret_cast<float*>(a.info + 2 * kMaxCtas);
  a.pl = a.pm + 2 * kMaxCtas * a.G;
  a.po = a.pl + 2 * kMaxCtas * a.G;
  a.shift = 4;
  while ((1 << a.shift) < pages->block_tokens) ++a.shift;
  a.num_blocks = pages->num_blocks, a.max_blocks = table->max_blocks;
  a.scale_log2 = (float)(scale * 1.4426950408889634);
  const int grid = sms < kMaxCtas ? sms : kMaxCtas;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = D == 128 ? launch_all<128>(mk, mv, a, grid, dev, s) : launch_all<64>(mk, mv, a, grid, dev, s);
  return e == cudaSuccess ? RKV_OK : fail_with(RKV_ECUDA, "page attention launch failed: %s", cudaGetErrorString(e));
}
