// k_prompt.cu - causal attention of packed prompts: o = softmax(scale q K^T) V.
//
// Bound by the tensor core: 4 D flops for each visible (query, key) pair and head.  A CTA
// works on two tiles of 128 query rows that read the same key/value head, so that the tensor
// core always has one tile's products while the other tile's softmax runs:
//   S_t = Q_t K^T   [128 rows x 128 keys] in TMEM, thread r of softmax group t owns row r
//   P_t = 2^(c s - c m) as bf16 over S_t in TMEM
//   O_t += P_t V    A = P_t from TMEM, V an MN-major B; accumulated in TMEM
// tcgen05 products execute in issue order, and a commit covers everything issued before it:
// S_t of key tile j is complete only when P_t V of tile j - 1 is, so one barrier a tile
// tells its group both.  No reduction crosses threads.  m is the row's maximum over some
// earlier tiles: it is raised (sum and accumulator rescaled) only when a score exceeds it
// by 2^8, so most tiles rescale nothing.  Sums are fp32 over the unrounded weights.
//
// Row tiles of one sequence and key/value head are numbered r = q_tile G + head and taken
// in consecutive pairs, so that both need the same keys (or one tile more): with an even G
// two heads of one query tile, with G = 1 two neighbouring query tiles.  One CTA an SM walks
// the pairs of all sequences, longest rows of a sequence first, in alternating directions,
// so that its shares of long and short pairs even out.
//
// Packed rows: a tile's rows behind its sequence are other sequences' rows.  Their queries
// fill lanes whose results are not stored; their keys are masked by position; their values
// are zeroed in shared memory, for 0 times what they hold must be 0.
//
// Warps: 0-3 and 4-7 softmax of tiles 0 and 1, 8 TMA, 9 MMA, 10 work list, 11 TMEM.
#include <cuda_bf16.h>

#include "pages.h"
#include "tc_common.cuh"

namespace rkv {
namespace {

constexpr int kRows = 128;                 // query rows of a tile
constexpr int kKeys = 128;                 // keys of a tile
constexpr int kPrThreads = 384;
constexpr int kItems = 2;                  // work items held ahead
constexpr float kPrRaise = 8.f;

// Two row tiles of one sequence and key/value head.
struct Item {
  int kvh;                                 // key/value head; -1 ends the list
  int k0, lk;                              // the sequence's first key row, its keys
  int row[2], rows[2];                     // first row of q / out, rows of the tile (0: none)
  int head[2];                             // query head
  int lim[2];                              // keys that the tile's row 0 sees (may be <= 0)
  int n[2];                                // key tiles; n[0] <= n[1]
};

struct PrArgs {
  __nv_bfloat16* out;
  float* lse;
  Strides ost;
  const int32_t *cu_q, *cu_k;
  int32_t* flags;
  int batch, total_q, total_k, Hq, N, G;
  float scale_log2;
};

template <int D>
struct PrCfg {
  static constexpr uint32_t kTileB = kKeys * D * 2;          // bytes of a Q, K or V tile
  static constexpr int kSlots = D == 128 ? 5 : 10;           // ring of K and V tiles
  static constexpr uint32_t kSmem = 1024 + (2 + kSlots) * kTileB;
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

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  const bool ok = warp_wait(bar, parity, abort, status);
  __syncwarp();
  return ok;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
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
  __shared__ __align__(8) uint64_t kv_full[kSlots], kv_empty[kSlots], q_full, q_empty, s_full[2], p_full[2],
      o_full[2], i_full[kItems], i_empty[kItems], drain;
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
    for (int i = 0; i < 2; ++i) mbar_init(&s_full[i], 1), mbar_init(&p_full[i], 128), mbar_init(&o_full[i], 1);
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
          if (!(ok = mbar_wait(&i_full[s], ph, abort, status))) break;
          const Item it = items[s];
          mbar_arrive(&i_empty[s]);
          if (it.kvh < 0) break;
          if (it.n[1] == 0) continue;
          if (!(ok = mbar_wait(&q_empty, q_ph, abort, status))) break;
          q_ph ^= 1u;
          mbar_arrive_expect_tx(&q_full, (it.n[0] > 0 ? 2 : 1) * C::kTileB);
          if (it.n[0] > 0) load_tile<D>(s_q, &tm_q, &q_full, it.head[0], it.row[0]);
          load_tile<D>(s_q + C::kTileB, &tm_q, &q_full, it.head[1], it.row[1]);
          for (int j = 0; j < 2 * it.n[1]; ++j) {            // K 0, V 0, K 1, V 1, ...
            if (!(ok = mbar_wait(&kv_empty[kv.stage], kv.phase ^ 1u, abort, status))) break;
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
        uint32_t q_ph = 0, p_ph[2] = {0, 0};
        bool ok = true;
        const uint32_t q_sm = smem_u32(s_q), kv_sm = smem_u32(s_kv);
        // S_t = Q_t K^T
        auto qk = [&](int t, int slot) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint32_t off = (uint32_t)(i >> 2) * (kKeys * 128) + (uint32_t)(i & 3) * 32;
            umma_bf16(tmem + t * 128, sdesc_sw128(q_sm + t * C::kTileB + off),
                      sdesc_sw128(kv_sm + slot * C::kTileB + off), id_s, i > 0);
          }
          umma_commit(&s_full[t]);
        };
        // O_t (+)= P_t V
        auto pv = [&](int t, int slot, bool acc) {
#pragma unroll
          for (int i = 0; i < kKeys / 16; ++i)
            umma_bf16_ta(tmem + 256 + t * 128, tmem + t * 128 + i * 8,
                         sdesc_mn(kv_sm + slot * C::kTileB + i * 2048, kKeys * 128), id_o, acc || i > 0);
        };
        for (int s = 0, ph = 0; ok; s == kItems - 1 ? (s = 0, ph ^= 1) : ++s) {
          if (!(ok = mbar_wait(&i_full[s], ph, abort, status))) break;
          const int kvh = items[s].kvh, n0 = items[s].n[0], n1 = items[s].n[1];
          mbar_arrive(&i_empty[s]);
          if (kvh < 0) break;
          if (n1 == 0) continue;
          if (!(ok = mbar_wait(&q_full, q_ph, abort, status))) break;
          q_ph ^= 1u;
          if (!(ok = mbar_wait(&kv_full[kv.stage], kv.phase, abort, status))) break;
          tc_fence_after();
          if (n0 > 0) qk(0, kv.stage);
          qk(1, kv.stage);
          umma_commit(&kv_empty[kv.stage]);
          if (n1 == 1) umma_commit(&q_empty);
          kv.next(kSlots);
          for (int j = 0; j < n1 && ok; ++j) {
            const Ring v = kv;                               // V j, then K j + 1
            kv.next(kSlots);
            if (!(ok = mbar_wait(&kv_full[v.stage], v.phase, abort, status))) break;
            if (j + 1 < n1 && !(ok = mbar_wait(&kv_full[kv.stage], kv.phase, abort, status))) break;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int n = t ? n1 : n0;
              if (j < n) {
                if (!(ok = mbar_wait(&p_full[t], p_ph[t], abort, status))) break;
                p_ph[t] ^= 1u;
                tc_fence_after();
                pv(t, v.stage, j > 0);
                if (t == 1) umma_commit(&kv_empty[v.stage]);
                if (j + 1 < n) qk(t, kv.stage);
                else umma_commit(&o_full[t]);
                if (t == 1 && j + 1 < n1) {
                  umma_commit(&kv_empty[kv.stage]);
                  if (j + 2 == n1) umma_commit(&q_empty);
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
      int64_t base = 0;                                      // items before sequence b
      int b = 0, chunk = -1;
      int q0 = 0, lq = 0, k0 = 0, lk = 0;                    // lane i: sequence chunk + i
      bool ok = true;
      const int64_t C0 = gridDim.x;
      int64_t round = 0;
      for (int s = 0, ph = 1; ok; s == kItems - 1 ? (s = 0, ph ^= 1) : ++s, ++round) {
        const int64_t i = round * C0 + ((round & 1) ? C0 - 1 - blockIdx.x : blockIdx.x);
        Item it;
        it.kvh = -1;
        while (b < a.batch) {
          if (chunk != (b & ~31)) {
            chunk = b & ~31;
            const int sb = chunk + lane;
            q0 = lq = k0 = lk = 0;
            if (sb < a.batch) {
              const int c0 = a.cu_q[sb], c1 = a.cu_q[sb + 1], d0 = a.cu_k[sb], d1 = a.cu_k[sb + 1];
              q0 = min(max(c0, 0), a.total_q), k0 = min(max(d0, 0), a.total_k);
              const int q1 = min(max(c1, q0), a.total_q), k1 = min(max(d1, k0), a.total_k);
              lq = q1 - q0, lk = k1 - k0;
              if (blockIdx.x == 0 && (q0 != c0 || q1 != c1 || k0 != d0 || k1 != d1))
                raise_flag(a.flags, RKV_FLAG_BAD_INDEX);
            }
          }
          const int my_pairs = ((lq + kRows - 1) / kRows * a.G + 1) / 2;
          if (b == chunk) {                                  // skip the chunk if it ends before i
            int64_t sum = (int64_t)my_pairs * a.N;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (i >= base + sum) {
              base += sum;
              b += 32;
              continue;
            }
          }
          const int pairs = __shfl_sync(0xffffffffu, my_pairs, b & 31);
          if (i >= base + (int64_t)pairs * a.N) {
            base += (int64_t)pairs * a.N;
            ++b;
            continue;
          }
          const int rel = (int)(i - base);
          const int LQ = __shfl_sync(0xffffffffu, lq, b & 31), Q0 = __shfl_sync(0xffffffffu, q0, b & 31);
          it.lk = __shfl_sync(0xffffffffu, lk, b & 31);
          it.k0 = __shfl_sync(0xffffffffu, k0, b & 31);
          it.kvh = rel % a.N;
          const int top = (LQ + kRows - 1) / kRows * a.G - 1 - 2 * (rel / a.N);   // longest first
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int r = top - 1 + t;
            const int qt = r >= 0 ? r / a.G : 0;
            it.row[t] = Q0 + qt * kRows;
            it.rows[t] = r >= 0 ? min(kRows, LQ - qt * kRows) : 0;
            it.head[t] = it.kvh * a.G + (r >= 0 ? r % a.G : 0);
            it.lim[t] = it.lk - LQ + qt * kRows + 1;
            const int seen = it.lim[t] + it.rows[t] - 1;     // by the tile's last row
            it.n[t] = it.rows[t] > 0 && seen > 0 ? (seen + kKeys - 1) / kKeys : 0;
          }
          break;
        }
        if (!(ok = wait_all(&i_empty[s], ph, abort, status))) break;
        if (lane == 0) {
          items[s] = it;
          mbar_arrive(&i_full[s]);
        }
        __syncwarp();
        if (it.kvh < 0) break;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // -------------------------------------------------------------------------- softmax
    const int t = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_tm = tmem + t * 128 + lanes, o_tm = tmem + 256 + t * 128 + lanes;
    uint32_t s_ph = 0, o_ph = 0;
    Ring kv;                                                 // slot of K j
    const float c = a.scale_log2;
    bool ok = true;
    for (int si = 0, ph = 0; ok; si == kItems - 1 ? (si = 0, ph ^= 1) : ++si) {
      if (!(ok = wait_all(&i_full[si], ph, abort, status))) break;
      const int kvh = items[si].kvh, n = items[si].n[t], n1 = items[si].n[1], lk = items[si].lk;
      const int row = items[si].row[t], rows = items[si].rows[t], head = items[si].head[t];
      // keys that this row sees
      const int see = min(items[si].lim[t] + r, lk);
      const int see0 = items[si].lim[t];
      __syncwarp();
      if (lane == 0) mbar_arrive(&i_empty[si]);
      if (kvh < 0) break;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n1; ++j) {
        kv.next(kSlots);                                     // now V j
        if (j < n) {
          if (!(ok = wait_all(&s_full[t], s_ph, abort, status))) break;
          s_ph ^= 1u;
          tc_fence_after();
          uint32_t x[128];
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld32(s_tm + 32 * i, x + 32 * i);
          tmem_ld_wait();
          if ((j + 1) * kKeys > see0) {                      // some row does not see every key
            const int vis = see - j * kKeys;
#pragma unroll
            for (int i = 0; i < 128; ++i) x[i] = i < vis ? x[i] : 0xFF800000u;
          }
          float mx[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = __uint_as_float(x[i]);
#pragma unroll
          for (int i = 4; i < 128; i += 8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              mx[e] = fmaxf(mx[e], __uint_as_float(x[i + e]));
              if (i + 4 + e < 128) mx[e] = fmaxf(mx[e], __uint_as_float(x[i + 4 + e]));
            }
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          const bool raise = top * c > m * c + kPrRaise;     // also from -inf
          if (__any_sync(0xffffffffu, raise)) {
            const float mn = raise ? top : m;
            const float f = raise ? ex2_approx((m - mn) * c) : 1.f;
            l *= f;
            m = mn;
            if (j > 0) {                                     // P V of tile j - 1 is complete
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                uint32_t o[16];
                tmem_ld16(o_tm + 16 * i, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(o_tm + 16 * i, o);
              }
            }
          }
          const float mc = m == -INFINITY ? 0.f : m * c;
          const uint64_t cc = f32x2_pack(c, c), nm = f32x2_pack(-mc, -mc);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const uint64_t y = fma2(f32x2_pack(__uint_as_float(x[64 * h + 2 * i]),
                                                 __uint_as_float(x[64 * h + 2 * i + 1])), cc, nm);
              float y0, y1;
              f32x2_unpack(y, y0, y1);
              y0 = ex2_approx(y0);
              y1 = ex2_approx(y1);
              sum[i & 1] = f32x2_add(sum[i & 1], f32x2_pack(y0, y1));
              w[i] = bf16x2(y0, y1);
            }
            tmem_st32(s_tm + 32 * h, w);
          }
          float a0, a1;
          f32x2_unpack(f32x2_add(sum[0], sum[1]), a0, a1);
          l += a0 + a1;
          if ((j + 1) * kKeys > lk) {                        // values behind the sequence
            if (!(ok = wait_all(&kv_full[kv.stage], kv.phase, abort, status))) break;
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
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&p_full[t]);
        }
        kv.next(kSlots);                                     // now K j + 1
      }
      if (!ok) break;
      // the rows' results
      const bool live = r < rows;
      const int64_t at = row + r;
      __nv_bfloat16* o = a.out + at * a.ost.row + head * a.ost.head;
      if (n > 0) {
        if (!(ok = wait_all(&o_full[t], o_ph, abort, status))) break;
        o_ph ^= 1u;
        tc_fence_after();
      }
      const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t x[32];
        if (n > 0) {
          tmem_ld32(o_tm + 32 * i, x);
          tmem_ld_wait();
        }
        if (live) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int d = 0; d < 4; ++d)
              w[d] = l != 0.f ? bf16x2(__uint_as_float(x[8 * e + 2 * d]) * inv, __uint_as_float(x[8 * e + 2 * d + 1]) * inv)
                              : 0u;
            *reinterpret_cast<uint4*>(o + 32 * i + 8 * e) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      tc_fence_before();
      if (live && a.lse)
        a.lse[at * a.Hq + head] = l != 0.f ? (m * c + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 11) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PrArgs& a, int grid,
                   int dev, cudaStream_t s) {
  static SmemOptIn opt_in;
  const cudaError_t e = opt_in(prompt_attention_kernel<D>, PrCfg<D>::kSmem, dev);
  if (e != cudaSuccess) return e;
  prompt_attention_kernel<D><<<grid, kPrThreads, PrCfg<D>::kSmem, s>>>(q, k, v, a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace rkv

using namespace rkv;

extern "C" rkv_status rkv_prompt_attention(const rkv_prompt* pr, int32_t* flags, void* stream) {
  if (!pr) return fail_with(RKV_EINVAL, "prompt is NULL");
  const rkv_prompt& p = *pr;
  if (p.head_dim != 64 && p.head_dim != 128) return fail_with(RKV_EINVAL, "head_dim must be 64 or 128");
  if (p.n_kv_heads < 1 || p.n_q_heads < 1 || p.n_q_heads > 65535 || p.n_q_heads % p.n_kv_heads)
    return fail_with(RKV_EINVAL, "n_q_heads must be a multiple of n_kv_heads, at most 65535");
  if (p.batch < 1 || p.batch > kMaxBatch) return fail_with(RKV_EINVAL, "batch must be in 1..%d", kMaxBatch);
  if (p.total_q < 0 || p.total_k < 0 || p.total_q > 1 << 30 || p.total_k > 1 << 30 ||
      (int64_t)p.total_q * p.n_q_heads > (int64_t)1 << 38)
    return fail_with(RKV_EINVAL, "total_q and total_k must be in 0..2^30, total_q * n_q_heads at most 2^38");
  if (!(p.scale > 0.0 && p.scale < 1e30)) return fail_with(RKV_EINVAL, "scale must be finite and > 0");
  if (p.total_q == 0) return RKV_OK;
  if (!p.q || !p.out || !p.cu_q || !p.cu_k || (p.total_k > 0 && (!p.k || !p.v)))
    return fail_with(RKV_EINVAL, "NULL pointer");
  const int64_t* strides[4] = {p.q_strides, p.k_strides, p.v_strides, p.out_strides};
  for (const int64_t* st : strides)
    if (st[0] < 0 || st[1] < 0 || st[0] % 8 || st[1] % 8)
      return fail_with(RKV_EALIGN, "strides must be >= 0 and multiples of 16 bytes");
  if (!is_aligned(p.q, 16) || !is_aligned(p.k, 16) || !is_aligned(p.v, 16) || !is_aligned(p.out, 16))
    return fail_with(RKV_EALIGN, "q, k, v and out must be 16-byte aligned");
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return fail_with(RKV_ECUDA, "no usable current device");
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
  a.cu_q = p.cu_q, a.cu_k = p.cu_k;
  a.flags = flags;
  a.batch = p.batch, a.total_q = p.total_q, a.total_k = p.total_k;
  a.Hq = p.n_q_heads, a.N = p.n_kv_heads, a.G = a.Hq / a.N;
  a.scale_log2 = (float)(p.scale * 1.4426950408889634);
  // no more CTAs than row tiles there can be
  const int64_t tiles = ((int64_t)p.total_q / kRows + p.batch) * p.n_q_heads;
  const int grid = (int)(tiles < sms ? tiles : sms);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = D == 128 ? launch<128>(mq, mk, mv, a, grid, dev, s) : launch<64>(mq, mk, mv, a, grid, dev, s);
  return e == cudaSuccess ? RKV_OK : fail_with(RKV_ECUDA, "prompt attention launch failed: %s", cudaGetErrorString(e));
}
