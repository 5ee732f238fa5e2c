// k_heads.cu - norm and rotation of query and key rows before the attention.
//
// A head's row x of D values becomes y = x / sqrt(mean(x^2) + eps) w (or x itself), and pair j
// of its first `rotary` values turns by the angle position freq_j:
//   y_a cos - y_b sin, y_b cos + y_a sin.
// The angle of a far position needs more bits than fp32 has, and only its place within a turn
// matters: freq_j / 2 pi is kept as a 64-bit binary fraction of a turn, an integer product with
// the position drops the whole turns by overflow, and the upper 32 bits, taken as a signed
// number, are the angle in [-pi, pi) to 2^-32 of a turn.  fp32 takes them to 24 bits, up to
// 2^-26 of a turn (1.6 2^-24 radians) near half of one, next to the sine's and cosine's 2 ulp.
//
// Bandwidth bounds many rows, one chain of loads few (16 rows of 40 heads of 128 2.9 us).  A warp
// takes a row: the sines are found once for its heads, a part of them in each lane.  The next
// heads' values, or the next row's, are on their way while some are turned.  32768 rows of 32 + 8
// heads of 128, normed and turned: 108 us, 6.2 TB/s (125 us with the sines found by every lane,
// nothing loaded ahead and products one by one; 111 with the next row's values not loaded ahead).
// Seven CTAs of 128 threads an SM: six are 112 us, eight spill (110); rows cut into two shares
// 118, several waves of CTAs 112 to 120 (each sets the turns up again).  That was chosen for bf16:
// with fp32 rows seven spill too (20 bytes a thread stored, 12 loaded), and 16384 of them take
// 124.5 us (5.4 TB/s) to fp32, 76.9 (6.5) to bf16.  Further from the copy's rate: adjacent pairs
// 129 us, rotary 32 of 128 128 (both 5.2 TB/s), and heads that do not fill a warp's groups, which
// leave lanes idle: 5 + 5 of 128 3.9 TB/s, 12 + 1 of 128 5.0, of 64 3.3.
#include <cuda_bf16.h>

#include "pages.h"
#include "ptx.cuh"

namespace rkv {
namespace {

constexpr int kHeadThreads = 128;
constexpr int kHeadWarps = kHeadThreads / 32;
constexpr int kHeadCtas = 7;         // resident CTAs an SM (fp32 rows spill a little)

struct HeadRows {
  const void* x[2];                  // q, k
  void* out[2];
  Strides st[2], ost[2];
  const void* weight[2];             // D values of x's type, or nullptr
  int heads[2];
};

struct HeadArgs {
  HeadRows h;
  const int32_t* positions;
  const double* freq;
  int n_rows, rotary, adjacent, shares;
  float eps;                         // below 0: no norm
};

__device__ __forceinline__ uint64_t f32x2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

__device__ __forceinline__ uint4 load16(const void* p) { return *static_cast<const uint4*>(p); }

// Eight consecutive values, as loaded; widen() gives four pairs of floats.
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  uint4 u = make_uint4(0, 0, 0, 0);
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = load16(p); }
  __device__ __forceinline__ void widen(uint64_t* f) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f32x2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
};
template <>
struct Chunk<float> {
  uint4 u[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  __device__ __forceinline__ void load(const float* p) { u[0] = load16(p), u[1] = load16(p + 4); }
  __device__ __forceinline__ void widen(uint64_t* f) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[2 * i] = f32x2_pack(__uint_as_float(u[i].x), __uint_as_float(u[i].y));
      f[2 * i + 1] = f32x2_pack(__uint_as_float(u[i].z), __uint_as_float(u[i].w));
    }
  }
};
__device__ __forceinline__ void store8(__nv_bfloat16* p, const uint64_t* f) {
  uint4 u;
  uint32_t* w = &u.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f32x2_unpack(f[i], lo, hi);
    const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    w[i] = *reinterpret_cast<const uint32_t*>(&t);
  }
  *reinterpret_cast<uint4*>(p) = u;
}
__device__ __forceinline__ void store8(float* p, const uint64_t* f) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f32x2_unpack(f[i], v[2 * i], v[2 * i + 1]);
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Sum over the lanes of a head of the squares of 16 values.
template <int kLanes>
__device__ __forceinline__ float sum_squares(const uint64_t* x) {
  uint64_t sum = f32x2_mul(x[0], x[0]);
#pragma unroll
  for (int e = 1; e < 8; ++e) sum = f32x2_fma(x[e], x[e], sum);
  float lo, hi;
  f32x2_unpack(sum, lo, hi);
  lo += hi;
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) lo += __shfl_xor_sync(0xffffffffu, lo, o);
  return lo;
}

// D / 16 lanes share a head's row: each has two chunks of eight values, a pair's two values
// both.  A warp takes a share of one row's heads, kPar at a time; the lanes that have a chunk of
// different heads turn the same pairs, and each finds the sines of some of them for all.
template <typename In, typename Out, int D>
__global__ void __launch_bounds__(kHeadThreads, kHeadCtas) head_norm_rotate_kernel(const __grid_constant__ HeadArgs p) {
  constexpr int kLanes = D / 16;
  constexpr int kPar = 32 / kLanes;  // heads that a warp takes at a time
  constexpr int kMine = 8 / kPar;    // pairs of which a lane finds the sines
  __shared__ uint64_t s_turn[D / 2];
  __shared__ __align__(16) float s_weight[2][D];
  const int tid = threadIdx.x, lane = tid & 31, l = lane % kLanes, sub = lane / kLanes;
  const int half = p.rotary / 2;
  // the lane's chunks, and whether they turn (rotary is a multiple of 16)
  const bool turns = l * 16 < p.rotary;
  int at0 = l * 16, at1 = at0 + 8;
  if (!p.adjacent && turns) at0 = l * 8, at1 = half + l * 8;
  const int parts_q = ceil_div(p.h.heads[0], kPar), parts = parts_q + ceil_div(p.h.heads[1], kPar);
  const int64_t tasks = (int64_t)p.n_rows * p.shares;
  const bool norm = p.eps >= 0.0f;
  const int64_t stride = (int64_t)gridDim.x * kHeadWarps;
  int64_t task = (int64_t)blockIdx.x * kHeadWarps + tid / 32;
  Chunk<In> next[2];
  auto fetch = [&](int row, int g) {
    const int which = g >= parts_q, head = (which ? g - parts_q : g) * kPar + sub;
    if (head < p.h.heads[which]) {
      const In* src = static_cast<const In*>(p.h.x[which]) + row * p.h.st[which].row + head * p.h.st[which].head;
      next[0].load(src + at0);
      next[1].load(src + at1);
    }
  };
  // a task's row and share of the parts; rows fit 32 bits
  int row, lo, hi;
  auto place = [&](int64_t t) {
    row = (int)(t / p.shares);
    const int share = (int)(t - (int64_t)row * p.shares);
    lo = (int)((int64_t)parts * share / p.shares), hi = (int)((int64_t)parts * (share + 1) / p.shares);
  };
  const bool any = task < tasks;
  pdl_wait_previous_grid();
  int pos = -1;
  if (any) {
    place(task);
    pos = p.positions[row];
    fetch(row, lo);
  }
  // while the first values are on their way: the turns, and the weights as floats
  for (int i = tid; i < D / 2; i += kHeadThreads) {
    double t = i < p.rotary / 2 ? p.freq[i] * 0.15915494309189533576888 : 0.0;      // 1 / (2 pi)
    t -= rint(t);
    s_turn[i] = (uint64_t)__double2ll_rn(t * 18446744073709551616.0);
  }
  for (int i = tid; i < 2 * D; i += kHeadThreads) {
    const In* w = static_cast<const In*>(p.h.weight[i / D]);
    s_weight[i / D][i % D] = w ? (float)w[i % D] : 1.0f;
  }
  __syncthreads();
  if (!any) return;
  while (true) {
    // the next task's first values are on their way before this one's last are done
    const int row_now = row, lo_now = lo, hi_now = hi, pos_now = pos;
    task += stride;
    const bool more = task < tasks;
    if (more) {
      place(task);
      pos = p.positions[row];
    }
    if (pos_now < 0) {
      if (!more) break;
      fetch(row, lo);
      continue;
    }
    // cosines and sines of the lane's pairs, two by two
    uint64_t c[4], s[4];
    {
      float cm[kMine], sm[kMine], cv[8], sv[8];
#pragma unroll
      for (int e = 0; e < kMine; ++e) {
        const int32_t t = (int32_t)((s_turn[l * 8 + sub * kMine + e] * (uint64_t)pos_now) >> 32);
        sincospif((float)t * 4.656612873077393e-10f, &sm[e], &cm[e]);            // 2^-31
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        cv[e] = __shfl_sync(0xffffffffu, cm[e % kMine], e / kMine * kLanes + l);
        sv[e] = __shfl_sync(0xffffffffu, sm[e % kMine], e / kMine * kLanes + l);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = f32x2_pack(cv[2 * i], cv[2 * i + 1]);
        s[i] = f32x2_pack(sv[2 * i], sv[2 * i + 1]);
      }
    }
    for (int g = lo_now; g < hi_now; ++g) {
      const int which = g >= parts_q, head = (which ? g - parts_q : g) * kPar + sub;
      uint64_t x[8];
      next[0].widen(x);
      next[1].widen(x + 4);
      if (g + 1 < hi_now) fetch(row_now, g + 1);
      else if (more) fetch(row, lo);
      if (norm) {
        const float sum = sum_squares<kLanes>(x);
        float r = rsqrtf(fmaf(sum, 1.0f / D, p.eps));
        if (__any_sync(0xffffffffu, !(sum < INFINITY))) {
          // squares past fp32: those of x 2^-70 are not, and eps, left out, is up to 4 10^-7 of their
          // mean (1e30 beside 2^128 / 128), 1.9 10^-7 of the result: below rsqrtf's 2 ulp
          const float down = sum < INFINITY ? 1.0f : 8.470329472543003e-22f;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = f32x2_mul(x[e], f32x2_pack(down, down));
          const float small = sum_squares<kLanes>(x);
          if (!(sum < INFINITY)) r = rsqrtf(small * (1.0f / D));
        }
        const float* w = s_weight[which];
        const uint64_t r2 = f32x2_pack(r, r);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4* wf = reinterpret_cast<const float4*>(w + (h ? at1 : at0));
          const float4 wa = wf[0], wb = wf[1];
          const uint64_t w2[4] = {f32x2_pack(wa.x, wa.y), f32x2_pack(wa.z, wa.w), f32x2_pack(wb.x, wb.y), f32x2_pack(wb.z, wb.w)};
#pragma unroll
          for (int e = 0; e < 4; ++e) x[4 * h + e] = f32x2_mul(f32x2_mul(x[4 * h + e], r2), w2[e]);
        }
      }
      if (turns) {
        if (p.adjacent) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float a, b, c0, c1, s0, s1;
            f32x2_unpack(x[e], a, b);
            f32x2_unpack(c[e / 2], c0, c1);
            f32x2_unpack(s[e / 2], s0, s1);
            const float ce = e % 2 ? c1 : c0, se = e % 2 ? s1 : s0;
            x[e] = f32x2_pack(a * ce - b * se, b * ce + a * se);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint64_t a = x[e], b = x[4 + e];
            x[e] = f32x2_sub(f32x2_mul(a, c[e]), f32x2_mul(b, s[e]));
            x[4 + e] = f32x2_fma(b, c[e], f32x2_mul(a, s[e]));
          }
        }
      }
      if (head < p.h.heads[which]) {
        Out* dst = static_cast<Out*>(p.h.out[which]) + row_now * p.h.ost[which].row + head * p.h.ost[which].head;
        store8(dst + at0, x);
        store8(dst + at1, x + 4);
      }
    }
    if (!more) break;
  }
}

template <typename In, typename Out, int D>
cudaError_t launch_heads(HeadArgs a, int sms, cudaStream_t s) {
  constexpr int kPar = 32 / (D / 16);
  const int parts = ceil_div(a.h.heads[0], kPar) + ceil_div(a.h.heads[1], kPar);
  // as many warps as the GPU holds; few rows are shared by warps
  const int64_t most = (int64_t)sms * kHeadCtas * kHeadWarps;
  int64_t shares = most / a.n_rows;
  a.shares = (int)(shares < 1 ? 1 : shares < parts ? shares : parts);
  const int64_t ctas = ((int64_t)a.n_rows * a.shares + kHeadWarps - 1) / kHeadWarps;
  const int64_t grid = ctas < (int64_t)sms * kHeadCtas ? ctas : (int64_t)sms * kHeadCtas;
  return launch_behind(head_norm_rotate_kernel<In, Out, D>, a, (unsigned)grid, kHeadThreads, 0, s);
}

template <int D>
cudaError_t launch_types(const HeadArgs& a, int dtype, int out_dtype, int sms, cudaStream_t s) {
  if (dtype == RKV_BF16) return launch_heads<__nv_bfloat16, __nv_bfloat16, D>(a, sms, s);
  return out_dtype == RKV_BF16 ? launch_heads<float, __nv_bfloat16, D>(a, sms, s)
                               : launch_heads<float, float, D>(a, sms, s);
}

}  // namespace
}  // namespace rkv

using namespace rkv;

extern "C" rkv_status rkv_head_norm_rotate(const rkv_head_rows* hr, void* stream) {
  if (!hr) return fail_with(RKV_EINVAL, "rows is NULL");
  const rkv_head_rows& r = *hr;
  if (r.head_dim != 64 && r.head_dim != 128) return fail_with(RKV_EINVAL, "head_dim must be 64 or 128");
  if (r.rotary_dim < 0 || r.rotary_dim > r.head_dim || r.rotary_dim % 16)
    return fail_with(RKV_EINVAL, "rotary_dim must be a multiple of 16 up to head_dim");
  if ((r.dtype != RKV_BF16 && r.dtype != RKV_F32) || (r.out_dtype != RKV_BF16 && r.out_dtype != r.dtype))
    return fail_with(RKV_EINVAL, "dtype must be RKV_F32 or RKV_BF16, out_dtype the same or RKV_BF16");
  if (r.n_rows < 0 || r.n_rows > 1 << 30) return fail_with(RKV_EINVAL, "n_rows must be in 0..2^30");
  if (r.n_q_heads < 0 || r.n_q_heads > 65535 || r.n_k_heads < 0 || r.n_k_heads > 65535)
    return fail_with(RKV_EINVAL, "head counts must be in 0..65535");
  if (r.norm && !(r.eps >= 1e-30 && r.eps <= 1e30)) return fail_with(RKV_EINVAL, "eps must be in 1e-30..1e30");
  if (!r.norm && (r.q_weight || r.k_weight)) return fail_with(RKV_EINVAL, "weights without a norm");
  if (r.n_rows == 0 || r.n_q_heads + r.n_k_heads == 0) return RKV_OK;
  if (!r.positions || (r.rotary_dim && !r.freq)) return fail_with(RKV_EINVAL, "NULL positions or freq");
  HeadArgs a;
  const void* x[2] = {r.q, r.k};
  void* out[2] = {r.q_out, r.k_out};
  const int64_t* st[2] = {r.q_strides, r.k_strides};
  const int64_t* ost[2] = {r.q_out_strides, r.k_out_strides};
  const void* w[2] = {r.q_weight, r.k_weight};
  const int heads[2] = {r.n_q_heads, r.n_k_heads};
  const int per16 = r.dtype == RKV_F32 ? 4 : 8, out16 = r.out_dtype == RKV_F32 ? 4 : 8;
  for (int i = 0; i < 2; ++i) {
    a.h.x[i] = x[i], a.h.out[i] = out[i], a.h.weight[i] = w[i], a.h.heads[i] = heads[i];
    a.h.st[i] = {st[i][0], st[i][1]}, a.h.ost[i] = {ost[i][0], ost[i][1]};
    if (heads[i] == 0) continue;
    if (!x[i] || !out[i]) return fail_with(RKV_EINVAL, "NULL rows");
    if (!is_aligned(x[i], 16) || !is_aligned(out[i], 16) || !is_aligned(w[i], 4))
      return fail_with(RKV_EALIGN, "rows must be 16-byte aligned, weights 4-byte");
    for (int j = 0; j < 2; ++j)
      if (st[i][j] < 0 || st[i][j] % per16 || ost[i][j] < 0 || ost[i][j] % out16)
        return fail_with(RKV_EALIGN, "strides must be >= 0 and multiples of 16 bytes");
    if (!rows_apart(r.n_rows, heads[i], r.head_dim, ost[i]))
      return fail_with(RKV_EINVAL, "rows of an output overlap");
  }
  if (r.rotary_dim && !is_aligned(r.freq, 8)) return fail_with(RKV_EALIGN, "freq must be 8-byte aligned");
  // other warps read rows while one writes: an output is its own input, or apart from both inputs
  RowBytes from[2], to[2];
  for (int i = 0; i < 2; ++i)
    if (heads[i] && (!row_bytes(x[i], r.n_rows, heads[i], r.head_dim, st[i], r.dtype == RKV_F32 ? 4 : 2, from[i]) ||
                     !row_bytes(out[i], r.n_rows, heads[i], r.head_dim, ost[i], r.out_dtype == RKV_F32 ? 4 : 2, to[i])))
      return fail_with(RKV_EINVAL, "strides pass the address space");
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      if (heads[i] && heads[j] && !(i == j && from[j] == to[i]) && rows_meet(from[j], to[i]))
        return fail_with(RKV_EINVAL, "an output overlaps an input and is not that input's own");
  if (heads[0] && heads[1] && rows_meet(to[0], to[1])) return fail_with(RKV_EINVAL, "q_out and k_out overlap");
  a.positions = r.positions;
  a.freq = r.freq;
  a.n_rows = r.n_rows, a.rotary = r.rotary_dim, a.adjacent = r.adjacent != 0;
  a.eps = r.norm ? (float)r.eps : -1.0f;
  int dev = 0, sms = 0;
  if (!current_device(dev, sms)) return fail_with(RKV_ECUDA, "no usable current device");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = r.head_dim == 128 ? launch_types<128>(a, r.dtype, r.out_dtype, sms, s)
                                          : launch_types<64>(a, r.dtype, r.out_dtype, sms, s);
  return e == cudaSuccess ? RKV_OK : fail_with(RKV_ECUDA, "head rows launch failed: %s", cudaGetErrorString(e));
}
