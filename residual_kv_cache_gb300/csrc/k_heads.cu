// k_heads.cu - norm and rotation of query and key rows before the attention.
//
// A head's row x of D values becomes y = x / sqrt(mean(x^2) + eps) w (or x itself), and pair j
// of its first `rotary` values turns by the angle position freq_j:
//   y_a cos - y_b sin, y_b cos + y_a sin.
// The angle of a far position needs more bits than fp32 has, and only its place within a turn
// matters: freq_j / 2 pi is kept as a 64-bit binary fraction of a turn, an integer product with
// the position drops the whole turns by overflow, and the upper 32 bits, taken as a signed
// number, are the angle in (-pi, pi] to 2^-32 of a turn.
#include <cuda_bf16.h>

#include "pages.h"

namespace rkv {
namespace {

constexpr int kHeadThreads = 256;
constexpr int kHeadWarps = kHeadThreads / 32;
constexpr int kHeadCtas = 4;         // resident CTAs an SM that the registers allow

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

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* f);
template <>
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* f) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void load8(const float* p, float* f) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* f) {
  uint4 u;
  uint32_t* w = &u.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&t);
  }
  *reinterpret_cast<uint4*>(p) = u;
}
__device__ __forceinline__ void store8(float* p, const float* f) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// D / 16 lanes share a head's row: each has two chunks of eight values, a pair's two values
// both.  A warp takes a share of one row's heads.
template <typename In, typename Out, int D>
__global__ void __launch_bounds__(kHeadThreads) head_norm_rotate_kernel(const __grid_constant__ HeadArgs p) {
  constexpr int kLanes = D / 16;
  constexpr int kPar = 32 / kLanes;  // heads that a warp takes at a time
  __shared__ uint64_t s_turn[D / 2];
  __shared__ float s_weight[2][D];
  const int tid = threadIdx.x, lane = tid & 31, l = lane % kLanes;
  if (tid < p.rotary / 2) {
    double t = p.freq[tid] * 0.15915494309189533576888;          // 1 / (2 pi)
    t -= rint(t);
    s_turn[tid] = (uint64_t)__double2ll_rn(t * 18446744073709551616.0);
  }
  for (int i = tid; i < 2 * D; i += kHeadThreads) {
    const In* w = static_cast<const In*>(p.h.weight[i / D]);
    s_weight[i / D][i % D] = w ? (float)w[i % D] : 1.0f;
  }
  __syncthreads();
  const int half = p.rotary / 2;
  // the lane's chunks, and whether they turn (rotary is a multiple of 16)
  const bool turns = l * 16 < p.rotary;
  int at[2];
  if (p.adjacent || !turns) at[0] = l * 16, at[1] = at[0] + 8;
  else at[0] = l * 8, at[1] = half + l * 8;
  const int parts_q = ceil_div(p.h.heads[0], kPar), parts = parts_q + ceil_div(p.h.heads[1], kPar);
  const int64_t tasks = (int64_t)p.n_rows * p.shares;
  const bool norm = p.eps >= 0.0f;
  for (int64_t task = (int64_t)blockIdx.x * kHeadWarps + tid / 32; task < tasks; task += (int64_t)gridDim.x * kHeadWarps) {
    const int row = (int)(task / p.shares), share = (int)(task - (int64_t)row * p.shares);
    const int pos = p.positions[row];
    if (pos < 0) continue;
    float c[8], s[8];
    if (turns) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int32_t t = (int32_t)((s_turn[l * 8 + e] * (uint64_t)pos) >> 32);
        sincospif((float)t * 4.656612873077393e-10f, &s[e], &c[e]);              // 2^-31
      }
    }
    const int lo = (int)((int64_t)parts * share / p.shares), hi = (int)((int64_t)parts * (share + 1) / p.shares);
    for (int g = lo; g < hi; ++g) {
      const int which = g >= parts_q;
      const int head = (which ? g - parts_q : g) * kPar + lane / kLanes;
      const bool live = head < p.h.heads[which];
      float x[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = 0.0f;
      if (live) {
        const In* src = static_cast<const In*>(p.h.x[which]) + row * p.h.st[which].row + head * p.h.st[which].head;
        load8(src + at[0], x);
        load8(src + at[1], x + 8);
      }
      if (norm) {
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        float r = rsqrtf(fmaf(sum, 1.0f / D, p.eps));
        if (__any_sync(0xffffffffu, !(sum < INFINITY))) {
          // squares past fp32: those of x 2^-70 are not, and eps is nothing beside them
          const float down = sum < INFINITY ? 1.0f : 8.470329472543003e-22f;
          float small = 0.0f;
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] *= down, small = fmaf(x[e], x[e], small);
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1) small += __shfl_xor_sync(0xffffffffu, small, o);
          if (!(sum < INFINITY)) r = rsqrtf(small * (1.0f / D));
        }
        const float* w = s_weight[which];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = x[e] * r * w[at[e / 8] + e % 8];
      }
      if (turns) {
        if (p.adjacent) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float a = x[2 * e], b = x[2 * e + 1];
            x[2 * e] = a * c[e] - b * s[e];
            x[2 * e + 1] = b * c[e] + a * s[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float a = x[e], b = x[8 + e];
            x[e] = a * c[e] - b * s[e];
            x[8 + e] = b * c[e] + a * s[e];
          }
        }
      }
      if (live) {
        Out* dst = static_cast<Out*>(p.h.out[which]) + row * p.h.ost[which].row + head * p.h.ost[which].head;
        store8(dst + at[0], x);
        store8(dst + at[1], x + 8);
      }
    }
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
  head_norm_rotate_kernel<In, Out, D><<<(unsigned)grid, kHeadThreads, 0, s>>>(a);
  return cudaGetLastError();
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
