// k_prompt.cu - causal attention of packed prompts: o = softmax(scale q K^T) V.
#include <cuda_bf16.h>

#include "pages.h"

namespace rkv {
namespace {

struct PromptArgs {
  rkv_prompt p;
  int32_t* flags;
};

// One warp per (query row, query head): a running maximum and sum over the keys.
template <int D>
__global__ void prompt_kernel(PromptArgs a) {
  const rkv_prompt& p = a.p;
  const int row = blockIdx.x, hq = blockIdx.y, lane = threadIdx.x;
  const int h = hq / (p.n_q_heads / p.n_kv_heads);
  if (row == 0 && hq == 0)
    for (int i = lane; i < p.batch; i += 32)
      if (p.cu_q[i] < 0 || p.cu_q[i + 1] < p.cu_q[i] || p.cu_q[i + 1] > p.total_q || p.cu_k[i] < 0 ||
          p.cu_k[i + 1] < p.cu_k[i] || p.cu_k[i + 1] > p.total_k)
        raise_flag(a.flags, RKV_FLAG_BAD_INDEX);
  int b = 0;
  while (b < p.batch && p.cu_q[b + 1] <= row) ++b;
  if (b == p.batch) return;
  const int q1 = min(p.cu_q[b + 1], p.total_q);
  const int k0 = min(max(p.cu_k[b], 0), p.total_k), k1 = min(max(p.cu_k[b + 1], k0), p.total_k);
  const int end = min(k1, k1 - (q1 - row) + 1);    // keys [k0, end) are visible
  constexpr int kE = D / 32;
  const __nv_bfloat16* q = (const __nv_bfloat16*)p.q + row * p.q_strides[0] + hq * p.q_strides[1];
  float qf[kE], o[kE], m = -INFINITY, l = 0.f;
  for (int e = 0; e < kE; ++e) qf[e] = __bfloat162float(q[lane * kE + e]) * (float)p.scale, o[e] = 0.f;
  for (int j = k0; j < end; ++j) {
    const __nv_bfloat16* k = (const __nv_bfloat16*)p.k + j * p.k_strides[0] + h * p.k_strides[1] + lane * kE;
    const __nv_bfloat16* v = (const __nv_bfloat16*)p.v + j * p.v_strides[0] + h * p.v_strides[1] + lane * kE;
    float s = 0.f;
    for (int e = 0; e < kE; ++e) s += qf[e] * __bfloat162float(k[e]);
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    const float mn = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.f : expf(m - mn), w = expf(s - mn);
    l = l * f + w;
    for (int e = 0; e < kE; ++e) o[e] = o[e] * f + w * __bfloat162float(v[e]);
    m = mn;
  }
  __nv_bfloat16* out = (__nv_bfloat16*)p.out + row * p.out_strides[0] + hq * p.out_strides[1];
  for (int e = 0; e < kE; ++e) out[lane * kE + e] = __float2bfloat16(l != 0.f ? o[e] / l : 0.f);
  if (p.lse && lane == 0) p.lse[(int64_t)row * p.n_q_heads + hq] = l != 0.f ? m + logf(l) : -INFINITY;
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
  if (p.total_q < 0 || p.total_k < 0) return fail_with(RKV_EINVAL, "total_q and total_k must be >= 0");
  if (!(p.scale > 0.0 && p.scale < 1e30)) return fail_with(RKV_EINVAL, "scale must be finite and > 0");
  if (p.total_q == 0) return RKV_OK;
  if (!p.q || !p.out || !p.cu_q || !p.cu_k || (p.total_k > 0 && (!p.k || !p.v)))
    return fail_with(RKV_EINVAL, "NULL pointer");
  for (const int64_t* st : {p.q_strides, p.k_strides, p.v_strides, p.out_strides})
    if (st[0] < 0 || st[1] < 0 || st[0] % 8 || st[1] % 8)
      return fail_with(RKV_EALIGN, "strides must be >= 0 and multiples of 16 bytes");
  if (!is_aligned(p.q, 16) || !is_aligned(p.k, 16) || !is_aligned(p.v, 16) || !is_aligned(p.out, 16))
    return fail_with(RKV_EALIGN, "q, k, v and out must be 16-byte aligned");
  PromptArgs a{p, flags};
  const dim3 grid(p.total_q, p.n_q_heads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.head_dim == 128) prompt_kernel<128><<<grid, 32, 0, s>>>(a);
  else prompt_kernel<64><<<grid, 32, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? RKV_OK : fail_with(RKV_ECUDA, "prompt attention launch failed: %s", cudaGetErrorString(e));
}
