// k_page_attention.cu - decode attention over 8-bit pages: o = softmax(scale q K^T) V.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "pages.h"

namespace rkv {
namespace {

struct PageAttnArgs {
  const uint8_t *k, *v;
  const float *ks, *vs;
  const int32_t *table, *seq_len;
  const __nv_bfloat16* q;
  Strides qst;
  __nv_bfloat16* out;
  float* lse;
  int32_t* flags;
  int N, Hq, shift, num_blocks, max_blocks;
  float scale;
};

// One warp per (sequence, query head): a running maximum and sum over the positions.
template <int D>
__global__ void page_attention_kernel(PageAttnArgs p) {
  const int b = blockIdx.x, hq = blockIdx.y, lane = threadIdx.x;
  const int h = hq / (p.Hq / p.N);
  constexpr int kE = D / 32;
  float q[kE], o[kE], m = -INFINITY, l = 0.f;
  for (int e = 0; e < kE; ++e) {
    q[e] = __bfloat162float(p.q[b * p.qst.row + hq * p.qst.head + lane * kE + e]) * p.scale;
    o[e] = 0.f;
  }
  int len = p.seq_len[b];
  const int cap = p.max_blocks << p.shift;
  if (len < 0 || len > cap) {
    raise_flag(p.flags, RKV_FLAG_BAD_INDEX);
    len = len < 0 ? 0 : cap;
  }
  for (int t = 0; t < len; ++t) {
    const int id = p.table[(int64_t)b * p.max_blocks + (t >> p.shift)];
    if (id < 0 || id >= p.num_blocks) {
      raise_flag(p.flags, RKV_FLAG_BAD_INDEX);
      continue;
    }
    const int64_t head = (int64_t)id * p.N + h;
    const int64_t row = ((head << p.shift) + (t & ((1 << p.shift) - 1))) * D + lane * kE;
    float s = 0.f;
    for (int e = 0; e < kE; ++e) {
      __nv_fp8_e4m3 c;
      c.__x = p.k[row + e];
      s += q[e] * (float)c;
    }
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    s *= p.ks[head];
    const float mn = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.f : expf(m - mn), w = expf(s - mn);
    l = l * f + w;
    for (int e = 0; e < kE; ++e) {
      __nv_fp8_e4m3 c;
      c.__x = p.v[row + e];
      o[e] = o[e] * f + w * (float)c * p.vs[head];
    }
    m = mn;
  }
  for (int e = 0; e < kE; ++e)
    p.out[((int64_t)b * p.Hq + hq) * D + lane * kE + e] = __float2bfloat16(l != 0.f ? o[e] / l : 0.f);
  if (p.lse && lane == 0) p.lse[(int64_t)b * p.Hq + hq] = l != 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace
}  // namespace rkv

using namespace rkv;

static rkv_status check_heads(const rkv_pages* pages, int n_q_heads) {
  if (n_q_heads < 1 || n_q_heads % pages->n_kv_heads || n_q_heads / pages->n_kv_heads > kPageMaxGroup)
    return fail_with(RKV_EINVAL, "n_q_heads must be a multiple of n_kv_heads, at most %d times it", kPageMaxGroup);
  return RKV_OK;
}

extern "C" rkv_status rkv_page_attention_workspace(const rkv_pages* pages, const rkv_page_table* table,
                                                   int32_t n_q_heads, size_t* bytes) {
  if (!bytes) return fail_with(RKV_EINVAL, "bytes is NULL");
  if (rkv_status st = check_pages(pages)) return st;
  if (rkv_status st = check_table(table, pages->block_tokens)) return st;
  if (rkv_status st = check_heads(pages, n_q_heads)) return st;
  *bytes = 16;
  return RKV_OK;
}

extern "C" rkv_status rkv_page_attention(const rkv_pages* pages, const rkv_page_table* table, const void* q,
                                         const int64_t q_strides[2], int32_t n_q_heads, double scale,
                                         void* out, float* lse, void* workspace, size_t workspace_bytes,
                                         int32_t* flags, void* stream) {
  size_t need = 0;
  if (rkv_status st = rkv_page_attention_workspace(pages, table, n_q_heads, &need)) return st;
  if (!q || !q_strides || !out || !workspace) return fail_with(RKV_EINVAL, "NULL pointer");
  if (!(scale > 0.0 && scale < 1e30)) return fail_with(RKV_EINVAL, "scale must be finite and > 0");
  if (workspace_bytes < need) return fail_with(RKV_ECAPACITY, "workspace has %zu of %zu bytes", workspace_bytes, need);
  if (!is_aligned(q, 16) || !is_aligned(out, 16) || !is_aligned(workspace, 16) || q_strides[0] < 0 ||
      q_strides[1] < 0 || q_strides[0] % 8 || q_strides[1] % 8)
    return fail_with(RKV_EALIGN, "q, out, workspace and q's strides must be whole 16 bytes");
  PageAttnArgs a;
  a.k = static_cast<const uint8_t*>(pages->k), a.v = static_cast<const uint8_t*>(pages->v);
  a.ks = pages->k_scale, a.vs = pages->v_scale;
  a.table = table->block_table, a.seq_len = table->seq_len;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.qst = {q_strides[0], q_strides[1]};
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse, a.flags = flags;
  a.N = pages->n_kv_heads, a.Hq = n_q_heads;
  a.shift = 4;
  while ((1 << a.shift) < pages->block_tokens) ++a.shift;
  a.num_blocks = pages->num_blocks, a.max_blocks = table->max_blocks;
  a.scale = (float)scale;
  const dim3 grid(table->batch, n_q_heads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (pages->head_dim == 128) page_attention_kernel<128><<<grid, 32, 0, s>>>(a);
  else page_attention_kernel<64><<<grid, 32, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? RKV_OK : fail_with(RKV_ECUDA, "page attention launch failed: %s", cudaGetErrorString(e));
}
