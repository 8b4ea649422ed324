// Attention over the paged cache, the plain way: one warp per (token, q-head) walks the keys.
#include <math_constants.h>

#include "attn.h"
#include "common.cuh"

namespace gdn {
namespace {

template <int D>
__global__ void __launch_bounds__(128) attn_simple_kernel(AttnParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (w >= (long long)p.tokens * p.hq) return;
  const int tok = (int)(w / p.hq), h = (int)(w % p.hq), hk = h / (p.hq / p.hkv);
  int n = tok, back = 1;
  if (p.cu_seqlens) {
    n = find_seq(p.cu_seqlens, p.num_seqs, tok, lane);
    int bos, eos;
    seq_range(p.cu_seqlens, n, p.tokens, bos, eos);
    back = eos - tok;
  }
  const int len = (int)min(max((long long)p.kv_lens[n], 0ll), (long long)p.max_pages * p.page_size);
  const int own = min(max(len - back + 1, 0), len);
  float q[E], acc[E] = {}, m = -CUDART_INF_F, l = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i)
    q[i] = __bfloat162float(((const __nv_bfloat16 *)p.q)[tok * p.qs[0] + h * p.qs[1] + lane + 32 * i]);
  for (int c = 0; c < p.prefix_len + own; ++c) {
    const int key = c < p.prefix_len ? c : c - p.prefix_len;
    const int pg = c < p.prefix_len ? p.prefix_table[key / p.page_size]
                                    : p.page_table[(long long)n * p.max_pages + key / p.page_size];
    if ((unsigned)pg >= (unsigned)p.num_pages) continue;
    const long long at = pg * p.page_stride + ((long long)hk * p.page_size + key % p.page_size) * D + lane;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(q[i], __bfloat162float(((const __nv_bfloat16 *)p.k_cache)[at + 32 * i]), s);
    s = warp_sum(s) * p.scale;
    const float m1 = fmaxf(m, s), a = __expf(m - m1), e = __expf(s - m1);
    m = m1;
    l = l * a + e;
#pragma unroll
    for (int i = 0; i < E; ++i)
      acc[i] = fmaf(acc[i], a, e * __bfloat162float(((const __nv_bfloat16 *)p.v_cache)[at + 32 * i]));
  }
#pragma unroll
  for (int i = 0; i < E; ++i) {
    float o = l > 0.f ? acc[i] / l : 0.f;
    if (p.gate) {
      const float g = __bfloat162float(((const __nv_bfloat16 *)p.gate)[tok * p.gs[0] + h * p.gs[1] + lane + 32 * i]);
      o = o / (1.f + __expf(-g));
    }
    ((__nv_bfloat16 *)p.o)[w * D + lane + 32 * i] = __float2bfloat16_rn(o);
  }
  if (p.lse && lane == 0) p.lse[w] = l > 0.f ? m + logf(l) : -CUDART_INF_F;
}

}  // namespace

cudaError_t launch_attn_simple(const AttnParams &p, cudaStream_t stream) {
  const unsigned blocks = (unsigned)(((long long)p.tokens * p.hq + 3) / 4);
  if (p.d == 128) attn_simple_kernel<128><<<blocks, 128, 0, stream>>>(p);
  else attn_simple_kernel<256><<<blocks, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gdn
