// Internal launch interface of the attention-layer operators.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

struct AppendParams {
  int num_seqs, tokens, hq, hkv, d, page_size, num_pages, max_pages, rot, axes, pos0;
  float eps;
  int64_t qs[2], ks[2], vs[2], page_stride;
  const void *q, *k, *v;
  const float *q_norm, *k_norm;
  const double *inv_freq;
  const int32_t *rope_axis, *positions, *page_table, *kv_lens, *cu_seqlens;
  void *q_out, *k_cache, *v_cache;
};
cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t stream);

struct AddNormParams {
  long long rows;
  int cols, group;
  float eps;
  const void *x, *residual;
  const float *weight;
  void *residual_out, *y;
  float *scale;
};
cudaError_t launch_add_rmsnorm(const AddNormParams &p, gdn_dtype dtype, cudaStream_t stream);

struct AttnParams {
  int num_seqs, tokens, hq, hkv, d, page_size, num_pages, max_pages, prefix_len;
  float scale;
  int64_t qs[2], gs[2], page_stride;
  const void *q, *gate, *k_cache, *v_cache;
  const int32_t *prefix_table, *page_table, *kv_lens, *cu_seqlens;
  void *o;
  float *lse;
};

constexpr int kSms = 152;          // persistent CTAs, and the shares that work is cut into
constexpr int kMostKeys = 0x7fffe000;  // that a row of an attention call may see
constexpr int kStepRows = 16;      // query heads per kv-head that the decode kernel takes
// Either attention call: picks the kernels and lays out the workspace (attn_tile.cu).
size_t attn_workspace(int num_seqs, int tokens, int hq, int hkv, int d, int prefix_len);
cudaError_t launch_attention(const AttnParams &p, void *ws, unsigned int *err, cudaStream_t stream);
// One token per sequence (attn_step.cu).
size_t attn_step_workspace(int d);
cudaError_t launch_attn_step(const AttnParams &p, void *ws, unsigned int *err, cudaStream_t stream);

// The library's device status word on the current device (gdn_api.cu), or NULL.
unsigned int *device_status_word();

// x <- x * sigmoid(gate), gate in bf16.
__device__ __forceinline__ float sigmoid(float g) {
  float e, r;  // 1 / (1 + 2^(-g log2 e)); 0 where the power overflows
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(1.f + e));
  return r;
}
__device__ __forceinline__ void gate4(float *x, const uint2 &g) {
  x[0] *= sigmoid(__uint_as_float(g.x << 16));
  x[1] *= sigmoid(__uint_as_float(g.x & 0xffff0000u));
  x[2] *= sigmoid(__uint_as_float(g.y << 16));
  x[3] *= sigmoid(__uint_as_float(g.y & 0xffff0000u));
}
__device__ __forceinline__ void gate8(float (&x)[8], const uint4 &g) {
  gate4(x, make_uint2(g.x, g.y));
  gate4(x + 4, make_uint2(g.z, g.w));
}

// Sequence that token t belongs to: the n with cu[n] <= t < cu[n + 1], by a warp that probes
// 32 places at a time (cu non-decreasing, cu[0] = 0; a malformed cu gives some n in range).
__device__ __forceinline__ int find_seq(const int32_t *cu, int num_seqs, int t, int lane) {
  int lo = 0, hi = num_seqs;  // cu[lo] <= t (taken), answer in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + (lane + 1) * step;
    const bool le = at < hi && cu[at] <= t;
    const int m = __popc(__ballot_sync(0xffffffffu, le));  // probes at or below t
    lo += m * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

}  // namespace gdn
