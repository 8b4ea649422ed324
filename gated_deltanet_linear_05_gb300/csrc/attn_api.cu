// C-ABI entry points of the attention-layer operators: host-side validation and launch.
// Declarations and the argument contract: include/gdn.h.
#include <cuda_runtime.h>
#include <math.h>

#include "attn.h"

namespace {

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
gdn_status cuda_status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

// Bytes from the first to past the last element of a [tokens, heads, D] bf16 tensor.
size_t extent(const gdn_attn_shape *s, const int64_t (&st)[2], int heads) {
  if (s->total_tokens == 0) return 0;
  return 2 * ((size_t)(s->total_tokens - 1) * st[0] + (size_t)(heads - 1) * st[1] + s->head_dim);
}
bool overlap(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na && nb && x < y + nb && y < x + na;
}

gdn_status check_stride(const int64_t (&st)[2], int d) {
  if (st[0] < d || st[1] < d || (st[0] & 7) || (st[1] & 7)) return GDN_ERR_INVALID_ARG;
  // what a tensor map can hold: 40-bit byte strides
  if (st[0] > (1ll << 38) || st[1] > (1ll << 38)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

gdn_status check_shape(const gdn_attn_shape *s) {
  if (!s) return GDN_ERR_INVALID_ARG;
  if (s->num_seqs < 0 || s->total_tokens < 0 || s->num_q_heads <= 0 || s->num_kv_heads <= 0 ||
      s->num_pages < 0 || s->max_pages < 0 || s->prefix_len < 0)
    return GDN_ERR_INVALID_ARG;
  if (s->num_q_heads % s->num_kv_heads != 0) return GDN_ERR_INVALID_ARG;
  if (s->head_dim != 128 && s->head_dim != 256) return GDN_ERR_UNSUPPORTED;
  if (s->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (s->num_q_heads / s->num_kv_heads > 128 || s->num_q_heads > 65535) return GDN_ERR_UNSUPPORTED;
  // tables of tiles, at most one a token and one a sequence with some hundred parts beside them, and
  // rows and (sequence, head) pairs are counted in 32 bits
  if ((long long)s->num_seqs + s->total_tokens > 0x7fffffffLL - 4096) return GDN_ERR_UNSUPPORTED;
  if ((long long)s->total_tokens * s->num_q_heads > 0x7fffffffLL ||
      (long long)s->num_seqs * s->num_q_heads > 0x7fffffffLL)
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// The paged cache's part of a shape.
gdn_status check_cache(const gdn_attn_shape *s) {
  if (s->page_size != 16 && s->page_size != 32 && s->page_size != 64 && s->page_size != 128)
    return GDN_ERR_UNSUPPORTED;
  if (s->page_stride < (int64_t)s->num_kv_heads * s->page_size * s->head_dim || (s->page_stride & 7))
    return GDN_ERR_INVALID_ARG;
  if (s->page_stride > (1ll << 38)) return GDN_ERR_UNSUPPORTED;
  // keys of a sequence and positions are counted in 32 bits
  if ((long long)s->max_pages * s->page_size + s->prefix_len > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

gdn_status check_tables(const gdn_attn_shape *s, const void *k_cache, const void *v_cache,
                        const int32_t *page_table, const int32_t *kv_lens, const int32_t *cu) {
  if (!cu && s->total_tokens != s->num_seqs) return GDN_ERR_INVALID_ARG;
  if (s->total_tokens > 0 && s->num_seqs == 0) return GDN_ERR_INVALID_ARG;
  if (s->num_seqs > 0 && (!kv_lens || (!page_table && s->max_pages > 0))) return GDN_ERR_INVALID_ARG;
  if (!aligned(kv_lens, 4) || !aligned(page_table, 4) || !aligned(cu, 4)) return GDN_ERR_INVALID_ARG;
  if (s->num_pages > 0 && (!k_cache || !v_cache)) return GDN_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

gdn_status attention(const gdn_attn_shape *s, const void *q, const void *gate, const void *k_cache,
                     const void *v_cache, const int32_t *prefix_table, const int32_t *page_table,
                     const int32_t *kv_lens, const int32_t *cu_seqlens, const int32_t *parents, void *o,
                     float *lse, void *workspace, size_t workspace_bytes, void *stream) {
  gdn_status st = check_cache(s);
  if (st != GDN_OK) return st;
  // key tiles are counted, and boxes of them addressed, up to some thousand keys past the last in 32 bits
  if ((long long)s->max_pages * s->page_size + s->prefix_len > gdn::kMostKeys) return GDN_ERR_UNSUPPORTED;
  if (!isfinite(s->scale * 1.4426950408889634f)) return GDN_ERR_INVALID_ARG;
  if ((st = check_stride(s->q_stride, s->head_dim)) != GDN_OK) return st;
  if (gate && (st = check_stride(s->gate_stride, s->head_dim)) != GDN_OK) return st;
  if ((st = check_tables(s, k_cache, v_cache, page_table, kv_lens, cu_seqlens)) != GDN_OK) return st;
  if (s->prefix_len > 0 && (!prefix_table || !aligned(prefix_table, 4) || s->num_pages == 0))
    return GDN_ERR_INVALID_ARG;
  if (s->total_tokens > 0 && (!q || !o)) return GDN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(gate, 16) || !aligned(o, 16) || !aligned(lse, 4))
    return GDN_ERR_INVALID_ARG;
  const size_t ob = (size_t)s->total_tokens * s->num_q_heads * s->head_dim * 2;
  if (overlap(o, ob, q, extent(s, s->q_stride, s->num_q_heads)) ||
      (gate && overlap(o, ob, gate, extent(s, s->gate_stride, s->num_q_heads))))
    return GDN_ERR_ALIAS;
  const size_t need = gdn_attn_workspace_size(s);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return GDN_ERR_WORKSPACE;
  if (s->total_tokens == 0) return GDN_OK;
  gdn::AttnParams p{};
  p.num_seqs = s->num_seqs;
  p.tokens = s->total_tokens;
  p.hq = s->num_q_heads;
  p.hkv = s->num_kv_heads;
  p.d = s->head_dim;
  p.page_size = s->page_size;
  p.num_pages = s->num_pages;
  p.max_pages = s->num_pages > 0 ? s->max_pages : 0;  // no page: no key
  p.prefix_len = s->prefix_len;
  // The kernels multiply by scale * log2(e) with subnormals flushed: one would turn a masked -inf into
  // NaN.  Below the normal range a scale counts as 0 (it would take a score of 2^100 to see it).
  p.scale = fabsf(s->scale) < 1.17549435e-38f ? 0.f : s->scale;
  for (int i = 0; i < 2; ++i) p.qs[i] = s->q_stride[i], p.gs[i] = s->gate_stride[i];
  p.page_stride = s->page_stride;
  p.q = q;
  p.gate = gate;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.prefix_table = prefix_table;
  p.page_table = page_table;
  p.kv_lens = kv_lens;
  p.cu_seqlens = cu_seqlens;
  p.parents = parents;
  p.o = o;
  p.lse = lse;
  return cuda_status(gdn::launch_attention(p, workspace, gdn::device_status_word(),
                                           static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t gdn_attn_workspace_size(const gdn_attn_shape *shape) {
  if (check_shape(shape) != GDN_OK) return (size_t)-1;
  return gdn::attn_workspace(shape->num_seqs, shape->total_tokens, shape->num_q_heads,
                             shape->num_kv_heads, shape->head_dim, shape->prefix_len);
}

gdn_status gdn_paged_attention(const gdn_attn_shape *shape, const void *q, const void *gate,
                               const void *k_cache, const void *v_cache,
                               const int32_t *page_table, const int32_t *kv_lens,
                               const int32_t *cu_seqlens, void *o, float *lse, void *workspace,
                               size_t workspace_bytes, void *stream) {
  const gdn_status st = check_shape(shape);
  if (st != GDN_OK) return st;
  if (shape->prefix_len != 0) return GDN_ERR_INVALID_ARG;
  return attention(shape, q, gate, k_cache, v_cache, nullptr, page_table, kv_lens, cu_seqlens, nullptr, o,
                   lse, workspace, workspace_bytes, stream);
}

gdn_status gdn_shared_prefix_attention(const gdn_attn_shape *shape, const void *q,
                                       const void *gate, const void *k_cache,
                                       const void *v_cache, const int32_t *prefix_table,
                                       const int32_t *page_table, const int32_t *kv_lens,
                                       const int32_t *cu_seqlens, void *o, float *lse,
                                       void *workspace, size_t workspace_bytes, void *stream) {
  const gdn_status st = check_shape(shape);
  if (st != GDN_OK) return st;
  if (shape->prefix_len == 0) return GDN_ERR_INVALID_ARG;
  return attention(shape, q, gate, k_cache, v_cache, prefix_table, page_table, kv_lens, cu_seqlens, nullptr,
                   o, lse, workspace, workspace_bytes, stream);
}

gdn_status gdn_tree_attention(const gdn_attn_shape *shape, const void *q, const void *gate,
                              const void *k_cache, const void *v_cache,
                              const int32_t *prefix_table, const int32_t *page_table,
                              const int32_t *kv_lens, const int32_t *cu_seqlens,
                              const int32_t *parents, void *o, float *lse, void *workspace,
                              size_t workspace_bytes, void *stream) {
  const gdn_status st = check_shape(shape);
  if (st != GDN_OK) return st;
  if (!cu_seqlens || !aligned(parents, 4) || (shape->total_tokens > 0 && !parents)) return GDN_ERR_INVALID_ARG;
  return attention(shape, q, gate, k_cache, v_cache, prefix_table, page_table, kv_lens, cu_seqlens, parents,
                   o, lse, workspace, workspace_bytes, stream);
}

gdn_status gdn_kv_append(const gdn_attn_shape *s, const void *q, const void *k, const void *v,
                         const float *q_norm, const float *k_norm, float eps,
                         const double *inv_freq, const int32_t *rope_axis,
                         const int32_t *positions, const int32_t *page_table,
                         const int32_t *kv_lens, const int32_t *cu_seqlens, void *q_out,
                         void *k_cache, void *v_cache, void *stream) {
  gdn_status st = check_shape(s);
  if (st == GDN_OK) st = check_cache(s);
  if (st != GDN_OK) return st;
  if (s->rotary_dim < 0 || s->rotary_dim > s->head_dim || s->rotary_dim % 16 != 0 || s->num_axes < 1 ||
      s->num_axes > 8)
    return GDN_ERR_INVALID_ARG;
  if ((st = check_stride(s->q_stride, s->head_dim)) != GDN_OK ||
      (st = check_stride(s->k_stride, s->head_dim)) != GDN_OK ||
      (st = check_stride(s->v_stride, s->head_dim)) != GDN_OK)
    return st;
  if ((st = check_tables(s, k_cache, v_cache, page_table, kv_lens, cu_seqlens)) != GDN_OK) return st;
  if (!(eps >= 0.f) || isinf(eps)) return GDN_ERR_INVALID_ARG;
  if (s->total_tokens > 0 && (!q || !k || !v || !q_out || (s->rotary_dim > 0 && !inv_freq)))
    return GDN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) ||
      !aligned(q_norm, 16) || !aligned(k_norm, 16) || !aligned(inv_freq, 8) || !aligned(rope_axis, 4) ||
      !aligned(positions, 4))
    return GDN_ERR_INVALID_ARG;
  const size_t row = (size_t)s->num_q_heads * s->head_dim;
  const size_t qb = (size_t)s->total_tokens * row * 2;
  const bool same = q_out == q && s->q_stride[0] == (int64_t)row && s->q_stride[1] == s->head_dim;
  if ((!same && overlap(q_out, qb, q, extent(s, s->q_stride, s->num_q_heads))) ||
      overlap(q_out, qb, k, extent(s, s->k_stride, s->num_kv_heads)) ||
      overlap(q_out, qb, v, extent(s, s->v_stride, s->num_kv_heads)))
    return GDN_ERR_ALIAS;
  if (s->total_tokens == 0) return GDN_OK;
  gdn::AppendParams p{};
  p.num_seqs = s->num_seqs;
  p.tokens = s->total_tokens;
  p.hq = s->num_q_heads;
  p.hkv = s->num_kv_heads;
  p.d = s->head_dim;
  p.page_size = s->page_size;
  p.num_pages = s->num_pages;
  p.max_pages = s->max_pages;
  p.rot = s->rotary_dim;
  p.axes = s->num_axes;
  p.pos0 = s->prefix_len;
  p.eps = eps;
  for (int i = 0; i < 2; ++i)
    p.qs[i] = s->q_stride[i], p.ks[i] = s->k_stride[i], p.vs[i] = s->v_stride[i];
  p.page_stride = s->page_stride;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_norm = q_norm;
  p.k_norm = k_norm;
  p.inv_freq = inv_freq;
  p.rope_axis = rope_axis;
  p.positions = positions;
  p.page_table = page_table;
  p.kv_lens = kv_lens;
  p.cu_seqlens = cu_seqlens;
  p.q_out = q_out;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  return cuda_status(gdn::launch_kv_append(p, static_cast<cudaStream_t>(stream)));
}

gdn_status gdn_add_rmsnorm(int64_t rows, int32_t cols, gdn_dtype dtype, const void *x,
                           const void *residual, const float *weight, float eps,
                           void *residual_out, void *y, float *scale, int32_t group,
                           void *stream) {
  if (rows < 0 || cols <= 0) return GDN_ERR_INVALID_ARG;
  if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (group != 0 && group != 128) return GDN_ERR_UNSUPPORTED;
  if (group != 0 && !scale) return GDN_ERR_INVALID_ARG;
  if (cols % 8 != 0 || (group && cols % group != 0) || cols > 65536 || rows > 0x7fffffffLL)
    return GDN_ERR_UNSUPPORTED;
  if (!(eps >= 0.f) || isinf(eps)) return GDN_ERR_INVALID_ARG;
  if (rows > 0 && (!x || !weight || !y || (residual && !residual_out))) return GDN_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(residual_out, 16) ||
      !aligned(y, 16) || !aligned(scale, 4))
    return GDN_ERR_INVALID_ARG;
  const size_t nb = (size_t)rows * cols * (dtype == GDN_BF16 ? 2 : 4);
  const size_t yb = scale ? (size_t)rows * cols : nb;
  const size_t sb = scale ? (size_t)rows * (group ? cols / group : 1) * 4 : 0;
  if ((residual_out != x && overlap(residual_out, nb, x, nb)) ||
      (residual_out != residual && overlap(residual_out, nb, residual, nb)) ||
      (!(y == x && !scale) && overlap(y, yb, x, nb)) || overlap(y, yb, residual, nb) ||
      overlap(y, yb, residual_out, nb) || overlap(scale, sb, x, nb) || overlap(scale, sb, residual, nb) ||
      overlap(scale, sb, residual_out, nb) || overlap(scale, sb, y, yb))
    return GDN_ERR_ALIAS;
  if (rows == 0) return GDN_OK;
  gdn::AddNormParams p{};
  p.rows = rows;
  p.cols = cols;
  p.group = group;
  p.eps = eps;
  p.x = x;
  p.residual = residual;
  p.weight = weight;
  p.residual_out = residual_out;
  p.y = y;
  p.scale = scale;
  return cuda_status(gdn::launch_add_rmsnorm(p, dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
