// C-ABI entry points of the beams' operators: host-side validation and launch.
// Declarations and the argument contract: include/gdn.h.
#include <cuda_runtime.h>

#include "beam.h"

namespace {

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
gdn_status cuda_status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

struct Range {
  const void *p;
  size_t bytes;
};
bool overlap(const Range &a, const Range &b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}

gdn_status check_shape(const gdn_beam_shape *s) {
  if (!s || s->num_groups < 0 || s->beams < 1 || s->vocab < 1 || s->top < 1 || s->top > s->vocab ||
      s->row_stride < s->vocab || s->pad_token < 0 || s->pad_token >= s->vocab)
    return GDN_ERR_INVALID_ARG;
  if (s->dtype != GDN_F32 && s->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (s->beams > 64 || s->top > 64 || s->vocab > 1 << 24) return GDN_ERR_UNSUPPORTED;
  // parts of rows, at most 4096 a request, are counted in 32 bits, logits' bytes in 63
  if (s->num_groups > 0x7fffffff / 4096 || s->row_stride > 1ll << 38) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

int parts(const gdn_beam_shape *s) {
  return gdn::beam_parts(s->num_groups, s->beams, s->vocab, s->dtype == GDN_BF16);
}
size_t lists(const gdn_beam_shape *s) {
  return gdn::beam_lists(s->num_groups, s->beams, s->vocab, s->dtype == GDN_BF16);
}
size_t sums_bytes(const gdn_beam_shape *s) {
  const size_t steps = ((size_t)s->vocab + gdn::kBeamStep - 1) / gdn::kBeamStep;
  return ((size_t)s->num_groups * s->beams * steps * sizeof(float2) + 255) / 256 * 256;
}

}  // namespace

extern "C" {

size_t gdn_beam_workspace_size(const gdn_beam_shape *shape) {
  if (check_shape(shape) != GDN_OK) return (size_t)-1;
  return sums_bytes(shape) + lists(shape) * shape->top * sizeof(uint64_t);
}

gdn_status gdn_beam_select(const gdn_beam_shape *shape, const void *logits, const float *scores,
                           const uint8_t *finished, float *scores_out, int32_t *parents,
                           int32_t *tokens, void *workspace, size_t workspace_bytes, void *stream) {
  const gdn_status st = check_shape(shape);
  if (st != GDN_OK) return st;
  const gdn_beam_shape *s = shape;
  if (s->num_groups == 0) return GDN_OK;
  if (!logits || !scores || !scores_out || !parents || !tokens) return GDN_ERR_INVALID_ARG;
  const size_t es = s->dtype == GDN_BF16 ? 2 : 4;
  if (!aligned(logits, (unsigned)es) || !aligned(scores, 4) || !aligned(scores_out, 4) || !aligned(parents, 4) ||
      !aligned(tokens, 4))
    return GDN_ERR_INVALID_ARG;
  const size_t rows = (size_t)s->num_groups * s->beams, need = gdn_beam_workspace_size(s);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return GDN_ERR_WORKSPACE;
  const size_t out = (size_t)s->num_groups * s->top * 4;
  const Range all[] = {{scores_out, out}, {parents, out}, {tokens, out}, {workspace, need},
                       {logits, ((rows - 1) * (size_t)s->row_stride + s->vocab) * es}, {scores, rows * 4}, {finished, rows}};
  for (int i = 0; i < 4; ++i)  // what is written
    for (int j = i + 1; j < 7; ++j)
      if (overlap(all[i], all[j])) return GDN_ERR_ALIAS;
  gdn::BeamParams p{};
  p.groups = s->num_groups;
  p.beams = s->beams;
  p.vocab = s->vocab;
  p.top = s->top;
  p.pad_token = s->pad_token;
  p.parts = parts(s);
  p.row_stride = s->row_stride;
  p.logits = logits;
  p.scores = scores;
  p.finished = finished;
  p.scores_out = scores_out;
  p.parents = parents;
  p.tokens = tokens;
  p.sums = static_cast<float2 *>(workspace);
  p.keys = reinterpret_cast<uint64_t *>(static_cast<char *>(workspace) + sums_bytes(s));
  return cuda_status(gdn::launch_beam_select(p, s->dtype, static_cast<cudaStream_t>(stream)));
}

gdn_status gdn_beam_reorder(int32_t num_layers, int32_t num_groups, int32_t beams,
                            int64_t row_bytes, const int32_t *parents, void *rows, void *stream) {
  if (num_layers < 0 || num_groups < 0 || beams < 1 || row_bytes < 0 || row_bytes % 4) return GDN_ERR_INVALID_ARG;
  if (beams > 64 || row_bytes > 1ll << 38) return GDN_ERR_UNSUPPORTED;
  // a grid in one dimension
  const long long items = (long long)num_layers * num_groups;
  if (items > 0x7fffffffLL || items * ((row_bytes + gdn::kReorderBytes - 1) / gdn::kReorderBytes) > 0x7fffffffLL)
    return GDN_ERR_UNSUPPORTED;
  if (items == 0 || row_bytes == 0) return GDN_OK;
  if (!parents || !rows || !aligned(parents, 4) || !aligned(rows, 4)) return GDN_ERR_INVALID_ARG;
  if (overlap({rows, (size_t)items * beams * row_bytes}, {parents, (size_t)num_groups * beams * 4})) return GDN_ERR_ALIAS;
  gdn::ReorderParams p{};
  p.layers = num_layers;
  p.groups = num_groups;
  p.beams = beams;
  p.row_bytes = row_bytes;
  p.parents = parents;
  p.rows = rows;
  return cuda_status(gdn::launch_beam_reorder(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
