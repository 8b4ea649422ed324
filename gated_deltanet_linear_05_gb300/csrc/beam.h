// Internal launch interface of the beams' operators (beam.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

struct BeamParams {
  int groups, beams, vocab, top, pad_token, parts, steps;  // steps: set by the launch
  long long row_stride;
  const void *logits;
  const float *scores;
  const uint8_t *finished;
  float *scores_out;
  int32_t *parents, *tokens;
  float2 *sums;    // [row][step] maximum and sum of powers
  uint64_t *keys;  // [row][part][top] the best logits
};
constexpr int kBeamStep = 4096;  // tokens of a step at least
int beam_parts(int groups, int beams, int vocab, bool bf16);
// (row, part) lists at most, which more requests, beams or vocabulary never make fewer
size_t beam_lists(int groups, int beams, int vocab, bool bf16);
cudaError_t launch_beam_select(const BeamParams &p, gdn_dtype dtype, cudaStream_t stream);

struct ReorderParams {
  int layers, groups, beams;
  long long row_bytes, blocks;
  const int32_t *parents;
  void *rows;
};
constexpr int kReorderBytes = 128 * 4;  // of a row to a CTA, at least
cudaError_t launch_beam_reorder(const ReorderParams &p, cudaStream_t stream);

}  // namespace gdn
