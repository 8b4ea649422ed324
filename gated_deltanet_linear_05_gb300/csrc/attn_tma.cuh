// What the attention kernels share: bounded waits, TMA loads and tensor maps of the paged
// cache, the output of a row, launches.
#pragma once

#include <cuda.h>
#include <math_constants.h>
#include <string.h>

#include <atomic>

#include "attn.h"
#include "common.cuh"

namespace gdn {

constexpr float kLn2 = 0.6931471805599453f;
// Counters at the start of an attention workspace: zero before the first call and after
// every one, at the same place for all shapes.
constexpr size_t kArrivedBytes = GDN_ATTN_COUNTER_BYTES;

__host__ __device__ inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

__device__ __forceinline__ bool try_bar(uint64_t *bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
// Bounded wait that remembers a lost signal: after the first time-out of a CTA every later
// wait returns soon, so the kernel ends.
__device__ __forceinline__ void wait_slow(uint64_t *bar, uint32_t parity, volatile int *dead,
                                          unsigned int *err) {
  for (int it = 0; it < (1 << 20); ++it) {
    if (try_bar(bar, parity)) return;
    if ((it & 255) == 255 && *dead) return;
  }
  *dead = 1;
  report_status(err, GDN_STATUS_WAIT_TIMEOUT);
}
__device__ __forceinline__ void wait_bar(uint64_t *bar, uint32_t parity, volatile int *dead,
                                         unsigned int *err) {
  if (!try_bar(bar, parity)) wait_slow(bar, parity, dead, err);
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
// A value that all lanes hold, known to the compiler as such (uniform registers).
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ void tma_4d(void *dst, const void *map, int x, int y, int z, int w,
                                       uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3, %4, %5}], [%6];\n" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void prefetch_map(const void *map) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}

// A row's maximum m (base 2) and sum of powers l.  m is -inf only while the row has seen no key: one
// that has, of scores that are all -inf (l = 0) or NaN (l = NaN), gets the lowest finite m.  So
// "no key" (0, as the contract says) and 0 / 0 or NaN (which must not pass for it) stay apart, and a
// row's result does not depend on how its keys were cut.
__device__ __forceinline__ float seen_max(float m, bool saw_key) {
  return m == -CUDART_INF_F && saw_key ? -3.402823466e38f : m;
}
__device__ __forceinline__ float row_inverse(float m, float l) {
  return l != 0.f ? 1.f / l : m == -CUDART_INF_F ? 0.f : CUDART_NAN_F;
}
__device__ __forceinline__ float row_lse(float m, float l) {
  return l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * kLn2;
}

// A row (token, head) of the output by one warp: lane l has columns 128 k + 4 l .. + 3 of the
// sum O (v[4 k ..]) with the maximum m (base 2) and the sum l.
template <int D>
__device__ __forceinline__ void emit_row(const AttnParams &p, int tok, int head, int lane, float m, float l,
                                         const float (&v)[D / 32]) {
  const long long row = (long long)tok * p.hq + head;
  const float inv = row_inverse(m, l);
#pragma unroll
  for (int k = 0; k < D / 128; ++k) {
    float x[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = v[4 * k + q] * inv;
    if (p.gate)
      gate4(x, *reinterpret_cast<const uint2 *>((const __nv_bfloat16 *)p.gate + tok * p.gs[0] + head * p.gs[1] +
                                                lane * 4 + 128 * k));
    *reinterpret_cast<uint2 *>((__nv_bfloat16 *)p.o + row * D + lane * 4 + 128 * k) =
        make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
  }
  if (p.lse && lane == 0) p.lse[row] = row_lse(m, l);
}

// Partial results of a shared prefix, left by the tile kernel for every row of the call: tile t of
// 2 tpt tokens has `parts` parts, part q of kv-head h in slot (t parts + q) Hkv + h, a slot 256
// rows of {m, l} and D sums, row (token / tpt) 128 + (token % tpt) G + g of the tile's tokens.
struct PrefixParts {
  const float *ml, *part;
  const int *head;  // not NULL: the number of parts is head[2], chosen on the device
  int parts, tpt;
};
constexpr int kTileRows = 256;
// One result {m, l}, D sums per row of the call, left for a join.
struct DenseRows {
  float *ml, *part;
};

// Adds `count` parts of a row, at `at`, `at` + pitch, ..., to (m, l, acc) by one warp:
//     M = max(m, max m_q),  l = sum 2^(m_q - M) l_q,  acc = sum 2^(m_q - M) O_q
// (m_q = -inf: no key, weight 0; a NaN in l_q reaches l whatever its weight).
// The statistics first, a part a lane, so that the sums' loads do not wait for one another
// (AHEAD of them at a time; 8 for the decode kernel's one CTA, 30 us for 32, two contexts of 30k; the
// join's many warps are slower with 8).
template <int D, int AHEAD = 4>
__device__ __forceinline__ void add_parts(float &m, float &l, float (&acc)[D / 32], const float *ml_of,
                                          const float *part_of, long long at, long long pitch, int count, int lane) {
  for (int q0 = 0; q0 < count; q0 += 32) {
    float2 ml = make_float2(-CUDART_INF_F, 0.f);
    if (q0 + lane < count) ml = __ldcg(reinterpret_cast<const float2 *>(ml_of + 2 * (at + (q0 + lane) * pitch)));
    float top = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top == -CUDART_INF_F) continue;
    const float m1 = fmaxf(m, top), a = ex2(m - m1), weight = ex2(ml.x - m1);
    m = m1;
    l = l * a + warp_sum(ml.y * weight);
#pragma unroll
    for (int k = 0; k < D / 32; ++k) acc[k] *= a;
    const int some = min(32, count - q0);
#pragma unroll (AHEAD)
    for (int q = 0; q < some; ++q) {  // (a part without keys holds zeros: its weight is 0)
      const float b = __shfl_sync(0xffffffffu, weight, q);
      const float *o = part_of + (at + (q0 + q) * pitch) * D + lane * 4;
#pragma unroll
      for (int k = 0; k < D / 128; ++k) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(o + 128 * k));
        acc[4 * k] = fmaf(v.x, b, acc[4 * k]);
        acc[4 * k + 1] = fmaf(v.y, b, acc[4 * k + 1]);
        acc[4 * k + 2] = fmaf(v.z, b, acc[4 * k + 2]);
        acc[4 * k + 3] = fmaf(v.w, b, acc[4 * k + 3]);
      }
    }
  }
}
// The prefix's parts of (token, head h G + g).
template <int D>
__device__ __forceinline__ void add_prefix(float &m, float &l, float (&acc)[D / 32], const PrefixParts &pre,
                                           int tok, int h, int g, int G, int hkv, int lane) {
  const int parts = pre.head ? pre.head[2] : pre.parts;
  if (parts == 0) return;
  const int tt = 2 * pre.tpt, off = tok % tt;
  const long long at =
      ((long long)(tok / tt) * parts * hkv + h) * kTileRows + off / pre.tpt * 128 + (off % pre.tpt) * G + g;
  add_parts<D>(m, l, acc, pre.ml, pre.part, at, (long long)hkv * kTileRows, parts, lane);
}

// Tensor map of a bf16 tensor with 128-byte swizzle (boxes of 64 columns).
cudaError_t bf16_map(CUtensorMap *map, const void *x, int rank, const cuuint64_t *dims,
                     const cuuint64_t *strides, const cuuint32_t *box);
// Map of q for boxes of `tokens` tokens x one kv-head's query heads x 64 columns.
cudaError_t q_map(CUtensorMap *map, const AttnParams &p, int tokens);
// Maps of K and V, [page][head][row][column], for boxes of min(page_size, tile) rows; zero
// (and never used) for a cache without pages.
cudaError_t cache_maps(CUtensorMap *k, CUtensorMap *v, const AttnParams &p, int tile);

// Allows `kernel` its dynamic shared memory, once per device (`done`: a bit per device).
template <typename... Args>
cudaError_t allow_smem(void (*kernel)(Args...), size_t smem, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return err;
}

// Launch, in clusters of `cluster` CTAs, as a programmatic dependent of the work before it on
// the stream.
template <typename... Args>
cudaError_t launch_dependent(void (*kernel)(Args...), unsigned grid, unsigned threads, size_t smem,
                             cudaStream_t stream, int cluster, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace gdn
