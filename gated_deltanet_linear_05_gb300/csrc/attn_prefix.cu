// One token per sequence behind a shared prefix: the prefix's tiles, bound by the tensor cores,
// and the sequences' own keys, bound by HBM, side by side in one launch.  Every CTA sees the lengths
// and comes to the same division of the SMs, so that both kinds of work end about together:
//     X : 152 - X  as  (row tiles x key tiles x cycles of a step) : (own bytes / 36 bytes a cycle),
// 2450 cycles a step of a CTA (4154 of a pair's two) as measured in long prompts; 36 bytes a cycle is
// about what an SM streams when not all of them do (from one shape, 128 requests of up to 1000 own keys behind 16389:
// 99 us with 48, 86 with 40 and 32, 89 with 26; 104 with the two one after the other).  A row tile is
// cut into as many parts as fill the X.
#include "attn_step.cuh"
#include "attn_tile.cuh"

namespace gdn {
namespace {

template <int D>
struct PrefixCfg {
  static constexpr int WORKERS = D == 128 ? 2 : 1;  // decode workers of a CTA
  static constexpr int WORKER_BYTES = (StepCfg<D>::SMEM + (int)sizeof(StepShared<D>) + 1023) / 1024 * 1024;
  static constexpr int SMEM = Cfg<D>::SMEM > WORKERS * WORKER_BYTES ? Cfg<D>::SMEM : WORKERS * WORKER_BYTES;
  static_assert(WORKERS * StepCfg<D>::THREADS <= Cfg<D>::WIDE, "threads");
  static_assert(SMEM + 1024 + 1024 <= 232448, "shared memory");
};

template <int D>
__global__ void __launch_bounds__(Cfg<D>::WIDE, 1)
    prefix_kernel(AttnParams p, TilePlan pre, StepPlan w, const __grid_constant__ CUtensorMap tile_q,
                  const __grid_constant__ CUtensorMap tile_k, const __grid_constant__ CUtensorMap tile_v,
                  const __grid_constant__ CUtensorMap step_q, const __grid_constant__ CUtensorMap step_k,
                  const __grid_constant__ CUtensorMap step_v) {
  using C = Cfg<D>;
  using P = PrefixCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Barriers bars;
  __shared__ float sh_sum[C::WIDE / 32];
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  float sum = 0.f;
  for (int n = tid; n < p.num_seqs; n += C::WIDE) sum += tiles_of(seq_len(p, n));
  sum = warp_sum(sum);
  if ((tid & 31) == 0) sh_sum[tid >> 5] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < C::WIDE / 32; ++i) sum += sh_sum[i];  // in the same order everywhere
  const int tt = 2 * (128 / (p.hq / p.hkv));
  const int items = (p.tokens + tt - 1) / tt * p.hkv;
  const float a = (float)items * pre.uniform_kt * (D == 128 ? 2450.f : 4154.f);
  const float b = sum * p.hkv * (kTile * D * 4.f / 36.f);
  const float want = C::UNITS * a / (a + b);
  int parts = min(pre.uniform_parts, max(1, (int)(want / items + 0.5f)));
  while (parts > 1 && items * parts > C::UNITS - 1) --parts;
  const int units = items * parts <= min(C::UNITS - 1, (int)(want * 1.5f)) ? items * parts
                                                                         : max(1, min(C::UNITS - 1, (int)(want + 0.5f)));
  if (blockIdx.x == 0 && tid == 0) pre.head[2] = parts;
  const int unit = (int)blockIdx.x / C::GRP;
  if (unit < units) {
    pre.uniform_parts = parts;
    tile_role<C, 8>(p, pre, tile_q, tile_k, tile_v, smem_raw, bars, unit, units, true);
    return;
  }
  const int v = tid / StepCfg<D>::THREADS;
  if (v >= P::WORKERS) return;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023) +
                  v * P::WORKER_BYTES;
  step_role<D>(p, w, step_q, step_k, step_v, smem, *reinterpret_cast<StepShared<D> *>(smem + StepCfg<D>::SMEM),
               tid - v * StepCfg<D>::THREADS, ((int)blockIdx.x - units * C::GRP) * P::WORKERS + v,
               (kSms - units * C::GRP) * P::WORKERS, 1 + 2 * v, true);
}

template <int D>
cudaError_t run(const AttnParams &p, char *ws, const TilePlan &pre, const DenseRows &dense, unsigned int *err_word,
                cudaStream_t stream) {
  using C = Cfg<D>;
  StepPlan w;
  step_layout<D>(&w, ws);
  w.dense = dense;
  w.err = err_word;
  CUtensorMap m[6];
  cudaError_t err = q_map(&m[0], p, 128 / (p.hq / p.hkv));
  if (err == cudaSuccess) err = cache_maps(&m[1], &m[2], p, C::KROWS);
  if (err == cudaSuccess) err = q_map(&m[3], p, 1);
  if (err == cudaSuccess) err = cache_maps(&m[4], &m[5], p, kTile);
  if (err != cudaSuccess) return err;
  const size_t smem = PrefixCfg<D>::SMEM + 1024;
  static std::atomic<uint64_t> allowed{0};
  err = allow_smem(prefix_kernel<D>, smem, allowed);
  if (err != cudaSuccess) return err;
  return launch_dependent(prefix_kernel<D>, kSms, C::WIDE, smem, stream, C::GRP, p, pre, w, m[0], m[1], m[2], m[3],
                          m[4], m[5]);
}

}  // namespace

cudaError_t launch_attn_prefix(const AttnParams &p, void *ws, const TilePlan &pre, const DenseRows &dense,
                               unsigned int *err, cudaStream_t stream) {
  return p.d == 128 ? run<128>(p, static_cast<char *>(ws), pre, dense, err, stream)
                    : run<256>(p, static_cast<char *>(ws), pre, dense, err, stream);
}

}  // namespace gdn
