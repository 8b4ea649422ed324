// Attention of one token per sequence over the paged cache (attn_step.cuh).
#include "attn_step.cuh"

namespace gdn {
namespace {

template <int D>
__global__ void __launch_bounds__(StepCfg<D>::THREADS, D == 128 ? 2 : 1)
    step_kernel(AttnParams p, StepPlan w, const __grid_constant__ CUtensorMap qmap,
                const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ StepShared<D> sh;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  step_role<D>(p, w, qmap, kmap, vmap, smem, sh, (int)threadIdx.x, (int)blockIdx.x, (int)gridDim.x, 1, false);
}

template <int D>
cudaError_t run(const AttnParams &p, char *ws, unsigned int *errw, cudaStream_t stream) {
  using C = StepCfg<D>;
  StepPlan w;
  step_layout<D>(&w, ws);
  w.err = errw;
  CUtensorMap q, k, v;
  cudaError_t err = q_map(&q, p, 1);
  if (err == cudaSuccess) err = cache_maps(&k, &v, p, kTile);
  if (err != cudaSuccess) return err;
  const size_t smem = C::SMEM + 1024;
  static std::atomic<uint64_t> allowed{0};
  err = allow_smem(step_kernel<D>, smem, allowed);
  if (err != cudaSuccess) return err;
  return launch_dependent(step_kernel<D>, C::CTAS, C::THREADS, smem, stream, 1, p, w, q, k, v);
}

}  // namespace

size_t attn_step_workspace(int d) {
  return d == 128 ? step_layout<128>(nullptr, nullptr) : step_layout<256>(nullptr, nullptr);
}

cudaError_t launch_attn_step(const AttnParams &p, void *ws, unsigned int *err, cudaStream_t stream) {
  return p.d == 128 ? run<128>(p, static_cast<char *>(ws), err, stream)
                    : run<256>(p, static_cast<char *>(ws), err, stream);
}

}  // namespace gdn
