// The attention layer's steps around its products: rotary positions + append to the paged
// cache, and the residual addition + RMS norm.  Both move each byte once and are bound by
// HBM, or at a few rows by the latency of a launch and of a chain of loads.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "attn.h"
#include "attn_tma.cuh"
#include "common.cuh"

namespace gdn {
namespace {

// Eight consecutive elements as floats.
__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}

// ------------------------------------------------------------------ append

// f / (2 pi) as a binary fraction of a turn, modulo 1, in 64 bits: f = m 2^e exactly (m < 2^53),
// 2^64 / (2 pi) = C, so the fraction is the low 64 bits of (m C) 2^e.  Integer arithmetic:
// the 64-bit floating units of this GPU are too slow for it, and 32-bit floats lose the
// angle (pos * f at pos = 10^6 has an error of 0.06 rad).
__device__ __forceinline__ uint64_t turn_fraction(double f) {
  constexpr uint64_t C = 0x28BE60DB9391054Aull;
  const uint64_t b = (uint64_t)__double_as_longlong(f);
  const int ex = (int)((b >> 52) & 0x7ff);
  const uint64_t m = (b & 0xfffffffffffffull) | (ex ? 1ull << 52 : 0);
  const int e = (ex ? ex : 1) - 1075;
  const uint64_t lo = m * C, hi = __umul64hi(m, C);
  uint64_t r;
  if (e >= 0) r = e < 64 ? lo << e : 0;
  else if (e > -64) r = (lo >> -e) | (hi << (64 + e));
  else r = e > -128 ? hi >> (-e - 64) : 0;
  return (b >> 63) ? 0 - r : r;
}

constexpr int kAppendWarps = 4;
constexpr int kAppendRows = 6;  // rows that a lane group has in flight (4: 83 us for packed prompts, 6: 76)

// A warp takes one token's head rows (or, with few tokens, `share` warps a token), a row in D / 8
// lanes of 8 elements.  The turns per position of a lane's frequencies are kept over the warp's
// tokens, cosines and sines over a token's rows; rows come kAppendRows at a time, so that
// loads are in flight while the ones before are rotated.  The rotation's other half reaches a
// lane as the raw bf16 words of the lane that has it.  Sine and cosine by the fast
// instructions on an angle already reduced to half a turn: 2^-21 absolute, against 2^-9 of bf16.
// Bound by HBM: packed prompts of 33k tokens, 48 head rows of 128: 75 us, 5.7 TB/s (84% of the copy
// rate); a decode step of 32 tokens by its chain of loads (length, page, row), about 4 us.
template <int D, bool NORM>
__global__ void __launch_bounds__(32 * kAppendWarps, 4) append_kernel(AppendParams p, int share) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, U = kAppendRows;
  const int lane = threadIdx.x & 31;
  const int part = (int)((blockIdx.x * kAppendWarps + (threadIdx.x >> 5)) % share);
  const int tokens_at_once = (int)(gridDim.x * kAppendWarps / share);
  const int col = (lane % LPR) * 8;
  const int half = p.rot >> 1;
  const bool rot = col < p.rot, low = col < half;
  const int f0 = rot ? (low ? col : col - half) : 0;  // first frequency of this lane's eight
  const int peer = (lane & ~(LPR - 1)) + ((low ? lane + half / 8 : lane - half / 8) & (LPR - 1));
  const int rows = p.hq + 2 * p.hkv;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  uint64_t turn[8];
  int axis[8];
  if (rot) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      turn[i] = turn_fraction(p.inv_freq[f0 + i]);
      axis[i] = p.rope_axis ? min(max(p.rope_axis[f0 + i], 0), p.axes - 1) : 0;
    }
  }
  for (int tok = (int)((blockIdx.x * kAppendWarps + (threadIdx.x >> 5)) / share); tok < p.tokens;
       tok += tokens_at_once) {
    const __nv_bfloat16 *q = (const __nv_bfloat16 *)p.q + tok * p.qs[0] + col;
    const __nv_bfloat16 *k = (const __nv_bfloat16 *)p.k + tok * p.ks[0] + col;
    const __nv_bfloat16 *v = (const __nv_bfloat16 *)p.v + tok * p.vs[0] + col;
    uint4 u[U];
    auto fetch = [&](int r0) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int r = r0 + i * share * RPW + lane / LPR;
        const __nv_bfloat16 *src = r < p.hq ? q + r * p.qs[1] : r < p.hq + p.hkv ? k + (r - p.hq) * p.ks[1]
                                                                                 : v + (r - p.hq - p.hkv) * p.vs[1];
        u[i] = r < rows ? *(const uint4 *)src : make_uint4(0, 0, 0, 0);
      }
    };
    fetch(part * RPW);
    // the token's place
    int n = tok, back = 1;  // back: tokens from this one to the sequence's end
    if (p.cu_seqlens) {
      n = find_seq(p.cu_seqlens, p.num_seqs, tok, lane);
      int bos, eos;
      seq_range(p.cu_seqlens, n, p.tokens, bos, eos);
      back = eos - tok;
    }
    const long long cap = (long long)p.max_pages * p.page_size;
    const int len = (int)min(max((long long)p.kv_lens[n], 0ll), cap);
    const int place = len - back;
    long long dst = -1;  // element offset of the token's rows of head 0
    if (place >= 0 && back > 0) {
      const int lps = 31 - __clz(p.page_size);
      const int pg = p.page_table[(long long)n * p.max_pages + (place >> lps)];
      if ((unsigned)pg < (unsigned)p.num_pages)
        dst = (long long)pg * p.page_stride + (long long)(place & (p.page_size - 1)) * D;
    }
    float cs[8], sn[8];
    if (rot) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int pos = p.positions ? p.positions[(long long)axis[i] * p.tokens + tok] : p.pos0 + place;
        const int32_t t = (int32_t)((turn[i] * (uint64_t)(int64_t)pos) >> 32);
        __sincosf((float)t * 1.4629180792671596e-9f, &sn[i], &cs[i]);  // 2 pi 2^-32
        if (low) sn[i] = -sn[i];  // out = x cos + other * sn
      }
    }
    for (int r0 = part * RPW; r0 < rows; r0 += U * share * RPW) {
      uint4 raw[U];
#pragma unroll
      for (int i = 0; i < U; ++i) raw[i] = u[i];
      if (r0 + U * share * RPW < rows) fetch(r0 + U * share * RPW);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int r = r0 + i * share * RPW + lane / LPR;
        const int kind = r < p.hq ? 0 : r < p.hq + p.hkv ? 1 : 2;
        uint4 o;
        o.x = __shfl_sync(0xffffffffu, raw[i].x, peer);
        o.y = __shfl_sync(0xffffffffu, raw[i].y, peer);
        o.z = __shfl_sync(0xffffffffu, raw[i].z, peer);
        o.w = __shfl_sync(0xffffffffu, raw[i].w, peer);
        float x[8], y[8];
        unpack8(raw[i], x);
        unpack8(o, y);
        if (NORM) {
          float s = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) s = fmaf(x[e], x[e], s);
#pragma unroll
          for (int m = LPR / 2; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
          const float *nw = kind == 0 ? p.q_norm : kind == 1 ? p.k_norm : nullptr;
          if (nw) {
            const float inv = rsqrtf(s * (1.f / D) + p.eps);
            const int other = rot ? (low ? col + half : col - half) : col;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * nw[col + e], y[e] = y[e] * inv * nw[other + e];
          }
        }
        if (rot) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = fmaf(x[e], cs[e], y[e] * sn[e]);
        }
        if (r >= rows) continue;
        if (kind == 0)
          *(uint4 *)((__nv_bfloat16 *)p.q_out + ((long long)tok * p.hq + r) * D + col) = pack8(x);
        else if (kind == 1 && dst >= 0)
          *(uint4 *)((__nv_bfloat16 *)p.k_cache + dst + (long long)(r - p.hq) * p.page_size * D + col) = pack8(x);
        else if (kind == 2 && dst >= 0)
          *(uint4 *)((__nv_bfloat16 *)p.v_cache + dst + (long long)(r - p.hq - p.hkv) * p.page_size * D + col) = raw[i];
      }
    }
  }
}

// ------------------------------------------------------------------ add + norm

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *p, float (&x)[8]) {
  unpack8(*(const uint4 *)p, x);
}
template <>
__device__ __forceinline__ void load8<float>(const float *p, float (&x)[8]) {
  const float4 a = *(const float4 *)p, b = *(const float4 *)(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) { *(uint4 *)p = pack8(x); }
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
  *(float4 *)p = make_float4(x[0], x[1], x[2], x[3]);
  *(float4 *)(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void round8(__nv_bfloat16 *, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __bfloat162float(__float2bfloat16_rn(x[i]));
}
__device__ __forceinline__ void round8(float *, float (&)[8]) {}

// Sum of squares / largest magnitude over the block.  Magnitudes as their bits: an
// unsigned maximum that keeps NaN (fmaxf would drop it).
__device__ __forceinline__ float block_sum(float s, float *sh, int warps) {
  s = warp_sum(s);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
  __syncthreads();
  const int l = threadIdx.x & 31;
  return warp_sum(l < warps ? sh[l] : 0.f);
}
__device__ __forceinline__ uint32_t block_max(uint32_t m, uint32_t *sh, int warps) {
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = m;
  __syncthreads();
  const int l = threadIdx.x & 31;
  return __reduce_max_sync(0xffffffffu, l < warps ? sh[l] : 0u);
}
__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
  const float a = __uint_as_float(amax_bits);
  return (a < 1e-12f ? 1e-12f : a) / 448.f;  // NaN stays
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// One CTA per row; a thread keeps NV vectors of 8 values of the row, so x and the residual are read
// once and h, y written once.  In registers up to 32768 columns; the variant for wider rows (NV = 8, 1024
// threads of 64 registers) keeps part of them in local memory, 0.5 to 0.9 KB a thread.  Bound by HBM: 16383 rows of 4096 bf16 to
// e4m3 in groups of 128: 76.6 us, 6.16 TB/s (91% of the copy rate).
template <typename T, int NV>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(AddNormParams p) {
  __shared__ float sh_sum[32];
  __shared__ uint32_t sh_max[32];
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int warps = blockDim.x >> 5;
  const long long at = (long long)blockIdx.x * p.cols;
  float v[NV][8];
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * blockDim.x + threadIdx.x) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
    if (c < p.cols) {
      load8((const T *)p.x + at + c, v[j]);
      if (p.residual) {
        float r[8];
        load8((const T *)p.residual + at + c, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] += r[i];
        round8((T *)nullptr, v[j]);
      }
      if (p.residual_out) store8((T *)p.residual_out + at + c, v[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(v[j][i], v[j][i], s);
    }
  }
  s = block_sum(s, sh_sum, warps);
  const float inv = 1.f / sqrtf(s / p.cols + p.eps);
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * blockDim.x + threadIdx.x) * 8;
    if (c < p.cols) {
      float w[8];
      load8(p.weight + c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[j][i] = v[j][i] * inv * w[i];
        amax = max(amax, __float_as_uint(fabsf(v[j][i])));
      }
      if (!p.scale) store8((T *)p.y + at + c, v[j]);
    }
  }
  if (!p.scale) return;
  float scale = 0.f;
  if (p.group == 0) {
    scale = scale_of(block_max(amax, sh_max, warps));
    if (threadIdx.x == 0) p.scale[blockIdx.x] = scale;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * blockDim.x + threadIdx.x) * 8;
    if (p.group) {  // 16 lanes hold a group of 128 columns
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(fabsf(v[j][i])));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      scale = scale_of(m);
      if (c < p.cols && (threadIdx.x & 15) == 0)
        p.scale[(long long)blockIdx.x * (p.cols >> 7) + (c >> 7)] = scale;
    }
    if (c < p.cols) {
      // y / scale by the reciprocal in two floats, q + less = 1 / scale within 2^-46: rounded once, and exact
      // where the quotient is, so that a tie between two codes stays one.  (q alone put codes next to a
      // tie off by one; by division the prompts' norm took 85 us for 76.  Of an infinite scale q is 0.)
      const float q = 1.f / scale, less = scale == CUDART_INF_F ? 0.f : fmaf(-scale, q, 1.f) * q;
      auto over = [&](float y) { return fmaf(y, q, y * less); };
      uint2 u;
      u.x = e4m3x4(over(v[j][0]), over(v[j][1]), over(v[j][2]), over(v[j][3]));
      u.y = e4m3x4(over(v[j][4]), over(v[j][5]), over(v[j][6]), over(v[j][7]));
      *(uint2 *)((uint8_t *)p.y + at + c) = u;
    }
  }
}

template <typename T>
cudaError_t launch_norm_t(const AddNormParams &p, cudaStream_t stream) {
  const int vecs = p.cols / 8;
  // vectors per thread: as few threads as hold the row with 2 each, so that several rows share
  // an SM; 1 each while there are too few rows to fill the SMs; more for very wide rows
  const int want = p.rows < 304 && vecs <= 1024 ? 1 : vecs <= 2048 ? 2 : vecs <= 4096 ? 4 : 8;
  const int threads = ((vecs + want - 1) / want + 31) / 32 * 32;
  const unsigned grid = (unsigned)p.rows;
  auto *kernel = want == 1   ? add_rmsnorm_kernel<T, 1>
                 : want == 2 ? add_rmsnorm_kernel<T, 2>
                 : want == 4 ? add_rmsnorm_kernel<T, 4>
                             : add_rmsnorm_kernel<T, 8>;
  return launch_dependent(kernel, grid, threads, 0, stream, 1, p);
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t stream) {
  const int rpw = 32 / (p.d / 8);
  const int rows = p.hq + 2 * p.hkv;
  // warps per token: enough to fill 152 SMs with 16 warps each, while each has rows to do
  int share = 1;
  while (share < 8 && (long long)p.tokens * share < 152 * 16 && share * rpw < rows) share *= 2;
  const long long blocks = ((long long)p.tokens * share + kAppendWarps - 1) / kAppendWarps;
  const unsigned grid = (unsigned)(blocks < 152 * 16 ? blocks : 152 * 16);
  const bool norm = p.q_norm || p.k_norm;
  auto *kernel = p.d == 128 ? (norm ? append_kernel<128, true> : append_kernel<128, false>)
                            : (norm ? append_kernel<256, true> : append_kernel<256, false>);
  return launch_dependent(kernel, grid, 32 * kAppendWarps, 0, stream, 1, p, share);
}

cudaError_t launch_add_rmsnorm(const AddNormParams &p, gdn_dtype dtype, cudaStream_t stream) {
  return dtype == GDN_BF16 ? launch_norm_t<__nv_bfloat16>(p, stream) : launch_norm_t<float>(p, stream);
}

}  // namespace gdn
