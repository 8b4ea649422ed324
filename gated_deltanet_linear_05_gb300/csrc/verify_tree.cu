// The delta rule over a tree of drafts ("New in v2", prompt lookup decoding, with more than one
// continuation): every node's output and delta from its path's state, none of which is written.
//
// With G_i the sum of g over node i's path (itself included), j < i for "j is an ancestor of i", and S
// the snapshot, the per-token rule of "How it works" along the path gives, as in its chunkwise form,
//     delta_i = beta_i (v_i - e^(G_i) S^T k_i - sum_{j < i} e^(G_i - G_j) (k_i.k_j) delta_j)
//     o_i     = e^(G_i) S^T q_i + sum_{j <= i} e^(G_i - G_j) (q_i.k_j) delta_j,
// so a tree is one block whose triangular mask is the ancestors', and all paths share the two products
// with S and the Gram matrix.
//
// A CTA of 128 threads takes a (sequence, v-head); thread c owns value column c.
//   products  [Q; K] (2 C rows) S on the tcgen05 tensor cores as D^T = S^T [Q; K]^T: S^T is the operand
//             with 128 rows, in tensor memory, where thread c writes its column of S straight from
//             coalesced loads, 32 keys at a time; S never passes through shared memory.  Each value of S is
//             split in three bf16 terms (24 bits, all that float32 has); q and k are bf16 as they
//             are, or three terms too (f32), of whose products the six above 2^-24 are taken.
//             Accumulation is float32, so both types come out as float32 arithmetic would.
//   Gram      [Q; K] K^T the same way into the columns that S^T takes later; the thread of each row
//             multiplies the entries of its node's ancestors by their decays and appends them to the
//             node's list in shared memory.  The exponents are differences of G in two floats.
//   solve     each thread walks the nodes in order down its own column: the deltas it needs are its own, so
//             there is no barrier, and the work is the sum of the depths, not the square of the nodes.
//
// Bound by HBM: the 64 KB of S per head are read once.
#include "attn_tma.cuh"
#include "internal.h"
#include "tc.cuh"

namespace gdn {
namespace {

constexpr int kTreeThreads = 128;
constexpr int kKeys = 32;  // keys of S to a step

// Bytes of shared memory: operand tiles, v, deltas and a row of zeros, coefficients, their nodes.
template <typename T, int C>
struct TreeCfg {
  static constexpr int TERMS = sizeof(T) == 2 ? 1 : 3;  // bf16 terms of a value of q or k
  static constexpr int CHUNK = 2 * C * 128;             // 64 columns of [Q; K]
  static constexpr int QK = TERMS * 2 * CHUNK;
  static constexpr int V = C * kD * (int)sizeof(T);
  static constexpr int DELTA = (C + 1) * kD * 4;
  static constexpr int PAIRS = C * (C - 1) / 2 + 3 * C;  // every list a multiple of 4 long
  static constexpr int SMEM = 1024 + QK + V + DELTA + PAIRS * 9;
  // Gram rows past 2 C are read from whatever follows the tiles; all of it is the CTA's own
  static_assert(QK - CHUNK + 16384 <= SMEM - 1024, "the Gram product's 128 rows");
  static constexpr int COLS = 2 * C + 64 <= 128 ? 128 : 256;  // tensor memory
};

// 64 columns x 2 C rows of bf16, 128-byte swizzle, K-major.
__device__ __forceinline__ uint64_t tile_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}
__device__ __forceinline__ int tile_off(int row, int unit) { return row * 128 + ((unit ^ (row & 7)) << 4); }

__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// Uses of the loaded registers stay behind the wait.
template <int N>
__device__ __forceinline__ void tie(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// The leading bf16 of two floats, packed; the floats keep what is left of them.
__device__ __forceinline__ uint32_t take_bf16(float &a, float &b) {
  const uint32_t p = pack_bf16(a, b);
  a -= __uint_as_float(p << 16);
  b -= __uint_as_float(p & 0xffff0000u);
  return p;
}

// beta, e^G, q.k of a node itself, its list: first entry << 8 | entries
struct Node {
  float beta, from_state, own;
  int list;
};

template <typename T, typename TO, int C>
__global__ void __launch_bounds__(kTreeThreads, C == 64 ? 2 : 4) verify_tree_kernel(TreeParams p) {
  using F = TreeCfg<T, C>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) Node nodes[C];
  __shared__ uint64_t above[C];
  __shared__ float2 path[C];  // G in two floats
  __shared__ int up[C], sum0;
  __shared__ float gates[C];
  __shared__ uint64_t bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int dead_flag;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t *qk = smem;
  T *sv = reinterpret_cast<T *>(smem + F::QK);
  float *sd = reinterpret_cast<float *>(smem + F::QK + F::V);
  float2 *coef = reinterpret_cast<float2 *>(smem + F::QK + F::V + F::DELTA);
  uint8_t *which = reinterpret_cast<uint8_t *>(coef + F::PAIRS);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  volatile int *dead = &dead_flag;

  if (warp == 0) tc::alloc<F::COLS>(&tmem_slot);
  if (tid == 32) {
    mbar_init(&bar, 1);
    mbar_fence_init();
    dead_flag = 0;
  }
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int n = blockIdx.x / p.hv, h = blockIdx.x - n * p.hv, kh = h / (p.hv / p.hk);
  int bos, eos;
  seq_range(p.cu_seqlens, n, p.total_tokens, bos, eos);
  const int t_n = min(eos - bos, C);

  // the state's first 64 keys, then the rows of q, k and v
  const float *state = p.state_in ? p.state_in + ((size_t)n * p.hv + h) * kD * kD + tid : nullptr;
  float s[2][kKeys];
  if (state && t_n > 0) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < kKeys; ++i) s[c][i] = __ldcs(state + (c * kKeys + i) * kD);
  }
  const T *q = static_cast<const T *>(p.q), *k = static_cast<const T *>(p.k), *v = static_cast<const T *>(p.v);
  if (F::TERMS == 1) {
#pragma unroll 4
    for (int e = tid; e < 2 * C * 16; e += kTreeThreads) {
      const int row = e >> 4, unit = e & 15, t = row & (C - 1);
      const T *src = (row < C ? q : k) + ((size_t)(bos + (t < t_n ? t : 0)) * p.hk + kh) * kD + unit * 8;
      cp_async16(qk + (unit >> 3) * F::CHUNK + tile_off(row, unit & 7), src, t < t_n ? 16 : 0);
    }
  } else {
#pragma unroll 4
    for (int e = tid; e < 2 * C * 32; e += kTreeThreads) {
      const int row = e >> 5, quad = e & 31, t = row & (C - 1);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t < t_n)
        x = *reinterpret_cast<const float4 *>((row < C ? q : k) + ((size_t)(bos + t) * p.hk + kh) * kD + quad * 4);
      uint8_t *at = qk + (quad >> 4) * F::CHUNK + tile_off(row, (quad & 15) >> 1) + (quad & 1) * 8;
#pragma unroll
      for (int term = 0; term < 3; ++term) {
        uint2 w;
        w.x = take_bf16(x.x, x.y);
        w.y = take_bf16(x.z, x.w);
        *reinterpret_cast<uint2 *>(at + term * 2 * F::CHUNK) = w;
      }
    }
  }
  constexpr int kUnits = kD * (int)sizeof(T) / 16;  // of a row of v
  for (int e = tid; e < t_n * kUnits; e += kTreeThreads) {
    const int t = e / kUnits, unit = e % kUnits;
    cp_async16(reinterpret_cast<uint8_t *>(sv) + e * 16,
               reinterpret_cast<const uint8_t *>(v + ((size_t)(bos + t) * p.hv + h) * kD) + unit * 16, 16);
  }
  cp_async_commit();

  // ancestors, path sums, and the places of the lists
  float beta = 0.f;
  if (tid < t_n) {
    up[tid] = p.parents[bos + tid];
    gates[tid] = p.g[(size_t)(bos + tid) * p.hv + h];
    beta = p.beta[(size_t)(bos + tid) * p.hv + h];
  }
  sd[C * kD + tid] = 0.f;
  __syncthreads();
  int entries = 0, list = 0;
  uint64_t mine = 0;
  if (tid < C) {
    float hi = 0.f, lo = 0.f;
    if (tid < t_n) {
      for (int j = tid, next; ; j = next) {  // (goes down at every step)
        mine |= 1ull << j;
        const float x = gates[j], y = hi + x, z = y - hi;  // two-sum: y + (what it lost) = hi + x
        lo += (hi - (y - z)) + (x - z);
        hi = y;
        next = up[j];
        if (next < 0 || next >= j) break;
      }
      mine &= ~(1ull << tid);
      above[tid] = mine;
      path[tid] = make_float2(hi, lo);
    }
    entries = (__popcll(mine) + 3) & ~3;
    list = entries;
#pragma unroll
    for (int o = 1; o < (C < 32 ? C : 32); o <<= 1) {
      const int x = __shfl_up_sync(C < 32 ? 0xffffu : 0xffffffffu, list, o);
      if (lane >= o) list += x;
    }
    if (tid == 31) sum0 = list;
    nodes[tid] = Node{beta, expf(hi + lo), 0.f, 0};
  }
  cp_async_wait<0>();
  tc::fence_proxy_async();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_slot;
  constexpr uint32_t kA = 2 * C;  // columns: D^T from 0, Gram and then S^T from here
  const uint64_t tiles = tile_desc(uniform(smem_u32(qk)));
  constexpr uint32_t kChunk = F::CHUNK >> 4;
  // terms of a product whose order is at most 2^-16 (2^-24 is left of their sum), small ones first
  constexpr int kTermA[6] = {2, 1, 0, 1, 0, 0}, kTermB[6] = {0, 1, 2, 0, 1, 0};
  if (warp == 0 && t_n > 0) {
    if (elect_one()) {
      constexpr uint32_t id = tc::idesc(128, C, 1, 0, 0);
      const uint64_t keys = tiles + (C * 128 >> 4);
      bool some = false;
#pragma unroll
      for (int x = F::TERMS == 1 ? 5 : 0; x < 6; ++x)
#pragma unroll
        for (int i = 0; i < kD / 16; ++i, some = true)
          tc::mma_ss(tmem + kA, tiles + (kTermA[x] * 2 + i / 4) * kChunk + (i % 4) * 2,
                     keys + (kTermB[x] * 2 + i / 4) * kChunk + (i % 4) * 2, id, some);
      tc::commit(&bar);
    }
    __syncwarp();
  }
  if (tid < t_n) {
    if (tid >= 32) list += sum0;
    nodes[tid].list = (list - entries) << 8 | entries;
    for (int i = __popcll(mine); i < entries; ++i) {
      coef[list - entries + i] = make_float2(0.f, 0.f);
      which[list - entries + i] = C;  // the row of zeros
    }
  }
  __syncthreads();
  uint32_t phase = 0;
  const uint32_t lanes = tmem + ((uint32_t)(32 * warp) << 16);
  if (t_n > 0) {
    wait_bar(&bar, phase, dead, p.err);
    tc::fence_after();
    if (32 * warp < 2 * C) {  // rows of the Gram matrix: of Q, then of K
      const int t = tid & (C - 1);
      const bool of_k = tid >= C, row = tid < 2 * C && t < t_n;
      const uint64_t bits = row ? above[t] : 0;
      const float2 mine2 = row ? path[t] : make_float2(0.f, 0.f);
      int at = row ? nodes[t].list >> 8 : 0;
#pragma unroll 1
      for (int j0 = 0; j0 < t_n; j0 += 16) {
        uint32_t x[16];
        ld16(lanes + kA + j0, x);
        tc::wait_ld();
        tie(x);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = j0 + i;
          if (bits >> j & 1) {
            const float2 g = path[j];
            const float y = __uint_as_float(x[i]) * expf((mine2.x - g.x) + (mine2.y - g.y));
            if (of_k) coef[at].x = y;
            else coef[at].y = y, which[at] = j;
            ++at;
          }
          if (row && !of_k && j == t) nodes[t].own = __uint_as_float(x[i]);
        }
      }
    }
    phase ^= 1;
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();

  // D^T = S^T [Q; K]^T
  if (state && t_n > 0) {
    constexpr uint32_t id = tc::idesc(128, 2 * C, 1, 0, 0);
#pragma unroll
    for (int c = 0; c < kD / kKeys; ++c) {
      float(&x)[kKeys] = s[c & 1];
#pragma unroll
      for (int term = 0; term < 3; ++term) {
        uint32_t w[kKeys / 2];
#pragma unroll
        for (int i = 0; i < kKeys / 2; ++i) w[i] = take_bf16(x[2 * i], x[2 * i + 1]);
        if (term == 0 && c > 0) {  // the products of the step before have read their operand
          wait_bar(&bar, phase, dead, p.err);
          phase ^= 1;
          tc::fence_after();
        }
        tc::st16(lanes + kA + 16 * term, w);
      }
      if (c + 2 < kD / kKeys) {
#pragma unroll
        for (int i = 0; i < kKeys; ++i) x[i] = __ldcs(state + ((c + 2) * kKeys + i) * kD);
      }
      tc::wait_st();
      tc::fence_before();
      __syncthreads();
      if (warp == 0) {
        tc::fence_after();
        if (elect_one()) {
          bool some = c > 0;
#pragma unroll
          for (int y = 0; y < 6; ++y) {
            if (F::TERMS == 1 && kTermB[y] > 0) continue;
#pragma unroll
            for (int i = 0; i < kKeys / 16; ++i, some = true)
              tc::mma_ts(tmem, tmem + kA + 16 * kTermA[y] + 8 * i,
                         tiles + (kTermB[y] * 2 + c / 2) * kChunk + ((c % 2) * 2 + i) * 2, id, some);
          }
          tc::commit(&bar);
        }
        __syncwarp();
      }
    }
    wait_bar(&bar, phase, dead, p.err);
    tc::fence_after();
  }

  // the nodes in order, each thread down its column
  TO *o = static_cast<TO *>(p.o);
#pragma unroll 1
  for (int t0 = 0; t0 < t_n; t0 += 8) {
    uint32_t qs[8] = {}, ks[8] = {};
    if (state) {
      ld8(lanes + t0, qs);
      ld8(lanes + C + t0, ks);
      tc::wait_ld();
      tie(qs);
      tie(ks);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = t0 + i;
      if (t < t_n) {
        const Node node = nodes[t];
        float below = 0.f, out = 0.f;
        const int first = node.list >> 8, last = first + (node.list & 255);
        for (int e = first; e < last; e += 4) {
          const uint32_t w = *reinterpret_cast<const uint32_t *>(which + e);
          const float4 c0 = *reinterpret_cast<const float4 *>(coef + e), c1 = *reinterpret_cast<const float4 *>(coef + e + 2);
          const float d0 = sd[(w & 255) * kD + tid], d1 = sd[(w >> 8 & 255) * kD + tid],
                      d2 = sd[(w >> 16 & 255) * kD + tid], d3 = sd[(w >> 24) * kD + tid];
          below = fmaf(c0.x, d0, below), out = fmaf(c0.y, d0, out);
          below = fmaf(c0.z, d1, below), out = fmaf(c0.w, d1, out);
          below = fmaf(c1.x, d2, below), out = fmaf(c1.y, d2, out);
          below = fmaf(c1.z, d3, below), out = fmaf(c1.w, d3, out);
        }
        const float d =
            node.beta * (Elem<T>::load(sv + t * kD + tid) - fmaf(node.from_state, __uint_as_float(ks[i]), below));
        sd[t * kD + tid] = d;
        const size_t at = ((size_t)(bos + t) * p.hv + h) * kD + tid;
        p.delta[at] = d;
        Elem<TO>::store(o + at, fmaf(node.own, d, fmaf(node.from_state, __uint_as_float(qs[i]), out)));
      }
    }
  }
  if (*dead) __nanosleep(1000000);  // products in flight end before tensor memory is given up
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::dealloc<F::COLS>(tmem);
}

template <typename T, typename TO, int C>
cudaError_t launch(const TreeParams &p, cudaStream_t stream) {
  constexpr size_t smem = TreeCfg<T, C>::SMEM;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t err = allow_smem(verify_tree_kernel<T, TO, C>, smem, allowed);
  if (err != cudaSuccess) return err;
  return launch_dependent(verify_tree_kernel<T, TO, C>, (unsigned)(p.num_seqs * p.hv), kTreeThreads, smem, stream, 1, p);
}
template <typename T, typename TO>
cudaError_t by_size(const TreeParams &p, cudaStream_t stream) {
  return p.chunk == 16 ? launch<T, TO, 16>(p, stream) : p.chunk == 32 ? launch<T, TO, 32>(p, stream)
                                                                     : launch<T, TO, 64>(p, stream);
}

}  // namespace

cudaError_t launch_verify_tree(const TreeParams &p, cudaStream_t stream) {
  if (p.dtype == GDN_F32) return by_size<float, float>(p, stream);
  return p.o_fp32 ? by_size<__nv_bfloat16, float>(p, stream) : by_size<__nv_bfloat16, __nv_bfloat16>(p, stream);
}

}  // namespace gdn
