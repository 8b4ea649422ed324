// The delta rule over a tree of drafts ("New in v2", prompt lookup decoding, with more than one
// continuation): every node's output and delta from its path's state, none of which is written.
//
// With G_i the sum of g over node i's path (itself included), j < i for "j is an ancestor of i", and S
// the snapshot, the per-token rule of "How it works" along the path gives, as in its chunkwise form,
//     delta_i = beta_i (r_i - sum_{j < i} e^(G_i - G_j) (k_i.k_j) delta_j),   r_i = v_i - e^(G_i) S^T k_i
//     o_i     = e^(G_i) S^T q_i + sum_{j <= i} e^(G_i - G_j) (q_i.k_j) delta_j,
// so a tree is one block whose triangular mask is the ancestors', and all paths share the two products
// with S and the Gram matrix.  The recursion is linear in r: with T its matrix, found by running it on the unit
// vectors (C columns, not the 128 of r), and W = (decays . Q K^T) T, both zero but for ancestors,
//     delta = T r,   o = diag(e^G) Q S + W r.
//
// A CTA takes a (sequence, v-head).  Threads 0..127 own a value column each, C / 32 warps more the tree.
//   products  [Q; K] (2 C rows) S on the tcgen05 tensor cores as D^T = S^T [Q; K]^T: S^T is the operand
//             with 128 rows, in tensor memory, where thread c writes its column of S straight from
//             coalesced loads, 32 keys at a time; S never passes through shared memory.  Each value of S is
//             split in three bf16 terms (24 bits, all that float32 has); q and k are bf16 as they
//             are, or three terms too (f32), of whose products the six above 2^-24 are taken.
//             Accumulation is float32, so both types come out as float32 arithmetic would.
//   tree      meanwhile: the Gram products K [Q; K]^T come the same way into D^T's columns before S needs
//             them; the thread of key j multiplies those of its descendants by the decays (exponents:
//             differences of G in two floats).  Then thread j runs the recursion on unit vector j, 16 nodes
//             at a time in registers.  (Down lists of the ancestors alone it took 90 cycles for each four of
//             them, one after another: 24 trees of 40 to 64 nodes, some of them chains, in f32 237 us for 168.)
//   results   r, in three terms over S^T's columns, times [W; T]^T in three terms, added to
//             diag(e^G) D^T in place.
//
// The 64 KB of S per head are read once.  64 trees of 11 to 32 nodes, 32 heads: 49 us, 3.8 TB/s (floor 27);
// bound by the chain of steps that a CTA goes through (loads under a busy HBM 6000 cycles, the state's steps
// 11000, results 5000 of 22000) at four CTAs an SM, all that tensor memory holds (128 of 512 columns each).
// 24 trees of 40 to 64 nodes: bf16 64 us, f32 86 (two CTAs).
//
// Tried and dropped: tf32 terms (two instructions a value in place of five and a half; q and k then go through
// registers to become 32 bits wide: 52 -> 66 us), the next CTA's state brought to L2 meanwhile (the same), T for two
// columns a lane and W by another warp (C = 64: 124 -> 134), the solution of 16 nodes in a rolled loop (52 -> 60).
#include "attn_tma.cuh"
#include "internal.h"
#include "tc.cuh"

namespace gdn {
namespace {

constexpr int kColumns = 128;  // threads with a value column
constexpr int kKeys = 32;      // keys of S to a step

// Shared memory: operand tiles, whose place [W; T] in three terms takes; N and A, whose place W and T
// take; v, if there is room.
template <typename T, int C>
struct TreeCfg {
  static constexpr int TERMS = sizeof(T) == 2 ? 1 : 3;  // bf16 terms of a value of q or k
  static constexpr int CHUNK = 2 * C * 128;             // 64 columns of [Q; K]
  // Chunks in shared memory at a time.  f32 rows of 32 and 64 nodes have 48 and 96 KB of terms, which leave an SM two
  // CTAs and one: their chunks come one after the other, the second once more for the state's products, and v straight
  // to registers (24 trees of 40 to 64 nodes 124 -> 86 us, 64 of 11 to 32 96 -> 88; 64 of 8 to 16 50 -> 57: not there).
  static constexpr int HALVES = TERMS == 3 && C >= 32 ? 1 : 2;
  static constexpr int QK = TERMS * HALVES * CHUNK;
  static constexpr int WT_TERM = 2 * C * C * 2;         // a term of [W; T]
  static constexpr int N_AT = QK > 3 * WT_TERM ? QK : 3 * WT_TERM;
  static constexpr int ROW = C + 4;                     // floats: 16-byte accesses of a column of rows spread over the banks
  static constexpr int A_AT = N_AT + C * ROW * 4;
  static constexpr int V_AT = A_AT + C * ROW * 4;
  static constexpr int USED = V_AT + (HALVES == 2 ? C * kD * (int)sizeof(T) : 0);
  // the Gram product reads 128 rows from K's first; past the tiles they are whatever follows
  static constexpr int GRAM = QK - CHUNK + C * 128 + 16384;
  static constexpr int SMEM = 1024 + (USED > GRAM ? USED : GRAM);
  static constexpr int A_COL = 2 * C, A_COLS = 3 * C / 2 > 48 ? 3 * C / 2 : 48;  // tensor memory: after D^T
  static constexpr int COLS = A_COL + A_COLS <= 128 ? 128 : 256;
  // The halves' Gram products stay apart until they are added in registers, the second's in the columns of A: on top of the
  // first's, the small terms of the second would be cut to its size (o at 32 and 64 nodes 8.0e-7 and 7.5e-7 of its rms
  // off, against 4.8e-7 and 3.2e-7 so).
  static_assert(HALVES == 2 || 4 * C <= COLS, "columns of the second half's Gram products");
  static constexpr int TREE_WARPS = C == 64 ? 2 : 1;
  static constexpr int THREADS = kColumns + 32 * TREE_WARPS;
  // CTAs on an SM by shared and by tensor memory; three where a fourth takes too many registers from the
  // reloading of chunks (3 us of 64 trees of 11 to 32; without it, at C = 16, 52 for 50)
  static constexpr int FIT = 227 * 1024 / (SMEM + 4096), MOST = HALVES == 1 && COLS == 128 ? 3 : 512 / COLS;
  static constexpr int CTAS = FIT < MOST ? FIT : MOST;
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

// The leading 8 bits of two floats as bf16, packed; the floats keep what is left of them (three times 8 bits
// are all that they have).
__device__ __forceinline__ uint32_t take_bf16(float &a, float &b) {
  const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
  a -= __uint_as_float(x & 0xffff0000u);
  b -= __uint_as_float(y & 0xffff0000u);
  return __byte_perm(x, y, 0x7632);
}

__device__ __forceinline__ void st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 z, x, y, z;\n mov.b64 {%0, %1}, z;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
// acc[i] += row[i] x for the entries FIRST and up of 16, in pairs.
template <int FIRST>
__device__ __forceinline__ void add_row(float2 (&acc)[8], const float *row, float x) {
#pragma unroll
  for (int i = FIRST / 4; i < 4; ++i) {
    const float4 c = *reinterpret_cast<const float4 *>(row + 4 * i);
    if (2 * (2 * i + 1) > FIRST) acc[2 * i] = fma2(make_float2(c.x, c.y), make_float2(x, x), acc[2 * i]);
    acc[2 * i + 1] = fma2(make_float2(c.z, c.w), make_float2(x, x), acc[2 * i + 1]);
  }
}
template <int I>
__device__ __forceinline__ float entry(const float2 (&x)[8]) {
  return I & 1 ? x[I / 2].y : x[I / 2].x;
}
// Nodes I and up of 16: r and w hold what the nodes before them add; d takes their column of T.
template <int I>
__device__ __forceinline__ void solve(float2 (&r)[8], float2 (&w)[8], float (&d)[16], const float *sn, const float *sa,
                                      int pitch, const float *beta, int unit) {
  d[I] = beta[I] * ((unit == I ? 1.f : 0.f) - entry<I>(r));
  if constexpr (I < 15) add_row<I + 1>(r, sn + I * pitch, d[I]);
  add_row<I>(w, sa + I * pitch, d[I]);
  if constexpr (I < 15) solve<I + 1>(r, w, d, sn, sa, pitch, beta, unit);
}

// Products of three-term operands whose order is at most 2^-16 (2^-24 is left of their sum), small first.
constexpr int kProducts = 6;
__device__ constexpr int kTermA[kProducts] = {2, 1, 0, 1, 0, 0}, kTermB[kProducts] = {0, 1, 2, 0, 1, 0};

template <typename T, typename TO, int C>
__global__ void __launch_bounds__(TreeCfg<T, C>::THREADS, TreeCfg<T, C>::CTAS) verify_tree_kernel(TreeParams p) {
  using F = TreeCfg<T, C>;
  constexpr int kTree = 32 * F::TREE_WARPS;
  constexpr int kGramRead = kTree + (F::HALVES == 1 ? kColumns : 32);  // threads at that barrier
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t above[C];    // a node's ancestors, itself among them
  __shared__ float2 path[C];       // G log2(e) in two floats
  __shared__ float from_state[C];  // e^G
  __shared__ float gates[C], beta[C];
  __shared__ int up[C];
  __shared__ uint64_t bar_gram, bar_s, bar_out;
  __shared__ uint32_t tmem_slot;
  __shared__ int dead_flag;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  // of key m and node t, at m ROW + t: the factors of delta_m in delta_t and in o_t; then W and T
  float *sn = reinterpret_cast<float *>(smem + F::N_AT), *sa = reinterpret_cast<float *>(smem + F::A_AT);
  T *sv = reinterpret_cast<T *>(smem + F::V_AT);
  const int tid = threadIdx.x, warp = uniform(tid >> 5);
  volatile int *dead = &dead_flag;

  if (warp == 0) tc::alloc<F::COLS>(&tmem_slot);
  if (tid == 32) {
    mbar_init(&bar_gram, 1);
    mbar_init(&bar_s, 1);
    mbar_init(&bar_out, 1);
    mbar_fence_init();
    dead_flag = 0;
  }
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int n = blockIdx.x / p.hv, h = blockIdx.x - n * p.hv, kh = h / (p.hv / p.hk);
  int bos, eos;
  seq_range(p.cu_seqlens, n, p.total_tokens, bos, eos);
  const int t_n = min(eos - bos, C);

  const T *q = static_cast<const T *>(p.q), *k = static_cast<const T *>(p.k), *v = static_cast<const T *>(p.v);
  // f32 rows of q and k in three terms, from column 64 `half` on, by `threads` threads; `ready` comes before the first
  // of them is written
  auto put_rows = [&](int half, int threads, auto ready) {
    constexpr int kBatch = 8;  // loads side by side (two at a time, the rows took 13k cycles of an item's 45k)
    constexpr int kQuads = 16 * F::HALVES;
#pragma unroll 1
    for (int e0 = tid; e0 < 2 * C * kQuads; e0 += kBatch * threads) {
      float4 x[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int e = e0 + b * threads, row = e / kQuads, t = row & (C - 1);
        x[b] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (e < 2 * C * kQuads && t < t_n)
          x[b] = *reinterpret_cast<const float4 *>((row < C ? q : k) + ((size_t)(bos + t) * p.hk + kh) * kD + half * 64 +
                                                   (e % kQuads) * 4);
      }
      if (e0 == tid) ready();
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int e = e0 + b * threads, row = e / kQuads, quad = e % kQuads;
        if (e >= 2 * C * kQuads) break;
        uint8_t *at = smem + (quad >> 4) * F::CHUNK + tile_off(row, (quad & 15) >> 1) + (quad & 1) * 8;
#pragma unroll
        for (int term = 0; term < 3; ++term) {
          uint2 w;
          w.x = take_bf16(x[b].x, x[b].y);
          w.y = take_bf16(x[b].z, x[b].w);
          *reinterpret_cast<uint2 *>(at + term * F::HALVES * F::CHUNK) = w;
        }
      }
    }
  };
  if (F::TERMS == 1) {
#pragma unroll 2
    for (int e = tid; e < 2 * C * 16; e += F::THREADS) {
      const int row = e >> 4, unit = e & 15, t = row & (C - 1);
      const T *src = (row < C ? q : k) + ((size_t)(bos + (t < t_n ? t : 0)) * p.hk + kh) * kD + unit * 8;
      cp_async16(smem + (unit >> 3) * F::CHUNK + tile_off(row, unit & 7), src, t < t_n ? 16 : 0);
    }
  } else {
    put_rows(F::HALVES == 1 ? 1 : 0, F::THREADS, [] {});
  }
  constexpr int kUnits = kD * (int)sizeof(T) / 16;  // of a row of v
  for (int e = tid; F::HALVES == 2 && e < t_n * kUnits; e += F::THREADS) {
    const int t = e / kUnits, unit = e % kUnits;
    cp_async16(reinterpret_cast<uint8_t *>(sv) + e * 16,
               reinterpret_cast<const uint8_t *>(v + ((size_t)(bos + t) * p.hv + h) * kD) + unit * 16, 16);
  }
  cp_async_commit();
  // the state's first 64 keys, then the rows of q, k and v
  const float *state = p.state_in ? p.state_in + ((size_t)n * p.hv + h) * kD * kD + (tid & 127) : nullptr;
  float s[2][kKeys];
  if (state && t_n > 0 && warp < 4) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < kKeys; ++i) s[c][i] = __ldcs(state + (c * kKeys + i) * kD);
  }

  // ancestors, path sums, and the places of the lists
  const int j = tid - kColumns;  // of a thread of the tree: its node, and its key
  if (warp >= 4) {
    const bool node = j < t_n;
    if (node) {
      up[j] = p.parents[bos + j];
      gates[j] = p.g[(size_t)(bos + j) * p.hv + h];
    }
    bar_sync(3, kTree);
    uint64_t mine = 0;
    float hi = 0.f, lo = 0.f;
    if (node) {
      for (int i = j, next; ; i = next) {  // (goes down at every step)
        mine |= 1ull << i;
        const float x = gates[i], y = hi + x, z = y - hi;  // two-sum: y + (what it lost) = hi + x
        lo += (hi - (y - z)) + (x - z);
        hi = y;
        next = up[i];
        if (next < 0 || next >= i) break;
      }
    }
    __syncwarp();
    if (j < C) {
      above[j] = mine;
      const float up2 = hi * 1.44269504f;  // (and what the product and the constant lose)
      const float low2 = fmaf(hi, 1.44269504f, -up2) + fmaf(lo, 1.44269504f, hi * 1.92596299e-8f);
      path[j] = make_float2(up2, low2);
      from_state[j] = ex2(up2 + low2);
      beta[j] = node ? p.beta[(size_t)(bos + j) * p.hv + h] : 0.f;
    }
  }
  cp_async_wait<0>();
  tc::fence_proxy_async();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_slot;
  const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
  const uint64_t tiles = tile_desc(uniform(smem_u32(smem)));
  constexpr uint32_t kChunk = F::CHUNK >> 4;
  constexpr uint32_t id_s = tc::idesc(128, 2 * C, 1, 0, 0);
  // Gram products of the chunks in shared memory, to tensor memory at `to`; by one thread
  auto gram = [&](uint32_t to) {
    bool some = false;
    const uint64_t keys = tiles + (C * 128 >> 4);
#pragma unroll
    for (int x = F::TERMS == 1 ? kProducts - 1 : 0; x < kProducts; ++x)
#pragma unroll
      for (int i = 0; i < F::HALVES * 4; ++i, some = true)
        tc::mma_ss(to, keys + (kTermA[x] * F::HALVES + i / 4) * kChunk + (i % 4) * 2,
                   tiles + (kTermB[x] * F::HALVES + i / 4) * kChunk + (i % 4) * 2, id_s, some);
    tc::commit(&bar_gram);
  };
  if (F::HALVES == 1 && t_n > 0) {  // the second half's, then the first half in its place
    if (warp == 4) {
      if (elect_one()) gram(tmem);
      __syncwarp();
    }
    put_rows(0, F::THREADS, [&] { wait_bar(&bar_gram, 0, dead, p.err); });
    tc::fence_proxy_async();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
  }
  if (t_n > 0 && warp >= 4) {
    // ---------------------------------------------------------------- the tree
    if (warp == 4) {
      if (elect_one()) gram(F::HALVES == 1 ? tmem + 2 * C : tmem);
      __syncwarp();
    }
    wait_bar(&bar_gram, F::HALVES == 1 ? 1 : 0, dead, p.err);
    tc::fence_after();
    const float2 own = path[j & (C - 1)];
#pragma unroll 1
    for (int t0 = 0; t0 < (t_n + 15) / 16 * 16; t0 += 8) {
      uint32_t x[8], y[8];
      ld8(lanes + t0, x);  // (by whole warps: at C = 16 half of the lanes have no key)
      ld8(lanes + C + t0, y);
      tc::wait_ld();
      tie(x);
      tie(y);
      if (F::HALVES == 1) {
        uint32_t x2[8], y2[8];
        ld8(lanes + 2 * C + t0, x2);
        ld8(lanes + 3 * C + t0, y2);
        tc::wait_ld();
        tie(x2);
        tie(y2);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = __float_as_uint(__uint_as_float(x[i]) + __uint_as_float(x2[i]));
          y[i] = __float_as_uint(__uint_as_float(y[i]) + __uint_as_float(y2[i]));
        }
      }
      float a[8], b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int t = t0 + i;
        const float2 g = path[t];
        const float decay = ex2((g.x - own.x) + (g.y - own.y));
        const bool on = above[t] >> j & 1;  // (its own: decay 1, and no factor of delta)
        a[i] = on ? __uint_as_float(x[i]) * decay : 0.f;
        b[i] = on && t != j ? __uint_as_float(y[i]) * decay : 0.f;
      }
      if (j < C) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          *reinterpret_cast<float4 *>(sa + j * F::ROW + t0 + i) = make_float4(a[i], a[i + 1], a[i + 2], a[i + 3]);
          *reinterpret_cast<float4 *>(sn + j * F::ROW + t0 + i) = make_float4(b[i], b[i + 1], b[i + 2], b[i + 3]);
        }
      }
    }
    tc::fence_before();
    bar_arrive(1, kGramRead);  // D^T's columns are free, and A's
    bar_sync(3, kTree);
    // column j of T and W, 16 nodes at a time; they take the place of the factors that have been used
#pragma unroll 1
    for (int t0 = 0; t0 < t_n; t0 += 16) {
      float2 r[8] = {}, w[8] = {};
      float d[16];
      // four at a time of the nodes before these 16, where one of them has one of these below
      uint64_t need = above[t0 + (j & 15)];
      need = (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(need >> 32)) << 32 |
             __reduce_or_sync(0xffffffffu, (uint32_t)need);
      if (j < C) {
#pragma unroll 1
        for (int m = 0; m < t0; m += 4) {
          if (!(need >> m & 15)) continue;
          const float4 x = *reinterpret_cast<const float4 *>(sa + j * F::ROW + m);
          const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            add_row<0>(r, sn + (m + i) * F::ROW + t0, xs[i]);
            add_row<0>(w, sa + (m + i) * F::ROW + t0, xs[i]);
          }
        }
        solve<0>(r, w, d, sn + t0 * F::ROW + t0, sa + t0 * F::ROW + t0, F::ROW, beta + t0, j - t0);
      }
      bar_sync(3, kTree);
      if (j < C) {
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          *reinterpret_cast<float4 *>(sa + j * F::ROW + t0 + i) = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
          *reinterpret_cast<float4 *>(sn + j * F::ROW + t0 + i) =
              make_float4(w[i / 2].x, w[i / 2].y, w[i / 2 + 1].x, w[i / 2 + 1].y);
        }
      }
    }
    bar_sync(3, kTree);
  } else if (t_n > 0) {
    // ---------------------------------------------------------------- D^T = S^T [Q; K]^T
    if (state) {
#pragma unroll 1
      for (int c0 = 0; c0 < kD / kKeys; c0 += 2) {
        if (F::HALVES == 1 && c0 > 0) {
          put_rows(1, kColumns, [&] { wait_bar(&bar_out, 1, dead, p.err); });
          tc::fence_proxy_async();  // (the next barrier is before these products)
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int c = c0 + half;
          float(&x)[kKeys] = s[half];
#pragma unroll
          for (int term = 0; term < 3; ++term) {
            uint32_t w[kKeys / 2];
#pragma unroll
            for (int i = 0; i < kKeys / 2; ++i) w[i] = take_bf16(x[2 * i], x[2 * i + 1]);
            if (F::HALVES == 1 && term == 0 && c == 0) {
              bar_sync(1, kGramRead);
              tc::fence_after();
            }
            if (term == 0 && c > 0) {  // the products of the step before have read their operand
              wait_bar(&bar_out, (c - 1) & 1, dead, p.err);
              tc::fence_after();
            }
            tc::st16(lanes + F::A_COL + 16 * term, w);
          }
          if (c0 == 0) {
#pragma unroll
            for (int i = 0; i < kKeys; ++i) x[i] = __ldcs(state + ((c + 2) * kKeys + i) * kD);
          }
          tc::wait_st();
          tc::fence_before();
          bar_sync(2, kColumns);
          if (warp == 0) {
            if (F::HALVES == 2 && c == 0) bar_sync(1, kGramRead);  // the Gram products have been read
            tc::fence_after();
            if (elect_one()) {
              uint32_t some = c > 0;
#pragma unroll
              for (int y = 0; y < kProducts; ++y) {
                if (F::TERMS == 1 && kTermB[y] > 0) continue;
#pragma unroll
                for (int i = 0; i < kKeys / 16; ++i, some = 1)
                  tc::mma_ts(tmem, tmem + F::A_COL + 16 * kTermA[y] + 8 * i,
                             tiles + (kTermB[y] * F::HALVES + (F::HALVES == 2 ? c0 >> 1 : 0)) * kChunk + (half * 2 + i) * 2, id_s, some);
              }
              tc::commit(c + 1 < kD / kKeys ? &bar_out : &bar_s);
            }
            __syncwarp();
          }
        }
      }
      wait_bar(&bar_s, 0, dead, p.err);
      tc::fence_after();
    } else {
      if (F::HALVES == 1 || warp == 0) bar_sync(1, kGramRead);
      bar_sync(2, kColumns);
      tc::fence_after();
    }
    // r, and what it will be added to
    const T *v_col = v + ((size_t)bos * p.hv + h) * kD + tid;
    float ahead[16];
    auto load_v = [&](int t0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) ahead[i] = t0 + i < t_n ? Elem<T>::load(v_col + (size_t)(t0 + i) * p.hv * kD) : 0.f;
    };
    if (F::HALVES == 1) load_v(0);
#pragma unroll 1
    for (int t0 = 0; t0 < t_n; t0 += 16) {
      uint32_t x[16], y[16];
      if (state) {
        ld16(lanes + t0, x);
        ld16(lanes + C + t0, y);
        tc::wait_ld();
        tie(x);
        tie(y);
      }
      float r[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int t = t0 + i;
        const bool node = t < t_n;
        const float scale = node && state ? from_state[t] : 0.f;
        if (F::HALVES == 2) r[i] = node ? Elem<T>::load(sv + t * kD + tid) : 0.f;
        else r[i] = ahead[i];
        if (state) r[i] = fmaf(-scale, __uint_as_float(y[i]), r[i]);
        x[i] = state ? __float_as_uint(scale * __uint_as_float(x[i])) : 0u;
        y[i] = 0u;
      }
      if (F::HALVES == 1) load_v(t0 + 16);
      tc::st16(lanes + t0, x);
      tc::st16(lanes + C + t0, y);
#pragma unroll
      for (int term = 0; term < 3; ++term) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = take_bf16(r[2 * i], r[2 * i + 1]);
        st8(lanes + F::A_COL + term * (C / 2) + t0 / 2, w);
      }
    }
    tc::wait_st();
  }
  __syncthreads();
  // [W; T] in three terms over the tiles, which every product has read: 8-row x 16-byte core matrices, rows of
  // a key column contiguous
  const int keys16 = (t_n + 15) / 16 * 16;
#pragma unroll 2
  for (int e = tid; e < keys16 * (C / 2); e += F::THREADS) {
    const int t = e & (C - 1), c = 2 * (e / C);
    const float *a = sn + c * F::ROW + t, *b = sa + c * F::ROW + t;
    float a0 = a[0], a1 = a[F::ROW], b0 = b[0], b1 = b[F::ROW];
    uint8_t *at = smem + (c >> 3) * (2 * C * 16) + t * 16 + (c & 7) * 2;
#pragma unroll
    for (int term = 0; term < 3; ++term) {
      *reinterpret_cast<uint32_t *>(at + term * F::WT_TERM) = take_bf16(a0, a1);
      *reinterpret_cast<uint32_t *>(at + term * F::WT_TERM + C * 16) = take_bf16(b0, b1);
    }
  }
  tc::fence_proxy_async();
  tc::fence_before();
  __syncthreads();
  if (t_n > 0 && warp < 4) {
    if (warp == 0) {
      tc::fence_after();
      const uint64_t wt = tc::sdesc(uniform(smem_u32(smem)), 2 * C * 16, 128);
      const int steps = (t_n + 15) / 16;
      if (elect_one()) {
#pragma unroll
        for (int y = 0; y < kProducts; ++y)
#pragma unroll 1
          for (int i = 0; i < steps; ++i)
            tc::mma_ts(tmem, tmem + F::A_COL + kTermA[y] * (C / 2) + 8 * i,
                       wt + ((kTermB[y] * F::WT_TERM + i * 2 * (2 * C * 16)) >> 4), id_s, 1);
        tc::commit(&bar_out);
      }
      __syncwarp();
    }
    wait_bar(&bar_out, state ? 1 : 0, dead, p.err);
    tc::fence_after();
    TO *o = static_cast<TO *>(p.o) + ((size_t)bos * p.hv + h) * kD + tid;
    float *delta = p.delta + ((size_t)bos * p.hv + h) * kD + tid;
    const size_t row = (size_t)p.hv * kD;
#pragma unroll 1
    for (int t0 = 0; t0 < t_n; t0 += 16) {
      uint32_t x[16], y[16];
      ld16(lanes + t0, x);
      ld16(lanes + C + t0, y);
      tc::wait_ld();
      tie(x);
      tie(y);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (t0 + i < t_n) {
          Elem<TO>::store(o + (t0 + i) * row, __uint_as_float(x[i]));
          delta[(t0 + i) * row] = __uint_as_float(y[i]);
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
  return launch_dependent(verify_tree_kernel<T, TO, C>, (unsigned)(p.num_seqs * p.hv), TreeCfg<T, C>::THREADS, smem, stream, 1, p);
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
