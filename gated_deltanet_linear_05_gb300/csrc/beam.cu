// Several beams of a request: the selection of their best continuations over beams and vocabulary, and the
// reordering of the rows that follow them.
#include <algorithm>

#include "attn_tma.cuh"
#include "beam.h"

namespace gdn {
namespace {

// ------------------------------------------------------------------ selection
//
// s(w, x) = score_w + logit_wx - lse_w.  Within a beam the order is the logits', so one pass over a
// row finds its maximum, its sum of powers and its `top` best logits without the sum being known; the
// second kernel puts the beams together.
//
// Pass 1: a CTA takes a part of a row, in steps of 256 threads x 32 values.  A thread keeps its own m and l
// with one rescaling a step.  What may still be among the best is told by a threshold: k lists whose best
// reach it hold k values that do, so the k-th largest of the lists' maxima (a list: what some threads
// have seen in this step, or what has been kept so far) is one, and no more than k lists have
// values above it.  Values that pass are appended to a buffer in shared memory, and the k best of it are found by
// counting how many are better.  Equal logits go by index: the keys are (value, index) in 64 bits, all
// different, so however the values lie the buffer holds what comes.
//
// Bound by HBM (the logits are read once) where rows are many; by latency where they are few.

constexpr int kThreads = 256;
constexpr int kVec = 4;                   // 16-byte loads of a thread and step
constexpr unsigned kAll = 0xffffffffu;

// Order-preserving images of floats (larger float, larger image; NaN as -inf, -0 as 0).
__device__ __forceinline__ uint32_t image(float x) {
  if (x != x) x = -CUDART_INF_F;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ uint64_t key_of(float x, int index) { return (uint64_t)image(x) << 32 | (uint32_t)~index; }
__device__ __forceinline__ uint64_t image(double x) {
  if (x != x) x = -CUDART_INF;
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double value_of(uint64_t u) {
  return __longlong_as_double((long long)(u >> 63 ? u & ~(1ull << 63) : ~u));
}

template <typename T>
struct Logits;
template <>
struct Logits<float> {
  static constexpr int PER = 4;
  static __device__ __forceinline__ void unpack(const uint4 &v, float *x) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
};
template <>
struct Logits<__nv_bfloat16> {
  static constexpr int PER = 8;
  static __device__ __forceinline__ void unpack(const uint4 &v, float *x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
};

// The `top` largest of keys[0 .. count) to out[0 ..), largest first.
__device__ __forceinline__ void rank_keys(const uint64_t *keys, int count, uint64_t *out, int top) {
  for (int i = threadIdx.x; i < count; i += kThreads) {
    const uint64_t mine = keys[i];
    int better = 0;
    for (int j = 0; j < count; ++j) better += keys[j] > mine;
    if (better < top) out[better] = mine;
  }
}

constexpr float kLog2e = 1.4426950408889634f;

// ALIGNED: every row starts on a 16-byte boundary, and a thread's loads are 16 bytes; else they are single
// values, coalesced over the threads.  Which thread has which value is the same for all rows of a
// call, so that equal rows give equal sums.
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 3) beam_rows_kernel(BeamParams p) {
  constexpr int MOST = kVec * Logits<T>::PER;           // values of a thread and step
  constexpr int UNIT = ALIGNED ? Logits<T>::PER : 1;    // consecutive ones
  __shared__ uint64_t best[64];  // the best so far, largest first (0: none)
  __shared__ uint64_t heads[kThreads], sh_limit;
  __shared__ int sh_count;
  __shared__ float2 sums[kThreads / 32];
  extern __shared__ uint64_t buffer[];  // what may count: `kept` from before, then new ones
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / p.parts, part = blockIdx.x - row * p.parts, top = p.top;
  if (tid < 64) best[tid] = 0;
  if (tid == 0) sh_count = 0;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if ((p.finished && p.finished[row]) || !isfinite(p.scores[row])) return;  // (its logits do not count)
  const T *x = static_cast<const T *>(p.logits) + (long long)row * p.row_stride;
  const int units = (p.vocab + UNIT - 1) / UNIT;
  const int u0 = (int)((long long)units * part / p.parts), u1 = (int)((long long)units * (part + 1) / p.parts);
  const int lists = top <= 16 ? 32 : kThreads, per_list = kThreads / lists;  // (32 lists are enough for few)
  const int end = min(u1 * UNIT, p.vocab);
  float m = -CUDART_INF_F, l = 0.f;
  int kept = 0;
  __syncthreads();
  for (int base = u0; base < u1; base += kThreads * (MOST / UNIT)) {
    auto index = [&](int i) { return (base + (i / UNIT) * kThreads + tid) * UNIT + i % UNIT; };
    float y[MOST];
#pragma unroll
    for (int i = 0; i < MOST; i += UNIT) {
      const int at = index(i);
      if (ALIGNED && at + UNIT <= end) {
        Logits<T>::unpack(__ldcs(reinterpret_cast<const uint4 *>(x + at)), y + i);
      } else {
#pragma unroll
        for (int e = 0; e < UNIT; ++e) y[i + e] = at + e < end ? Elem<T>::load(x + at + e) : -CUDART_INF_F;
      }
    }
    float big = y[0];
#pragma unroll
    for (int i = 1; i < MOST; ++i) big = fmaxf(big, y[i]);
    // The differences are taken first: a product with log2 e less its own maximum's would put the
    // rounding of that maximum, up to 1e-6, into every power alike.
    const float m1 = fmaxf(m, big), ref = m1 == -CUDART_INF_F ? 0.f : m1;
    float sum = 0.f, sum2 = 0.f;
#pragma unroll
    for (int i = 0; i < MOST; i += 2) {
      sum += ex2((y[i] - ref) * kLog2e);
      sum2 += ex2((y[i + 1] - ref) * kLog2e);
    }
    l = l * ex2((m - ref) * kLog2e) + (sum + sum2);
    m = m1;

    // threads with a value that may count; with few of them all such values are taken
    const uint64_t last = best[top - 1];  // 0 while there are fewer
    const bool some = last == 0 || big >= value_of((uint32_t)(last >> 32));
    const int busy = __syncthreads_count(some);
    if (busy == 0) continue;
    uint64_t limit = last;
    if (busy > top) {
      uint64_t head = 0;
      if (some) {
#pragma unroll
        for (int i = 0; i < MOST; ++i)
          if (index(i) < end) head = max(head, key_of(y[i], index(i)));
      }
      for (int o = 1; o < per_list; o <<= 1) head = max(head, __shfl_xor_sync(kAll, head, o));
      if (tid % per_list == 0) heads[tid / per_list] = head;
      __syncthreads();
      if (tid < lists) {  // the top-th largest; 0 where fewer lists have a value
        const uint64_t mine = heads[tid];
        int better = 0;
        for (int j = 0; j < lists; ++j) better += heads[j] > mine;
        if (better < top && (better == top - 1 || mine == 0)) sh_limit = mine;
      }
      __syncthreads();
      limit = max(limit, sh_limit);
    }
    if (some) {
#pragma unroll
      for (int i = 0; i < MOST; ++i) {
        const uint64_t key = key_of(y[i], index(i));
        if (index(i) < end && key >= limit) buffer[kept + atomicAdd(&sh_count, 1)] = key;
      }
    }
    __syncthreads();
    const int total = kept + sh_count;
    if (total > kept) {
      rank_keys(buffer, total, best, top);
      kept = min(top, total);
      __syncthreads();
      if (tid < kept) buffer[tid] = best[tid];
      if (tid == 0) sh_count = 0;
    }
  }
  // the part's maximum, sum of powers and best
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(kAll, m, o), l2 = __shfl_xor_sync(kAll, l, o), m1 = fmaxf(m, m2);
    const float ref = m1 == -CUDART_INF_F ? 0.f : m1;
    l = l * ex2((m - ref) * kLog2e) + l2 * ex2((m2 - ref) * kLog2e);
    m = m1;
  }
  if (lane == 0) sums[warp] = make_float2(m, l);
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kThreads / 32; ++i) m = fmaxf(m, sums[i].x);
    const float ref = m == -CUDART_INF_F ? 0.f : m;
    l = 0.f;
    for (int i = 0; i < kThreads / 32; ++i) l += sums[i].y * ex2((sums[i].x - ref) * kLog2e);
    p.sums[blockIdx.x] = make_float2(m, l);
  }
  if (tid < top) p.keys[(long long)blockIdx.x * top + tid] = best[tid];
}

// A continuation by its score and its place w V + x: larger scores first, then smaller places.
struct Cand {
  uint64_t score;
  uint32_t place;
};
__device__ __forceinline__ bool better(const Cand &a, const Cand &b) {
  return a.score > b.score || (a.score == b.score && a.place < b.place);
}

// Pass 2: a request.  Each (beam, part) list is in order, so the top-th best of the lists' heads bounds what
// counts, and the lists are walked down to it.
constexpr int kHeads = 4096;  // lists whose heads are kept
__global__ void __launch_bounds__(kThreads) beam_join_kernel(BeamParams p) {
  __shared__ double shift[64];     // score_w - lse_w: what a logit's score adds; NaN: see kind
  __shared__ int kind[64];         // 0: as the logits say; 1: every continuation -inf; 2: finished
  __shared__ Cand bound;
  __shared__ int count;
  extern __shared__ uint64_t raw[];
  const int tid = threadIdx.x, group = blockIdx.x, w_n = p.beams, parts = p.parts, top = p.top;
  const int lists = w_n * parts;
  Cand *heads = reinterpret_cast<Cand *>(raw);        // [lists]
  Cand *pool = heads + lists;                         // [top * top]
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (tid == 0) count = 0;
  for (int w = tid >> 5; w < w_n; w += kThreads / 32) {  // a warp a beam
    const int row = group * w_n + w, lane = tid & 31;
    float m = -CUDART_INF_F;
    for (int i = lane; i < parts; i += 32) m = fmaxf(m, p.sums[(long long)row * parts + i].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    const float r = m == -CUDART_INF_F ? 0.f : m;
    double l = 0.0;
    for (int i = lane; i < parts; i += 32) {
      const float2 s = p.sums[(long long)row * parts + i];
      l += (double)s.y * exp((double)s.x - (double)r);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kAll, l, o);
    if (lane == 0) {
      const float score = p.scores[row];
      const bool done = p.finished && p.finished[row];
      shift[w] = done ? (double)score : (double)score - ((double)m + log(l));
      kind[w] = done ? 2 : isfinite(score) && l > 0.0 && isfinite(l) && isfinite(m) ? 0 : 1;
    }
  }
  __syncthreads();
  // entry i of list (w, part)
  auto entry = [&](int list, int i, Cand &c) {
    const int w = list / parts, part = list - w * parts;
    const uint32_t base = (uint32_t)w * (uint32_t)p.vocab;
    if (kind[w] == 0) {
      const uint64_t key = p.keys[((long long)group * lists + list) * top + i];
      if (key == 0) return false;
      c = Cand{image(shift[w] + (double)value_of((uint32_t)(key >> 32))), base + ~(uint32_t)key};
      return true;
    }
    if (part > 0) return false;  // in order of the token, a finished beam's own before them
    if (kind[w] == 2) {
      if (i == 0) {
        c = Cand{image(shift[w]), base + (uint32_t)p.pad_token};
        return true;
      }
      i = i - 1 < p.pad_token ? i - 1 : i;
      if (i >= p.vocab) return false;
    }
    c = Cand{image(-CUDART_INF), base + (uint32_t)i};
    return true;
  };
  for (int i = tid; i < lists; i += kThreads)
    if (!entry(i, 0, heads[i])) heads[i] = Cand{0, ~0u};
  if (tid == 0) bound = Cand{0, ~0u};
  __syncthreads();
  if (lists > top) {
    for (int i = tid; i < lists; i += kThreads) {
      const Cand mine = heads[i];
      int b = 0;
      for (int j = 0; j < lists; ++j) b += better(heads[j], mine);
      if (b == top - 1 && mine.score != 0) bound = mine;
    }
    __syncthreads();
  }
  for (int i = tid; i < lists; i += kThreads) {
    Cand c = heads[i];
    for (int e = 0; c.score != 0 && !better(bound, c);) {
      pool[atomicAdd(&count, 1)] = c;
      if (++e == top || !entry(i, e, c)) break;
    }
  }
  __syncthreads();
  const int n = count;
  for (int i = tid; i < n; i += kThreads) {
    const Cand mine = pool[i];
    int b = 0;
    for (int j = 0; j < n; ++j) b += better(pool[j], mine);
    if (b < top) {
      const long long at = (long long)group * top + b;
      p.scores_out[at] = (float)value_of(mine.score);
      p.parents[at] = (int)(mine.place / (uint32_t)p.vocab);
      p.tokens[at] = (int)(mine.place % (uint32_t)p.vocab);
    }
  }
}

// Parts of a row: enough CTAs to fill the GPU three times over, of a step at least, and no more lists
// a request than the join keeps.
int parts_of(int rows, int beams, int vocab, int step) {
  const int most = std::max(1, std::min(vocab / step, kHeads / beams));
  const int fill = (int)((3LL * 3 * kSms + rows - 1) / std::max(rows, 1));
  return std::max(1, std::min(most, fill));
}

// ------------------------------------------------------------------ reordering
//
// Thread by thread: a thread has one 16-byte (or 4-byte) column of all W rows of a (layer, request).  It
// copies what moves into its own column of shared memory, then writes the rows that change.  No
// thread reads what another writes, so the rows may be in place whatever the parents are.
template <typename U>
__global__ void __launch_bounds__(128) reorder_kernel(ReorderParams p) {
  extern __shared__ __align__(16) uint8_t stage_raw[];
  U *stage = reinterpret_cast<U *>(stage_raw);
  __shared__ int from[64];
  const int tid = threadIdx.x, w_n = p.beams;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const long long item = blockIdx.x / p.blocks;  // (layer, request)
  const int block = (int)(blockIdx.x - item * p.blocks), group = (int)(item % p.groups);
  if (tid < w_n) {
    const int f = p.parents[(long long)group * w_n + tid];
    from[tid] = f < 0 || f >= w_n ? tid : f;
  }
  __syncthreads();
  uint64_t need = 0;
  for (int w = 0; w < w_n; ++w)
    if (from[w] != w) need |= 1ull << from[w];
  if (need == 0) return;
  const long long per_row = p.row_bytes / (long long)sizeof(U);
  U *rows = reinterpret_cast<U *>(p.rows) + item * w_n * per_row;
  const long long col = (long long)block * 128 + tid;
  if (col >= per_row) return;
  for (int w = 0; w < w_n; ++w)
    if (need >> w & 1) {
      if (sizeof(U) == 16) cp_async16(stage + w * 128 + tid, rows + w * per_row + col, 16);
      else cp_async4(stage + w * 128 + tid, rows + w * per_row + col, 4);
    }
  cp_async_commit();
  asm volatile("cp.async.wait_all;\n" ::: "memory");
  for (int w = 0; w < w_n; ++w)
    if (from[w] != w) rows[w * per_row + col] = stage[from[w] * 128 + tid];
}

template <typename T, bool ALIGNED>
cudaError_t select(const BeamParams &p, cudaStream_t stream) {
  const size_t lists = (size_t)p.top * (p.top <= 16 ? kThreads / 32 : 1);  // threads whose values may all count
  const size_t rows = sizeof(uint64_t) * (lists * kVec * Logits<T>::PER + p.top);
  const size_t join = sizeof(Cand) * ((size_t)p.beams * p.parts + (size_t)p.top * p.top);
  static std::atomic<uint64_t> allowed{0}, allowed2{0};
  cudaError_t err = allow_smem(beam_rows_kernel<T, ALIGNED>, 64 * 1024, allowed);
  if (err == cudaSuccess) err = allow_smem(beam_join_kernel, 160 * 1024, allowed2);
  if (err == cudaSuccess)
    err = launch_dependent(beam_rows_kernel<T, ALIGNED>, (unsigned)(p.groups * p.beams * p.parts), kThreads, rows, stream, 1, p);
  if (err != cudaSuccess) return err;
  return launch_dependent(beam_join_kernel, (unsigned)p.groups, kThreads, join, stream, 1, p);
}
template <typename T>
cudaError_t by_alignment(const BeamParams &p, cudaStream_t stream) {
  const bool aligned = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 && p.row_stride % (16 / (int)sizeof(T)) == 0;
  return aligned ? select<T, true>(p, stream) : select<T, false>(p, stream);
}

}  // namespace

int beam_parts(int groups, int beams, int vocab, bool bf16) {
  return parts_of(groups * beams, beams, vocab, kThreads * kVec * (bf16 ? 8 : 4));
}

cudaError_t launch_beam_select(const BeamParams &p, gdn_dtype dtype, cudaStream_t stream) {
  return dtype == GDN_BF16 ? by_alignment<__nv_bfloat16>(p, stream) : by_alignment<float>(p, stream);
}

cudaError_t launch_beam_reorder(const ReorderParams &given, cudaStream_t stream) {
  ReorderParams p = given;
  const bool wide = p.row_bytes % 16 == 0 && reinterpret_cast<uintptr_t>(p.rows) % 16 == 0;
  const size_t smem = (size_t)p.beams * 128 * (wide ? 16 : 4);
  const long long cols = p.row_bytes / (wide ? 16 : 4);
  p.blocks = (cols + 127) / 128;
  const long long grid = p.blocks * p.layers * p.groups;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  static std::atomic<uint64_t> allowed{0};
  if (!wide) return launch_dependent(reorder_kernel<uint32_t>, (unsigned)grid, 128, smem, stream, 1, p);
  const cudaError_t err = allow_smem(reorder_kernel<uint4>, 128 * 1024, allowed);
  return err != cudaSuccess ? err : launch_dependent(reorder_kernel<uint4>, (unsigned)grid, 128, smem, stream, 1, p);
}

}  // namespace gdn
