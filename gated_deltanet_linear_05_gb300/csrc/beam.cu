// Several beams of a request: the selection of their best continuations over beams and vocabulary, and the
// reordering of the rows that follow them.
#include <algorithm>

#include "attn_tma.cuh"
#include "beam.h"

namespace gdn {
namespace {

// ------------------------------------------------------------------ selection
//
// s(w, x) = score_w + (logit_wx - m_w) - ln l_w, with m_w the row's maximum and l_w its sum of exp(logit - m_w).  Within a
// beam the order is the logits', so one pass over a row finds its maximum, its sum of powers and its `top` best
// logits without the sum being known; the second kernel puts the beams together.
//
// Pass 1: a CTA takes a part of a row, in steps of 256 threads x MOST values, the next step's loads under way
// while this one's are looked at.  Each step has its own maximum and sum of powers, in an order that does not go by the
// parts, so that a request's scores are the same to the bit in any batch: the threads' go to shared memory, and eight
// steps' at a time are put together by a warp each (64 x 8 rows of 150001 57.4 -> 58.9 us; by shuffles in each step 61.7).
// What may still be among the best is told by a limit: once `top` are kept the last of them, and where more threads
// than that reach it, a value that at least `top` threads' largest reach, found by halving the range of their largest
// (a barrier that counts for each halving; some 8 of them in a part's first step, seldom any later).  Values that
// pass are appended to a buffer in shared memory, and the k best of it found by counting how many are better.
// Equal logits go by index: the keys there are (value, index) in 64 bits, all different.  Where equal values
// pass in numbers that the buffer does not hold, the limit is the top-th largest of the threads' largest keys, which
// no more than `top` threads have values above.
//
// Bound by HBM (the logits are read once) where rows are many; by latency where they are few.

constexpr int kThreads = 256;
constexpr int kSumSteps = kThreads / 32;  // whose sums are put together at a time
constexpr unsigned kAll = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;

// The largest of a warp's floats, NaN apart.
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(r) : "f"(x));
  return r;
}

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

// A thread's values of a step: 16-byte units as loaded, where every row starts on a 16-byte boundary; else single
// values, coalesced over the threads.  Which thread has which value is the same for all rows of a call, so that
// equal rows give equal sums.
template <typename T, bool ALIGNED, int VEC>
struct Values {
  static constexpr int PER = 16 / (int)sizeof(T);
  static constexpr int MOST = VEC * PER, UNIT = ALIGNED ? PER : 1;  // values, consecutive ones
  uint32_t w[ALIGNED ? VEC * 4 : MOST];

  static __device__ __forceinline__ int index(int base, int i) {
    return base + ((i / UNIT) * kThreads + (int)threadIdx.x) * UNIT + i % UNIT;
  }
  // those from `base` on of x[0 .. end), -inf beyond
  __device__ __forceinline__ void load(const T *x, int base, int end) {
    if (base + MOST * kThreads <= end) {
      const T *mine = x + base + threadIdx.x * UNIT;
#pragma unroll
      for (int i = 0; i < MOST; i += UNIT) {
        if (ALIGNED) {
          const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(mine + i * kThreads));
          uint32_t *to = w + i / UNIT * 4;
          to[0] = v.x, to[1] = v.y, to[2] = v.z, to[3] = v.w;
        } else {
          w[i] = __float_as_uint(Elem<T>::load(mine + i * kThreads));
        }
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < MOST; i += UNIT) {
      const int at = index(base, i);
      if (ALIGNED && at + UNIT <= end) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(x + at));
        uint32_t *to = w + i / UNIT * 4;
        to[0] = v.x, to[1] = v.y, to[2] = v.z, to[3] = v.w;
      } else if (!ALIGNED) {
        w[i] = __float_as_uint(at < end ? Elem<T>::load(x + at) : -CUDART_INF_F);
      } else if (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < UNIT; ++e)
          w[i + e] = __float_as_uint(at + e < end ? Elem<T>::load(x + at + e) : -CUDART_INF_F);
      } else {
#pragma unroll
        for (int e = 0; e < UNIT; e += 2) {
          const float lo = at + e < end ? Elem<T>::load(x + at + e) : -CUDART_INF_F;
          const float hi = at + e + 1 < end ? Elem<T>::load(x + at + e + 1) : -CUDART_INF_F;
          w[(i + e) / 2] = __float_as_uint(lo) >> 16 | (__float_as_uint(hi) & 0xffff0000u);
        }
      }
    }
  }
  __device__ __forceinline__ float operator[](int i) const {
    if (!ALIGNED || sizeof(T) == 4) return __uint_as_float(w[i]);
    return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
};

// The `top` largest of keys[0 .. count) to out[0 ..), largest first.
__device__ __forceinline__ void rank_keys(const uint64_t *keys, int count, uint64_t *out, int top) {
  for (int i = threadIdx.x; i < count; i += kThreads) {
    const uint64_t mine = keys[i];
    int better = 0;
#pragma unroll 4
    for (int j = 0; j < count; ++j) better += keys[j] > mine;
    if (better < top) out[better] = mine;
  }
}

// A value that at least `top` threads' reach, and not many more if it can be helped: `mine` of the threads that take
// part (0 for the others), of which there are `top` at least.
template <int WARPS>
__device__ __forceinline__ uint32_t common_limit(uint32_t mine, int top, uint32_t (&sh)[2][WARPS]) {
  const uint32_t big = __reduce_max_sync(kAll, mine), small = __reduce_min_sync(kAll, mine == 0 ? ~0u : mine);
  if ((threadIdx.x & 31) == 0) sh[0][threadIdx.x >> 5] = big, sh[1][threadIdx.x >> 5] = small;
  __syncthreads();
  uint32_t lo = ~0u, hi = 0;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) hi = max(hi, sh[0][i]), lo = min(lo, sh[1][i]);
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo + 1) / 2;
    const int count = __syncthreads_count(mine >= mid);
    if (count >= top) lo = mid;
    else hi = mid - 1;
    if (count >= top && count <= top + top / 2 + 8) break;
  }
  return lo;
}

template <typename T, bool ALIGNED, int VEC>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && ALIGNED ? 3 : 4) beam_rows_kernel(BeamParams p) {
  using V = Values<T, ALIGNED, VEC>;
  constexpr int MOST = V::MOST, STEP = MOST * kThreads;
  __shared__ uint64_t best[64];  // the best so far, largest first
  __shared__ uint64_t heads[kThreads], sh_limit;
  __shared__ uint32_t sh_range[2][kThreads / 32];
  __shared__ int sh_count;
  extern __shared__ uint64_t buffer[];  // what may count: `kept` from before, then new ones
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / p.parts, part = blockIdx.x - row * p.parts, top = p.top, room = top * MOST;
  if (tid < 64) best[tid] = 0;
  if (tid == 0) sh_count = 0;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if ((p.finished && p.finished[row]) || !isfinite(p.scores[row])) return;  // (its logits do not count)
  const T *x = static_cast<const T *>(p.logits) + (long long)row * p.row_stride;
  const int steps = p.steps;  // of the row: parts take whole ones
  const int from = (int)((long long)steps * part / p.parts) * STEP;
  const int end = (int)min((long long)((long long)steps * (part + 1) / p.parts) * STEP, (long long)p.vocab);
  int kept = 0, late = 0;  // kept: in order; late: threads (at most) that have appended since
  float last = 0.f;        // of the `top` that are kept
  // The best of what is kept and what has been appended; after a barrier, and ends with one.
  auto settle = [&]() {
    const int total = kept + sh_count;
    if (total > kept) rank_keys(buffer, total, best, top);
    kept = min(top, total);
    late = 0;
    __syncthreads();
    if (tid < kept) buffer[tid] = best[tid];
    if (tid == 0) sh_count = 0;
    last = kept == top ? value_of((uint32_t)(best[top - 1] >> 32)) : 0.f;
    __syncthreads();
  };
  float2 *sums = reinterpret_cast<float2 *>(buffer + top * (MOST + 1));  // [kSumSteps + 1][kThreads], in turn: the step after those that are read has one of its own
  // The sums of up to kSumSteps steps of the row, to `step`; after its barrier.
  auto put_sums = [&](int step) {
    const int mine = step / kSumSteps * kSumSteps + warp;
    if (mine > step || mine * STEP < from) return;
    const float2 *of = sums + mine % (kSumSteps + 1) * kThreads + lane;
    float m = of[0].x;
#pragma unroll 4
    for (int i = 1; i < kThreads / 32; ++i) m = fmaxf(m, of[32 * i].x);
    m = warp_max(m);
    const float ref = m == -CUDART_INF_F ? 0.f : m;
    float l = 0.f;
#pragma unroll 4
    for (int i = 0; i < kThreads / 32; ++i) l = fmaf(of[32 * i].y, ex2((of[32 * i].x - ref) * kLog2e), l);
#pragma unroll 4
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kAll, l, o);
    if (lane == 0) p.sums[(long long)row * steps + mine] = make_float2(m, l);
  };
  V y, ahead;
  ahead.load(x, from, end);
  __syncthreads();
#pragma unroll 1
  for (int base = from; base < end; base += STEP) {
    y = ahead;
    if (base + STEP < end) ahead.load(x, base + STEP, end);
    float big = y[0];
#pragma unroll
    for (int i = 1; i < MOST; ++i) big = fmaxf(big, y[i]);
    // The differences are taken first: a product with log2 e less its own maximum's would put the
    // rounding of that maximum, up to 1e-6, into every power alike.
    const int step = base / STEP;
    const float ref = big == -CUDART_INF_F ? 0.f : big;
    float sum[4];
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      const float e = ex2((y[i] - ref) * kLog2e);
      sum[i % 4] = i < 4 ? e : sum[i % 4] + e;
    }
    sums[step % (kSumSteps + 1) * kThreads + tid] = make_float2(big, (sum[0] + sum[1]) + (sum[2] + sum[3]));

    // Threads with a value that may count.  Equal ones from here on come after those that are kept.
    auto may = [&]() { return kept < top ? V::index(base, 0) < end : big > last; };
    int busy = __syncthreads_count(may());
    if (step % kSumSteps == kSumSteps - 1) put_sums(step);
    if (busy == 0) continue;
    if (late > 0 && late + busy > top) {  // (the buffer holds all values of `top` threads)
      settle();
      busy = __syncthreads_count(may());
      if (busy == 0) continue;
    }
    const bool some = may();
    float limit = -CUDART_INF_F;
    if (busy > top) limit = value_of(common_limit(some ? image(big) : 0u, top, sh_range));
    if (some && big >= limit) {
      uint32_t bits = 0;
#pragma unroll
      for (int i = 0; i < MOST; ++i) bits |= y[i] >= limit && (kept < top || y[i] > last) ? 1u << i : 0u;
      const bool alone = (bits & (bits - 1)) == 0;  // (then it is the largest; else they are read again)
      for (; bits; bits &= bits - 1) {
        const int at = V::index(base, __ffs(bits) - 1);
        if (at >= end) break;
        const int to = atomicAdd(&sh_count, 1);
        if (to < room) buffer[kept + to] = key_of(alone ? big : Elem<T>::load(x + at), at);
      }
    }
    late += busy;
    if (busy <= top) continue;
    __syncthreads();
    if (sh_count > room) {  // (by so many equal values)
      __syncthreads();
      uint64_t head = 0;
      if (some) {
#pragma unroll 1
        for (int i = 0; i < MOST; ++i) {
          const int at = V::index(base, i);
          if (at < end) head = max(head, key_of(Elem<T>::load(x + at), at));
        }
      }
      heads[tid] = head;
      if (tid == 0) sh_count = 0;
      __syncthreads();
      int better = 0;
      for (int j = 0; j < kThreads; ++j) better += heads[j] > head;
      // the top-th largest; 0 where fewer threads have a value
      if (better < top && (better == top - 1 || head == 0)) sh_limit = head;
      __syncthreads();
      if (some && head >= sh_limit) {
#pragma unroll 1
        for (int i = 0; i < MOST; ++i) {
          const int at = V::index(base, i);
          const uint64_t key = at < end ? key_of(Elem<T>::load(x + at), at) : 0;
          if (key >= sh_limit && key > (kept == top ? best[top - 1] : 0)) buffer[kept + atomicAdd(&sh_count, 1)] = key;
        }
      }
      __syncthreads();
    }
    settle();
  }
  const int last_step = (end - 1) / STEP;
  if (last_step % kSumSteps != kSumSteps - 1) put_sums(last_step);
  __syncthreads();
  if (late > 0) settle();
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

// Pass 2: a request.  The (beam, part) lists are in order.  Their first entries, up to kSample of them, tell a score
// that at least `top` reach and not many more, found by halving: first by threads' largest, then by all.  What
// reaches it, and what follows in lists whose sampled entries all do, is ranked by counting.  The halving is done on
// scores in float32, less what their rounding may make of them; only what passes gets its score in float64 (slow on
// this GPU).
constexpr int kLists = 4096;   // lists of a request at most
constexpr int kSample = 4096;
constexpr int kRoom = kLists;  // what may pass, but for equal scores: no less than 64 entries of 64 lists

// sampled entries of a list
__host__ __device__ constexpr int sampled_of(int lists, int top) {
  const int most = kSample / lists > 1 ? kSample / lists : 1;
  return top < most ? top : most;
}

// ln(a + b), b small beside a > 0, to 2^-28: a = 2^e f with f in [1/sqrt 2, sqrt 2), ln f = 2 artanh(s) with
// s = (f - 1) / (f + 1), |s| < 0.172; s in two floats, its series from s^3 on (to s^11) in one.
__device__ __forceinline__ double log_of(float a, float b) {
  const int e = (__float_as_int(a) - 0x3f3504f3) >> 23;
  const float scale = __int_as_float((127 - e) << 23), f = a * scale, g = b * scale;
  const float x = f - 1.f, y = f + 1.f, y_low = f - (y - 1.f);  // (x is exact; y + y_low = f + 1)
  const float s = x / y;
  const float low = (fmaf(-s, y, x) + (g - s * (g + y_low))) / y;
  const float q = s * s;
  const float tail = s * q * fmaf(q, fmaf(q, fmaf(q, fmaf(q, 1.f / 11, 1.f / 9), 1.f / 7), 1.f / 5), 1.f / 3);
  return (double)e * 0.693147180559945309 + 2.0 * ((double)s + (double)(low + tail));
}

__device__ __forceinline__ uint64_t pick(const uint64_t (&x)[8], int i) {
  uint64_t r = x[0];
#pragma unroll
  for (int k = 1; k < 8; ++k) r = i == k ? x[k] : r;
  return r;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) beam_join_kernel(BeamParams p) {
  __shared__ double ln_sum[64];   // of a beam (dead or finished: 0)
  __shared__ float peak[64];      // its largest logit (dead or finished: 0)
  __shared__ float score_of[64];  // (dead: 0)
  __shared__ float shift[64];     // score less ln_sum, for the bound
  __shared__ int kind[64];      // 0: as the logits say; 1: every continuation -inf; 2: finished
  __shared__ uint32_t sh_range[2][THREADS / 32];
  __shared__ Cand sh_bound;
  __shared__ int sh_count, sh_sum[3], sh_widest;  // widest: the largest |shift|, as its float's bits
  extern __shared__ uint64_t raw[];
  const int tid = threadIdx.x, group = blockIdx.x, w_n = p.beams, parts = p.parts, top = p.top;
  const int lists = w_n * parts, deep = sampled_of(lists, top);
  Cand *found = reinterpret_cast<Cand *>(raw);  // [kRoom]
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (tid == 0) sh_count = sh_widest = sh_sum[0] = sh_sum[1] = sh_sum[2] = 0;
  __syncthreads();
  // Beams' sums, by threads enough for four steps each (32 at most): what is added in which order goes by the steps
  // alone, not by the threads that the kernel has.
  const int steps = p.steps;
  const int log_per = steps <= 16 ? 2 : steps <= 32 ? 3 : steps <= 64 ? 4 : 5, per = 1 << log_per, turn = tid & (per - 1);
#pragma unroll 1
  for (int w0 = 0; w0 < w_n; w0 += THREADS >> log_per) {
    const int w = w0 + (tid >> log_per), row = group * w_n + w;
    const float2 *sums = p.sums + (long long)row * steps;
    const bool here = w < w_n;
    const float score = here ? p.scores[row] : 0.f;
    const bool done = here && isfinite(score) && p.finished && p.finished[row];
    float m = -CUDART_INF_F;
    float2 some[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = turn + u * per;
      some[u] = here && i < steps ? sums[i] : make_float2(-CUDART_INF_F, 0.f);
      m = fmaxf(m, some[u].x);
    }
#pragma unroll 4
    for (int i = turn + 4 * per; here && i < steps; i += per) m = fmaxf(m, sums[i].x);
#pragma unroll 1
    for (int o = 1; o < per; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    const float ref = m == -CUDART_INF_F ? 0.f : m;
    float l = 0.f, low = 0.f;  // the sum in two floats
    auto add = [&](float x) {
      const float y = l + x, z = y - l;
      low += (l - (y - z)) + (x - z);
      l = y;
    };
#pragma unroll
    for (int u = 0; u < 4; ++u) add(some[u].y * ex2((some[u].x - ref) * kLog2e));
#pragma unroll 1
    for (int i = turn + 4 * per; here && i < steps; i += per) {
      const float2 s = sums[i];
      add(s.y * ex2((s.x - ref) * kLog2e));
    }
#pragma unroll 1
    for (int o = 1; o < per; o <<= 1) {
      const float x = __shfl_xor_sync(kAll, l, o), y = __shfl_xor_sync(kAll, low, o);
      // (both sides add the same two in the same order)
      const bool first = (tid & o) == 0;
      const float a = first ? l : x, b = first ? x : l, sum = a + b, z = sum - a;
      low = low + y + ((a - (sum - z)) + (b - z));
      l = sum;
    }
    if (here && turn == 0) {
      const bool alive = isfinite(score) && l > 0.f && isfinite(l) && isfinite(m);
      const double ln = alive && !done ? log_of(l, low) : 0.0;
      ln_sum[w] = ln;
      peak[w] = alive && !done ? m : 0.f;
      score_of[w] = done || alive ? score : 0.f;
      shift[w] = (float)((double)score_of[w] - ln);
      kind[w] = done ? 2 : alive ? 0 : 1;
      atomicMax(&sh_widest, __float_as_int(fabsf(shift[w])));
    }
  }
  __syncthreads();
  // entry i of list (w, part), whose key (where its logits say) is `key`: its logit (a finished or dead
  // beam's: 0 or -inf) and its place
  const uint64_t *keys = p.keys + (long long)group * lists * top;
  auto entry = [&](int list, int i, uint64_t key, float &logit, uint32_t &place) {
    const int w = list / parts, part = list - w * parts;
    const uint32_t base = (uint32_t)w * (uint32_t)p.vocab;
    if (kind[w] == 0) {
      logit = value_of((uint32_t)(key >> 32));
      place = base + ~(uint32_t)key;
      return key != 0;
    }
    if (part > 0) return false;  // in order of the token, a finished beam's own before them
    logit = -CUDART_INF_F;
    if (kind[w] == 2) {
      if (i == 0) {
        logit = 0.f;
        place = base + (uint32_t)p.pad_token;
        return true;
      }
      i = i - 1 < p.pad_token ? i - 1 : i;
    }
    place = base + (uint32_t)i;
    return i < p.vocab;
  };
  // The maximum is taken off first: a row far from 0, as a mask of the lowest value leaves it, would swallow score and
  // logarithm.  (Difference and sum are exact but for far exponents, so that beams of equal rows tie where score and logit do.)
  auto exactly = [&](float logit, uint32_t place) {
    const int w = place / (uint32_t)p.vocab;
    return Cand{image(((double)score_of[w] + ((double)logit - (double)peak[w])) - ln_sum[w]), place};
  };
  auto about = [&](int list, float logit) {
    const int w = list / parts;
    return shift[w] + (logit - peak[w]);
  };
  // (loops stay rolled but for a few loads side by side: a kernel this short waits for its instructions)
  uint32_t *sample = reinterpret_cast<uint32_t *>(found + kRoom), most = 0;  // [kSample]
  const int sampled = lists * deep;
#pragma unroll 1
  for (int k = tid; k < sampled; k += 4 * THREADS) {
    uint64_t key[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int at = k + u * THREADS, list = at / deep;
      key[u] = at < sampled ? keys[(long long)list * top + (at - list * deep)] : 0;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int at = k + u * THREADS, list = at / deep;
      float logit;
      uint32_t place, score = 0;
      if (at >= sampled) break;
      if (entry(list, at - list * deep, key[u], logit, place)) score = image(about(list, logit));
      sample[at] = score;
      most = max(most, score);
    }
  }
  uint32_t lo = 0;
  if (__syncthreads_count(most != 0) > top) lo = common_limit(most, top, sh_range);
  auto reach = [&](uint32_t limit, int turn) {
    int count = 0;
#pragma unroll 4
    for (int k = tid; k < sampled; k += THREADS) count += sample[k] >= limit && sample[k] != 0;
    count = __reduce_add_sync(kAll, count);
    if ((tid & 31) == 0 && count) atomicAdd(&sh_sum[turn], count);
    __syncthreads();
    count = sh_sum[turn];
    if (tid == 0) sh_sum[turn == 0 ? 2 : turn - 1] = 0;  // (three counters in turn: this one is read, the next one free)
    return count;
  };
  const int enough = top + top / 2 + 32;
  if (reach(lo, 0) > enough) {
    most = __reduce_max_sync(kAll, most);
    if ((tid & 31) == 0) sh_range[0][tid >> 5] = most;
    __syncthreads();
    uint32_t hi = 0;
    for (int i = 0; i < THREADS / 32; ++i) hi = max(hi, sh_range[0][i]);
    for (int turn = 1; lo < hi; turn = turn == 2 ? 0 : turn + 1) {
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      const int count = reach(mid, turn);
      if (count >= top) lo = mid;
      else hi = mid - 1;
      if (count >= top && count <= enough) break;
    }
  }
  // (a score in float32 is off by three roundings of 2^-24, of shift, difference and sum: by 2^-23 (|score| + |shift|), which
  // both that of `low` and one at the bound may be, 2.4e-7 in all; 1e-13: float64's own, ln V 2^-53 at most)
  const float low = lo == 0 ? -CUDART_INF_F : value_of(lo);
  const float bound = low > -CUDART_INF_F ? low - (3.6e-7f * (fabsf(low) + __int_as_float(sh_widest)) + 1e-13f) : low;
  // What reaches the bound and is no worse than `least`.
  auto gather = [&](const Cand *least) {
    auto put = [&](float logit, uint32_t place) {
      const Cand c = exactly(logit, place);
      if (least && better(*least, c)) return;
      const int to = atomicAdd(&sh_count, 1);
      if (to < kRoom) found[to] = c;
    };
#pragma unroll 1
    for (int at = tid; at < sampled; at += THREADS) {
      if (sample[at] == 0 || value_of(sample[at]) < bound) continue;
      const int list = at / deep, first = at - list * deep;
      float logit;
      uint32_t place;
      entry(list, first, keys[(long long)list * top + first], logit, place);
      put(logit, place);
      if (first < deep - 1) continue;
#pragma unroll 1
      for (int e = deep, more = 1; more && e < top; e += 8) {
        uint64_t key[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) key[u] = e + u < top ? keys[(long long)list * top + e + u] : 0;
#pragma unroll 1
        for (int u = 0; u < 8 && e + u < top; ++u) {
          more = entry(list, e + u, pick(key, u), logit, place) && about(list, logit) >= bound;
          if (!more) break;
          put(logit, place);
        }
      }
    }
    __syncthreads();
    return sh_count;
  };
  int n = gather(nullptr);
  if (n > kRoom) {  // equal scores: bounded by the top-th best head itself
    __syncthreads();
    if (tid == 0) sh_count = 0, sh_bound = Cand{0, ~0u};
    for (int i = tid; i < lists; i += THREADS) {
      float logit;
      uint32_t place;
      found[i] = entry(i, 0, keys[(long long)i * top], logit, place) ? exactly(logit, place) : Cand{0, ~0u};
    }
    __syncthreads();
    for (int i = tid; i < lists; i += THREADS) {
      const Cand mine = found[i];
      int b = 0;
      for (int j = 0; j < lists; ++j) b += better(found[j], mine);
      if (b == top - 1 && mine.score != 0) sh_bound = mine;
    }
    __syncthreads();
    n = gather(&sh_bound);
  }
  for (int i = tid; i < n; i += THREADS) {
    const Cand mine = found[i];
    int b = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) b += better(found[j], mine);
    if (b < top) {
      const long long at = (long long)group * top + b;
      p.scores_out[at] = (float)value_of(mine.score);
      p.parents[at] = (int)(mine.place / (uint32_t)p.vocab);
      p.tokens[at] = (int)(mine.place % (uint32_t)p.vocab);
    }
  }
}

// Lists that are made of `rows` rows at most, whatever their length: eight waves of CTAs, which the cost below seldom wants
// more than, and two a row.  A workspace's size goes by this, not by the parts themselves: fewer rows have more
// parts each, and a workspace must do for them too.
long long most_lists(int rows, int slots) { return 2ll * rows + 8 * slots; }

// Parts of a row, each of whole steps: the number that by its cost ends first if `slots` CTAs run at a time, the last of
// them half a CTA's time longer than the rest, and a CTA's start and end take one and a half steps; no more lists a
// request than the join takes.  In 1, 2, ... parts: 64 x 8 rows of 150001 in f32 (37 steps) 61.6, 60.1, 55.8, 58.7,
// 62.7 us, of which it takes 4, not the best; 64 x 8 of 151936 in bf16 (19 steps) 55.6, 55.4, 60.5, of which 2; 4 x 48 of
// 99999 52.7, 45.7, 43.8, 50.1, of which 3; 2 x 4 of 32000 (4 steps) 11.9, 10.1, 9.3, 8.1, of which 4.  It does not
// go by where rows start: for bf16 it counts steps of 8192 tokens and three CTAs an SM, also where rows that start
// anywhere are read in steps of 4096 by four.
int parts_of(int rows, int beams, int vocab, int step, int slots) {
  const int steps = (vocab + step - 1) / step;
  const int most = std::min<long long>(std::min(steps, kLists / beams), most_lists(rows, slots) / std::max(rows, 1));
  int best = 1;
  float least = 0.f;
  for (int parts = 1; parts <= most; ++parts) {
    const float all = (float)rows / slots * (steps + 1.5f * parts);  // (grows with the parts)
    if (parts > 1 && all > least) break;
    const float cost = all + 0.5f * ((steps + parts - 1) / parts + 1.5f);
    if (parts == 1 || cost < least) best = parts, least = cost;
  }
  return best;
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

template <typename T, bool ALIGNED, int VEC>
cudaError_t select(const BeamParams &given, cudaStream_t stream) {
  constexpr int STEP = Values<T, ALIGNED, VEC>::MOST * kThreads;
  static_assert(STEP >= kBeamStep, "a place in the workspace for each step's sums");
  BeamParams p = given;
  p.steps = (p.vocab + STEP - 1) / STEP;
  auto rows_smem = [](int top) {
    return sizeof(uint64_t) * (size_t)top * (Values<T, ALIGNED, VEC>::MOST + 1) + sizeof(float2) * (kSumSteps + 1) * kThreads;
  };
  const size_t rows = rows_smem(p.top);
  constexpr size_t join = sizeof(Cand) * kRoom + sizeof(uint32_t) * kSample;
  const int lists = p.beams * p.parts;
  static std::atomic<uint64_t> allowed{0}, allowed_wide{0}, allowed_rows{0};
  // A CTA of 256 threads walks up to four sampled entries a thread as fast as one of 1024 (2 x 4 beams of 32000, 64 entries:
  // 8.1 against 9.3 us a call; 16 beams of 32000, 1024: 11.2, 11.8); with more it is slower (64 beams of 32000, 8 best,
  // 2048: 13.8, 12.7; 4 x 48 of 99999, 48 best, 4032: 50.7, 43.9).
  const bool wide = lists * sampled_of(lists, p.top) > 1024;
  cudaError_t err = wide ? allow_smem(beam_join_kernel<1024>, join, allowed_wide) : allow_smem(beam_join_kernel<256>, join, allowed);
  if (err == cudaSuccess) err = allow_smem(beam_rows_kernel<T, ALIGNED, VEC>, rows_smem(64), allowed_rows);
  if (err == cudaSuccess)
    err = launch_dependent(beam_rows_kernel<T, ALIGNED, VEC>, (unsigned)(p.groups * p.beams * p.parts), kThreads, rows, stream, 1, p);
  if (err != cudaSuccess) return err;
  return wide ? launch_dependent(beam_join_kernel<1024>, (unsigned)p.groups, 1024, join, stream, 1, p)
              : launch_dependent(beam_join_kernel<256>, (unsigned)p.groups, 256, join, stream, 1, p);
}
template <typename T>
cudaError_t by_alignment(const BeamParams &p, cudaStream_t stream) {
  const bool alone = p.groups * p.beams == 1;  // (its stride says nothing)
  const bool aligned = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 && (alone || p.row_stride % (16 / (int)sizeof(T)) == 0);
  // (single values of 16 bits take a register each: half as many)
  return aligned ? select<T, true, 4>(p, stream) : select<T, false, sizeof(T) == 2 ? 2 : 4>(p, stream);
}

}  // namespace

constexpr int step_of(bool bf16) { return kThreads * 4 * (bf16 ? 8 : 4); }
constexpr int slots_of(bool bf16) { return kSms * (bf16 ? 3 : 4); }

int beam_parts(int groups, int beams, int vocab, bool bf16) {
  return parts_of(groups * beams, beams, vocab, step_of(bf16), slots_of(bf16));
}
size_t beam_lists(int groups, int beams, int vocab, bool bf16) {
  const long long steps = (vocab + step_of(bf16) - 1) / step_of(bf16);
  return (size_t)std::min(groups * std::min(beams * steps, (long long)kLists), groups ? most_lists(groups * beams, slots_of(bf16)) : 0);
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
