// Attention of one token per sequence over the paged cache (decode): bound by reading every
// key and value once from HBM.
//
// The batch's key tiles of 64, over all sequences and kv-heads in a row, are dealt out to the
// CTAs in equal runs, so that ragged contexts load every SM alike; a run may begin and end
// inside a sequence.  A (sequence, kv-head) pair that lies in one run is finished there; else
// each run leaves a partial result (m, l, O) in the workspace and the CTA that arrives last
// joins them in the order of the keys.
//
// The G <= 16 query heads of a kv-head are the rows of m16n8k16 products.  A warp takes 16
// keys of each tile with a running maximum and sum of its own, so that the warps meet only
// at the end of a pair; with D = 256 a second set of warps takes the upper half of V's
// columns (and repeats the scores: the shared memory they are read from has the bandwidth to spare).
// One warp keeps a ring of K and V tiles full by TMA: 160 KB in flight per SM.
//
// 64 contexts of 255 to 8191 keys, 32 heads of 128 on 8: 170 us, 6.65 TB/s (98% of the copy rate).  Two
// contexts of 90k to 131k keys, 16 heads of 256 on 2: 79 us, 5.6 TB/s with 7 us of start and join.  One of
// 66k, 4 heads of 128 on 1: 20 us (its floor is 5).
#pragma once

#include <cuda.h>
#include <math_constants.h>

#include "attn.h"
#include "attn_tma.cuh"

namespace gdn {

constexpr int kTile = 64;  // keys

template <int D_>
struct StepCfg {
  static constexpr int D = D_;
  static constexpr int HALVES = D / 128;
  static constexpr int WARPS = 4 * HALVES;             // consumers
  static constexpr int THREADS = 32 * (WARPS + 1);
  static constexpr int CTAS = kSms * (D == 128 ? 2 : 1);
  static constexpr int UNIT = kTile * D * 2;           // bytes of a K or V tile
  static constexpr int STAGES = 5;
  static constexpr int CH = D / 64;
  static constexpr int RP = 132;                       // padded row of the join buffers (floats)
  static constexpr int R_BYTES = HALVES * 2 * 16 * RP * 4;
  static constexpr int Q_BYTES = 16 * D * 2;           // a pair's query rows
  static constexpr int SMEM = STAGES * UNIT + 2 * Q_BYTES + R_BYTES;
};

struct StepPlan {
  unsigned int *arrived;  // [CTAS] parts finished of the pair that begins in that CTA's run
  float *ml, *part;       // [2 CTAS][16] {m, l}, [2 CTAS][16][D]
  DenseRows dense;        // the results are left there instead of finished
  unsigned int *err;
};

__device__ __forceinline__ int seq_len(const AttnParams &p, int n) {
  return (int)min(max((long long)p.kv_lens[n], 0ll), (long long)p.max_pages * p.page_size);
}
__device__ __forceinline__ int tiles_of(int len) { return max(1, (len + kTile - 1) / kTile); }

// Byte offset of (row, col) in a tile of 64 rows: 64-column chunks in TMA's 128-byte swizzle.
__device__ __forceinline__ uint32_t sw_off(int row, int col) {
  return (uint32_t)((col >> 6) * (kTile * 128) + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4));
}

template <int D>
struct StepShared {
  using C = StepCfg<D>;
  uint64_t full[C::STAGES], empty[C::STAGES], q_full[2], q_empty[2];
  long long base;
  int dead, last, n, scan[C::WARPS + 1];
  float m[2][C::WARPS][16], l[C::WARPS][16];
};

// The run of worker `worker` of `workers` by its StepCfg<D>::THREADS threads (tid 0 ..), which have the
// named barriers `bar` and `bar` + 1.  `smem`: StepCfg<D>::SMEM bytes on a 1024-byte boundary.  `waited`: the
// work before this kernel is known to be complete.
template <int D>
__device__ __forceinline__ void step_role(const AttnParams &p, const StepPlan &w, const CUtensorMap &qmap,
                                          const CUtensorMap &kmap, const CUtensorMap &vmap, uint8_t *smem,
                                          StepShared<D> &sh, int tid, int worker, int workers, int bar, bool waited) {
  using C = StepCfg<D>;
  uint64_t *full = sh.full, *empty = sh.empty, *q_full = sh.q_full, *q_empty = sh.q_empty;
  uint8_t *ring = smem;
  uint8_t *sq = ring + C::STAGES * C::UNIT;
  float *sr = reinterpret_cast<float *>(sq + 2 * C::Q_BYTES);
  const int warp = uniform(tid >> 5), lane = tid & 31;
  const int G = p.hq / p.hkv;
  volatile int *dead = &sh.dead;
  if (tid == 0) {
    prefetch_map(&qmap);
    if (p.num_pages > 0) {  // else there are no such maps
      prefetch_map(&kmap);
      prefetch_map(&vmap);
    }
    for (int i = 0; i < C::STAGES; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], C::WARPS);
    for (int i = 0; i < 2; ++i) mbar_init(&q_full[i], 1), mbar_init(&q_empty[i], C::WARPS);
    mbar_fence_init();
    sh.dead = 0;
  }
  if (!waited) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  }
  // The run of this CTA: tiles [x0, x1) of all, and the sequence that x0 lies in.  A scan of
  // the sequences' tiles gives the total; with more sequences than threads a second one finds
  // the place.
  auto scan = [&](int n, int &tiles, long long &sum) {  // tiles before sequence n in the chunk, their sum
    tiles = n < p.num_seqs ? tiles_of(seq_len(p, n)) : 0;
    int s = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += v;
    }
    bar_sync(bar + 1, C::THREADS);
    if (lane == 31) sh.scan[warp] = s;
    bar_sync(bar + 1, C::THREADS);
    long long at = s - tiles;
    sum = 0;
#pragma unroll
    for (int i = 0; i <= C::WARPS; ++i) {
      at += i < warp ? sh.scan[i] : 0;
      sum += sh.scan[i];
    }
    return at;
  };
  long long all = 0, sum, at;
  int tiles;
  for (int n0 = 0; n0 < p.num_seqs; n0 += C::THREADS) {
    at = scan(n0 + tid, tiles, sum);
    all += sum;
  }
  const long long total = all * p.hkv;
  const long long ctas = min((long long)workers, total);
  if (worker >= ctas) return;
  const long long x0 = total * worker / ctas, x1 = total * (worker + 1) / ctas;
  for (long long n0 = 0, before = 0; n0 < p.num_seqs && before * p.hkv <= x0; n0 += C::THREADS, before += sum) {
    if (p.num_seqs > C::THREADS) at = scan((int)n0 + tid, tiles, sum);
    const long long first = (before + at) * p.hkv;
    if (tiles > 0 && first <= x0 && x0 < first + (long long)tiles * p.hkv) sh.n = (int)n0 + tid, sh.base = first;
  }
  bar_sync(bar + 1, C::THREADS);
  // This CTA's pairs in order: sequence, head, first and last + 1 key tile.
  struct Walk {
    int n, h, len, tiles, j0, j1, ahead;
    long long x;
  };
  auto start = [&]() {
    Walk k;
    k.n = sh.n;
    k.x = x0;
    k.len = seq_len(p, k.n);
    k.tiles = tiles_of(k.len);
    const long long rem = x0 - sh.base;
    k.h = (int)(rem / k.tiles);
    k.j0 = (int)(rem % k.tiles);
    k.j1 = (int)min((long long)k.tiles, k.j0 + (x1 - x0));
    k.ahead = k.n + 1 < p.num_seqs ? seq_len(p, k.n + 1) : 0;  // the next length is at hand when needed
    return k;
  };
  auto step = [&](Walk &k) {
    k.x += k.j1 - k.j0;
    if (k.x >= x1) return;
    if (++k.h == p.hkv) {
      k.h = 0;
      ++k.n;
      k.len = k.ahead;
      k.tiles = tiles_of(k.len);
      k.ahead = k.n + 1 < p.num_seqs ? seq_len(p, k.n + 1) : 0;
    }
    k.j0 = 0;
    k.j1 = (int)min((long long)k.tiles, x1 - k.x);
  };
  const float asl = p.scale == 0.f ? 1.f : fabsf(p.scale) * 1.4426950408889634f;
  const float flip = p.scale == 0.f ? 0.f : p.scale < 0.f ? -1.f : 1.f;
  uint32_t ld = 0, pairs = 0, turn = 0;  // tiles and pairs so far

  if (warp == C::WARPS) {
    // ---------------------------------------------------------------- loads
    const int box = min(p.page_size, kTile), boxes = kTile / box, lps = 31 - __clz(p.page_size);
    const int pi = lane / C::CH, ch = lane % C::CH;
    for (Walk k = start(); k.x < x1; step(k)) {
      if (k.len == 0) continue;
      const int32_t *table = p.page_table + (long long)k.n * p.max_pages;
      auto page_of = [&](int j) {
        const int key = j * kTile + pi * box;
        return pi < boxes && j < k.j1 && key < k.len ? table[key >> lps] : -1;
      };
      int next = page_of(k.j0);
      const uint32_t qb = pairs & 1;
      wait_bar(&q_empty[qb], ((pairs >> 1) & 1) ^ 1, dead, w.err);
      if (lane == 0) {
        mbar_arrive_expect_tx(&q_full[qb], (uint32_t)G * D * 2);
        for (int c = 0; c < C::CH; ++c)
          tma_load_3d(sq + qb * C::Q_BYTES + c * 2048, &qmap, c * 64, k.h * G, k.n, &q_full[qb]);
      }
      __syncwarp();
      ++pairs;
      for (int j = k.j0; j < k.j1; ++j) {
        const int key = j * kTile + pi * box;
        const bool on = pi < boxes && key < k.len;
        // (a page out of range reads as zeros)
        const int pg = (unsigned)next < (unsigned)p.num_pages ? next : p.num_pages;
        next = page_of(j + 1);
        const int count = __popc(__ballot_sync(0xffffffffu, on));
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++ld) {
          const uint32_t st = ld % C::STAGES;
          wait_bar(&empty[st], ((ld / C::STAGES) & 1) ^ 1, dead, w.err);
          if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)count * box * 128);
          __syncwarp();
          if (on)
            tma_4d(ring + st * C::UNIT + ch * (kTile * 128) + pi * box * 128, kv ? &vmap : &kmap, ch * 64,
                   key & (p.page_size - 1), k.h, pg, &full[st]);
        }
      }
    }
    if (*dead) __nanosleep(1000000);  // copies in flight land before shared memory is given up
    return;
  }

  // ------------------------------------------------------------------ scores, softmax, sums
  const int kg = warp & 3, hf = warp >> 2;
  const int gid = lane >> 2, tig = lane & 3;
  const int kr = kg * 16;                                       // this warp's keys in a tile
  const int nthr = 32 * C::WARPS;
  for (Walk k = start(); k.x < x1; step(k)) {
    const int n = k.n, h = k.h, len = k.len, j0 = k.j0, j1 = k.j1;
    const long long pair0 = k.x - j0;  // first tile of the pair
    // the pair's G query rows; what lies in the rows after them reaches no result
    const uint32_t qb = pairs & 1;
    const uint8_t *qs = sq + qb * C::Q_BYTES;
    if (len > 0) wait_bar(&q_full[qb], (pairs >> 1) & 1, dead, w.err);
    const int qrow = (lane & 7) + ((lane >> 3) & 1) * 8;
    auto q_frag = [&](uint32_t (&a)[4], int k) {
      const int c = k * 16 + (lane >> 4) * 8;
      ldsm_x4(a, qs + (c >> 6) * 2048 + qrow * 128 + ((((c >> 3) & 7) ^ (qrow & 7)) << 4));
    };
    uint32_t qa[D == 128 ? 8 : 1][4];
    if (D == 128)
#pragma unroll
      for (int k = 0; k < (D == 128 ? 8 : 1); ++k) q_frag(qa[k], k);
    float o[16][4] = {};
    float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};
    for (int j = j0; j < j1 && len > 0; ++j) {
      // scores of 16 rows and this warp's 16 keys
      uint32_t st = ld % C::STAGES;
      wait_bar(&full[st], (ld / C::STAGES) & 1, dead, w.err);
      const uint8_t *kt = ring + st * C::UNIT;
      float s[2][4] = {};
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t b[4];
        ldsm_x4(b, kt + sw_off(kr + (lane & 7) + (lane >> 4) * 8, k * 16 + ((lane >> 3) & 1) * 8));
        if (D == 128) {
          mma_bf16(s[0], qa[k & 7], b[0], b[1]);
          mma_bf16(s[1], qa[k & 7], b[2], b[3]);
        } else {
          uint32_t a[4];
          q_frag(a, k);
          mma_bf16(s[0], a, b[0], b[1]);
          mma_bf16(s[1], a, b[2], b[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
      ++ld;
      const int left = len - j * kTile - kr;  // live keys among the warp's 16
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[t][i] *= flip;
          if (t * 8 + 2 * tig + (i & 1) >= left) s[t][i] = -CUDART_INF_F;
        }
      float top[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        top[r] = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2)) * asl;
      }
      // the reference moves when it would rise by more than 8 (2^8 is far from overflow)
      if (__any_sync(0xffffffffu, (gid < G && top[0] > m[0] + 8.f) || (gid + 8 < G && top[1] > m[1] + 8.f))) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float m1 = fmaxf(m[r], top[r]);
          const float a = m1 == -CUDART_INF_F ? 1.f : ex2(m[r] - m1);
          m[r] = m1;
          l[r] *= a;
#pragma unroll
          for (int t = 0; t < 16; ++t) o[t][2 * r] *= a, o[t][2 * r + 1] *= a;
        }
      }
      uint32_t pa[4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float ref = m[r] == -CUDART_INF_F ? 0.f : m[r];
        float e[2][2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            e[t][i] = ex2(fmaf(s[t][2 * r + i], asl, -ref));
            l[r] += e[t][i];
          }
        pa[r] = pack_bf16(e[0][0], e[0][1]);
        pa[2 + r] = pack_bf16(e[1][0], e[1][1]);
      }
      // O += P V over the 16 keys; V rows past the last key count as zero whatever they hold
      st = ld % C::STAGES;
      wait_bar(&full[st], (ld / C::STAGES) & 1, dead, w.err);
      const uint8_t *vt = ring + st * C::UNIT;
      uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
      if (left < 16) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int k = 2 * tig + 8 * i;
          keep[i] = (k < left ? 0xffffu : 0u) | (k + 1 < left ? 0xffff0000u : 0u);
        }
      }
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        uint32_t b[4];
        ldsm_x4_t(b, vt + sw_off(kr + (lane & 7) + ((lane >> 3) & 1) * 8, hf * 128 + t * 16 + (lane >> 4) * 8));
        mma_bf16(o[2 * t], pa, b[0] & keep[0], b[1] & keep[1]);
        mma_bf16(o[2 * t + 1], pa, b[2] & keep[0], b[3] & keep[1]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
      ++ld;
    }

    if (len > 0) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_empty[qb]);
      ++pairs;
    }

    // Join the warps: one maximum per row, then each half of the key groups sums O in a buffer.
    // (The maxima are in two places by turns: a warp may be here while another still reads the
    // last pair's; everything else is written after the first barrier.)
    float (*sh_m)[16] = sh.m[turn];
    turn ^= 1;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (tig == 0) sh_m[warp][gid + 8 * r] = m[r];
    }
    bar_sync(bar, nthr);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = gid + 8 * r;
      const float top = fmaxf(fmaxf(sh_m[hf * 4][row], sh_m[hf * 4 + 1][row]),
                              fmaxf(sh_m[hf * 4 + 2][row], sh_m[hf * 4 + 3][row]));
      const float a = top == -CUDART_INF_F ? 0.f : ex2(m[r] - top);
      if (tig == 0) sh.l[warp][row] = l[r] * a;
#pragma unroll
      for (int t = 0; t < 16; ++t) o[t][2 * r] *= a, o[t][2 * r + 1] *= a;
    }
    float *buf = sr + (hf * 2 + (kg & 1)) * 16 * C::RP;
    auto put = [&](bool add) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (gid + 8 * r < G)
#pragma unroll
          for (int t = 0; t < 16; ++t) {
            float2 *at = reinterpret_cast<float2 *>(buf + (gid + 8 * r) * C::RP + 8 * t + 2 * tig);
            float2 v = make_float2(o[t][2 * r], o[t][2 * r + 1]);
            if (add) v.x += at->x, v.y += at->y;
            *at = v;
          }
    };
    if (kg >= 2) put(false);
    bar_sync(bar, nthr);
    if (kg < 2) put(true);
    bar_sync(bar, nthr);

    // a row of the pair: finished, or left for a join
    auto emit = [&](int r, float mm, float ll, const float (&v)[D / 32]) {
      if (w.dense.part) {
        const long long row = (long long)n * p.hq + h * G + r;
        if (lane == 0) *reinterpret_cast<float2 *>(w.dense.ml + 2 * row) = make_float2(mm, ll);
#pragma unroll
        for (int c = 0; c < D / 128; ++c)
          *reinterpret_cast<float4 *>(w.dense.part + row * D + 128 * c + 4 * lane) =
              make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
        return;
      }
      emit_row<D>(p, n, h * G + r, lane, mm, ll, v);
    };
    const bool whole = j0 == 0 && j1 == k.tiles;
    const long long slot = 2ll * worker + (j0 == 0);
    for (int r = warp; r < G; r += C::WARPS) {
      const float mm = seen_max(fmaxf(fmaxf(sh_m[0][r], sh_m[1][r]), fmaxf(sh_m[2][r], sh_m[3][r])), len > 0);
      const float ll = (sh.l[0][r] + sh.l[1][r]) + (sh.l[2][r] + sh.l[3][r]);
      float v[D / 32];
#pragma unroll
      for (int c = 0; c < D / 128; ++c) {
        const float *at = sr + c * 2 * 16 * C::RP + r * C::RP + 4 * lane;
        const float4 a = *reinterpret_cast<const float4 *>(at);
        const float4 b = *reinterpret_cast<const float4 *>(at + 16 * C::RP);
        v[4 * c] = a.x + b.x, v[4 * c + 1] = a.y + b.y, v[4 * c + 2] = a.z + b.z, v[4 * c + 3] = a.w + b.w;
      }
      if (whole) {
        emit(r, mm, ll, v);
      } else {
        if (lane == 0) *reinterpret_cast<float2 *>(w.ml + 2 * (slot * 16 + r)) = make_float2(mm, ll);
#pragma unroll
        for (int k = 0; k < D / 128; ++k)
          *reinterpret_cast<float4 *>(w.part + (slot * 16 + r) * D + 128 * k + 4 * lane) =
              make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
      }
    }
    if (!whole) {
      // The runs c0 .. c1 that the pair lies in (c owns tile x iff total c / ctas <= x < total (c + 1) / ctas).
      // Many parts are joined in two levels, groups of `size` runs (the last takes the rest) and then the
      // groups, whose sums replace their first run's: a part costs a row's join about 0.2 us, and one
      // sequence of 66k keys with one kv-head has 304.  A counter per group, of a run that lies inside the
      // pair, so that no other pair has it (a group has `size` runs at least); the pair's is c0's.
      const int c0 = (int)(((pair0 + 1) * ctas - 1) / total), c1 = (int)(((pair0 + k.tiles) * ctas - 1) / total);
      const int count = c1 - c0 + 1, size = count < 64 ? 8 : 16, groups = count < 16 ? 1 : count / size;
      const int g = min((worker - c0) / size, groups - 1), first = c0 + g * size;
      const int runs = g == groups - 1 ? count - g * size : size;
      auto last_of = [&](unsigned int *arrived, int all) {  // all threads, after their writes
        __threadfence();
        bar_sync(bar, nthr);
        if (tid == 0) {
          sh.last = atomicAdd(arrived, 1u) == (unsigned)(all - 1);
          if (sh.last) *arrived = 0;  // ready for the next call
        }
        bar_sync(bar, nthr);
        if (sh.last) __threadfence();
        return sh.last != 0;
      };
      // (the run that began the pair has slot 2 c0 + 1, the others 2 c)
      if (last_of(&w.arrived[groups > 1 ? first + 1 : c0], runs)) {
        for (int r = warp; r < G; r += C::WARPS) {
          float mm = -CUDART_INF_F, ll = 0.f, v[D / 32] = {};
          const long long own = (2ll * first + (g == 0)) * 16 + r;
          add_parts<D, 8>(mm, ll, v, w.ml, w.part, own, 0, 1, lane);
          add_parts<D, 8>(mm, ll, v, w.ml, w.part, (2ll * first + 2) * 16 + r, 32, runs - 1, lane);
          if (groups == 1) {
            emit(r, mm, ll, v);
          } else {
            if (lane == 0) *reinterpret_cast<float2 *>(w.ml + 2 * own) = make_float2(mm, ll);
#pragma unroll
            for (int c = 0; c < D / 128; ++c)
              *reinterpret_cast<float4 *>(w.part + own * D + 128 * c + 4 * lane) =
                  make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
          }
        }
        if (groups > 1 && last_of(&w.arrived[c0], groups)) {
          for (int r = warp; r < G; r += C::WARPS) {
            float mm = -CUDART_INF_F, ll = 0.f, v[D / 32] = {};
            add_parts<D, 8>(mm, ll, v, w.ml, w.part, (2ll * c0 + 1) * 16 + r, 0, 1, lane);
            add_parts<D, 8>(mm, ll, v, w.ml, w.part, 2ll * (c0 + size) * 16 + r, 32 * size, groups - 1, lane);
            emit(r, mm, ll, v);
          }
        }
      }
    }
  }
}

template <int D>
size_t step_layout(StepPlan *out, char *ws) {
  using C = StepCfg<D>;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char *r = ws ? ws + at : nullptr;
    at += up256(bytes);
    return r;
  };
  StepPlan a{};
  a.arrived = (unsigned int *)take(kArrivedBytes);
  a.ml = (float *)take(sizeof(float) * 2 * 16 * 2 * C::CTAS);
  a.part = (float *)take(sizeof(float) * 16 * D * 2 * C::CTAS);
  if (out) *out = a;
  return at;
}

}  // namespace gdn
