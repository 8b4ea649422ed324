// Attention over the paged cache on the tcgen05 tensor cores, for prompts, drafts and shared
// prefixes: tiles of query rows against the keys, one pass with a running maximum and sum.
//
// Rows.  A kv-head's G = Hq / Hkv query heads share its keys, so a tile packs (token, head)
// rows: row r of a 128-row sub-tile is token r / G, head r % G, tpt = 128 / G tokens in all.
//
// Per tile of BN keys, with S = Q K^T in tensor memory and one thread per row:
//     m' = max(m, scale max_c S_c);  p_c = 2^(scale S_c - m');  l = l 2^(m - m') + sum p_c
//     O <- O 2^(m - m') + P V
// (scale includes log2 e).  The reference m only moves when it would rise by more than 8, so
// that O is rescaled a few times per row at most: p then stays below 2^8 and the result is the
// same, as l and O share the reference.  P goes to tensor memory as bf16 (V is held in
// bf16: the product's other operand has no more bits) and l sums the unrounded p in float32.
//
// A tile has two sub-tiles of 128 rows that share each K and V tile of 128 keys.
// D = 128: one CTA; while the softmax warps of one sub-tile work, the tensor cores run the
// other's products.  Tensor memory: S 2 x 128 columns (P over S), O 2 x 128.
// D = 256: a pair of CTAs with a sub-tile each (O takes 256 of the 512 columns) and the
// products of cta_group::2, so that each CTA loads and reads half of every K and V tile (one CTA
// alone had 64-key tiles, whose score products are bound by shared memory: 48 cycles for 32).
// Two S buffers: the next tile's scores are computed while this one's softmax runs.
// Both: 64 KB of Q and a ring of five 32 KB tiles in shared memory, loaded by TMA page by page.
// Narrow tiles have one sub-tile and one CTA: D = 128 two CTAs to an SM, with half its tensor memory and
// two 32 KB stages each; D = 256 two 64 KB stages and two S buffers.
//
// Warps: 4 per sub-tile for the softmax and the epilogue, one for the loads, one for the products.
//
// Bound by the tensor cores for prompts: 8192 tokens, 32 heads of 128 take 338 us (1625 TFLOP/s, 85%
// of cuBLAS's rate; a step of 128 keys 2450 cycles against the products' 2048); 4096 tokens, 16
// heads of 256 take 89 us (1540), with a gate 104 (the epilogue's sigmoids).  Drafts of 16 tokens on
// contexts of 200 to 4000 are bound by HBM: 103 us, 5.3 TB/s with the plan.
#pragma once

#include <cuda.h>
#include <math_constants.h>

#include "attn.h"
#include "attn_tma.cuh"
#include "tc.cuh"

namespace gdn {

constexpr int kBN = 128;        // keys per tile

template <int D_, bool NARROW = false>
struct Cfg {
  static constexpr int D = D_;
  static constexpr bool PAIR = D == 256 && !NARROW;  // two CTAs share a tile, one sub-tile each
  static constexpr int GRP = PAIR ? 2 : 1;          // tcgen05 cta_group
  static constexpr int SUBS = PAIR || NARROW ? 1 : 2;  // sub-tiles of 128 rows in a CTA
  static constexpr int ROWS = 128 * SUBS * GRP;     // of a tile
  static constexpr int CTAS = NARROW && D == 128 ? 2 : 1;  // on an SM
  static constexpr int NBUF = D == 256 ? 2 : 1;     // S buffers of a sub-tile
  static constexpr int STAGES = NARROW ? 2 : 5;
  static constexpr int CH = D / 64;                 // 128-byte column chunks of a row of q or K
  static constexpr int KROWS = PAIR ? 64 : kBN;     // keys of a K tile in this CTA
  static constexpr int Q_BYTES = 128 * D * 2;       // one sub-tile
  static constexpr int VCH = PAIR ? 2 : D / 64;     // 64-column chunks of a V tile in this CTA
  static constexpr int KV_BYTES = VCH * 16384;      // a CTA's part of a K or V tile
  static constexpr int O_COL = CTAS == 2 ? 128 : 256;  // tensor memory: S from column 0, O from here
  static constexpr int COLS = CTAS == 2 ? 256 : 512;
  static constexpr int SMEM = SUBS * Q_BYTES + STAGES * KV_BYTES;
  static constexpr int THREADS = SUBS == 1 ? 192 : 384;  // of the tile kernel (384: two warps are idle)
  static constexpr int WIDE = 384;                  // of the kernel that shares the SMs with decode workers
  static constexpr int UNITS = kSms * CTAS / GRP;   // CTAs, or pairs of them
  static constexpr int SLOTS = 2 * UNITS;           // partial results of split tiles
};

// ------------------------------------------------------------------ operands

// Descriptors of 128-byte-swizzled operands: K-major (rows of 128 bytes, eight rows per
// 1024-byte atom) and MN-major (rows along K; `mn` bytes from one 64-column chunk to the next).
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t mn) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)(mn >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

// tcgen05 of one CTA (GRP = 1) or of a pair (2): there the CTA of even rank issues for both,
// each holding its 128 rows of A and of the result and half of B's N, at the same addresses.
template <int GRP>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  if (GRP == 1) {
    tc::mma_ss(d, a, b, id, accumulate);
  } else {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(accumulate)
        : "memory");
  }
}
template <int GRP>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  if (GRP == 1) {
    tc::mma_ts(d, a, b, id, accumulate);
  } else {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(accumulate)
        : "memory");
  }
}
// Arrive on `bar` (of both CTAs of a pair) once every product issued so far has completed.
template <int GRP>
__device__ __forceinline__ void commit(uint64_t *bar) {
  if (GRP == 1) {
    tc::commit(bar);
  } else {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  }
}
template <int GRP, int COLS>
__device__ __forceinline__ void tmem_alloc(uint32_t *slot) {
  if (GRP == 1) {
    tc::alloc<COLS>(slot);
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
  }
}
template <int GRP, int COLS>
__device__ __forceinline__ void tmem_dealloc(uint32_t base) {
  if (GRP == 1) tc::dealloc<COLS>(base);
  else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;\n" ::"r"(base) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// The address of a shared-memory object of this CTA in the pair's first CTA.
__device__ __forceinline__ uint32_t in_first(const void *p) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;\n" : "=r"(r) : "r"(smem_u32(p)));
  return r;
}
// Arrive in the first CTA.  The second form also orders this thread's writes to shared memory
// before it for the cluster; what the first one signals lies in tensor memory and is ordered by
// tcgen05's own fences (with .release.cluster a tile's softmax took 2000 cycles longer).
__device__ __forceinline__ void arrive_first(uint64_t *bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(in_first(bar)) : "memory");
}
__device__ __forceinline__ void release_first(uint64_t *bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(in_first(bar)) : "memory");
}
// TMA loads; in a pair they count on the first CTA's barrier.
template <bool PAIR>
__device__ __forceinline__ void load_q(void *dst, const void *map, int x, int y, int z, uint64_t *bar) {
  if (!PAIR) {
    tma_load_3d(dst, map, x, y, z, bar);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%2, %3, %4}], [%5];\n" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(in_first(bar))
        : "memory");
  }
}
template <bool PAIR>
__device__ __forceinline__ void load_kv(void *dst, const void *map, int x, int y, int z, int w, uint64_t *bar) {
  if (!PAIR) {
    tma_4d(dst, map, x, y, z, w, bar);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%2, %3, %4, %5}], [%6];\n" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(in_first(bar))
        : "memory");
  }
}
// A load that stays where it stands (the compiler would move it down to its use).
__device__ __forceinline__ uint4 load_now(const void *p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// Four lanes' 16-byte units: unit k of lane i to unit i of lane k.
__device__ __forceinline__ void swap_units(uint4 &a, uint4 &b, bool up, int mask) {
  uint4 s = up ? a : b;
  s.x = __shfl_xor_sync(0xffffffffu, s.x, mask);
  s.y = __shfl_xor_sync(0xffffffffu, s.y, mask);
  s.z = __shfl_xor_sync(0xffffffffu, s.z, mask);
  s.w = __shfl_xor_sync(0xffffffffu, s.w, mask);
  if (up) a = s;
  else b = s;
}
__device__ __forceinline__ void transpose4(uint4 (&u)[4], int lane) {
  swap_units(u[0], u[1], lane & 1, 1);
  swap_units(u[2], u[3], lane & 1, 1);
  swap_units(u[0], u[2], lane & 2, 2);
  swap_units(u[1], u[3], lane & 2, 2);
}

// Rows of a V tile (CHUNKS chunks of 64 columns, 128 rows) from `valid` on to zero, by one warp:
// they lie past the last key, and 0 * NaN is not 0.
template <int CHUNKS>
__device__ __forceinline__ void clear_rows(uint8_t *tile, int valid, int lane) {
  for (int x = lane; x < (128 - valid) * (8 * CHUNKS); x += 32) {
    const int r = valid + x / (8 * CHUNKS), y = x % (8 * CHUNKS);
    *reinterpret_cast<uint4 *>(tile + (y >> 3) * 16384 + r * 128 + (y & 7) * 16) = make_uint4(0, 0, 0, 0);
  }
  tc::fence_proxy_async();
  __syncwarp();
}

// Ties loaded registers to the wait before them, so that no use moves above it.
__device__ __forceinline__ void tie32(uint32_t (&r)[32]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                 "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]),
                 "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]),
                 "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}

// Pairs of floats in one instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.ftz.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.ftz.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 32 columns of O, or zeros where no product was taken.
__device__ __forceinline__ void read_o(uint32_t (&o)[32], uint32_t addr, bool some) {
  if (some) {
    tc::ld32(addr, o);
    tc::wait_ld();
    tie32(o);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = 0;
  }
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// ------------------------------------------------------------------ plan

// One piece of work of a kv-head: tokens tok0 .. tok0 + ntok - 1 of a sequence against its
// key tiles kt0 .. kt1 - 1.
struct Entry {
  int tok0, ntok, seq, place0;  // place0: place of tok0 (kMostKeys: every key is seen)
  int kt0, kt1, slot, kvlen;    // slot: partial result's (of kv-head 0, then Hkv apart), -1: final
};
struct Split {  // a tile whose parts are joined afterwards
  int tok0, ntok, slot, parts;
};

// The plan and the partial results, in the caller's workspace.
struct TilePlan {
  int *head;      // [0] entries, [1] tiles to join
  int *base;      // first tile of each sequence
  Entry *rec;     // tiles
  Entry *entry;   // pieces of work, longest first
  Split *split;   // tiles to join
  float *ml;      // [slot][row] {m, l}
  float *part;    // [slot][row][D]
  int max_tiles, max_entries, units, slots, all_slots;
  int uniform_parts, uniform_kt;  // > 0: no plan, equal parts of equal tiles (shared prefix)
  unsigned int *err;
};

// Keys that the last of `ntok` tokens from place0 on sees.
__device__ __forceinline__ int visible(int place0, int ntok, int kvlen) {
  return min(max(place0 + ntok, 0), kvlen);
}

// Parts of a tile of kvt key tiles in chunks of `chunk` (inv = 1 / chunk): about
// ceil(kvt / chunk), at least 1; every user computes the same.
__device__ __forceinline__ int parts_in(int kvt, int chunk, float inv) {
  return kvt <= chunk ? 1 : (int)ceilf(kvt * inv * 0.999999f);
}

__device__ __forceinline__ void seq_info(const AttnParams &p, int n, int &bos, int &t, int &len) {
  bos = n;
  t = 1;
  if (p.cu_seqlens) {
    int eos;
    seq_range(p.cu_seqlens, n, p.tokens, bos, eos);
    t = eos - bos;
  }
  len = (int)min(max((long long)p.kv_lens[n], 0ll), (long long)p.max_pages * p.page_size);
}

// ------------------------------------------------------------------ the tile kernel

struct Barriers {
  uint64_t q_full, q_empty, kv_full[5], kv_empty[5], s_full[2], p_full[2][2], pv_done[2];
  uint64_t v_tail, tail_ok[5];  // D = 256: a last V tile has come; it has been cleared past the last key
  uint32_t tmem;
  int dead;
};

// Work item of this round: the entry and its kv-head.
__device__ __forceinline__ bool item_at(const AttnParams &p, const TilePlan &w, int unit, int units, int round,
                                        int tt, Entry &e, int &h) {
  // back and forth over the units, so that who had the longest entry gets the shortest next
  const int c = (round & 1) ? units - 1 - unit : unit;
  const long long i = (long long)round * units + c;
  if (w.uniform_parts > 0) {  // shared prefix: equal parts of equal tiles
    const int tiles = (p.tokens + tt - 1) / tt;
    if (i >= (long long)tiles * w.uniform_parts * p.hkv) return false;
    h = (int)(i % p.hkv);
    const int at = (int)(i / p.hkv), tile = at / w.uniform_parts, q = at % w.uniform_parts;
    const int kvt = w.uniform_kt;
    e.tok0 = tile * tt;
    e.ntok = min(tt, p.tokens - e.tok0);
    e.seq = 0;
    e.place0 = kMostKeys;
    e.kt0 = (int)((long long)kvt * q / w.uniform_parts);
    e.kt1 = (int)((long long)kvt * (q + 1) / w.uniform_parts);
    e.slot = at * p.hkv;
    e.kvlen = p.prefix_len;
    return true;
  }
  if (i / p.hkv >= w.max_entries) return false;
  h = (int)(i % p.hkv);
  const int4 *src = reinterpret_cast<const int4 *>(w.entry + i / p.hkv);
  const int4 a = src[0], b = src[1];
  if (i / p.hkv >= w.head[0]) return false;  // (three loads side by side, not one after another)
  e = Entry{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  return true;
}

// Key tiles that sub-tile `i` of an entry takes part in.
__device__ __forceinline__ int sub_tiles(const Entry &e, int i, int tpt) {
  const int first = i * tpt;
  if (first >= e.ntok) return 0;
  const int vis = visible(e.place0, min(e.ntok, first + tpt), e.kvlen);
  return max(0, min((vis + kBN - 1) / kBN, e.kt1) - e.kt0);
}

// The work of unit `unit` of `units` (a CTA, or a pair of them) by all of its threads.  `waited`: the
// work before this kernel is known to be complete.  The warps are 4 SUBS for the softmax, LOADER that
// loads and the next that issues the products.
template <class C, int LOADER>
__device__ __forceinline__ void tile_role(const AttnParams &p, const TilePlan &w, const CUtensorMap &qmap,
                                          const CUtensorMap &kmap, const CUtensorMap &vmap, uint8_t *smem_raw,
                                          Barriers &bars, int unit, int units, bool waited) {
  constexpr int D = C::D;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t *sq = smem, *skv = smem + C::SUBS * C::Q_BYTES;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  volatile int *dead = &bars.dead;
  const int G = p.hq / p.hkv, tpt = 128 / G, tt = tpt * (C::ROWS / 128);
  const int rank = C::PAIR ? (int)(blockIdx.x & 1) : 0;  // CTA of the pair

  if (threadIdx.x == 0) {
    mbar_init(&bars.q_full, 1);
    mbar_init(&bars.q_empty, 1);
    for (int i = 0; i < C::STAGES; ++i)
      mbar_init(&bars.kv_full[i], 1), mbar_init(&bars.kv_empty[i], 1), mbar_init(&bars.tail_ok[i], 2);
    for (int i = 0; i < 2; ++i)
      mbar_init(&bars.s_full[i], 1), mbar_init(&bars.p_full[i][0], 4 * C::GRP),
          mbar_init(&bars.p_full[i][1], 4 * C::GRP), mbar_init(&bars.pv_done[i], 1);
    mbar_init(&bars.v_tail, 1);
    mbar_fence_init();
    bars.dead = 0;
  }
  if (warp == LOADER) {
    if (lane == 0) {
      prefetch_map(&qmap);
      if (p.num_pages > 0) {  // else there are no such maps
        prefetch_map(&kmap);
        prefetch_map(&vmap);
      }
    }
    __syncwarp();
    tmem_alloc<C::GRP, C::COLS>(&bars.tmem);
  }
  tc::fence_before();
  __syncthreads();
  if (C::PAIR) cluster_sync();  // the other CTA's barriers are ready
  tc::fence_after();
  const uint32_t tmem = bars.tmem;
  if (!waited) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  }

  Entry e;
  int h;
  // 12 warps start with 168 registers each.  D = 128: the eight softmax warps take 208, the other
  // four keep 88 (with 224 and 56 the warps that load and issue ran short: packed prompts 949 us
  // against 905).  D = 256 in 12 warps: the four softmax warps take 232, four idle ones give theirs
  // away; in 6 warps there are enough.  8 x 208 + 4 x 88 = 4 x 232 + 4 x 24 + 4 x 248 = 12 x 168.
  constexpr bool kMove = LOADER == 8;
  if (warp < 4 * C::SUBS) {
    // ---------------------------------------------------------------- softmax, epilogue
    if (kMove && C::PAIR) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;\n");
    else if (kMove) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;\n");
    const int sub = C::PAIR ? rank : warp >> 2;
    const int row = threadIdx.x & 127;
    const float asl = p.scale == 0.f ? 1.f : fabsf(p.scale) * 1.4426950408889634f;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t o_base = lanes + C::O_COL + (C::PAIR ? 0 : sub * 128);
    uint32_t cnt = 0;  // tiles of this sub-tile so far, over all items
    for (int round = 0; item_at(p, w, unit, units, round, tt, e, h); ++round) {
      // (a pair's sub-tiles run through the same tiles: one product is for both)
      const int n = C::PAIR ? max(sub_tiles(e, 0, tpt), sub_tiles(e, 1, tpt)) : sub_tiles(e, sub, tpt);
      const int dt = sub * tpt + row / G;
      const bool live = row < tpt * G && dt < e.ntok;
      // keys this row sees, counted from the entry's first
      const int limit = (live ? visible(e.place0, dt + 1, e.kvlen) : 0) - e.kt0 * kBN;
      float m = -CUDART_INF_F, l = 0.f;
      if (p.gate && live && e.slot < 0) {  // the epilogue's gate, into L2 meanwhile (4096 tokens: 112 -> 107 us)
        const char *at = (const char *)((const __nv_bfloat16 *)p.gate + (e.tok0 + dt) * p.gs[0] + (h * G + row % G) * p.gs[1]);
#pragma unroll
        for (int c = 0; c < 2 * D; c += 128) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(at + c));
      }
      for (int j = 0; j < n; ++j, ++cnt) {
        const int b = C::NBUF == 2 ? (cnt & 1) : sub;
        const uint32_t s_addr = lanes + b * 128;
        wait_bar(&bars.s_full[b], C::NBUF == 2 ? (cnt >> 1) & 1 : cnt & 1, dead, w.err);
        // Every completion of P V is waited for in its turn (it has come, or is about to: these
        // scores were issued after it), so that no wait mistakes an older phase for its own.
        if (C::NBUF == 2 && j >= 2) wait_bar(&bars.pv_done[b], ((cnt - 2) >> 1) & 1, dead, w.err);
        if (C::NBUF == 1 && j >= 1) wait_bar(&bars.pv_done[b], (cnt - 1) & 1, dead, w.err);
        tc::fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::ld32(s_addr + 32 * c, s[c]);
        tc::wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) tie32(s[c]);
        if (p.scale <= 0.f) {
#pragma unroll
          for (int c = 0; c < kBN; ++c) {
            const float x = __uint_as_float(s[c / 32][c % 32]);
            s[c / 32][c % 32] = __float_as_uint(p.scale == 0.f ? 0.f : -x);
          }
        }
        const int lim = limit - j * kBN;
        if (__any_sync(0xffffffffu, lim < kBN)) {
#pragma unroll
          for (int c = 0; c < kBN; ++c)
            if (c >= lim) s[c / 32][c % 32] = 0xff800000u;
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) mx[c] = __uint_as_float(s[0][c]);
#pragma unroll
        for (int c = 4; c < kBN; c += 2)
          mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], __uint_as_float(s[c / 32][c % 32]),
                                  __uint_as_float(s[c / 32][c % 32 + 1]));
        const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * asl;
        if (__any_sync(0xffffffffu, top > m + 8.f)) {
          const float m1 = fmaxf(m, top);
          const float a = m1 == -CUDART_INF_F ? 1.f : ex2(m - m1);
          if (j > 0) {
            if (C::NBUF == 2) {
              wait_bar(&bars.pv_done[b ^ 1], ((cnt - 1) >> 1) & 1, dead, w.err);
              tc::fence_after();
            }
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tc::ld32(o_base + c, o);
              tc::wait_ld();
              tie32(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
              tc::st32(o_base + c, o);
            }
          }
          l *= a;
          m = m1;
        }
        const float ref = m == -CUDART_INF_F ? 0.f : m;
        const uint64_t asl2 = pack2(asl, asl), ref2 = pack2(-ref, -ref);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 x =
                unpack2(fma2(pack2(__uint_as_float(s[c][2 * i]), __uint_as_float(s[c][2 * i + 1])), asl2, ref2));
            const float a = ex2(x.x), b2 = ex2(x.y);
            sum[i & 1] = add2(sum[i & 1], pack2(a, b2));
            pk[i] = pack_bf16(a, b2);
          }
          tc::st16(s_addr + 16 * c, pk);
          if (c & 1) {  // 64 keys of P are handed over
            tc::wait_st();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) {
              if (C::PAIR) arrive_first(&bars.p_full[b][c >> 1]);
              else mbar_arrive(&bars.p_full[b][c >> 1]);
            }
          }
        }
        const float2 su = unpack2(add2(sum[0], sum[1]));
        l += su.x + su.y;
      }
      // epilogue
      auto settle = [&]() {  // the last P V
        if (C::NBUF == 2) {
          if (n > 1) wait_bar(&bars.pv_done[cnt & 1], ((cnt - 2) >> 1) & 1, dead, w.err);
          wait_bar(&bars.pv_done[(cnt - 1) & 1], ((cnt - 1) >> 1) & 1, dead, w.err);
        } else {
          wait_bar(&bars.pv_done[sub], (cnt - 1) & 1, dead, w.err);
        }
        tc::fence_after();
      };
      // A lane has a row; for global memory four lanes exchange 16-byte units (transpose4), so that
      // an access covers 64 bytes of eight rows and not 16 of 32 (a line a cycle is the limit).
      const int tok = e.tok0 + dt, head = h * G + row % G;
      const int orow = live ? tok * p.hq + head : -1;
      const int unit4 = lane & 3;
      int rowk[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) rowk[k] = __shfl_sync(0xffffffffu, orow, (lane & 28) + k);
      if (e.slot >= 0) {
        const long long at = (long long)(e.slot + h) * C::ROWS + sub * 128 + row;
        if (live) *reinterpret_cast<float2 *>(w.ml + 2 * at) = make_float2(seen_max(m, limit > 0), l);
        float *part = w.part + (at - unit4) * D + 4 * unit4;
        if (n > 0) settle();
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          read_o(o, o_base + c, n > 0);
#pragma unroll
          for (int i = 0; i < 32; i += 16) {
            uint4 u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              u[k] = make_uint4(o[i + 4 * k], o[i + 4 * k + 1], o[i + 4 * k + 2], o[i + 4 * k + 3]);
            transpose4(u, lane);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (rowk[k] >= 0) *reinterpret_cast<uint4 *>(part + k * D + c + i) = u[k];
          }
        }
      } else {
        if (live && p.lse) p.lse[orow] = row_lse(m, l);
        // as row_inverse, which took 0.5% longer here (a NaN in l is in every column of O too)
        float inv = l > 0.f ? 1.f / l : 0.f;
        if (l == 0.f && limit > 0) inv = CUDART_NAN_F;
        const __nv_bfloat16 *gk[4];
        uint4 gate[4];
        if (p.gate) {
          const long long off = live ? tok * p.gs[0] + head * p.gs[1] : 0;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            gk[k] = (const __nv_bfloat16 *)p.gate + __shfl_sync(0xffffffffu, off, (lane & 28) + k) + 8 * unit4;
        }
        auto fetch = [&](uint4 (&to)[4], int c) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            to[k] = make_uint4(0, 0, 0, 0);
            if (rowk[k] >= 0) to[k] = load_now(gk[k] + c);
          }
        };
        if (p.gate) fetch(gate, 0);
        if (n > 0) settle();
        // A pair's loop stays rolled (16 heads of 256, 4096 tokens: 89 us, by two 91); the other is
        // unrolled by two (8192 tokens, 32 heads of 128: 338 us, rolled 346).
        // With the registers for it (D = 256) the next columns' gate is fetched before these ones' sigmoids
        // and not after (107 -> 104 us; D = 128: 353 -> 369).
        constexpr int kUnroll = C::PAIR ? 1 : 2;
        constexpr bool kEarly = D == 256;
#pragma unroll (kUnroll)
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          uint4 u[4];
          uint4 next[4];
          if (kEarly && p.gate && c + 32 < D) fetch(next, c + 32);
          read_o(o, o_base + c, n > 0);
          if (p.gate) transpose4(gate, lane);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(o[8 * k + i]) * inv;
            if (p.gate) gate8(x, gate[k]);
            u[k] = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                              pack_bf16(x[6], x[7]));
          }
          if (!kEarly && p.gate && c + 32 < D) fetch(gate, c + 32);
#pragma unroll
          for (int k = 0; kEarly && k < 4; ++k) gate[k] = next[k];
          transpose4(u, lane);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (rowk[k] >= 0)
              *reinterpret_cast<uint4 *>((__nv_bfloat16 *)p.o + (long long)rowk[k] * D + c + 8 * unit4) = u[k];
        }
      }
      tc::fence_before();
    }
  } else if (warp < LOADER) {
    if (kMove) asm volatile("setmaxnreg.dec.sync.aligned.u32 24;\n");
  } else {
   if (kMove && C::PAIR) asm volatile("setmaxnreg.inc.sync.aligned.u32 248;\n");
   else if (kMove) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
   if (warp == LOADER) {
    // ---------------------------------------------------------------- loads
    // A tile comes in boxes of box rows x 64 columns; lane b keeps the page of box b of the tile
    // after the present one, so that no load waits for the table.  In a pair, CTA r holds keys
    // 64 r .. + 63 of K and columns 128 r .. + 127 of V.  Uniform values for the same reason
    // as in the products.
    const int lps = 31 - __clz(p.page_size), box = min(p.page_size, C::KROWS);
    const int kb0 = C::PAIR ? rank * (64 / box) : 0, kb1 = kb0 + C::KROWS / box;  // this CTA's boxes of K
    uint32_t st = 0, ph = 1, items = 0, tails = 0;
    for (int round = 0; item_at(p, w, unit, units, round, tt, e, h); ++round) {
      const int n0 = uniform(sub_tiles(e, 0, tpt)), n1 = uniform(sub_tiles(e, 1, tpt)), n = max(n0, n1);
      if (n == 0) continue;
      const int32_t *table = w.uniform_parts > 0 ? p.prefix_table : p.page_table + (long long)e.seq * p.max_pages;
      const int kvlen = uniform(e.kvlen), first = uniform(e.kt0 * kBN), head = uniform(h);
      auto page_of = [&](int j) {
        const int key = first + j * kBN + lane * box;
        return j < n && lane * box < kBN && key < kvlen ? table[key >> lps] : 0;
      };
      int ahead = page_of(0);
      wait_bar(&bars.q_empty, (items & 1) ^ 1, dead, w.err);
      if (elect_one()) {
        const uint32_t sub_bytes = (uint32_t)C::CH * tpt * G * 128;
        if (rank == 0) mbar_arrive_expect_tx(&bars.q_full, ((n0 > 0) + (n1 > 0)) * sub_bytes);
        for (int i = 0; i < 2; ++i)
          if ((i ? n1 : n0) > 0 && (!C::PAIR || i == rank))
            for (int c = 0; c < C::CH; ++c)
              load_q<C::PAIR>(sq + (C::PAIR ? 0 : i * C::Q_BYTES) + c * 16384, &qmap, c * 64, head * G,
                              e.tok0 + i * tpt, &bars.q_full);
      }
      __syncwarp();
      ++items;
      for (int j = 0; j < n; ++j) {
        const int page = ahead;
        ahead = page_of(j + 1);
        const int key0 = first + j * kBN, left = kvlen - key0;
        const int boxes = (min(left, kBN) + box - 1) / box;        // up to the last key
        const uint32_t bytes = (uint32_t)boxes * box * D * 2;      // of both CTAs
        auto page_in = [&](int b) {  // (a page out of range reads as zeros)
          const int pg = __shfl_sync(0xffffffffu, page, b);
          return (unsigned)pg < (unsigned)p.num_pages ? pg : p.num_pages;
        };
        // K
        wait_bar(&bars.kv_empty[st], ph, dead, w.err);
        uint8_t *dst = skv + st * C::KV_BYTES;
        if (rank == 0 && elect_one()) mbar_arrive_expect_tx(&bars.kv_full[st], bytes);
        __syncwarp();
        for (int b = kb0; b < min(boxes, kb1); ++b) {
          const int pg = page_in(b), row = (key0 + b * box) & (p.page_size - 1);
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < C::CH; ++c)
              load_kv<C::PAIR>(dst + c * (C::KROWS * 128) + (b - kb0) * box * 128, &kmap, c * 64, row, head, pg,
                               &bars.kv_full[st]);
          }
          __syncwarp();
        }
        if (++st == C::STAGES) st = 0, ph ^= 1;
        // V
        wait_bar(&bars.kv_empty[st], ph, dead, w.err);
        dst = skv + st * C::KV_BYTES;
        const bool tail = C::PAIR && left < kBN;
        if (elect_one()) {
          if (tail) mbar_arrive_expect_tx(&bars.v_tail, bytes / 2);
          if (rank == 0) {
            if (tail) mbar_arrive(&bars.kv_full[st]);
            else mbar_arrive_expect_tx(&bars.kv_full[st], bytes);
          }
        }
        __syncwarp();
        for (int b = 0; b < boxes; ++b) {
          const int pg = page_in(b), row = (key0 + b * box) & (p.page_size - 1);
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < C::VCH; ++c) {
              const int x = (C::PAIR ? rank * 128 : 0) + c * 64;
              uint8_t *at = dst + c * (kBN * 128) + b * box * 128;
              if (tail) tma_4d(at, &vmap, x, row, head, pg, &bars.v_tail);
              else load_kv<C::PAIR>(at, &vmap, x, row, head, pg, &bars.kv_full[st]);
            }
          }
          __syncwarp();
        }
        if (tail) {  // both CTAs clear their columns past the last key, then the products may start
          wait_bar(&bars.v_tail, tails & 1, dead, w.err);
          ++tails;
          clear_rows<C::VCH>(dst, left, lane);
          if (lane == 0) release_first(&bars.tail_ok[st]);
        }
        if (++st == C::STAGES) st = 0, ph ^= 1;
      }
    }
   } else if (warp == LOADER + 1 && rank == 0) {
    // ---------------------------------------------------------------- products
    // All values here are the same in every lane and known as such (uniform()): the
    // instruction takes its descriptors from uniform registers, and building them from
    // lane-varying ones made issuing a product (95 cycles) slower than the product (64).
    constexpr int M = 128 * C::GRP;
    constexpr uint32_t id_qk = tc::idesc(M, kBN, 1, 0, 0), id_pv = tc::idesc(M, D, 1, 0, 1);
    constexpr uint32_t kStage = C::KV_BYTES >> 4;
    const uint32_t tm = uniform(tmem);
    const uint64_t dq = desc_k(uniform(smem_u32(sq))), dk = desc_k(uniform(smem_u32(skv))),
                   dv = desc_mn(uniform(smem_u32(skv)), kBN * 128);
    uint32_t st = 0, ph = 0, items = 0, tails = 0;  // ring position of the next K or V tile, its parity
    uint32_t cnt[2] = {0, 0};
    auto qk = [&](int i, uint32_t at, uint32_t c) {
      const int buf = C::NBUF == 2 ? (c & 1) : i;
      const uint64_t a = dq + i * (C::Q_BYTES >> 4), b = dk + at * kStage;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ss<C::GRP>(tm + buf * 128, a + (((k / 4) * 16384 + (k % 4) * 32) >> 4),
                         b + (((k / 4) * (C::KROWS * 128) + (k % 4) * 32) >> 4), id_qk, k > 0);
        commit<C::GRP>(&bars.s_full[buf]);
      }
      __syncwarp();
    };
    auto done = [&](uint64_t *bar) {
      if (elect_one()) commit<C::GRP>(bar);
      __syncwarp();
    };
    for (int round = 0; item_at(p, w, unit, units, round, tt, e, h); ++round) {
      int n[2] = {uniform(sub_tiles(e, 0, tpt)), uniform(sub_tiles(e, 1, tpt))};
      const int nmax = max(n[0], n[1]);
      if (C::PAIR) n[0] = nmax, n[1] = 0;  // one product for both sub-tiles
      const int keys = uniform(e.kvlen - e.kt0 * kBN);
      if (nmax == 0) continue;
      wait_bar(&bars.q_full, items & 1, dead, w.err);
      ++items;
      auto next = [&](uint32_t &at, uint32_t &parity) {  // takes the ring's next tile
        at = st;
        parity = ph;
        if (++st == C::STAGES) st = 0, ph ^= 1;
      };
      uint32_t sk, pk, sv, pv;
      next(sk, pk);
      wait_bar(&bars.kv_full[sk], pk, dead, w.err);
      tc::fence_after();
#pragma unroll
      for (int i = 0; i < C::SUBS; ++i)
        if (n[i] > 0) qk(i, sk, cnt[i]);
      done(&bars.kv_empty[sk]);
      if (nmax == 1) done(&bars.q_empty);
      for (int j = 0; j < nmax; ++j) {
        const bool more = j + 1 < nmax;
        next(sv, pv);
        if (more) next(sk, pk);
        if (C::NBUF == 2 && more) {
          wait_bar(&bars.kv_full[sk], pk, dead, w.err);
          tc::fence_after();
          qk(0, sk, cnt[0] + 1);
          done(&bars.kv_empty[sk]);
          if (j + 2 == nmax) done(&bars.q_empty);
        }
        wait_bar(&bars.kv_full[sv], pv, dead, w.err);
        const int valid = keys - j * kBN;
        if (valid < kBN) {
          if (C::PAIR) {
            wait_bar(&bars.tail_ok[sv], tails >> sv & 1, dead, w.err);
            tails ^= 1u << sv;  // parity of each stage's own
          } else {
            clear_rows<C::VCH>(skv + sv * C::KV_BYTES, valid, lane);
          }
        }
        if (C::SUBS == 2 && more) wait_bar(&bars.kv_full[sk], pk, dead, w.err);
#pragma unroll
        for (int i = 0; i < C::SUBS; ++i) {
          if (j >= n[i]) continue;
          const uint32_t c = cnt[i]++;
          const int buf = C::NBUF == 2 ? (c & 1) : i;
          const uint32_t pa = tm + buf * 128;
          const uint64_t b = dv + sv * kStage;
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            wait_bar(&bars.p_full[buf][part], C::NBUF == 2 ? (c >> 1) & 1 : c & 1, dead, w.err);
            tc::fence_after();
            if (elect_one()) {
#pragma unroll
              for (int k = 4 * part; k < 4 * part + 4; ++k)
                mma_ts<C::GRP>(tm + C::O_COL + i * 128, pa + k * 8, b + (k * 2048 >> 4), id_pv, j > 0 || k > 0);
              if (part) commit<C::GRP>(&bars.pv_done[buf]);
            }
            __syncwarp();
          }
          if (C::NBUF == 1 && j + 1 < n[i]) {
            if (C::SUBS == 1) {
              wait_bar(&bars.kv_full[sk], pk, dead, w.err);
              tc::fence_after();
            }
            qk(i, sk, c + 1);
          }
        }
        done(&bars.kv_empty[sv]);
        if (C::NBUF == 1 && more) {
          done(&bars.kv_empty[sk]);
          if (j + 2 == nmax) done(&bars.q_empty);
        }
      }
    }
   }
  }
  if (*dead) __nanosleep(1000000);  // copies in flight land before shared memory is given up
  tc::fence_before();
  __syncthreads();
  if (C::PAIR) cluster_sync();  // no signal is on its way to a CTA that has gone
  tc::fence_after();
  if (warp == LOADER) tmem_dealloc<C::GRP, C::COLS>(tmem);
}

// A shared prefix beside the sequences' own keys, one token per sequence (attn_prefix.cu): the
// prefix's parts go to `pre`, their number to pre.head[2], the own results to `dense`.
cudaError_t launch_attn_prefix(const AttnParams &p, void *ws, const TilePlan &pre, const DenseRows &dense,
                               unsigned int *err, cudaStream_t stream);

}  // namespace gdn
