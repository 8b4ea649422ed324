// Attention over the paged cache for prompts, drafts and shared prefixes: the plan that cuts a
// batch into pieces of work, the tile kernel that does them (attn_tile.cuh), the join of split
// tiles, and the choice of kernels for a call.
#include <string.h>

#include <algorithm>

#include "attn_tile.cuh"

namespace gdn {
namespace {

// ------------------------------------------------------------------ plan

constexpr int kPlanThreads = 512;
constexpr int kCand = 16;
constexpr int kPlanTiles = 4096;  // tiles whose lengths are kept in shared memory

// The nodes that each node of the trees sees, by the blocks beside the planning one: 64 threads to a
// sequence walk up from a node each, through parents in shared memory (a chain of 64: 2 us of the plan's 6).
constexpr int kTreesABlock = kPlanThreads / GDN_TREE_NODES;
__device__ __forceinline__ void ancestors(const AttnParams &p, int block, int blocks, int (*up)[GDN_TREE_NODES]) {
  const int i = threadIdx.x % GDN_TREE_NODES, mine = threadIdx.x / GDN_TREE_NODES;
  for (int n0 = block * kTreesABlock; n0 < p.num_seqs; n0 += blocks * kTreesABlock) {
    const int n = n0 + mine;
    int bos = 0, eos = 0;
    if (n < p.num_seqs) seq_range(p.cu_seqlens, n, p.tokens, bos, eos);
    const int t = min(eos - bos, GDN_TREE_NODES);
    if (i < t) up[mine][i] = p.parents[bos + i];
    __syncthreads();
    if (i < t) {
      uint64_t above = 0;
      for (int j = i, next; ; j = next) {  // (goes down at every step)
        above |= 1ull << j;
        next = up[mine][j];
        if (next < 0 || next >= j) break;
      }
      p.above[bos + i] = above;
    }
    for (int j = bos + GDN_TREE_NODES + i; j < eos; j += GDN_TREE_NODES) p.above[j] = 0;  // too many: no bit left
    __syncthreads();
  }
}

// Cuts the batch into entries, one block.  Tiles with many key tiles are split so that the
// SMs get even shares: of kCand chunk lengths the one with the smallest
//     max(chunk, ceil(entries / units) * mean entry) + 3 ceil(entries / units) + join
// (in key tiles; 3 is about what starting and ending an entry costs), where the join costs 0.12 a part of
// the longest tile and 2.4e-6 a float of partial sums (one prompt of 1200 tokens, 12 gated heads of 256:
// 54 us if it is taken to be free, 30 so; any factor from 0.6e-6 to 5e-6 does within 3 us).  Entries are ordered by
// length, longest first, in 64 classes, for the kernel's back-and-forth assignment.  All of it
// is latency: the lengths stay in shared memory and a warp tries each chunk length.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(AttnParams p, TilePlan w, int tt) {
  constexpr int kWarps = kPlanThreads / 32;
  __shared__ int sh_scan[kWarps], sh_total, sh_kvmax, sh_hist[64], sh_slot, sh_nsplit, sh_nbig;
  __shared__ int sh_big[kPlanThreads], sh_kvt[kPlanTiles];
  __shared__ float sh_cost[kCand];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  if (blockIdx.x > 0) {
    ancestors(p, (int)blockIdx.x - 1, (int)gridDim.x - 1, reinterpret_cast<int (*)[GDN_TREE_NODES]>(sh_kvt));
    return;
  }
  if (tid == 0) sh_total = sh_kvmax = sh_slot = sh_nsplit = sh_nbig = 0;
  if (tid < 64) sh_hist[tid] = 0;
  int kvmax = 1;
  auto put = [&](int at, int n, int bos, int t, int len, int i) {
    if (at >= w.max_tiles) return;  // only with a malformed cu_seqlens
    const int tok0 = i * tt, ntok = min(tt, t - tok0);
    const int place0 = p.parents ? kMostKeys : len - t + tok0;  // (a tree's nodes may see any key)
    const int kvt = (visible(place0, ntok, len) + kBN - 1) / kBN;
    w.rec[at] = Entry{bos + tok0, ntok, n, place0, 0, kvt, 0, len};
    if (at < kPlanTiles) sh_kvt[at] = kvt;
    kvmax = max(kvmax, kvt);
  };
  auto length = [&](int i) { return i < kPlanTiles ? sh_kvt[i] : w.rec[i].kt1; };
  for (int n0 = 0; n0 < p.num_seqs; n0 += kPlanThreads) {
    const int n = n0 + tid;
    int bos = 0, t = 0, len = 0;
    if (n < p.num_seqs) seq_info(p, n, bos, t, len);
    const int tiles = (t + tt - 1) / tt;
    int s = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += v;
    }
    if (lane == 31) sh_scan[warp] = s;
    __syncthreads();
    int at = sh_total + s - tiles;
    for (int i = 0; i < warp; ++i) at += sh_scan[i];
    if (tiles > 4) {  // long sequences: all threads over the tiles, below
      sh_big[atomicAdd(&sh_nbig, 1)] = n;
      w.base[n] = at;
    } else {
      for (int i = 0; i < tiles; ++i) put(at + i, n, bos, t, len, i);
    }
    __syncthreads();
    if (tid == kPlanThreads - 1) sh_total = at + tiles;
    for (int b = 0; b < sh_nbig; ++b) {
      const int m = sh_big[b];
      seq_info(p, m, bos, t, len);
      const int first = w.base[m];
      for (int i = tid; i < (t + tt - 1) / tt; i += kPlanThreads) put(first + i, m, bos, t, len, i);
    }
    __syncthreads();
    if (tid == 0) sh_nbig = 0;
  }
  kvmax = __reduce_max_sync(0xffffffffu, kvmax);
  if (lane == 0) atomicMax(&sh_kvmax, kvmax);
  __syncthreads();
  const int tiles = min(sh_total, w.max_tiles);
  kvmax = sh_kvmax;
  constexpr int parts_of[kCand] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 19, 25, 38, 50, 76, 152};
  for (int c = warp; c < kCand; c += kWarps) {
    const int chunk = (kvmax + parts_of[c] - 1) / parts_of[c];
    const float inv = 1.f / chunk;
    int cnt = 0, spl = 0;
    float work = 0.f;
    for (int i = lane; i < tiles; i += 32) {
      const int kvt = length(i), parts = parts_in(kvt, chunk, inv);
      cnt += parts;
      spl += parts > 1 ? parts : 0;
      work += kvt;
    }
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    spl = __reduce_add_sync(0xffffffffu, spl);
    work = warp_sum(work);
    if (lane == 0) {
      const float items = (float)cnt * p.hkv, rounds = ceilf(items / w.units);
      const float floats = (float)spl * p.tokens * p.hq * p.d / max(tiles, 1);  // of partial sums
      const float join = spl > 0 ? 0.12f * parts_in(kvmax, chunk, inv) + 2.4e-6f * floats : 0.f;
      sh_cost[c] = c > 0 && (long long)spl * p.hkv > w.slots
                       ? CUDART_INF_F
                       : fmaxf((float)chunk, rounds * (work * p.hkv / fmaxf(items, 1.f))) + 3.f * rounds + join;
    }
  }
  __syncthreads();
  int best = 0;
#pragma unroll
  for (int c = 1; c < kCand; ++c)
    if (sh_cost[c] < sh_cost[best]) best = c;
  const int chunk = (kvmax + parts_of[best] - 1) / parts_of[best];
  const float inv = 1.f / chunk;
  auto cls = [&](int len) { return 63 - min(63, (int)(len * 63 * inv)); };
  auto cut = [&](int kvt, int q, int parts) { return parts == 1 ? q * kvt : (int)((long long)kvt * q / parts); };
  for (int i = tid; i < tiles; i += kPlanThreads) {
    const int kvt = length(i), parts = parts_in(kvt, chunk, inv);
    for (int q = 0; q < parts; ++q) atomicAdd(&sh_hist[cls(cut(kvt, q + 1, parts) - cut(kvt, q, parts))], 1);
  }
  __syncthreads();
  if (warp == 0) {  // exclusive scan of the 64 classes
    int a = sh_hist[2 * lane], b = sh_hist[2 * lane + 1], s = a + b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += v;
    }
    sh_hist[2 * lane] = s - a - b;
    sh_hist[2 * lane + 1] = s - b;
    if (lane == 31) w.head[0] = s;  // number of entries
  }
  __syncthreads();
  for (int i = tid; i < tiles; i += kPlanThreads) {
    Entry e = w.rec[i];
    const int kvt = length(i), parts = parts_in(kvt, chunk, inv);
    int slot = -1;
    if (parts > 1 || w.all_slots) {
      slot = atomicAdd(&sh_slot, parts) * p.hkv;
      w.split[atomicAdd(&sh_nsplit, 1)] = Split{e.tok0, e.ntok, slot, parts};
    }
    for (int q = 0; q < parts; ++q) {
      e.kt0 = cut(kvt, q, parts);
      e.kt1 = cut(kvt, q + 1, parts);
      e.slot = slot < 0 ? -1 : slot + q * p.hkv;
      w.entry[atomicAdd(&sh_hist[cls(e.kt1 - e.kt0)], 1)] = e;
    }
  }
  __syncthreads();
  if (tid == 0) w.head[1] = sh_nsplit;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::CTAS)
    tile_kernel(AttnParams p, TilePlan w, const __grid_constant__ CUtensorMap qmap,
                const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Barriers bars;
  tile_role<C, C::SUBS == 2 ? 8 : 4>(p, w, qmap, kmap, vmap, smem_raw, bars, (int)blockIdx.x / C::GRP, C::UNITS, false);
}

// ------------------------------------------------------------------ join

// One warp per row: its parts and the shared prefix's.  Rows of the split tiles in the plan's table,
// or with `dense` all rows of the call, whose own result the decode kernel left there.
template <int D>
__global__ void __launch_bounds__(256)
    join_kernel(AttnParams p, TilePlan w, DenseRows dense, PrefixParts pre, int tpt, int tile_rows) {
  const int lane = threadIdx.x & 31;
  const int G = p.hq / p.hkv, per_head = tile_rows / 128 * tpt * G;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const long long rows = dense.part ? (long long)p.tokens * p.hq : (long long)w.head[1] * p.hkv * per_head;
  const long long step = (long long)gridDim.x * 8;
  for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < rows; i += step) {
    float acc[D / 32] = {}, m = -CUDART_INF_F, l = 0.f;
    int tok, h, g;
    if (dense.part) {
      tok = (int)(i / p.hq);
      h = (int)(i % p.hq) / G;
      g = (int)(i % p.hq) % G;
      add_parts<D>(m, l, acc, dense.ml, dense.part, i, 0, 1, lane);
    } else {
      const int r = (int)(i % per_head), dt = r / G;
      const Split s = w.split[i / per_head / p.hkv];
      if (dt >= s.ntok) continue;
      h = (int)(i / per_head % p.hkv);
      g = r % G;
      tok = s.tok0 + dt;
      add_parts<D>(m, l, acc, w.ml, w.part, (long long)(s.slot + h) * tile_rows + dt / tpt * 128 + dt % tpt * G + g,
                   (long long)p.hkv * tile_rows, s.parts, lane);
    }
    add_prefix<D>(m, l, acc, pre, tok, h, g, G, p.hkv, lane);
    emit_row<D>(p, tok, h * G + g, lane, m, l, acc);
  }
}

// ------------------------------------------------------------------ host

// Tokens of a tile, tiles of a call at most, tiles of the shared prefix's pass.
template <int D>
struct Sizes {
  int tpt, tt, max_tiles, prefix_tiles;
  Sizes(int tokens, int num_seqs, int hq, int hkv) {
    tpt = 128 / (hq / hkv);
    tt = tpt * 2;
    max_tiles = tokens / tt + num_seqs;
    prefix_tiles = (tokens + tt - 1) / tt;
  }
};

// Parts that each tile of the prefix pass is cut into: as many as fill the SMs once, of at
// least two key tiles each.
template <int D>
int prefix_parts(int tiles, int hkv, int prefix_len) {
  constexpr int units = Cfg<D>::UNITS;
  const int kt = (prefix_len + kBN - 1) / kBN;
  const long long items = (long long)tiles * hkv;
  const int fill = units / (int)(items < 1 ? 1 : items < units ? items : units);  // (no tokens: no tiles)
  const int most = (kt + 1) / 2;
  return fill < 1 ? 1 : fill < most ? fill : most;
}

template <int D>
size_t layout(TilePlan *own, TilePlan *pre, DenseRows *dense, uint64_t **above, char *ws, int num_seqs, int tokens, int hq,
              int hkv, int prefix_len) {
  const Sizes<D> z(tokens, num_seqs, hq, hkv);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char *r = ws ? ws + at : nullptr;
    at += up256(bytes);
    return r;
  };
  // Tables for the narrow tiles, which are more; partial rows for the wide ones, which have no fewer.
  constexpr int split_slots = Cfg<D, true>::SLOTS;
  static_assert(split_slots * Cfg<D, true>::ROWS == Cfg<D>::SLOTS * Cfg<D>::ROWS, "rows");
  const int narrow_tiles = tokens / z.tpt + num_seqs, entries = narrow_tiles + split_slots;
  const size_t own_slots = prefix_len > 0 ? (size_t)z.max_tiles * hkv + Cfg<D>::SLOTS : Cfg<D>::SLOTS;
  const size_t slot = (size_t)kTileRows * sizeof(float);
  TilePlan a{}, b{};
  DenseRows c{};
  a.head = (int *)take(256);
  a.base = (int *)take(sizeof(int) * (size_t)(num_seqs + 1));
  a.rec = (Entry *)take(sizeof(Entry) * (size_t)narrow_tiles);
  a.entry = (Entry *)take(sizeof(Entry) * (size_t)entries);
  a.split = (Split *)take(sizeof(Split) * (size_t)(prefix_len > 0 ? narrow_tiles : split_slots));
  a.ml = (float *)take(own_slots * slot * 2);
  a.part = (float *)take(own_slots * slot * D);
  a.max_entries = entries;
  if (prefix_len > 0) {
    b.uniform_parts = prefix_parts<D>(z.prefix_tiles, hkv, prefix_len);
    b.uniform_kt = (prefix_len + kBN - 1) / kBN;
    // (no fewer than the units: a batch of fewer rows may have more parts)
    const size_t items = (size_t)z.prefix_tiles * hkv, slots = items > Cfg<D>::UNITS ? items : Cfg<D>::UNITS;
    b.ml = (float *)take(slots * slot * 2);
    b.part = (float *)take(slots * slot * D);
    a.all_slots = 1;
    const size_t rows = (size_t)tokens * hq;
    c.ml = (float *)take(rows * 2 * sizeof(float));
    c.part = (float *)take(rows * D * sizeof(float));
  }
  uint64_t *nodes = (uint64_t *)take(sizeof(uint64_t) * (size_t)tokens);
  if (above) *above = nodes;
  if (dense) *dense = c;
  if (own) *own = a;
  if (pre) *pre = b;
  return at;
}

// The sequences' own keys in tiles of configuration C: plan, tiles, join.
template <class C>
cudaError_t run_tiles(const AttnParams &p, TilePlan own, const PrefixParts &parts, int tpt, const CUtensorMap &q,
                      unsigned int *errw, cudaStream_t stream) {
  const int tt = tpt * (C::ROWS / 128);
  own.err = errw;
  own.max_tiles = p.tokens / tt + p.num_seqs;
  own.units = C::UNITS;
  own.slots = C::SLOTS;
  CUtensorMap k, v;
  cudaError_t err = cache_maps(&k, &v, p, C::KROWS);
  if (err != cudaSuccess) return err;
  const size_t smem = C::SMEM + 1024;
  static std::atomic<uint64_t> allowed{0};
  err = allow_smem(tile_kernel<C>, smem, allowed);
  // (blocks of 8 trees beside the plan's)
  const int trees = C::TREE ? std::min((p.num_seqs + kTreesABlock - 1) / kTreesABlock, kSms - 1) : 0;
  if (err == cudaSuccess)
    err = launch_dependent(plan_kernel, 1 + trees, kPlanThreads, 0, stream, 1, p, own, tt);
  if (err == cudaSuccess)
    err = launch_dependent(tile_kernel<C>, C::UNITS * C::GRP, C::THREADS, smem, stream, C::GRP, p, own, q, k, v);
  if (err != cudaSuccess) return err;
  return launch_dependent(join_kernel<C::D>, 4 * kSms, 256, 0, stream, 1, p, own, DenseRows{}, parts, tpt, C::ROWS);
}

template <int D>
cudaError_t run(const AttnParams &call, char *ws, unsigned int *errw, cudaStream_t stream) {
  // one token per sequence: the decode kernel does the sequences' own keys
  const bool step = !call.cu_seqlens && call.hq / call.hkv <= kStepRows;
  char *tile_ws = ws + attn_step_workspace(D);
  using C = Cfg<D>;
  const Sizes<D> z(call.tokens, call.num_seqs, call.hq, call.hkv);
  if (step && call.prefix_len == 0) return launch_attn_step(call, ws, errw, stream);
  TilePlan own, pre;
  DenseRows dense;
  AttnParams p = call;
  layout<D>(&own, &pre, &dense, &p.above, tile_ws, p.num_seqs, p.tokens, p.hq, p.hkv, p.prefix_len);
  pre.err = errw;
  if (step) {  // the prefix and the sequences' own keys side by side, then their join
    pre.head = own.head;
    cudaError_t err = launch_attn_prefix(p, ws, pre, dense, errw, stream);
    if (err != cudaSuccess) return err;
    const PrefixParts parts{pre.ml, pre.part, pre.head, 0, z.tpt};
    return launch_dependent(join_kernel<D>, 4 * kSms, 256, 0, stream, 1, p, own, dense, parts, z.tpt, C::ROWS);
  }
  CUtensorMap q;
  cudaError_t err = q_map(&q, p, z.tpt);
  if (err != cudaSuccess) return err;
  if (p.prefix_len > 0) {
    CUtensorMap k, v;
    err = cache_maps(&k, &v, p, C::KROWS);
    const size_t smem = C::SMEM + 1024;
    static std::atomic<uint64_t> allowed{0};
    if (err == cudaSuccess) err = allow_smem(tile_kernel<C>, smem, allowed);
    if (err == cudaSuccess)
      err = launch_dependent(tile_kernel<C>, kSms, C::THREADS, smem, stream, C::GRP, p, pre, q, k, v);
    if (err != cudaSuccess) return err;
  }
  const PrefixParts parts{pre.ml, pre.part, nullptr, pre.uniform_parts, z.tpt};
  // Narrow tiles where a sequence's rows fill half a wide one at most, as drafts' do: twice the tiles are
  // under way, and starts and ends overlap (105 drafts of 9 to 18 tokens after 34, 32 heads of 128: 26 us,
  // wide 40; 128 of 16 after 200 to 4000: 103 and 107).  At D = 256 two stages of 64 KB hold long contexts
  // back (28 drafts after 367 to 1469 keys: 74 us, wide 63; 54 after 480: 58 and 66, after 900: 83 and 85).
  // The host knows neither lengths nor rows of a sequence: the rule takes the mean rows, so that a prompt
  // among many single tokens gets narrow tiles, and at D = 256 the most keys that the page table can hold,
  // so that behind a table of more than 1024 keys drafts get wide ones whatever their contexts.
  const bool narrow = (long long)p.tokens <= (long long)p.num_seqs * z.tpt &&
                      (D == 128 || (long long)p.max_pages * p.page_size <= 1024);
  if (p.parents)
    return narrow ? run_tiles<Cfg<D, true, true>>(p, own, parts, z.tpt, q, errw, stream)
                  : run_tiles<Cfg<D, false, true>>(p, own, parts, z.tpt, q, errw, stream);
  return narrow ? run_tiles<Cfg<D, true>>(p, own, parts, z.tpt, q, errw, stream)
                : run_tiles<C>(p, own, parts, z.tpt, q, errw, stream);
}

}  // namespace

size_t attn_workspace(int num_seqs, int tokens, int hq, int hkv, int d, int prefix_len) {
  // the decode kernel's part first: its counters stay in one place for all shapes
  return attn_step_workspace(d) + (d == 128 ? layout<128>(nullptr, nullptr, nullptr, nullptr, nullptr, num_seqs, tokens, hq, hkv, prefix_len)
                                            : layout<256>(nullptr, nullptr, nullptr, nullptr, nullptr, num_seqs, tokens, hq, hkv, prefix_len));
}

cudaError_t launch_attention(const AttnParams &p, void *ws, unsigned int *err, cudaStream_t stream) {
  return p.d == 128 ? run<128>(p, static_cast<char *>(ws), err, stream)
                    : run<256>(p, static_cast<char *>(ws), err, stream);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t bf16_map(CUtensorMap *map, const void *x, int rank, const cuuint64_t *dims,
                     const cuuint64_t *strides, const cuuint32_t *box) {
  // cuTensorMapEncodeTiled from the driver, looked up once (no link against libcuda)
  static EncodeTiledFn enc = []() -> EncodeTiledFn {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  if (!enc) return cudaErrorNotSupported;
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(x), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

cudaError_t q_map(CUtensorMap *map, const AttnParams &p, int tokens) {
  const cuuint64_t dims[3] = {(cuuint64_t)p.d, (cuuint64_t)p.hq, (cuuint64_t)p.tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)p.qs[1] * 2, (cuuint64_t)p.qs[0] * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)(p.hq / p.hkv), (cuuint32_t)tokens};
  return bf16_map(map, p.q, 3, dims, strides, box);
}

cudaError_t cache_maps(CUtensorMap *k, CUtensorMap *v, const AttnParams &p, int tile) {
  memset(k, 0, sizeof(*k));
  memset(v, 0, sizeof(*v));
  if (p.num_pages == 0) return cudaSuccess;
  const cuuint64_t dims[4] = {(cuuint64_t)p.d, (cuuint64_t)p.page_size, (cuuint64_t)p.hkv,
                              (cuuint64_t)p.num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)p.d * 2, (cuuint64_t)p.page_size * p.d * 2,
                                 (cuuint64_t)p.page_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)(p.page_size < tile ? p.page_size : tile), 1, 1};
  const cudaError_t err = bf16_map(k, p.k_cache, 4, dims, strides, box);
  return err != cudaSuccess ? err : bf16_map(v, p.v_cache, 4, dims, strides, box);
}

}  // namespace gdn
