// Eviction by accumulated attention weight, in place, per (sequence, KV head): keep the protected
// entries (the first tokens and the last ones, by their ordinals) and then those of the largest
// weight, `budget` in all. Three launches:
//
//   own     writes into owner[page] which table place names the page, so that the next step can see
//           a page that is named twice (its place does not read back what it wrote);
//   select  a cluster of CTAs per (sequence, KV head) finds the budget-th largest key by a radix
//           descent (11, 11 and 10 bits; the histograms are summed over the cluster through
//           distributed shared memory) and lists the evicted places e < budget and the kept
//           entries e >= budget, both in ascending order: there are as many of one as of the other;
//   move    copies kept entry j of the second list over place j of the first. Sources and targets
//           never overlap, so every row moves on its own, and a bounded cache that is one entry over its
//           budget moves one row per head, not the cache.
//
// Bound: 8 bytes (weight, ordinal) per entry and head read, and the moved rows read and written.
// The keys stay in shared memory between the digits (up to kKeysInShared per CTA; longer shares are
// read again).
#include <cooperative_groups.h>

#include <algorithm>

#include "cache_device.cuh"

namespace rra {

namespace cg = cooperative_groups;

namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kKeysInShared = 32768;

__global__ void __launch_bounds__(256) evict_own_kernel(const __grid_constant__ EvictParams p) {
  const CacheView &c = p.c;
  const int b = blockIdx.x;
  const int raw = c.len[b];
  const int n = cache_len(c, b);
  const int pages = (n + c.ps - 1) / c.ps;
  if (threadIdx.x == 0) {
    p.skip[b] = 0;
    p.plan[c.batch * c.hkv + b] = n;
    if (raw != n) raise(c.status, kErrBadLength);
  }
  for (int i = threadIdx.x; i < pages; i += 256) {
    const int pg = page_at(c, b, i);
    if (pg >= 0) p.owner[pg] = b * c.max_pages + i;
  }
}

// Orders entries by what is kept first: protected entries, then the weight. Weights that are not
// above zero are 0; positive floats order like their bits.
__device__ __forceinline__ uint32_t entry_key(const EvictParams &p, int b, int head, int e,
                                              int64_t recent_from) {
  int slot, off;
  split_entry(p.c, e, slot, off);
  const int pg = page_at(p.c, b, slot);
  if (pg < 0) return 0;   // the sequence is skipped
  const int64_t at = track_at(p.c, pg, head, off);
  const int32_t order = __ldg(p.c.order + at);
  const float w = __ldg(p.c.weight + at);
  if (order < p.sinks || order >= recent_from) return 0xffffffffu;
  return w > 0.f ? __float_as_uint(w) : 0u;
}

// Exclusive prefix of `mine` over the warps of the block, then over the CTAs of the cluster before
// this one. s_warp: [kSelWarps], s_cta: one word that the other CTAs read.
__device__ int2 exclusive(cg::cluster_group &cl, int2 mine, int2 *s_warp, int2 *s_cta) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) s_warp[warp] = mine;
  __syncthreads();
  int2 before = make_int2(0, 0), all = make_int2(0, 0);
  for (int w = 0; w < kSelWarps; ++w) {
    const int2 x = s_warp[w];
    if (w < warp) {
      before.x += x.x;
      before.y += x.y;
    }
    all.x += x.x;
    all.y += x.y;
  }
  if (threadIdx.x == 0) *s_cta = all;
  cl.sync();
  for (unsigned k = 0; k < cl.block_rank(); ++k) {
    const int2 x = *cl.map_shared_rank(s_cta, k);
    before.x += x.x;
    before.y += x.y;
  }
  return before;
}

__global__ void __launch_bounds__(kSelThreads)
    evict_select_kernel(const __grid_constant__ EvictParams p, int keys_room) {
  extern __shared__ uint32_t s_keys[];
  __shared__ __align__(16) uint32_t s_hist[3][kBins];
  __shared__ uint32_t s_scan[kSelWarps];
  __shared__ int2 s_warp[3][kSelWarps];
  __shared__ int2 s_cta[3];
  __shared__ uint32_t s_found[3];

  const CacheView &c = p.c;
  cg::cluster_group cl = cg::this_cluster();
  const int ranks = cl.num_blocks(), rank = cl.block_rank();
  const int item = blockIdx.x / ranks;
  const int b = item / c.hkv, head = item - b * c.hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = p.plan[c.batch * c.hkv + b];

  // a page that the tables name twice: both of its sequences stay as they are
  if (head == 0) {
    const int pages = (n + c.ps - 1) / c.ps;
    for (int i = rank * kSelThreads + tid; i < pages; i += ranks * kSelThreads) {
      const int pg = page_at(c, b, i);
      const int me = b * c.max_pages + i;
      if (pg < 0) {
        p.skip[b] = 1;
      } else if (p.owner[pg] != me) {
        p.skip[b] = 1;
        p.skip[p.owner[pg] / c.max_pages] = 1;
        raise(c.status, kErrSharedPage);
      }
    }
  }
  if (n <= p.budget) {   // the same for the whole cluster
    if (rank == 0 && tid == 0) p.plan[item] = 0;
    return;
  }

  // each CTA takes a run of entries, each of its warps a run of those
  const int per_warp = ((n + ranks * kSelWarps - 1) / (ranks * kSelWarps) + 31) / 32 * 32;
  const int per = per_warp * kSelWarps;
  const int lo = min(rank * per, n), hi = min(lo + per, n);
  const int wlo = min(lo + warp * per_warp, hi), whi = min(wlo + per_warp, hi);
  const int64_t recent_from = static_cast<int64_t>(c.seen[b]) - p.recent;
  const bool kept_here = per <= keys_room;
  auto key_of = [&](int e) -> uint32_t {
    return kept_here ? s_keys[e - lo] : entry_key(p, b, head, e, recent_from);
  };

  for (int i = tid; i < 3 * kBins; i += kSelThreads) (&s_hist[0][0])[i] = 0;
  __syncthreads();
  uint32_t want = p.budget;    // the want-th largest key among those that match the digits so far
  uint32_t prefix = 0;
  uint32_t ties = 0;           // keys equal to the found one
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const int bits = pass == 2 ? 10 : 11;
    const uint32_t mask = pass == 0 ? 0u : (pass == 1 ? 0xffe00000u : 0xfffffc00u);
    for (int e0 = wlo; e0 < whi; e0 += 32) {
      const int e = e0 + lane;
      bool in = e < whi;
      uint32_t key = 0;
      if (in) {
        if (pass == 0) {
          key = entry_key(p, b, head, e, recent_from);
          if (kept_here) s_keys[e - lo] = key;
        } else {
          key = key_of(e);
        }
        in = (key & mask) == prefix;
      }
      const uint32_t bin = in ? (key >> shift) & ((1u << bits) - 1u) : 0xffffffffu;
      // equal bins of a warp are added once: most weights share their exponent
      const uint32_t peers = __match_any_sync(0xffffffffu, bin);
      if (in && lane == __ffs(peers) - 1)
        atomicAdd(&s_hist[pass][bin], static_cast<uint32_t>(__popc(peers)));
    }
    cl.sync();
    // thread i holds the bins from the top: kBins - 1 - 4 i and the three below it
    uint32_t cnt[4] = {0, 0, 0, 0};
    const int top = kBins - 1 - 4 * tid;
    for (int k = 0; k < ranks; ++k) {
      const uint32_t *h = cl.map_shared_rank(&s_hist[pass][0], k);
      const uint4 x = *reinterpret_cast<const uint4 *>(h + top - 3);
      cnt[0] += x.w;
      cnt[1] += x.z;
      cnt[2] += x.y;
      cnt[3] += x.x;
    }
    uint32_t sum = cnt[0] + cnt[1] + cnt[2] + cnt[3];
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    uint32_t above = incl - sum;
    for (int w = 0; w < warp; ++w) above += s_scan[w];
    if (above < want && want <= above + sum) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (above < want && want <= above + cnt[k]) {
          s_found[0] = (static_cast<uint32_t>(top - k) << shift);
          s_found[1] = want - above;
          s_found[2] = cnt[k];
        }
        above += cnt[k];
      }
    }
    __syncthreads();
    prefix |= s_found[0];
    want = s_found[1];
    ties = s_found[2];
    __syncthreads();
  }

  // keys above `prefix` are kept, and the first `want` of the `ties` equal ones
  int tie_rank = 0;
  const bool some = want < ties;
  if (some) {
    int mine = 0;
    for (int e0 = wlo; e0 < whi; e0 += 32) {
      const int e = e0 + lane;
      mine += __popc(__ballot_sync(0xffffffffu, e < whi && key_of(e) == prefix));
    }
    tie_rank = exclusive(cl, make_int2(mine, 0), s_warp[0], &s_cta[0]).x;
  }
  const uint32_t below = (1u << lane) - 1u;
  int32_t *holes = p.moves + static_cast<int64_t>(item) * 2 * p.moves_cap;
  int32_t *movers = holes + p.moves_cap;
  int2 at = make_int2(0, 0);
  for (int write = 0; write < 2; ++write) {
    int rank_now = tie_rank;
    int2 seen = make_int2(0, 0);
    for (int e0 = wlo; e0 < whi; e0 += 32) {
      const int e = e0 + lane;
      const bool in = e < whi;
      const uint32_t key = in ? key_of(e) : 0u;
      const bool tie = in && key == prefix;
      const uint32_t tied = __ballot_sync(0xffffffffu, tie);
      const bool kept =
          in && (key > prefix ||
                 (tie && (!some || rank_now + __popc(tied & below) < static_cast<int>(want))));
      rank_now += __popc(tied);
      const bool hole = in && !kept && e < p.budget, mover = kept && e >= p.budget;
      const uint32_t hs = __ballot_sync(0xffffffffu, hole);
      const uint32_t ms = __ballot_sync(0xffffffffu, mover);
      if (write) {
        if (hole) holes[at.x + seen.x + __popc(hs & below)] = e;
        if (mover) movers[at.y + seen.y + __popc(ms & below)] = e;
      }
      seen.x += __popc(hs);
      seen.y += __popc(ms);
    }
    if (!write) {
      at = exclusive(cl, seen, s_warp[1], &s_cta[1]);
    } else if (rank == ranks - 1 && tid == kSelThreads - 1) {
      p.plan[item] = at.x + seen.x;
    }
  }
  cl.sync();   // no CTA leaves while another reads its shared memory
}

// One warp per move: the lower half of its lanes takes the key row, the upper the value row.
template <int D>
__global__ void __launch_bounds__(256) evict_move_kernel(const __grid_constant__ EvictParams p,
                                                         int chunks) {
  constexpr int VECS = D / 8;                  // 16-byte vectors of a row
  constexpr int LANES = 2 * VECS;              // lanes of one move: 32 or 16
  const CacheView &c = p.c;
  const int item = blockIdx.x / chunks, part = blockIdx.x - item * chunks;
  const int b = item / c.hkv, head = item - b * c.hkv;
  if (p.skip[b]) return;
  const int n = p.plan[c.batch * c.hkv + b];
  if (p.advance && head == 0 && part == 0 && threadIdx.x == 0 && n > p.budget)
    c.len[b] = p.budget;
  const int moves = p.plan[item];
  const int32_t *holes = p.moves + static_cast<int64_t>(item) * 2 * p.moves_cap;
  const int32_t *movers = holes + p.moves_cap;
  const int sub = threadIdx.x % LANES;
  uint8_t *base = (sub < VECS ? c.k : c.v) + head * c.head_bytes + (sub % VECS) * 16;
  for (int j = part * (256 / LANES) + threadIdx.x / LANES; j < moves;
       j += chunks * (256 / LANES)) {
    int slot, doff, soff;
    split_entry(c, __ldg(holes + j), slot, doff);
    const int dst = page_at(c, b, slot);
    split_entry(c, __ldg(movers + j), slot, soff);
    const int src = page_at(c, b, slot);
    if (dst < 0 || src < 0) continue;
    *reinterpret_cast<uint4 *>(base + dst * c.page_bytes + doff * c.entry_bytes) =
        *reinterpret_cast<const uint4 *>(base + src * c.page_bytes + soff * c.entry_bytes);
    const int64_t to = track_at(c, dst, head, doff), from = track_at(c, src, head, soff);
    if (sub == 0) c.weight[to] = c.weight[from];
    if (sub == 1) c.order[to] = c.order[from];
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, int num_sms, cudaStream_t stream) {
  const CacheView &c = p.c;
  const int items = c.batch * c.hkv;
  evict_own_kernel<<<c.batch, 256, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;

  // CTAs per cluster by what the table can hold: a CTA's share should stay near 2048 entries
  int ranks = 1;
  while (ranks < 8 && c.cap > ranks * 2048) ranks *= 2;
  int64_t room = (static_cast<int64_t>(c.cap) + ranks - 1) / ranks + 32 * kSelWarps;
  if (room > kKeysInShared) room = kKeysInShared;
  const size_t smem = static_cast<size_t>(room) * 4;
  e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kKeysInShared * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items) * ranks);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ranks;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p, static_cast<int>(room));
  if (e != cudaSuccess) return e;

  const int chunks = std::min(512, (num_sms * 8 + items - 1) / items);
  const unsigned grid = static_cast<unsigned>(items) * chunks;
  if (c.d == 128)
    evict_move_kernel<128><<<grid, 256, 0, stream>>>(p, chunks);
  else
    evict_move_kernel<64><<<grid, 256, 0, stream>>>(p, chunks);
  return cudaGetLastError();
}

}  // namespace rra
