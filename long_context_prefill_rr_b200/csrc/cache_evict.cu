// Eviction by accumulated attention weight, in place, per (sequence, KV head): keep the protected
// entries (the first tokens and the last ones, by their ordinals) and then those of the largest
// weight, `budget` in all. Two launches:
//
//   select  a cluster of CTAs per (sequence, KV head) finds the budget-th largest key by a radix
//           descent (11, 11 and 10 bits; the histograms are summed over the cluster through
//           distributed shared memory) and lists the evicted places e < budget and the kept
//           entries e >= budget, both in ascending order: there are as many of one as of the other.
//           Along the way it claims the sequences' pages: a page claimed twice in a call is named twice by
//           the tables, and its sequences are left alone;
//   move    copies kept entry j of the second list over place j of the first. Sources and targets
//           never overlap, so every row moves on its own, and a bounded cache that is one entry over its
//           budget moves one row per head, not the cache.
//
// Bound: 8 bytes (weight, ordinal) per entry and head read, and the moved rows read and written; for
// short caches the chain of dependent steps (length, page, weight, three digits).
#include <cooperative_groups.h>

#include <algorithm>

#include "cache_device.cuh"

namespace rra {

namespace cg = cooperative_groups;

namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMoveWarps = 8;

// Orders entries by what is kept first: protected entries, then the weight. Weights that are not
// above zero are 0; positive floats order like their bits.
__device__ __forceinline__ uint32_t entry_key(const EvictParams &p, int32_t order, float w,
                                              int64_t recent_from) {
  if (order < p.sinks || order >= recent_from) return 0xffffffffu;
  return w > 0.f ? __float_as_uint(w) : 0u;
}

// All threads of the cluster; of the block where it is alone.
__device__ __forceinline__ void sync_all(cg::cluster_group &cl, int ranks) {
  if (ranks > 1)
    cl.sync();
  else
    __syncthreads();
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
  if (cl.num_blocks() == 1) return before;
  if (threadIdx.x == 0) *s_cta = all;
  cl.sync();
  for (unsigned k = 0; k < cl.block_rank(); ++k) {
    const int2 x = *cl.map_shared_rank(s_cta, k);
    before.x += x.x;
    before.y += x.y;
  }
  return before;
}

// KPT: keys that a thread holds in registers; a CTA's share of more than KPT * kSelThreads entries is
// taken in rounds and read again for every digit.
template <int KPT>
__global__ void __launch_bounds__(kSelThreads)
    evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ __align__(16) uint32_t s_hist[3][kBins];
  __shared__ uint32_t s_scan[kSelWarps];
  __shared__ int2 s_warp[2][kSelWarps];
  __shared__ int2 s_cta[2];
  __shared__ uint32_t s_found[3];

  const CacheView &c = p.c;
  cg::cluster_group cl = cg::this_cluster();
  const int ranks = cl.num_blocks(), rank = cl.block_rank();
  const int item = blockIdx.x / ranks;
  const int b = item / c.hkv, head = item - b * c.hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  for (int i = tid; i < 3 * kBins / 4; i += kSelThreads)
    reinterpret_cast<uint4 *>(&s_hist[0][0])[i] = make_uint4(0, 0, 0, 0);
  grid_dependency_wait();
  grid_dependents_go();
  const int raw = c.len[b];
  const uint32_t tag = *p.epoch + 1u;   // the same for the whole call; the move kernel moves it on
  const int64_t recent_from = static_cast<int64_t>(c.seen[b]) - p.recent;
  const int n = raw < 0 ? 0 : min(raw, c.cap);
  if (rank == 0 && head == 0 && tid == 0) {
    if (raw != n) raise(c.status, kErrBadLength);
    p.lens[b] = n;
    p.tags[b] = tag;
  }
  // The pages of the sequence, shared out over its heads. A page that comes back with this call's tag was
  // claimed before: both of its sequences stay as they are.
  const int pages = (n + c.ps - 1) / c.ps;
  for (int i = (head * ranks + rank) * kSelThreads + tid; i < pages;
       i += c.hkv * ranks * kSelThreads) {
    const int pg = page_at(c, b, i);
    if (pg < 0) {
      p.skip[b] = tag;
      continue;
    }
    const unsigned long long me =
        (static_cast<unsigned long long>(tag) << 32) | static_cast<unsigned>(b);
    const unsigned long long was = atomicExch(p.owner + pg, me);
    if (static_cast<uint32_t>(was >> 32) == tag) {
      p.skip[b] = tag;
      p.skip[static_cast<uint32_t>(was)] = tag;
      raise(c.status, kErrSharedPage);
    }
  }
  if (n <= p.budget) {   // the same for the whole cluster
    if (rank == 0 && tid == 0) p.plan[item] = 0;
    return;
  }

  // each CTA takes a run of entries, each of its warps a run of those
  const int per_warp = ((n + ranks * kSelWarps - 1) / (ranks * kSelWarps) + 31) / 32 * 32;
  const int wlo = min((rank * kSelWarps + warp) * per_warp, n), whi = min(wlo + per_warp, n);
  const int rounds = (per_warp + KPT * 32 - 1) / (KPT * 32);
  uint32_t key[KPT];
  // key[k] of entry wlo + (round * KPT + k) * 32 + lane. The pages of a batch are looked up together, then
  // its weights and ordinals; a page that is none (the sequence is left alone) reads as page 0.
  auto load = [&](int round) {
    constexpr int BATCH = KPT < 8 ? KPT : 8;
    const int e0 = wlo + round * KPT * 32 + lane;
#pragma unroll
    for (int k0 = 0; k0 < KPT; k0 += BATCH) {
      int64_t at[BATCH];
      int32_t order[BATCH];
      float w[BATCH];
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const int e = min(e0 + (k0 + k) * 32, n - 1);
        int slot, off;
        split_entry(c, e, slot, off);
        const int pg = c.table[b * c.table_stride + slot];
        at[k] = track_at(c, static_cast<unsigned>(pg) < static_cast<unsigned>(c.num_pages) ? pg : 0,
                         head, off);
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        order[k] = __ldcg(c.order + at[k]);
        w[k] = __ldcg(c.weight + at[k]);
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k) key[k0 + k] = entry_key(p, order[k], w[k], recent_from);
    }
  };
  load(0);
  __syncthreads();

  uint32_t want = p.budget;    // the want-th largest key among those that match the digits so far
  uint32_t prefix = 0;
  uint32_t ties = 0;           // keys equal to the found one
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t digit = pass == 2 ? 0x3ffu : 0x7ffu;
    const uint32_t mask = pass == 0 ? 0u : (pass == 1 ? 0xffe00000u : 0xfffffc00u);
    uint32_t *hist = s_hist[pass];
    for (int round = 0; round < rounds; ++round) {
      if (rounds > 1) load(round);
      const int e0 = wlo + round * KPT * 32 + lane;
#pragma unroll
      for (int k = 0; k < KPT; ++k) {
        const bool in = e0 + k * 32 < whi && (key[k] & mask) == prefix;
        const uint32_t votes = __ballot_sync(0xffffffffu, in);
        if (votes == 0) continue;
        // one add where all the lanes agree (equal weights, protected runs), else one per lane
        const uint32_t bin = (key[k] >> shift) & digit;
        const int first = __ffs(votes) - 1;
        const uint32_t lead = __shfl_sync(0xffffffffu, bin, first);
        if (__all_sync(0xffffffffu, !in || bin == lead)) {
          if (lane == first) atomicAdd(&hist[bin], static_cast<uint32_t>(__popc(votes)));
        } else if (in) {
          atomicAdd(&hist[bin], 1u);
        }
      }
    }
    sync_all(cl, ranks);
    // thread i holds the bins from the top: kBins - 1 - 4 i and the three below it
    uint32_t cnt[4] = {0, 0, 0, 0};
    const int top = kBins - 1 - 4 * tid;
    for (int k = 0; k < ranks; ++k) {
      const uint32_t *h = cl.map_shared_rank(hist, k);
      const uint4 x = *reinterpret_cast<const uint4 *>(h + top - 3);
      cnt[0] += x.w;
      cnt[1] += x.z;
      cnt[2] += x.y;
      cnt[3] += x.x;
    }
    const uint32_t sum = cnt[0] + cnt[1] + cnt[2] + cnt[3];
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    uint32_t above = incl - sum;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) above += w < warp ? s_scan[w] : 0u;
    if (above < want && want <= above + sum) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (above < want && want <= above + cnt[k]) {
          s_found[0] = static_cast<uint32_t>(top - k) << shift;
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
  }

  // keys above `prefix` are kept, and the first `want` of the `ties` equal ones
  int tie_rank = 0;
  const bool some = want < ties;
  if (some) {
    int mine = 0;
    for (int round = 0; round < rounds; ++round) {
      if (rounds > 1) load(round);
      const int e0 = wlo + round * KPT * 32 + lane;
#pragma unroll
      for (int k = 0; k < KPT; ++k)
        mine += __popc(__ballot_sync(0xffffffffu, e0 + k * 32 < whi && key[k] == prefix));
    }
    tie_rank = exclusive(cl, make_int2(mine, 0), s_warp[0], &s_cta[0]).x;
  }
  const uint32_t below = (1u << lane) - 1u;
  int32_t *holes = p.moves + static_cast<int64_t>(item) * 2 * p.moves_cap;
  int32_t *movers = holes + p.moves_cap;
  int2 at = make_int2(0, 0);
#pragma unroll 1
  for (int write = 0; write < 2; ++write) {
    int rank_now = tie_rank;
    int2 seen = make_int2(0, 0);
    for (int round = 0; round < rounds; ++round) {
      if (rounds > 1) load(round);
      const int e0 = wlo + round * KPT * 32 + lane;
#pragma unroll
      for (int k = 0; k < KPT; ++k) {
        const int e = e0 + k * 32;
        const bool in = e < whi;
        const bool tie = in && key[k] == prefix;
        const uint32_t tied = __ballot_sync(0xffffffffu, tie);
        const bool kept =
            in && (key[k] > prefix ||
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
    }
    if (!write) {
      at = exclusive(cl, seen, s_warp[1], &s_cta[1]);
    } else if (rank == ranks - 1 && tid == kSelThreads - 1) {
      p.plan[item] = at.x + seen.x;
    }
  }
  if (ranks > 1) cl.sync();   // no CTA leaves while another reads its shared memory
}

// A warp takes kFlight moves (twice as many for head_dim 64, whose two rows fill half a warp) of a
// (sequence, KV head) at a time: as many lanes find the places of one each and move its weight and
// ordinal, then the warp copies the rows, all loads before the first store.
constexpr int kFlight = 8;

template <int D>
__global__ void __launch_bounds__(kMoveWarps * 32)
    evict_move_kernel(const __grid_constant__ EvictParams p, int parts) {
  constexpr int VECS = D / 8;                  // 16-byte vectors of a row
  constexpr int PER = 32 / (2 * VECS);         // moves whose key and value rows fill a warp: 1 or 2
  constexpr int TAKE = kFlight * PER;
  const CacheView &c = p.c;
  const int lane = threadIdx.x & 31;
  const int items = c.batch * c.hkv;
  grid_dependency_wait();
  grid_dependents_go();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.epoch += 1u;
  const int sub = lane % (2 * VECS), which = lane / (2 * VECS);
  const int warps = gridDim.x * kMoveWarps;
  for (int64_t w = blockIdx.x * kMoveWarps + (threadIdx.x >> 5);
       w < static_cast<int64_t>(items) * parts; w += warps) {
    const int item = static_cast<int>(w / parts);
    const int part = static_cast<int>(w - static_cast<int64_t>(item) * parts);
    const int b = item / c.hkv, head = item - b * c.hkv;
    const uint32_t skip = p.skip[b], tag = p.tags[b];
    const int moves = p.plan[item], n = p.lens[b];
    if (skip == tag) continue;
    if (p.advance && head == 0 && part == 0 && lane == 0 && n > p.budget) c.len[b] = p.budget;
    const int32_t *holes = p.moves + static_cast<int64_t>(item) * 2 * p.moves_cap;
    const int32_t *movers = holes + p.moves_cap;
    uint8_t *base = (sub < VECS ? c.k : c.v) + head * c.head_bytes + (sub % VECS) * 16;
    for (int j0 = part * TAKE; j0 < moves; j0 += parts * TAKE) {
      int64_t to = -1, from = -1;
      if (lane < TAKE && j0 + lane < moves) {
        int dslot, sslot, doff, soff;
        split_entry(c, __ldcg(holes + j0 + lane), dslot, doff);
        split_entry(c, __ldcg(movers + j0 + lane), sslot, soff);
        const int dst = c.table[b * c.table_stride + dslot];
        const int src = c.table[b * c.table_stride + sslot];
        // the pages of a sequence that is not skipped were checked when they were claimed
        to = dst * c.page_bytes + doff * c.entry_bytes;
        from = src * c.page_bytes + soff * c.entry_bytes;
        const int64_t tw = track_at(c, dst, head, doff), fw = track_at(c, src, head, soff);
        c.weight[tw] = __ldcg(c.weight + fw);
        c.order[tw] = __ldcg(c.order + fw);
      }
      uint4 row[kFlight];
      int64_t dst[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int64_t s = __shfl_sync(0xffffffffu, from, i * PER + which);
        dst[i] = __shfl_sync(0xffffffffu, to, i * PER + which);
        if (dst[i] >= 0) row[i] = ld_stream(base + s);
      }
#pragma unroll
      for (int i = 0; i < kFlight; ++i)
        if (dst[i] >= 0) *reinterpret_cast<uint4 *>(base + dst[i]) = row[i];
    }
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, int num_sms, cudaStream_t stream) {
  const CacheView &c = p.c;
  const int items = c.batch * c.hkv;
  // CTAs per cluster and keys per thread by what the table can hold: one CTA up to 4096 entries, up
  // to eight of them for longer ones
  int ranks = 1;
  while (ranks < 8 && c.cap > ranks * 4096) ranks *= 2;
  const int share = (c.cap + ranks * kSelThreads - 1) / (ranks * kSelThreads);
  auto kern = share <= 4 ? evict_select_kernel<4>
                         : (share <= 8 ? evict_select_kernel<8> : evict_select_kernel<32>);
  cudaError_t e = launch_dependent(kern, dim3(static_cast<unsigned>(items) * ranks), kSelThreads, 0,
                                   ranks, stream, p);
  if (e != cudaSuccess) return e;
  const int warps = num_sms * 4 * kMoveWarps;
  const int parts = std::max(1, warps / items);
  const int64_t blocks = (static_cast<int64_t>(items) * parts + kMoveWarps - 1) / kMoveWarps;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(num_sms * 4, blocks)));
  return c.d == 128 ? launch_dependent(evict_move_kernel<128>, grid, kMoveWarps * 32, 0, 1, stream,
                                       p, parts)
                    : launch_dependent(evict_move_kernel<64>, grid, kMoveWarps * 32, 0, 1, stream,
                                       p, parts);
}

}  // namespace rra
