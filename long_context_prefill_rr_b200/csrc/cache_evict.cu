// Eviction by accumulated attention weight, in place, per (sequence, KV head): keep the protected
// entries (the first tokens and the last ones, by their ordinals) and then those of the largest
// weight, `budget` in all. Two launches:
//
//   select  a block or a cluster per (sequence, KV head) finds the budget-th largest key by a radix
//           descent (digits of 8 bits; the histograms are summed over the cluster through
//           distributed shared memory) and lists the evicted places e < budget and the kept
//           entries e >= budget, both in ascending order: there are as many of one as of the other.
//           Along the way it claims the sequences' pages: a page claimed twice in a call is named twice by
//           the tables, and its sequences are left alone;
//   move    copies kept entry j of the second list over place j of the first. Sources and targets
//           never overlap, so every row moves on its own, and a bounded cache that is one entry over its
//           budget moves one row per head, not the cache.
//
// Bound: 8 bytes (weight, ordinal) per entry and head read, and the moved rows read and written. Measured
// from cold caches (8 KV heads of 128, bf16): 32 sequences one entry over 2048, select 11 us and move 6; one
// of 128K cut to 16K, 25 and 24 (the bytes take 18); eight of 32K cut to 8K, 26 and 74 (62). The move runs
// at 75-83% of the copy rate; select is bound by its chain of dependent steps: length, page, weight, four
// digits and the ranks of the lists, each with a barrier of the block or cluster. Taking the entries four
// at a time halved its instructions and saved 2 us of 28; digits found bit by bit took 760 cycles a bit
// against 1700 a digit; keys in registers, unrolled, were no faster than these rolled loops (each stretch
// of new instructions has to be fetched first); a third launch that marked the pages beforehand cost 3 us;
// dealing the moves out over warps that stay made the move slower (52 us against 44, five ragged sequences).
#include <cooperative_groups.h>

#include <limits.h>

#include <algorithm>
#include <atomic>

#include "cache_device.cuh"

namespace rra {

namespace cg = cooperative_groups;

namespace {

constexpr int kBins = 256;
constexpr int kPasses = 4;         // digits of 8, 8, 8 and 7 bits from bit 30 down
constexpr uint32_t kProtected = 0x7fffffffu;
constexpr int kKeyRoom = 16384;    // keys that a CTA of a cluster holds in shared memory, 64 KB
constexpr int kMoveWarps = 8;
constexpr int kRanks = 8;          // CTAs of a cluster at most

// What a sequence is cut by.
struct Cut {
  int n;               // entries
  uint32_t tag;        // the call's mark, one above the count of calls (the move kernel moves that on)
  int recent_from;     // ordinals from here on are protected
};

__device__ __forceinline__ Cut read_cut(const EvictParams &p, int b, bool first) {
  const CacheView &c = p.c;
  const int raw = c.len[b];
  Cut cut;
  cut.tag = *p.epoch + 1u;
  // seen - recent, or the lowest ordinal if that is below it
  const int seen = c.seen[b];
  cut.recent_from = seen < INT_MIN + p.recent ? INT_MIN : seen - p.recent;
  cut.n = raw < 0 ? 0 : min(raw, c.cap);
  if (first) {
    if (raw != cut.n) raise(c.status, kErrBadLength);
    p.lens[b] = cut.n;
    p.tags[b] = cut.tag;
  }
  return cut;
}

// Claims the pages `part`, `part` + `parts`, ... of the sequence. A page that comes back with this
// call's tag was claimed before: both of its sequences stay as they are.
__device__ __forceinline__ void claim_pages(const EvictParams &p, int b, const Cut &cut, int part,
                                            int parts) {
  const CacheView &c = p.c;
  const int pages = (cut.n + c.ps - 1) / c.ps;
  for (int i = part; i < pages; i += parts) {
    const int pg = page_at(c, b, i);
    if (pg < 0) {
      p.skip[b] = cut.tag;
      continue;
    }
    const unsigned long long me =
        (static_cast<unsigned long long>(cut.tag) << 32) | static_cast<unsigned>(b);
    const unsigned long long was = atomicExch(p.owner + pg, me);
    if (static_cast<uint32_t>(was >> 32) == cut.tag) {
      // (a sequence of this cache, unless the workspace was laid out for another and not zero-filled since)
      const int other = static_cast<int>(min(static_cast<uint32_t>(was), c.batch - 1u));
      p.skip[b] = cut.tag;
      p.skip[other] = cut.tag;
      // no mistake as long as neither of them is to be cut
      if (cut.n > p.budget || cache_len(c, other) > p.budget) raise(c.status, kErrSharedPage);
    }
  }
}

// Sum over the lanes below, of x.
__device__ __forceinline__ uint32_t lane_prefix(uint32_t x, int lane) {
  uint32_t incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  return incl - x;
}

__device__ __forceinline__ int digit_shift(int pass) { return pass == 3 ? 0 : 23 - 8 * pass; }

// What the descent has found: `prefix` holds the digits of the want-th largest key so far, `ties` the
// keys that share them.
struct Found {
  uint32_t prefix, want, ties, more;   // more: there is a next digit
};

// One digit, found by one warp (lane i holds eight of the bins, from the top). Returns false if the bins
// hold fewer than f->want keys, which are taken off f->want.
__device__ __forceinline__ bool descend(const uint32_t *bins, int pass, Found *f) {
  const int lane = threadIdx.x & 31;
  const int top = kBins - 8 - 8 * lane;
  const uint4 hi = *reinterpret_cast<const uint4 *>(bins + top + 4);
  const uint4 lo = *reinterpret_cast<const uint4 *>(bins + top);
  const uint32_t cnt[8] = {hi.w, hi.z, hi.y, hi.x, lo.w, lo.z, lo.y, lo.x};
  uint32_t sum = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum += cnt[i];
  const uint32_t before = lane_prefix(sum, lane);
  const uint32_t here = __ballot_sync(0xffffffffu, before < f->want && f->want <= before + sum);
  if (here == 0) {
    f->want -= __shfl_sync(0xffffffffu, before + sum, 31);
    return false;
  }
  uint32_t passed = before, above = before, mine = 0, ties = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (passed < f->want) {      // the last bin that satisfies this is the one
      mine = i;
      above = passed;
      ties = cnt[i];
    }
    passed += cnt[i];
  }
  const int from = __ffs(here) - 1;
  f->want -= __shfl_sync(0xffffffffu, above, from);
  f->ties = __shfl_sync(0xffffffffu, ties, from);
  f->prefix |= __shfl_sync(0xffffffffu, static_cast<uint32_t>(top) + 7u - mine, from)
               << digit_shift(pass);
  return true;
}

// Prefix of the warps' values `mine` over the block, and with CLUSTER over the CTAs before this one too.
// s_warp: [WARPS]; s_cta: a pair that the other CTAs read.
template <int WARPS, bool CLUSTER>
__device__ __forceinline__ int2 prefix_of_warps(int2 mine, int2 *s_warp, int2 *s_cta, int2 *all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) s_warp[warp] = mine;
  __syncthreads();
  const int2 v = lane < WARPS ? s_warp[lane] : make_int2(0, 0);
  const int x = static_cast<int>(lane_prefix(v.x, lane)), y = static_cast<int>(lane_prefix(v.y, lane));
  *all = make_int2(__shfl_sync(0xffffffffu, x + v.x, 31), __shfl_sync(0xffffffffu, y + v.y, 31));
  int2 before = make_int2(__shfl_sync(0xffffffffu, x, warp), __shfl_sync(0xffffffffu, y, warp));
  if (CLUSTER) {
    cg::cluster_group cl = cg::this_cluster();
    if (threadIdx.x == 0) *s_cta = *all;
    cl.sync();
    const int ranks = cl.num_blocks(), rank = cl.block_rank();
    const int2 z = lane < ranks ? *cl.map_shared_rank(s_cta, lane) : make_int2(0, 0);
    const int zx = static_cast<int>(lane_prefix(z.x, lane)), zy = static_cast<int>(lane_prefix(z.y, lane));
    before.x += __shfl_sync(0xffffffffu, zx, rank);
    before.y += __shfl_sync(0xffffffffu, zy, rank);
    *all = make_int2(__shfl_sync(0xffffffffu, zx, 31), __shfl_sync(0xffffffffu, zy, 31));
  }
  return before;
}

// What the keys of a (sequence, KV head) are made of; passed by value, so that it stays in registers.
struct KeySource {
  const int32_t *table, *order;   // the sequence's pages; the head's ordinals and
  const float *weight;            // weights in page 0
  int page_stride, num_pages, ps;
  uint32_t ps_magic, ps_shift;
  int sinks, recent_from;
  bool four;                      // four consecutive entries from a multiple of four are one aligned vector

  __device__ __forceinline__ int64_t at(int e) const {
    const int slot = static_cast<int>(__umulhi(static_cast<uint32_t>(e) * 2u, ps_magic) >> ps_shift);
    const int pg = table[slot];
    // a page that is none (the sequence is left alone) reads as page 0
    const int page = static_cast<unsigned>(pg) < static_cast<unsigned>(num_pages) ? pg : 0;
    return static_cast<int64_t>(page) * page_stride + (e - slot * ps);
  }
  __device__ __forceinline__ uint32_t key(int32_t ordinal, float w) const {
    if (ordinal < sinks || ordinal >= recent_from) return kProtected;
    return w > 0.f ? __float_as_uint(w) : 0u;
  }
};

// Keys of the entries e0 + 128 g + 4 lane + (0 .. 3), g < groups, to keys[128 g + 4 lane + ...]: what is kept
// first has the larger key. Protected entries come first, then the weight: those not above zero are 0,
// positive floats order like their bits and infinity is 0x7f800000, so 31 bits do. Entries at or past
// `end` get key 0. Returns the protected entries of the lane.
__device__ __noinline__ int load_keys(const KeySource src, int e0, int end, int groups, uint32_t *keys) {
  const int lane = threadIdx.x & 31;
  int safe = 0;
  int64_t next = 0;
  if (groups > 0) next = src.at(min(e0 + lane * 4, end - 1));
#pragma unroll 1
  for (int g = 0; g < groups; ++g) {
    const int e = e0 + g * 128 + lane * 4;
    int32_t order[4];
    float w[4];
    if (src.four && e < end) {
      // (the rest of a vector whose first entries exist lies in the same page)
      const int4 o = __ldcg(reinterpret_cast<const int4 *>(src.order + next));
      const float4 x = __ldcg(reinterpret_cast<const float4 *>(src.weight + next));
      order[0] = o.x, order[1] = o.y, order[2] = o.z, order[3] = o.w;
      w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else {
      int64_t at[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) at[j] = src.at(min(e + j, end - 1));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        order[j] = __ldcg(src.order + at[j]);
        w[j] = __ldcg(src.weight + at[j]);
      }
    }
    next = src.at(min(e + 128, end - 1));   // the next page, while the weights are on their way
    uint32_t key[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      key[j] = e + j < end ? src.key(order[j], w[j]) : 0u;
      safe += key[j] == kProtected;
    }
    *reinterpret_cast<uint4 *>(keys + g * 128 + lane * 4) = make_uint4(key[0], key[1], key[2], key[3]);
  }
  return safe;
}

// One block, or one cluster of blocks, per (sequence, KV head). room: keys that the dynamic shared
// memory holds; a CTA's share of more entries is taken in rounds and read again for every digit. Loops are
// kept rolled: a short call is bound by latencies, instruction fetches among them.
template <int THREADS, bool CLUSTER>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
    evict_select_kernel(const __grid_constant__ EvictParams p, int room) {
  constexpr int WARPS = THREADS / 32;
  extern __shared__ __align__(16) uint32_t s_keys[];
  __shared__ __align__(16) uint32_t s_hist[kPasses][kBins], s_sum[2][kBins];
  __shared__ uint32_t s_safe;
  __shared__ Found s_found;
  __shared__ int2 s_warp[2][WARPS];
  __shared__ int2 s_cta[3];

  const CacheView &c = p.c;
  cg::cluster_group cl = cg::this_cluster();
  const int ranks = CLUSTER ? cl.num_blocks() : 1, rank = CLUSTER ? cl.block_rank() : 0;
  const int item = blockIdx.x / ranks;
  const int b = item / c.hkv, head = item - b * c.hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  for (int i = tid; i < kPasses * kBins; i += THREADS) (&s_hist[0][0])[i] = 0;
  if (tid == 0) s_safe = 0;
  grid_dependency_wait();
  grid_dependents_go();
  const Cut cut = read_cut(p, b, rank == 0 && head == 0 && tid == 0);
  const int n = cut.n;
  int moves = 0;
  if (n > p.budget) {   // the same for the whole cluster
    // each CTA takes a run of entries, each of its warps a run of those, in rounds of `take` groups of 128
    const int per_warp = (n + ranks * THREADS * 4 - 1) / (ranks * THREADS * 4) * 128;
    const int wlo = min((rank * WARPS + warp) * per_warp, n), whi = min(wlo + per_warp, n);
    const int take = room / (THREADS * 4);
    const int rounds = (per_warp / 128 + take - 1) / take;
    uint32_t *keys = s_keys + warp * take * 128;
    const KeySource src = {c.table + b * c.table_stride,
                           c.order + static_cast<int64_t>(head) * c.ps,
                           c.weight + static_cast<int64_t>(head) * c.ps,
                           c.hkv * c.ps, c.num_pages, c.ps, c.ps_magic, c.ps_shift,
                           p.sinks, cut.recent_from, p.four != 0};
    int safe = 0;
    // groups of a round, after reading its keys unless they are there
    auto groups_of = [&](int round, bool first) {
      const int e0 = wlo + round * take * 128;
      const int groups = (max(0, min(whi - e0, take * 128)) + 127) / 128;
      if (first || rounds > 1) {
        const int found = load_keys(src, e0, whi, groups, keys);
        if (first) safe += found;
      }
      return groups;
    };
    auto keys_of = [&](int g) { return *reinterpret_cast<const uint4 *>(keys + g * 128 + lane * 4); };

    // protected entries are counted apart, and entries of weight 0 not at all: both come in numbers
    for (int round = 0; round < rounds; ++round) groups_of(round, true);
    safe = __reduce_add_sync(0xffffffffu, safe);
    __syncthreads();
    if (lane == 0) atomicAdd(&s_safe, static_cast<uint32_t>(safe));

    Found f{0u, static_cast<uint32_t>(p.budget), 0u, 1u};
    bool exact = false;        // the keys at or above the prefix are as many as wanted
#pragma unroll 1
    for (int pass = 0; pass < kPasses && !exact; ++pass) {
      // the keys that share the digits found so far, without the zeros and the protected ones: a range
      const int shift = digit_shift(pass);
      const uint32_t span = pass == 0 ? 0x7fffffffu : (1u << digit_shift(pass - 1)) - 1u;
      const uint32_t low = max(f.prefix, 1u);
      const uint32_t width = min(f.prefix + span, kProtected - 1u) - low;
      for (int round = 0; round < rounds; ++round) {
        const int groups = groups_of(round, false);
#pragma unroll 2
        for (int g = 0; g < groups; ++g) {
          const uint4 k = keys_of(g);
          if (k.x - low <= width) atomicAdd(&s_hist[pass][(k.x - f.prefix) >> shift], 1u);
          if (k.y - low <= width) atomicAdd(&s_hist[pass][(k.y - f.prefix) >> shift], 1u);
          if (k.z - low <= width) atomicAdd(&s_hist[pass][(k.z - f.prefix) >> shift], 1u);
          if (k.w - low <= width) atomicAdd(&s_hist[pass][(k.w - f.prefix) >> shift], 1u);
        }
      }
      const uint32_t *bins = s_hist[pass];
      if (CLUSTER) {
        cl.sync();
        if (tid < kBins) {
          uint32_t sum = 0, part[kRanks];      // all of them asked for before the first is used
#pragma unroll
          for (int k = 0; k < kRanks; ++k)
            part[k] = k < ranks ? *cl.map_shared_rank(&s_hist[pass][tid], k) : 0u;
#pragma unroll
          for (int k = 0; k < kRanks; ++k) sum += part[k];
          s_sum[pass & 1][tid] = sum;
        }
        bins = s_sum[pass & 1];
      }
      __syncthreads();
      if (warp == 0) {
        Found g = f;
        g.more = 1;
        uint32_t in_front = 0;
        if (pass == 0)
          in_front = CLUSTER ? __reduce_add_sync(
                                   0xffffffffu, lane < ranks ? *cl.map_shared_rank(&s_safe, lane) : 0u)
                             : s_safe;
        if (in_front >= g.want) {          // more protected entries than places: the first of them
          g.prefix = kProtected;
          g.ties = in_front;
          g.more = 0;
        } else {
          g.want -= in_front;
          // every weight above 0 stays, and the first of the zeros
          if (!descend(bins, pass, &g)) g.more = 0;
        }
        if (lane == 0) s_found = g;
      }
      __syncthreads();
      f = s_found;
      exact = f.want == f.ties;
      if (!f.more) break;
    }
    if (exact && f.prefix == 0) f.prefix = 1;   // the zeros were not counted
    // kept: the keys at or above the prefix if exact, else those above it and the first f.want of those
    // equal to it
    const uint32_t least = exact ? f.prefix : f.prefix + 1u;
    int2 all;
    auto ties_of = [&](int e, const uint4 &k) -> uint32_t {     // as a mask of the lane's four
      const uint32_t m = (k.x == f.prefix ? 1u : 0u) | (k.y == f.prefix ? 2u : 0u) |
                         (k.z == f.prefix ? 4u : 0u) | (k.w == f.prefix ? 8u : 0u);
      return m & ((1u << max(0, min(whi - e, 4))) - 1u);
    };
    int tie_rank = 0;
    if (!exact) {
      int ties = 0;
      for (int round = 0; round < rounds; ++round) {
        const int groups = groups_of(round, false), e0 = wlo + round * take * 128 + lane * 4;
        for (int g = 0; g < groups; ++g) ties += __popc(ties_of(e0 + g * 128, keys_of(g)));
      }
      ties = __reduce_add_sync(0xffffffffu, ties);
      tie_rank = prefix_of_warps<WARPS, CLUSTER>(make_int2(ties, 0), s_warp[0], &s_cta[0], &all).x;
    }
    int32_t *holes = p.moves + static_cast<int64_t>(item) * 2 * p.moves_cap;
    int32_t *movers = holes + p.moves_cap;
    int rank_now = tie_rank;
    // Masks of the lane's four entries from e: the places to fill (x) and the entries to move (y).
    auto masks = [&](int e, const uint4 &k) {
      uint32_t kept = (k.x >= least ? 1u : 0u) | (k.y >= least ? 2u : 0u) | (k.z >= least ? 4u : 0u) |
                      (k.w >= least ? 8u : 0u);
      const uint32_t in = (1u << max(0, min(whi - e, 4))) - 1u;
      const uint32_t front = (1u << max(0, min(p.budget - e, 4))) - 1u;
      if (!exact) {
        const uint32_t tied = ties_of(e, k);
        const int before = static_cast<int>(lane_prefix(__popc(tied), lane));
        int left = static_cast<int>(f.want) - rank_now - before;   // ties of this lane that stay
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if ((tied >> j) & 1u) {
            if (left > 0) kept |= 1u << j;
            --left;
          }
        rank_now += __shfl_sync(0xffffffffu, before + __popc(tied), 31);
      }
      kept &= in;
      return make_uint2(in & front & ~kept, kept & ~front);
    };
    int2 seen = make_int2(0, 0);
    for (int round = 0; round < rounds; ++round) {
      const int groups = groups_of(round, false), e0 = wlo + round * take * 128 + lane * 4;
      for (int g = 0; g < groups; ++g) {
        const uint2 m = masks(e0 + g * 128, keys_of(g));
        seen.x += __popc(m.x);
        seen.y += __popc(m.y);
      }
    }
    seen.x = __reduce_add_sync(0xffffffffu, seen.x);
    seen.y = __reduce_add_sync(0xffffffffu, seen.y);
    int2 to = prefix_of_warps<WARPS, CLUSTER>(seen, s_warp[1], &s_cta[1], &all);
    moves = all.x;
    rank_now = tie_rank;
    for (int round = 0; round < rounds; ++round) {
      const int groups = groups_of(round, false), e0 = wlo + round * take * 128 + lane * 4;
      for (int g = 0; g < groups; ++g) {
        const int e = e0 + g * 128;
        const uint2 m = masks(e, keys_of(g));
        // both ranks in one prefix: a group has 128 entries
        const uint32_t mine = __popc(m.x) | (__popc(m.y) << 16);
        const uint32_t before = lane_prefix(mine, lane);
        const uint32_t total = __shfl_sync(0xffffffffu, before + mine, 31);
        // a group lies before the budget or behind it, but for one
        if (total & 0xffffu) {
          int32_t *h = holes + to.x + static_cast<int>(before & 0xffffu);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if ((m.x >> j) & 1u) *h++ = e + j;
          to.x += static_cast<int>(total & 0xffffu);
        }
        if (total >> 16) {
          int32_t *v = movers + to.y + static_cast<int>(before >> 16);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if ((m.y >> j) & 1u) *v++ = e + j;
          to.y += static_cast<int>(total >> 16);
        }
      }
    }
  }
  if (rank == 0 && tid == 0) p.plan[item] = moves;
  claim_pages(p, b, cut, (head * ranks + rank) * THREADS + tid, c.hkv * ranks * THREADS);
  if (CLUSTER) cl.sync();   // no CTA leaves while another reads its shared memory
}

// A warp takes kFlight moves (twice as many for head_dim 64, whose two rows fill half a warp) of a
// (sequence, KV head) at a time: as many lanes move a weight and an ordinal each, then the warp copies the
// rows, all loads before the first store.
constexpr int kFlight = 4;
constexpr int kMoveBlocks = 4;     // blocks that share an SM

template <int D>
__global__ void __launch_bounds__(kMoveWarps * 32, kMoveBlocks)
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
    int j0 = part * TAKE;
    // The lane's move, -1: none. Its entries are read two batches ahead and its pages one. (The pages of a
    // sequence that is not skipped were checked when they were claimed.)
    int hole = -1, mover = -1, doff = -1, soff = 0, dpage = 0, spage = 0;
    auto read_entries = [&](int j) {
      const bool in = lane < TAKE && j + lane < moves;
      hole = in ? __ldcg(holes + j + lane) : -1;
      mover = in ? __ldcg(movers + j + lane) : -1;
    };
    auto read_pages = [&]() {
      doff = -1;
      if (hole >= 0) {
        int slot;
        split_entry(c, hole, slot, doff);
        dpage = c.table[b * c.table_stride + slot];
        split_entry(c, mover, slot, soff);
        spage = c.table[b * c.table_stride + slot];
      }
    };
    read_entries(j0);
    read_pages();
    read_entries(j0 + parts * TAKE);
    while (j0 < moves) {
      int64_t to = -1, from = 0, tw = 0;
      float weight = 0.f;
      int32_t order = 0;
      const bool mine = doff >= 0;
      if (mine) {
        to = dpage * c.page_bytes + doff * c.entry_bytes;
        from = spage * c.page_bytes + soff * c.entry_bytes;
        const int64_t fw = track_at(c, spage, head, soff);
        tw = track_at(c, dpage, head, doff);
        weight = __ldcg(c.weight + fw);
        order = __ldcg(c.order + fw);
      }
      const int count = min(TAKE, moves - j0);
      uint4 row[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int64_t s = __shfl_sync(0xffffffffu, from, i * PER + which);
        if (i * PER + which < count) row[i] = ld_stream(base + s);
      }
      j0 += parts * TAKE;
      read_pages();
      read_entries(j0 + parts * TAKE);
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int64_t d = __shfl_sync(0xffffffffu, to, i * PER + which);
        if (i * PER + which < count) *reinterpret_cast<uint4 *>(base + d) = row[i];
      }
      if (mine) {
        c.weight[tw] = weight;
        c.order[tw] = order;
      }
    }
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, int num_sms, cudaStream_t stream) {
  const CacheView &c = p.c;
  const int items = c.batch * c.hkv;
  // One block where there are blocks enough or little to share, else up to eight that share the work of one,
  // as long as all of them find an SM and a share is more than 1024 entries. Long shares take the
  // largest blocks: two smaller ones would be put on one SM while others idle. But clusters of eight of them find
  // places on only four fifths of the SMs (a cluster stays within a group of SMs); more than those would
  // wait for a second round, 90 us against 86 for the smaller blocks (five sequences of up to 128K, 4 heads).
  int ranks = 1;
  while (ranks < kRanks &&
         (c.cap > ranks * kKeyRoom || (c.cap > ranks * 1024 && items * ranks * 2 <= num_sms)))
    ranks *= 2;
  const bool crowded = ranks == kRanks && items * ranks > num_sms * 4 / 5;
  const int threads = c.cap > ranks * 4096 && !crowded ? 1024 : 512;
  // keys per CTA, in whole groups of 128 for each warp
  const int64_t share = (static_cast<int64_t>(c.cap) + ranks - 1) / ranks;
  const int room = static_cast<int>(
      std::min<int64_t>(kKeyRoom, (share + threads * 4 - 1) / (threads * 4) * (threads * 4)));
  static std::atomic<uint64_t> allowed[4];
  const auto kern =
      ranks > 1 ? (threads == 1024 ? evict_select_kernel<1024, true> : evict_select_kernel<512, true>)
                : (threads == 1024 ? evict_select_kernel<1024, false> : evict_select_kernel<512, false>);
  cudaError_t e = allow_shared(kern, kKeyRoom * 4, &allowed[(ranks > 1) * 2 + threads / 1024]);
  if (e == cudaSuccess)
    e = launch_dependent(kern, dim3(static_cast<unsigned>(items) * ranks), threads, room * 4, ranks,
                         stream, p, room);
  if (e != cudaSuccess) return e;
  // Blocks of the move kernel: as many as its longest possible lists can use, up to two rounds of those that fit,
  // so that the hardware evens out items with many moves and with none. Whole passes over five ragged sequences of
  // up to 128K, and over eight of 32K: one round 83 and 113 us, two 81 and 114, five 81 and 118; eight moves in
  // flight and three blocks per SM 85 and 124.
  const int64_t most = std::max(1, std::min(p.budget, c.cap - p.budget));
  const int per_block = kMoveWarps * kFlight * (c.d == 128 ? 1 : 2);
  const int64_t blocks =
      std::min<int64_t>(num_sms * kMoveBlocks * 2, items * ((most + per_block - 1) / per_block));
  const dim3 grid(static_cast<unsigned>(blocks));
  const int parts = static_cast<int>(std::max<int64_t>(1, blocks * kMoveWarps / items));
  return c.d == 128 ? launch_dependent(evict_move_kernel<128>, grid, kMoveWarps * 32, 0, 1, stream,
                                       p, parts)
                    : launch_dependent(evict_move_kernel<64>, grid, kMoveWarps * 32, 0, 1, stream,
                                       p, parts);
}

}  // namespace rra
