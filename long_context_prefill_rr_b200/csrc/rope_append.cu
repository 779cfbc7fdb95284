// Rotary positions with several axes, from a view to a view and into the pages of a cache.
//
// Pair i of a head turns by phi = position[axis(i)] * f_i: (x, y) -> (x cos - y sin, y cos + x sin);
// the gradient turns back (sin negated). f_i is kept as F_i = f_i / (2 pi) * 2^64, an integer, so
// position * F_i mod 2^64 is the fraction of a turn with the full turns dropped, exact to 2^-64 *
// position; its top 32 bits, as a signed number, go to sincospif. An fp32 product
// position * f_i would be off by 2^-24 * position radians, 0.06 at a million.
//
// Memory bound: every row is read once and written once (twice where the prefill's copy and the
// cache both want it). A thread owns one unit of 16 dimensions (two 16-byte vectors: for halves one
// from each half, 8 pairs) of one token and walks over heads, so the eight sines and cosines are
// taken once for all of them.
#include "cache_device.cuh"

namespace rra {

struct RopeUnit {
  float c[8], s[8];
};

template <class T, bool ADJACENT>
__device__ __forceinline__ void turn(const RopeUnit &r, uint4 &a, uint4 &b) {
  uint32_t *pa = reinterpret_cast<uint32_t *>(&a);
  uint32_t *pb = reinterpret_cast<uint32_t *>(&b);
  if (ADJACENT) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = Elem<T>::unpack(pa[i]), y = Elem<T>::unpack(pb[i]);
      pa[i] = Elem<T>::pack(x.x * r.c[i] - x.y * r.s[i], x.y * r.c[i] + x.x * r.s[i]);
      pb[i] = Elem<T>::pack(y.x * r.c[4 + i] - y.y * r.s[4 + i],
                            y.y * r.c[4 + i] + y.x * r.s[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = Elem<T>::unpack(pa[i]), y = Elem<T>::unpack(pb[i]);
      const float c0 = r.c[2 * i], s0 = r.s[2 * i], c1 = r.c[2 * i + 1], s1 = r.s[2 * i + 1];
      pa[i] = Elem<T>::pack(x.x * c0 - y.x * s0, x.y * c1 - y.y * s1);
      pb[i] = Elem<T>::pack(y.x * c0 + x.x * s0, y.y * c1 + x.y * s1);
    }
  }
}

template <class T, bool ADJACENT, bool CACHED>
__global__ void __launch_bounds__(256)
    rope_kernel(const __grid_constant__ RopeParams p, const __grid_constant__ CacheView c) {
  grid_dependency_wait();
  grid_dependents_go();
  const int units = p.d / 16;
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t row = idx / units;
  const int u = static_cast<int>(idx - row * units);
  const int b = static_cast<int>(row / p.tokens);
  const int t = static_cast<int>(row - static_cast<int64_t>(b) * p.tokens);
  bool real = b < p.batch;
  if (real && p.new_len) real = t < p.new_len[b];
  int page = -1, off = 0, ordinal = 0;
  if (CACHED && real) {
    const int e = cache_len(c, b) + t;
    if (e < c.cap) {
      int slot;
      split_entry(c, e, slot, off);
      page = page_at(c, b, slot);
      if (c.order) ordinal = c.seen[b] + t;
    }
  }
  if (real) {
    const bool turned = u < p.rot / 16;
    const int a0 = (!ADJACENT && turned) ? u * 16 : u * 32;             // byte offsets in a row
    const int b0 = (!ADJACENT && turned) ? p.rot + u * 16 : u * 32 + 16;
    RopeUnit r;
    if (turned) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int pair = u * 8 + i;
        const int64_t pos = p.pos.data[p.axis[pair] * p.pos.axis + b * p.pos.batch +
                                       t * p.pos.token];
        const uint64_t frac = static_cast<uint64_t>(pos) * p.turn[pair];
        const float half_turns = static_cast<float>(static_cast<int32_t>(frac >> 32)) * 0x1p-31f;
        sincospif(half_turns, &r.s[i], &r.c[i]);
        if (p.inverse) r.s[i] = -r.s[i];
      }
    }
    const int h0 = blockIdx.y * p.heads_per_thread;
    const int h1 = min(h0 + p.heads_per_thread, p.heads);
    const int nq = p.q.data ? p.hq : 0;
    const int nk = p.k.data ? p.hkv : 0;
#pragma unroll 4
    for (int h = h0; h < h1; ++h) {
      const bool is_q = h < nq, is_v = h >= nq + nk;
      const rra_view &src = is_q ? p.q : (is_v ? p.v : p.k);
      const rra_view &dst = is_q ? p.qo : (is_v ? p.vo : p.ko);
      const int hh = is_q ? h : (is_v ? h - nq - nk : h - nq);
      const uint8_t *in = static_cast<const uint8_t *>(src.data) + b * src.batch +
                          hh * src.head + t * src.token;
      uint4 x = *reinterpret_cast<const uint4 *>(in + a0);
      uint4 y = *reinterpret_cast<const uint4 *>(in + b0);
      if (turned && !is_v) rra::turn<T, ADJACENT>(r, x, y);
      if (dst.data) {
        uint8_t *o = static_cast<uint8_t *>(dst.data) + b * dst.batch + hh * dst.head +
                     t * dst.token;
        *reinterpret_cast<uint4 *>(o + a0) = x;
        *reinterpret_cast<uint4 *>(o + b0) = y;
      }
      if (CACHED && !is_q && page >= 0) {
        uint8_t *o = (is_v ? c.v : c.k) + page * c.page_bytes + hh * c.head_bytes +
                     off * c.entry_bytes;
        *reinterpret_cast<uint4 *>(o + a0) = x;
        *reinterpret_cast<uint4 *>(o + b0) = y;
        if (c.order && is_v && u == 0) {
          const int64_t at = track_at(c, page, hh, off);
          c.weight[at] = 0.f;
          c.order[at] = ordinal;
        }
      }
    }
  }
  if (!CACHED) return;
  // lengths outside the table, reported once per sequence
  if (blockIdx.y == 0 && real && t == 0 && u == 0) {
    const int n = c.len[b];
    const int add = p.new_len ? min(p.new_len[b], p.tokens) : p.tokens;
    if (n < 0 || static_cast<int64_t>(n) + add > c.cap) raise(c.status, kErrBadLength);
  }
  if (!p.advance) return;
  // The last block to have read len and seen moves them on and resets the count.
  __shared__ uint32_t s_last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0)
    s_last = atomicAdd(p.done, 1u) == gridDim.x * gridDim.y - 1u ? 1u : 0u;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  for (int i = threadIdx.x; i < p.batch; i += 256) {
    int add = p.new_len ? min(p.new_len[i], p.tokens) : p.tokens;
    if (add < 0) add = 0;
    const int64_t n = static_cast<int64_t>(cache_len(c, i)) + add;
    c.len[i] = n > c.cap ? c.cap : static_cast<int>(n);
    if (c.seen) c.seen[i] += add;
  }
  if (threadIdx.x == 0) *p.done = 0;
}

template <class T>
static cudaError_t launch_rope_t(const RopeParams &p, const CacheView *cache, int pairing,
                                 dim3 grid, cudaStream_t stream) {
  const bool adjacent = pairing == RRA_PAIRS_ADJACENT;
  const auto kern = cache ? (adjacent ? rope_kernel<T, true, true> : rope_kernel<T, false, true>)
                          : (adjacent ? rope_kernel<T, true, false> : rope_kernel<T, false, false>);
  return launch_dependent(kern, grid, 256, 0, 1, stream, p, cache ? *cache : CacheView{});
}

cudaError_t launch_rope(const RopeParams &in, const CacheView *cache, int dtype, int pairing,
                        int num_sms, cudaStream_t stream) {
  RopeParams p = in;
  const int64_t threads = static_cast<int64_t>(p.batch) * p.tokens * (p.d / 16);
  const int64_t blocks = (threads + 255) / 256;
  // heads are shared out over blockIdx.y until every SM has its fill of threads
  const int64_t want = (static_cast<int64_t>(num_sms) * 8 + blocks - 1) / blocks;
  const int split = static_cast<int>(want < 1 ? 1 : (want > p.heads ? p.heads : want));
  p.heads_per_thread = (p.heads + split - 1) / split;
  const dim3 grid(static_cast<unsigned>(blocks),
                  static_cast<unsigned>((p.heads + p.heads_per_thread - 1) / p.heads_per_thread));
  if (dtype == RRA_BF16) return launch_rope_t<__nv_bfloat16>(p, cache, pairing, grid, stream);
  return launch_rope_t<__half>(p, cache, pairing, grid, stream);
}

}  // namespace rra
