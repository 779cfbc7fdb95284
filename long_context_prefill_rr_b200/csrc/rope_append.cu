// Rotary positions with several axes, from a view to a view and into the pages of a cache.
//
// Pair i of a head turns by phi = position[axis(i)] * f_i: (x, y) -> (x cos - y sin, y cos + x sin);
// the gradient turns back (sin negated). f_i is kept as F_i = f_i / (2 pi) * 2^64, an integer, so
// position * F_i mod 2^64 is the fraction of a turn with the full turns dropped, exact to 2^-64 *
// position. (An fp32 product position * f_i would be off by 2^-24 * position radians, 0.06 at a million.)
// Its top two bits, rounded, are the quadrant; sine and cosine of the rest, at most an eighth of a turn,
// come from their Taylor series.
//
// Memory bound: every row is read once and written once (twice where the prefill's copy and the
// cache both want it). A thread owns one unit of 16 dimensions (two 16-byte vectors: for halves one
// from each half, 8 pairs) of one token and walks over heads, so the eight sines and cosines are
// taken once for all of them. Measured (65536 tokens, 28 + 4 heads of 128, bf16, 1.07 GB): 175 us, 94% of
// the copy rate; with four blocks per SM 187, with two heads in flight per thread and spills 181, with
// sincospif in place of the series and four heads in flight 195. 7500 tokens, a quarter of them padding,
// into pages (104 MB): 25 us against 16 for the bytes; it is the reads of lengths, pages and positions in
// front of the first row, and blocks of padding that leave their place idle, that cost there.
#include "cache_device.cuh"

namespace rra {

constexpr int kBlocks = 5;   // blocks that share an SM

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

// Top 32 bits of position * turn mod 2^64.
__device__ __forceinline__ uint32_t fraction(int32_t position, uint64_t turn) {
  const uint32_t lo = static_cast<uint32_t>(turn), hi = static_cast<uint32_t>(turn >> 32);
  const uint32_t x = static_cast<uint32_t>(position);
  return __umulhi(x, lo) + x * hi - (position < 0 ? lo : 0u);
}

// Cosine and sine of f / 2^32 turns. With |x| <= pi / 4 the series are cut below 2^-25 (x^11 / 11!, x^10 / 10!).
__device__ __forceinline__ void cos_sin(uint32_t f, float &c, float &s) {
  const uint32_t quadrant = (f + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(f - (quadrant << 30))) * 1.4629180792671596e-9f;
  const float xx = x * x;
  float sine = fmaf(xx, 1.f / 362880.f, -1.f / 5040.f);
  sine = fmaf(xx, sine, 1.f / 120.f);
  sine = fmaf(xx, sine, -1.f / 6.f);
  sine = fmaf(x * xx, sine, x);
  float cosine = fmaf(xx, 1.f / 40320.f, -1.f / 720.f);
  cosine = fmaf(xx, cosine, 1.f / 24.f);
  cosine = fmaf(xx, cosine, -0.5f);
  cosine = fmaf(xx, cosine, 1.f);
  // a quarter turn takes (cos, sin) to (-sin, cos)
  const float a = (quadrant & 1u) ? sine : cosine, b = (quadrant & 1u) ? cosine : sine;
  c = __uint_as_float(__float_as_uint(a) ^ (((quadrant + 1u) & 2u) << 30));
  s = __uint_as_float(__float_as_uint(b) ^ ((quadrant & 2u) << 30));
}

// Heads h0 .. h1 - 1 of one tensor: from `in` to `out` and to `page`, where those are given (byte offsets
// of the two vectors: a and b).
template <class T, bool ADJACENT, bool TURN>
__device__ __forceinline__ void heads(const RopeUnit &r, int h0, int h1, int a, int b,
                                      const uint8_t *in, int64_t in_head, uint8_t *out,
                                      int64_t out_head, uint8_t *page, int64_t page_head) {
  in += h0 * in_head;
  out += h0 * out_head;
  page += h0 * page_head;
  const bool to_out = out_head >= 0, to_page = page_head >= 0;
#pragma unroll 1
  for (int h = h0; h < h1; ++h, in += in_head, out += out_head, page += page_head) {
    uint4 x = *reinterpret_cast<const uint4 *>(in + a);
    uint4 y = *reinterpret_cast<const uint4 *>(in + b);
    if (TURN) rra::turn<T, ADJACENT>(r, x, y);
    if (to_out) {
      *reinterpret_cast<uint4 *>(out + a) = x;
      *reinterpret_cast<uint4 *>(out + b) = y;
    }
    if (to_page) {
      *reinterpret_cast<uint4 *>(page + a) = x;
      *reinterpret_cast<uint4 *>(page + b) = y;
    }
  }
}

template <class T, bool ADJACENT, bool CACHED>
__global__ void __launch_bounds__(256, kBlocks)
    rope_kernel(const __grid_constant__ RopeParams p, const __grid_constant__ CacheView c) {
  grid_dependency_wait();
  grid_dependents_go();
  const int units = p.d / 16;
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t row = idx / units;
  const int u = static_cast<int>(idx - row * units);
  const int b = static_cast<int>(row / p.tokens);
  const int t = static_cast<int>(row - static_cast<int64_t>(b) * p.tokens);
  // everything that the token's rows do not depend on is asked for at once
  const bool there = b < p.batch;
  const bool turned = u < p.rot / 16;
  int32_t pos[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  int first = 0, new_tokens = p.tokens, ordinal = 0;
  if (there) {
    if (p.new_len) new_tokens = p.new_len[b];
    if (CACHED) first = c.len[b];
    if (CACHED && c.order) ordinal = c.seen[b] + t;
    if (turned) {
      const int32_t *at = p.pos.data + b * p.pos.batch + t * p.pos.token;
#pragma unroll
      for (int i = 0; i < 8; ++i) pos[i] = at[p.axis[u * 8 + i] * p.pos.axis];
    }
  }
  const bool real = there && t < new_tokens;
  if (real) {
    int page = -1, off = 0;
    if (CACHED) {
      const int e = max(0, min(first, c.cap)) + t;
      int slot;
      split_entry(c, e, slot, off);
      if (e < c.cap) page = c.table[b * c.table_stride + slot];
    }
    const int va = (!ADJACENT && turned) ? u * 16 : u * 32;             // byte offsets in a row
    const int vb = (!ADJACENT && turned) ? p.rot + u * 16 : u * 32 + 16;
    RopeUnit r;
    if (turned) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cos_sin(fraction(pos[i], p.turn[u * 8 + i]), r.c[i], r.s[i]);
        if (p.inverse) r.s[i] = -r.s[i];
      }
    }
    if (CACHED && static_cast<unsigned>(page) >= static_cast<unsigned>(c.num_pages)) {
      if (max(0, min(first, c.cap)) + t < c.cap) raise(c.status, kErrBadPage);
      page = -1;
    }
    // the heads of q, then of k, then of v are shared out over blockIdx.y
    const int h0 = blockIdx.y * p.heads_per_thread, h1 = h0 + p.heads_per_thread;
    auto part = [&](const rra_view &src, const rra_view &dst, int first, int count, uint8_t *cache,
                    bool turn_it) {
      if (!src.data) return;
      const int lo = max(h0 - first, 0), hi = min(h1 - first, count);
      if (lo >= hi) return;
      const uint8_t *in = static_cast<const uint8_t *>(src.data) + b * src.batch + t * src.token;
      uint8_t *out = static_cast<uint8_t *>(dst.data) + b * dst.batch + t * dst.token;
      const bool paged = CACHED && cache != nullptr && page >= 0;
      uint8_t *to = paged ? cache + page * c.page_bytes + off * c.entry_bytes : nullptr;
      const int64_t out_head = dst.data ? dst.head : -1, to_head = paged ? c.head_bytes : -1;
      if (turn_it)
        heads<T, ADJACENT, true>(r, lo, hi, va, vb, in, src.head, out, out_head, to, to_head);
      else
        heads<T, ADJACENT, false>(r, lo, hi, va, vb, in, src.head, out, out_head, to, to_head);
    };
    const int nq = p.q.data ? p.hq : 0, nk = p.k.data ? p.hkv : 0;
    part(p.q, p.qo, 0, nq, nullptr, turned);
    part(p.k, p.ko, nq, nk, c.k, turned);
    part(p.v, p.vo, nq + nk, p.v.data ? p.hkv : 0, c.v, false);
    if (CACHED && c.order && page >= 0 && u == 0)
      for (int h = max(h0 - nq - nk, 0); h < min(h1 - nq - nk, p.hkv); ++h) {
        const int64_t at = track_at(c, page, h, off);
        c.weight[at] = 0.f;
        c.order[at] = ordinal;
      }
  }
  if (!CACHED) return;
  // lengths outside the table, reported once per sequence, whether it has new tokens or not
  if (blockIdx.y == 0 && there && t == 0 && u == 0 &&
      (first < 0 || static_cast<int64_t>(first) + max(min(new_tokens, p.tokens), 0) > c.cap))
    raise(c.status, kErrBadLength);
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
  // Heads are shared out over blockIdx.y as long as all blocks find a place at once: a second,
  // partly filled round costs more than longer blocks.
  const int64_t fit = static_cast<int64_t>(num_sms) * kBlocks / blocks;
  const int split = static_cast<int>(fit < 1 ? 1 : (fit > p.heads ? p.heads : fit));
  p.heads_per_thread = (p.heads + split - 1) / split;
  const dim3 grid(static_cast<unsigned>(blocks),
                  static_cast<unsigned>((p.heads + p.heads_per_thread - 1) / p.heads_per_thread));
  if (dtype == RRA_BF16) return launch_rope_t<__nv_bfloat16>(p, cache, pairing, grid, stream);
  return launch_rope_t<__half>(p, cache, pairing, grid, stream);
}

}  // namespace rra
