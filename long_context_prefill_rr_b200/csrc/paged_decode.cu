// Attention of one new token per sequence over a paged key-value cache, split over the entries
// and joined: o = sum_e softmax(scale q.k_e) v_e with the running maximum and sum of an online
// softmax, one pass over K and V.
//
// Memory bound: 4 d bytes per entry and KV head against 4 d flop per query head, so K and V have to
// be read once, at HBM speed, and everything else stays in registers. (More than 16 query heads to a KV
// head read them once per 16.)
//
// Work. The entries of all (sequence, KV head, head tile) items are laid end to end in units of 64
// and cut into equal runs, one per CTA, whatever the lengths are (they are read on the device, so a
// captured graph follows them). A run touches a few items; its share of one item is a piece. An
// item of one piece is finished where it is computed; otherwise each piece leaves its unnormalised
// output, maximum and sum in the workspace and the CTA that finishes last joins them in order of
// the entries, so equal calls give equal bits.
//
// Inner loop. A warp takes 16 entries at a time through a ring of its own, filled by cp.async, and
// shares nothing with the other warps until its piece ends: no block barrier in the loop. The MMA
// fragments come out of the ring by 16-byte reads: the contraction index of q.k may be permuted freely
// as long as q is permuted alike, so a thread takes 16 bytes of a key row as the B fragments of two
// k-steps; the columns of p.v may be permuted as well, so a thread takes 16 bytes of each of four
// value rows and pairs up the rows' elements. The 8 query heads fill rows 0-7 of the 16-row MMA
// tile. Rows 8-15 of the p.v product hold the low parts of the same weights (p = hi + lo, both 16-bit),
// so the weights keep twice the bits of the element type at no cost: 2^-17 of themselves in bf16; in fp16
// 2^-22 of themselves or 2^-40 of the largest weight, whichever is more, because they are raised by 2^15
// first (unraised, entries 17.3 nats below an attention sink were 0 here and counted in the denominator).
// With more than 8 heads to a KV head rows 8-15 hold 8 more of them, and the low parts take a second product.
//
// Measured on the way (128K entries, 32 / 8 heads of 128, 537 MB; the copy rate gives 82 us): fragments
// loaded straight into registers 107 us (64-byte requests, 56% of the load pipe's wavefronts); the
// same loads through cp.async into places private to each thread 136; a ring of rows filled by one bulk
// copy per row 106 (a warp issues its 32 copies one by one); this ring, whose copies cover whole rows,
// 92, and 90 with the rows marked to leave L2 first. Two stages and two CTAs per SM (three for head_dim
// 64) keep 128 KB in flight; more bytes in flight are slower (three stages 97, three CTAs 101;
// head_dim 64 with four stages and three CTAs 106 against 88). 16 heads to a KV head take 66 us where
// two passes of 8 took 106 (4 x 40000 entries, 328 MB).
// A call of 1000 entries takes 8 us, 2 of them the join of 16 pieces; reading eight pieces at a time
// there made it slower (10: the longer code has to be fetched).
#include <float.h>
#include <math.h>

#include "cache_device.cuh"

namespace rra {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

// A warp's ring: kStages stages of 16 key rows and 16 value rows. Rows lie D * 2 + 32 bytes apart, 8
// banks past a multiple of 32, which with the order of the entries below keeps every 16-byte read
// of a warp free of bank conflicts.
constexpr int kStages = 2;
template <int D>
constexpr uint32_t kPitch = D * 2 + 32;
template <int D>
constexpr uint32_t kStageBytes = 32 * kPitch<D>;
template <int D>
constexpr size_t kRingBytes = static_cast<size_t>(kWarps) * kStages * kStageBytes<D>;

// Keys and values leave L2 first, before the logits and pieces that are read again. That holds with more than 16
// query heads to a KV head too, which read them once per head tile, from CTAs that do not run side by
// side: 4 x 128K entries, 32 heads over one, take 115 us so, and 127 with rows that leave L2 in turn or last.
__device__ __forceinline__ uint64_t once_policy() {
  uint64_t policy;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool valid, uint64_t policy) {
  const int n = valid ? 16 : 0;   // 0: nothing is read, the place is filled with zeros
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst),
               "l"(src), "r"(n), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// What a mean is its weighted sum times: a sum of 0 (no weight at all) leaves 0, and NaN stays. (The hardware's
// quotient, off by 2^-22 at most: the sums are well within its range. The exact one cost 0.3 us of a call of 7.)
__device__ __forceinline__ float reciprocal_of_sum(float sum) {
  return sum == 0.f ? 0.f : __fdividef(1.f, sum);
}
// A factor that joins means, 2^-126 at least (nothing beside the largest of them): an infinite or NaN mean
// stays what it is.
__device__ __forceinline__ float share_of(float f) { return fmaxf(f, FLT_MIN); }

// Entry (of 8) behind column 2 t + e of an MMA tile. Columns may stand for the entries in any order, as
// long as logits, weights and value rows agree; this one puts the rows that a read touches together
// (columns 2 t, 2 t + 1 of the keys; the four values of t for the value rows) into different banks.
__device__ __forceinline__ int entry_of(int t, int e) { return e ? 4 + ((t + 2) & 3) : t; }

// Where a CTA's run of units starts.
struct Cursor {
  int b;         // sequence
  int start;     // first unit of the sequence
  int units;     // units of one of its items
  int len;
};

__device__ __forceinline__ int units_of(int len) { return (len + kDecodeUnit - 1) / kDecodeUnit; }

// Units of all sequences, and the sequence that holds unit `per * cta`. All threads of the block
// call it; items: items per sequence. Returns the number of units per CTA.
__device__ int locate(const CacheView &c, int items, int grid, int cta, int *s_scan, Cursor *cur,
                      int *total_out) {
  const int tid = threadIdx.x, nt = blockDim.x;
  const int lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  if (c.batch <= 32) {
    // a lane per sequence, and every warp for itself
    const int len = lane < c.batch ? cache_len(c, lane) : 0;
    const int mine = units_of(len) * items;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const int total = __shfl_sync(0xffffffffu, incl, 31);
    const int per = max(1, (total + grid - 1) / grid);
    const uint32_t past = __ballot_sync(0xffffffffu, incl > per * cta);
    const int b = past ? __ffs(past) - 1 : 0;
    cur->b = b;
    cur->start = __shfl_sync(0xffffffffu, incl - mine, b);
    cur->len = __shfl_sync(0xffffffffu, len, b);
    cur->units = units_of(cur->len);
    *total_out = total;
    return per;
  }
  const int chunk = (c.batch + nt - 1) / nt;
  const int b0 = min(tid * chunk, c.batch), b1 = min(b0 + chunk, c.batch);
  int sum = 0;
  for (int b = b0; b < b1; ++b) sum += units_of(cache_len(c, b)) * items;
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
  for (int w = 0; w < nw; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  const int per = max(1, (total + grid - 1) / grid);
  const int first = per * cta;
  int excl = before + incl - sum;
  if (first >= excl && first < excl + sum) {
    for (int b = b0; b < b1; ++b) {
      const int len = cache_len(c, b);
      const int n = units_of(len) * items;
      if (first < excl + n) {
        s_scan[16] = b;
        s_scan[17] = excl;
        s_scan[18] = len;
        break;
      }
      excl += n;
    }
  }
  __syncthreads();
  if (first < total) {
    cur->b = s_scan[16];
    cur->start = s_scan[17];
    cur->len = s_scan[18];
    cur->units = units_of(cur->len);
  }
  *total_out = total;
  return per;
}

// The next sequence with entries.
__device__ __forceinline__ void next_sequence(const CacheView &c, int items, Cursor *cur) {
  cur->start += cur->units * items;
  do {
    ++cur->b;
    cur->len = cache_len(c, cur->b);
  } while (cur->len == 0 && cur->b + 1 < c.batch);
  cur->units = units_of(cur->len);
}

// One query head's mean of a warp's entries of a piece, again: where values that are infinite or NaN meet
// weights of 0 (logits of -inf) or the low parts of others, the matrix product has 0 * inf; and sums of bf16's
// largest values pass fp32's range. Here an entry without a weight is left out, the other values that
// are not finite are noted for each dimension apart from the sum, and the sum is kept 2^-31 as large (a
// sequence has at most 2^30 entries). A lane takes D / 32 dimensions of eight entries at a time, for the heads and warps that
// it happens to: 128K entries, 32 / 8 heads of 128, take 1.1 ms with an infinity under every KV head and 1.6 with
// nothing but NaN, against 90 us. Code of its own, because the same within the loop below cost every call
// 0.4 us, and 2 of 93 (32 sequences of up to 8K).
template <class T, int D>
__device__ __noinline__ void add_up_again(const DecodeParams &p, int b, int kv_head, int head, int e0,
                                          int key1, float *out, float *max_out, float *sum_out) {
  constexpr int PER = D / 32, BATCH = 8;   // BATCH: entries in flight
  const CacheView &c = p.c;
  const int lane = threadIdx.x & 31;
  auto read = [&](int64_t at, const uint8_t *base, float (&x)[PER]) {
#pragma unroll
    for (int i = 0; i < PER; i += 2) {
      const int byte = (lane * PER + i) * 2;
      const float2 y = Elem<T>::unpack(at < 0 ? 0u : *reinterpret_cast<const uint32_t *>(base + at + byte));
      x[i] = y.x, x[i + 1] = y.y;
    }
  };
  float q[PER], acc[PER] = {}, top = -INFINITY, sum = 0.f;
  read(b * p.q_batch + head * p.q_head, p.q, q);
  uint32_t plus = 0, minus = 0;        // dimensions with a value of +inf or NaN, and of -inf or NaN
#pragma unroll 1
  for (int kb = e0; kb < key1; kb += kDecodeUnit) {
    int64_t mine = -1;
    if (kb + (lane & 15) < key1) {
      int slot, off;
      split_entry(c, kb + (lane & 15), slot, off);
      const int pg = page_at(c, b, slot);
      if (pg >= 0) mine = pg * c.page_bytes + off * c.entry_bytes;
    }
#pragma unroll 1
    for (int j = 0; j < 16; j += BATCH) {
      float x[BATCH], v[BATCH][PER];
#pragma unroll
      for (int n = 0; n < BATCH; ++n) {
        const int64_t at = __shfl_sync(0xffffffffu, mine, j + n);
        float k[PER];
        read(at, c.k + kv_head * c.head_bytes, k);
        read(at, c.v + kv_head * c.head_bytes, v[n]);
        x[n] = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) x[n] = fmaf(q[i], k[i], x[n]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < BATCH; ++n) x[n] += __shfl_xor_sync(0xffffffffu, x[n], o);
#pragma unroll
      for (int n = 0; n < BATCH; ++n) {
        x[n] *= p.scale_log2;          // the same in all lanes
        if (x[n] == -INFINITY || __shfl_sync(0xffffffffu, mine, j + n) < 0) continue;
        const float top_new = fmaxf(top, x[n]), alpha = exp2f(top - top_new), w = exp2f(x[n] - top_new);
        top = top_new;
        sum = sum * alpha + w;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const float y = v[n][i];
          const bool finite = fabsf(y) < INFINITY;
          acc[i] = acc[i] * alpha + (finite ? w * 0x1p-31f * y : 0.f);
          if (!finite && !(y < 0.f)) plus |= 1u << i;
          if (!finite && !(y > 0.f)) minus |= 1u << i;
        }
      }
    }
  }
  const float inv = reciprocal_of_sum(sum);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    acc[i] *= inv * 0x1p31f;
    if ((plus >> i) & 1u) acc[i] += INFINITY;
    if ((minus >> i) & 1u) acc[i] -= INFINITY;
    out[lane * PER + i] = acc[i];
  }
  if (lane == 0) *max_out = top, *sum_out = sum;
}

// TILE: query heads of a KV head that a warp carries, 8 or 16.
template <class T, int D, int TILE>
__global__ void __launch_bounds__(kThreads, decode_ctas(D))
    paged_decode_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int NJ = D / 32;        // 16-byte vectors of a key row per thread
  constexpr int NH = D / 64;        // 64-dimension halves of a value row
  constexpr int HT = TILE / 8;      // heads of a thread: r and r + 8
  constexpr int S = kStages;
  constexpr uint32_t PITCH = kPitch<D>, STAGE = kStageBytes<D>;
  constexpr int ROW = D + 4;        // padded row of the merge buffer
  // Weights, their sums and the outputs are 2^RAISE times too large in the registers, where they are divided
  // by one another.
  constexpr int RAISE = Elem<T>::kRaise;
  static_assert(S <= 4 && S * STAGE >= TILE * ROW * 4, "exist masks, merge buffer");
  extern __shared__ __align__(128) uint8_t s_ring[];
  __shared__ int s_scan[20];
  __shared__ float s_m[kWarps][TILE], s_l[kWarps][TILE];

  const CacheView &c = p.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, t = lane & 3;
  const int items = c.hkv * p.head_tiles;
  const int cta = blockIdx.x;
  const uint32_t ring = smem_u32(s_ring) + warp * S * STAGE;
  // the merge buffer of a warp lies over its ring, which is idle then
  auto s_o = [&](int w) { return reinterpret_cast<float *>(s_ring + w * S * STAGE); };

  const uint64_t policy = once_policy();
  grid_dependency_wait();
  grid_dependents_go();
  // sequences without entries, and lengths outside the table
  for (int b = cta; b < c.batch; b += gridDim.x) {
    const int raw = c.len[b];
    if ((raw < 0 || raw > c.cap) && threadIdx.x == 0) raise(c.status, kErrBadLength);
    if (raw > 0) continue;
    for (int i = threadIdx.x; i < c.hq * (D / 8); i += kThreads) {
      const int h = i / (D / 8), v = i - h * (D / 8);
      *reinterpret_cast<uint4 *>(p.out + b * p.o_batch + h * p.o_head + v * 16) =
          make_uint4(0, 0, 0, 0);
      if (v == 0) {
        if (p.lse) p.lse[b * c.hq + h] = -INFINITY;
        p.lse2[b * c.hq + h] = -INFINITY;
      }
    }
  }

  Cursor cur;
  int total;
  const int per = locate(c, items, gridDim.x, cta, s_scan, &cur, &total);
  int pos = per * cta;
  const int end = min(pos + per, total);

  while (pos < end) {
    const int in_seq = pos - cur.start;
    const int m = in_seq / cur.units;                    // item of the sequence
    const int unit0 = in_seq - m * cur.units;
    const int n = min(cur.units - unit0, end - pos);
    const int head = m / p.head_tiles;                   // KV head
    const int tile = m - head * p.head_tiles;
    const int rows = min(TILE, c.g - tile * TILE);
    const int h0 = head * c.g + tile * TILE;     // first query head
    const int b = cur.b;
    const int key1 = min(cur.len, (unit0 + n) * kDecodeUnit);

    uint4 qf[HT][NJ];
#pragma unroll
    for (int h = 0; h < HT; ++h)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        qf[h][j] = r + 8 * h < rows
                       ? *reinterpret_cast<const uint4 *>(
                             p.q + b * p.q_batch + (h0 + r + 8 * h) * p.q_head + (4 * j + t) * 16)
                       : make_uint4(0, 0, 0, 0);

    float acc[NH * 8][4];
#pragma unroll
    for (int i = 0; i < NH * 8; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i][q] = 0.f;
    float m_run[HT], l_run[HT];
#pragma unroll
    for (int h = 0; h < HT; ++h) m_run[h] = -INFINITY, l_run[h] = 0.f;

    // byte offset of entry kb + (lane & 15), or -1 if there is none
    auto place = [&](int kb) -> int64_t {
      const int e = kb + (lane & 15);
      if (e >= key1) return -1;
      int slot, off;
      split_entry(c, e, slot, off);
      const int pg = page_at(c, b, slot);
      return pg < 0 ? -1 : pg * c.page_bytes + off * c.entry_bytes;
    };
    // Starts the copies of 16 entries into a stage: LANES lanes to a row, so that a warp's copy reads whole
    // rows. Entries that do not exist become rows of zeros. Returns which do.
    constexpr int LANES = D / 8, ROWS = 32 / LANES;
    const uint8_t *kh = c.k + head * c.head_bytes + (lane % LANES) * 16;
    const uint8_t *vh = c.v + head * c.head_bytes + (lane % LANES) * 16;
    auto fetch = [&](int st, int64_t at) -> uint32_t {
      const uint32_t dst = ring + st * STAGE + (lane / LANES) * PITCH + (lane % LANES) * 16;
#pragma unroll
      for (int i = 0; i < 16 / ROWS; ++i) {
        const int64_t o = __shfl_sync(0xffffffffu, at, i * ROWS + lane / LANES);
        const int64_t from = o >= 0 ? o : 0;
        copy16(dst + i * ROWS * PITCH, kh + from, o >= 0, policy);
        copy16(dst + (16 + i * ROWS) * PITCH, vh + from, o >= 0, policy);
      }
      return __ballot_sync(0xffffffffu, at >= 0) & 0xffffu;
    };

    // Step i is fetched into stage i mod S and used S - 1 steps later.
    int kb = unit0 * kDecodeUnit + (warp - (S - 1) * kWarps) * 16;   // entries that are used
    int ahead = unit0 * kDecodeUnit + warp * 16;                     // entries that are fetched
    uint64_t exist = 0;                // 16 bits per stage in flight, the newest on top
    int64_t at = place(ahead);
    for (int in = 0, st = 1 % S; kb < key1; kb += kDecodeUnit) {
      exist >>= 16;
      if (ahead < key1) {
        exist |= static_cast<uint64_t>(fetch(in, at)) << (16 * (S - 1));
        ahead += kDecodeUnit;
        at = place(ahead);
      }
      copy_commit();
      in = in + 1 == S ? 0 : in + 1;
      const int now = st;
      st = st + 1 == S ? 0 : st + 1;
      if (kb < unit0 * kDecodeUnit) continue;
      copy_wait<S - 1>();
      __syncwarp();                    // the other lanes' copies of the stage have landed too
      const uint32_t kst = ring + now * STAGE + t * 16;
      const uint32_t vst = ring + now * STAGE + 16 * PITCH + r * 16;
      // logits of heads r and r + 8 for columns 2t, 2t + 1 of the first MMA tile and of the second
      float s[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const uint4 kf = lds16(kst + (8 * i + entry_of(r >> 1, r & 1)) * PITCH + j * 64);
          const uint4 q1 = HT == 2 ? qf[HT - 1][j] : make_uint4(0, 0, 0, 0);
          Elem<T>::mma(s[i], qf[0][j].x, q1.x, qf[0][j].y, q1.y, kf.x, kf.y);
          Elem<T>::mma(s[i], qf[0][j].z, q1.z, qf[0][j].w, q1.w, kf.z, kf.w);
        }
      }
      float x[HT][4], mx[HT];
      bool grows = false;
#pragma unroll
      for (int h = 0; h < HT; ++h) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = entry_of(t, i & 1) + (i >> 1) * 8;
          x[h][i] = (exist >> e) & 1u ? s[i >> 1][2 * h + (i & 1)] * p.scale_log2 : -INFINITY;
          if (p.logits && r + 8 * h < rows && kb + e < key1)
            p.logits[(static_cast<int64_t>(b) * c.hq + h0 + r + 8 * h) * p.cap64 + kb + e] = x[h][i];
        }
        mx[h] = fmaxf(fmaxf(x[h][0], x[h][1]), fmaxf(x[h][2], x[h][3]));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
        grows = grows || mx[h] > m_run[h];
      }
      if (__any_sync(0xffffffffu, grows)) {
        float alpha[HT];
#pragma unroll
        for (int h = 0; h < HT; ++h) {
          const float m_new = fmaxf(m_run[h], mx[h]);
          // a row that has met no logit yet stays at -inf with sums of zero
          alpha[h] = m_new == -INFINITY ? 1.f : exp2f(m_run[h] - m_new);
          m_run[h] = m_new;
          l_run[h] *= alpha[h];
        }
#pragma unroll
        for (int i = 0; i < NH * 8; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[i][q] *= alpha[q / 2 * (HT - 1)];
      }
      uint32_t hi[HT][2], lo[HT][2];
#pragma unroll
      for (int h = 0; h < HT; ++h) {
        const float base = m_run[h] == -INFINITY ? 0.f : m_run[h];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // (the difference is rounded before the factor is added: it is never above 0)
          float y0 = x[h][2 * i] - base, y1 = x[h][2 * i + 1] - base;
          if (RAISE) y0 += RAISE, y1 += RAISE;
          const float w0 = fast_exp2(y0), w1 = fast_exp2(y1);
          l_run[h] += w0 + w1;
          hi[h][i] = Elem<T>::pack(w0, w1);
          const float2 f = Elem<T>::unpack(hi[h][i]);
          lo[h][i] = Elem<T>::pack(w0 - f.x, w1 - f.y);
        }
      }
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        uint4 vf[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          vf[i] = lds16(vst + (entry_of(t, i & 1) + (i >> 1) * 8) * PITCH + h * 128);
        const uint32_t *v0 = reinterpret_cast<const uint32_t *>(&vf[0]);
        const uint32_t *v1 = reinterpret_cast<const uint32_t *>(&vf[1]);
        const uint32_t *v2 = reinterpret_cast<const uint32_t *>(&vf[2]);
        const uint32_t *v3 = reinterpret_cast<const uint32_t *>(&vf[3]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t pick = (e & 1) ? 0x7632u : 0x5410u;
          const uint32_t b0 = __byte_perm(v0[e >> 1], v1[e >> 1], pick);
          const uint32_t b1 = __byte_perm(v2[e >> 1], v3[e >> 1], pick);
          if (HT == 1) {
            Elem<T>::mma(acc[h * 8 + e], hi[0][0], lo[0][0], hi[0][1], lo[0][1], b0, b1);
          } else {
            Elem<T>::mma(acc[h * 8 + e], hi[0][0], hi[HT - 1][0], hi[0][1], hi[HT - 1][1], b0, b1);
            Elem<T>::mma(acc[h * 8 + e], lo[0][0], lo[HT - 1][0], lo[0][1], lo[HT - 1][1], b0, b1);
          }
        }
      }
      __syncwarp();                    // every lane's reads fed the MMAs above: the stage is free
    }
    copy_wait<0>();
    __syncwarp();

    // ---- the warps' results meet in shared memory
    float inv_run[HT], not_finite[HT] = {};
#pragma unroll
    for (int h = 0; h < HT; ++h) {
      l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], 1);
      l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], 2);
      if (t == 0) {
        s_m[warp][r + 8 * h] = m_run[h];
        s_l[warp][r + 8 * h] = l_run[h] / static_cast<float>(1 << RAISE);
      }
      inv_run[h] = reciprocal_of_sum(l_run[h]);
    }
    // the thread's columns 2t and 2t + 1 of the permuted tiles are dimensions 16t .. 16t + 15 of
    // each half; with one head per thread the products of the low parts are added here. Products with 0 tell
    // heads with a mean that is not finite.
#pragma unroll
    for (int w = 0; w < HT; ++w)
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            float y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float *o = acc[h * 8 + e + k];
              y[k] = (HT == 1 ? o[q] + o[q + 2] : o[q + 2 * w]) * inv_run[w];
              not_finite[w] += y[k] * 0.f;
            }
            *reinterpret_cast<float4 *>(s_o(warp) + (r + 8 * w) * ROW + h * 64 + t * 16 + q * 8 + e) =
                make_float4(y[0], y[1], y[2], y[3]);
          }
    uint32_t again[HT];
#pragma unroll
    for (int h = 0; h < HT; ++h)       // (a denominator of NaN stays)
      again[h] = __ballot_sync(0xffffffffu, r + 8 * h < rows && not_finite[h] != 0.f && l_run[h] == l_run[h]);
    if (__builtin_expect((again[0] | again[HT - 1]) != 0u, 0)) {
      __syncwarp();
#pragma unroll 1
      for (int row = 0; row < rows; ++row)
        if (((row < 8 ? again[0] : again[HT - 1]) >> (row & 7) * 4) & 0xfu)
          add_up_again<T, D>(p, b, head, h0 + row, unit0 * kDecodeUnit + warp * 16, key1,
                             s_o(warp) + row * ROW, &s_m[warp][row], &s_l[warp][row]);
    }
    __syncthreads();

    const int first_unit = cur.start + m * cur.units;
    const int cta0 = first_unit / per, cta1 = (first_unit + cur.units - 1) / per;
    const int item = b * items + m;
    const int64_t slot = static_cast<int64_t>(cta) + item;
    const bool whole = cta0 == cta1;
    for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
      const int row = i / (D / 4), col = (i - row * (D / 4)) * 4;
      float mt = s_m[0][row];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) mt = fmaxf(mt, s_m[w][row]);
      const float base = mt == -INFINITY ? 0.f : mt;
      float l = 0.f, part[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        part[w] = exp2f(s_m[w][row] - base) * s_l[w][row];
        l += part[w];
      }
      const float inv = reciprocal_of_sum(l);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = share_of(part[w] * inv);
        const float4 x = *reinterpret_cast<const float4 *>(s_o(w) + row * ROW + col);
        o.x += f * x.x;
        o.y += f * x.y;
        o.z += f * x.z;
        o.w += f * x.w;
      }
      if (whole) {
        *reinterpret_cast<uint2 *>(p.out + b * p.o_batch + (h0 + row) * p.o_head + col * 2) =
            make_uint2(Elem<T>::pack(o.x, o.y), Elem<T>::pack(o.z, o.w));
        if (col == 0) {
          const float l2 = base + log2f(l);
          p.lse2[b * c.hq + h0 + row] = l2;
          if (p.lse) p.lse[b * c.hq + h0 + row] = l2 * 0.6931471805599453f;
        }
      } else {
        *reinterpret_cast<float4 *>(p.part_o + (slot * TILE + row) * D + col) = o;
        if (col == 0) p.part_ml[slot * TILE + row] = make_float2(mt, l);
      }
    }

    if (!whole) {
      // ---- the last of the item's CTAs joins its pieces, in the order of the entries
      __syncthreads();
      if (threadIdx.x == 0) {
        // releases the block's writes (which the barrier orders before it) and acquires the others'
        const int done = atomic_add_acq_rel(&p.counters[item], 1);
        s_scan[19] = done == cta1 - cta0;
        if (done == cta1 - cta0) p.counters[item] = 0;
      }
      __syncthreads();
      if (s_scan[19]) {
        for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
          const int row = i / (D / 4), col = (i - row * (D / 4)) * 4;
          float mt, l, lower = 1.f;
          float4 o;
          // sums past fp32's range are taken once more, 2^-31 as large
          for (;; lower = 0x1p-31f) {
            mt = -INFINITY, l = 0.f;
            o = make_float4(0.f, 0.f, 0.f, 0.f);
            const float2 *ml = p.part_ml + (static_cast<int64_t>(item) + cta0) * TILE + row;
            const float *po =
                p.part_o + ((static_cast<int64_t>(item) + cta0) * TILE + row) * D + col;
            for (int k = cta0; k <= cta1; ++k, ml += TILE, po += TILE * D) {
              const float2 y = __ldcg(ml);
              const float4 x = __ldcg(reinterpret_cast<const float4 *>(po));
              const float mn = fmaxf(mt, y.x);
              const float base = mn == -INFINITY ? 0.f : mn;
              const float fa = exp2f(mt - base), part = y.y * exp2f(y.x - base);
              const float ga = share_of(fa), gb = share_of(part * lower);
              mt = mn;
              l = l * fa + part;
              o.x = o.x * ga + x.x * gb;
              o.y = o.y * ga + x.y * gb;
              o.z = o.z * ga + x.z * gb;
              o.w = o.w * ga + x.w * gb;
            }
            if (lower != 1.f || o.x * 0.f + o.y * 0.f + o.z * 0.f + o.w * 0.f == 0.f) break;
          }
          const float inv = reciprocal_of_sum(l * lower);
          *reinterpret_cast<uint2 *>(p.out + b * p.o_batch + (h0 + row) * p.o_head + col * 2) =
              make_uint2(Elem<T>::pack(o.x * inv, o.y * inv),
                         Elem<T>::pack(o.z * inv, o.w * inv));
          if (col == 0) {
            const float l2 = (mt == -INFINITY ? 0.f : mt) + log2f(l);
            p.lse2[b * c.hq + h0 + row] = l2;
            if (p.lse) p.lse[b * c.hq + h0 + row] = l2 * 0.6931471805599453f;
          }
        }
      }
    }
    __syncthreads();   // the merge buffer is free again
    pos += n;
    if (pos < end && pos - cur.start == cur.units * items) next_sequence(c, items, &cur);
  }
}

// weight[entry, KV head] += sum over the KV head's query heads of 2^(logit - lse2). A thread takes four
// entries; the logits of the pass before are read once, most of them from L2. Bound by its chain (length,
// logits, page) in one round of blocks. 6 prompts, 223000 entries, 28 heads: 15 us behind cold caches, and 5
// more for the logits' stores in a decode of 83; lanes on consecutive entries with single-word loads took
// 6 us more.
constexpr int kWeightThreads = 256;

__global__ void __launch_bounds__(kWeightThreads, 6)
    add_weight_kernel(const __grid_constant__ DecodeParams p) {
  __shared__ int s_scan[20];
  const CacheView &c = p.c;
  grid_dependency_wait();
  grid_dependents_go();
  Cursor cur;
  int total;
  const int per = locate(c, c.hkv, gridDim.x, blockIdx.x, s_scan, &cur, &total);
  int pos = per * blockIdx.x;
  const int end = min(pos + per, total);
  while (pos < end) {
    const int in_seq = pos - cur.start;
    const int head = in_seq / cur.units;
    const int unit0 = in_seq - head * cur.units;
    const int n = min(cur.units - unit0, end - pos);
    const int key1 = min(cur.len, (unit0 + n) * kDecodeUnit);
    const int64_t row0 = static_cast<int64_t>(cur.b) * c.hq + head * c.g;
    for (int e = unit0 * kDecodeUnit + threadIdx.x * 4; e < key1; e += kWeightThreads * 4) {
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int h = 0; h < c.g; ++h) {
        const float4 x = __ldcg(reinterpret_cast<const float4 *>(p.logits + (row0 + h) * p.cap64 + e));
        const float l2 = p.lse2[row0 + h];
        // a row whose every logit is -inf has no weights
        const float base = l2 == -INFINITY ? INFINITY : l2;
        sum[0] += exp2f(x.x - base);
        sum[1] += exp2f(x.y - base);
        sum[2] += exp2f(x.z - base);
        sum[3] += exp2f(x.w - base);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (e + i >= key1) break;
        int slot, off;
        split_entry(c, e + i, slot, off);
        const int pg = page_at(c, cur.b, slot);
        if (pg >= 0) atomicAdd(c.weight + track_at(c, pg, head, off), sum[i]);
      }
    }
    pos += n;
    if (pos < end && pos - cur.start == cur.units * c.hkv) next_sequence(c, c.hkv, &cur);
  }
}

template <class T, int D, int TILE>
cudaError_t launch_decode_t(const DecodeParams &p, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed{0};
  const auto kern = paged_decode_kernel<T, D, TILE>;
  const cudaError_t e = allow_shared(kern, kRingBytes<D>, &allowed);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(p.grid), kThreads, kRingBytes<D>, 1, stream, p);
}

template <class T>
cudaError_t launch_decode_d(const DecodeParams &p, cudaStream_t stream) {
  if (p.c.d == 128)
    return p.tile == 8 ? launch_decode_t<T, 128, 8>(p, stream) : launch_decode_t<T, 128, 16>(p, stream);
  return p.tile == 8 ? launch_decode_t<T, 64, 8>(p, stream) : launch_decode_t<T, 64, 16>(p, stream);
}

}  // namespace

cudaError_t launch_decode(const DecodeParams &p, int dtype, int num_sms, cudaStream_t stream) {
  const cudaError_t e = dtype == RRA_BF16 ? launch_decode_d<__nv_bfloat16>(p, stream)
                                          : launch_decode_d<__half>(p, stream);
  if (e != cudaSuccess || !p.logits) return e;
  return launch_dependent(add_weight_kernel, dim3(num_sms * 6), kWeightThreads, 0, 1, stream, p);
}

}  // namespace rra
