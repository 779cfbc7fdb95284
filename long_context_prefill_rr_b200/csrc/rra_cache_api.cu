// C ABI of the cache operators (declared in include/rra_cache.h): argument checks, workspace
// carve-up and kernel launches. Nothing is allocated and nothing synchronises.
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "cache_internal.h"

namespace rra {

static size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

CacheLayout cache_layout(const CacheView &c, bool tracked, int num_sms) {
  CacheLayout w{};
  const int tile = decode_tile(c.g);
  w.head_tiles = (c.g + tile - 1) / tile;
  const int64_t items = static_cast<int64_t>(c.batch) * c.hkv * w.head_tiles;
  w.cap64 = (static_cast<int64_t>(c.cap) + kDecodeUnit - 1) / kDecodeUnit * kDecodeUnit;
  // one CTA for every place on the SMs, but no more than there can be units of work
  const int64_t most = items * (w.cap64 / kDecodeUnit);
  w.grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(num_sms * decode_ctas(c.d), most)));
  size_t off = 256;
  w.status = 0;
  w.done = 4;
  w.epoch = 8;
  w.counters = off;
  off = align_up(off + items * 4, 256);
  w.part_ml = off;
  off = align_up(off + (items + w.grid) * tile * 8, 256);
  w.part_o = off;
  off = align_up(off + (items + w.grid) * tile * c.d * 4, 256);
  w.lse2 = off;
  off = align_up(off + static_cast<size_t>(c.batch) * c.hq * 4, 256);
  if (tracked) {
    w.skip = off;
    off = align_up(off + static_cast<size_t>(c.batch) * 4, 256);
    w.tags = off;
    off = align_up(off + static_cast<size_t>(c.batch) * 4, 256);
    w.lens = off;
    off = align_up(off + static_cast<size_t>(c.batch) * 4, 256);
    w.plan = off;
    off = align_up(off + static_cast<size_t>(c.batch) * c.hkv * 4, 256);
    w.owner = off;
    off = align_up(off + static_cast<size_t>(c.num_pages) * 8, 256);
    w.big = off;
    w.moves = c.cap / 2 + 1;   // a list holds at most min(budget, len - budget) entries
    const size_t logits = static_cast<size_t>(c.batch) * c.hq * w.cap64 * 4;
    const size_t lists = static_cast<size_t>(c.batch) * c.hkv * 2 * w.moves * 4;
    off = align_up(off + std::max(logits, lists), 256);
  }
  w.total = off;
  return w;
}

}  // namespace rra

using rra::CacheLayout;
using rra::CacheView;

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool row_stride(int64_t s) { return s >= 0 && s % 8 == 0; }

// SMs of the current device (asked once per device).
int current_sms() {
  static std::atomic<int> cache[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  if (dev >= 0 && dev < 64 && (n = cache[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
  if (dev >= 0 && dev < 64) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

template <class T>
T *at(void *ws, size_t off) {
  return reinterpret_cast<T *>(static_cast<uint8_t *>(ws) + off);
}

// The sizes alone (no pointer is looked at).
rra_status resolve_sizes(const rra_cache *s, CacheView *c) {
  if (!s) return RRA_ERR_INVALID_ARG;
  if (s->batch < 0 || s->heads_q < 1 || s->heads_kv < 1 || s->heads_q % s->heads_kv != 0 ||
      s->page_size < 1 || s->num_pages < 1 || s->max_pages < 1 || s->reserved != 0)
    return RRA_ERR_INVALID_ARG;
  if (s->dtype != RRA_BF16 && s->dtype != RRA_F16) return RRA_ERR_UNSUPPORTED;
  if (s->head_dim != 64 && s->head_dim != 128) return RRA_ERR_UNSUPPORTED;
  const int64_t cap = static_cast<int64_t>(s->max_pages) * s->page_size;
  if (cap > (1 << 30)) return RRA_ERR_UNSUPPORTED;
  const int g = s->heads_q / s->heads_kv;
  // units of work, table places and heads are counted in 32 bits, with room for one more round of CTAs
  const int64_t tiles = (g + rra::decode_tile(g) - 1) / rra::decode_tile(g);
  const int64_t units = (cap + rra::kDecodeUnit - 1) / rra::kDecodeUnit;
  if (s->batch > 0 && (static_cast<int64_t>(s->heads_kv) * tiles > (1 << 30) / s->batch / units ||
                       s->heads_q > INT_MAX / 1024 / s->batch ||
                       s->max_pages > INT_MAX / s->batch))
    return RRA_ERR_UNSUPPORTED;
  *c = CacheView{};
  c->batch = s->batch;
  c->hq = s->heads_q;
  c->hkv = s->heads_kv;
  c->g = g;
  c->d = s->head_dim;
  c->ps = s->page_size;
  // ps_magic = ceil(2^(31 + k) / ps) with 2^k >= ps: it exceeds the quotient by less than 2^k / ps, so
  // e * ps_magic / 2^(31 + k) exceeds e / ps by less than e / (2^31 ps), too little to reach the next
  // integer while e < 2^31; and ps_magic < 2^32
  while ((int64_t{1} << c->ps_shift) < s->page_size) ++c->ps_shift;
  c->ps_magic = static_cast<uint32_t>(((uint64_t{1} << (31 + c->ps_shift)) + s->page_size - 1) /
                                      s->page_size);
  c->num_pages = s->num_pages;
  c->max_pages = s->max_pages;
  c->cap = static_cast<int>(cap);
  return RRA_OK;
}

// A view as the kernels take it: strides in bytes, 0 for a dimension of one place (whatever was given).
rra_view bytes(const rra_view &v, int batch, int heads, int tokens) {
  return {v.data, batch > 1 ? v.batch * 2 : 0, heads > 1 ? v.head * 2 : 0,
          tokens > 1 ? v.token * 2 : 0};
}

// A view that is read: aligned rows, strides of 0 allowed.
bool readable(const rra_view &v, int batch, int heads, int tokens) {
  return aligned16(v.data) && (batch <= 1 || row_stride(v.batch)) &&
         (heads <= 1 || row_stride(v.head)) && (tokens <= 1 || row_stride(v.token));
}

// A view that is written: its rows do not overlap either. With the strides of the dimensions that have
// more than one place in ascending order, each has to step over everything below it.
bool writable(const rra_view &v, int batch, int heads, int tokens, int d) {
  if (!readable(v, batch, heads, tokens)) return false;
  int64_t stride[3] = {v.batch, v.head, v.token}, size[3] = {batch, heads, tokens};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (stride[j] < stride[i]) {
        std::swap(stride[i], stride[j]);
        std::swap(size[i], size[j]);
      }
  int64_t span = d;
  for (int i = 0; i < 3; ++i) {
    if (size[i] <= 1) continue;
    if (stride[i] < span) return false;
    span += stride[i] * (size[i] - 1);
  }
  return true;
}

// Sizes, strides and pointers of a call (no device call is made).
rra_status resolve_cache(const rra_cache *s, CacheView *c) {
  const rra_status st = resolve_sizes(s, c);
  if (st != RRA_OK) return st;
  if (s->batch == 0) return RRA_OK;
  const rra_view rows = {s->k, s->page_stride, s->head_stride, s->entry_stride};
  if (!writable(rows, s->num_pages, s->heads_kv, s->page_size, s->head_dim) ||
      (s->batch > 1 && s->table_stride < s->max_pages))
    return RRA_ERR_INVALID_ARG;
  if (!s->k || !s->v || !s->page_table || !s->len || !s->workspace || !aligned16(s->k) ||
      !aligned16(s->v) || !aligned4(s->page_table) || !aligned4(s->len) || !aligned16(s->workspace))
    return RRA_ERR_INVALID_ARG;
  const bool tracked = s->weight != nullptr;
  if (tracked != (s->order != nullptr) || tracked != (s->seen != nullptr) ||
      !aligned4(s->weight) || !aligned4(s->order) || !aligned4(s->seen))
    return RRA_ERR_INVALID_ARG;
  const rra_view strides = bytes(rows, s->num_pages, s->heads_kv, s->page_size);
  c->page_bytes = strides.batch;
  c->head_bytes = strides.head;
  c->entry_bytes = strides.token;
  c->table_stride = s->batch > 1 ? s->table_stride : 0;
  c->k = static_cast<uint8_t *>(s->k);
  c->v = static_cast<uint8_t *>(s->v);
  c->table = s->page_table;
  c->len = s->len;
  c->weight = s->weight;
  c->order = s->order;
  c->seen = s->seen;
  return RRA_OK;
}

// The workspace of a call whose arguments are right; *w is its carve-up.
rra_status carve(const rra_cache *s, CacheView *c, CacheLayout *w, int *sms) {
  *sms = current_sms();
  if (*sms <= 0) return RRA_ERR_CUDA;
  *w = rra::cache_layout(*c, s->weight != nullptr, *sms);
  if (s->workspace_bytes < w->total) return RRA_ERR_WORKSPACE;
  c->status = at<uint32_t>(s->workspace, w->status);
  return RRA_OK;
}

// Checks the tokens of a call and fills the kernel's parameters.
rra_status resolve_tokens(const rra_rope *r, const rra_tokens *t, rra::RopeParams *p) {
  if (!r || !t) return RRA_ERR_INVALID_ARG;
  if (t->batch < 0 || t->tokens < 0 || t->heads_q < 0 || t->heads_kv < 0)
    return RRA_ERR_INVALID_ARG;
  if (t->dtype != RRA_BF16 && t->dtype != RRA_F16) return RRA_ERR_UNSUPPORTED;
  if ((r->head_dim != 64 && r->head_dim != 128) || r->rotary_dim < 16 ||
      r->rotary_dim % 16 != 0 || r->rotary_dim > r->head_dim || r->axes < 1 ||
      r->axes > RRA_ROPE_MAX_AXES ||
      (r->pairing != RRA_PAIRS_HALVES && r->pairing != RRA_PAIRS_ADJACENT))
    return RRA_ERR_INVALID_ARG;
  if (t->tokens > (1 << 30) || t->heads_q > 65535 || t->heads_kv > 65535)
    return RRA_ERR_UNSUPPORTED;
  const int64_t rows = static_cast<int64_t>(t->batch) * t->tokens;
  if (rows > (static_cast<int64_t>(1) << 35)) return RRA_ERR_UNSUPPORTED;
  if (rows == 0) return RRA_OK;
  const bool hq = t->q.data && t->heads_q > 0, hk = t->k.data && t->heads_kv > 0;
  const bool hv = t->v.data && t->heads_kv > 0;
  if (!t->positions.data || !aligned4(t->positions.data)) return RRA_ERR_INVALID_ARG;
  if ((t->q_out.data && !hq) || (t->k_out.data && !hk) || (t->v_out.data && !hv))
    return RRA_ERR_INVALID_ARG;
  if ((hq && !readable(t->q, t->batch, t->heads_q, t->tokens)) ||
      (hk && !readable(t->k, t->batch, t->heads_kv, t->tokens)) ||
      (hv && !readable(t->v, t->batch, t->heads_kv, t->tokens)))
    return RRA_ERR_INVALID_ARG;
  if ((t->q_out.data && !writable(t->q_out, t->batch, t->heads_q, t->tokens, r->head_dim)) ||
      (t->k_out.data && !writable(t->k_out, t->batch, t->heads_kv, t->tokens, r->head_dim)) ||
      (t->v_out.data && !writable(t->v_out, t->batch, t->heads_kv, t->tokens, r->head_dim)))
    return RRA_ERR_INVALID_ARG;
  if (hq && !t->q_out.data) return RRA_ERR_INVALID_ARG;   // a q that is turned for nothing
  p->batch = t->batch;
  p->hq = t->heads_q;
  p->hkv = t->heads_kv;
  p->tokens = t->tokens;
  p->d = r->head_dim;
  p->rot = r->rotary_dim;
  p->heads = (hq ? t->heads_q : 0) + (hk ? t->heads_kv : 0) + (hv ? t->heads_kv : 0);
  p->pos = t->positions;
  const rra_view none = {nullptr, 0, 0, 0};
  auto q_view = [&](const rra_view &v) { return bytes(v, t->batch, t->heads_q, t->tokens); };
  auto kv_view = [&](const rra_view &v) { return bytes(v, t->batch, t->heads_kv, t->tokens); };
  p->q = hq ? q_view(t->q) : none;
  p->k = hk ? kv_view(t->k) : none;
  p->v = hv ? kv_view(t->v) : none;
  p->qo = q_view(t->q_out);
  p->ko = kv_view(t->k_out);
  p->vo = kv_view(t->v_out);
  std::copy(r->turn, r->turn + RRA_ROPE_MAX_PAIRS, p->turn);
  std::copy(r->axis, r->axis + RRA_ROPE_MAX_PAIRS, p->axis);
  for (int i = 0; i < r->rotary_dim / 2; ++i)
    if (p->axis[i] >= r->axes) return RRA_ERR_INVALID_ARG;
  return RRA_OK;
}

rra_status cuda_status(cudaError_t e) { return e == cudaSuccess ? RRA_OK : RRA_ERR_CUDA; }

}  // namespace

extern "C" {

rra_status rra_rope_init(rra_rope *rope, int head_dim, int rotary_dim, int axes, int pairing,
                         double theta, const double *inv_freq, const int32_t *sections,
                         const int32_t *axis_of_pair) {
  if (!rope) return RRA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return RRA_ERR_UNSUPPORTED;
  if (rotary_dim < 16 || rotary_dim > head_dim || rotary_dim % 16 != 0 || axes < 1 ||
      axes > RRA_ROPE_MAX_AXES ||
      (pairing != RRA_PAIRS_HALVES && pairing != RRA_PAIRS_ADJACENT))
    return RRA_ERR_INVALID_ARG;
  const int pairs = rotary_dim / 2;
  rra_rope r{};
  r.head_dim = head_dim;
  r.rotary_dim = rotary_dim;
  r.axes = axes;
  r.pairing = pairing;
  if (!inv_freq && !(theta > 0.0 && isfinite(theta))) return RRA_ERR_INVALID_ARG;
  // theta^(-2 i / rotary_dim) by multiplication: 64 bits of mantissa lose six of them at most
  const long double step =
      inv_freq ? 1.0L : powl(static_cast<long double>(theta), -2.0L / rotary_dim);
  long double power = 1.0L;
  for (int i = 0; i < pairs; ++i, power *= step) {
    const long double f = inv_freq ? static_cast<long double>(inv_freq[i]) : power;
    if (!isfinite(f)) return RRA_ERR_INVALID_ARG;
    long double turns = f / (2.0L * 3.14159265358979323846264338327950288L);
    turns -= floorl(turns);                       // [0, 1)
    const long double scaled = roundl(turns * 0x1p64L);
    r.turn[i] = scaled >= 0x1p64L ? 0 : static_cast<uint64_t>(scaled);
  }
  if (axis_of_pair) {
    for (int i = 0; i < pairs; ++i) {
      if (axis_of_pair[i] < 0 || axis_of_pair[i] >= axes) return RRA_ERR_INVALID_ARG;
      r.axis[i] = static_cast<uint8_t>(axis_of_pair[i]);
    }
  } else if (sections) {
    int at_pair = 0;
    for (int a = 0; a < axes; ++a) {
      if (sections[a] < 0 || sections[a] > pairs - at_pair) return RRA_ERR_INVALID_ARG;
      for (int i = 0; i < sections[a]; ++i) r.axis[at_pair++] = static_cast<uint8_t>(a);
    }
    if (at_pair != pairs) return RRA_ERR_INVALID_ARG;
  } else if (axes != 1) {
    return RRA_ERR_INVALID_ARG;
  }
  *rope = r;
  return RRA_OK;
}

rra_status rra_rope_rotate(const rra_rope *rope, const rra_tokens *tokens, int inverse,
                           rra_stream_t stream) {
  rra::RopeParams p{};
  const rra_status s = resolve_tokens(rope, tokens, &p);
  if (s != RRA_OK) return s;
  if (p.heads == 0) return RRA_OK;
  if ((p.k.data && !p.ko.data) || (p.v.data && !p.vo.data)) return RRA_ERR_INVALID_ARG;
  p.inverse = inverse != 0;
  const int sms = current_sms();
  if (sms <= 0) return RRA_ERR_CUDA;
  return cuda_status(rra::launch_rope(p, nullptr, tokens->dtype, rope->pairing, sms,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

size_t rra_cache_workspace_bytes(const rra_cache *cache) {
  CacheView c;
  if (resolve_sizes(cache, &c) != RRA_OK) return 0;
  const int sms = current_sms();
  if (sms <= 0) return 0;
  return rra::cache_layout(c, cache->weight != nullptr, sms).total;
}

rra_status rra_cache_append(const rra_cache *cache, const rra_rope *rope,
                            const rra_tokens *tokens, const int32_t *new_len, int advance,
                            rra_stream_t stream) {
  CacheView c;
  CacheLayout w;
  int sms = 0;
  rra::RopeParams p{};
  rra_status s = resolve_cache(cache, &c);
  if (s == RRA_OK) s = resolve_tokens(rope, tokens, &p);
  if (s != RRA_OK) return s;
  if (tokens->batch != cache->batch || tokens->heads_kv != cache->heads_kv ||
      tokens->dtype != cache->dtype || rope->head_dim != cache->head_dim)
    return RRA_ERR_INVALID_ARG;
  if (p.heads == 0) return RRA_OK;   // no tokens
  if (!p.k.data || !p.v.data || !aligned4(new_len)) return RRA_ERR_INVALID_ARG;
  s = carve(cache, &c, &w, &sms);
  if (s != RRA_OK) return s;
  p.new_len = new_len;
  p.advance = advance != 0;
  p.done = at<uint32_t>(cache->workspace, w.done);
  return cuda_status(rra::launch_rope(p, &c, tokens->dtype, rope->pairing, sms,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

rra_status rra_cache_decode(const rra_cache *cache, const rra_view *q, const rra_view *out,
                            float *lse, int add_weight, rra_stream_t stream) {
  rra::DecodeParams p{};
  CacheLayout w;
  int sms = 0;
  rra_status s = resolve_cache(cache, &p.c);
  if (s != RRA_OK) return s;
  if (cache->batch == 0) return RRA_OK;
  if (!q || !out || !q->data || !out->data || !aligned4(lse) ||
      !readable(*q, cache->batch, cache->heads_q, 1) ||
      !writable(*out, cache->batch, cache->heads_q, 1, cache->head_dim))
    return RRA_ERR_INVALID_ARG;
  if (add_weight && !cache->weight) return RRA_ERR_INVALID_ARG;
  s = carve(cache, &p.c, &w, &sms);
  if (s != RRA_OK) return s;
  p.q = static_cast<const uint8_t *>(q->data);
  p.out = static_cast<uint8_t *>(out->data);
  const rra_view qs = bytes(*q, cache->batch, cache->heads_q, 1);
  const rra_view os = bytes(*out, cache->batch, cache->heads_q, 1);
  p.q_batch = qs.batch;
  p.q_head = qs.head;
  p.o_batch = os.batch;
  p.o_head = os.head;
  p.lse = lse;
  const float scale = cache->softmax_scale > 0.f
                          ? cache->softmax_scale
                          : 1.0f / sqrtf(static_cast<float>(cache->head_dim));
  p.scale_log2 = scale * 1.4426950408889634f;
  p.tile = rra::decode_tile(p.c.g);
  p.head_tiles = w.head_tiles;
  p.grid = w.grid;
  p.part_o = at<float>(cache->workspace, w.part_o);
  p.part_ml = at<float2>(cache->workspace, w.part_ml);
  p.counters = at<int32_t>(cache->workspace, w.counters);
  p.lse2 = at<float>(cache->workspace, w.lse2);
  p.logits = add_weight ? at<float>(cache->workspace, w.big) : nullptr;
  p.cap64 = w.cap64;
  return cuda_status(
      rra::launch_decode(p, cache->dtype, sms, reinterpret_cast<cudaStream_t>(stream)));
}

rra_status rra_cache_evict(const rra_cache *cache, int budget, int sinks, int recent, int advance,
                           rra_stream_t stream) {
  rra::EvictParams p{};
  CacheLayout w;
  int sms = 0;
  rra_status s = resolve_cache(cache, &p.c);
  if (s != RRA_OK) return s;
  if (budget < 1 || sinks < 0 || recent < 0 || sinks > budget || recent > budget - sinks)
    return RRA_ERR_INVALID_ARG;
  if (cache->batch == 0) return RRA_OK;
  if (!cache->weight) return RRA_ERR_INVALID_ARG;
  s = carve(cache, &p.c, &w, &sms);
  if (s != RRA_OK) return s;
  p.budget = budget;
  p.sinks = sinks;
  p.recent = recent;
  p.advance = advance != 0;
  // a page's rows of weights then start at multiples of 16 bytes
  p.four = cache->page_size % 4 == 0 && aligned16(cache->weight) && aligned16(cache->order);
  p.epoch = at<uint32_t>(cache->workspace, w.epoch);
  p.skip = at<uint32_t>(cache->workspace, w.skip);
  p.tags = at<uint32_t>(cache->workspace, w.tags);
  p.lens = at<int32_t>(cache->workspace, w.lens);
  p.plan = at<int32_t>(cache->workspace, w.plan);
  p.owner = at<unsigned long long>(cache->workspace, w.owner);
  p.moves = at<int32_t>(cache->workspace, w.big);
  p.moves_cap = w.moves;
  return cuda_status(rra::launch_evict(p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
