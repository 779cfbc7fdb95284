/*
 * rra_cache.h - C ABI of the cache operators: what stands before and behind the prefill of rra.h.
 *
 *   rotary positions - rra_rope_rotate turns the query and key rows of a prompt by positions with
 *                      one or several axes (time, height, width), or back (the gradient);
 *                      rra_cache_append does the same for new tokens and writes their keys and
 *                      values into a paged key-value cache;
 *   decode attention - rra_cache_decode: attention of one new token per sequence over its cached
 *                      entries, split over the cache's length and joined;
 *   eviction         - rra_cache_evict keeps the entries with the largest accumulated attention
 *                      weight (rra_cache_decode accumulates it) and compacts the cache in place.
 *
 * Conventions, beside those of rra.h (device pointers, 16-byte alignment, no allocation, work
 * enqueued on `stream` without synchronising, argument errors reported before anything is enqueued)
 *   - Element type: bf16 or fp16, the same for queries, keys, values and outputs. head_dim 64 or
 *     128. Query head h reads KV head h / (heads_q / heads_kv).
 *   - A view is a tensor [batch, heads, tokens, head_dim] whose last dimension is contiguous; its
 *     other strides are counted in elements and are multiples of 8, so that every row is 16-byte
 *     aligned. Input strides may be 0 (a broadcast input); the rows of an output do not overlap.
 *   - Cache entry e of sequence b is row e % page_size of page page_table[b][e / page_size]. The
 *     key of KV head h of that entry is at k + page * page_stride + h * head_stride +
 *     (e % page_size) * entry_stride, its value at the same place of v.
 *   - Softmax does not depend on the order of the entries: eviction changes it, and keys carry their
 *     position from the rotation. A tracked cache also holds, per entry and KV head, the attention
 *     weight accumulated so far and the token's ordinal, both [num_pages, heads_kv, page_size]. Weights
 *     come from rra_cache_decode alone, or from the caller: after a prompt that went through
 *     rra_prefill and rra_cache_append they are all 0. len and seen are arrays of their own.
 *   - Lengths, page tables and ordinals live on the device and are read there: calls can be captured
 *     into a CUDA graph and replayed while they change.
 *   - A device-side mistake never reads or writes outside the cache; it sets the workspace's sticky
 *     error word (rra_check_device_status of rra.h reads and clears it, RRA_ERR_INVALID_ARG): a
 *     length below 0 or beyond the page table counts as the nearest valid one, an entry on a page
 *     outside [0, num_pages) as absent.
 *   - The calls that share a workspace must not overlap on the GPU, nor must the calls that write a
 *     cache and any other call on that cache. A workspace may serve several caches of the same sizes (the
 *     layers of a model); for other sizes it is laid out otherwise and has to be zero-filled again. That of
 *     a tracked cache has room for the logits of a decode that adds weights, 4 bytes per sequence,
 *     query head and entry of the page table's width.
 */
#ifndef RRA_CACHE_H_
#define RRA_CACHE_H_

#include "rra.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { RRA_BF16 = 0, RRA_F16 = 1 } rra_dtype;
typedef enum {
  RRA_PAIRS_HALVES = 0,   /* pair i is (i, i + rotary_dim / 2) */
  RRA_PAIRS_ADJACENT = 1  /* pair i is (2 i, 2 i + 1) */
} rra_pairing;

#define RRA_ROPE_MAX_PAIRS 64
#define RRA_ROPE_MAX_AXES 4

/* Filled by rra_rope_init; a plain host value that may be copied. */
typedef struct {
  int head_dim, rotary_dim, axes, pairing;
  uint64_t turn[RRA_ROPE_MAX_PAIRS]; /* turns per position, as a fraction of 2^64 */
  uint8_t axis[RRA_ROPE_MAX_PAIRS];  /* the axis whose position turns the pair */
} rra_rope;

/* One tensor [batch, heads, tokens, head_dim] of q, k or v; data == NULL: not given. */
typedef struct {
  void *data;
  int64_t batch, head, token;        /* strides in elements */
} rra_view;

/* int32 positions [axes, batch, tokens]. */
typedef struct {
  const int32_t *data;
  int64_t axis, batch, token;        /* strides in elements, may be 0 */
} rra_positions;

/* The tokens of a call. */
typedef struct {
  int batch, heads_q, heads_kv, tokens, dtype;
  rra_positions positions;
  rra_view q, k, v;                  /* inputs */
  rra_view q_out, k_out, v_out;      /* outputs; an output may be its own input, stride for stride */
} rra_tokens;

typedef struct {
  int batch;             /* sequences (rows of page_table) >= 0 */
  int heads_q, heads_kv; /* heads_q % heads_kv == 0 */
  int head_dim;          /* 64 or 128 */
  int dtype;             /* rra_dtype of k, v, queries and outputs */
  int page_size;         /* entries per page >= 1 */
  int num_pages;         /* pages of k and v >= 1 */
  int max_pages;         /* page_table entries per sequence >= 1; max_pages * page_size <= 2^30 */
  float softmax_scale;   /* <= 0 means 1/sqrt(head_dim) */
  int reserved;          /* 0 */
  int64_t page_stride, head_stride, entry_stride; /* of k and v, in elements, multiples of 8 */
  int64_t table_stride;  /* elements between rows of page_table */
  void *k, *v;
  const int32_t *page_table;
  int32_t *len;          /* [batch] entries of each sequence */
  float *weight;         /* accumulated attention weight; weight, order and seen all or none */
  int32_t *order;        /* token ordinal of each entry */
  int32_t *seen;         /* [batch] tokens that each sequence has seen */
  void *workspace;       /* rra_cache_workspace_bytes, zero-filled once before its first use */
  size_t workspace_bytes;
} rra_cache;

/* Describes a rotation of the first rotary_dim of head_dim dimensions (rotary_dim a multiple of 16,
 * head_dim 64 or 128, 1 <= axes <= 4). Pair i turns by position[axis of i] * frequency of i.
 * inv_freq: rotary_dim / 2 frequencies in radians per position, or NULL for
 * theta^(-2 i / rotary_dim). axis_of_pair: rotary_dim / 2 axes, or NULL for `sections`: the first
 * sections[0] pairs follow axis 0, the next sections[1] axis 1, and so on (their sum is
 * rotary_dim / 2; NULL with one axis). Frequencies are kept as 64-bit fractions of a turn, so the
 * angle of a far position loses nothing to its size: the multiple of the full turn drops out of an
 * integer product. Runs on the host. */
rra_status rra_rope_init(rra_rope *rope, int head_dim, int rotary_dim, int axes, int pairing,
                         double theta, const double *inv_freq, const int32_t *sections,
                         const int32_t *axis_of_pair);

/* Rotates q into q_out and k into k_out; either pair may be left out. inverse != 0 turns back,
 * which takes the gradients of the outputs to those of the inputs. v and v_out, if given, are
 * copied. Batch, heads and tokens may be 0 (nothing is enqueued). */
rra_status rra_rope_rotate(const rra_rope *rope, const rra_tokens *tokens, int inverse,
                           rra_stream_t stream);

/* Bytes of workspace of the cache calls for these sizes on the current device (k, v and the other
 * pointers are not read; weight != NULL or not says whether the cache is tracked). 0 if invalid. */
size_t rra_cache_workspace_bytes(const rra_cache *cache);

/* Rotates q and k and appends k and v to the cache: token t of sequence b becomes entry
 * len[b] + t. tokens->batch == cache->batch; q and q_out, k_out, v_out may be left out. new_len:
 * int32 [batch] with the tokens of each sequence that are real, or NULL for all; padding (t >=
 * new_len[b]) is neither read nor written. Tracked caches get weight 0 and ordinal seen[b] + t.
 * advance != 0 adds the new tokens to len and seen; layers that share them advance with the last
 * one. Entries past the page table are dropped and flagged. Sequences may share pages as long as no
 * two tokens of a call fall on the same row (theirs would mix). */
rra_status rra_cache_append(const rra_cache *cache, const rra_rope *rope,
                            const rra_tokens *tokens, const int32_t *new_len, int advance,
                            rra_stream_t stream);

/* out[b, h] = sum over the entries e < len[b] of softmax(softmax_scale q_h . k_e) v_e; lse[b, h]
 * (fp32 [batch, heads_q], may be NULL) the natural logarithm of the softmax's denominator. q and
 * out are views with one token (their token stride is not used); out may be q. A sequence without
 * entries gets out 0 and lse -inf. A logit of -inf counts as absent, whatever its value. Any other
 * entry has a weight above 0, however small: an infinite value makes its output infinite, a NaN or
 * infinities of both signs make it NaN. A logit of +inf or NaN makes its head's out and lse NaN (and
 * the weights that the head gives, with add_weight). Logits, sums and outputs are held in fp32 and
 * rounded once, to the element type. add_weight != 0 (tracked caches)
 * adds to the weight of every entry and KV head the softmax weights that the KV head's query heads
 * gave it. Rows of page_table may share pages here; with add_weight a shared entry then gets
 * the sum of its rows, added in no fixed order. Otherwise equal calls give equal bits. */
rra_status rra_cache_decode(const rra_cache *cache, const rra_view *q, const rra_view *out,
                            float *lse, int add_weight, rra_stream_t stream);

/* Cuts every sequence with more than `budget` entries down to budget, per KV head: entries whose
 * ordinal is below `sinks` or at least seen[b] - recent are kept, then those of the largest weight
 * (negative and NaN weights count as 0; ties: the lower entry). sinks + recent <= budget. The kept
 * entries at or behind `budget`, in ascending order, move into the places of the evicted ones
 * before it, in ascending order, with their weight and ordinal; nothing else moves, and entries at or
 * behind `budget` stay as they were. advance != 0 sets len[b] = budget; layers that share len
 * advance with the last one. Needs a tracked cache. Sequences that share a page, with another or with
 * themselves, or have a bad one are left as they are, since their entries could not move apart; this is
 * flagged if one of the sharing sequences is over the budget. The launch is sized by the page table's
 * width, since lengths are on the device: a table much wider than its sequences costs time. */
rra_status rra_cache_evict(const rra_cache *cache, int budget, int sinks, int recent, int advance,
                           rra_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RRA_CACHE_H_ */
