// Internal interface between the C ABI of the cache operators (rra_cache_api.cu) and their kernels
// (rope_append.cu, paged_decode.cu, cache_evict.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "rra_cache.h"

namespace rra {

// Entries that one CTA step of the decode kernel covers (4 warps of 16), and the granule in which
// its work is split over the grid.
constexpr int kDecodeUnit = 64;
// Query heads of a KV head that one warp of the decode kernel carries: 8 fill half of its MMA tiles and leave
// the other half to the low parts of their weights; more than 8 are cheaper 16 at a time than K and V
// read once more.
constexpr int decode_tile(int g) { return g > 8 ? 16 : 8; }

// CTAs of the decode kernel that share an SM.
constexpr int decode_ctas(int head_dim) { return head_dim == 128 ? 2 : 3; }

// The cache as the kernels see it.
struct CacheView {
  int batch, hq, hkv, g, d;
  int ps;                      // page size
  uint32_t ps_magic, ps_shift; // e / ps = (2 e * ps_magic >> 32) >> ps_shift for 0 <= e < 2^31
  int num_pages, max_pages, cap;   // cap = max_pages * ps
  int64_t page_bytes, head_bytes, entry_bytes;
  int64_t table_stride;
  uint8_t *k, *v;
  const int32_t *table;
  int32_t *len;
  float *weight;
  int32_t *order;
  int32_t *seen;
  uint32_t *status;            // sticky error word of the workspace
};

// Workspace of a cache (byte offsets). Header: the status word, the append kernel's count of
// finished blocks and the eviction's call count. The counters are zero between calls: the block that
// completes a count resets it.
struct CacheLayout {
  size_t status, done, epoch, counters;   // counters: int32 per (sequence, KV head, head tile)
  size_t part_o, part_ml;          // partial outputs and (max, sum) of the decode pieces
  size_t lse2;                     // fp32 [batch, hq]: log2 of the softmax denominators
  size_t skip, tags, lens, plan;   // 32-bit [batch], [batch], [batch] and [batch * hkv]
  size_t owner;                    // uint64 [num_pages]
  size_t big;                      // logits [batch, hq, cap64], or the evict kernel's move lists
  size_t total;
  int grid;                        // CTAs of the decode kernel
  int head_tiles;                  // ceil(g / decode_tile(g))
  int64_t cap64;                   // cap rounded up to kDecodeUnit
  int64_t moves;                   // places of one move list
};

CacheLayout cache_layout(const CacheView &c, bool tracked, int num_sms);

struct RopeParams {
  int batch, hq, hkv, tokens, d, rot;
  int heads;          // rows of heads per token: hq + hkv (+ hkv with v), those that are given
  int heads_per_thread;
  int inverse;
  rra_positions pos;
  rra_view q, k, v, qo, ko, vo;   // byte strides
  const int32_t *new_len;
  int advance;
  uint32_t *done;
  uint64_t turn[RRA_ROPE_MAX_PAIRS];
  uint8_t axis[RRA_ROPE_MAX_PAIRS];
};

struct DecodeParams {
  CacheView c;
  const uint8_t *q;
  uint8_t *out;
  int64_t q_batch, q_head, o_batch, o_head;   // bytes
  float *lse;
  float scale_log2;
  int tile, head_tiles, grid;
  float *part_o;
  float2 *part_ml;
  int32_t *counters;
  float *lse2;
  float *logits;      // NULL unless weights are accumulated
  int64_t cap64;
};

struct EvictParams {
  CacheView c;
  int budget, sinks, recent, advance;
  int four;                    // weights and ordinals may be read four at a time
  uint32_t *epoch;             // calls so far; a call marks what it finds with epoch + 1
  uint32_t *skip, *tags;       // [batch]: the call that left the sequence alone; the current one
  int32_t *lens, *plan;        // [batch] lengths; [batch * hkv] moves
  unsigned long long *owner;   // [num_pages]: tag << 32 | sequence of the last claim
  int32_t *moves;
  int64_t moves_cap;
};

// Allows a kernel more than 48 KB of shared memory, once per device (`allowed`: a bit for each).
template <class... Params>
cudaError_t allow_shared(void (*kern)(Params...), size_t bytes, std::atomic<uint64_t> *allowed) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (allowed->load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes));
  if (e == cudaSuccess) allowed->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launches a kernel that begins with griddepcontrol.wait: its blocks may be set up while the kernel before
// it on the stream drains. cluster: blocks per cluster.
template <class... Params, class... Args>
cudaError_t launch_dependent(void (*kern)(Params...), dim3 grid, int threads, size_t smem,
                             int cluster, cudaStream_t stream, const Args &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

cudaError_t launch_rope(const RopeParams &p, const CacheView *cache, int dtype, int pairing,
                        int num_sms, cudaStream_t stream);
cudaError_t launch_decode(const DecodeParams &p, int dtype, int num_sms, cudaStream_t stream);
cudaError_t launch_evict(const EvictParams &p, int num_sms, cudaStream_t stream);

}  // namespace rra
