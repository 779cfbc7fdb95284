// Device helpers of the cache operators: entry addresses and the two 16-bit element types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache_internal.h"
#include "common.cuh"

namespace rra {

// Waits until the kernels before this one on the stream are complete and their writes visible; every
// thread calls it before it touches global memory.
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// Lets the next kernel's blocks be set up from now on (it waits for this grid's end all the same).
__device__ __forceinline__ void grid_dependents_go() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ int atomic_add_acq_rel(int32_t *p, int x) {
  int old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(x) : "memory");
  return old;
}

__device__ __forceinline__ void raise(uint32_t *status, uint32_t bit) { atomicOr(status, bit); }

// Length of sequence b, clamped to what the page table can hold.
__device__ __forceinline__ int cache_len(const CacheView &c, int b) {
  const int n = c.len[b];
  return n < 0 ? 0 : (n > c.cap ? c.cap : n);
}

__device__ __forceinline__ void split_entry(const CacheView &c, int e, int &slot, int &off) {
  slot = static_cast<int>(__umulhi(static_cast<uint32_t>(e) * 2u, c.ps_magic) >> c.ps_shift);
  off = e - slot * c.ps;
}

// Page of table place `slot` of sequence b, or -1 (flagged) if it is not a page of the cache.
__device__ __forceinline__ int page_at(const CacheView &c, int b, int slot) {
  const int pg = c.table[b * c.table_stride + slot];
  if (static_cast<unsigned>(pg) < static_cast<unsigned>(c.num_pages)) return pg;
  raise(c.status, kErrBadPage);
  return -1;
}

// Place of an entry in weight and order.
__device__ __forceinline__ int64_t track_at(const CacheView &c, int page, int head, int off) {
  return (static_cast<int64_t>(page) * c.hkv + head) * c.ps + off;
}

// A row that is read once. (None of these kernels reads through the non-coherent path: they may be set
// up while the kernel that writes what they read still runs.)
__device__ __forceinline__ uint4 ld_stream(const void *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// kRaise: decode multiplies the softmax weights, which are 1 at most, by 2^kRaise before it rounds them to
// the element type. fp16 has a smallest step of 2^-24: raised by 15 (32768 is still below its largest
// value) a weight keeps 2^-40 of the largest one. bf16 reaches as far as fp32.
template <class T>
struct Elem;

template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kRaise = 0;
  static __device__ __forceinline__ float2 unpack(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  // D (16 x 8, fp32) += A (16 x 16) B (16 x 8)
  static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
};

template <>
struct Elem<__half> {
  static constexpr int kRaise = 15;
  static __device__ __forceinline__ float2 unpack(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
};

}  // namespace rra
