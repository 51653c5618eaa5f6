// Device helpers of the attention operators: 16-bit element types, the rows of a sequence, page
// lookup.
#pragma once
#include "attention.h"
#include "ptx.cuh"

namespace mlap {

template <bool BF16>
struct Half16;
template <>
struct Half16<false> {
  using T = __half;
  using T2 = __half2;
  static __device__ __forceinline__ float to_f(T v) { return __half2float(v); }
  static __device__ __forceinline__ T from_f(float v) { return __float2half_rn(v); }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const T2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <>
struct Half16<true> {
  using T = __nv_bfloat16;
  using T2 = __nv_bfloat162;
  static __device__ __forceinline__ float to_f(T v) { return __bfloat162float(v); }
  static __device__ __forceinline__ T from_f(float v) { return __float2bfloat16_rn(v); }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const T2 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

// Two int8 codes (bytes of a word with 0x80 added to each) as exact f16: 0x6400 | u is 1024 + u.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t codes_f16(uint32_t biased) {
  const uint32_t h = __byte_perm(biased, 0x64646464u, SEL);
  const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&h),
                            __half2half2(__ushort_as_half(static_cast<unsigned short>(0x6480u))));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The same, times 2^-14, as exact bf16: the bits 0x00uu are u 2^-133 for every byte u, below the
// normal range and in its first binade alike, and (u - 128) 2^-14 has eight bits.  So reduced, 128
// products with a bf16 query add up inside fp32's range whatever the query's values are (128 * 128 *
// 2^-14 = 1).
constexpr float kCodeUnits = 16384.f;      // of a bf16 code: what a score has to be multiplied by
template <uint32_t SEL>
__device__ __forceinline__ uint32_t codes_bf16(uint32_t biased) {
  const uint32_t h = __byte_perm(biased, 0u, SEL);
  uint32_t v;                              // h * 2^119 - 128 * 2^-14
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v) : "r"(h), "r"(0x7b007b00u), "r"(0xbc00bc00u));
  return v;
}
// A word's codes as operands of the queries' type.
template <bool BF16, uint32_t SEL>
__device__ __forceinline__ uint32_t codes16(uint32_t w) {
  if constexpr (BF16) return codes_bf16<SEL>(w ^ 0x80808080u);
  return codes_f16<SEL>(w ^ 0x80808080u);
}

__device__ __forceinline__ uint32_t div_fast(uint32_t n, const FastDiv& f) {
  return f.d > 1 ? static_cast<uint32_t>(__umul64hi(n, f.magic)) : n;
}

// Value scales below 2^-90 count as 0: their inverses, which the sums of the weights carry, and
// 2^20 keys of weight 2^14 then stay inside fp32.
constexpr float kTinyScale = 8.0779356e-28f;

// Token rows and positions of a sequence; len 0 for one that is empty or skipped.
struct SeqRows {
  int64_t row0;                // first token row
  int32_t len;                 // token rows
  int32_t ctx;                 // position of the first one
  bool bad;                    // skipped: its entries are out of range
};

__device__ __forceinline__ SeqRows seq_rows(const Ragged& r, int b) {
  const int64_t lo = r.cu[b], hi = r.cu[b + 1];
  const int64_t ctx = r.ctx == nullptr ? 0 : r.ctx[b];
  SeqRows s;
  s.bad = lo < 0 || hi < lo || hi > r.T || hi - lo > r.max_new || ctx < 0 || ctx > kMaxContext;
  s.row0 = s.bad ? 0 : lo;
  s.len = s.bad ? 0 : static_cast<int32_t>(hi - lo);
  s.ctx = s.bad ? 0 : static_cast<int32_t>(ctx);
  return s;
}

// Page of sequence b that holds position pos, or -1: no page, or one that does not exist (bad).
__device__ __forceinline__ int64_t page_of(const Pages& pg, int b, int blk, bool* bad) {
  if (blk >= pg.max_blocks) {
    *bad = true;
    return -1;
  }
  const int64_t id = pg.table[static_cast<int64_t>(b) * pg.max_blocks + blk];
  if (id < -1 || id >= pg.block_num) *bad = true;
  return id >= 0 && id < pg.block_num ? id : -1;
}

}  // namespace mlap
