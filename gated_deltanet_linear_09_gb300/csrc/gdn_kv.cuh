// gdn_kv.cuh -- the paged key/value cache as the kernels see it: geometry, a token's place, and
// the exact e4m3 -> bf16 conversion.
#pragma once

#include <cuda_fp16.h>

#include "gdn_internal.h"

namespace gdn {

// Where a packed token lives: page < 0 when it has no place; its position in the sequence.
struct Place {
  int page, off, pos;
};

// The sequence holding packed token t: the largest s with cu[s] <= t, by a 32-way search of the
// whole warp (all lanes with the same t, or each lane its own: the search follows the least t of
// the warp and every lane then steps forward to its own).
__device__ __forceinline__ int find_seq(const KvBatchView& b, int t) {
  const int lane = threadIdx.x & 31;
  const int t0 = __reduce_min_sync(0xffffffffu, t);
  int lo = 0, hi = b.num_seqs;                  // cu[lo] <= t0 (cu[0] = 0), answer in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5;
    const int i = lo + lane * step;
    const bool le = i < hi && (lane == 0 || __ldg(b.cu + i) <= t0);
    const int k = __popc(__ballot_sync(0xffffffffu, le));   // lanes 0..k-1 when cu is monotone
    lo += (k - 1) * step;
    hi = min(hi, lo + step);
  }
  while (lo + 1 < b.num_seqs && __ldg(b.cu + lo + 1) <= t) ++lo;
  return lo;
}

// The place of packed token t (all 32 lanes of the warp call this together).
__device__ __forceinline__ Place find_place(const KvView& c, const KvBatchView& b, int t) {
  const int s = find_seq(b, t);
  const int c0 = __ldg(b.cu + s), c1 = __ldg(b.cu + s + 1);
  Place p{-1, 0, 0};
  if (t >= c1 && s == b.num_seqs - 1 && c1 >= c0) return p;    // padding past the last sequence
  const long long len = __ldg(b.lens + s);
  if (c0 < 0 || t < c0 || t >= c1 || c1 > b.total || len < 0 || len > ((long long)b.table_cols << c.page_shift)) {
    set_status(c.status, GDN_STATUS_BAD_SEQLENS);
    return p;
  }
  const long long pos = len - (c1 - t);
  if (pos < 0) return p;
  const int page = __ldg(b.table + (long long)s * b.table_ld + (pos >> c.page_shift));
  if (page < 0 || page >= c.num_pages) {
    set_status(c.status, GDN_STATUS_PAGE_RANGE);
    return p;
  }
  p.page = page;
  p.pos = (int)pos;
  p.off = (int)(pos & ((1 << c.page_shift) - 1));
  return p;
}

// ------------------------------------------------------------------ e4m3 -> bf16

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The e4m3 codes in the upper bytes of w's two halves as bf16 values.  A code's exponent and
// mantissa, moved to the low four exponent bits and the high three mantissa bits of a bf16, are
// the value times 2^-120 (the biases 127 and 7 apart; subnormals included), so one exact multiply
// by 2^120 finishes.  The NaN codes 0x7f / 0xff (which the cache never holds) come out as +-480.
__device__ __forceinline__ uint32_t e4m3_hi_bits(uint32_t w) {
  return ((w >> 4) & 0x07f007f0u) | (w & 0x80008000u);
}
__device__ __forceinline__ uint32_t e4m3_hi_to_bf16x2(uint32_t w) { return mul_bf16x2(e4m3_hi_bits(w), 0x7b807b80u); }

// Four codes b0..b3 (b0 lowest) -> the bf16 pairs (b0, b1) and (b2, b3).
__device__ __forceinline__ void e4m3x4_to_bf16(uint32_t w, uint32_t& p01, uint32_t& p23) {
  p01 = e4m3_hi_to_bf16x2(__byte_perm(w, 0, 0x1404));
  p23 = e4m3_hi_to_bf16x2(__byte_perm(w, 0, 0x3424));
}

// The bf16 bits of the scale with exponent byte b (255: NaN).
__device__ __forceinline__ uint32_t scale_bits(uint32_t b) { return b == 255 ? 0x7fc0u : b << 7; }

// The same as an f32.
__device__ __forceinline__ float scale_f32(uint32_t b) { return __uint_as_float(scale_bits(b) << 16); }

// The exponent byte of a vector whose largest magnitude has the bf16 bits `top` (sign cleared):
// 1.m * 2^(E - 127) <= 448 = 1.75 * 2^8 asks for 2^(E - 135), one more when 1.m > 1.75.  Bytes
// below 10 would put the least e4m3 value times the scale outside bf16's normal range.
__device__ __forceinline__ int scale_byte(uint32_t top) {
  if (top >= 0x7f80u) return 255;
  if (top == 0) return 127;
  const int e = (int)(top >> 7) - 8 + ((top & 0x7f) > 0x60 ? 1 : 0);
  return e < 10 ? 10 : e;
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_to_e4m3(uint32_t w) {
  uint16_t h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
      : "=h"(h)
      : "f"(__uint_as_float(w & 0xffff0000u)), "f"(__uint_as_float(w << 16)));
  return h;
}

// Two elements of a query row as hi + lo in e4m3 codes.  A row brought to (224, 448] by a power of two
// is the sum of two e4m3 vectors: bf16 has eight significant bits and e4m3 four, and splitting by the
// product with 2^4 + 1 (Veltkamp) leaves four and four, exactly.  Elements below 2^-10 of the row's
// largest, whose parts fall out of e4m3's exponents, lose bits at 2^-17 of it.
__device__ __forceinline__ void split_e4m3(uint32_t x, uint32_t& hi, uint32_t& lo) {
  const uint32_t c = mul_bf16x2(x, 0x41884188u), h = sub_bf16x2(c, sub_bf16x2(c, x));
  hi = bf16x2_to_e4m3(h);
  lo = bf16x2_to_e4m3(sub_bf16x2(x, h));
}
// What brings a row of this scale byte there, as two bf16 (a row that reads as NaN: ones).
__device__ __forceinline__ uint32_t split_factor(int b) { return (uint32_t)(b == 255 ? 127 : 254 - b) * 0x00800080u; }

}  // namespace gdn
