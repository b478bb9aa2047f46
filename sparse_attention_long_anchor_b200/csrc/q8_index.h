// Index arithmetic of the 8-bit paged cache: plain functions for the kernels
// and for host code, with no CUDA dependency, so that their bounds are tested
// on the CPU.
#pragma once

#include <stdint.h>

#if defined(__CUDACC__)
#define Q8_HD __host__ __device__ __forceinline__
#else
#define Q8_HD inline
#endif

namespace kascade {

// A page-table entry as a page of the pool: itself, or 0 with `bad` set.
Q8_HD uint32_t q8_page(int32_t entry, int32_t num_pages, bool& bad) {
  if ((uint32_t)entry < (uint32_t)num_pages) return (uint32_t)entry;
  bad = true;
  return 0;
}

// A list entry as one of the row's n >= 1 keys: itself, or the nearest with `bad` set.
Q8_HD int32_t q8_key(int32_t key, int32_t n, bool& bad) {
  if ((uint32_t)key < (uint32_t)n) return key;
  bad = true;
  return key < 0 ? 0 : n - 1;
}

// Whether a slot lies in the pool (slot -1, a padding token, does not).
Q8_HD bool q8_slot_ok(int32_t slot, int32_t num_pages, int page_shift) {
  return (uint32_t)slot < ((uint32_t)num_pages << page_shift);
}

// Slot of row `in_page` of the page that a table or free-list entry names.  No
// pool has a page whose slots pass 31 bits, or a negative one: kBadSlot stands
// for their rows, which lies in no pool either and is not the padding mark.
constexpr int32_t kBadSlot = -2147483647 - 1;
Q8_HD int32_t q8_slot(int32_t entry, uint32_t in_page, int page_shift) {
  return (uint32_t)entry <= 0x7fffffffu >> page_shift ? (int32_t)((uint32_t)entry << page_shift | in_page) : kBadSlot;
}

// Row of kv head h at row `in_page` of `page`: below num_pages Hkv P < 2^31.
Q8_HD uint32_t q8_row(uint32_t page, uint32_t in_page, uint32_t h, uint32_t Hkv, int page_shift) {
  return ((page * Hkv + h) << page_shift) + in_page;
}

// Last b with pre[b] <= x, for pre[0] = 0 <= x < pre[n]: of requests that
// share a first element, the one that is not empty.
Q8_HD int q8_owner(const int* pre, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// ceil(n num / den), 0 <= n, num, den <= 2^20, by den's 64-bit reciprocal
// inv = floor((2^64 - 1) / den) + 1: inv exceeds 2^64 / den by at most 1, so the
// product is off by less than x / 2^64 < 2^-23, which is less than 1 / den
// (x < 2^41).  A 64-bit quotient would cost a kernel's first load hundreds of
// cycles.
Q8_HD uint64_t q8_reciprocal(uint32_t den) { return ~(uint64_t)0 / den + 1; }
Q8_HD int32_t q8_count(int32_t n, uint32_t num, uint32_t den, uint64_t inv) {
  const uint64_t x = (uint64_t)n * num + (den - 1);
  if (den == 1) return (int32_t)x;
#if defined(__CUDA_ARCH__)
  return (int32_t)__umul64hi(x, inv);
#else
  return (int32_t)(((unsigned __int128)x * inv) >> 64);
#endif
}

// Exponent of a block's scale: the smallest e with amax <= top 2^e, top =
// 448 = 1.75 2^8 (e4m3) or 127 = 1.984375 2^6 (int8), from the bits of amax
// (finite, >= 0), held in [-100, 122] so that 2^e and 2^-e are normal.
// Powers of two make x / s exact, so a new row is rounded once, and a block
// whose scale grows keeps its e4m3 rows exactly unless they turn subnormal.
constexpr int kScaleMinExp = -100, kScaleMaxExp = 122;
Q8_HD int q8_scale_exp(uint32_t amax_bits, bool int8) {
  const uint32_t top_frac = int8 ? 0x7e0000u : 0x600000u;
  const int top_exp = int8 ? 6 : 8;
  const int e = (int)(amax_bits >> 23) - 127 - top_exp + ((amax_bits & 0x7fffffu) > top_frac ? 1 : 0);
  return e < kScaleMinExp ? kScaleMinExp : e > kScaleMaxExp ? kScaleMaxExp : e;
}

}  // namespace kascade
