// The 8-bit paged KV cache: layout, element conversions and the argument
// blocks of its kernels (q8_cache.cu, q8_decode.cu).
//
// Pages are [num_pages, Hkv, P, D] bytes for K and for V, and scales
// [num_pages, Hkv, P / S] float2 (K scale, V scale): one pair per S consecutive
// rows of a page and kv head.  Row r = (page Hkv + h) P + slot starts at byte
// r D and takes scale pair r / S.  A byte stands for its e4m3 or int8 value
// times its scale.  Rows and slots fit 31 bits (checked on the host); byte
// offsets are 64-bit.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "q8_index.h"

namespace kascade {

constexpr int kErrIndexRange = 7;   // device error word: a list entry outside its row's keys
constexpr int kErrPage = 8;         // device error word: a slot or page-table entry outside the page pool

enum : int { kE4M3 = 0, kInt8 = 1 };        // cache element types
enum : int { kInBf16 = 0, kInF32 = 1, kInF16 = 2 };   // element types of q, k, v, o (KASCADE_DTYPE_*)

struct Q8Cache {
  uint8_t* k;
  uint8_t* v;
  float2* scales;
  int num_pages, Hkv, D;
  int page_shift, block_shift;   // P = 1 << page_shift, S = 1 << block_shift
};

// a packed pair of 8-bit values (bits 0-15 or 16-31 of w) as exact fp16 pairs
template <int CT>
__device__ __forceinline__ void q8_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (CT == kE4M3) {
    // every e4m3 value is an fp16 value; the conversion is one instruction
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // x + 128 in the low bits of fp16 1024 (spacing 1 there), less 1152
    const uint32_t u = w ^ 0x80808080u;
    const __half2 c = __half2half2(__ushort_as_half((unsigned short)0x6480));   // 1152
    uint32_t p = __byte_perm(u, 0x64646464u, 0x4140), r = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 a = __hsub2(*reinterpret_cast<__half2*>(&p), c), b = __hsub2(*reinterpret_cast<__half2*>(&r), c);
    lo = *reinterpret_cast<uint32_t*>(&a);
    hi = *reinterpret_cast<uint32_t*>(&b);
  }
}

// four values to bytes: round to nearest even, saturated to the type's
// largest magnitude (infinities too); NaN is e4m3's NaN and int8's 0
template <int CT>
__device__ __forceinline__ uint32_t q8_pack4(float a, float b, float c, float d) {
  if constexpr (CT == kE4M3) {
    uint32_t r;
    asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n"
        " mov.b32 %0, {l, h};\n}\n"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
  } else {
    auto one = [](float x) -> uint32_t {
      const int i = x == x ? __float2int_rn(fminf(fmaxf(x, -127.f), 127.f)) : 0;
      return (uint32_t)i & 0xffu;
    };
    return one(a) | (one(b) << 8) | (one(c) << 16) | (one(d) << 24);
  }
}

// 2^e as a float, -126 <= e <= 127
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// ---------------------------------------------------------------------------
// kernel arguments

struct PageTablesArgs {
  const int32_t* kv_lens;      // [B] tokens held
  const int32_t* new_lens;     // [B] tokens to add
  const int32_t* free_pages;   // [num_free]
  int32_t* page_table;         // [B, max_pages], entries of new pages written
  int32_t* lens_out;           // [B]
  int32_t* offsets;            // [B + 1]
  int32_t* slot_map;           // [capacity]
  int32_t* info;               // (pages taken or -1, tokens)
  int B, page_shift, max_pages, num_free, capacity;
};
cudaError_t launch_page_tables(const PageTablesArgs& a, cudaStream_t stream);

struct Q8AppendArgs {
  Q8Cache c;
  const void* k;
  const void* v;
  int64_t k_token, k_head, v_token, v_head;   // strides in elements
  const int32_t* slots;
  int T;
  int* err;
};
cudaError_t launch_q8_append(const Q8AppendArgs& a, int in_type, int cache_type, cudaStream_t stream);

struct Q8GatherArgs {
  Q8Cache c;
  const int32_t* page_table;   // [B, max_pages]
  const int32_t* kv_lens;      // [B] or NULL: N
  void* k;                     // [B, Hkv, N, D], either may be NULL
  void* v;
  int B, N, max_pages;
  int* err;
};
cudaError_t launch_q8_gather(const Q8GatherArgs& a, int out_type, int cache_type, cudaStream_t stream);

struct Q8DecodeArgs {
  Q8Cache c;
  const void* q;
  const int32_t* page_table;
  const int32_t* kv_lens;      // NULL: N
  const int32_t* idx;          // NULL: dense
  const int32_t* head_map;
  void* o;
  float* lse;                  // may be NULL
  float2* part_ml;             // [part, G] (max, sum)
  float* part_o;               // [part, G, D]
  int* share;                  // the tiles of a CTA that the lengths gave
  int* err;
  int B, Hq, Hp, G, Gkv, N, num, den, n_lists, max_pages;
  int stride;                  // entries of a list (dense: N)
  uint64_t den_inv;            // q8_reciprocal(den)
  bool one_list;
  int longest;                 // tiles of the longest list
  int ctas;                    // CTAs (not of clusters)
  int per;                     // tiles of a CTA, 0: found on the device (set at launch)
  int flags;
};
// The split of `problems` lists of up to `count` keys: tiles of the longest
// list, CTAs, and partial results (of G heads each) that they may leave; 0: a
// CTA per problem, and none.
struct Q8Plan {
  int longest;
  int64_t ctas, parts;
};
Q8Plan q8_decode_plan(int64_t problems, int count);
cudaError_t launch_q8_decode(const Q8DecodeArgs& a, int in_type, int cache_type, cudaStream_t stream);

}  // namespace kascade
