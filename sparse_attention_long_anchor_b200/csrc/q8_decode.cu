// Attention of one query token over the 8-bit paged cache (Kascade README,
// Abstract: reuse layers attend over an anchor's Top-k indices, head-aware; a
// paged cache stores the same keys in pages): for each query head of problem
// (b, h), over the keys of its index list or over all keys of its row,
//   s_j = (q . k8_j) ks_j / sqrt(D),  p = softmax(s),  o = sum_j p_j vs_j v8_j,
// k8, v8 the stored bytes' values and ks, vs their blocks' scales.
//
// Bound by HBM: 2 D bytes per key and kv head against 4 G D flops.  So rows go
// straight from global memory into the registers of the 16x8x16 MMA (no trip
// through shared memory), each warp one slice of 16 keys ahead:
//   * S^T = K q^T: the contraction runs over the dims, so a lane may hold any
//     permutation of them as long as q has the same: lane (g, c) takes dims
//     [64 s + 16 c, +16) of keys g and g + 8, one 16-byte load each, whose
//     byte pairs are the MMA's operand pairs once widened;
//   * O^T += V^T P^T: the dims are the rows of the product, which may be
//     permuted too: lane (g, c) takes dims [g D/8, +D/8) of keys 2c, 2c + 1,
//     2c + 8, 2c + 9; a byte permute pairs two keys of one dim.
// Bytes widen to fp16, which holds every e4m3 and int8 value exactly.  The two
// other operands are brought into fp16's range without giving up bits:
//   * q is scaled per head by a power of two to a largest magnitude in
//     [2^14, 2^15); bf16's 8 bits (fp16's 11) then stay exact down to 2^-28
//     (2^-25) of that magnitude, smaller ones lose at most 2^-40 of it;
//   * p vs (p <= 1) is scaled by 2^(14 - E), E the largest exponent of vs that
//     the warp has met (the accumulators are rescaled when it grows, as they
//     are for the running maximum), and rounds to fp16: 2^-12 relative.
// Scores, softmax statistics and accumulators are fp32.
//
// A CTA takes `per` keys of one problem and merges its warps in shared
// memory; with more than one split per problem the partials (max, sum, fp32
// output) go to the workspace and a second kernel, launched to overlap, joins
// them.  No atomics: results do not depend on the order of the CTAs.
#include <type_traits>

#include "kernels.h"
#include "q8.cuh"

namespace kascade {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kCtasPerSM = 3;
constexpr int kStage = 1024;   // row numbers staged in shared memory at a time
constexpr int kPlanSMs = 148;

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint2 ldg_nc_v2(const void* p) {
  uint2 r;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];\n" : "=r"(r.x), "=r"(r.y) : "l"(p));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// weight of a partial result with running maximum m when joined at M
__device__ __forceinline__ float join_weight(float m, float M) { return m == -INFINITY ? 0.0f : exp2f(m - M); }

// one slice's rows in registers: K chunks of keys g and g + 8, V chunks of
// keys 2c, 2c + 1, 2c + 8, 2c + 9, and the scales of keys g and g + 8
template <int D>
struct Slice {
  uint32_t k[2][D / 64][4];
  uint32_t v[4][D / 32];
  float2 s0, s1;
};

template <int D, int QT, int CT>
__global__ void __launch_bounds__(kThreads, kCtasPerSM) q8_decode_kernel(const Q8DecodeArgs a) {
  constexpr int KQ = D / 64;        // 16-byte K loads per lane and key
  constexpr int VW = D / 32;        // 4-byte words of V per lane and key
  constexpr int MT = D / 16;        // MMA row tiles of O^T
  constexpr int RO = D + 4;         // padded row of the warps' outputs
  __shared__ uint32_t rows[kStage];
  __shared__ float red_o[kWarps][8][RO];
  __shared__ float2 red_ml[kWarps][8];
  __shared__ float red_e[kWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int prob = blockIdx.x / a.splits, split = blockIdx.x - prob * a.splits;
  const int b = prob / a.Hp, h = prob - b * a.Hp;
  const int G = a.G;

  // the problem's keys: an index list (of another head's problem, by the
  // map; an entry out of range is an empty list) or all keys of the row
  const int hm_raw = a.one_list ? 0 : (a.idx && a.head_map ? __ldg(a.head_map + h) : h);
  const bool hm_ok = hm_raw >= 0 && (a.idx == nullptr || hm_raw < a.n_lists);
  const int n_b = a.kv_lens ? min(max(__ldg(a.kv_lens + b), 0), a.N) : a.N;
  const int count = hm_ok ? (a.idx ? topk_count(n_b, a.num, a.den) : n_b) : 0;
  const int c0 = min(count, split * a.per), c1 = min(count, c0 + a.per);
  if (c0 >= c1 && split > 0) return;   // the join counts the splits of a problem the same way
  const int32_t* list =
      a.idx ? a.idx + (size_t)(b * a.n_lists + (hm_ok ? hm_raw : 0)) * topk_count(a.N, a.num, a.den) : nullptr;
  const int kvh = (h * G) / a.Gkv;
  const int32_t* ptab = a.page_table + (size_t)b * a.max_pages;
  const int ps = a.c.page_shift, bs = a.c.block_shift;

  // row numbers of keys [base, base + n) of this split; a slice's tail repeats the last key
  auto stage = [&](int base, int n) {
    const int n16 = (n + 15) & ~15;
    for (int i = tid; i < n16; i += kThreads) {
      int key = base + min(i, n - 1);
      bool bad = false;
      if (list) {
        key = q8_key(__ldg(list + key), n_b, bad);
        if (bad) raise_error(a.err, kErrIndexRange);
        bad = false;
      }
      const uint32_t pg = q8_page(__ldg(ptab + (key >> ps)), a.c.num_pages, bad);
      if (bad) raise_error(a.err, kErrPage);
      rows[i] = q8_row(pg, (uint32_t)key & ((1u << ps) - 1u), kvh, a.c.Hkv, ps);
    }
  };

  // q: B operand of S^T, head g's dims [64 s + 16 c, +16), scaled into fp16
  uint32_t qf[KQ][4][2];
  float sc0, sc1;   // score scale of heads 2c and 2c + 1: log2(e) / sqrt(D) and q's power of two
  {
    float x[KQ][16];
    uint32_t am = 0;
#pragma unroll
    for (int s = 0; s < KQ; ++s) {
      uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (g < G) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                        (size_t)(b * a.Hq + h * G + g) * D + 64 * s + 16 * c);
        const uint4 u = p[0], v = p[1];
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w, w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (QT == kInBf16) {
          x[s][2 * i] = bf16_lo(w[i]);
          x[s][2 * i + 1] = bf16_hi(w[i]);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
          x[s][2 * i] = f.x;
          x[s][2 * i + 1] = f.y;
        }
        am = max(am, max(__float_as_uint(x[s][2 * i]) & 0x7fffffffu, __float_as_uint(x[s][2 * i + 1]) & 0x7fffffffu));
      }
    }
    am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
    am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
    // exponent of the head's largest magnitude, brought to 14 (an infinity or
    // NaN stays one; magnitudes under 2^-100 are left to fp16's own range)
    const int e = min(max((int)(am >> 23) - 127, -100), 127);
    const float up = pow2f(14 - e);
#pragma unroll
    for (int s = 0; s < KQ; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        qf[s][i][0] = pack_f16(x[s][4 * i] * up, x[s][4 * i + 1] * up);
        qf[s][i][1] = pack_f16(x[s][4 * i + 2] * up, x[s][4 * i + 3] * up);
      }
    const float mine = kLog2e * rsqrtf((float)D) * pow2f(e - 14);
    sc0 = __shfl_sync(0xffffffffu, mine, 8 * c);       // lane (2c, 0)
    sc1 = __shfl_sync(0xffffffffu, mine, 8 * c + 4);   // lane (2c + 1, 0)
  }

  auto load = [&](Slice<D>& t, int sl) {
    const uint32_t* r = rows + sl * 16;
    const uint32_t r0 = r[g], r1 = r[g + 8];
#pragma unroll
    for (int s = 0; s < KQ; ++s) {
      const uint4 x = ldg_nc_v4(a.c.k + (size_t)r0 * D + 64 * s + 16 * c);
      const uint4 y = ldg_nc_v4(a.c.k + (size_t)r1 * D + 64 * s + 16 * c);
      t.k[0][s][0] = x.x, t.k[0][s][1] = x.y, t.k[0][s][2] = x.z, t.k[0][s][3] = x.w;
      t.k[1][s][0] = y.x, t.k[1][s][1] = y.y, t.k[1][s][2] = y.z, t.k[1][s][3] = y.w;
    }
    t.s0 = __ldg(a.c.scales + (r0 >> bs));
    t.s1 = __ldg(a.c.scales + (r1 >> bs));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t rv = r[2 * c + (j & 1) + 4 * (j & 2)];
      if constexpr (D == 128) {
        const uint4 x = ldg_nc_v4(a.c.v + (size_t)rv * D + 16 * g);
        t.v[j][0] = x.x, t.v[j][1] = x.y, t.v[j][VW - 2] = x.z, t.v[j][VW - 1] = x.w;
      } else {
        const uint2 x = ldg_nc_v2(a.c.v + (size_t)rv * D + 8 * g);
        t.v[j][0] = x.x, t.v[j][1] = x.y;
      }
    }
  };

  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;   // heads 2c, 2c + 1; sums over this lane's keys
  int e_run = 27;                                             // biased exponent E of the V scales met so far
  float oacc[MT][4];   // tile t: dim g D/8 + 2t of heads 2c, 2c + 1, then dim g D/8 + 2t + 1
#pragma unroll
  for (int t = 0; t < MT; ++t) oacc[t][0] = oacc[t][1] = oacc[t][2] = oacc[t][3] = 0.f;

  auto step = [&](const Slice<D>& t, int k0) {   // keys [k0, k0 + 16), those past c1 masked
    float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < KQ; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t a0, a1, a2, a3;
        q8_to_f16<CT>(t.k[0][s][i], a0, a2);
        q8_to_f16<CT>(t.k[1][s][i], a1, a3);
        mma_f16_16816(i & 1 ? sb : sa, a0, a1, a2, a3, qf[s][i][0], qf[s][i][1]);
      }
    const bool in0 = k0 + g < c1, in1 = k0 + g + 8 < c1;
    const float x0 = in0 ? (sa[0] + sb[0]) * (sc0 * t.s0.x) : -INFINITY;   // key g, head 2c
    const float x1 = in0 ? (sa[1] + sb[1]) * (sc1 * t.s0.x) : -INFINITY;   // key g, head 2c + 1
    const float x2 = in1 ? (sa[2] + sb[2]) * (sc0 * t.s1.x) : -INFINITY;   // key g + 8
    const float x3 = in1 ? (sa[3] + sb[3]) * (sc1 * t.s1.x) : -INFINITY;
    float n0 = fmaxf(x0, x2), n1 = fmaxf(x1, x3);
    // (a slice's tail repeats a key that is attended, so its scale may count too)
    const uint32_t vm = __reduce_max_sync(0xffffffffu, max(__float_as_uint(t.s0.y) & 0x7fffffffu,
                                                           __float_as_uint(t.s1.y) & 0x7fffffffu));
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, o));
      n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, o));
    }
    n0 = fmaxf(n0, m0);
    n1 = fmaxf(n1, m1);
    const int e_new = max(e_run, (int)(vm >> 23));
    float al0 = join_weight(m0, n0), al1 = join_weight(m1, n1);
    const float p0 = exp2f(x0 - n0), p1 = exp2f(x1 - n1), p2 = exp2f(x2 - n0), p3 = exp2f(x3 - n1);
    l0 = l0 * al0 + (p0 + p2);
    l1 = l1 * al1 + (p1 + p3);
    m0 = n0;
    m1 = n1;
    const float f = e_run == e_new ? 1.0f : pow2f(max(e_run - e_new, -126));
    al0 *= f;
    al1 *= f;
    e_run = e_new;
    const float ve = __uint_as_float((uint32_t)(268 - e_new) << 23);   // 2^(14 - E)
    const float v0 = t.s0.y * ve, v1 = t.s1.y * ve;
    // P^T (keys x heads) from accumulator to operand layout
    const uint32_t b0 = movmatrix_trans(pack_f16(p0 * v0, p1 * v0));
    const uint32_t b1 = movmatrix_trans(pack_f16(p2 * v1, p3 * v1));
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      // word i / 2 of each key's chunk holds dims 4 (i / 2) .. + 3 of the lane's
      const uint32_t sel = i & 1 ? 0x7362 : 0x5140;
      uint32_t a0, a1, a2, a3;
      q8_to_f16<CT>(__byte_perm(t.v[0][i >> 1], t.v[1][i >> 1], sel), a0, a1);
      q8_to_f16<CT>(__byte_perm(t.v[2][i >> 1], t.v[3][i >> 1], sel), a2, a3);
      float d[4] = {oacc[i][0] * al0, oacc[i][1] * al1, oacc[i][2] * al0, oacc[i][3] * al1};
      mma_f16_16816(d, a0, a1, a2, a3, b0, b1);
      oacc[i][0] = d[0], oacc[i][1] = d[1], oacc[i][2] = d[2], oacc[i][3] = d[3];
    }
  };

  for (int base = c0; base < c1; base += kStage) {
    const int n = min(kStage, c1 - base);
    if (base > c0) __syncthreads();   // the rows before are no longer read
    stage(base, n);
    __syncthreads();
    const int slices = (n + 15) >> 4;
    Slice<D> t0, t1;
    if (warp < slices) load(t0, warp);
    for (int sl = warp; sl < slices; sl += 2 * kWarps) {
      if (sl + kWarps < slices) load(t1, sl + kWarps);
      step(t0, base + sl * 16);
      if (sl + 2 * kWarps < slices) load(t0, sl + 2 * kWarps);
      if (sl + kWarps < slices) step(t1, base + (sl + kWarps) * 16);
    }
  }

  // ---- join the warps
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, o);
    l1 += __shfl_xor_sync(0xffffffffu, l1, o);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float* ro = &red_o[warp][2 * c + j][g * (D / 8)];
#pragma unroll
    for (int t = 0; t < MT; ++t)
      *reinterpret_cast<float2*>(ro + 2 * t) = make_float2(oacc[t][j], oacc[t][2 + j]);
  }
  if (g == 0) {
    red_ml[warp][2 * c] = make_float2(m0, l0);
    red_ml[warp][2 * c + 1] = make_float2(m1, l1);
  }
  if (lane == 0) red_e[warp] = __uint_as_float((uint32_t)max(e_run - 14, 0) << 23);   // 2^(E - 14)
  __syncthreads();
  constexpr int Q4 = D / 4;
  for (int i = tid; i < G * Q4; i += kThreads) {
    const int hh = i / Q4, d4 = (i - hh * Q4) * 4;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red_ml[w][hh].x);
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = red_ml[w][hh];
      const float f = join_weight(ml.x, M);
      l += f * ml.y;
      const float fe = f * red_e[w];
      const float4 x = *reinterpret_cast<const float4*>(&red_o[w][hh][d4]);
      acc.x += fe * x.x, acc.y += fe * x.y, acc.z += fe * x.z, acc.w += fe * x.w;
    }
    const size_t orow = (size_t)b * a.Hq + h * G + hh;
    if (a.splits > 1) {
      const size_t pr = ((size_t)prob * a.splits + split) * G + hh;
      *reinterpret_cast<float4*>(a.part_o + pr * D + d4) = acc;
      if (d4 == 0) a.part_ml[pr] = make_float2(M, l);
    } else {
      const float inv = l == 0.f ? 0.f : 1.0f / l;   // no key: zero
      uint32_t lo, hi;
      if constexpr (QT == kInBf16) {
        lo = pack_bf16(acc.x * inv, acc.y * inv), hi = pack_bf16(acc.z * inv, acc.w * inv);
      } else {
        lo = pack_f16(acc.x * inv, acc.y * inv), hi = pack_f16(acc.z * inv, acc.w * inv);
      }
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + orow * D + d4) = make_uint2(lo, hi);
      if (d4 == 0 && a.lse) a.lse[orow] = l == 0.f ? -INFINITY : (M + log2f(l)) * (float)kLn2;
    }
  }
}

// Joins the splits of one (problem, head): CTA = one row of o.
constexpr int kJoinThreads = 128;

template <int D, int QT>
__global__ void __launch_bounds__(kJoinThreads) q8_join_kernel(const Q8DecodeArgs a) {
  constexpr int Q4 = D / 4, GROUPS = kJoinThreads / Q4;   // lanes per row, splits side by side
  __shared__ float4 acc_s[GROUPS][Q4];
  __shared__ float red[kJoinThreads / 32][2];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int prob = blockIdx.x / a.G, hh = blockIdx.x - prob * a.G;
  const int b = prob / a.Hp, h = prob - b * a.Hp;
  const int hm = a.one_list ? 0 : (a.idx && a.head_map ? __ldg(a.head_map + h) : h);
  const bool hm_ok = hm >= 0 && (a.idx == nullptr || hm < a.n_lists);
  const int n_b = a.kv_lens ? min(max(__ldg(a.kv_lens + b), 0), a.N) : a.N;
  const int count = hm_ok ? (a.idx ? topk_count(n_b, a.num, a.den) : n_b) : 0;
  const int n = max(1, (count + a.per - 1) / a.per);   // split 0 always writes
  const size_t p0 = (size_t)prob * a.splits * a.G + hh;
  float M = -INFINITY;
  for (int s = tid; s < n; s += kJoinThreads) M = fmaxf(M, a.part_ml[p0 + (size_t)s * a.G].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) red[warp][0] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) M = fmaxf(M, red[w][0]);
  float l = 0.f;
  for (int s = tid; s < n; s += kJoinThreads) {
    const float2 ml = a.part_ml[p0 + (size_t)s * a.G];
    l += join_weight(ml.x, M) * ml.y;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane == 0) red[warp][1] = l;
  const int grp = tid / Q4, d4 = (tid - grp * Q4) * 4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = grp; s < n; s += GROUPS) {
    const size_t pr = p0 + (size_t)s * a.G;
    const float f = join_weight(a.part_ml[pr].x, M);
    const float4 x = *reinterpret_cast<const float4*>(a.part_o + pr * D + d4);
    acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
  }
  acc_s[grp][d4 / 4] = acc;
  __syncthreads();
  if (grp != 0) return;
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) l += red[w][1];
#pragma unroll
  for (int r = 1; r < GROUPS; ++r) {
    const float4 x = acc_s[r][d4 / 4];
    acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  uint32_t lo, hi;
  if constexpr (QT == kInBf16) {
    lo = pack_bf16(acc.x * inv, acc.y * inv), hi = pack_bf16(acc.z * inv, acc.w * inv);
  } else {
    lo = pack_f16(acc.x * inv, acc.y * inv), hi = pack_f16(acc.z * inv, acc.w * inv);
  }
  const size_t orow = (size_t)b * a.Hq + h * a.G + hh;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + orow * D + d4) = make_uint2(lo, hi);
  if (d4 == 0 && a.lse) a.lse[orow] = l == 0.f ? -INFINITY : (M + log2f(l)) * (float)kLn2;
}

template <int D, int QT, int CT>
cudaError_t run(const Q8DecodeArgs& a, cudaStream_t st) {
  const int64_t problems = (int64_t)a.B * a.Hp;
  cudaError_t e = launch_ex(q8_decode_kernel<D, QT, CT>, dim3((unsigned)(problems * a.splits)), dim3(kThreads), 0, st,
                            (a.flags & 1) != 0, 1, a);
  if (e != cudaSuccess || a.splits == 1) return e;
  // the join waits for the kernel above before it reads anything, so it may always be launched early
  return launch_ex(q8_join_kernel<D, QT>, dim3((unsigned)(problems * a.G)), dim3(kJoinThreads), 0, st, true, 1, a);
}

template <int D, int QT>
cudaError_t run_ct(const Q8DecodeArgs& a, int cache_type, cudaStream_t st) {
  return cache_type == kInt8 ? run<D, QT, kInt8>(a, st) : run<D, QT, kE4M3>(a, st);
}

}  // namespace

void q8_decode_plan(int64_t problems, int count, int* per, int* splits) {
  const int64_t slots = (int64_t)kPlanSMs * kCtasPerSM;
  int64_t want = slots / problems;                       // splits that fit one wave
  if (want < 1) want = 1;
  int64_t p = (count + want - 1) / want;
  const int64_t unit = 16 * kWarps;                      // a slice for every warp
  p = (p + unit - 1) / unit * unit;
  if (p < unit) p = unit;
  if (p > 1024) p = 1024;
  *per = (int)p;
  *splits = (int)((count + p - 1) / p);
  if (*splits < 1) *splits = 1;
}

cudaError_t launch_q8_decode(const Q8DecodeArgs& a, int in_type, int cache_type, cudaStream_t stream) {
  if (a.c.D == 128)
    return in_type == kInF16 ? run_ct<128, kInF16>(a, cache_type, stream) : run_ct<128, kInBf16>(a, cache_type, stream);
  return in_type == kInF16 ? run_ct<64, kInF16>(a, cache_type, stream) : run_ct<64, kInBf16>(a, cache_type, stream);
}

}  // namespace kascade
