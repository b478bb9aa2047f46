// Attention of one query token over the 8-bit paged cache (Kascade README,
// Abstract: reuse layers attend over an anchor's Top-k indices, head-aware; a
// paged cache stores the same keys in pages): for each query head of problem
// (b, h), over the keys of its index list or over all keys of its row,
//   s_j = (q . k8_j) ks_j / sqrt(D),  p = softmax(s),  o = sum_j p_j vs_j v8_j,
// k8, v8 the stored bytes' values and ks, vs their blocks' scales.
//
// Bound by HBM: 2 D bytes per key and kv head against 4 G D flops.  Every warp
// works alone on tiles of 16 keys, whose rows travel by cp.async into a ring of
// kStages stages of its own (no barrier between warps, copies of two tiles
// under way while one is computed), and feeds the 16x8x16 MMA from there:
//   * S^T = K q^T: the contraction runs over the dims, so a lane may hold any
//     permutation of them as long as q has the same: lane (g, c) takes 16-byte
//     chunks of keys g and g + 8 (D = 128: chunks 2c and 2c + 1 of the row's
//     eight; D = 64: chunk c of four), whose byte pairs are the MMA's operand
//     pairs once widened;
//   * O^T += V^T P^T: the dims are the rows of the product, which may be
//     permuted too: lane (g, c) takes dims [g D/8, +D/8) of keys 2c, 2c + 1,
//     2c + 8, 2c + 9; a byte permute pairs two keys of one dim.
// Rows are stored with their chunks swizzled so that both kinds of read are
// free of bank conflicts (see chunk_at).
// Bytes widen to fp16, which holds every e4m3 and int8 value exactly.  The two
// other operands are brought into fp16's range without giving up bits:
//   * q is scaled per head by a power of two to a largest magnitude in
//     [2^14, 2^15); bf16's 8 bits (fp16's 11) then stay exact down to 2^-31
//     (2^-28) of that magnitude, smaller ones lose at most half of fp16's
//     smallest step, 2^-25, which is 2^-39 of it;
//   * p vs (p <= 1) is scaled by 2^(14 - E), E the largest exponent of vs that
//     the warp has met (the accumulators are rescaled when it grows, as they
//     are for the running maximum), and rounds to fp16: by 2^-11 of itself, or,
//     where that is more (products below fp16's normal range), by 2^-25 in
//     units of 2^(E - 14).
// Scores, softmax statistics and accumulators are fp32.
//
// Three ways to split the work, by the problems' number and length (see run);
// in each, a CTA takes tiles of one problem:
//   * few short lists: a thread-block cluster per problem, whose CTAs take
//     `per` tiles each and push their partial results into one another's
//     shared memory (st.async on the receiver's mbarrier; the one wait is
//     bounded).  One launch, no workspace; latency is what counts there;
//   * longer lists, up to a quarter as many problems as CTAs are resident at
//     once: all tiles are cut into shares, as many CTAs to a problem as its
//     length asks for and all of them resident together (see find_share).  A
//     ragged batch is balanced that way whatever its lengths are, which only
//     the device knows;
//   * more problems: `per` tiles to a CTA, in several waves.  A share would be
//     most of a problem, and the longest would be waited for.
// The last two leave a partial result (max, sum, fp32 output) per CTA in the
// workspace where a problem has several, and a second kernel, launched to
// overlap, joins them.  The split depends on the lengths alone and there are
// no atomics: results do not depend on the order in which CTAs run.
#include <atomic>

#include "cluster_choice.h"
#include "kernels.h"
#include "q8.cuh"

namespace kascade {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCtasPerSM = 2;
constexpr int kPlanSMs = 148;
constexpr int kResident = kPlanSMs * kCtasPerSM;
constexpr int kTile = 16;     // keys of one step of a warp
constexpr int kStages = 3;    // tiles of a warp's ring
constexpr int kMaxCS = 16;    // largest cluster
constexpr int kErrMerge = 3;  // device error word: a peer CTA's partial result never arrived
constexpr uint32_t kNoRow = 0xffffffffu;

// A stage: 16 K rows, 16 V rows, 16 scale pairs.  Chunk ch (16 bytes) of row r
// lies in 128-byte line r (D = 128) or r / 2 (D = 64), at its place in the
// line XOR a number that changes from line to line: the eight lanes that a
// 16-byte read serves at once (rows g, g + 1 with four chunks of K; four rows
// 2c + j with chunks g, g + 1 of V) and the sixteen of an 8-byte read (D = 64:
// four rows, two chunks of V) then fall on different banks.
template <int D>
struct Stage {
  static constexpr int TB = 16 * D;            // bytes of 16 rows
  static constexpr int K = 0, V = TB, S = 2 * TB;
  static constexpr int BYTES = 2 * TB + 16 * 8;
};
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int ch) {
  if constexpr (D == 128) return (uint32_t)(r * 128 + ((ch ^ (r & 7)) << 4));
  return (uint32_t)((r >> 1) * 128 + ((((r & 1) * 4 + ch) ^ (2 * ((r >> 1) & 3))) << 4));
}

// From the place of a chunk in row r to that of the same chunk in row r + 1 (r
// even), and in row r + n (n a multiple of 4; D = 64: of 8).
template <int D>
__device__ __forceinline__ uint32_t next_row(uint32_t at) {
  return D == 128 ? (at + 128) ^ 16 : at ^ 64;
}
template <int D>
__device__ __forceinline__ uint32_t row_step(uint32_t at, int n) {
  return D == 128 && (n & 4) ? ((at + n * D) ^ 64) : at + n * D;
}

// shared memory: the rings [kWarps][kStages]; after the tiles each warp's ring
// holds its output for the join of the warps
template <int D>
struct Smem {
  static constexpr int RO = D + 4;             // padded row of a warp's output (floats)
  static constexpr size_t WARPB = (size_t)kStages * Stage<D>::BYTES;
  static constexpr size_t ml = kWarps * WARPB; // [kWarps][8] (max, sum)
  static constexpr size_t e = ml + kWarps * 8 * 8;             // [kWarps] 2^(E - 14)
  // clusters: written by the CTAs of the cluster, slot r by CTA r
  static constexpr size_t recv_ml = e + kWarps * 4;            // [kMaxCS][8] (max, sum)
  static constexpr size_t recv_o = recv_ml + kMaxCS * 8 * 8;   // [cluster size][units of 4 outputs]
  static constexpr size_t q = recv_o + (8 * D / 4 + kMaxCS) * 16;   // [D / 32][32 lanes] uint4: the q operand
  static constexpr size_t bar = q + D / 32 * 32 * 16;
  static constexpr size_t total = bar + 8;
  static_assert(8 * RO * 4 <= WARPB && WARPB % 16 == 0, "a warp's output fits its ring");
  static_assert(recv_ml % 16 == 0 && recv_o % 16 == 0 && q % 16 == 0 && bar % 8 == 0, "alignment");
  static_assert(total <= (228 * 1024 - kCtasPerSM * 1024) / kCtasPerSM, "CTAs per SM");
};

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint2 lds_v2(uint32_t addr) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];\n" : "=r"(r.x), "=r"(r.y) : "r"(addr));
  return r;
}
__device__ __forceinline__ void cp_async_8(uint32_t dst, const void* src, int src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(dst), "l"(src), "r"(src_bytes));
}
__device__ __forceinline__ int cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;\n" : "=r"(r));
  return (int)r;
}
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctaid.x;\n" : "=r"(r));
  return (int)r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A running maximum starts at kNoScore, so that scores of minus infinity weigh
// ex2(-inf) = 0 whatever comes before them; it is -inf where there was no key.
constexpr float kNoScore = -3.402823466e+38f;   // fp32's lowest
// weight of a partial result with running maximum m when joined at M
__device__ __forceinline__ float join_weight(float m, float M) { return m == -INFINITY ? 0.0f : ex2_fast(m - M); }

// (Inputs are read by plain loads, not through the read-only path: under
// programmatic dependent launch another kernel may write them while this one
// is already running, up to its wait.)
// keys that batch row b's problems attend over, and their tiles
__device__ __forceinline__ int row_keys(const Q8DecodeArgs& a, int b) {
  return a.kv_lens ? min(max(a.kv_lens[b], 0), a.N) : a.N;
}
__device__ __forceinline__ int row_count(const Q8DecodeArgs& a, int n) {
  return a.idx ? q8_count(n, a.num, a.den, a.den_inv) : n;
}
__device__ __forceinline__ int row_tiles(const Q8DecodeArgs& a, int b) {
  return (row_count(a, row_keys(a, b)) + kTile - 1) / kTile;
}
__device__ __forceinline__ int warp_inclusive_scan(int x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Shares.  With S tiles to a CTA, row b's problems have ceil(T_b / S) CTAs
// each; S is the smallest (within the search) at which all of them are at most
// a.ctas, which S = total / (ctas - problems) is in any case.  Each warp counts
// for itself, 32 rows at a time: cheaper than a barrier for the batches there
// are.  mine: this lane's row's tiles, of the first 32 rows.
__device__ __forceinline__ int ceil_div(int x, int y) { return (x + y - 1) / y; }
__device__ __forceinline__ int first_rows(const Q8DecodeArgs& a) {
  const int lane = threadIdx.x & 31;
  return lane < a.B ? row_tiles(a, lane) : 0;
}
// sum over the rows [0, end) of f(tiles of the row)
template <class F>
__device__ __forceinline__ int sum_rows(const Q8DecodeArgs& a, int mine, int end, F&& f) {
  const int lane = threadIdx.x & 31;
  int s = lane < end ? f(mine) : 0;
  for (int x = lane + 32; x < end; x += 32) s += f(row_tiles(a, x));
  return __reduce_add_sync(0xffffffffu, s);
}
constexpr int kSearch = 6;   // halvings of the interval in which S is sought
__device__ __forceinline__ int find_share(const Q8DecodeArgs& a, int mine) {
  if (!a.kv_lens) {
    // equal rows: as many CTAs to a problem as there are for each
    return max(ceil_div(row_tiles(a, 0), max(a.ctas / (a.B * a.Hp), 1)), kWarps);
  }
  const int tiles = sum_rows(a, mine, a.B, [](int t) { return t; });
  const int64_t total = (int64_t)tiles * a.Hp;
  const int spare = a.ctas - a.B * a.Hp;
  int hi = spare > 0 ? (int)min((total + spare - 1) / spare, (int64_t)a.longest) : a.longest;
  int lo = (int)((total + a.ctas - 1) / a.ctas);
  lo = max(lo, kWarps);
  hi = max(hi, lo);
  for (int i = 0; i < kSearch && lo < hi; ++i) {
    const int s = i == 0 ? lo : (lo + hi) >> 1;
    const int n = sum_rows(a, mine, a.B, [&](int t) { return ceil_div(t, s); });
    if ((int64_t)n * a.Hp <= a.ctas) hi = s;
    else lo = s + 1;
  }
  return hi;
}
// The problem and the part of it that CTA `cta` has: false if none.
struct Part {
  int b, h, part;
};
__device__ __forceinline__ bool part_of_cta(const Q8DecodeArgs& a, int mine, int share, int cta, Part& r) {
  if (!a.kv_lens) {
    const int n = ceil_div(row_tiles(a, 0), share), prob = cta / n;
    r.b = prob / a.Hp;
    r.h = prob - r.b * a.Hp;
    r.part = cta - prob * n;
    return prob < a.B * a.Hp;
  }
  const int lane = threadIdx.x & 31;
  int base = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int t = b0 == 0 ? mine : b0 + lane < a.B ? row_tiles(a, b0 + lane) : 0;
    const int n = ceil_div(t, share);
    const int incl = base + warp_inclusive_scan(n * a.Hp);
    const uint32_t past = __ballot_sync(0xffffffffu, incl > cta);
    if (past) {   // the first row that ends behind this CTA
      const int l = __ffs(past) - 1;
      const int each = __shfl_sync(0xffffffffu, n, l), off = cta - (__shfl_sync(0xffffffffu, incl, l) - each * a.Hp);
      r.b = b0 + l;
      r.h = off / each;
      r.part = off - r.h * each;
      return true;
    }
    base = __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

// four consecutive outputs, normalised and rounded once
template <int QT>
__device__ __forceinline__ void store_out(const Q8DecodeArgs& a, size_t at, float4 x, float M, float l) {
  const float inv = M == -INFINITY ? 0.f : 1.0f / l;   // no key: zero (none but weights of zero: 0 / 0)
  uint32_t lo, hi;
  if constexpr (QT == kInBf16) {
    lo = pack_bf16(x.x * inv, x.y * inv), hi = pack_bf16(x.z * inv, x.w * inv);
  } else {
    lo = pack_f16(x.x * inv, x.y * inv), hi = pack_f16(x.z * inv, x.w * inv);
  }
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + at) = make_uint2(lo, hi);
}
__device__ __forceinline__ float lse_of(float M, float l) {
  return l == 0.f ? -INFINITY : (M + log2f(l)) * (float)kLn2;
}

// kCluster: blockIdx.x / (cluster size) is the problem
template <int D, int QT, int CT, bool kCluster>
__global__ void __launch_bounds__(kThreads, kCtasPerSM) q8_decode_kernel(const Q8DecodeArgs a) {
  using St = Stage<D>;
  using L = Smem<D>;
  constexpr int KQ = D / 64;        // 16-byte K chunks per lane and key
  constexpr int VW = D / 32;        // 4-byte words of V per lane and key
  constexpr int MT = D / 16;        // MMA row tiles of O^T
  constexpr int LPR = D / 16;       // lanes that copy a row (a chunk each)
  constexpr int RPC = 32 / LPR;     // rows per copy instruction
  extern __shared__ __align__(128) char smem[];
  float2* red_ml = reinterpret_cast<float2*>(smem + L::ml);
  float* red_e = reinterpret_cast<float*>(smem + L::e);
  // with inputs that the caller vouches for, everything up to the copies of
  // the first tiles comes before the wait for the previous kernel; what that
  // may have written (q) or still reads (the workspace, o) comes behind it
  const bool early = (a.flags & 3) == 3;
  if (!early) {
    pdl_wait();
    pdl_launch_dependents();
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int G = a.G;
  const int ps = a.c.page_shift, bs = a.c.block_shift;
  const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * L::WARPB);
  const uint8_t* kp = a.c.k + 16 * (lane % LPR);   // the chunk that this lane copies of each row
  const uint8_t* vp = a.c.v + 16 * (lane % LPR);

  // the head map's entries, a lane each: they do not wait for (b, h)
  const bool mapped = a.idx && a.head_map && !a.one_list;
  const int hm_lane = mapped && lane < a.Hp ? a.head_map[lane] : 0;
  const int stride = a.stride;   // entries of a list, -1 past a row's own (dense: N)
  // this CTA's tiles, from tile ta of problem (b, h) on
  int b, h, ta, per = a.per;
  [[maybe_unused]] int cs = 1, rank = 0, units = 0;   // clusters: outputs are owned in units of four
  [[maybe_unused]] const uint32_t bar = smem_u32(smem) + (uint32_t)L::bar;
  if constexpr (kCluster) {
    cs = cluster_size();
    rank = cluster_rank();
    const int prob = blockIdx.x / cs;
    b = prob / a.Hp;
    h = prob - b * a.Hp;
    ta = rank * per;
    if (cs > 1) {
      const int n = G * (D / 4);
      units = (n + cs - 1) / cs;
      if (tid == 0) {
        mbar_init(bar, 1);
        mbar_fence_init();
        // every CTA of the cluster sends this CTA's outputs and G (max, sum) pairs
        mbar_arrive_expect_tx(bar, (uint32_t)(cs * (max(0, min(units, n - rank * units)) * 16 + G * 8)));
      }
      cluster_arrive_release();   // the matching wait comes before the first push
    }
  } else {
    Part pt;
    if (per > 0) {
      const int n = ceil_div(a.longest, per), prob = blockIdx.x / n;
      pt.part = blockIdx.x - prob * n;
      pt.b = prob / a.Hp;
      pt.h = prob - pt.b * a.Hp;
    } else {
      const int mine = first_rows(a);
      per = find_share(a, mine);
      if (blockIdx.x == 0) {   // for the join
        if (early) pdl_wait();
        if (tid == 0) *a.share = per;
      }
      if (!part_of_cta(a, mine, per, blockIdx.x, pt)) {
        if (early) pdl_wait();   // (no kernel of ours is done before its predecessor)
        return;
      }
    }
    b = pt.b;
    h = pt.h;
    ta = pt.part * per;
  }

  // Loads that wait for nothing but (b, h) come first: each is a trip of its
  // own to L2 or HBM.  q's rows: the dims of the lane's K chunks for head g.
  uint4 qw[KQ][2];
  auto load_q = [&]() {
#pragma unroll
    for (int s = 0; s < KQ; ++s) {
      qw[s][0] = qw[s][1] = make_uint4(0, 0, 0, 0);
      if (g < G) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                        ((size_t)b * a.Hq + h * G + g) * D + 16 * (KQ * c + s));
        qw[s][0] = p[0];
        qw[s][1] = p[1];
      }
    }
  };
  if (!early) load_q();
  const int n_b = row_keys(a, b);
  // the problem's keys: an index list (of another head's problem, by the
  // map; an entry out of range is an empty list) or all keys of the row
  int hm = a.one_list ? 0 : h;
  if (mapped) hm = h < 32 ? __shfl_sync(0xffffffffu, hm_lane, h) : a.head_map[h];
  const bool hm_ok = hm >= 0 && (a.idx == nullptr || hm < a.n_lists);
  const int32_t* list = a.idx ? a.idx + ((size_t)b * a.n_lists + (hm_ok ? hm : 0)) * stride : nullptr;
  const int kvh = (h * G) / a.Gkv;
  const int32_t* ptab = a.page_table + (size_t)b * a.max_pages;

  // A lane finds the row of one key, for two of the warp's tiles at a time
  // (the pair's first by lanes 0-15): the list entries of a pair ahead of its
  // page-table entries, those ahead of the rows' copies.  Keys past the list
  // have no row: zeros are filled in for them and their scores masked.
  const int t0 = ta + warp;   // this warp's tiles: t0, t0 + kWarps, ...
  constexpr int kPairStep = 2 * kWarps * kTile;   // from a pair's keys to the next pair's
  const int place = (t0 + (lane >> 4) * kWarps) * kTile + (lane & 15);   // the lane's key of pair 0, in the list
  auto entry = [&](int k) -> int {
    k = min(k, stride - 1);
    return list ? list[k] : k;
  };
  // list entries of the first pairs; e_n is that of the pair whose pages are looked up next
  const int e0 = entry(place), e1 = entry(place + kPairStep);
  int e_n = entry(place + 2 * kPairStep), k_n = place + 2 * kPairStep;

  const int count_b = row_count(a, n_b);
  const int tiles_b = (count_b + kTile - 1) / kTile;
  if (!kCluster && ta >= tiles_b) {   // (a row without keys is the join's)
    if (early) pdl_wait();
    return;
  }
  const int tb = min(tiles_b, ta + per);    // tiles [ta, tb) of the problem
  const int t_end = hm_ok ? tb : ta;
  // Entries out of range are replaced and noted; reported once, at the end.
  bool bad_key = false, bad_page = false;
  auto key_of = [&](int k, int e) -> int {
    bool bad = false;
    const int key = q8_key(e, n_b, bad);
    bad_key |= bad && k < count_b;
    return key;
  };
  auto row_of = [&](int k, int key, int page) -> uint32_t {
    bool bad = false;
    const uint32_t pg = q8_page(page, a.c.num_pages, bad);
    bad_page |= bad && k < count_b;
    const uint32_t row = q8_row(pg, (uint32_t)key & ((1u << ps) - 1u), kvh, a.c.Hkv, ps);
    return k < count_b ? row : kNoRow;
  };
  // copies of a tile (the second of its pair: `odd`) into a stage of the ring
  const int whole_tiles = count_b / kTile;   // tiles without a masked tail
  const uint32_t copy0 = chunk_at<D>(lane / LPR, lane % LPR);
  const uint32_t copy_s = St::S + (lane & 15) * 8;
  auto issue = [&](uint32_t mine, int t, int odd, uint32_t st) {
    const int r0 = lane / LPR + 16 * odd;
    if (t < whole_tiles) {
#pragma unroll
      for (int i = 0; i < 16 / RPC; ++i) {
        const uint32_t row = __shfl_sync(0xffffffffu, mine, r0 + i * RPC);
        const uint32_t to = st + row_step<D>(copy0, i * RPC);
        cp_async_16(to + St::K, kp + (size_t)row * D, 16);
        cp_async_16(to + St::V, vp + (size_t)row * D, 16);
      }
      if ((lane >> 4) == odd) cp_async_8(st + copy_s, a.c.scales + (mine >> bs), 8);
    } else {
#pragma unroll 1
      for (int i = 0; i < 16 / RPC; ++i) {
        const uint32_t row = __shfl_sync(0xffffffffu, mine, r0 + i * RPC);
        const int bytes = row == kNoRow ? 0 : 16;   // 0: zeros, and nothing is read
        const size_t off = row == kNoRow ? 0 : (size_t)row * D;
        const uint32_t to = st + chunk_at<D>(lane / LPR + i * RPC, lane % LPR);
        cp_async_16(to + St::K, kp + off, bytes);
        cp_async_16(to + St::V, vp + off, bytes);
      }
      if ((lane >> 4) == odd)
        cp_async_8(st + copy_s, a.c.scales + (mine == kNoRow ? 0u : mine >> bs), mine == kNoRow ? 0 : 8);
    }
  };
  // the first kStages tiles on their way
  static_assert(kStages == 3, "two pairs cover the tiles issued up front and the next one");
  uint32_t rows = kNoRow, rows_n = kNoRow;   // rows of the pair that is issued from, and of the next one
  if (t0 < t_end) {
    const int k0 = key_of(place, e0), k1 = key_of(place + kPairStep, e1);
    const int p0 = ptab[k0 >> ps], p1 = ptab[k1 >> ps];
    const uint32_t r0 = row_of(place, k0, p0);
    rows = row_of(place + kPairStep, k1, p1);
    issue(r0, t0, 0, ring);
    cp_async_commit();   // one group per stage, empty past the last tile
    if (t0 + kWarps < t_end) issue(r0, t0 + kWarps, 1, ring + St::BYTES);
    cp_async_commit();
    if (t0 + 2 * kWarps < t_end) issue(rows, t0 + 2 * kWarps, 0, ring + 2 * St::BYTES);
    cp_async_commit();
  }

  if (early) {
    pdl_wait();
    pdl_launch_dependents();
    load_q();
  }
  // q as B operand of S^T, scaled into fp16.  It is kept in shared memory, the
  // same for every warp: registers are short (128 a thread) and the four reads
  // a tile cost less (Llama-shaped 32K lists, rows in L2, 7.75 -> 7.6 us; dense 101
  // -> 100).
  uint4* qs = reinterpret_cast<uint4*>(smem + L::q) + lane;
  float sc0, sc1;   // score scale of heads 2c and 2c + 1: log2(e) / sqrt(D) and q's power of two
  {
    float x[KQ][16];
    uint32_t am = 0;
#pragma unroll
    for (int s = 0; s < KQ; ++s) {
      const uint4 u = qw[s][0], v = qw[s][1];
      const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
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
    if (warp == 0) {
#pragma unroll
      for (int s = 0; s < KQ; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          qs[(2 * s + i) * 32] = make_uint4(pack_f16(x[s][8 * i] * up, x[s][8 * i + 1] * up),
                                            pack_f16(x[s][8 * i + 2] * up, x[s][8 * i + 3] * up),
                                            pack_f16(x[s][8 * i + 4] * up, x[s][8 * i + 5] * up),
                                            pack_f16(x[s][8 * i + 6] * up, x[s][8 * i + 7] * up));
    }
    const float mine = kLog2e * rsqrtf((float)D) * pow2f(e - 14);
    sc0 = __shfl_sync(0xffffffffu, mine, 8 * c);       // lane (2c, 0)
    sc1 = __shfl_sync(0xffffffffu, mine, 8 * c + 4);   // lane (2c + 1, 0)
  }
  __syncthreads();

  float m0 = t0 < t_end ? kNoScore : -INFINITY, m1 = m0, l0 = 0.f, l1 = 0.f;   // heads 2c, 2c + 1; sums over this lane's keys
  int e_run = 27;                                             // biased exponent E of the V scales met so far
  float oacc[MT][4];   // tile t: dim g D/8 + 2t of heads 2c, 2c + 1, then dim g D/8 + 2t + 1
#pragma unroll
  for (int t = 0; t < MT; ++t) oacc[t][0] = oacc[t][1] = oacc[t][2] = oacc[t][3] = 0.f;

  // this lane's chunks in a stage: K rows g and g + 8, V rows 2c, 2c + 1, + 8
  const uint32_t k_at = St::K + chunk_at<D>(g, KQ * c);
  const uint32_t v_at = St::V + (D == 128 ? chunk_at<D>(2 * c, g) : chunk_at<D>(2 * c, g >> 1) + (g & 1) * 8);
  uint32_t st = ring;
  int it = 0;
#pragma unroll 1
  for (int t = t0; t < t_end; t += kWarps, ++it) {
    // tile it + kStages is issued below: the first of pair (it + 3) / 2 when
    // `it` is odd, and then the next pair's rows have been found
    const bool find = !(it & 1) && t + (kStages + 1) * kWarps < t_end;
    int key2 = 0, page2 = 0;
    if (find) {
      key2 = key_of(k_n, e_n);
      page2 = ptab[key2 >> ps];
      e_n = entry(k_n + kPairStep);
    }
    cp_async_wait<kStages - 1>();   // this lane's copies of the tile
    __syncwarp();                   // ... and every other lane's
    const uint2 s0 = lds_v2(st + St::S + g * 8), s1 = lds_v2(st + St::S + (g + 8) * 8);
    float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < KQ; ++s) {
      const uint32_t at = st + (k_at ^ (16u * s));   // (KQ c is even: the next chunk's place is the other of a pair)
      const uint4 ka = lds_v4(at), kb = lds_v4(at + 8 * D);
      const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
      const uint4 q0 = qs[2 * s * 32], q1 = qs[(2 * s + 1) * 32];
      const uint32_t qf[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t a0, a1, a2, a3;
        q8_to_f16<CT>(wa[i], a0, a2);
        q8_to_f16<CT>(wb[i], a1, a3);
        mma_f16_16816(i & 1 ? sb : sa, a0, a1, a2, a3, qf[2 * i], qf[2 * i + 1]);
      }
    }
    const float ks0 = __uint_as_float(s0.x), ks1 = __uint_as_float(s1.x);
    float x0 = (sa[0] + sb[0]) * (sc0 * ks0), x1 = (sa[1] + sb[1]) * (sc1 * ks0);   // key g, heads 2c, 2c + 1
    float x2 = (sa[2] + sb[2]) * (sc0 * ks1), x3 = (sa[3] + sb[3]) * (sc1 * ks1);   // key g + 8
    if (t * kTile + kTile > count_b) {   // the last tile: its tail is masked
      if (t * kTile + g >= count_b) x0 = x1 = -INFINITY;
      if (t * kTile + g + 8 >= count_b) x2 = x3 = -INFINITY;
    }
    const uint32_t vm = __reduce_max_sync(0xffffffffu, max(s0.y & 0x7fffffffu, s1.y & 0x7fffffffu));
    float n0 = fmaxf(x0, x2), n1 = fmaxf(x1, x3);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, o));
      n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, o));
    }
    n0 = fmaxf(n0, m0);
    n1 = fmaxf(n1, m1);
    const int e_new = max(e_run, (int)(vm >> 23));
    // a maximum that grew rescales what is summed so far; most tiles have none
    if (__any_sync(0xffffffffu, n0 != m0 || n1 != m1 || e_new != e_run)) {
      const float al0 = join_weight(m0, n0), al1 = join_weight(m1, n1);
      const float f = pow2f(max(e_run - e_new, -126));
      l0 *= al0;
      l1 *= al1;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        oacc[i][0] *= al0 * f;
        oacc[i][1] *= al1 * f;
        oacc[i][2] *= al0 * f;
        oacc[i][3] *= al1 * f;
      }
      m0 = n0;
      m1 = n1;
      e_run = e_new;
    }
    const float ve = __uint_as_float((uint32_t)(268 - e_run) << 23);   // 2^(14 - E)
    const float v0 = __uint_as_float(s0.y) * ve, v1 = __uint_as_float(s1.y) * ve;
    const float p0 = ex2_fast(x0 - m0), p1 = ex2_fast(x1 - m1), p2f = ex2_fast(x2 - m0), p3 = ex2_fast(x3 - m1);
    l0 += p0 + p2f;
    l1 += p1 + p3;
    // P^T (keys x heads) from accumulator to operand layout
    const uint32_t b0 = movmatrix_trans(pack_f16(p0 * v0, p1 * v0));
    const uint32_t b1 = movmatrix_trans(pack_f16(p2f * v1, p3 * v1));
    uint32_t v[4][VW];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t at = st + (j & 1 ? next_row<D>(v_at) : v_at) + (j >> 1) * 8 * D;
      if constexpr (D == 128) {
        const uint4 x = lds_v4(at);
        v[j][0] = x.x, v[j][1] = x.y, v[j][VW - 2] = x.z, v[j][VW - 1] = x.w;
      } else {
        const uint2 x = lds_v2(at);
        v[j][0] = x.x, v[j][1] = x.y;
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      // word i / 2 of each key's chunk holds dims 4 (i / 2) .. + 3 of the lane's
      const uint32_t sel = i & 1 ? 0x7362 : 0x5140;
      uint32_t a0, a1, a2, a3;
      q8_to_f16<CT>(__byte_perm(v[0][i >> 1], v[1][i >> 1], sel), a0, a1);
      q8_to_f16<CT>(__byte_perm(v[2][i >> 1], v[3][i >> 1], sel), a2, a3);
      mma_f16_16816(oacc[i], a0, a1, a2, a3, b0, b1);
    }
    __syncwarp();   // every lane has read the stage
    if (it & 1) rows = rows_n;
    if (t + kStages * kWarps < t_end) issue(rows, t + kStages * kWarps, (it + kStages) & 1, st);
    cp_async_commit();
    if (find) {
      rows_n = row_of(k_n, key2, page2);
      k_n += kPairStep;
    }
    st = st + St::BYTES == ring + kStages * St::BYTES ? ring : st + St::BYTES;
  }
  if (bad_key) raise_error(a.err, kErrIndexRange);
  if (bad_page) raise_error(a.err, kErrPage);
  cp_async_wait<0>();
  __syncwarp();

  // ---- join the warps
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, o);
    l1 += __shfl_xor_sync(0xffffffffu, l1, o);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float* ro = reinterpret_cast<float*>(smem + warp * L::WARPB) + (2 * c + j) * L::RO + g * (D / 8);
#pragma unroll
    for (int t = 0; t < MT; ++t)
      *reinterpret_cast<float2*>(ro + 2 * t) = make_float2(oacc[t][j], oacc[t][2 + j]);
  }
  if (g == 0) {
    red_ml[warp * 8 + 2 * c] = make_float2(m0, l0);
    red_ml[warp * 8 + 2 * c + 1] = make_float2(m1, l1);
  }
  if (lane == 0) red_e[warp] = __uint_as_float((uint32_t)max(e_run - 14, 0) << 23);   // 2^(E - 14)
  __syncthreads();
  constexpr int Q4 = D / 4;   // units of four outputs per head: at most one per thread
  static_assert(8 * Q4 <= kThreads && Q4 >= kMaxCS, "a unit and a (max, sum) receiver per thread");
  const int hh = tid / Q4, d4 = (tid - hh * Q4) * 4;
  float M = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (hh < G) {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red_ml[w * 8 + hh].x);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = red_ml[w * 8 + hh];
      const float f = join_weight(ml.x, M);
      l += f * ml.y;
      const float fe = f * red_e[w];
      const float4 x = *reinterpret_cast<const float4*>(smem + w * L::WARPB + (hh * L::RO + d4) * 4);
      acc.x += fe * x.x, acc.y += fe * x.y, acc.z += fe * x.z, acc.w += fe * x.w;
    }
  }
  const size_t orow = (size_t)b * a.Hq + h * G + hh;
  if constexpr (kCluster) {
    if (cs == 1) {
      if (hh < G) {
        store_out<QT>(a, orow * D + d4, acc, M, l);
        if (d4 == 0 && a.lse) a.lse[orow] = lse_of(M, l);
      }
      return;
    }
    __syncwarp();   // (converged for the aligned barrier)
    // each unit goes to the CTA that owns it, each head's (max, sum) to every CTA
    cluster_wait_acquire();   // every CTA's mbarrier is initialised
    const uint32_t recv_ml = smem_u32(smem) + (uint32_t)L::recv_ml, recv_o = smem_u32(smem) + (uint32_t)L::recv_o;
    if (hh < G) {
      const int q = tid / units;
      st_async_v4(mapa(recv_o + (uint32_t)(rank * units + tid - q * units) * 16, q), acc, mapa(bar, q));
      const int r = tid - hh * Q4;
      if (r < cs) st_async_v2(mapa(recv_ml + (uint32_t)(rank * 8 + hh) * 8, r), make_float2(M, l), mapa(bar, r));
    }
    if (!mbar_wait_cluster_bounded(bar, 0)) raise_error(a.err, kErrMerge);
    // this CTA's units, the cluster's partial results of each side by side in cs lanes
    const int v = tid >> (31 - __clz(cs)), r = tid & (cs - 1), u = rank * units + v;   // (cs is a power of two: v < kThreads / cs)
    const bool have = v < units && u < G * Q4;
    const int uh = u / Q4, ud = (u - uh * Q4) * 4;
    float2 ml = make_float2(-INFINITY, 0.f);
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (have) {
      ml = reinterpret_cast<const float2*>(smem + L::recv_ml)[r * 8 + uh];
      acc = reinterpret_cast<const float4*>(smem + L::recv_o)[r * units + v];
    }
    M = ml.x;
    for (int o = 1; o < cs; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float f = join_weight(ml.x, M);
    l = f * ml.y;
    acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
    for (int o = 1; o < cs; o <<= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, o);
      acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
      acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
      acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
      acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
    }
    if (have && r == 0) {
      const size_t row = (size_t)b * a.Hq + h * G + uh;
      store_out<QT>(a, row * D + ud, acc, M, l);
      if (ud == 0 && a.lse) a.lse[row] = lse_of(M, l);
    }
    return;
  }
  if (hh < G) {
    if (ta == 0 && tb == tiles_b) {   // the problem whole
      store_out<QT>(a, orow * D + d4, acc, M, l);
      if (d4 == 0 && a.lse) a.lse[orow] = lse_of(M, l);
    } else {
      const size_t pr = (size_t)blockIdx.x * G + hh;
      *reinterpret_cast<float4*>(a.part_o + pr * D + d4) = acc;
      if (d4 == 0) a.part_ml[pr] = make_float2(M, l);
    }
  }
}

// Joins the partial results of one (problem, head): CTA = one row of o, and
// thread (group, 4 dims) the partial results group, group + GROUPS, ...
constexpr int kJoinThreads = 128;

template <int D, int QT>
__global__ void __launch_bounds__(kJoinThreads) q8_join_kernel(const Q8DecodeArgs a) {
  constexpr int Q4 = D / 4, GROUPS = kJoinThreads / Q4;
  constexpr int BATCH = 4;   // partial results whose loads are under way together
  __shared__ float4 acc_s[GROUPS][Q4];
  __shared__ float2 ml_s[GROUPS];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  const int prob = blockIdx.x / a.G, hh = blockIdx.x - prob * a.G;
  const int b = prob / a.Hp, h = prob - b * a.Hp;
  const int grp = tid / Q4, d4 = (tid - grp * Q4) * 4;
  const size_t orow = (size_t)b * a.Hq + h * a.G + hh;
  const int share = a.per > 0 ? a.per : *a.share;
  const int mine = a.per > 0 || !a.kv_lens ? 0 : first_rows(a);
  const int tiles = row_tiles(a, b);
  if (tiles == 0) {   // no key: zeros (no CTA above had this problem)
    if (grp == 0) store_out<QT>(a, orow * D + d4, make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f);
    if (tid == 0 && a.lse) a.lse[orow] = -INFINITY;
    return;
  }
  const int n = ceil_div(tiles, share);
  if (n == 1) return;   // written whole
  int first;            // the CTA above that had the problem's first part
  if (a.per > 0) first = prob * ceil_div(a.longest, share);
  else if (!a.kv_lens) first = prob * n;
  else first = sum_rows(a, mine, b, [&](int t) { return ceil_div(t, share); }) * a.Hp + h * n;
  float M = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = grp; s0 < n; s0 += GROUPS * BATCH) {
    float2 ml[BATCH];
    float4 x[BATCH];
    float m = M;
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int s = s0 + u * GROUPS;
      const size_t pr = (size_t)(first + min(s, n - 1)) * a.G + hh;
      ml[u] = a.part_ml[pr];
      x[u] = *reinterpret_cast<const float4*>(a.part_o + pr * D + d4);
      if (s >= n) ml[u] = make_float2(-INFINITY, 0.f);
    }
#pragma unroll
    for (int u = 0; u < BATCH; ++u) m = fmaxf(m, ml[u].x);
    const float f0 = join_weight(M, m);
    l *= f0;
    acc.x *= f0, acc.y *= f0, acc.z *= f0, acc.w *= f0;
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      if (s0 + u * GROUPS >= n) break;
      const float f = join_weight(ml[u].x, m);
      l += f * ml[u].y;
      acc.x += f * x[u].x, acc.y += f * x[u].y, acc.z += f * x[u].z, acc.w += f * x[u].w;
    }
    M = m;
  }
  acc_s[grp][d4 / 4] = acc;
  if (d4 == 0) ml_s[grp] = make_float2(M, l);
  __syncthreads();
  if (grp != 0) return;
#pragma unroll
  for (int r = 1; r < GROUPS; ++r) M = fmaxf(M, ml_s[r].x);
  l = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int r = 0; r < GROUPS; ++r) {
    const float2 ml = ml_s[r];
    const float f = join_weight(ml.x, M);
    const float4 x = acc_s[r][d4 / 4];
    l += f * ml.y;
    acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
  }
  store_out<QT>(a, orow * D + d4, acc, M, l);
  if (d4 == 0 && a.lse) a.lse[orow] = lse_of(M, l);
}

// cluster sizes of the first way, and how many clusters of each run at once
constexpr int kSizes[] = {16, 8, 4, 2};
constexpr int kNumSizes = 4;
constexpr int kClusterTiles = 16;  // most tiles of a warp in the first way
// The second way up to this many problems, the third from there on: 128 problems
// of 64K keys 342 against 322 us, 256 ragged ones up to 8K 77 against 58 us; 64
// ragged ones up to 64K 104 against 112 us.
constexpr int kShareProblems = kResident / 4;
// Tiles of a CTA in the third way: 256 problems ragged up to 512 tiles 58 us by
// 128 and 63 by 256, 128 problems of 4096 tiles 344 and 322 us.
int wave_tiles(int longest) { return longest < 2048 ? 128 : 256; }

template <int D, int QT, int CT>
const int* active_clusters() {
  // (host threads may come here at once: each fills the same numbers in, and
  // `ready` is set behind them)
  static int cached[64][kNumSizes];
  static std::atomic<bool> ready[64];
  static const int none[kNumSizes] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return none;
  if (!ready[dev].load(std::memory_order_acquire)) {
    for (int i = 0; i < kNumSizes; ++i) {
      int m = 0;
      const auto fn = q8_decode_kernel<D, QT, CT, true>;
      if (ensure_func_attrs(reinterpret_cast<const void*>(fn), Smem<D>::total, kSizes[i] > 8) == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        cfg.gridDim = dim3(kSizes[i]);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = Smem<D>::total;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kSizes[i];
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&m, fn, &cfg) != cudaSuccess) m = 0;
      }
      cached[dev][i] = m;
    }
    cudaGetLastError();
    ready[dev].store(true, std::memory_order_release);
  }
  return cached[dev];
}

template <int D, int QT, int CT>
cudaError_t run(Q8DecodeArgs a, cudaStream_t st) {
  const int64_t problems = (int64_t)a.B * a.Hp;
  const int tiles = a.longest;
  const bool pdl = (a.flags & 1) != 0;
  // a CTA per problem, or a cluster if its warps get few tiles each and all
  // problems run at once
  int cs = tiles <= kWarps ? 1 : 0;
  if (!cs) {
    const int* active = active_clusters<D, QT, CT>();
    bool fits[kNumSizes];
    for (int i = 0; i < kNumSizes; ++i)
      fits[i] = active[i] >= problems && tiles <= kSizes[i] * kWarps * kClusterTiles && tiles > (kSizes[i] / 2) * kWarps;
    cs = choose_cluster_size(problems, kSizes, active, fits, kNumSizes);
  }
  if (cs) {
    const auto fn = q8_decode_kernel<D, QT, CT, true>;
    const cudaError_t e = ensure_func_attrs(reinterpret_cast<const void*>(fn), Smem<D>::total, cs > 8);
    if (e != cudaSuccess) return e;
    a.per = max((tiles + cs - 1) / cs, kWarps);   // a tile for every warp, then the next CTA
    return launch_ex(fn, dim3((unsigned)(problems * cs)), dim3(kThreads), Smem<D>::total, st, pdl, cs, a);
  }
  const auto fn = q8_decode_kernel<D, QT, CT, false>;
  cudaError_t e = ensure_func_attrs(reinterpret_cast<const void*>(fn), Smem<D>::total, false);
  if (e != cudaSuccess) return e;
  a.per = problems > kShareProblems ? wave_tiles(tiles) : 0;
  e = launch_ex(fn, dim3((unsigned)a.ctas), dim3(kThreads), Smem<D>::total, st, pdl, 1, a);
  if (e != cudaSuccess) return e;
  // the join waits for the kernel above before it reads anything, so it may always be launched early
  return launch_ex(q8_join_kernel<D, QT>, dim3((unsigned)((int64_t)a.B * a.Hq)), dim3(kJoinThreads), 0, st, true, 1, a);
}

template <int D, int QT>
cudaError_t run_ct(const Q8DecodeArgs& a, int cache_type, cudaStream_t st) {
  return cache_type == kInt8 ? run<D, QT, kInt8>(a, st) : run<D, QT, kE4M3>(a, st);
}

}  // namespace

Q8Plan q8_decode_plan(int64_t problems, int count) {
  Q8Plan p;
  p.longest = (count + kTile - 1) / kTile;
  if (p.longest <= kWarps) {
    p.ctas = problems;
    p.parts = 0;
  } else if (problems > kShareProblems) {
    const int n = (p.longest + wave_tiles(p.longest) - 1) / wave_tiles(p.longest);
    p.ctas = problems * n;
    p.parts = p.ctas;
  } else {
    const int64_t most = problems * ((p.longest + kWarps - 1) / kWarps);
    p.ctas = p.parts = most < kResident ? most : kResident;
  }
  return p;
}

cudaError_t launch_q8_decode(const Q8DecodeArgs& a, int in_type, int cache_type, cudaStream_t stream) {
  if (a.c.D == 128)
    return in_type == kInF16 ? run_ct<128, kInF16>(a, cache_type, stream) : run_ct<128, kInBf16>(a, cache_type, stream);
  return in_type == kInF16 ? run_ct<64, kInF16>(a, cache_type, stream) : run_ct<64, kInBf16>(a, cache_type, stream);
}

}  // namespace kascade
