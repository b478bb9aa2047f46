// Book-keeping and data movement of the 8-bit paged KV cache: page tables and
// slot maps from request lengths, the append that quantises new K and V rows
// into their pages, and the gather that turns pages back into contiguous
// slabs (a paged cache stores the same keys in fixed-size pages: README,
// Kernel Benchmarks note on paged kernels).
#include "q8.cuh"

namespace kascade {

namespace {

// ------------------------------------------------------------- page tables
//
// Request b holds n_b tokens and adds m_b: first_b = ceil(n_b / P) pages held,
// need_b = ceil((n_b + m_b) / P) - first_b to take.  With c and f the exclusive
// prefix sums of m and need, the call writes page_table[b, first_b + i] =
// free[f_b + i] and the slots of b's new tokens at slot_map[c_b ...].
//
// Bound by latency (a few dependent loads), not by its bytes.  Each CTA
// computes the prefix sums of all requests for itself (two scans of B
// integers out of L2) and then writes its share of the slots, the new table
// entries and the lengths: one launch, no exchange between CTAs.  That is why
// lens_out must not overlap kv_lens: another CTA may still be reading it.

constexpr int kTabThreads = 256;
constexpr int kTabTokens = 4;                 // slots per thread and step
constexpr int kMaxBatch = 4096;               // two prefix-sum arrays in 32 KB of shared memory
constexpr int kMaxLen = 1 << 20;              // tokens of a request

__global__ void __launch_bounds__(kTabThreads) page_tables_kernel(const PageTablesArgs a) {
  __shared__ int tok[kMaxBatch + 1], pag[kMaxBatch + 1];
  __shared__ int scan[kTabThreads / 32 + 1];
  const int tid = threadIdx.x, P1 = (1 << a.page_shift) - 1;
  // prefix sums, kTabThreads requests at a time; 64-bit totals, since a sum
  // of invalid lengths may pass 31 bits before it is refused
  bool bad = false;
  long long toks = 0, pages = 0;
  for (int b0 = 0; b0 < a.B; b0 += kTabThreads) {
    const int b = b0 + tid;
    int m = 0, need = 0;
    if (b < a.B) {
      const int n = a.kv_lens[b], add = a.new_lens[b];
      const bool ok = n >= 0 && add >= 0 && n <= kMaxLen && add <= kMaxLen && n + add <= kMaxLen &&
                      ((n + add + P1) >> a.page_shift) <= a.max_pages;
      bad |= !ok;
      if (ok) {
        m = add;
        need = ((n + add + P1) >> a.page_shift) - ((n + P1) >> a.page_shift);
      }
    }
    // at most 256 requests of 2^20 tokens: 2^28 per step
    int mt, nt;
    const int mi = block_inclusive_scan<kTabThreads>(m, scan, &mt);
    const int ni = block_inclusive_scan<kTabThreads>(need, scan, &nt);
    if (b < a.B) {
      // the low 32 bits; read only once the totals are known to fit
      tok[b] = (int)(toks + mi - m);
      pag[b] = (int)(pages + ni - need);
    }
    toks += mt;
    pages += nt;
  }
  if (tid == 0) {
    tok[a.B] = (int)toks;
    pag[a.B] = (int)pages;
  }
  bad |= toks > a.capacity || pages > a.num_free;
  const bool fail = __syncthreads_or(bad);   // the same verdict in every CTA
  const int T = fail ? 0 : (int)toks;
  const int gtid = blockIdx.x * kTabThreads + tid, gthreads = gridDim.x * kTabThreads;

  for (int b = gtid; b < a.B; b += gthreads) {
    a.lens_out[b] = fail ? a.kv_lens[b] : a.kv_lens[b] + a.new_lens[b];
    a.offsets[b] = fail ? 0 : tok[b];
  }
  if (gtid == 0) {
    a.offsets[a.B] = T;
    a.info[0] = fail ? -1 : (int)pages;
    a.info[1] = T;
  }
  if (!fail)
    for (int i = gtid; i < (int)pages; i += gthreads) {
      const int b = q8_owner(pag, a.B, i);
      const int first = (a.kv_lens[b] + P1) >> a.page_shift;
      a.page_table[(size_t)b * a.max_pages + first + i - pag[b]] = a.free_pages[i];
    }

  // slots, kTabTokens consecutive ones per thread and step, the tail -1.
  // Pages held before are read from the table, new ones from the free list
  // (their table entries are being written by other CTAs).
  for (long long t0 = (long long)gtid * kTabTokens; t0 < a.capacity; t0 += (long long)gthreads * kTabTokens) {
    int out[kTabTokens];
    int b = t0 < T ? q8_owner(tok, a.B, (int)t0) : 0;
    int page = 0, page_of = -1, page_b = -1;   // the page looked up last
#pragma unroll
    for (int u = 0; u < kTabTokens; ++u) {
      const int t = (int)t0 + u;
      out[u] = -1;
      if (t < T) {
        while (tok[b + 1] <= t) ++b;
        const int n = a.kv_lens[b], pos = n + t - tok[b];
        const int pi = pos >> a.page_shift, first = (n + P1) >> a.page_shift;
        if (pi != page_of || b != page_b) {
          page = pi < first ? a.page_table[(size_t)b * a.max_pages + pi] : a.free_pages[pag[b] + pi - first];
          page_of = pi;
          page_b = b;
        }
        out[u] = (int)(((unsigned)page << a.page_shift) | (unsigned)(pos & P1));
      }
    }
    if (t0 + kTabTokens <= a.capacity && (((uintptr_t)a.slot_map) & 15) == 0) {
      *reinterpret_cast<int4*>(a.slot_map + t0) = make_int4(out[0], out[1], out[2], out[3]);
    } else {
#pragma unroll
      for (int u = 0; u < kTabTokens; ++u)
        if (t0 + u < a.capacity) a.slot_map[t0 + u] = out[u];
    }
  }
}

// ------------------------------------------------------------------ append
//
// A run is a maximal stretch of tokens whose slots lie in one block (S rows of
// one page); skipped tokens (slots outside the pool) inside it do not end it
// unless 32 follow one another.  For each run, kv head and tensor:
//   s = 2^e, the smallest with max |x| <= top s over the run's finite values;
//   if rows of the block precede the run: s = max(s_old, s), and where that
//   grew, those rows become rn(y s_old / s);
//   the new rows become rn(x / s).
// Bound by HBM: each input value is read once from HBM (a second time from
// L1/L2, once the maximum is known) and each byte written once.
//
// A CTA takes `tile` tokens of one (kv head, tensor) and owns the runs that
// start there.  Runs of up to kShortRun rows (a decode step) go to a warp
// each, which keeps the rows in registers; longer ones (a prompt) are done by
// the whole CTA.

constexpr int kAppThreads = 256;
constexpr int kAppWarps = kAppThreads / 32;
constexpr int kShortRun = 8;
constexpr int kMaxTile = 256;

// eight consecutive input values as floats
template <int IN>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&x)[8]) {
  if constexpr (IN == kInF32) {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = __ldg(f), b = __ldg(f + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 r = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (IN == kInBf16) {
        x[2 * j] = bf16_lo(w[j]);
        x[2 * j + 1] = bf16_hi(w[j]);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
      }
    }
  }
}

// bits of the largest finite magnitude (non-negative floats order like their bits)
__device__ __forceinline__ uint32_t amax_bits(const float (&x)[8], uint32_t m) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t u = __float_as_uint(x[j]) & 0x7fffffffu;
    m = max(m, u < 0x7f800000u ? u : 0u);
  }
  return m;
}

// x s and x / s to 24 bits, rounded to odd (towards zero, the last bit set
// where something was dropped): rounding that to at most 8 bits then gives
// what rounding the exact value would, which a nearest fp32 value next to a
// border does not.  (A remainder below fp32's range belongs to a value that
// rounds to zero.)
__device__ __forceinline__ float odd_if(float y, float rest) {
  return rest != 0.0f ? __uint_as_float(__float_as_uint(y) | 1u) : y;
}
__device__ __forceinline__ float mul_odd(float x, float s) {
  const float y = __fmul_rz(x, s);
  return odd_if(y, __fmaf_rn(x, s, -y));
}
__device__ __forceinline__ float div_odd(float x, float s) {
  const float y = __fdiv_rz(x, s);
  return odd_if(y, __fmaf_rn(-y, s, x));
}

// rn(x / s).  For a power of two the product with 1 / s is the quotient; a
// block that keeps a scale of the caller's own may have any other.
template <int CT>
__device__ __forceinline__ uint2 pack8(const float (&x)[8], float s) {
  float y[8];
  if ((__float_as_uint(s) & 0x7fffffu) == 0) {
    const float inv = 1.0f / s;
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = x[j] * inv;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = div_odd(x[j], s);
  }
  return make_uint2(q8_pack4<CT>(y[0], y[1], y[2], y[3]), q8_pack4<CT>(y[4], y[5], y[6], y[7]));
}

// rn(y r) of sixteen bytes
template <int CT>
__device__ __forceinline__ uint4 requant16(uint4 y, float r) {
  const uint32_t w[4] = {y.x, y.y, y.z, y.w};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t lo, hi;
    q8_to_f16<CT>(w[j], lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    o[j] = q8_pack4<CT>(mul_odd(a.x, r), mul_odd(a.y, r), mul_odd(b.x, r), mul_odd(b.y, r));
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int D, int IN, int CT>
__global__ void __launch_bounds__(kAppThreads) q8_append_kernel(const Q8AppendArgs a, int tile) {
  constexpr int LPR = D / 8;           // lanes per input row
  constexpr int RPW = 32 / LPR;        // input rows per warp and pass
  constexpr int CPR = D / 16;          // 16-byte chunks per cache row
  constexpr int PASSES = kShortRun / RPW;
  __shared__ int long_t[kMaxTile], long_n[kMaxTile];
  __shared__ int n_long;
  __shared__ uint32_t red[kAppWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const void* src = is_v ? a.v : a.k;
  const int64_t ts = is_v ? a.v_token : a.k_token;
  const int64_t hoff = (int64_t)h * (is_v ? a.v_head : a.k_head);
  uint8_t* pages = is_v ? a.c.v : a.c.k;
  float* scales = reinterpret_cast<float*>(a.c.scales) + (is_v ? 1 : 0);
  const int ps = a.c.page_shift, bs = a.c.block_shift;
  const int sub = lane / LPR, col = (lane % LPR) * 8;

  auto row_of = [&](int slot) -> uint32_t {
    return q8_row((uint32_t)slot >> ps, (uint32_t)slot & ((1u << ps) - 1u), h, a.c.Hkv, ps);
  };
  auto valid = [&](int slot) { return q8_slot_ok(slot, a.c.num_pages, ps); };
  // the block's scale once the run's maximum is known: (scale, ratio for the
  // rows before the run, 1 when they stay)
  auto new_scale = [&](uint32_t amax, uint32_t offset, float old, float& ratio) -> float {
    float s = pow2f(q8_scale_exp(amax, CT == kInt8));
    ratio = 1.0f;
    if (offset > 0) {
      if (s > old) ratio = old / s;   // exact: s is a power of two
      else if (old >= s) s = old;     // (a NaN old scale is dropped)
    }
    return s;
  };
  if (tid == 0) n_long = 0;
  __syncthreads();

  const int t0 = blockIdx.x * tile, t1 = min(a.T, t0 + tile);
  for (int t = t0 + warp; t < t1; t += kAppWarps) {
    const int slot = __ldg(a.slots + t);
    if (!valid(slot)) {   // -1: a padding token
      if (slot != -1 && lane == 0) raise_error(a.err, kErrPage);
      continue;
    }
    const uint32_t blk = (uint32_t)slot >> bs;
    // the last token before this one that is not skipped, 32 back at most: in
    // the same block, this one is inside a run that starts earlier
    {
      const int u = t - 1 - lane;
      const int x = u >= 0 ? __ldg(a.slots + u) : -1;
      const uint32_t m = __ballot_sync(0xffffffffu, valid(x));
      if (m && __shfl_sync(0xffffffffu, (uint32_t)x >> bs, __ffs(m) - 1) == blk) continue;
    }
    // tokens of the run: to the last one before a token of another block or 32 skipped ones
    int n = 1;
    for (;;) {
      const int u = t + n + lane;
      const int x = u < a.T ? __ldg(a.slots + u) : -1;
      const bool ok = valid(x), here = ok && ((uint32_t)x >> bs) == blk;
      uint32_t in = __ballot_sync(0xffffffffu, here);
      const uint32_t other = __ballot_sync(0xffffffffu, ok && !here);
      if (other) in &= (other & (0u - other)) - 1u;   // up to the first of another block
      if (in) n += 32 - __clz(in);
      if (!in || other) break;
    }
    if (n > kShortRun) {
      if (lane == 0) {
        const int i = atomicAdd(&n_long, 1);
        long_t[i] = t;
        long_n[i] = n;
      }
      continue;
    }
    float x[PASSES][8];
    int at[PASSES];
    uint32_t am = 0;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int i = p * RPW + sub;
      at[p] = i < n ? __ldg(a.slots + t + i) : -1;
      if (valid(at[p])) {
        load8<IN>(src, (int64_t)(t + i) * ts + hoff + col, x[p]);
        am = amax_bits(x[p], am);
      }
    }
    am = __reduce_max_sync(0xffffffffu, am);
    const uint32_t offset = (uint32_t)slot & ((1u << bs) - 1u);
    const uint32_t row = row_of(slot), row0 = row - offset;
    float* sp = scales + 2 * (size_t)(row >> bs);
    const float old = offset ? *sp : 0.0f;
    float ratio;
    const float s = new_scale(am, offset, old, ratio);
    __syncwarp();
    if (lane == 0) *sp = s;
    if (ratio != 1.0f)
      for (int c = lane; c < (int)offset * CPR; c += 32) {
        uint4* p = reinterpret_cast<uint4*>(pages + (size_t)row0 * D) + c;
        *p = requant16<CT>(*p, ratio);
      }
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      if (valid(at[p]))
        *reinterpret_cast<uint2*>(pages + (size_t)row_of(at[p]) * D + col) = pack8<CT>(x[p], s);
    }
  }
  __syncthreads();

  const int runs = n_long;
  for (int q = 0; q < runs; ++q) {
    const int t = long_t[q], n = long_n[q];
    uint32_t am = 0;
    for (int i = warp * RPW + sub; i < n; i += kAppWarps * RPW) {
      float x[8];
      if (!valid(__ldg(a.slots + t + i))) continue;
      load8<IN>(src, (int64_t)(t + i) * ts + hoff + col, x);
      am = amax_bits(x, am);
    }
    am = __reduce_max_sync(0xffffffffu, am);
    if (lane == 0) red[warp] = am;
    const int slot = __ldg(a.slots + t);
    const uint32_t offset = (uint32_t)slot & ((1u << bs) - 1u);
    const uint32_t row = row_of(slot), row0 = row - offset;
    float* sp = scales + 2 * (size_t)(row >> bs);
    const float old = offset ? *sp : 0.0f;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppWarps; ++w) am = max(am, red[w]);
    float ratio;
    const float s = new_scale(am, offset, old, ratio);
    if (ratio != 1.0f)
      for (int c = tid; c < (int)offset * CPR; c += kAppThreads) {
        uint4* p = reinterpret_cast<uint4*>(pages + (size_t)row0 * D) + c;
        *p = requant16<CT>(*p, ratio);
      }
    for (int i = warp * RPW + sub; i < n; i += kAppWarps * RPW) {
      const int sl = __ldg(a.slots + t + i);
      if (!valid(sl)) continue;
      float x[8];
      load8<IN>(src, (int64_t)(t + i) * ts + hoff + col, x);
      *reinterpret_cast<uint2*>(pages + (size_t)row_of(sl) * D + col) = pack8<CT>(x, s);
    }
    __syncthreads();   // every thread has read the old scale (and red) of this run
    if (tid == 0) *sp = s;
  }
}

// ------------------------------------------------------------------ gather
//
// out[b, h, j] = byte x scale, rounded once to the output type, for j <
// kv_lens[b]; later rows are not touched.  Bound by HBM (1 byte read and 2 or
// 4 written per element): every thread turns 8 bytes into one or two 16-byte
// stores, so a warp writes whole 512-byte stretches.

constexpr int kGatThreads = 256;
constexpr int kGatUnroll = 4;

template <int D, int OUT, int CT>
__global__ void __launch_bounds__(kGatThreads) q8_gather_kernel(const Q8GatherArgs a, int chunks) {
  constexpr int CPR = D / 8;                      // 8-byte chunks per row
  constexpr int ROWS = kGatThreads / CPR;         // rows per pass
  const int bh = blockIdx.x / chunks, chunk = blockIdx.x - bh * chunks;
  const int b = bh / a.c.Hkv, h = bh - b * a.c.Hkv;
  const bool is_v = blockIdx.y != 0 || !a.k;
  const int len = a.kv_lens ? min(max(__ldg(a.kv_lens + b), 0), a.N) : a.N;
  const uint8_t* pages = is_v ? a.c.v : a.c.k;
  void* out = is_v ? a.v : a.k;
  const int ps = a.c.page_shift;
  const int ch = threadIdx.x % CPR, r0 = chunk * ROWS * kGatUnroll + threadIdx.x / CPR;
  uint2 raw[kGatUnroll];
  float sc[kGatUnroll];
#pragma unroll
  for (int u = 0; u < kGatUnroll; ++u) {
    const int j = r0 + u * ROWS;
    if (j < len) {
      bool bad = false;
      const uint32_t pg = q8_page(__ldg(a.page_table + (size_t)b * a.max_pages + (j >> ps)), a.c.num_pages, bad);
      if (bad) raise_error(a.err, kErrPage);
      const uint32_t row = q8_row(pg, (uint32_t)j & ((1u << ps) - 1u), h, a.c.Hkv, ps);
      raw[u] = __ldg(reinterpret_cast<const uint2*>(pages + (size_t)row * D) + ch);
      sc[u] = __ldg(reinterpret_cast<const float*>(a.c.scales) + 2 * (size_t)(row >> a.c.block_shift) + (is_v ? 1 : 0));
    }
  }
#pragma unroll
  for (int u = 0; u < kGatUnroll; ++u) {
    const int j = r0 + u * ROWS;
    if (j >= len) continue;
    float x[8];
    const uint32_t w[2] = {raw[u].x, raw[u].y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t lo, hi;
      q8_to_f16<CT>(w[i], lo, hi);
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&lo));
      const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      x[4 * i] = p.x * sc[u], x[4 * i + 1] = p.y * sc[u], x[4 * i + 2] = q.x * sc[u], x[4 * i + 3] = q.y * sc[u];
    }
    const size_t at = ((size_t)bh * a.N + j) * D + 8 * ch;
    if constexpr (OUT == kInF32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
      __stcs(o, make_float4(x[0], x[1], x[2], x[3]));
      __stcs(o + 1, make_float4(x[4], x[5], x[6], x[7]));
    } else {
      uint32_t y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (OUT == kInBf16) {
          y[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
        } else {
          const __half2 t = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
          y[i] = *reinterpret_cast<const uint32_t*>(&t);
        }
      }
      __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at), make_uint4(y[0], y[1], y[2], y[3]));
    }
  }
}

template <int D, int IN, int CT>
cudaError_t run_append(const Q8AppendArgs& a, cudaStream_t st) {
  // eight tokens per CTA (one per warp) as long as that is not many CTAs, as
  // in a decode step; else a tile of a block's size, so that a prompt's runs
  // start one to a CTA and few CTAs find nothing to do
  const int64_t small = ((int64_t)a.T + kAppWarps - 1) / kAppWarps * a.c.Hkv * 2;
  int tile = kAppWarps;
  if (small > 4096) tile = min(max(1 << a.c.block_shift, 64), kMaxTile);
  const dim3 grid((a.T + tile - 1) / tile, a.c.Hkv, 2);
  return launch_ex(q8_append_kernel<D, IN, CT>, grid, dim3(kAppThreads), 0, st, false, 1, a, tile);
}

template <int D, int CT>
cudaError_t append_in(const Q8AppendArgs& a, int in_type, cudaStream_t st) {
  if (in_type == kInF32) return run_append<D, kInF32, CT>(a, st);
  if (in_type == kInF16) return run_append<D, kInF16, CT>(a, st);
  return run_append<D, kInBf16, CT>(a, st);
}

template <int D, int OUT, int CT>
cudaError_t run_gather(const Q8GatherArgs& a, cudaStream_t st) {
  const int rows = kGatThreads / (D / 8) * kGatUnroll;
  const int chunks = (a.N + rows - 1) / rows;
  const dim3 grid((unsigned)((int64_t)chunks * a.B * a.c.Hkv), a.k && a.v ? 2 : 1, 1);
  return launch_ex(q8_gather_kernel<D, OUT, CT>, grid, dim3(kGatThreads), 0, st, false, 1, a, chunks);
}

template <int D, int CT>
cudaError_t gather_out(const Q8GatherArgs& a, int out_type, cudaStream_t st) {
  if (out_type == kInF32) return run_gather<D, kInF32, CT>(a, st);
  if (out_type == kInF16) return run_gather<D, kInF16, CT>(a, st);
  return run_gather<D, kInBf16, CT>(a, st);
}

}  // namespace

cudaError_t launch_page_tables(const PageTablesArgs& a, cudaStream_t stream) {
  const int per = kTabThreads * kTabTokens;
  const int work = a.capacity > a.B ? a.capacity : a.B;
  const int blocks = (work + per - 1) / per;
  return launch_ex(page_tables_kernel, dim3(blocks < 1 ? 1 : blocks > 296 ? 296 : blocks), dim3(kTabThreads), 0, stream,
                   false, 1, a);
}

cudaError_t launch_q8_append(const Q8AppendArgs& a, int in_type, int cache_type, cudaStream_t stream) {
  if (a.c.D == 128)
    return cache_type == kInt8 ? append_in<128, kInt8>(a, in_type, stream) : append_in<128, kE4M3>(a, in_type, stream);
  return cache_type == kInt8 ? append_in<64, kInt8>(a, in_type, stream) : append_in<64, kE4M3>(a, in_type, stream);
}

cudaError_t launch_q8_gather(const Q8GatherArgs& a, int out_type, int cache_type, cudaStream_t stream) {
  if (a.c.D == 128)
    return cache_type == kInt8 ? gather_out<128, kInt8>(a, out_type, stream) : gather_out<128, kE4M3>(a, out_type, stream);
  return cache_type == kInt8 ? gather_out<64, kInt8>(a, out_type, stream) : gather_out<64, kE4M3>(a, out_type, stream);
}

}  // namespace kascade
