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
// Bound by latency (a few dependent loads), not by its bytes: 3.4 us for a step
// of 8 requests, 8.2 us for 2048 requests and a million slots.  Each CTA
// computes the prefix sums of all requests for itself (2 B integers out of L2)
// and then writes its share of the slots, the new table entries and the
// lengths: one launch, no exchange between CTAs.  That is why lens_out must not
// overlap kv_lens: another CTA may still be reading it.

constexpr int kTabThreads = 256;
constexpr int kTabTokens = 4;                 // slots per thread and step
constexpr int kTabCtas = 148 * 4;             // 2048 requests, 1M slots: 8.1 us; 148 * 2: 8.7, 148 * 6: 9.6
constexpr int kMaxBatch = 4096;               // two prefix-sum arrays in 32 KB of shared memory
constexpr int kMaxLen = 1 << 20;              // tokens of a request
constexpr int kTokBits = 33;
constexpr unsigned long long kTokMask = (1ull << kTokBits) - 1;

__global__ void __launch_bounds__(kTabThreads) page_tables_kernel(const PageTablesArgs a) {
  __shared__ int tok[kMaxBatch + 1], pag[kMaxBatch + 1];
  __shared__ unsigned long long scan[kTabThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, P1 = (1 << a.page_shift) - 1;
  // prefix sums.  The lengths come in by coalesced loads; then a thread takes
  // `per` consecutive requests (an odd number: no bank conflicts), and one scan
  // over the CTA joins the threads.  Tokens (at most 4096 2^20 < 2^33) and
  // pages (< 2^29) share a 64-bit word; an invalid request adds nothing and is
  // refused below.
  for (int b = tid; b < a.B; b += kTabThreads) {
    tok[b] = __ldg(a.kv_lens + b);
    pag[b] = __ldg(a.new_lens + b);
  }
  __syncthreads();
  const int per = (a.B + kTabThreads - 1) / kTabThreads | 1, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  bool bad = false;
  unsigned long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = tok[b], add = pag[b];
    const bool ok = n >= 0 && add >= 0 && n <= kMaxLen && add <= kMaxLen && n + add <= kMaxLen &&
                    ((n + add + P1) >> a.page_shift) <= a.max_pages;
    bad |= !ok;
    // this thread's own sums for now
    tok[b] = (int)(mine & kTokMask);
    pag[b] = (int)(mine >> kTokBits);
    if (ok)
      mine += (unsigned long long)add |
              (unsigned long long)(((n + add + P1) >> a.page_shift) - ((n + P1) >> a.page_shift)) << kTokBits;
  }
  unsigned long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  unsigned long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kTabThreads / 32; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  for (int b = b0; b < b1; ++b) {   // (read only once the totals are known to fit 31 bits)
    tok[b] += (int)(before & kTokMask);
    pag[b] += (int)(before >> kTokBits);
  }
  const long long toks = (long long)(total & kTokMask), pages = (long long)(total >> kTokBits);
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
        out[u] = q8_slot(page, (uint32_t)(pos & P1), a.page_shift);
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
// Bound by HBM for prompts: each input value is read once and waits on the SM
// for its run's maximum, each byte is written once: 36.6 us for a 32K prompt of 8
// kv heads, d = 128, blocks of 64 in bf16 (5.5 TB/s), 58 us in fp32 (5.8 TB/s).  A
// decode step is bound by latency: 2.5 us for 8 requests.
//
// Three kernels, by the block's size and the number of tokens (see run_append).
// The heads of a token are worked on next to one another: together they read
// whole stretches of memory.
constexpr int kAppThreads = 256;
constexpr int kAppWarps = kAppThreads / 32;
constexpr int kShortRun = 8;   // rows of a run that a warp does alone
constexpr int kMaxTile = 256;
// CTAs of the form for few tokens (8 tokens of a set each) up to which it is
// taken.  8 kv heads, d = 128 in bf16, few against many: decode steps of 512
// 6.0 and 14.5 us, of 1024 9.9 and 14.4, of 2048 17.7 and 14.6; prompts of 1000
// tokens 7.7 and 7.1, of 2048 12.0 and 4.4 (8 of 250 13.4 and 13.5).  13 ragged
// chunks of d = 64 in fp32, blocks of 16, where the form for many takes 10 us
// whatever their length: 1392 CTAs 7.3 and 10.0 us, 1808 8.0 and 10.2, 3148
// 10.7 and 10.6, 4024 12.8 and 10.3; one prompt of those rows, 1024 CTAs 5.9 and
// 5.8, 2000 8.0 and 7.4, 4096 13.3 and 6.6.
constexpr int kFewCtas = 2048;
constexpr uint32_t kNoRow = 0xffffffffu;
constexpr int kLook = 32;      // skipped tokens that part two runs of one block

// eight consecutive input values, as they are and as floats
template <int IN>
struct Raw8 {
  uint4 w[IN == kInF32 ? 2 : 1];
};
template <int IN>
__device__ __forceinline__ Raw8<IN> load8(const void* p, int64_t i) {
  Raw8<IN> r;
  if constexpr (IN == kInF32) {
    const uint4* f = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
    r.w[0] = __ldg(f);
    r.w[1] = __ldg(f + 1);
  } else {
    r.w[0] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i));
  }
  return r;
}
template <int IN>
__device__ __forceinline__ void floats(const Raw8<IN>& r, float (&x)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (IN == kInF32) {
      const uint4 v = r.w[1];
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
      x[j] = __uint_as_float(w[j]);
      x[4 + j] = __uint_as_float(u[j]);
    } else if constexpr (IN == kInBf16) {
      x[2 * j] = bf16_lo(w[j]);
      x[2 * j + 1] = bf16_hi(w[j]);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
      x[2 * j] = f.x;
      x[2 * j + 1] = f.y;
    }
  }
}

// Largest magnitude of the values added.  Magnitudes order like their bits, so
// 16-bit types take the maximum of two values at once.  add() takes infinities
// and NaN too (they come out largest: finite() is false), add_finite() leaves
// them out.
template <int IN>
struct MaxAcc {
  uint32_t m = 0;
  __device__ __forceinline__ void add(const Raw8<IN>& r) {
    if constexpr (IN == kInF32) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        m = max(max(m, max(r.w[j].x & 0x7fffffffu, r.w[j].y & 0x7fffffffu)),
                max(r.w[j].z & 0x7fffffffu, r.w[j].w & 0x7fffffffu));
    } else {
      m = max2(max2(m, max2(r.w[0].x & 0x7fff7fffu, r.w[0].y & 0x7fff7fffu)),
               max2(r.w[0].z & 0x7fff7fffu, r.w[0].w & 0x7fff7fffu));
    }
  }
  __device__ __forceinline__ void add_finite(const Raw8<IN>& r) {
    float x[8];
    floats<IN>(r, x);
    uint32_t f = 0;   // as fp32
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t u = __float_as_uint(x[j]) & 0x7fffffffu;
      f = max(f, u < 0x7f800000u ? u : 0u);
    }
    if constexpr (IN == kInF32) m = max(m, f);
    if constexpr (IN == kInBf16) m = max2(m, f >> 16);
    if constexpr (IN == kInF16) m = max2(m, (uint32_t)__half_as_ushort(__float2half_rn(__uint_as_float(f))));
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ __forceinline__ uint32_t top() const { return IN == kInF32 ? m : max(m & 0xffffu, m >> 16); }
  __device__ __forceinline__ bool finite() const {
    return top() < (IN == kInF32 ? 0x7f800000u : IN == kInBf16 ? 0x7f80u : 0x7c00u);
  }
  __device__ __forceinline__ uint32_t bits() const {   // of the fp32 value
    if constexpr (IN == kInF32) return m;
    if constexpr (IN == kInBf16) return top() << 16;
    return __float_as_uint(__half2float(__ushort_as_half((unsigned short)top())));
  }
};

// x s and x / s to 24 bits, rounded to odd (towards zero, the last bit set
// where something was dropped): rounding that to at most 8 bits then gives
// what rounding the exact value would, which a nearest fp32 value next to a
// border does not.  (A remainder below fp32's range belongs to a value that
// rounds to zero; that of an infinity is NaN, which is no remainder.)
__device__ __forceinline__ float odd_if(float y, float rest) {
  return fabsf(rest) > 0.0f ? __uint_as_float(__float_as_uint(y) | 1u) : y;
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
__device__ __forceinline__ bool is_pow2(float s) { return (__float_as_uint(s) & 0x7fffffu) == 0; }   // (infinity too)
constexpr float kMaxEasy = 0x1p126f;   // the largest scale whose reciprocal is a normal number
template <int IN, int CT>
__device__ __forceinline__ uint2 pack8_pow2(const Raw8<IN>& r, float inv) {
  float x[8];
  floats<IN>(r, x);
  return make_uint2(q8_pack4<CT>(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                    q8_pack4<CT>(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
}
// The same for finite values that s does not saturate.  To int8 by one fused
// multiply-add each, whose rounding at 1.5 2^23 is the one to an integer (a
// conversion instruction goes through a pipe of a quarter of the rate: a 32K
// prompt in int8 43.4 us with those).
template <int IN, int CT>
__device__ __forceinline__ uint2 pack8_finite(const Raw8<IN>& r, float inv) {
  if constexpr (CT != kInt8) return pack8_pow2<IN, CT>(r, inv);
  float x[8];
  floats<IN>(r, x);
  uint32_t y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = __float_as_uint(__fmaf_rn(x[j], inv, 12582912.0f));
  return make_uint2(__byte_perm(__byte_perm(y[0], y[1], 0x0040), __byte_perm(y[2], y[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(y[4], y[5], 0x0040), __byte_perm(y[6], y[7], 0x0040), 0x5410));
}
template <int IN, int CT>
__device__ __forceinline__ uint2 pack8(const Raw8<IN>& r, float s) {
  if (is_pow2(s)) return pack8_pow2<IN, CT>(r, 1.0f / s);
  float x[8];
  floats<IN>(r, x);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = div_odd(x[j], s);
  return make_uint2(q8_pack4<CT>(x[0], x[1], x[2], x[3]), q8_pack4<CT>(x[4], x[5], x[6], x[7]));
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

// What the kernels know of their (kv head, tensor).
template <int D, int IN, int CT>
struct Appender {
  static constexpr int LPR = D / 8;           // lanes per input row
  static constexpr int RPW = 32 / LPR;        // input rows per warp and pass
  static constexpr int CPR = D / 16;          // 16-byte chunks per cache row
  static constexpr int STEP = kAppWarps * RPW;   // rows of the CTA's pass
  const Q8AppendArgs& a;
  const void* src;
  uint8_t* pages;
  float* scales;
  int64_t ts, off;   // token stride; this lane's offset in a row of the head
  int h, col;
  // set: 0 .. Hkv - 1 the K heads, then the V heads
  __device__ __forceinline__ Appender(const Q8AppendArgs& args, int set) : a(args) {
    const bool is_v = set >= a.c.Hkv;
    h = is_v ? set - a.c.Hkv : set;
    src = is_v ? a.v : a.k;
    pages = is_v ? a.c.v : a.c.k;
    scales = reinterpret_cast<float*>(a.c.scales) + (is_v ? 1 : 0);
    ts = is_v ? a.v_token : a.k_token;
    col = (threadIdx.x % LPR) * 8;
    off = (int64_t)h * (is_v ? a.v_head : a.k_head) + col;
  }
  __device__ __forceinline__ bool valid(int slot) const { return q8_slot_ok(slot, a.c.num_pages, a.c.page_shift); }
  __device__ __forceinline__ uint32_t block_of(int slot) const { return (uint32_t)slot >> a.c.block_shift; }
  __device__ __forceinline__ uint32_t offset_in_block(int slot) const {
    return (uint32_t)slot & ((1u << a.c.block_shift) - 1u);
  }
  __device__ __forceinline__ uint32_t row_of(int slot) const {
    const int ps = a.c.page_shift;
    return q8_row((uint32_t)slot >> ps, (uint32_t)slot & ((1u << ps) - 1u), h, a.c.Hkv, ps);
  }
  __device__ __forceinline__ float* scale_at(uint32_t row) const { return scales + 2 * (size_t)(row >> a.c.block_shift); }
  __device__ __forceinline__ Raw8<IN> load(int t) const { return load8<IN>(src, (int64_t)t * ts + off); }
  __device__ __forceinline__ const char* address(int t) const {
    return static_cast<const char*>(src) + ((int64_t)t * ts + off) * (IN == kInF32 ? 4 : 2);
  }
  __device__ __forceinline__ int64_t token_bytes() const { return ts * (IN == kInF32 ? 4 : 2); }
  __device__ __forceinline__ void store_row(uint32_t row, const Raw8<IN>& r, float s) const {
    *reinterpret_cast<uint2*>(pages + (size_t)row * D + col) = pack8<IN, CT>(r, s);
  }
  __device__ __forceinline__ void store(int slot, const Raw8<IN>& r, float s) const { store_row(row_of(slot), r, s); }
  // the block's scale once the run's maximum is known; ratio: of the rows
  // before the run, 1 when they stay
  __device__ __forceinline__ float new_scale(uint32_t amax, uint32_t offset, float old, float& ratio) const {
    float s = pow2f(q8_scale_exp(amax, CT == kInt8));
    ratio = 1.0f;
    if (offset > 0) {
      if (s > old) ratio = old / s;   // exact: s is a power of two
      else if (old >= s) s = old;     // (a NaN old scale is dropped)
    }
    return s;
  }
  // rows [row0, row0 + n) times ratio, by `step` threads
  __device__ __forceinline__ void requant(uint32_t row0, int n, float ratio, int first, int step) const {
    for (int c = first; c < n * CPR; c += step) {
      uint4* p = reinterpret_cast<uint4*>(pages + (size_t)row0 * D) + c;
      *p = requant16<CT>(*p, ratio);
    }
  }
  // tokens of the run that starts at token t: to the last one before a token of
  // another block or kLook skipped ones (a whole warp)
  // the slots of tokens t .. t + have - 1 are in near
  __device__ int run_length(int t, uint32_t blk, const int* near = nullptr, int have = 0) const {
    int n = 1;
    for (;;) {
      const int i = n + (int)(threadIdx.x & 31), u = t + i;
      const int y = i < have ? near[i] : u < a.T ? __ldg(a.slots + u) : -1;
      const bool ok = valid(y), here = ok && block_of(y) == blk;
      uint32_t in = __ballot_sync(0xffffffffu, here);
      const uint32_t other = __ballot_sync(0xffffffffu, ok && !here);
      if (other) in &= (other & (0u - other)) - 1u;   // up to the first of another block
      if (in) n += 32 - __clz(in);
      if (!in || other) return n;
    }
  }
};

// One scale per row (S = 1): rows have nothing to do with one another.  The lanes
// of a row read it, find its maximum and scale, and write it, from registers;
// kRowBatch rows per lane under way together.  32K tokens of 8 kv heads, d = 128
// in bf16: 50 us (83 as runs of one row each).
constexpr int kRowBatch = 2;
template <int D, int IN, int CT>
__global__ void __launch_bounds__(kAppThreads) q8_append_rows_kernel(const Q8AppendArgs a) {
  using A = Appender<D, IN, CT>;
  constexpr int GROUPS = kAppThreads / A::LPR;
  const int sets = 2 * a.c.Hkv, total = a.T * sets;   // (31 bits: checked on the host)
  int u = blockIdx.x * (GROUPS * kRowBatch) + (int)threadIdx.x / A::LPR;
  const int lane = threadIdx.x & 31;
  const uint32_t row_lanes = ((1u << A::LPR) - 1u) << (lane / A::LPR * A::LPR);
  Raw8<IN> v[kRowBatch];
  int slot[kRowBatch], t[kRowBatch];
#pragma unroll
  for (int i = 0; i < kRowBatch; ++i, u += GROUPS) {   // neighbouring lanes: the heads of a token
    t[i] = u / sets;
    slot[i] = -1;
    if (u < total) {
      const A ap(a, u - t[i] * sets);
      slot[i] = __ldg(a.slots + t[i]);
      v[i] = ap.load(t[i]);
    }
  }
  u -= kRowBatch * GROUPS;
#pragma unroll
  for (int i = 0; i < kRowBatch; ++i, u += GROUPS) {
    const A ap(a, u - t[i] * sets);
    if (!ap.valid(slot[i])) {   // (the lanes of a row agree)
      if (slot[i] != -1) raise_error(a.err, kErrPage);
      continue;
    }
    MaxAcc<IN> acc;
    acc.add(v[i]);
    if (__any_sync(row_lanes, !acc.finite())) {
      acc.m = 0;
      acc.add_finite(v[i]);
    }
    const uint32_t row = ap.row_of(slot[i]);
    float ratio;
    const float s = ap.new_scale(__reduce_max_sync(row_lanes, acc.bits()), 0, 0.0f, ratio);
    if (lane % A::LPR == 0) *ap.scale_at(row) = s;
    *reinterpret_cast<uint2*>(ap.pages + (size_t)row * D + ap.col) = pack8_pow2<IN, CT>(v[i], 1.0f / s);
  }
}

// Few tokens (a decode step): a token to a warp, which looks around it.  Runs of
// up to kShortRun rows are the warp's, kept in registers; longer ones the CTA's.
template <int D, int IN, int CT>
__global__ void __launch_bounds__(kAppThreads) q8_append_kernel(const Q8AppendArgs a) {
  using A = Appender<D, IN, CT>;
  constexpr int PASSES = kShortRun / A::RPW;
  __shared__ int long_t[kAppWarps], long_n[kAppWarps], n_long;
  __shared__ uint32_t red[kAppWarps];
  const int sets = 2 * a.c.Hkv;
  const A ap(a, blockIdx.x % sets);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane / A::LPR;
  const int t = blockIdx.x / sets * kAppWarps + warp;
  const int slot = t < a.T ? __ldg(a.slots + t) : -1;
  const int back = t - 1 - lane, prev = back >= 0 && t < a.T ? __ldg(a.slots + back) : -1;
  if (tid == 0) n_long = 0;
  __syncthreads();
  if (ap.valid(slot)) {
    // a run starts here unless the last token before that is not skipped, kLook
    // back at most, is in the same block
    const uint32_t m = __ballot_sync(0xffffffffu, ap.valid(prev)), blk = ap.block_of(slot);
    const bool starts = !m || __shfl_sync(0xffffffffu, ap.block_of(prev), __ffs(m) - 1) != blk;
    const int n = starts ? ap.run_length(t, blk) : 0;
    if (n > kShortRun) {
      if (lane == 0) {
        const int i = atomicAdd(&n_long, 1);
        long_t[i] = t;
        long_n[i] = n;
      }
    } else if (n > 0) {
      Raw8<IN> v[PASSES];
      int at[PASSES];
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int i = p * A::RPW + sub;
        at[p] = i < n ? __ldg(a.slots + t + i) : -1;
        if (ap.valid(at[p])) v[p] = ap.load(t + i);
      }
      MaxAcc<IN> acc;
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
        if (ap.valid(at[p])) acc.add_finite(v[p]);
      const uint32_t offset = ap.offset_in_block(slot), row = ap.row_of(slot);
      float* sp = ap.scale_at(row);
      const float old = offset ? *sp : 0.0f;
      const uint32_t am = __reduce_max_sync(0xffffffffu, acc.bits());
      float ratio;
      const float s = ap.new_scale(am, offset, old, ratio);
      __syncwarp();
      if (lane == 0) *sp = s;
      if (ratio != 1.0f) ap.requant(row - offset, offset, ratio, lane, 32);
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
        if (ap.valid(at[p])) ap.store(at[p], v[p], s);
    }
  } else if (slot != -1 && lane == 0) {   // (-1: a padding token)
    raise_error(a.err, kErrPage);
  }
  __syncthreads();

  const int runs = n_long, i0 = warp * A::RPW + sub;
  for (int q = 0; q < runs; ++q) {
    const int rt = long_t[q], n = long_n[q];
    MaxAcc<IN> acc;
    for (int i = i0; i < n; i += A::STEP)
      if (ap.valid(__ldg(a.slots + rt + i))) acc.add_finite(ap.load(rt + i));
    const int first = __ldg(a.slots + rt);
    const uint32_t offset = ap.offset_in_block(first), row = ap.row_of(first);
    float* sp = ap.scale_at(row);
    const float old = offset ? *sp : 0.0f;
    uint32_t am = __reduce_max_sync(0xffffffffu, acc.bits());
    if (lane == 0) red[warp] = am;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppWarps; ++w) am = max(am, red[w]);
    float ratio;
    const float s = ap.new_scale(am, offset, old, ratio);
    if (ratio != 1.0f) ap.requant(row - offset, offset, ratio, tid, kAppThreads);
    for (int i = i0; i < n; i += A::STEP) {   // (the rows come from L1 or L2)
      const int y = __ldg(a.slots + rt + i);
      if (ap.valid(y)) ap.store(y, ap.load(rt + i), s);
    }
    __syncthreads();   // every thread has read the old scale (and red) of this run
    if (tid == 0) *sp = s;
  }
}

// Many tokens (prompts): one, two or four warps take a tile's runs of one (kv
// head, tensor), all at once whatever their lengths are; the CTA's warps take
// neighbouring heads of the same tile.  Every row from the first start to the
// end of the last run is read into shared memory, where it waits for its run's
// scale: the maxima are joined per run (integer maxima: order does not matter),
// then the rows are rounded and written.  (A window that does not fit, as at a
// border of two long runs, comes in chunks, all but one of them twice.)
// Instructions bound this kernel as much as bytes do: a warp's fixed part, run
// one after the other, takes as long as its rows.  So a tile of whole blocks in
// order, the rule in a prompt, is told by one test per token and needs none of
// the search for runs (32K tokens: 42.8 us with the search, 35.8 without), a
// CTA has four warps (two: 53 us) and a set as few as hold its rows (two where
// one does: 49 us).
constexpr int kTileWarps = 4;
constexpr int kTileThreads = kTileWarps * 32;
constexpr int kKept = 16384;   // bytes of shared memory per warp: three CTAs, 192 KB under way per SM

template <int D, int IN, int CT>
__global__ void __launch_bounds__(kTileThreads, 5)
    q8_append_tiled_kernel(const Q8AppendArgs a, int tile, int groups, int wps, int hold) {
  using A = Appender<D, IN, CT>;
  constexpr int PIECES = (int)sizeof(Raw8<IN>) / 16;
  extern __shared__ __align__(128) char kept[];   // [kTileWarps][hold][PIECES * 512], then:
  uint2* const rows = reinterpret_cast<uint2*>(kept + kTileWarps * hold * PIECES * 512);   // [2 tile + 16] row of the token's
                                                  // slot for head 0 (kNoRow: skipped), and its run
  uint32_t* const run_top = reinterpret_cast<uint32_t*>(rows + 2 * tile + 16);   // [kTileWarps][tile] largest magnitude
                                                  // of a run, then its scale, as bits
  int* const sl = reinterpret_cast<int*>(run_top + kTileWarps * tile);   // [kLook + 2 tile] slots of tokens t0 - kLook ..
  __shared__ uint32_t lead[kMaxTile / 32];        // bit x: a run starts at token t0 + x
  __shared__ int flags[kTileWarps][2];            // of a set: an infinity or NaN met; a scale that is not easy (below)
  __shared__ int end_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int mine = warp / wps, part = warp - mine * wps;   // the warp's set in the CTA, and its part of the rows
  const int set = blockIdx.x % groups * (kTileWarps / wps) + mine;
  const bool active = set < 2 * a.c.Hkv;
  const A ap(a, min(set, 2 * a.c.Hkv - 1));
  const int t0 = blockIdx.x / groups * tile;
  const int ps = a.c.page_shift;
  // a set's warps go on by themselves once they know their runs
  auto sync_set = [&]() {
    if (wps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;\n" ::"r"(1 + mine), "r"(wps * 32) : "memory");
  };
  auto any_of_set = [&](bool p, int which) -> bool {   // (a barrier of the set too)
    p = __any_sync(0xffffffffu, p);
    if (wps > 1) {
      if (p && lane == 0) flags[mine][which] = 1;
      sync_set();
      return flags[mine][which] != 0;
    }
    __syncwarp();
    return p;
  };
  // the warp's passes: rows sub, sub + step ..
  const int step = wps * A::RPW, sub = part * A::RPW + lane / A::LPR;
  uint32_t* const top = run_top + mine * tile;
  const uint32_t head_row = (uint32_t)ap.h << ps;
  uint8_t* const pages = ap.pages + (size_t)head_row * D + ap.col;
  // The lanes of a row copy 16 bytes next to one another (whole sectors), which
  // for fp32 are not all the columns that they work on: kept_at finds those,
  // 32 bytes of a row, of which every other four lanes read the second half
  // first, so that eight lanes meet all banks.
  const int l = lane % A::LPR;
  const char* const home = kept + warp * hold * PIECES * 512 + lane * 16;
  const uint32_t to = smem_u32(home);
  const bool swap = l & 4;
  const int own = PIECES == 1 ? 0 : (2 * l >= A::LPR ? 512 + (l - A::LPR) * 16 : l * 16) + (swap ? 16 : 0);
  auto copy = [&](int q, const char* from, int bytes) {
#pragma unroll
    for (int w = 0; w < PIECES; ++w)
      cp_async_16(to + (q * PIECES + w) * 512, from - (PIECES - 1) * l * 16 + w * A::LPR * 16, bytes);
  };
  auto kept_at = [&](int q) -> Raw8<IN> {
    Raw8<IN> r;
    const char* const at = home + own + q * PIECES * 512;
    if constexpr (PIECES == 1) {
      r.w[0] = *reinterpret_cast<const uint4*>(at);
    } else {
      const uint4 x = *reinterpret_cast<const uint4*>(at), y = *reinterpret_cast<const uint4*>(at + (swap ? -16 : 16));
      r.w[0] = swap ? y : x;
      r.w[1] = swap ? x : y;
    }
    return r;
  };

  // Whole blocks, in order, from token x_s on (a prompt, once past its first
  // block): their rows follow one another, and there is no earlier scale.
  const int shift = a.c.block_shift, block = 1 << shift;
  {
    const int x_s = (int)((0u - (uint32_t)__ldg(a.slots + t0)) & (uint32_t)(block - 1));
    bool whole = t0 + x_s + tile <= a.T && block >= step && tile <= hold * step;
    if (whole)
      for (int x = tid; x < x_s + tile; x += kTileThreads) {   // (those before x_s go on with a run from before)
        const int slot = __ldg(a.slots + t0 + x), before = t0 + x > 0 ? __ldg(a.slots + t0 + x - 1) : -1;
        const int o = (int)ap.offset_in_block(slot);
        whole &= ap.valid(slot) && o == ((x - x_s) & (block - 1)) && (o == 0 || slot - 1 == before);
        if (whole && x >= x_s && o == 0)
          rows[(x - x_s) >> shift].x = q8_row((uint32_t)slot >> ps, (uint32_t)slot & ((1u << ps) - 1u), 0, a.c.Hkv, ps);
      }
    if (part == 0)
      for (int r = lane; r < tile >> shift; r += 32) top[r] = 0;
    if (__syncthreads_and(whole)) {
      if (!active) return;
      const char* from = ap.address(t0 + x_s + sub);
      const int64_t skip = step * ap.token_bytes();
      const int n = block / step, runs = tile >> shift;
#pragma unroll 4
      for (int q = 0; q < tile / step; ++q, from += skip) copy(q, from, 16);
      cp_async_commit();
      cp_async_wait<0>();
      __syncwarp();
      uint32_t odd = 0;   // bit r: run r (of 32 at most: a step is two rows) has an infinity or NaN in this warp's rows
      for (int r = 0; r < runs; ++r) {
        MaxAcc<IN> acc;
#pragma unroll 4
        for (int q = r * n; q < (r + 1) * n; ++q) acc.add(kept_at(q));
        if (__any_sync(0xffffffffu, !acc.finite())) {
          odd |= 1u << r;
          acc.m = 0;
          for (int q = r * n; q < (r + 1) * n; ++q) acc.add_finite(kept_at(q));
        }
        const uint32_t m = __reduce_max_sync(0xffffffffu, acc.bits());
        if (lane == 0) atomicMax(top + r, m);
      }
      sync_set();
      for (int r = 0; r < runs; ++r) {
        float ratio;
        const float s = ap.new_scale(top[r], 0, 0.0f, ratio), inv = 1.0f / s;
        const uint32_t row = rows[r].x;
        if (part == 0 && lane == 0) *ap.scale_at(row + head_row) = s;
        uint8_t* out = pages + (size_t)(row + sub) * D;
        if (CT == kInt8 && (odd >> r & 1u)) {
          for (int q = r * n; q < (r + 1) * n; ++q, out += step * D)
            *reinterpret_cast<uint2*>(out) = pack8_pow2<IN, CT>(kept_at(q), inv);
        } else {
#pragma unroll 4
          for (int q = r * n; q < (r + 1) * n; ++q, out += step * D)
            *reinterpret_cast<uint2*>(out) = pack8_finite<IN, CT>(kept_at(q), inv);
        }
      }
      return;
    }
  }
  for (int x = tid; x < kLook + 2 * tile; x += kTileThreads) {
    const int t = t0 - kLook + x;
    const int slot = t >= 0 && t < a.T ? __ldg(a.slots + t) : -1;
    const bool ok = ap.valid(slot);
    sl[x] = slot;
    if (x >= kLook) {
      rows[x - kLook].x = ok ? q8_row((uint32_t)slot >> ps, (uint32_t)slot & ((1u << ps) - 1u), 0, a.c.Hkv, ps) : kNoRow;
      if (slot != -1 && !ok && x < kLook + tile) raise_error(a.err, kErrPage);
    }
  }
  __syncthreads();
  for (int x = tid; x < tile; x += kTileThreads) {   // (tiles are whole warps)
    bool starts = rows[x].x != kNoRow;
    if (starts)
      for (int k = 1; k <= kLook; ++k)
        if (ap.valid(sl[kLook + x - k])) {
          starts = ap.block_of(sl[kLook + x - k]) != ap.block_of(sl[kLook + x]);
          break;
        }
    const uint32_t m = __ballot_sync(0xffffffffu, starts);
    if (lane == 0) lead[x / 32] = m;
  }
  __syncthreads();
  int x_s = tile, x_l = 0, runs = 0;   // first and last start, and how many
  for (int w = 0; w < tile / 32; ++w) {
    const uint32_t m = lead[w];
    // a token's run: the starts up to it, less 1
    if (w % kTileWarps == warp) rows[32 * w + lane].y = runs + __popc(m & (0xffffffffu >> (31 - lane))) - 1;
    if (m) {
      x_s = min(x_s, 32 * w + __ffs(m) - 1);
      x_l = 32 * w + 31 - __clz(m);
      runs += __popc(m);
    }
  }
  if (runs == 0) return;   // (the same for every warp)
  for (int x = tile + tid; x < 2 * tile; x += kTileThreads) rows[x].y = runs - 1;   // (what is left of the last)
  if (warp == 0) {         // the last run may end behind the tile
    const int n = ap.run_length(t0 + x_l, ap.block_of(sl[kLook + x_l]), sl + kLook + x_l, 2 * tile - x_l);
    if (lane == 0) end_s = x_l + n;
  }
  if (part == 0) {
    for (int r = lane; r < runs; r += 32) top[r] = 0;
    if (lane < 2) flags[mine][lane] = 0;
  }
  __syncthreads();
  if (!active) return;
  const int end = end_s;
  const int first = x_s + sub;
  const int passes = (end - x_s + step - 1) / step;   // rows of a lane
  // row of token t0 + x (past the window only where many are skipped)
  auto row_at = [&](int x) -> uint32_t {
    if (x >= end) return kNoRow;
    if (x < 2 * tile) return rows[x].x;
    const int slot = __ldg(a.slots + t0 + x);
    return ap.valid(slot) ? q8_row((uint32_t)slot >> ps, (uint32_t)slot & ((1u << ps) - 1u), 0, a.c.Hkv, ps) : kNoRow;
  };
  auto run_of = [&](int x) -> int { return (int)rows[min(x, tile - 1)].y; };
  bool plain = end <= 2 * tile;   // no row is skipped: no test per row
  for (int x = x_s + lane; plain && x < end; x += 32) plain = rows[x].x != kNoRow;
  plain = __all_sync(0xffffffffu, plain);
  // rows come to shared memory hold passes at a time
  const int chunks = (passes + hold - 1) / hold;
  int here = -1;                  // the chunk that is in shared memory
  auto fetch = [&](int c) -> int {   // returns the chunk's passes
    const int p0 = c * hold, n = min(hold, passes - p0);
    if (c == here) return n;
    here = c;
    __syncwarp();
    if (plain) {
      const char* from = ap.address(t0 + first + p0 * step);
      const int64_t skip = step * ap.token_bytes();
#pragma unroll 4
      for (int q = 0; q < n - 1; ++q, from += skip) copy(q, from, 16);
      copy(n - 1, ap.address(t0 + min(first + (p0 + n - 1) * step, end - 1)), 16);   // (past the end the last row again)
    } else {
      for (int q = 0; q < n; ++q) {   // zeros for skipped rows and past the end
        const int x = first + (p0 + q) * step;
        const bool have = row_at(x) != kNoRow;
        copy(q, ap.address(have ? t0 + x : t0), have ? 16 : 0);
      }
    }
    cp_async_commit();
    cp_async_wait<0>();
    __syncwarp();
    return n;
  };
  // f(chunk's first pass, its passes) over all rows, the chunk that is here first
  auto sweep = [&](auto&& f) {
    const int c0 = max(here, 0), dir = c0 > 0 ? -1 : 1;
    for (int i = 0, c = c0; i < chunks; ++i, c += dir) {
      const int n = fetch(c);
      f(c * hold, n);
    }
  };
  // f(values, token) of every row; skipped ones are zeros
  auto for_rows = [&](auto&& f) {
    sweep([&](int p0, int n) {
#pragma unroll 2
      for (int q = 0; q < n; ++q) f(kept_at(q), first + (p0 + q) * step);
    });
  };
  // maxima: a lane keeps its own while its rows stay in one run; the lanes of a
  // row (which change runs together) join theirs before the shared maximum
  const uint32_t row_lanes = ((1u << A::LPR) - 1u) << (lane / A::LPR * A::LPR);
  bool odd = false;                         // an infinity or NaN was met
  auto maxima = [&](bool finite_only) {
    MaxAcc<IN> acc;
    int cur = run_of(first);
    auto flush = [&]() {
      odd |= !acc.finite();
      const uint32_t m = __reduce_max_sync(row_lanes, acc.bits());
      if (lane % A::LPR == 0) atomicMax(top + cur, m);
      acc.m = 0;
    };
    if (plain && !finite_only) {
      sweep([&](int p0, int n) {   // (the last pass may be past the end: the last row again, of its run)
        const uint2* row = rows + first + p0 * step;
#pragma unroll 2
        for (int q = 0; q < n; ++q, row += step) {
          const int r = q < n - 1 ? (int)row->y : run_of(min(first + (p0 + q) * step, end - 1));
          if (r != cur) {
            flush();
            cur = r;
          }
          acc.add(kept_at(q));
        }
      });
    } else {
      for_rows([&](const Raw8<IN>& v, int x) {
        const int r = run_of(x);
        if (r != cur) {
          flush();
          cur = r;
        }
        if (finite_only) acc.add_finite(v);
        else acc.add(v);
      });
    }
    flush();
  };
  maxima(false);
  if (any_of_set(odd, 0)) {   // once more without them
    if (part == 0)
      for (int r = lane; r < runs; r += 32) top[r] = 0;
    sync_set();
    maxima(true);
    sync_set();
  }
  // scales, a lane per run; rows before a run whose scale grew, by the warp
  bool easy = true;   // every scale's reciprocal is a normal power of two
  if (part == 0) {
    for (int x0 = 0; x0 < tile; x0 += 32) {
      const int x = x0 + lane;
      const bool starts = lead[x0 / 32] >> lane & 1u;
      float ratio = 1.0f;
      uint32_t row = 0, offset = 0;
      if (starts) {   // token t0 + x starts a run
        const int r = (int)rows[x].y;
        offset = ap.offset_in_block(sl[kLook + x]);
        row = rows[x].x + head_row;
        float* sp = ap.scale_at(row);
        const float s = ap.new_scale(top[r], offset, offset ? *sp : 0.0f, ratio);
        *sp = s;
        top[r] = __float_as_uint(s);
        easy &= is_pow2(s) && s <= kMaxEasy;
      }
      for (uint32_t grew = __ballot_sync(0xffffffffu, ratio != 1.0f); grew; grew &= grew - 1) {
        const int l = __ffs(grew) - 1;
        const uint32_t n = __shfl_sync(0xffffffffu, offset, l);
        ap.requant(__shfl_sync(0xffffffffu, row, l) - n, (int)n, __shfl_sync(0xffffffffu, ratio, l), lane, 32);
      }
    }
  }
  if (any_of_set(!easy, 1)) {
    for_rows([&](const Raw8<IN>& v, int x) {
      const uint32_t r = row_at(x);
      if (r != kNoRow) ap.store_row(r + head_row, v, __uint_as_float(top[run_of(x)]));
    });
  } else if (plain) {
    sweep([&](int p0, int n) {
      const uint2* row = rows + first + p0 * step;
#pragma unroll 4
      for (int q = 0; q < n - 1; ++q, row += step) {
        const uint2 r = *row;
        // 1 / s by its exponent: s = 2^e, -100 <= e <= 126
        const float inv = __uint_as_float((254u << 23) - top[r.y]);
        *reinterpret_cast<uint2*>(pages + (size_t)r.x * D) = pack8_pow2<IN, CT>(kept_at(q), inv);
      }
      if (first + (p0 + n - 1) * step < end)
        *reinterpret_cast<uint2*>(pages + (size_t)row->x * D) =
            pack8_pow2<IN, CT>(kept_at(n - 1), 1.0f / __uint_as_float(top[row->y]));
    });
  } else {
    for_rows([&](const Raw8<IN>& v, int x) {
      const uint32_t r = row_at(x);
      const uint2 y = pack8_pow2<IN, CT>(v, 1.0f / __uint_as_float(top[run_of(x)]));
      if (r != kNoRow) *reinterpret_cast<uint2*>(pages + (size_t)r * D) = y;
    });
  }
}

// ------------------------------------------------------------------ gather
//
// out[b, h, j] = byte x scale, rounded once to the output type, for j <
// kv_lens[b]; later rows are not touched.  Bound by HBM writes (1 byte read and
// 2 or 4 written per element): every thread turns 8 bytes into one or two
// 16-byte stores, so a warp writes whole 512-byte stretches.  Eight 32K
// sequences of 8 kv heads, d = 128 to bf16: 292 us for 0.54 GB read and 1.07 GB
// written, where writing alone takes 275 us.  Four rows under way per thread:
// two take 310 us, eight 407.

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
  // rows by themselves; a token per warp as long as that is not many CTAs, as
  // in a decode step; else tiles of a block's size, so that a prompt's runs
  // start one to a tile
  const int sets = 2 * a.c.Hkv;
  if (a.c.block_shift == 0) {
    const int rows = kAppThreads / (D / 8) * kRowBatch;
    const int64_t ctas = ((int64_t)a.T * sets + rows - 1) / rows;
    return launch_ex(q8_append_rows_kernel<D, IN, CT>, dim3((unsigned)ctas), dim3(kAppThreads), 0, st, false, 1, a);
  }
  const int64_t few = ((int64_t)a.T + kAppWarps - 1) / kAppWarps * sets;
  if (few <= kFewCtas)
    return launch_ex(q8_append_kernel<D, IN, CT>, dim3((unsigned)few), dim3(kAppThreads), 0, st, false, 1, a);
  // as many warps to a (head, tensor) as hold a tile's rows: a block's where a
  // run is a tile, else the tile's and those of a run that reaches over its end.
  // (128 KB of rows, as in fp32 blocks of 256 at d = 128, are twice what the four
  // hold: they come in two chunks, one of them twice, and never as whole blocks.
  // 32K tokens of 8 kv heads take 89 us then, and 62 in blocks of 128.)
  constexpr int ROW = D * (IN == kInF32 ? 4 : 2), PASS = IN == kInF32 ? 1024 : 512;   // bytes of a row, and a warp's pass
  const int block = 1 << a.c.block_shift, tile = min(max(block, 64), kMaxTile);
  const int window = (block >= tile ? tile : tile + block) * ROW;
  const int wps = window <= kKept ? 1 : window <= 2 * kKept ? 2 : 4;
  const int hold = min(window / wps, kKept) / PASS;
  const int per_cta = kTileWarps / wps, groups = (sets + per_cta - 1) / per_cta;
  const int64_t ctas = ((int64_t)a.T + tile - 1) / tile * groups;
  const auto fn = q8_append_tiled_kernel<D, IN, CT>;
  const size_t smem = (size_t)kTileWarps * hold * PASS + (2 * tile + 16) * 8 + kTileWarps * tile * 4 + (kLook + 2 * tile) * 4;
  const cudaError_t e = ensure_func_attrs(reinterpret_cast<const void*>(fn), smem, false);
  if (e != cudaSuccess) return e;
  return launch_ex(fn, dim3((unsigned)ctas), dim3(kTileThreads), smem, st, false, 1, a, tile, groups, wps, hold);
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
  return launch_ex(page_tables_kernel, dim3(blocks < 1 ? 1 : blocks > kTabCtas ? kTabCtas : blocks), dim3(kTabThreads), 0, stream,
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
