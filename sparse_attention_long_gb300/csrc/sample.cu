// Sampling of one token per row of logits (dsa_sample): temperature, min-p, top-k,
// top-p, and a draw by a given uniform number.
//
// All three cuts keep a run of the tokens in the order (logit descending, index
// ascending), so a cut is a logit and a number of tokens that have exactly this logit,
// lowest index first.  min-p gives its logit outright, from the maximum.
//
// Borders between tokens lie dense in a large vocabulary, so fp32 sums would draw
// neighbours of the right token now and then (131,072 borders, sums off by 1e-7: one row in
// fifty).  Weights are computed to 2^-29 of themselves and summed as integers, in units of 2^-44
// of the largest one or finer: sums are exact, whatever their order, and so is what follows
// from them.
//
// A thread-block cluster per row, as many CTAs as hold it in shared memory, 32 KB each
// (more for a few rows).  Then one of
//  - a list, where few tokens can be kept: ceil(k / CTAs) of a CTA's threads have a logit that
//    reaches a number, so k of the row do, and few more than k reach the smallest such
//    number; or those that min-p keeps; or, of logits in the thousands for their temperature,
//    those that weigh anything.  CTA 0 gets them and does the rest;
//  - nothing to cut: one pass of weights;
//  - a histogram of distances to the maximum in 1/128 powers of two: it tells the bin of the
//    k-th logit, and by the bins' middles about where top-p's border lies.  One pass of
//    weights sums exactly what lies above and below; the few logits at the border go to CTA 0,
//    which finds the cuts;
//  - bisection over all logits, where too many lie at a cut (equal ones, say);
// and a draw: the CTA, warp, step, thread and token at which the mass passes its part.
// With a row for each SM or more, a row that needs but a list is read by one CTA
// (stream_kernel), which keeps nothing of it but the candidates.
//
// Measured (us, calls back to back; in brackets the logits' bytes at 6.8 TB/s): one row of
// 32,001 fp32, top-k and top-p 7 (0.02); 768 rows of 64,000 bf16, top-k and top-p 33 (14.5), of
// which stream_kernel 30; 256 rows of 131,071 bf16 at a temperature 50 (9.9), fp32 69 (19.7); 48 rows of
// 64,000 fp32, top-p alone and large nuclei 30 (1.8); 64 rows of 131,071 bf16, top-p alone 46, a
// mixture 29 to 34 (2.5), top-k 2,000 51, all at a temperature of 0.01 13, at 0 10.
// Bound: the first by the latency of loads and two cluster barriers; stream_kernel by
// instructions and the phases without loads (settings, bounds, the end); a pass of weights by
// instructions (20 per bf16 logit, 25 else; 2.4 per cycle and SM); the histogram's path by
// such a pass and its seven cluster barriers, 1 us each with what they wait for.
#include <float.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "bound.h"
#include "dsa_common.cuh"

namespace dsa {

bool ext_dev_ctx(DevCtx* c);

namespace sample {

constexpr int kMaxCluster = 8;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kVec = 8;                            // consecutive logits of a thread
constexpr int kMaxVocab = 1 << 18;
constexpr int kList = 2048;                        // tokens that one CTA can order, 2^n
constexpr int kCounted = 256;                      // up to so many by counting, or, of logits alone,
constexpr int kListed = 512;                       // so many
constexpr int kSmallK = 1024;                      // top_k up to which candidates are listed at first

typedef unsigned long long u64;

struct Args {
  int rows, vocab, requests, bits;                 // vocab <= 2^bits
  long long ld;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t *top_k, *index;
  int32_t* token;
  float* prob;
};

// 2^31 * 2^(j / 1024)
struct Powers {
  uint32_t at[1024];
  constexpr Powers() : at() {
    for (int j = 0; j < 1024; ++j) {
      const double x = j / 1024.0 * 0.69314718055994530942;
      double term = 1, sum = 1;
      for (int k = 1; k < 20; ++k) {
        term *= x / k;
        sum += term;
      }
      at[j] = (uint32_t)(sum * 2147483648.0 + 0.5);
    }
  }
};
__device__ __align__(16) const Powers kPowers{};

__device__ __forceinline__ void store_remote(u64* local, uint32_t rank, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa_shared(smem_u32(local), rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void store_remote(uint32_t* local, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(local), rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void store_remote(float* local, uint32_t rank, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(smem_u32(local), rank)), "f"(v) : "memory");
}
__device__ __forceinline__ float load_remote(const float* local, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_u32(local), rank)) : "memory");
  return v;
}
__device__ __forceinline__ float ordered_value(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? u ^ 0x80000000u : ~u);
}
// The type's values as consecutive integers, and back; `up`: of the least value that is not below x.
template <typename T>
struct Grid;
template <>
struct Grid<float> {
  static __device__ __forceinline__ uint32_t up(float x) { return ordered_key(x); }
  static __device__ __forceinline__ float value(uint32_t k) { return ordered_value(k); }
};
template <>
struct Grid<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t up(float x) {
    const uint32_t k = ordered_key(x);
    return (k & 0x80000000u) ? (k + 0xFFFFu) >> 16 : k >> 16;
  }
  static __device__ __forceinline__ float value(uint32_t k) {
    return ordered_value((k & 0x8000u) ? k << 16 : (k << 16) | 0xFFFFu);
  }
};

// the largest value of the type below x (-0 has a number of its own, but is no other value than 0)
template <typename T>
__device__ __forceinline__ float next_below(float x) {
  const uint32_t k = Grid<T>::up(x) - 1;
  return Grid<T>::value(k == Grid<T>::up(0.f) - 1 ? k - 1 : k);
}

// two floats in one register pair
__device__ __forceinline__ u64 pair(float lo, float hi) {
  u64 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void halves(u64 v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
  u64 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// w = 2^-x as a whole number of units, x = (max - l) * log2(e) / temperature.  Two logits
// at once: max - l = d + e and d * scale = x + f without error, -x = q + r with q a
// multiple of 2^-10, 2^q from the table and 2^r by a series.  Off by 2^-29 of itself
// (the table by half a step of 2^-31, r by as much, the series without the cube of |r| < 2^-9 by 0.4
// 2^-30, the product below by one step of 2^-30 at most) and the last unit.
struct Weight {
  float max, hi, lo;                               // log2(e) / temperature in two floats
  int shift;                                       // the largest weight is 2^(62 - shift) units

  __device__ __forceinline__ u64 of(bool counts, uint32_t y, float z, const uint32_t* __restrict__ powers) const {
    // (what is further down, the exponent of 2 out of reach, weighs nothing)
    const uint32_t p = counts && __uint_as_float(y) > kY - 62.5f + (float)shift ? powers[y & 1023u] : 0u;
    const uint32_t w = __umulhi(p, __float_as_uint(z) - __float_as_uint(kZ) + (1u << 31));  // 2^30 * 2^(q's fraction + r)
    return ((u64)w << 32) >> (((shift << 10) + 1023 + __float_as_uint(kY) - y) >> 10 & 63u);
  }
  static constexpr float kY = 12288.f;             // 1.5 * 2^13: steps of 2^-10
  static constexpr float kZ = 0.005859375f;        // 1.5 * 2^-8: steps of 2^-31, for |r| below 2^-9
  static constexpr float kLn2 = 0.693147181f, kHalfLn2Sq = 0.240226507f;
  // whether l0 and l1 count; y0, y1: bits of the step numbers, see bin_at
  __device__ __forceinline__ void two(float l0, float l1, bool counts0, bool counts1, u64& w0, u64& w1, uint32_t& y0,
                                      uint32_t& y1, const uint32_t* __restrict__ powers) const {
    const u64 m = pair(max, max), nm = pair(-max, -max), h = pair(hi, hi), nh = pair(-hi, -hi), one = pair(-1.f, -1.f);
    const u64 nl = pair(-l0, -l1);
    const u64 d = add2(m, nl), t = add2(d, nm);
    const u64 e = add2(fma2(fma2(t, one, d), one, m), fma2(t, one, nl));
    const u64 nx = mul2(d, nh);
    const u64 f = fma2(d, pair(lo, lo), fma2(e, h, fma2(d, h, nx)));
    const u64 y = add2(nx, pair(kY, kY)), q = add2(y, pair(-kY, -kY));
    const u64 r = fma2(f, one, fma2(q, one, nx));
    const u64 z = fma2(r, fma2(r, pair(kHalfLn2Sq, kHalfLn2Sq), pair(kLn2, kLn2)), pair(kZ, kZ));
    float a0, a1, z0, z1;
    halves(y, a0, a1), halves(z, z0, z1);
    w0 = of(counts0, __float_as_uint(a0), z0, powers), w1 = of(counts1, __float_as_uint(a1), z1, powers);
    y0 = __float_as_uint(a0), y1 = __float_as_uint(a1);
  }
  __device__ __forceinline__ u64 operator()(float l, const uint32_t* __restrict__ powers) const {
    u64 a, b;
    uint32_t y;
    two(l, l, true, false, a, b, y, y, powers);
    return a;
  }
  __device__ __forceinline__ uint32_t step(float l) const {
    return __float_as_uint(__fadd_rn(__fmul_rn(__fsub_rn(max, l), -hi), kY));
  }
};

// The same for bf16 logits that are not too large, with fewer steps: a logit's eight bits
// times sixteen of the scale is exact, so l * scale - max * scale needs no exact
// difference first.  (20 instead of 25 instructions per logit: 256 rows of 131,071 51 us
// instead of 59, with top-p alone 143 instead of 169.)
struct DirectWeight {
  float high, low, from, left;                     // scale in 16 bits and the rest; kY - max * scale in two parts
  int shift;
  __device__ __forceinline__ explicit DirectWeight(const Weight& w) {
    high = __uint_as_float((__float_as_uint(w.hi) + 0x80u) & 0xFFFFFF00u);
    low = __fadd_rn(__fsub_rn(w.hi, high), w.lo);
    const float t = __fmul_rn(w.max, high), y = __fadd_rn(t, Weight::kY), q = __fsub_rn(y, Weight::kY);
    from = __fsub_rn(Weight::kY, q);               // both multiples of 2^-10 below 2^14: exact
    left = __fmaf_rn(-w.max, low, __fsub_rn(q, t));
    shift = w.shift;
  }
  __device__ __forceinline__ void two(float l0, float l1, bool counts0, bool counts1, u64& w0, u64& w1, uint32_t& s0,
                                      uint32_t& s1, const uint32_t* __restrict__ powers) const {
    const u64 l = pair(l0, l1), t = mul2(l, pair(high, high));
    const u64 y = add2(t, pair(from, from)), q = add2(y, pair(-from, -from));
    const u64 r = add2(fma2(q, pair(-1.f, -1.f), t), fma2(l, pair(low, low), pair(left, left)));
    const u64 z = fma2(r, fma2(r, pair(Weight::kHalfLn2Sq, Weight::kHalfLn2Sq), pair(Weight::kLn2, Weight::kLn2)),
                       pair(Weight::kZ, Weight::kZ));
    float y0, y1, z0, z1;
    halves(y, y0, y1), halves(z, z0, z1);
    const Weight g{0.f, 0.f, 0.f, shift};
    w0 = g.of(counts0, __float_as_uint(y0), z0, powers), w1 = g.of(counts1, __float_as_uint(y1), z1, powers);
    s0 = __float_as_uint(y0), s1 = __float_as_uint(y1);
  }
  __device__ __forceinline__ u64 operator()(float l, const uint32_t* __restrict__ powers) const {
    u64 a, b;
    uint32_t y;
    two(l, l, true, false, a, b, y, y, powers);
    return a;
  }
  __device__ __forceinline__ uint32_t step(float l) const { return __float_as_uint(__fadd_rn(__fmul_rn(l, high), from)); }
};

// A row's weights: all of one kind, whatever else is done for the row.
template <typename T>
struct RowWeight {
  static constexpr bool kDirect = sizeof(T) == 2;
  Weight plain;
  typename std::conditional<kDirect, DirectWeight, Weight>::type fine;
  bool fits;                                       // (false: plain)
  __device__ __forceinline__ explicit RowWeight(const Weight& w)
      : plain(w), fine(w), fits(!kDirect || fabsf(w.max) * w.hi < 2000.f) {}
  __device__ __forceinline__ u64 operator()(float l, const uint32_t* __restrict__ powers) const {
    return fits ? fine(l, powers) : plain(l, powers);
  }
};

// p * z rounded up or down to an integer, for a float 0 <= p <= 1
__device__ __forceinline__ u64 scaled(float p, u64 z, bool up) {
  int e;
  const float m = frexpf(p, &e);                   // p = m * 2^e, m in [1/2, 1)
  const u64 i = (u64)(m * 16777216.f);             // exact
  const int sh = 24 - e;                           // p = i * 2^-sh, sh >= 23
  const u64 lo = i * z, hi = __umul64hi(i, z);
  if (sh >= 128) return up && (lo | hi) ? 1 : 0;
  u64 q, left;
  if (sh >= 64) {
    const int r = sh - 64;
    q = hi >> r;
    left = lo | (r ? hi << (64 - r) : 0);
  } else {
    q = (lo >> sh) | (hi << (64 - sh));            // below 2^64: the result is at most z
    left = lo << (64 - sh);
  }
  return q + (up && left ? 1 : 0);
}

__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

struct __align__(16) Shared {
  uint32_t powers[1024];
  double far;                                      // how far below the largest logit min-p goes
  u64 warp_sum[kWarps];
  uint32_t warp_count[kWarps];
  u64 sum[2][kMaxCluster], more[2][kMaxCluster];   // of every CTA of the cluster, two exchanges deep
  uint32_t count[2][kMaxCluster];
  u64 scan_sum[kWarps];
  u64 note;                                        // of CTA 0 to all
  float warp_mass[kWarps], z;
  int bin[3];
  uint32_t rank_in, listed;
  int who;                                         // where the token lies: warp, kept mass before it, ...
  uint32_t seen;
  u64 before, target, total;
};

__device__ __forceinline__ void load_powers(Shared& s) {
  static_assert(kThreads == 256, "four powers per thread");
  reinterpret_cast<uint4*>(s.powers)[threadIdx.x] = reinterpret_cast<const uint4*>(kPowers.at)[threadIdx.x];
}

// What a CTA sums, and what the cluster does.  An exchange's numbers stay readable until
// the next but one.
struct Team {
  Shared& s;
  int rank, size, turn;
  __device__ __forceinline__ void exchange(u64 sum, uint32_t count) {
    turn ^= 1;
    if ((int)threadIdx.x < size) {
      store_remote(&s.sum[turn][rank], threadIdx.x, sum);
      store_remote(&s.count[turn][rank], threadIdx.x, count);
    }
    cluster_sync_all();
  }
  __device__ __forceinline__ void exchange(u64 sum, u64 more, uint32_t count) {
    if ((int)threadIdx.x < size) store_remote(&s.more[turn ^ 1][rank], threadIdx.x, more);
    exchange(sum, count);
  }
  // this CTA's totals; the same of all threads that come between two barriers
  __device__ __forceinline__ void add_cta(u64& sum, uint32_t& count) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    count = __reduce_add_sync(0xFFFFFFFFu, count);
    if (lane == 0) s.warp_sum[warp] = sum, s.warp_count[warp] = count;
    __syncthreads();
    sum = 0, count = 0;
    for (int w = 0; w < kWarps; ++w) sum += s.warp_sum[w], count += s.warp_count[w];
  }
  __device__ __forceinline__ void add_cta(u64& a, u64& b) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o), b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    if (lane == 0) s.warp_sum[warp] = a, s.scan_sum[warp] = b;
    __syncthreads();
    a = b = 0;
    for (int w = 0; w < kWarps; ++w) a += s.warp_sum[w], b += s.scan_sum[w];
  }
  // totals over the cluster
  __device__ __forceinline__ void add(u64& sum, uint32_t& count) {
    add_cta(sum, count);                           // (read again before the exchange's barrier only)
    exchange(sum, count);
    sum = 0, count = 0;
    for (int r = 0; r < size; ++r) sum += s.sum[turn][r], count += s.count[turn][r];
  }
};

// Eight consecutive logits as they lie in memory.  A NaN among them is never the largest,
// reaches no bound and weighs nothing, as comparisons with it fail; +inf is taken out.
template <typename T>
struct Run;
// A row as runs of sixteen-byte alignment: places `skew` to `behind` - 1 from `at` on hold
// its logits, the token at place i is i - skew.  (A run's other places are -inf.)
template <typename T>
struct RowOf {
  const T* at;
  int skew, behind;
  __device__ __forceinline__ RowOf(const T* row, int vocab) {
    skew = (int)(((uintptr_t)row & 15) / sizeof(T));
    at = row - skew, behind = vocab + skew;
  }
  __device__ __forceinline__ void load(Run<T>& run, int i) const {
    if (i >= skew && i + 8 <= behind) run.load(at + i);
    else run.load_some(at + i, skew - i, behind - i);
  }
};
template <>
struct Run<float> {
  uint32_t w[8];
  static constexpr uint32_t kNone = 0xFF800000u;   // -inf
  __device__ __forceinline__ void load(const float* p) {
    const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 4);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
  __device__ __forceinline__ void store(float* p) const {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(p + 4) = make_uint4(w[4], w[5], w[6], w[7]);
  }
  __device__ __forceinline__ void load_some(const float* p, int lo, int hi) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = j >= lo && j < hi ? __float_as_uint(p[j]) : kNone;
  }
  __device__ __forceinline__ float get(int j) const { return __uint_as_float(w[j]); }
  __device__ __forceinline__ float largest() const {
    float m = get(0);
#pragma unroll
    for (int j = 1; j < 8; ++j) m = fmaxf(m, get(j));
    return m;
  }
  // +inf becomes -inf; returns the largest
  __device__ __forceinline__ float clean() {
    float m = largest();
    if (!(m < INFINITY)) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!(get(j) < INFINITY)) w[j] = kNone;
      m = largest();
    }
    return m;
  }
};
template <>
struct Run<__nv_bfloat16> {
  uint32_t w[4];
  static constexpr uint32_t kNone = 0xFF80u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void load_some(const __nv_bfloat16* p, int lo, int hi) {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
    const auto at = [&](int j) { return j >= lo && j < hi ? q[j] : kNone; };
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = at(2 * j) | at(2 * j + 1) << 16;
  }
  __device__ __forceinline__ float get(int j) const {
    return __uint_as_float((j & 1) ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
  }
  __device__ __forceinline__ float largest() const {
    const uint32_t m = max2(max2(w[0], w[1]), max2(w[2], w[3]));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
  }
  __device__ __forceinline__ float clean() {
    float m = largest();
    if (!(m < INFINITY)) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (!(__uint_as_float(w[j] << 16) < INFINITY)) w[j] = (w[j] & 0xFFFF0000u) | kNone;
        if (!(__uint_as_float(w[j] & 0xFFFF0000u) < INFINITY)) w[j] = (w[j] & 0xFFFFu) | kNone << 16;
      }
      m = largest();
    }
    return m;
  }
};

// The largest grid value that `want` of what f counts (or weighs) reach: grid numbers lo
// (reached) and hi (not); above: f at the grid number behind it.  f(v, w): of the logits
// in [v, w), w infinite at first.
template <typename T, typename S, typename F>
__device__ __forceinline__ float bisect(uint32_t lo, uint32_t hi, S want, S& above, F f) {
  float w = INFINITY;
  while (hi - lo > 1) {
    const uint32_t mid = lo + (hi - lo) / 2;
    const float v = Grid<T>::value(mid);
    const S some = above + f(v, w);
    if (some >= want) lo = mid;
    else hi = mid, w = v, above = some;
  }
  return Grid<T>::value(lo);
}

// A CTA's histogram: bin b holds logits whose distance to the largest is b / 128 to
// (b + 1) / 128 powers of two; the last one also what lies further down.
constexpr int kBins = 4096;
constexpr float kPerUnit = 128.f;
__device__ __forceinline__ int bin_at(uint32_t y) {  // (y's bits fall with the distance, past a change of sign too)
  return (int)min((__float_as_uint(Weight::kY) - y) >> 3, (uint32_t)(kBins - 1));
}

// The cluster's histograms summed in every CTA's: each CTA sums a part of the bins for all.
// Between two barriers of the cluster.
__device__ __forceinline__ void sum_histograms(uint32_t* __restrict__ hist, int rank, int size) {
  const int part = (kBins / 2 + size - 1) / size * 2, first = rank * part, behind = min(first + part, kBins);
  for (int i = first + 2 * (int)threadIdx.x; i < behind; i += 2 * kThreads) {
    uint32_t x[kMaxCluster] = {}, y[kMaxCluster] = {};
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      if (r >= size) break;
      asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];"
                   : "=r"(x[r]), "=r"(y[r])
                   : "r"(mapa_shared(smem_u32(hist + i), r))
                   : "memory");
    }
#pragma unroll
    for (int r = 1; r < kMaxCluster; ++r) x[0] += x[r], y[0] += y[r];
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < size)
        asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(mapa_shared(smem_u32(hist + i), r)), "r"(x[0]), "r"(y[0])
                     : "memory");
  }
}

// The choice of bins.  bin[2]: where the k-th logit lies (kBins: none does), rank_in of
// its bin's tokens are kept; bin[0] to bin[1], with p < 1: where top-p's border lies, by the counts and
// the weights of the bins' middles, with a part `margin` of the mass to either side, or, if
// more than `limit` tokens lie there, less of it, down to 2^-13.  Who has the exact sums
// looks whether the border lies there.
__device__ __forceinline__ void choose_bins(Shared& s, const uint32_t* __restrict__ hist, int k, bool cuts, float p,
                                            float margin, uint32_t limit, uint32_t& rank_in) {
  constexpr int kMine = kBins / kThreads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t n[kMine];
  float w[kMine];
#pragma unroll
  for (int i = 0; i < kMine; i += 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(hist + tid * kMine + i);
    n[i] = v.x, n[i + 1] = v.y, n[i + 2] = v.z, n[i + 3] = v.w;
  }
  if (tid < 2) s.bin[tid] = kBins - 1;
  if (tid == 0) s.bin[2] = kBins;
  uint32_t count = 0;
  float mass = 0;
  const float first_weight = exp2f(-((float)(tid * kMine) + 0.5f) / kPerUnit);
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    w[i] = n[i] * (first_weight * exp2f(-i / kPerUnit));
    count += n[i], mass += w[i];
  }
  uint32_t c_run = count;
  float m_run = mass;
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t c = __shfl_up_sync(0xFFFFFFFFu, c_run, o);
    const float a = __shfl_up_sync(0xFFFFFFFFu, m_run, o);
    if (lane >= o) c_run += c, m_run += a;
  }
  if (lane == 31) s.warp_count[warp] = c_run, s.warp_mass[warp] = m_run;
  __syncthreads();
  // of the threads before this one (sums of positive numbers: nothing cancels)
  c_run -= count, m_run = __shfl_up_sync(0xFFFFFFFFu, m_run, 1);
  if (lane == 0) m_run = 0.f;
  float z = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) c_run += s.warp_count[i], m_run += s.warp_mass[i];
    z += s.warp_mass[i];
  }
  if (cuts && c_run < (uint32_t)k && (uint32_t)k <= c_run + count) {
    uint32_t c = c_run;
    float a = m_run;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      if (c < (uint32_t)k && (uint32_t)k <= c + n[i]) {
        s.bin[2] = tid * kMine + i;
        s.rank_in = k - c;
        s.z = a + w[i] / n[i] * (k - c);
      }
      c += n[i], a += w[i];
    }
  }
  __syncthreads();
  rank_in = 0;
  if (s.bin[2] < kBins) rank_in = s.rank_in, z = s.z;
  if (p < 1.f) {
    for (;; margin *= margin > 0x1p-12f ? 0.25f : 0.5f) {
      const float from = p * z * (1.f - margin), upto = p * z * (1.f + margin);
      float a = m_run;
      int b1 = kBins - 1, b2 = kBins - 1;
      // (sums of other threads may differ in the last bits: a little more of them look)
      if (m_run <= upto * 1.001f && m_run + mass >= from * 0.999f) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          a += w[i];
          if (a >= from) b1 = min(b1, tid * kMine + i);
          if (a >= upto) b2 = min(b2, tid * kMine + i);
        }
      }
      if (b1 < kBins - 1) atomicMin(&s.bin[0], b1);
      if (b2 < kBins - 1) atomicMin(&s.bin[1], b2);
      __syncthreads();
      b1 = min(s.bin[0], s.bin[2]), b2 = max(b1, min(s.bin[1], s.bin[2]));
      uint32_t in = 0;
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        if (b1 <= tid * kMine + i && tid * kMine + i <= b2) in += n[i];
      in = __reduce_add_sync(0xFFFFFFFFu, in);
      if (lane == 0) s.warp_count[warp] = in;
      __syncthreads();
      in = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) in += s.warp_count[i];
      const bool enough = in <= limit || margin <= 0x1p-13f;
      if (tid < 2) s.bin[tid] = !enough ? kBins - 1 : tid ? b2 : b1;
      if (enough) break;
      __syncthreads();
    }
  } else if (tid == 0) {
    s.bin[0] = s.bin[1] = s.bin[2];
  }
  __syncthreads();
}

// The masses of a thread's logits from the cut on: of those in bins before b1 and of those
// between b2 and bk; list(logit, step) for the others up to bk.
template <typename T, typename W, typename F>
__device__ __forceinline__ void mass_around(const T* x, int steps, float cut, const W& weight,
                                            const uint32_t* __restrict__ powers, int b1, int b2, int bk, u64& above,
                                            u64& between, F list) {
  // (bins as ranges of steps: bin b begins 8 b steps below kY, the last one ends nowhere)
  const auto begin = [](int b) { return __uint_as_float(__float_as_uint(Weight::kY) - 8 * (uint32_t)b); };
  const auto end = [&](int b) { return b < kBins - 1 ? __uint_as_float(__float_as_uint(begin(b)) - 7) : -INFINITY; };
  const float begin1 = begin(b1), end2 = end(b2), begin_k = bk < kBins ? begin(bk) : -INFINITY,
              end_k = bk < kBins ? end(bk) : INFINITY;
  for (int s = 0; s < steps; ++s) {
    Run<T> run;
    run.load(x + s * 32 * kVec);
    uint32_t hits = 0;
#pragma unroll
    for (int j = 0; j < kVec; j += 2) {
      u64 w[2];
      uint32_t y[2];
      const float l[2] = {run.get(j), run.get(j + 1)};
      const bool in[2] = {l[0] >= cut, l[1] >= cut};
      weight.two(l[0], l[1], in[0], in[1], w[0], w[1], y[0], y[1], powers);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float at = __uint_as_float(y[i]);
        if (at > begin1) above += w[i];
        else if (at < end2 && at > begin_k) between += w[i];
        else if (at >= end2 || at >= end_k) hits |= (uint32_t)in[i] << (j + i);
      }
    }
    if (hits) list(s, hits);
  }
}

// larger logit first, then lower index
__device__ __forceinline__ u64 make_key(float l, uint32_t idx) {
  return ((u64)ordered_key(l) << 32) | (0xFFFFFFFFu - idx);
}
__device__ __forceinline__ float key_logit(u64 k) { return ordered_value((uint32_t)(k >> 32)); }

// The end for n listed tokens, by one CTA: list[] in any order, other[] room for as many
// (kList).  The first k are kept at most, p as in top-p.  A scan's sums go by turns to
// two places, so that one barrier is enough.
__device__ __forceinline__ u64 scan(u64 v, u64* __restrict__ sums, u64& all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  u64 run = v;
  for (int o = 1; o < 32; o <<= 1) {
    const u64 r = __shfl_up_sync(0xFFFFFFFFu, run, o);
    if (lane >= o) run += r;
  }
  if (lane == 31) sums[warp] = run;
  __syncthreads();
  u64 at = run - v;
  all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const u64 x = sums[w];
    if (w < warp) at += x;
    all += x;
  }
  return at;
}
// The largest number c such that the keys from c on weigh `want` or more, eight bits at a
// time, until one key is left (or, with `some`, until what is left is needed whole: c is
// then less than the reaching key, but more than the next).  in(key): which ones count;
// of(key): a weight.  sums: 768 numbers; a weight goes to limbs of 21 bits, which 2,048 of
// them do not overflow, the upper bits of the third (of 2,048 weights it has 20 bits at
// most) count the keys.
template <typename I, typename W>
__device__ __forceinline__ u64 reaching_key(Shared& s, uint32_t* __restrict__ sums, const u64* __restrict__ list, int n,
                                            bool some, u64 want, I in, W of) {
  const int tid = threadIdx.x, warp = tid >> 5;
  // from the first bit that not all share
  u64 any = 0, every = ~0ull;
  for (int i = tid; i < n; i += kThreads)
    if (in(list[i])) any |= list[i], every &= list[i];
  any = (u64)__reduce_or_sync(0xFFFFFFFFu, (uint32_t)(any >> 32)) << 32 | __reduce_or_sync(0xFFFFFFFFu, (uint32_t)any);
  every = (u64)__reduce_and_sync(0xFFFFFFFFu, (uint32_t)(every >> 32)) << 32 | __reduce_and_sync(0xFFFFFFFFu, (uint32_t)every);
  if ((tid & 31) == 0) s.scan_sum[warp] = any, s.warp_sum[warp] = every;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) any |= s.scan_sum[w], every &= s.warp_sum[w];
  int shift = max(56 - __clzll((long long)(any & ~every)), 0);
  u64 fixed = shift > 55 ? 0 : ~0ull << (shift + 8), prefix = every & fixed, base = 0;  // fixed: bits that are known
  for (;;) {
    sums[tid] = sums[tid + 256] = sums[tid + 512] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const u64 key = list[i];
      if (!in(key) || ((key ^ prefix) & fixed)) continue;
      const u64 w = of(key);
      uint32_t* at = sums + (key >> shift & 255);
      atomicAdd(at, (uint32_t)w & 0x1FFFFFu);
      if (w >> 21) atomicAdd(at + 256, (uint32_t)(w >> 21) & 0x1FFFFFu);
      atomicAdd(at + 512, (uint32_t)(w >> 42) + (1u << 21));
    }
    __syncthreads();
    const int bin = 255 - tid;                     // from the largest down
    const u64 mine = sums[bin] + ((u64)sums[bin + 256] << 21) + ((u64)(sums[bin + 512] & 0x1FFFFFu) << 42);
    u64 all;
    const u64 before = base + scan(mine, s.warp_sum, all);
    if (before < want && want <= before + mine) {
      s.before = before, s.who = bin;
      s.seen = sums[bin + 512] >> 21 == 1 || (some && before + mine == want);
    }
    __syncthreads();
    prefix |= (u64)s.who << shift;
    base = s.before;
    if (shift == 0 || s.seen) break;
    fixed = ~0ull << shift;
    shift = max(shift - 8, 0);
    __syncthreads();
  }
  __syncthreads();
  return prefix;
}
template <typename W>
__device__ __forceinline__ void finish(const Args& a, Shared& s, const W& weight, u64* __restrict__ list,
                                       u64* __restrict__ other, int n, int k, float p, float u, int row) {
  const int tid = threadIdx.x, kk = min(n, k);
  if (n <= kCounted) {
    // A token's place is the number of larger ones, by logit and index and by index alone.
    u64 key = 0, w = 0;
    int place = 0, at_index = 0;
    if (tid < n) {
      key = list[tid];
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const u64 o = list[j];
        place += o > key;
        at_index += (uint32_t)o > (uint32_t)key;
      }
      w = weight(key_logit(key), s.powers);
      other[place] = w;
    }
    int kept = kk;
    if (p < 1.f) {
      __syncthreads();
      u64 all;
      const u64 at = scan(tid < kk ? other[tid] : 0, s.warp_sum, all);
      const u64 want = scaled(p, all, true);       // the mass before a kept token is below this
      kept = __syncthreads_count(tid < kk && at < want);
    } else {
      __syncthreads();
    }
    if (tid < n) {
      other[at_index] = place < kept ? w : 0;
      list[at_index + kCounted] = key;
    }
    __syncthreads();
    u64 total;
    const u64 mine = tid < n ? other[tid] : 0, at = scan(mine, s.scan_sum, total), target = scaled(u, total, false);
    if (at <= target && target < at + mine) {
      a.token[row] = (int32_t)(0xFFFFFFFFu - (uint32_t)list[tid + kCounted]);
      if (a.prob) a.prob[row] = (float)((double)mine / (double)total);
    }
    return;
  }
  // More tokens: the last key that is kept, by number, then by mass; then the token, which is
  // the reaching one in the order of the indices.
  uint32_t* sums = (uint32_t*)other;
  const auto of = [&](u64 key) { return weight(key_logit(key), s.powers); };
  u64 least = 0;
  if (kk < n)
    least = reaching_key(s, sums, list, n, true, (u64)kk, [](u64) { return true; }, [](u64) { return (u64)1; });
  const auto kept = [&](u64 key) { return key >= least; };
  const auto mass = [&] {
    u64 mine = 0, all;
    for (int i = tid; i < n; i += kThreads)
      if (kept(list[i])) mine += of(list[i]);
    scan(mine, s.scan_sum, all);
    __syncthreads();
    return all;
  };
  u64 total = mass();
  if (p < 1.f) {
    // (the mass before a kept token is below the wanted one)
    least = max(least, reaching_key(s, sums, list, n, true, scaled(p, total, true), kept, of));
    total = mass();
  }
  const u64 target = scaled(u, total, false);
  // by index alone: the logits change places with it, what is not kept becomes 0
  for (int i = tid; i < n; i += kThreads) list[i] = kept(list[i]) ? list[i] << 32 | list[i] >> 32 : 0;
  __syncthreads();
  const auto of_turned = [&](u64 key) { return weight(ordered_value((uint32_t)key), s.powers); };
  const u64 found = reaching_key(s, sums, list, n, false, target + 1, [](u64 key) { return key != 0; }, of_turned);
  // (one key is left: the smallest from there on)
  u64 best = ~0ull;
  for (int i = tid; i < n; i += kThreads)
    if (list[i] >= found) best = min(best, list[i]);
  for (int o = 16; o; o >>= 1) best = min(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
  if ((tid & 31) == 0) s.scan_sum[tid >> 5] = best;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kWarps; ++w) best = min(best, s.scan_sum[w]);
    a.token[row] = (int32_t)(0xFFFFFFFFu - (uint32_t)(best >> 32));
    if (a.prob) a.prob[row] = (float)((double)of_turned(best) / (double)total);
  }
}

// The cut by n listed logits (values), with the masses above and between their bins: the
// logit at the cut and how many equal to it are kept.  bin bk, where there is one, keeps
// its first rank_in; then p as in top-p, among the bins up to b2 (or in bk at its cut).
// below: less than all of them.  False: top-p's border is not among them.
template <typename W, typename B>
__device__ __forceinline__ bool cut_of_few(Shared& s, const W& weight, B bin_of, float* __restrict__ values, int n,
                                           float below, int b2, int bk, uint32_t rank_in, float p, u64 above, u64 between,
                                           float& cut, uint32_t& ties) {
  // A logit's place is the number of larger ones, and of equal ones in any order.
  static_assert(kListed == 2 * kThreads, "two per thread");
  float* sorted = values + 1024;
  uint32_t* equal = (uint32_t*)sorted + kListed;
  u64* masses = (u64*)(values + 2048);
  const int tid = threadIdx.x, second = tid + kThreads;
  const bool in0 = tid < n, in1 = second < n;
  const float l0 = in0 ? values[tid] : 0.f, l1 = in1 ? values[second] : 0.f;
  if (tid < 4) values[n + tid] = -INFINITY;
  equal[tid] = equal[second] = 0;
  __syncthreads();
  int place0 = 0, place1 = 0;
  if (n <= kThreads) {
    if (in0)
      for (int j = 0; j < n; j += 4) {
        const float4 v = *reinterpret_cast<const float4*>(values + j);
        place0 += (v.x > l0) + (v.y > l0) + (v.z > l0) + (v.w > l0);
      }
  } else {
    for (int j = 0; j < n; j += 4) {
      const float4 v = *reinterpret_cast<const float4*>(values + j);
      place0 += (v.x > l0) + (v.y > l0) + (v.z > l0) + (v.w > l0);
      place1 += (v.x > l1) + (v.y > l1) + (v.z > l1) + (v.w > l1);
    }
  }
  const auto put = [&](float l, int place) {
    place += (int)atomicAdd(&equal[place], 1u);
    sorted[place] = l;
    masses[place] = weight(l, s.powers);
  };
  if (in0) put(l0, place0);
  if (in1) put(l1, place1);
  const int bin0 = in0 ? bin_of(l0) : kBins + 1, bin1 = in1 ? bin_of(l1) : kBins + 1;
  const int before_k = __syncthreads_count(bin0 < bk) + __syncthreads_count(bin1 < bk);
  const int in_p = __syncthreads_count(bin0 <= b2) + __syncthreads_count(bin1 <= b2);
  const int limit = bk < kBins ? before_k + (int)rank_in : n;
  // two neighbours per thread
  const int i0 = 2 * tid, i1 = i0 + 1;
  int kept = limit;
  if (p < 1.f) {
    u64 all;
    const u64 m0 = i0 < limit ? masses[i0] : 0, m1 = i1 < limit ? masses[i1] : 0;
    const u64 at = above + scan(m0 + m1, s.warp_sum, all);
    // (`all` and the masses between: what lies behind the border)
    const u64 want = scaled(p, above + between + all, true);
    const int last = min(in_p, limit);
    kept = __syncthreads_count(i0 < last && at < want) + __syncthreads_count(i1 < last && at + m0 < want);
    // the border is among them if one that may be kept reaches it
    const int reached = __syncthreads_or((i0 < last && at + m0 >= want) || (i1 < last && at + m0 + m1 >= want));
    if (above >= want || kept == 0 || !reached) return false;
  }
  cut = kept ? sorted[kept - 1] : below;
  ties = (uint32_t)(__syncthreads_count(i0 < kept && sorted[i0] == cut) + __syncthreads_count(i1 < kept && sorted[i1] == cut));
  return true;
}
template <typename T, typename W, typename B>
__device__ __forceinline__ bool cut_of_many(Team& team, const W& weight, B bin_of, const float* __restrict__ values,
                                            int n, float below, int b2, int bk, uint32_t rank_in, float p, u64 above,
                                            u64 between, float& cut, uint32_t& ties) {
  Shared& s = team.s;
  const auto each_listed = [&](auto f) {
    for (int i = threadIdx.x; i < n; i += kThreads) f(values[i]);
  };
  const auto block_min = [&](uint32_t v) {
    v = __reduce_min_sync(0xFFFFFFFFu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.warp_count[threadIdx.x >> 5] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v = min(v, s.warp_count[w]);
    return v;
  };
  const auto mass_of = [&](float v, float w, int to_bin) {
    u64 some = 0;
    uint32_t none = 0;
    each_listed([&](float l) {
      if (l >= v && l < w && bin_of(l) <= to_bin) some += weight(l, s.powers);
    });
    __syncthreads();
    team.add_cta(some, none);
    return some;
  };
  uint32_t least = 0xFFFFFFFFu, most = 0, k_least = 0xFFFFFFFFu, k_most = 0;
  each_listed([&](float l) {
    const int b = bin_of(l);
    const uint32_t g = Grid<T>::up(l);
    if (b <= b2) least = min(least, g), most = max(most, g);
    if (b == bk) k_least = min(k_least, g), k_most = max(k_most, g);
  });
  cut = below, ties = 0;
  if (bk < kBins) {                                // the rank_in-th of its bin
    uint32_t over = 0;
    k_least = block_min(k_least), k_most = ~block_min(~k_most);
    cut = bisect<T>(k_least, k_most + 1, rank_in, over, [&](float v, float w) {
      uint32_t in = 0;
      u64 none = 0;
      each_listed([&](float l) { in += l >= v && l < w && bin_of(l) == bk; });
      __syncthreads();
      team.add_cta(none, in);
      return in;
    });
    ties = rank_in - over;
  }
  if (p >= 1.f) return true;
  u64 some = 0;
  uint32_t none = 0;
  each_listed([&](float l) {
    if (l > cut) some += weight(l, s.powers);
  });
  __syncthreads();
  team.add_cta(some, none);
  some += above + between;                         // mass above the cut so far
  const u64 each = weight(cut, s.powers), want = scaled(p, some + ties * each, true);
  if (above >= want) return false;
  if (some < want) {                               // tokens at the cut are among the kept
    ties = (uint32_t)((want - some + each - 1) / each);
    return true;
  }
  if (above + mass_of(-FLT_MAX, INFINITY, b2) < want) return false;
  u64 over = above;
  least = block_min(least), most = ~block_min(~most);
  cut = bisect<T>(least, most + 1, want, over, [&](float v, float w) { return mass_of(v, w, b2); });
  const u64 one = weight(cut, s.powers);
  ties = (uint32_t)((want - over + one - 1) / one);
  return true;
}

// A request's settings, checked; what a greedy one does not use is left out.
struct Settings {
  float temp, p, least, u;
  int k;
  bool ok, greedy;
  __device__ __forceinline__ Settings(const Args& a, int row) {
    const int q = a.index ? a.index[row] : row;
    ok = q >= 0 && q < a.requests;
    temp = ok && a.temperature ? a.temperature[q] : 1.f;
    p = ok && a.top_p ? a.top_p[q] : 1.f, least = ok && a.min_p ? a.min_p[q] : 0.f;
    u = a.u[row], k = ok && a.top_k ? a.top_k[q] : 0;
    ok = ok && temp >= 0.f && temp <= 0x1p100f;
    greedy = temp == 0.f;
    if (!ok || greedy) p = 1.f, least = 0.f, u = 0.f, k = 0;
    ok = ok && k >= 0 && p > 0.f && p <= 1.f && least >= 0.f && least <= 1.f && u >= 0.f && u < 1.f;
    if (k == 0 || k > a.vocab) k = a.vocab;
    if (greedy) k = 1;
  }
  // how far below the largest logit min-p goes
  __device__ __forceinline__ double far() const { return -log((double)least) * (double)temp; }
  __device__ __forceinline__ Weight weight(float m, int bits) const {
    Weight w{m, 0.f, 0.f, bits};
    if (!greedy) {
      // (no fp64: its units are few)
      constexpr float kHi = 1.44269502162933349609375f, kLo = 1.9259629911e-8f;
      w.hi = __fdiv_rn(kHi, temp);
      w.lo = __fdiv_rn(__fadd_rn(__fmaf_rn(-w.hi, temp, kHi), kLo), temp);
      if (!(w.hi < 1e38f)) w.hi = 1e38f, w.lo = 0.f;
    }
    return w;
  }
};

// reached_by over a CTA's threads
__device__ __forceinline__ uint32_t reached_by_threads(int need, uint32_t best, uint32_t top, uint32_t lo) {
  return reached_by(need, top, lo, [&](uint32_t key) { return __syncthreads_count(best >= key); });
}
__device__ __forceinline__ uint32_t largest_of_cta(uint32_t best, uint32_t* __restrict__ of_warps) {
  best = __reduce_max_sync(0xFFFFFFFFu, best);
  if ((threadIdx.x & 31) == 0) of_warps[threadIdx.x >> 5] = best;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) best = max(best, of_warps[w]);
  return best;
}

// Many rows: one CTA per row, which reads it once and lists what a top_k up to kStreamK or a
// min-p can keep.  The first 4,096 (fp32: 2,048) logits give a bound that top_k of them reach,
// more logits a better one.  Rows that need anything else, or have too many candidates, are
// left to sample_kernel.  Logits on their way lie in shared memory, so that six CTAs fit an
// SM's registers.  768 rows of 64,000 bf16: 30 us, 3.3 TB/s; 2,700 instructions per warp, a
// third of them for settings, bounds and the end, at 2.2 per cycle and SM.
constexpr int kStreamK = 192, kLater = -2;
template <typename T>
__global__ void __launch_bounds__(kThreads, 6)
    stream_kernel(const __grid_constant__ Args a, const T* __restrict__ logits, DevCtx c) {
  __shared__ Shared sh;
  __shared__ __align__(16) u64 list[kList], other[kList / 2];
  constexpr int kRunList = kList;
  int* runs = (int*)other;                         // runs with a logit that reached the bound when they were read
  // Logits on their way, in the list's place: 64 bytes per thread, in two groups.
  constexpr int kRuns = 32 / (int)sizeof(Run<T>), kGroup = kRuns * kThreads * kVec;
  T* ring = (T*)list + threadIdx.x * kVec;
  const int tid = threadIdx.x, row = blockIdx.x;
  load_powers(sh);
  if (tid == 0) sh.listed = sh.rank_in = 0;
  wait_for_earlier();
  const RowOf<T> src(logits + row * a.ld, a.vocab);
  const T* mine = src.at + tid * kVec;
  const uint32_t slot = smem_u32(ring);
  constexpr int kStep = kThreads * kVec, kPieces = (int)sizeof(Run<T>) / 16;
  const auto fetch = [&](int at, int half) {       // (each thread looks at what it fetched itself)
    if (at >= src.skew && at + kGroup <= src.behind) {
#pragma unroll
      for (int s = 0; s < kRuns * kPieces; ++s)
        cp_async16_cg(slot + (half * kRuns + s / kPieces) * kStep * sizeof(T) + s % kPieces * 16,
                      (const uint8_t*)(mine + at + s / kPieces * kStep) + s % kPieces * 16);
    } else if (at < src.behind) {
#pragma unroll 1
      for (int s = 0; s < kRuns; ++s) {
        Run<T> run;
        src.load(run, at + s * kStep + tid * kVec);
        run.store(ring + (half * kRuns + s) * kStep);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  fetch(0, 0);
  fetch(kGroup, 1);
  const Settings set(a, row);
  const bool by_k = set.k < a.vocab;
  if (!set.ok || !(by_k ? set.k <= kStreamK : set.least > 0.f)) {
    if (tid == 0) {
      a.token[row] = set.ok ? kLater : -1;
      if (a.prob) a.prob[row] = 0.f;
      if (!set.ok) set_status(c, DSA_ERR_INDEX);
    }
    cp_async_wait_all();
    return;
  }
  if (tid == 0 && set.least > 0.f) sh.far = set.far();  // (read behind a barrier)
  const auto cut_at = [&](float m) {
    return set.greedy ? m : set.least > 0.f ? fmaxf(__double2float_ru((double)m - sh.far), -FLT_MAX) : -FLT_MAX;
  };
  float m = -INFINITY, low = -FLT_MAX;
  uint32_t top = 0, bound = 0;
  for (int at = 0, group = 1, bound_at = 1; at < src.behind; at += kGroup, ++group) {
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    const int half = (group - 1) & 1;
    float of_run[kRuns];
#pragma unroll
    for (int s = 0; s < kRuns; ++s) {
      Run<T> run;
      run.load(ring + (half * kRuns + s) * kThreads * kVec);
      m = fmaxf(m, of_run[s] = run.clean());
    }
    // (m, which is never +inf, is known when the logits have been read: only then new ones may come)
    if (m < INFINITY) fetch(at + 2 * kGroup, half);
    const bool last = at + kGroup >= src.behind;
    if (group == bound_at || last) {               // after 1, 3, 9, ... groups and the last
      bound_at *= 3;
      const uint32_t best = ordered_key(m);
      const bool by_top = group == 1 || last || !by_k || set.k == 1 || !bound;
      if (by_top) top = largest_of_cta(best, sh.warp_count);
      if (by_k) bound = reached_by_threads(set.k, best, by_top ? top : 0xFFFFFFF0u, bound);
      low = fmaxf(low, ordered_value(bound));      // (a bound once found holds)
      if (by_top) low = fmaxf(low, cut_at(ordered_value(top)));
      __syncthreads();
    }
#pragma unroll
    for (int s = 0; s < kRuns; ++s)
      if (of_run[s] >= low) {
        const uint32_t to = atomicAdd(&sh.listed, 1u);
        if (to < kRunList) runs[to] = at + (s * kThreads + tid) * kVec;
      }
  }
  // The next launch comes here and not at the beginning: CTAs that come while others hold
  // an SM's places fill what is left, and some SMs get twice as many as others.  (300 rows of
  // 16,000 12 us instead of 20; 48 rows of 64,000 by top-p 31 instead of 36.)
  let_next_launch();
  cp_async_wait_all();
  __syncthreads();
  m = ordered_value(top);
  const int n = (int)sh.listed;
  if (m == -INFINITY || n > kRunList) {
    if (tid == 0) {
      a.token[row] = m == -INFINITY ? -1 : kLater;
      if (a.prob) a.prob[row] = 0.f;
    }
    return;
  }
  for (int i = tid; i < n; i += kThreads) {        // the logits that reach the last bound
    const int at = runs[i];
    Run<T> run;
    src.load(run, at);
    run.clean();
    uint32_t hits = 0;
#pragma unroll
    for (int j = 0; j < kVec; ++j) hits |= (uint32_t)(run.get(j) >= low) << j;
    uint32_t to = hits ? atomicAdd(&sh.rank_in, __popc(hits)) : 0;
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (hits >> j & 1) {
        if (to < kList) list[to] = make_key(run.get(j), (uint32_t)(at + j - src.skew));
        ++to;
      }
  }
  __syncthreads();
  if (sh.rank_in > kList) {
    if (tid == 0) a.token[row] = kLater;
    return;
  }
  finish(a, sh, RowWeight<T>(set.weight(m, a.bits)), list, other, (int)sh.rank_in, set.k, set.p, set.u, row);
}

// A row by a cluster; called between an arrive at the cluster's barrier and the next.
// chunk: logits of a CTA; steps: runs of eight per thread, so that the chunk fits the CTA.
// kCuts: there may be a top-k, top-p or min-p (and dyn begins with room for a list).
template <typename T, bool kCuts>
__device__ __forceinline__ void sample_row(const Args& a, const T* __restrict__ logits, int chunk, int steps, const DevCtx& c,
                                           Shared& sh, uint8_t* dyn, int row) {
  u64* list = (u64*)dyn;
  T* mine = (T*)(dyn + (kCuts ? kList * sizeof(u64) : 0));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int size = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  if (tid == 0) sh.listed = 0;
  // The row's logits of this CTA to shared memory: a warp's together in index order, a
  // thread's in runs of eight.
  const int first = (warp * steps * 32 + lane) * kVec;
  const RowOf<T> src(logits + row * a.ld, a.vocab);
  T* x = mine + first;
  float m = -INFINITY;
  constexpr int kAhead = sizeof(T) == 2 ? 8 : 4;   // runs in flight
  Run<T> run[kAhead];
  const auto load_runs = [&](int s0) {
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      const int i = first + (s0 + s) * 32 * kVec;
      if (s0 + s >= steps) break;
      if (i < chunk) src.load(run[s], rank * chunk + i);  // (chunks are whole runs)
      else run[s].load_some(src.at, 0, 0);
    }
  };
  load_runs(0);
  const Settings set(a, row);                      // (while they are on their way)
  const bool ok = set.ok, greedy = set.greedy;
  const float p = kCuts ? set.p : 1.f, least = kCuts ? set.least : 0.f, u = set.u;
  const int k = kCuts || greedy ? set.k : a.vocab;
  if (kCuts && tid == 0 && least > 0.f) sh.far = set.far();
  for (int s0 = 0; s0 < steps; s0 += kAhead) {
    if (s0) load_runs(s0);
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      if (s0 + s >= steps) break;
      m = fmaxf(m, run[s].clean());
      run[s].store(x + (s0 + s) * 32 * kVec);
    }
  }
  // f(logit) over this thread's logits
  const auto each_logit = [&](auto f) {
    for (int s = 0; s < steps; ++s) {
      Run<T> run;
      run.load(x + s * 32 * kVec);
#pragma unroll
      for (int j = 0; j < kVec; ++j) f(run.get(j));
    }
  };
  Team team{sh, rank, size, 0};
  // The CTA's largest logit; and with a small k a logit that at least k of the row reach:
  // ceil(k / size) threads of each CTA have one.
  const uint32_t best = ordered_key(m);
  uint32_t top = largest_of_cta(best, sh.warp_count);
  const bool small_k = kCuts && k <= kSmallK && k < a.vocab;
  uint32_t bound = small_k ? reached_by_threads((k + size - 1) / size, best, top, 0) : 0;
  cluster_wait();
  team.exchange(top, bound);
  for (int r = 0; r < size; ++r) {
    top = max(top, (uint32_t)sh.sum[team.turn][r]);
    bound = min(bound, sh.count[team.turn][r]);
  }
  m = ordered_value(top);
  if (!ok || m == -INFINITY) {                     // the same for the whole cluster
    if (rank == 0 && tid == 0) {
      a.token[row] = -1;
      if (a.prob) a.prob[row] = 0.f;
      if (!ok) set_status(c, DSA_ERR_INDEX);
    }
    return;
  }
  // kept: logits above `cut`, and of those equal to it the first `ties`; first what min-p keeps
  const RowWeight<T> weight(set.weight(m, a.bits));
  float cut = greedy ? m : -FLT_MAX;
  if (least > 0.f) cut = fmaxf(__double2float_ru((double)m - sh.far), -FLT_MAX);
  // Logits in the thousands for their temperature are far apart: what is 64 powers of two
  // below the largest weighs nothing, and few are not.
  const bool cold = kCuts && !greedy && !weight.fits;
  if (cold) cut = fmaxf(cut, m - 64.f / weight.plain.hi);
  if (kCuts && (small_k || cold || least > 0.f || (p < 1.f && a.vocab <= kList))) {
    // Few tokens can be kept as a rule, or are there: CTA 0 gets them listed.
    const float low = small_k ? fmaxf(cut, fmaxf(ordered_value(bound), -FLT_MAX)) : cut;
    const uint32_t room = kList / size;
    for (int s = 0; s < steps; ++s) {
      Run<T> run;
      run.load(x + s * 32 * kVec);
      if (run.largest() < low) continue;
      uint32_t hits = 0;
#pragma unroll
      for (int j = 0; j < kVec; ++j) hits |= (uint32_t)(run.get(j) >= low) << j;
      uint32_t to = atomicAdd(&sh.listed, __popc(hits));
      for (; hits && to < room; hits &= hits - 1, ++to) {
        const int i = s * 32 * kVec + __ffs(hits) - 1;
        store_remote(&list[rank * room + to], 0, make_key(to_f32(x[i]), (uint32_t)(rank * chunk + first + i - src.skew)));
      }
    }
    __syncthreads();
    team.exchange(0, sh.listed);
    bool all = true;
    int total = 0;
    for (int r = 0; r < size; ++r) {
      all = all && sh.count[team.turn][r] <= room;
      total += (int)sh.count[team.turn][r];
    }
    if (all) {
      let_next_launch();
      if (rank != 0) return;
      u64* packed = (u64*)mine;                    // (this CTA's logits are not looked at again)
      int r = 0, begin = 0;
      for (int i = tid; i < total; i += kThreads) {
        while (i - begin >= (int)sh.count[team.turn][r]) begin += (int)sh.count[team.turn][r++];
        packed[i] = list[r * room + i - begin];
      }
      __syncthreads();
      finish(a, sh, weight, packed, list, total, k, p, u, row);
      return;
    }
  }
  // Any number of tokens.
  u64 sum = 0;                                     // this thread's part of what is kept: logits above the cut,
  uint32_t count = 0, ties = greedy ? 1u : 0x7FFFFFFFu;  // and those equal to it
  const auto masses = [&](const auto& weight) {
    for (int s = 0; s < steps; ++s) {
      Run<T> run;
      run.load(x + s * 32 * kVec);
#pragma unroll
      for (int j = 0; j < kVec; j += 2) {
        u64 w0, w1;
        uint32_t y;
        weight.two(run.get(j), run.get(j + 1), run.get(j) > cut, run.get(j + 1) > cut, w0, w1, y, y, sh.powers);
        sum += w0 + w1;
      }
    }
  };
  const auto keep = [&] {
    sum = 0, count = 0;
    if (greedy) {                                  // (nothing above the largest)
    } else if (weight.fits) {
      masses(weight.fine);
    } else {
      masses(weight.plain);
    }
    if (ties)
      each_logit([&](float l) { count += l == cut; });
  };
  bool cuts = kCuts && k < a.vocab && !greedy;
  bool found = !cuts && p >= 1.f;
  if (!greedy) cut = Grid<T>::value(Grid<T>::up(cut));
  if (found) {                                     // nothing to cut, or the first of the largest
    if (!greedy) cut = next_below<T>(cut), ties = 0;
    keep();
  }
  // A histogram tells near which logits the cuts lie; CTA 0 gets those listed.  The bins'
  // middles are off by a part in 370 at most, a sum over many bins by much less: 2^-11 of
  // the mass to either side is enough as a rule, 2^-8 the second time.  (48 rows of 64,000: 9
  // us more from 2^-13 on, as 3 rows need a second time, 8 more from 2^-8 on, as lists get longer.)
  for (int time = 0; kCuts && weight.fits && !found && time < 2; ++time) {
    uint32_t* hist = (uint32_t*)list;
    static_assert(kBins * 4 <= kList * 8, "the histogram takes the list's place");
    const auto bin_of = [&](float l) { return bin_at(weight.fine.step(l)); };
    __syncthreads();
    if (tid == 0) sh.listed = 0;
    for (int i = tid; i < kBins / 4; i += kThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    each_logit([&](float l) {
      if (l >= cut) atomicAdd(&hist[bin_of(l)], 1u);
    });
    cluster_sync_all();
    sum_histograms(hist, rank, size);
    cluster_sync_all();
    uint32_t rank_in = 0;
    choose_bins(sh, hist, k, cuts, p, time ? 0x1p-8f : 0x1p-11f, time ? 2 * kList : kCounted, rank_in);
    const int b1 = sh.bin[0], b2 = sh.bin[1], bk = sh.bin[2];
    if (bk == kBins && p >= 1.f) {                 // fewer than k reach the cut: nothing more to cut
      cuts = false;
      break;
    }
    const auto is_listed = [&](int b) { return (uint32_t)(b - b1) <= (uint32_t)(b2 - b1) || b == bk; };
    float* values = (float*)list;                  // in the histogram's place
    const uint32_t room = 2 * kList / size;
    u64 above = 0, between = 0;                    // exact masses of what lies above and between the listed bins
    uint32_t with = 0;                             // steps with listed logits
    mass_around<T>(x, steps, cut, weight.fine, sh.powers, b1, b2, bk, above, between, [&](int s, uint32_t hits) {
      with |= 1u << s;
      uint32_t to = atomicAdd(&sh.listed, __popc(hits));
      for (; hits && to < room; hits &= hits - 1) values[to++] = to_f32(x[s * 32 * kVec + __ffs(hits) - 1]);
    });
    const u64 above_here = above, between_here = between;
    team.add_cta(above, between);
    team.exchange(above, between, sh.listed);
    bool all = true;
    above = between = 0;
    for (int r = 0; r < size; ++r) {
      all = all && sh.count[team.turn][r] <= room;
      above += sh.sum[team.turn][r], between += sh.more[team.turn][r];
    }
    if (!all) break;
    if (rank == 0) {
      int n = (int)sh.count[team.turn][0];
      for (int r = 1; r < size; ++r) {             // the others' behind its own
        const int more = (int)sh.count[team.turn][r];
        for (int i = tid; i < more; i += kThreads) values[n + i] = load_remote(&values[i], r);
        n += more;
      }
      __syncthreads();
      float at_cut;
      uint32_t tied;
      const bool right = n <= kListed ? cut_of_few(sh, weight.fine, bin_of, values, n, next_below<T>(cut), b2, bk, rank_in, p,
                                                    above, between, at_cut, tied)
                                      : cut_of_many<T>(team, weight.fine, bin_of, values, n, next_below<T>(cut), b2, bk,
                                                        rank_in, p, above, between, at_cut, tied);
      if (tid < size) store_remote(&sh.note, tid, right ? (u64)__float_as_uint(at_cut) << 32 | tied : ~0ull);
    }
    cluster_sync_all();
    found = sh.note != ~0ull;
    if (found) {
      cut = __uint_as_float((uint32_t)(sh.note >> 32));
      ties = (uint32_t)sh.note;
      sum = above_here + (bin_of(cut) > b2 ? between_here : 0);
      for (; with; with &= with - 1) {
        Run<T> run;
        run.load(x + (__ffs(with) - 1) * 32 * kVec);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const float l = run.get(j);
          if (l > cut && is_listed(bin_of(l))) sum += weight.fine(l, sh.powers);
          count += l == cut;
        }
      }
    }
  }
  if (kCuts && !found) {
    // Nothing more to cut, or too many near a cut (equal logits, say): bisection over all of them.
    const auto count_of = [&](float v, float w) {
      uint32_t n = 0;
      u64 none = 0;
      each_logit([&](float l) { n += l >= v && l < w; });
      team.add(none, n);
      return n;
    };
    const uint32_t end = Grid<T>::up(m) + 1;
    __syncthreads();
    if (cuts && count_of(cut, INFINITY) > (uint32_t)k) {
      uint32_t over = 0;
      cut = bisect<T>(Grid<T>::up(cut), end, (uint32_t)k, over, count_of);
      ties = k - over;
    }
    keep();
    if (p < 1.f) {
      u64 mass = sum;
      uint32_t tied = count;
      team.add(mass, tied);
      ties = min(ties, tied);
      const u64 each = weight(cut, sh.powers);
      const u64 want = scaled(p, mass + ties * each, true);  // the mass before a kept token is below this
      if (mass < want) {                           // tokens at the cut are among them
        ties = (uint32_t)((want - mass + each - 1) / each);
      } else {
        u64 over = 0;
        cut = bisect<T>(Grid<T>::up(cut), end, want, over, [&](float v, float w) {
          u64 some = 0;
          uint32_t none = 0;
          each_logit([&](float l) {
            if (l >= v && l < w) some += weight(l, sh.powers);
          });
          team.add(some, none);
          return some;
        });
        const u64 one = weight(cut, sh.powers);
        ties = (uint32_t)((want - over + one - 1) / one);
        keep();
      }
    }
  }
  // What each warp keeps, in the order of the tokens.
  const u64 each = ties ? weight(cut, sh.powers) : 0;
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  count = __reduce_add_sync(0xFFFFFFFFu, count);
  if (lane == 0) sh.warp_sum[warp] = sum, sh.warp_count[warp] = count;
  __syncthreads();
  if (warp == 0) {
    u64 s = lane < kWarps ? sh.warp_sum[lane] : 0;
    for (int o = kWarps / 2; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    const uint32_t n = __reduce_add_sync(0xFFFFFFFFu, lane < kWarps ? sh.warp_count[lane] : 0u);
    sum = s, count = n;
  }
  team.exchange(sum, count);                       // (its stores are the first warp's)
  // mass of n tokens at the cut when `seen` of them came before
  const auto tie_mass = [&](uint32_t seen, uint32_t n) { return (u64)(min(ties, seen + n) - min(ties, seen)) * each; };
  if (warp == 0) {
    // a CTA's, then a warp's, per lane: the kept mass before it and its own
    u64 before, kept;
    uint32_t seen;
    const auto in_order = [&](u64 s, uint32_t n, u64 base, uint32_t base_seen) {
      static_assert(kWarps <= 8 && kMaxCluster <= 8, "three steps");
      uint32_t n_run = n;
      for (int o = 1; o < 8; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, n_run, o);
        if (lane >= o) n_run += v;
      }
      seen = base_seen + n_run - n;
      kept = s + (ties ? tie_mass(seen, n) : 0);
      u64 run = kept;
      for (int o = 1; o < 8; o <<= 1) {
        const u64 v = __shfl_up_sync(0xFFFFFFFFu, run, o);
        if (lane >= o) run += v;
      }
      before = base + run - kept;
    };
    in_order(lane < size ? sh.sum[team.turn][lane] : 0, lane < size ? sh.count[team.turn][lane] : 0u, 0, 0);
    const u64 total = __shfl_sync(0xFFFFFFFFu, before + kept, 7), target = scaled(u, total, false);
    const bool here = __shfl_sync(0xFFFFFFFFu, before <= target && target < before + kept, rank);
    const u64 base = __shfl_sync(0xFFFFFFFFu, before, rank);
    const uint32_t base_seen = __shfl_sync(0xFFFFFFFFu, seen, rank);
    if (lane == 0) sh.who = -1;
    __syncwarp();
    if (here) {
      in_order(lane < kWarps ? sh.warp_sum[lane] : 0, lane < kWarps ? sh.warp_count[lane] : 0u, base, base_seen);
      if (lane < kWarps && before <= target && target < before + kept)
        sh.who = lane, sh.before = before, sh.seen = seen, sh.target = target, sh.total = total;
    }
  }
  __syncthreads();
  const int who = sh.who;
  let_next_launch();                               // (late, as in stream_kernel)
  if (who < 0) return;
  // The CTA that holds the token: one step of the warp that does per warp, one of its lanes.
  u64 before = sh.before;
  uint32_t seen = sh.seen;
  const u64 target = sh.target, total = sh.total;
  const T* at_x = mine + (who * steps * 32 + lane) * kVec;
  for (int s0 = 0; s0 < steps; s0 += kWarps) {
    const int s = s0 + warp;
    Run<T> v;
    u64 run = 0, own[kVec];
    uint32_t tie_run = 0;
    if (s < steps) {
      v.load(at_x + s * 32 * kVec);
#pragma unroll
      for (int j = 0; j < kVec; j += 2) {
        const float l0 = v.get(j), l1 = v.get(j + 1);
        uint32_t y;
        if (weight.fits) weight.fine.two(l0, l1, l0 > cut, l1 > cut, own[j], own[j + 1], y, y, sh.powers);
        else weight.plain.two(l0, l1, l0 > cut, l1 > cut, own[j], own[j + 1], y, y, sh.powers);
        run += own[j] + own[j + 1];
        tie_run += (v.get(j) == cut) + (v.get(j + 1) == cut);
      }
    }
    const u64 mine_run = run;
    const uint32_t mine_ties = tie_run;
    for (int o = 1; o < 32; o <<= 1) {
      const u64 r = __shfl_up_sync(0xFFFFFFFFu, run, o);
      const uint32_t n = __shfl_up_sync(0xFFFFFFFFu, tie_run, o);
      if (lane >= o) run += r, tie_run += n;
    }
    if (lane == 31) sh.warp_sum[warp] = run, sh.warp_count[warp] = tie_run;
    __syncthreads();
    u64 at = before;
    uint32_t at_ties = seen;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const u64 some = sh.warp_sum[w] + tie_mass(seen, sh.warp_count[w]);
      before += some;
      seen += sh.warp_count[w];
      if (w < warp) at += some, at_ties = seen;
    }
    if (s < steps) {
      at += run - mine_run + tie_mass(at_ties, tie_run - mine_ties);
      at_ties += tie_run - mine_ties;
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const bool tie = v.get(j) == cut;
        const u64 w = tie ? (at_ties < ties ? each : 0) : own[j];
        at_ties += tie;
        if (at <= target && target < at + w) {
          a.token[row] = rank * chunk + (who * steps * 32 + s * 32 + lane) * kVec + j - src.skew;
          if (a.prob) a.prob[row] = (float)((double)w / (double)total);
        }
        at += w;
      }
    }
    __syncthreads();
  }
}

// kLeft: only the rows that stream_kernel left.  (A grid of all rows whose other CTAs end at
// once: 3 us for 768 rows of 64,000; fewer clusters that look for rows take 60 % longer
// where most are left.)
template <typename T, bool kCuts, bool kLeft>
__global__ void __launch_bounds__(kThreads, 4)
    sample_kernel(const __grid_constant__ Args a, const T* __restrict__ logits, int chunk, int steps, DevCtx c) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ Shared sh;
  cluster_arrive();                                // no CTA writes to one that has not begun
  const int row = blockIdx.x / cluster_nctarank();
  if (!kLeft) load_powers(sh);
  wait_for_earlier();
  if (kLeft) {
    if (a.token[row] != kLater) {                  // (written after barriers behind this read)
      cluster_wait();
      return;
    }
    load_powers(sh);
  }
  sample_row<T, kCuts>(a, logits, chunk, steps, c, sh, dyn, row);
}

static int check(const dsa_sampler* p) {
  if (!p) return DSA_ERR_INVALID_ARG;
  if (p->dtype != DSA_BF16 && p->dtype != DSA_FP32) return DSA_ERR_UNSUPPORTED;
  if (p->rows < 1 || p->vocab < 1 || p->ld < p->vocab || p->requests < 1) return DSA_ERR_INVALID_ARG;
  if (p->vocab > kMaxVocab || p->ld > (1ll << 40) || p->rows >= (1ll << 27) || p->requests >= (1ll << 31))
    return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}
static bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && x < y + nb && y < x + na;
}

template <typename T>
static bool launch(const Args& a, const void* logits, DevCtx c, cudaStream_t st) {
  // 32 KB of logits per CTA, so that four fit an SM, and more CTAs for a few rows
  int dev = 0, sms = 0, size = 1;
  if (!cuda_ok(cudaGetDevice(&dev)) || !cuda_ok(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)))
    return false;
  const int full = 32768 / (int)sizeof(T);
  size = std::min(kMaxCluster, (a.vocab + full - 1) / full);
  while (size < kMaxCluster && (long long)a.rows * size * 2 <= sms && size * 2048 < a.vocab) ++size;
  // (rows that do not begin at sixteen bytes take up to a run's places more)
  const bool whole = (((uintptr_t)logits | (uintptr_t)(a.ld * sizeof(T))) & 15u) == 0;
  const int places = a.vocab + (whole ? 0 : kVec - 1);
  const int chunk = (places + size * kVec - 1) / (size * kVec) * kVec, step = kThreads * kVec;
  const int steps = (chunk + step - 1) / step;
  const bool cuts = a.top_k || a.top_p || a.min_p;
  const size_t room = (size_t)steps * step * sizeof(T);
  const size_t smem = cuts ? kList * 8 + std::max(room, (size_t)kList * 8) : room;
  const bool stream = a.rows >= sms && (a.top_k || a.min_p);
  auto kernel = stream ? sample_kernel<T, true, true> : cuts ? sample_kernel<T, true, false> : sample_kernel<T, false, false>;
  // (the most that any call takes: another thread's call may come between this one and the launch)
  constexpr int kMost = kList * 8 + (kMaxVocab / kMaxCluster + kThreads * kVec) * (int)sizeof(T);
  if (smem > kMost || !cuda_ok(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost))) return false;
  if (stream && !launch_programmatic(stream_kernel<T>, dim3((unsigned)a.rows), dim3(kThreads), 0, st, 1, a,
                                     (const T*)logits, c))
    return false;
  return launch_programmatic(kernel, dim3((unsigned)(a.rows * size)), dim3(kThreads), smem, st, size, a,
                             (const T*)logits, chunk, steps, c);
}

}  // namespace sample
}  // namespace dsa

using namespace dsa;
using namespace dsa::sample;

extern "C" int dsa_sample(const dsa_sampler* p, const void* logits, const float* u, const float* temperature,
                          const int32_t* top_k, const float* top_p, const float* min_p, const int32_t* index,
                          int32_t* token, float* prob, dsa_stream_t stream) {
  int rc = check(p);
  if (rc) return rc;
  if (!logits || !u || !token || (!index && p->requests != p->rows)) return DSA_ERR_INVALID_ARG;
  const size_t esz = p->dtype == DSA_BF16 ? 2 : 4, rows = (size_t)p->rows * 4, req = (size_t)p->requests * 4;
  if (((uintptr_t)logits & (esz - 1)) ||
      (((uintptr_t)u | (uintptr_t)temperature | (uintptr_t)top_k | (uintptr_t)top_p | (uintptr_t)min_p |
        (uintptr_t)index | (uintptr_t)token | (uintptr_t)prob) & 3u))
    return DSA_ERR_INVALID_ARG;
  for (const void* o : {(const void*)token, (const void*)prob})
    if (overlap(o, rows, logits, ((size_t)(p->rows - 1) * p->ld + p->vocab) * esz) || overlap(o, rows, u, rows) ||
        overlap(o, rows, index, rows) || overlap(o, rows, temperature, req) || overlap(o, rows, top_k, req) ||
        overlap(o, rows, top_p, req) || overlap(o, rows, min_p, req))
      return DSA_ERR_INVALID_ARG;
  if (overlap(token, rows, prob, rows)) return DSA_ERR_INVALID_ARG;
  DevCtx c;
  if (!ext_dev_ctx(&c)) return DSA_ERR_CUDA;
  int bits = 0;
  while ((1ll << bits) < p->vocab) ++bits;
  const Args a{(int)p->rows, (int)p->vocab, (int)p->requests, bits, p->ld, u, temperature, top_p, min_p,
               top_k, index, token, prob};
  const bool ok = p->dtype == DSA_BF16 ? launch<__nv_bfloat16>(a, logits, c, (cudaStream_t)stream)
                                       : launch<float>(a, logits, c, (cudaStream_t)stream);
  return ok ? DSA_OK : DSA_ERR_CUDA;
}
