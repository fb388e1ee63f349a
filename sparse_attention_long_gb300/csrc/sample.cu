// Sampling of one token per row of logits (dsa_sample): temperature, min-p, top-k,
// top-p, and a draw by a given uniform number.
//
// One thread-block cluster per row; the row stays in shared memory.
// All three cuts keep a run of the tokens in the order (logit descending, index
// ascending), so a cut is a logit and a number of tokens that have exactly this logit,
// lowest index first.  min-p gives its logit outright, from the maximum.  top-k's and
// top-p's are found by bisection over the logits' order-preserving bits: a step counts
// (or weighs) the logits above a middle one.
//
// Borders between tokens lie dense in a large vocabulary, so fp32 sums would draw
// neighbours of the right token now and then.  Weights are computed to some 2^-31 of themselves
// (the exponent in two floats, a table of 2^(j/256) and a short series) and summed as
// integers, in units of 2^-44 of the largest one or finer: sums are exact, whatever
// their order.
#include <float.h>
#include <math.h>

#include "dsa_common.cuh"

namespace dsa {

bool ext_dev_ctx(DevCtx* c);

namespace sample {

constexpr int kMaxCluster = 8;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kVec = 8;                            // consecutive logits of a thread
constexpr int kMaxVocab = 1 << 18;
constexpr int kList = 2048;                        // tokens that one CTA can order, 2^n
constexpr int kCounted = 256;                      // up to so many by counting
constexpr int kSmallK = 1024;                      // top_k up to which candidates are listed

typedef unsigned long long u64;

struct Args {
  int rows, vocab, requests, unit;                 // weights in units of 2^-unit
  long long ld;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t *top_k, *index;
  int32_t* token;
  float* prob;
};

// 2^31 * 2^(j / 256)
struct Powers {
  uint32_t at[256];
  constexpr Powers() : at() {
    for (int j = 0; j < 256; ++j) {
      const double x = j / 256.0 * 0.69314718055994530942;
      double term = 1, sum = 1;
      for (int k = 1; k < 24; ++k) {
        term *= x / k;
        sum += term;
      }
      at[j] = (uint32_t)(sum * 2147483648.0 + 0.5);
    }
  }
};
__device__ const Powers kPowers{};

__device__ __forceinline__ void store_remote(u64* local, uint32_t rank, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa_shared(smem_u32(local), rank)), "l"(v) : "memory");
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

// w = 2^-x in units of 2^-unit, x = (max - l) * log2(e) / temperature
struct Weight {
  float max, hi, lo;                               // log2(e) / temperature in two floats
  int unit;
  __device__ __forceinline__ u64 operator()(float l, const uint32_t* __restrict__ powers) const {
    const float d = __fsub_rn(max, l), t = __fsub_rn(d, max);
    const float e = __fadd_rn(__fsub_rn(max, __fsub_rn(d, t)), -__fadd_rn(l, t));  // max - l = d + e
    const float x = __fmul_rn(d, hi);
    if (!(x < 62.f)) return 0;
    const float y = __fmaf_rn(d, lo, __fmaf_rn(e, hi, __fmaf_rn(d, hi, -x)));
    const float n = rintf(x);
    const u64 z = -(((u64)(int64_t)n << 32) + (int64_t)__float2int_rn((x - n) * 4294967296.f) +
                    (int64_t)__float2int_rn(y * 4294967296.f));               // -x, 32 bits behind the point
    const int k = (int)((int64_t)z >> 32);
    const uint32_t f = (uint32_t)z, p = powers[f >> 24];
    const float r = (float)(f & 0xFFFFFFu) * (0.69314718056f / 4294967296.f);
    const float s = r * __fmaf_rn(r, __fmaf_rn(r, 1.f / 6, 0.5f), 1.f);        // e^r - 1 < 2^-8
    const u64 w = (u64)(p + __float2uint_rn((float)p * s)) << (unit - 31);
    return k > 0 ? w : w >> -k;
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

struct Shared {
  uint32_t powers[256];
  double far;                                      // how far below the largest logit min-p goes
  u64 warp_sum[kWarps];
  uint32_t warp_count[kWarps];
  u64 sum[2][kMaxCluster], count[2][kMaxCluster];  // of every CTA of the cluster, two exchanges deep
};

// What a CTA sums, and what the cluster does.  An exchange's numbers stay readable until
// the next but one.
struct Team {
  Shared& s;
  int rank, size, turn;
  __device__ __forceinline__ void exchange(u64 sum, u64 count) {
    turn ^= 1;
    if ((int)threadIdx.x < size) {
      store_remote(&s.sum[turn][rank], threadIdx.x, sum);
      store_remote(&s.count[turn][rank], threadIdx.x, count);
    }
    cluster_sync_all();
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
  // totals over the cluster
  __device__ __forceinline__ void add(u64& sum, uint32_t& count) {
    add_cta(sum, count);                           // (read again before the exchange's barrier only)
    exchange(sum, count);
    sum = 0, count = 0;
    for (int r = 0; r < size; ++r) sum += s.sum[turn][r], count += (uint32_t)s.count[turn][r];
  }
  // the sum of the threads before this one, and of all
  __device__ __forceinline__ u64 before(u64 v, u64& all) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    u64 run = v;
    for (int o = 1; o < 32; o <<= 1) {
      const u64 r = __shfl_up_sync(0xFFFFFFFFu, run, o);
      if (lane >= o) run += r;
    }
    __syncthreads();
    if (lane == 31) s.warp_sum[warp] = run;
    __syncthreads();
    u64 at = run - v;
    all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += s.warp_sum[w];
      all += s.warp_sum[w];
    }
    return at;
  }
};

// eight consecutive logits as they lie in memory
template <typename T>
struct Run;
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
  __device__ __forceinline__ void load_some(const float* p, int n) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = j < n ? __float_as_uint(p[j]) : kNone;
  }
  __device__ __forceinline__ float get(int j) const { return __uint_as_float(w[j]); }
  // infinities and NaN become -inf; returns the largest
  __device__ __forceinline__ float clean() {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v = fabsf(get(j)) <= FLT_MAX ? get(j) : -INFINITY;
      w[j] = __float_as_uint(v);
      m = fmaxf(m, v);
    }
    return m;
  }
  __device__ __forceinline__ float largest() const {
    float m = get(0);
#pragma unroll
    for (int j = 1; j < 8; ++j) m = fmaxf(m, get(j));
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
  __device__ __forceinline__ void load_some(const __nv_bfloat16* p, int n) {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = (2 * j < n ? q[2 * j] : kNone) | (2 * j + 1 < n ? q[2 * j + 1] : kNone) << 16;
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
    uint32_t bad = 0;                              // an exponent of all ones carries into the sign
#pragma unroll
    for (int j = 0; j < 4; ++j) bad |= (w[j] & 0x7F807F80u) + 0x00800080u;
    if (bad & 0x80008000u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if ((w[j] & 0x7F80u) == 0x7F80u) w[j] = (w[j] & 0xFFFF0000u) | kNone;
        if ((w[j] & 0x7F800000u) == 0x7F800000u) w[j] = (w[j] & 0xFFFFu) | kNone << 16;
      }
    return largest();
  }
};

// larger logit first, then lower index
__device__ __forceinline__ u64 make_key(float l, uint32_t idx) {
  return ((u64)ordered_key(l) << 32) | (0xFFFFFFFFu - idx);
}
__device__ __forceinline__ float key_logit(u64 k) { return ordered_value((uint32_t)(k >> 32)); }

// The end for n listed tokens, by one CTA: list[] in index order, sorted[] room for as
// many (kList).  k: how many are kept at most; want(mass of these): as in top-p.
__device__ __forceinline__ void finish(const Args& a, Team& team, const Weight& weight, const u64* __restrict__ list,
                                       u64* __restrict__ sorted, int n, int k, float p, float u, int row) {
  const Shared& s = team.s;
  const int tid = threadIdx.x;
  const int kk = min(n, k);
  u64 least = 0;                                   // the last key that is kept
  u64 total = 0;
  if (kk < n || p < 1.f) {
    if (n <= kCounted) {
      // every key's place is the number of larger ones
      if (tid < n) {
        const u64 mine = list[tid];
        int place = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) place += list[j] > mine;
        sorted[place] = mine;
      }
      __syncthreads();
    } else {
      int m = kCounted;
      while (m < n) m *= 2;
      for (int i = tid; i < m; i += kThreads) sorted[i] = i < n ? list[i] : 0;
      for (int size = 2; size <= m; size *= 2)
        for (int step = size / 2; step; step /= 2) {
          __syncthreads();
          for (int i = tid; i < m / 2; i += kThreads) {
            const int lo = 2 * i - (i & (step - 1)), hi = lo + step;
            const u64 x = sorted[lo], y = sorted[hi];
            if ((x < y) == ((lo & size) == 0)) sorted[lo] = y, sorted[hi] = x;
          }
        }
      __syncthreads();
    }
    // masses in that order, `each` places per thread
    const int each = (n + kThreads - 1) / kThreads, first = tid * each, behind = min(first + each, kk);
    int kept = kk;
    if (p < 1.f) {
      u64 mine = 0, all;
      for (int i = first; i < behind; ++i) mine += weight(key_logit(sorted[i]), s.powers);
      u64 at = team.before(mine, all);
      const u64 want = scaled(p, all, true);       // the mass before a kept token is below this
      int more = 0;
      for (int i = first; i < behind; ++i) {
        more += at < want;
        at += weight(key_logit(sorted[i]), s.powers);
      }
      u64 none = 0;
      uint32_t count = more;
      __syncthreads();
      team.add_cta(none, count);
      kept = max(1, (int)count);
    }
    least = sorted[kept - 1];
  }
  const int each = (n + kThreads - 1) / kThreads, first = tid * each, behind = min(first + each, n);
  u64 mine = 0;
  for (int i = first; i < behind; ++i)
    if (list[i] >= least) mine += weight(key_logit(list[i]), s.powers);
  u64 at = team.before(mine, total);
  const u64 target = scaled(u, total, false);
  if (at > target || at + mine <= target) return;
  for (int i = first; i < behind; ++i) {
    const u64 w = list[i] >= least ? weight(key_logit(list[i]), s.powers) : 0;
    if (at <= target && target < at + w) {
      a.token[row] = (int32_t)(0xFFFFFFFFu - (uint32_t)list[i]);
      if (a.prob) a.prob[row] = (float)((double)w / (double)total);
    }
    at += w;
  }
}

// chunk: logits of a CTA; steps: runs of eight per thread, so that the chunk fits the CTA
template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
    sample_kernel(const __grid_constant__ Args a, const T* __restrict__ logits, int chunk, int steps, int vec, DevCtx c) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ Shared sh;
  u64* list = (u64*)dyn;
  T* mine = (T*)(dyn + kList * sizeof(u64));
  let_next_launch();
  cluster_arrive();                                // no CTA writes to one that has not begun
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int size = (int)cluster_nctarank(), rank = (int)cluster_ctarank(), row = blockIdx.x / size;
  for (int i = tid; i < 256; i += kThreads) sh.powers[i] = kPowers.at[i];
  wait_for_earlier();
  // the request's settings
  const int q = a.index ? a.index[row] : row;
  bool ok = q >= 0 && q < a.requests;
  const float temp = ok && a.temperature ? a.temperature[q] : 1.f;
  ok = ok && temp >= 0.f && temp <= FLT_MAX;
  const bool greedy = temp == 0.f, draws = ok && !greedy;
  const float p = draws && a.top_p ? a.top_p[q] : 1.f, least = draws && a.min_p ? a.min_p[q] : 0.f;
  const float u = draws ? a.u[row] : 0.f;
  int k = draws && a.top_k ? a.top_k[q] : 0;
  ok = ok && k >= 0 && p > 0.f && p <= 1.f && least >= 0.f && least <= 1.f && u >= 0.f && u < 1.f;
  if (k == 0 || k > a.vocab) k = a.vocab;
  if (greedy) k = 1;
  if (tid == 0 && least > 0.f) sh.far = -log((double)least) * (double)temp;
  // The row's logits of this CTA to shared memory: a warp's together in index order, a
  // thread's in runs of eight.
  const int first = (warp * steps * 32 + lane) * kVec;
  const int there = min(chunk, a.vocab - rank * chunk);
  const T* src = logits + row * a.ld + rank * chunk;
  T* x = mine + first;
  float m = -INFINITY;
  constexpr int kAhead = sizeof(T) == 2 ? 8 : 4;   // runs in flight
  for (int s0 = 0; s0 < steps; s0 += kAhead) {
    Run<T> run[kAhead];
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      const int i = first + (s0 + s) * 32 * kVec;
      if (s0 + s >= steps) break;
      if (vec && i + kVec <= there) run[s].load(src + i);
      else run[s].load_some(src + i, there - i);
    }
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
  const uint32_t of_warp = __reduce_max_sync(0xFFFFFFFFu, best);
  if (lane == 0) sh.warp_count[warp] = of_warp;
  __syncthreads();
  uint32_t top = 0;
  for (int w = 0; w < kWarps; ++w) top = max(top, sh.warp_count[w]);
  uint32_t bound = 0;
  const bool small_k = k <= kSmallK && k < a.vocab;
  if (small_k) {
    const int need = (k + size - 1) / size;
    bound = top;
    if (need > 1) {
      uint32_t lo = 0, hi = top + 1, step = 1u << 18;  // fewer than `need` threads reach hi, at least as many lo
      while (hi - lo > 1) {
        const uint32_t mid = lo == 0 && hi > step ? hi - step : lo + (hi - lo) / 2;
        const int n = __syncthreads_count(best >= mid);
        if (n >= need) lo = mid;
        else hi = mid, step *= 2;
        if (n >= need && n <= need + need / 4 + 1) break;
        if (lo == 0 && step >= (1u << 30)) break;  // a CTA with few logits: all are candidates
      }
      bound = lo;
    }
  }
  cluster_wait();
  team.exchange(top, bound);
  for (int r = 0; r < size; ++r) {
    top = max(top, (uint32_t)sh.sum[team.turn][r]);
    bound = min(bound, (uint32_t)sh.count[team.turn][r]);
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
  Weight weight{m, 0.f, 0.f, a.unit};
  if (draws) {
    // (no fp64: its units are few)
    constexpr float kHi = 1.44269502162933349609375f, kLo = 1.9259629911e-8f;
    weight.hi = __fdiv_rn(kHi, temp);
    weight.lo = __fdiv_rn(__fadd_rn(__fmaf_rn(-weight.hi, temp, kHi), kLo), temp);
    if (!(weight.hi < 1e38f)) weight.hi = 1e38f, weight.lo = 0.f;
  }
  float cut = greedy ? m : -FLT_MAX;
  if (least > 0.f) {
    cut = fmaxf(__double2float_ru((double)m - sh.far), -FLT_MAX);
  }
  if (small_k || least > 0.f) {
    // Few tokens can be kept as a rule: CTA 0 gets them listed, in index order.
    const float low = small_k ? fmaxf(cut, fmaxf(ordered_value(bound), -FLT_MAX)) : cut;
    const int room = kList / size;
    uint32_t n = 0, with = 0;                      // steps with some (steps <= 32)
    for (int s = 0; s < steps; ++s) {
      Run<T> run;
      run.load(x + s * 32 * kVec);
      if (run.largest() >= low) {
        with |= 1u << s;
#pragma unroll
        for (int j = 0; j < kVec; ++j) n += run.get(j) >= low;
      }
    }
    with = __reduce_or_sync(0xFFFFFFFFu, with);
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if (lane == 0) sh.warp_count[warp] = n;
    __syncthreads();
    uint32_t at = 0, in_cta = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += sh.warp_count[w];
      in_cta += sh.warp_count[w];
    }
    if (in_cta <= (uint32_t)room)
      for (; with; with &= with - 1) {
        const int s = __ffs(with) - 1;
        Run<T> run;
        run.load(x + s * 32 * kVec);
        uint32_t hits = 0;
#pragma unroll
        for (int j = 0; j < kVec; ++j) hits |= (uint32_t)(run.get(j) >= low) << j;
        const uint32_t have = __popc(hits);
        uint32_t upto = have;
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t r = __shfl_up_sync(0xFFFFFFFFu, upto, o);
          if (lane >= o) upto += r;
        }
        uint32_t to = rank * room + at + upto - have;
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          if (hits >> j & 1)
            store_remote(&list[to++], 0, make_key(run.get(j), (uint32_t)(rank * chunk + first + s * 32 * kVec + j)));
        at += __shfl_sync(0xFFFFFFFFu, upto, 31);
      }
    team.exchange(0, in_cta);
    bool all = true;
    int total = 0;
    for (int r = 0; r < size; ++r) {
      all = all && sh.count[team.turn][r] <= (u64)room;
      total += (int)sh.count[team.turn][r];
    }
    if (all) {
      if (rank != 0) return;
      // together; each CTA's part moves towards the front
      if (size > 1) {
        u64 keep[kList / kThreads];
#pragma unroll
        for (int i = 0; i < kList / kThreads; ++i) keep[i] = list[tid + i * kThreads];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kList / kThreads; ++i) {
          const int from = tid + i * kThreads, r = from / room, o = from - r * room;
          int to = o;
          for (int b = 0; b < r; ++b) to += (int)sh.count[team.turn][b];
          if (o < (int)sh.count[team.turn][r]) list[to] = keep[i];
        }
        __syncthreads();
      }
      finish(a, team, weight, list, (u64*)mine, total, k, p, u, row);
      return;
    }
  }
  // Any number of tokens: bisection over the logits' bits.
  u64 mass = 0, sum = 0;
  uint32_t count = 0, ties = greedy ? 1u : 0x7FFFFFFFu;
  const uint32_t end = Grid<T>::up(m) + 1;
  uint32_t lo = Grid<T>::up(cut), hi = end;
  if (k < a.vocab && !greedy) {
    u64 none = 0;
    count = 0;
    each_logit([&](float l) { count += l >= cut; });
    team.add(none, count);
    if (count > (uint32_t)k) {
      uint32_t above = 0;                          // logits at hi and above
      while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        const float v = Grid<T>::value(mid);
        none = count = 0;
        each_logit([&](float l) { count += l >= v; });
        team.add(none, count);
        if (count >= (uint32_t)k) lo = mid;
        else hi = mid, above = count;
      }
      ties = k - above;
    }
  }
  if (!greedy) cut = Grid<T>::value(lo);
  // this thread's part of what is kept so far
  const auto kept_here = [&] {
    sum = 0, count = 0;
    each_logit([&](float l) {
      if (l > cut) sum += weight(l, sh.powers);
      count += l == cut;
    });
  };
  kept_here();
  if (p < 1.f) {
    mass = sum;
    uint32_t tied = count;
    team.add(mass, tied);
    ties = min(ties, tied);
    const u64 each = weight(cut, sh.powers);
    const u64 want = scaled(p, mass + ties * each, true);  // the mass before a kept token is below this
    if (mass < want) {                             // tokens at the cut are among them
      ties = (uint32_t)((want - mass + each - 1) / each);
    } else {
      u64 above = 0;                               // mass at hi and above
      hi = end;
      while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        const float v = Grid<T>::value(mid), w = hi == end ? INFINITY : Grid<T>::value(hi);
        u64 some = 0;
        uint32_t none = 0;
        each_logit([&](float l) {
          if (l >= v && l < w) some += weight(l, sh.powers);
        });
        team.add(some, none);
        some += above;
        if (some >= want) lo = mid;
        else hi = mid, above = some;
      }
      cut = Grid<T>::value(lo);
      const u64 one = weight(cut, sh.powers);
      ties = (uint32_t)((want - above + one - 1) / one);
      kept_here();
    }
  }
  // what each warp keeps, in the order of the tokens
  const u64 each = weight(cut, sh.powers);
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  count = __reduce_add_sync(0xFFFFFFFFu, count);
  if (lane == 0) sh.warp_sum[warp] = sum, sh.warp_count[warp] = count;
  __syncthreads();
  u64 cta_sum = 0;
  uint32_t cta_count = 0;
  for (int w = 0; w < kWarps; ++w) cta_sum += sh.warp_sum[w], cta_count += sh.warp_count[w];
  team.exchange(cta_sum, cta_count);
  u64 total = 0, before = 0;
  uint32_t tied = 0, tied_before = 0;
  // mass of n tokens at the cut when `seen` of them came before
  const auto tie_mass = [&](uint32_t seen, uint32_t n) { return (u64)(min(ties, seen + n) - min(ties, seen)) * each; };
  for (int r = 0; r < size; ++r) {
    const uint32_t n = (uint32_t)sh.count[team.turn][r];
    const u64 kept = sh.sum[team.turn][r] + tie_mass(tied, n);
    if (r < rank) before += kept, tied_before += n;
    total += kept;
    tied += n;
  }
  const u64 target = scaled(u, total, false);
  for (int w = 0; w < warp; ++w) {
    const uint32_t n = sh.warp_count[w];
    before += sh.warp_sum[w] + tie_mass(tied_before, n);
    tied_before += n;
  }
  if (before > target || before + sum + tie_mass(tied_before, count) <= target) return;
  // the one warp that holds the token, thread by thread
  for (int s = 0; s < steps; ++s) {
    Run<T> v;
    v.load(x + s * 32 * kVec);
    u64 run = 0;
    uint32_t tie_run = 0;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      if (v.get(j) > cut) run += weight(v.get(j), sh.powers);
      tie_run += v.get(j) == cut;
    }
    const u64 own = run;
    const uint32_t own_ties = tie_run;
    for (int o = 1; o < 32; o <<= 1) {
      const u64 r = __shfl_up_sync(0xFFFFFFFFu, run, o);
      const uint32_t n = __shfl_up_sync(0xFFFFFFFFu, tie_run, o);
      if (lane >= o) run += r, tie_run += n;
    }
    uint32_t seen = tied_before + (tie_run - own_ties);
    u64 at = before + (run - own) + tie_mass(tied_before, tie_run - own_ties);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const float l = v.get(j);
      u64 w = 0;
      if (l > cut) w = weight(l, sh.powers);
      else if (l == cut && seen++ < ties) w = each;
      if (at <= target && target < at + w) {
        a.token[row] = rank * chunk + first + s * 32 * kVec + j;
        if (a.prob) a.prob[row] = (float)((double)w / (double)total);
      }
      at += w;
    }
    run = __shfl_sync(0xFFFFFFFFu, run, 31);
    tie_run = __shfl_sync(0xFFFFFFFFu, tie_run, 31);
    before += run + tie_mass(tied_before, tie_run);
    tied_before += tie_run;
  }
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
  while (size < kMaxCluster && (size * (32768ll / (int)sizeof(T)) < a.vocab ||
                                ((long long)a.rows * size * 2 <= sms && size * 2048 < a.vocab)))
    size *= 2;
  const int chunk = (a.vocab + size * kVec - 1) / (size * kVec) * kVec, step = kThreads * kVec;
  const int steps = (chunk + step - 1) / step;
  const size_t room = (size_t)steps * step * sizeof(T), smem = kList * 8 + (room > kList * 8 ? room : kList * 8);
  const int vec = (((uintptr_t)logits | (uintptr_t)(a.ld * sizeof(T))) & 15u) == 0;
  return cuda_ok(cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) &&
         launch_programmatic(sample_kernel<T>, dim3((unsigned)(a.rows * size)), dim3(kThreads), smem, st, size, a,
                             (const T*)logits, chunk, steps, vec, c);
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
  const Args a{(int)p->rows, (int)p->vocab, (int)p->requests, 62 - bits, p->ld, u, temperature, top_p, min_p,
               top_k, index, token, prob};
  const bool ok = p->dtype == DSA_BF16 ? launch<__nv_bfloat16>(a, logits, c, (cudaStream_t)stream)
                                       : launch<float>(a, logits, c, (cudaStream_t)stream);
  return ok ? DSA_OK : DSA_ERR_CUDA;
}
