// Beam selection (dsa_beam_select): per request, the best beams_out of
//   cand(w, v) = score[w] + x[w, v] - log sum_u exp x[w, u]
// over its beams w and the vocabulary, ties to the lower w * vocab + v.
//
// Two kernels.  beam_part_kernel reads the logits once: one CTA per (beam row,
// chunk of the vocabulary), the chunk in registers.  Within a beam the order of
// the candidates is the order of the logits, so a chunk only has to give its
// best beams_out logits, its maximum m and its sum of exp(x - m).  With c =
// ceil(beams_out / 4), the smallest of the 4 warps' c-th largest thread maxima
// bounds the chunk's beams_out-th largest logit from below (4 c threads have a
// logit at least that large); some 20 logits of a chunk pass it for 8 beams.
// Those are ranked by counting, as keys (order-preserving bits of the logit,
// inverted index), which are unique.  Should too many pass (equal logits), the
// bound is taken again over keys, which lets the logits of at most beams_out threads pass.
// An infinity or NaN shows in the maximum or the sum; only then are the logits
// looked at one by one.
// beam_join_kernel (one CTA per request) adds the chunks' sums in 64 bits and
// ranks the candidates by their 64-bit scores.
//
// Candidates of different beams can lie close together, and their order is an
// output: the sums are fp32 only inside a thread, a warp adds them as integers
// (2^-40 of its largest term: the order does not matter), everything after that
// is fp64 or as exact.  A row gives the same bits wherever it lies: which element a
// thread takes depends on its index alone, not on alignment.
//
// Bound: for a batch, the logits' way from HBM and some 10 instructions per logit,
// of which the CTAs of a wave do first the one and then the other: 64 x 8 beams x
// 131071 bf16 take 33 us, 4.1 TB/s; the first kernel alone 26 us, 5.1 TB/s.
// Loading the next chunk ahead of the sums took more registers than it gave.  One
// request of 4 x 32001: 7.8 us, the two launches and their latencies.
#include <math.h>

#include "dsa_common.cuh"

namespace dsa {

bool ext_dev_ctx(DevCtx* c);

namespace beam {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kVec = 8;                            // consecutive elements per thread and step
// elements per thread and CTA: 8,192 (bf16) or 4,096 (fp32) logits, 32 registers
// (CTAs of 256 threads and twice the logits took 0.6 us less for 64 x 8 beams x
// 131071 bf16, but 1.1 us more for one request of 4 x 32001)
constexpr int kStepsBf16 = 8, kStepsFp32 = 4;
constexpr int kMaxPerThread = kStepsBf16 * kVec;
constexpr int chunk_of(int dtype) { return kThreads * kVec * (dtype == DSA_BF16 ? kStepsBf16 : kStepsFp32); }
constexpr int kMaxBeams = 32;                      // in and out
constexpr int kMaxRuns = 128;                      // runs of eight logits that hold some
constexpr int kMaxCand = kMaxPerThread * kMaxBeams;  // candidates of a chunk at most, see beam_part_kernel

struct Args {
  int n_batch, win, wout, vocab, chunks;
  long long ld;
  int eos;
};
// per (row, chunk, warp): maximum, and sum of exp(x - max) in units of 2^-40
struct Stat {
  unsigned long long sum;
  float max, pad;
};
constexpr float kUnit = 1099511627776.f;           // 2^40

// larger logit first, then lower index; 0: no logit
__device__ __forceinline__ unsigned long long make_key(float x, uint32_t idx) {
  return ((unsigned long long)ordered_key(x) << 32) | (0xFFFFFFFFu - idx);
}
__device__ __forceinline__ float ordered_value(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  return ordered_value((uint32_t)(k >> 32));
}
__device__ __forceinline__ uint32_t key_index(unsigned long long k) { return 0xFFFFFFFFu - (uint32_t)k; }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two floats in one register pair
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
constexpr float kLog2e = 1.4426950408889634f;
// Below this size of the maximum m, x log2e - m log2e is one fused product.  From here on
// the difference comes first: m log2e's rounding error, 2^-25 of it, would be more than a
// few terms' own errors, and from 2^31 on its power of two overflows.  (64 x 8 beams x
// 131071 bf16 of which 99 % are masked by -1e9: 37 us; read again one by one 93.)
constexpr float kFused = 1048576.f;

// a thread's logits in registers, in runs of eight.  kResident: CTAs per SM; bf16
// 64 x 8 beams x 131071 35.5 / 33.6 / 32.2 / 36.2 us with 7 / 8 / 9 / 10 (registers
// against loads in flight), fp32 64 x 8 x 64000 31.0 / 33.0 us with 8 / 9.
template <typename T>
struct Logits;
template <>
struct Logits<float> {
  static constexpr int kSteps = kStepsFp32, kResident = 8;
  float x[kSteps][kVec];
  __device__ __forceinline__ void load16(int s, const float* p) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    x[s][0] = a.x, x[s][1] = a.y, x[s][2] = a.z, x[s][3] = a.w;
    x[s][4] = b.x, x[s][5] = b.y, x[s][6] = b.z, x[s][7] = b.w;
  }
  __device__ __forceinline__ void load1(int s, const float* p, int n) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) x[s][i] = i < n ? __ldcs(p + i) : -INFINITY;
  }
  __device__ __forceinline__ float get(int s, int e) const { return x[s][e]; }
  __device__ __forceinline__ void put_run(int s, float* p) const {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[s][0], x[s][1], x[s][2], x[s][3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[s][4], x[s][5], x[s][6], x[s][7]);
  }
  __device__ __forceinline__ float run_max(int s) const {
    float m = x[s][0];
#pragma unroll
    for (int e = 1; e < kVec; ++e) m = fmaxf(m, x[s][e]);
    return m;
  }
  __device__ __forceinline__ float max() const {
    float m = run_max(0);
#pragma unroll
    for (int s = 1; s < kSteps; ++s) m = fmaxf(m, run_max(s));
    return m;
  }
  // logits that may not be chosen count as -inf
  __device__ __forceinline__ void clean() {
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int e = 0; e < kVec; ++e) x[s][e] = x[s][e] < INFINITY ? x[s][e] : -INFINITY;
  }
};
template <>
struct Logits<__nv_bfloat16> {
  static constexpr int kSteps = kStepsBf16, kResident = 9;
  uint32_t w[kSteps][kVec / 2];                    // two each, the first in the low half
  __device__ __forceinline__ void load16(int s, const __nv_bfloat16* p) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
    w[s][0] = a.x, w[s][1] = a.y, w[s][2] = a.z, w[s][3] = a.w;
  }
  __device__ __forceinline__ void load1(int s, const __nv_bfloat16* p, int n) {
    const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
    for (int i = 0; i < kVec / 2; ++i) {
      const uint32_t lo = 2 * i < n ? __ldcs(q + 2 * i) : 0xFF80u, hi = 2 * i + 1 < n ? __ldcs(q + 2 * i + 1) : 0xFF80u;
      w[s][i] = lo | (hi << 16);
    }
  }
  __device__ __forceinline__ float get(int s, int e) const {
    return __uint_as_float((e & 1) ? w[s][e >> 1] & 0xFFFF0000u : w[s][e >> 1] << 16);
  }
  __device__ __forceinline__ void put_run(int s, __nv_bfloat16* p) const {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[s][0], w[s][1], w[s][2], w[s][3]);
  }
  __device__ __forceinline__ uint32_t run_max2(int s) const {
    uint32_t t = w[s][0];
#pragma unroll
    for (int i = 1; i < kVec / 2; ++i) asm("max.bf16x2 %0, %0, %1;" : "+r"(t) : "r"(w[s][i]));
    return t;
  }
  static __device__ __forceinline__ float larger(uint32_t t) {
    return fmaxf(__uint_as_float(t << 16), __uint_as_float(t & 0xFFFF0000u));
  }
  __device__ __forceinline__ float run_max(int s) const { return larger(run_max2(s)); }
  __device__ __forceinline__ float max() const {
    uint32_t t = run_max2(0);
#pragma unroll
    for (int s = 1; s < kSteps; ++s) asm("max.bf16x2 %0, %0, %1;" : "+r"(t) : "r"(run_max2(s)));
    return larger(t);
  }
  __device__ __forceinline__ void clean() {
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int i = 0; i < kVec / 2; ++i) {
        const float lo = __uint_as_float(w[s][i] << 16), hi = __uint_as_float(w[s][i] & 0xFFFF0000u);
        w[s][i] = (lo < INFINITY ? w[s][i] & 0xFFFFu : 0xFF80u) | (hi < INFINITY ? w[s][i] & 0xFFFF0000u : 0xFF800000u);
      }
  }
};

// f(logit, index) for a thread's logits, read again (from L2): for the rare
// paths, whose unrolled code would crowd the instruction cache
template <typename T, typename F>
__device__ __forceinline__ void reread(const T* row, int first, int vocab, F f) {
#pragma unroll 1
  for (int s = 0; s < Logits<T>::kSteps; ++s)
#pragma unroll 1
    for (int e = 0; e < kVec; ++e) {
      const int i = first + s * kThreads * kVec + e;
      if (i >= vocab) continue;
      const float y = to_f32<T>(row[i]);
      f(y < INFINITY ? y : -INFINITY, i);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, Logits<T>::kResident)
    beam_part_kernel(Args a, const T* __restrict__ logits, const float* __restrict__ scores,
                     const uint8_t* __restrict__ finished, Stat* __restrict__ stats,
                     unsigned long long* __restrict__ keys, int vec) {
  constexpr int kSteps = Logits<T>::kSteps, kChunk = kThreads * kVec * kSteps;
  __shared__ unsigned long long cand[kMaxCand], tmax[kThreads], kth;
  __shared__ __align__(16) T runs[kMaxRuns][kVec];
  __shared__ int run_at[kMaxRuns];
  __shared__ uint32_t wleast[kWarps];
  __shared__ int n_cand, n_runs;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = a.wout;
  const uint32_t item = blockIdx.x, row = item / (uint32_t)a.chunks;
  const int first = (int)(item - row * (uint32_t)a.chunks) * kChunk + tid * kVec;  // this thread's first logit
  let_next_launch();
  wait_for_earlier();
  // a finished beam has no logits, a beam of score -inf no candidates
  if ((finished && finished[row]) || !(scores[row] > -INFINITY)) return;
  if (tid == 0) n_cand = n_runs = 0;
  Logits<T> x;
  const T* xrow = logits + (long long)row * a.ld;
  {
    const T* base = xrow + first;
    if (vec && first + (kSteps - 1) * kThreads * kVec + kVec <= a.vocab) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) x.load16(s, base + s * kThreads * kVec);
    } else {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int left = a.vocab - first - s * kThreads * kVec;
        if (vec && left >= kVec) x.load16(s, base + s * kThreads * kVec);
        else x.load1(s, base + s * kThreads * kVec, left);
      }
    }
  }
  float m;
  for (int pass = 0; pass < 2; ++pass) {
    m = x.max();
    // sum of exp(x - m) over the thread
    float part = 0.f;
    if (fabsf(m) < kFused) {
      // 2^(x log2e - mu) with mu = m log2e as rounded; its rounding error, below 2^-4,
      // which a fused product gives exactly, is taken out of the sum at the end
      const float mu = m * kLog2e;
      const uint64_t minus = pack2(-mu, -mu);
      uint64_t p[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int e = 0; e < kVec; e += 2) {
          float lo, hi;
          unpack2(ffma2(kLog2e, kLog2e, x.get(s, e), x.get(s, e + 1), minus), lo, hi);
          p[e >> 1] = add2(p[e >> 1], pack2(ex2(lo), ex2(hi)));
        }
      float lo, hi;
      unpack2(add2(add2(p[0], p[1]), add2(p[2], p[3])), lo, hi);
      part = (lo + hi) * ex2(-fmaf(m, kLog2e, -mu));
    } else if (m == INFINITY || m != m) {
      part = m;                                    // the vote below sees it
    } else if (m != -INFINITY) {                   // (a finite mask, say)
      const uint64_t minus = pack2(-m, -m);
      uint64_t p[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int e = 0; e < kVec; e += 2) {
          float lo, hi;
          unpack2(add2(pack2(x.get(s, e), x.get(s, e + 1)), minus), lo, hi);
          p[e >> 1] = add2(p[e >> 1], pack2(ex2(lo * kLog2e), ex2(hi * kLog2e)));
        }
      float lo, hi;
      unpack2(add2(add2(p[0], p[1]), add2(p[2], p[3])), lo, hi);
      part = lo + hi;
    }
    // the warp's c-th largest thread maximum
    uint32_t v = ordered_key(m), top = 0, largest = 0;
    for (int r = (k + kWarps - 1) / kWarps; r > 0; --r) {
      top = __reduce_max_sync(0xffffffffu, v);
      if (largest == 0) largest = top;
      if (__ffs(__ballot_sync(0xffffffffu, v == top)) - 1 == lane) v = 0;
    }
    const float wm = ordered_value(largest);
    // at most 64 terms of at most 1 per thread: below 2^50, two halves of 25 bits
    const unsigned long long fix = m == -INFINITY ? 0ull : __float2ull_rn(part * ex2((m - wm) * kLog2e) * kUnit);
    const uint32_t lo = __reduce_add_sync(0xffffffffu, (uint32_t)fix & 0x1FFFFFFu);
    const uint32_t hi = __reduce_add_sync(0xffffffffu, (uint32_t)(fix >> 25));
    if (lane == 0) {
      wleast[warp] = top;
      Stat& o = stats[(size_t)item * kWarps + warp];
      o.sum = ((unsigned long long)hi << 25) + lo;
      o.max = wm;
    }
    // an infinity or NaN among the logits: once more without them
    if (!__syncthreads_or(part != part || m == INFINITY || m != m) || pass == 1) break;
    x.clean();
  }
  uint32_t least = wleast[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) least = least < wleast[w] ? least : wleast[w];
  // (too few logits for a bound: every one passes)
  const float from = least == 0 ? -3.402823466e38f : fmaxf(ordered_value(least), -3.402823466e38f);
  // the runs with such a logit go to shared memory as they are (to pick their
  // logits out here, every lane of the warp would wait for each of them)
  if (m >= from) {
    uint32_t hit = 0;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) hit |= x.run_max(s) >= from ? 1u << s : 0u;
    int at = atomicAdd(&n_runs, __popc(hit));
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      if ((hit >> s) & 1u) {
        if (at < kMaxRuns) {
          x.put_run(s, runs[at]);
          run_at[at] = first + s * kThreads * kVec;
        }
        ++at;
      }
  }
  __syncthreads();
  const int nr = n_runs;
  if (nr <= kMaxRuns) {
    for (int i = tid; i < nr * kVec; i += kThreads) {
      const float y = to_f32<T>(runs[i / kVec][i % kVec]);
      if (y >= from) cand[atomicAdd(&n_cand, 1)] = make_key(y, run_at[i / kVec] + i % kVec);
    }
  } else {                                         // many equal logits: bound by unique keys
    unsigned long long best = 0;
    reread(xrow, first, a.vocab, [&](float y, int i) {
      if (y == m && m != -INFINITY) best = best > make_key(y, i) ? best : make_key(y, i);
    });
    tmax[tid] = best;
    const int have = __syncthreads_count(best != 0);  // threads with a logit
    int rank = 0;
    for (int t = 0; t < kThreads; ++t) rank += tmax[t] > best;
    if (rank == k - 1 && best != 0) kth = best;
    __syncthreads();
    const unsigned long long lowest = have < k ? 1ull : kth;
    reread(xrow, first, a.vocab, [&](float y, int i) {
      const unsigned long long key = make_key(y, i);
      if (y != -INFINITY && key >= lowest) cand[atomicAdd(&n_cand, 1)] = key;  // only k threads have such keys
    });
  }
  __syncthreads();
  const int n = n_cand;
  unsigned long long* out = keys + (size_t)item * k;
  for (int i = tid; i < n; i += kThreads) {
    const unsigned long long mine = cand[i];
    int r = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) r += cand[j] > mine;
    if (r < k) out[r] = mine;
  }
  for (int i = n + tid; i < k; i += kThreads) out[i] = 0;
}

// order-preserving map of a double (no NaN)
__device__ __forceinline__ unsigned long long ordered64(double x) {
  const long long u = __double_as_longlong(x + 0.0);
  return (unsigned long long)u ^ ((unsigned long long)(u >> 63) | 0x8000000000000000ull);
}

// ln(t 2^-unit) for t >= 2^(unit-1), to 2e-11: t = f 2^e with f in [0.707, 1.414],
// ln f = 2 artanh s, s = (f - 1) / (f + 1), |s| < 0.172, by its power series.  fp64
// instructions are slow here (some 15 cycles of the SM each), so the quotient is an fp32
// one and its remainder, and the series is fp32 from s^5 on (at most 2e-4 of the whole;
// up to s^13, the next term is below 1e-12).  One request took 7.3 us with the logarithm
// all in fp32, but candidates of different beams that lie closer than 2^-25 changed
// places; 7.8 like this, 8.0 all in fp64.
__device__ __forceinline__ double log_of(unsigned long long t, int unit) {
  int e = 63 - __clzll((long long)t);
  const unsigned long long frac = e > 52 ? t >> (e - 52) : t << (52 - e);  // 53 bits, the first one 1
  double f = __longlong_as_double((long long)((frac & 0xFFFFFFFFFFFFFull) | 0x3FF0000000000000ull));
  if (f > 1.4142135623730951) {
    f *= 0.5;
    ++e;
  }
  // the quotient: fp32, corrected by its remainder
  const double a = f - 1.0, b = f + 1.0;
  const float bf = __frcp_rn((float)b), s0 = (float)a * bf;
  const double s = (double)s0 + (double)((float)fma(-(double)s0, b, a) * bf), z = s * s;
  const float y = s0 * s0;
  float p = 1.f / 13.f;
  p = fmaf(p, y, 1.f / 11.f);
  p = fmaf(p, y, 1.f / 9.f);
  p = fmaf(p, y, 1.f / 7.f);
  p = fmaf(p, y, 1.f / 5.f);
  const double c = 2.0 * s, r = z * (1.0 / 3.0 + (double)(p * y));
  return fma((double)(e - unit), 0.6931471805599453, fma(c, r, c));
}

// sum w / 4, w <= 1 taken to 2^-32: the product of integers keeps the sum's bits
__device__ __forceinline__ unsigned long long scaled(unsigned long long sum, float w) {
  return __umul64hi(sum, (unsigned long long)__float2uint_rn(w * 2147483648.f) << 31);
}

// A beam's `k` best keys out of its chunks' sorted lists kr[chunk][k] (one warp, a
// lane has NL lists); how many there are.
template <int NL>
__device__ __forceinline__ int merge_lists(const unsigned long long* kr, int chunks, int k, unsigned long long* list) {
  const int lane = threadIdx.x & 31;
  int pos[NL];
  unsigned long long head[NL];
#pragma unroll
  for (int q = 0; q < NL; ++q) {
    pos[q] = 0;
    head[q] = lane + 32 * q < chunks ? kr[(lane + 32 * q) * k] : 0;
  }
  int got = 0;
  for (; got < k; ++got) {
    unsigned long long best = head[0];
#pragma unroll
    for (int q = 1; q < NL; ++q) best = head[q] > best ? head[q] : best;
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
    const unsigned long long win = ((unsigned long long)hi << 32) | lo;
    if (win == 0) break;
    if (best == win) {                             // keys are unique: one list of one lane
      list[got] = win;
#pragma unroll
      for (int q = 0; q < NL; ++q)
        if (head[q] == win) head[q] = ++pos[q] < k ? kr[(lane + 32 * q) * k + pos[q]] : 0;
    }
  }
  return got;
}
// the same for any number of chunks: each time the largest key below the last one
__device__ __forceinline__ int merge_any(const unsigned long long* kr, int chunks, int k, unsigned long long* list) {
  const int lane = threadIdx.x & 31;
  unsigned long long last = ~0ull;
  int got = 0;
  for (; got < k; ++got) {
    unsigned long long best = 0;
    for (int i = lane; i < chunks * k; i += 32) {
      const unsigned long long v = kr[i];
      if (v < last && v > best) best = v;
    }
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
    last = ((unsigned long long)hi << 32) | lo;
    if (last == 0) break;
    if (lane == 0) list[got] = last;
  }
  return got;
}

// One CTA per request.  Per beam, one warp merges its chunks' sorted lists (lane =
// chunk and every 32nd after it, the largest head taken each time) while another
// adds the chunks' sums and takes the logarithm; then every candidate has a thread,
// which computes its score and, by a binary search in each beam's list, its place.
// One warp takes the logarithms of all beams (lane = beam), in the time of the merges.
// Bound: latency, of which beams_out rounds of warp reductions and the logarithm are the
// most; the lists are read from global memory once, all loads in flight, where they fit
// (with a load per round, sum and merge in one warp, and the beams merged by a warp,
// 2 us more for one request).
constexpr int kJoinWarps = 8, kJoinThreads = 2 * 32 * kJoinWarps;
constexpr int kLists = 4;                           // per lane: 128 chunks, 1M (bf16) or 512K logits
constexpr int kKeyRoom = 512;                       // keys per warp
__global__ void __launch_bounds__(kJoinThreads)
    beam_join_kernel(Args a, const float* __restrict__ scores, const uint8_t* __restrict__ finished,
                     const Stat* __restrict__ stats, const unsigned long long* __restrict__ keys,
                     int32_t* __restrict__ parent, int32_t* __restrict__ token, float* __restrict__ scores_out,
                     uint8_t* __restrict__ finished_out) {
  __shared__ unsigned long long room[kJoinWarps][kKeyRoom];
  __shared__ unsigned long long list[kMaxBeams][kMaxBeams + 1];  // best first: keys, then ordered scores; 0: none
  __shared__ int32_t index[kMaxBeams][kMaxBeams];  // their tokens
  __shared__ float top[kMaxBeams];                 // a beam's largest logit, and the logarithm of
  __shared__ double ln[kMaxBeams];                 // its sum of exp(x - top): added, a large top would take its bits
  __shared__ unsigned long long sum[kMaxBeams];    // that sum, in units of 2^-38; 0: no logit
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, k = a.wout;
  const int wj = (tid >> 5) % kJoinWarps;
  const bool merges = tid < 32 * kJoinWarps;
  let_next_launch();
  wait_for_earlier();
  for (int w = wj; w < a.win; w += kJoinWarps) {
    const long long row = (long long)b * a.win + w;
    const float sc = scores[row];
    const bool done = finished && finished[row];
    const bool open = !done && sc > -INFINITY;      // (what other beams' lists and sums hold is unspecified)
    if (merges) {
      const int have = a.chunks * k;
      const unsigned long long* kr = keys + row * have;
      if (have <= kKeyRoom) {
#pragma unroll 4
        for (int i = lane; i < have; i += 32) room[wj][i] = kr[i];
        __syncwarp();
        kr = room[wj];
      }
      int got = 0;
      if (open) {
        got = a.chunks <= 32            ? merge_lists<1>(kr, a.chunks, k, list[w])
              : a.chunks <= 32 * kLists ? merge_lists<kLists>(kr, a.chunks, k, list[w])
                                        : merge_any(kr, a.chunks, k, list[w]);
      }
      if (done && sc > -INFINITY) {
        if (lane == 0) list[w][0] = ~0ull;         // the end token at the beam's score
        got = 1;
      }
      for (int r = got + lane; r < k; r += 32) list[w][r] = 0;
      __syncwarp();                                // room is read
    } else if (open) {
      const Stat* s = stats + row * a.chunks * kWarps;
      const int ns = a.chunks * kWarps;
      float m = -INFINITY;
#pragma unroll 4
      for (int c = lane; c < ns; c += 32) m = fmaxf(m, s[c].max);
      m = ordered_value(__reduce_max_sync(0xffffffffu, ordered_key(m)));
      unsigned long long t = 0;
      if (m != -INFINITY) {
#pragma unroll 4
        for (int c = lane; c < ns; c += 32)
          t += scaled(s[c].sum, expf(s[c].max - m));  // (no logit in a warp: 0 * 0)
#pragma unroll
        for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      }
      if (lane == 0) {
        top[w] = m;
        sum[w] = t;
      }
    } else if (lane == 0) {
      sum[w] = 0;
    }
  }
  if (!merges) {                                   // the logarithms, lane = beam, while the lists are merged
    named_bar_sync(1, 32 * kJoinWarps);
    if (wj == 0 && lane < a.win && sum[lane] != 0) ln[lane] = log_of(sum[lane], 38);
  }
  __syncthreads();
  for (int i = tid; i < a.win * k; i += kJoinThreads) {
    const int w = i / k, r = i - w * k;
    const unsigned long long key = list[w][r];
    if (key == 0) continue;
    const long long row = (long long)b * a.win + w;
    const double sc = (double)scores[row];
    const bool done = finished && finished[row];
    list[w][r] = ordered64(done ? sc : sc + (((double)key_value(key) - (double)top[w]) - ln[w]));
    index[w][r] = done ? a.eos : (int)key_index(key);
  }
  __syncthreads();
  // a candidate's place: how many of every beam's (sorted) list are better.  Equal
  // scores: the lower beam, within a beam the list's order.
  const int items = a.win * k;
  int n = 0;
  for (int i0 = 0; i0 < items; i0 += kJoinThreads) {
    const int i = i0 + tid, w = i / k, r = i - w * k;
    const unsigned long long cs = i < items ? list[w][r] : 0;
    n += __syncthreads_count(cs != 0);
    if (cs == 0) continue;
    int place = r;
#pragma unroll 4
    for (int v = 0; v < a.win; ++v) {
      if (v == w) continue;
      const unsigned long long least = v < w ? cs : cs + 1;  // scores from here on are better
      int lo = 0, hi = k;                          // entries below lo are better, from hi on they are not
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (list[v][mid] >= least) lo = mid + 1;
        else hi = mid;
      }
      place += lo;
    }
    if (place >= k) continue;
    const long long o = (long long)b * k + place, row = (long long)b * a.win + w;
    const int v = index[w][r];
    const unsigned long long u = (cs & 0x8000000000000000ull) ? cs ^ 0x8000000000000000ull : ~cs;
    parent[o] = (int32_t)row;
    token[o] = v;
    scores_out[o] = (float)__longlong_as_double((long long)u);
    if (finished_out) finished_out[o] = (finished && finished[row]) || v == a.eos;
  }
  for (int r = n + tid; r < k; r += kJoinThreads) {  // too few candidates
    const long long o = (long long)b * k + r;
    parent[o] = token[o] = -1;
    scores_out[o] = -INFINITY;
    if (finished_out) finished_out[o] = 0;
  }
}

static int check(const dsa_beam* p, Args* a) {
  if (!p) return DSA_ERR_INVALID_ARG;
  if (p->dtype != DSA_BF16 && p->dtype != DSA_FP32) return DSA_ERR_UNSUPPORTED;
  if (p->n_batch < 1 || p->beams_in < 1 || p->beams_out < 1 || p->vocab < 1 || p->ld < p->vocab || p->eos < -1 ||
      p->eos >= p->vocab)
    return DSA_ERR_INVALID_ARG;
  if (p->beams_in > kMaxBeams || p->beams_out > kMaxBeams || p->vocab > (1 << 24) || p->ld > (1ll << 40) ||
      p->n_batch >= (1ll << 31) ||
      p->n_batch * p->beams_in * ((p->vocab + chunk_of(p->dtype) - 1) / chunk_of(p->dtype)) >= (1ll << 31))
    return DSA_ERR_UNSUPPORTED;
  a->n_batch = (int)p->n_batch;
  a->win = (int)p->beams_in;
  a->wout = (int)p->beams_out;
  a->vocab = (int)p->vocab;
  a->chunks = (int)((p->vocab + chunk_of(p->dtype) - 1) / chunk_of(p->dtype));
  a->ld = p->ld;
  a->eos = (int)p->eos;
  return DSA_OK;
}
static bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}
static size_t stat_bytes(const Args& a) { return (size_t)a.n_batch * a.win * a.chunks * kWarps * sizeof(Stat); }

}  // namespace beam
}  // namespace dsa

using namespace dsa;
using namespace dsa::beam;

extern "C" {

size_t dsa_beam_workspace_size(const dsa_beam* p) {
  Args a;
  if (check(p, &a) != DSA_OK) return 0;
  return stat_bytes(a) + (size_t)a.n_batch * a.win * a.chunks * a.wout * 8;
}

int dsa_beam_select(const dsa_beam* p, const void* logits, const float* scores, const uint8_t* finished,
                    int32_t* parent, int32_t* token, float* scores_out, uint8_t* finished_out, void* workspace,
                    dsa_stream_t stream) {
  Args a;
  int rc = check(p, &a);
  if (rc) return rc;
  if (!logits || !scores || !parent || !token || !scores_out) return DSA_ERR_INVALID_ARG;
  if (finished && p->eos < 0) return DSA_ERR_INVALID_ARG;
  const uintptr_t esz = p->dtype == DSA_BF16 ? 2 : 4;
  if (((uintptr_t)logits & (esz - 1)) != 0 ||
      (((uintptr_t)scores | (uintptr_t)parent | (uintptr_t)token | (uintptr_t)scores_out) & 3u) != 0)
    return DSA_ERR_INVALID_ARG;
  // one request's results over another's beams
  const size_t in = (size_t)a.n_batch * a.win, out = (size_t)a.n_batch * a.wout;
  if (overlap(scores, 4 * in, scores_out, 4 * out) ||
      (finished && finished_out && overlap(finished, in, finished_out, out)))
    return DSA_ERR_INVALID_ARG;
  if (!workspace || ((uintptr_t)workspace & 15u) != 0) return DSA_ERR_WORKSPACE;
  DevCtx c;
  if (!ext_dev_ctx(&c)) return DSA_ERR_CUDA;
  Stat* stats = (Stat*)workspace;
  unsigned long long* keys = (unsigned long long*)((uint8_t*)workspace + stat_bytes(a));
  cudaStream_t st = (cudaStream_t)stream;
  const int vec = (((uintptr_t)logits | (uintptr_t)(p->ld * esz)) & 15u) == 0;
  const long long items = (long long)a.n_batch * a.win * a.chunks;
  const unsigned grid = (unsigned)items;
  const bool ok =
      p->dtype == DSA_BF16
          ? launch_programmatic(beam_part_kernel<__nv_bfloat16>, dim3(grid), dim3(kThreads), 0, st, 1, a,
                                (const __nv_bfloat16*)logits, scores, finished, stats, keys, vec)
          : launch_programmatic(beam_part_kernel<float>, dim3(grid), dim3(kThreads), 0, st, 1, a, (const float*)logits,
                                scores, finished, stats, keys, vec);
  if (!ok) return DSA_ERR_CUDA;
  return launch_programmatic(beam_join_kernel, dim3(a.n_batch), dim3(kJoinThreads), 0, st, 1, a, scores, finished,
                             (const Stat*)stats, (const unsigned long long*)keys, parent, token, scores_out,
                             finished_out)
             ? DSA_OK
             : DSA_ERR_CUDA;
}

}  // extern "C"
