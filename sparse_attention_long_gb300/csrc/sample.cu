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
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kVec = 8;                            // consecutive logits of a thread
constexpr int kChunk = 32768;                      // logits of a CTA at most
constexpr int kMaxVocab = kMaxCluster * kChunk;

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
  u64 warp_sum[kWarps];
  uint32_t warp_count[kWarps];
  float warp_max[kWarps];
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
  // totals over the cluster
  __device__ __forceinline__ void add(u64& sum, uint32_t& count) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    count = __reduce_add_sync(0xFFFFFFFFu, count);
    // (the last exchange's barrier came after its reads of these)
    if (lane == 0) s.warp_sum[warp] = sum, s.warp_count[warp] = count;
    __syncthreads();
    sum = 0, count = 0;
    for (int w = 0; w < kWarps; ++w) sum += s.warp_sum[w], count += s.warp_count[w];
    exchange(sum, count);
    sum = 0, count = 0;
    for (int r = 0; r < size; ++r) sum += s.sum[turn][r], count += (uint32_t)s.count[turn][r];
  }
  __device__ __forceinline__ float largest(float x) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
    if (lane == 0) s.warp_max[warp] = x;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) x = fmaxf(x, s.warp_max[w]);
    exchange(__float_as_uint(x), 0);
    for (int r = 0; r < size; ++r) x = fmaxf(x, __uint_as_float((uint32_t)s.sum[turn][r]));
    return x;
  }
};

// eight consecutive logits
__device__ __forceinline__ void load8(const float* p, float (&v)[kVec]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[kVec]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}

__device__ __forceinline__ void store8(float* p, const float (&v)[kVec]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[kVec]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7]));
}

// chunk: logits of a CTA; steps: runs of eight per thread, so that the chunk fits the CTA
template <typename T>
__global__ void __launch_bounds__(kThreads)
    sample_kernel(const __grid_constant__ Args a, const T* __restrict__ logits, int chunk, int steps, int vec, DevCtx c) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ Shared sh;
  let_next_launch();
  cluster_arrive();                                // no CTA writes to one that has not begun
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int size = (int)cluster_nctarank(), rank = (int)cluster_ctarank(), row = blockIdx.x / size;
  if (tid < 256) sh.powers[tid] = kPowers.at[tid];
  wait_for_earlier();
  // the request's settings
  const int q = a.index ? a.index[row] : row;
  bool ok = q >= 0 && q < a.requests;
  const float temp = ok && a.temperature ? a.temperature[q] : 1.f;
  ok = ok && temp >= 0.f && temp <= FLT_MAX;
  const bool greedy = temp == 0.f, draws = ok && !greedy;
  const float p = draws && a.top_p ? a.top_p[q] : 1.f, least = draws && a.min_p ? a.min_p[q] : 0.f;
  const float u = draws ? a.u[row] : 0.f;
  const int k = draws && a.top_k ? a.top_k[q] : 0;
  ok = ok && k >= 0 && p > 0.f && p <= 1.f && least >= 0.f && least <= 1.f && u >= 0.f && u < 1.f;
  // The row's logits of this CTA to shared memory: a warp's together in index order, a
  // thread's in runs of eight.
  const int first = (warp * steps * 32 + lane) * kVec;
  const int there = min(chunk, a.vocab - rank * chunk);
  const T* src = logits + row * a.ld + rank * chunk;
  T* x = (T*)dyn + first;
  float m = -INFINITY;
#pragma unroll 4
  for (int s = 0; s < steps; ++s) {
    const int i = first + s * 32 * kVec;
    float v[kVec];
    if (vec && i + kVec <= there) {
      load8(src + i, v);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[j] = i + j < there ? to_f32(src[i + j]) : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      v[j] = fabsf(v[j]) <= FLT_MAX ? v[j] : -INFINITY;  // infinities and NaN are never chosen
      m = fmaxf(m, v[j]);
    }
    store8(x + s * 32 * kVec, v);
  }
  // f(logit) over this thread's logits
  const auto each_logit = [&](auto f) {
    for (int s = 0; s < steps; ++s) {
      float v[kVec];
      load8(x + s * 32 * kVec, v);
#pragma unroll
      for (int j = 0; j < kVec; ++j) f(v[j]);
    }
  };
  Team team{sh, rank, size, 0};
  cluster_wait();
  m = team.largest(m);
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
    const double f = fmin(1.4426950408889634 / (double)temp, 1e38);
    weight.hi = (float)f;
    weight.lo = (float)(f - (double)weight.hi);
  }
  float cut = greedy ? m : -FLT_MAX;
  if (least > 0.f) {
    const double far = -log((double)least) * (double)temp;
    cut = fmaxf(__double2float_ru((double)m - far), -FLT_MAX);
  }
  u64 mass = 0;
  uint32_t count = 0, ties = 0x7FFFFFFFu;
  const uint32_t top = Grid<T>::up(m) + 1;
  uint32_t lo = Grid<T>::up(cut), hi = top;
  if (greedy) {
    ties = 1;
  } else {
    if (k > 0 && k < a.vocab) {
      u64 none = 0;
      count = 0;
      each_logit([&](float l) { count += l >= cut; });
      team.add(none, count);
      if (count > (uint32_t)k) {
        uint32_t above = 0;                        // logits at hi and above
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
    cut = Grid<T>::value(lo);
    // the mass of what is kept so far
    count = 0;
    each_logit([&](float l) {
      if (l > cut) mass += weight(l, sh.powers);
      count += l == cut;
    });
    team.add(mass, count);
    ties = min(ties, count);
    const u64 each = weight(cut, sh.powers);
    if (p < 1.f) {
      const u64 want = scaled(p, mass + ties * each, true);  // the mass before a kept token is below this
      if (mass < want) {                           // tokens at the cut are among them
        ties = (uint32_t)((want - mass + each - 1) / each);
      } else {
        u64 above = 0;                             // mass at hi and above
        hi = top;
        while (hi - lo > 1) {
          const uint32_t mid = lo + (hi - lo) / 2;
          const float v = Grid<T>::value(mid), w = hi == top ? INFINITY : Grid<T>::value(hi);
          u64 some = 0;
          count = 0;
          each_logit([&](float l) {
            if (l >= v && l < w) some += weight(l, sh.powers);
          });
          team.add(some, count);
          some += above;
          if (some >= want) lo = mid;
          else hi = mid, above = some;
        }
        cut = Grid<T>::value(lo);
        const u64 one = weight(cut, sh.powers);
        ties = (uint32_t)((want - above + one - 1) / one);
      }
    }
  }
  // what each warp keeps, in the order of the tokens
  const u64 each = weight(cut, sh.powers);
  u64 sum = 0;
  count = 0;
  each_logit([&](float l) {
    if (l > cut) sum += weight(l, sh.powers);
    count += l == cut;
  });
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
    float v[kVec];
    load8(x + s * 32 * kVec, v);
    u64 mine = 0;
    uint32_t t = 0;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      if (v[j] > cut) mine += weight(v[j], sh.powers);
      t += v[j] == cut;
    }
    u64 run = mine;
    uint32_t tie_run = t;
    for (int o = 1; o < 32; o <<= 1) {
      const u64 r = __shfl_up_sync(0xFFFFFFFFu, run, o);
      const uint32_t n = __shfl_up_sync(0xFFFFFFFFu, tie_run, o);
      if (lane >= o) run += r, tie_run += n;
    }
    uint32_t seen = tied_before + (tie_run - t);
    u64 at = before + (run - mine) + tie_mass(tied_before, tie_run - t);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      u64 w = 0;
      if (v[j] > cut) w = weight(v[j], sh.powers);
      else if (v[j] == cut && seen++ < ties) w = each;
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
  int size = 1;
  while (size < kMaxCluster && size * kChunk < a.vocab) size *= 2;
  const int chunk = (a.vocab + size * kVec - 1) / (size * kVec) * kVec, step = kThreads * kVec;
  const int steps = (chunk + step - 1) / step;
  const size_t smem = (size_t)steps * step * sizeof(T);
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
