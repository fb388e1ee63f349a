// Beam selection (dsa_beam_select): per request, the best beams_out of
//   cand(w, v) = score[w] + x[w, v] - log sum_u exp x[w, u]
// over its beams w and the vocabulary, ties to the lower w * vocab + v.
//
// Two kernels.  beam_part_kernel reads the logits once: one CTA per (beam row,
// chunk of the vocabulary), the chunk in registers.  Within a beam the order of
// the candidates is the order of the logits, so a chunk only has to give its
// best beams_out logits, its maximum m and its sum of exp(x - m).  The k-th
// largest of the threads' own maxima bounds the chunk's k-th largest logit from
// below (each of those k threads has a logit at least that large), so few
// logits pass it; those are ranked by counting.  Keys are (order-preserving
// bits of the logit, inverted index): unique, so ties need no care.
// beam_join_kernel (one CTA per request) adds the chunks' sums in 64 bits and
// ranks the candidates by their 64-bit scores.
//
// Candidates of different beams can lie close together, and their order is an
// output: the sums are fp32 only inside a thread and a chunk's total and
// everything after it is fp64.  A row gives the same bits wherever it lies:
// which element a thread takes depends on its index alone, not on alignment.
//
// Bound: reading the logits (HBM) for a batch; the two launches for one request.
#include <math.h>

#include "dsa_common.cuh"

namespace dsa {

bool ext_dev_ctx(DevCtx* c);

namespace beam {

constexpr int kThreads = 256;
constexpr int kVec = 8;                            // consecutive elements per thread and step
constexpr int kSteps = 4;
constexpr int kChunk = kThreads * kVec * kSteps;   // 8192 logits per CTA
constexpr int kMaxBeams = 32;                      // in and out
constexpr int kMaxCand = 32 * kMaxBeams;           // candidates of a chunk at most, see beam_part_kernel

struct Args {
  int n_batch, win, wout, vocab, chunks;
  long long ld;
  int eos;
};
// per (row, chunk): maximum and sum, then wout keys
struct Stat {
  double sum;
  float max, pad;
};

// larger logit first, then lower index; 0: no logit
__device__ __forceinline__ unsigned long long make_key(float x, uint32_t idx) {
  return ((unsigned long long)ordered_key(x) << 32) | (0xFFFFFFFFu - idx);
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return __uint_as_float((u & 0x80000000u) ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ uint32_t key_index(unsigned long long k) { return 0xFFFFFFFFu - (uint32_t)k; }

// logits that may not be chosen count as -inf: -inf itself, +inf and NaN
__device__ __forceinline__ float clean(float x) { return x < INFINITY ? x : -INFINITY; }

template <typename T>
__device__ __forceinline__ void load8(const T* p, bool vec, int n, float* x);
template <>
__device__ __forceinline__ void load8<float>(const float* p, bool vec, int n, float* x) {
  if (vec && n >= 8) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < n ? __ldcs(p + i) : -INFINITY;
  }
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, bool vec, int n, float* x) {
  if (vec && n >= 8) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = i < n ? __uint_as_float((uint32_t)__ldcs(reinterpret_cast<const unsigned short*>(p) + i) << 16) : -INFINITY;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    beam_part_kernel(Args a, const T* __restrict__ logits, const float* __restrict__ scores,
                     const uint8_t* __restrict__ finished, Stat* __restrict__ stats,
                     unsigned long long* __restrict__ keys, int vec) {
  __shared__ unsigned long long tmax[kThreads], cand[kMaxCand], kth;
  __shared__ float wmax[kThreads / 32];
  __shared__ double wsum[kThreads / 32];
  __shared__ int n_cand;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long row = blockIdx.x / a.chunks;
  const int chunk = blockIdx.x % a.chunks;
  // a finished beam has no logits, a beam of score -inf no candidates
  if ((finished && finished[row]) || !(scores[row] > -INFINITY)) return;
  const T* base = logits + row * a.ld;
  float x[kSteps][kVec];
  float m = -INFINITY;
  unsigned long long best = 0;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int i0 = chunk * kChunk + (s * kThreads + tid) * kVec;
    load8<T>(base + i0, vec != 0, a.vocab - i0, x[s]);
  }
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      x[s][e] = clean(x[s][e]);
      m = fmaxf(m, x[s][e]);
    }
  // the thread's best key: its first element equal to its maximum
  if (m > -INFINITY) {
#pragma unroll
    for (int s = kSteps - 1; s >= 0; --s)
#pragma unroll
      for (int e = kVec - 1; e >= 0; --e)
        if (x[s][e] == m) best = make_key(m, chunk * kChunk + (s * kThreads + tid) * kVec + e);
  }
  tmax[tid] = best;
  if (tid == 0) n_cand = 0;
  float wm = m;
#pragma unroll
  for (int o = 16; o; o >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
  if (lane == 0) wmax[warp] = wm;
  __syncthreads();
  float cm = wmax[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) cm = fmaxf(cm, wmax[w]);
  // rank of this thread's best key among all threads'
  const int k = a.wout;
  int rank = 0;
#pragma unroll 8
  for (int t = 0; t < kThreads; ++t) rank += tmax[t] > best;
  if (rank == k - 1 && best != 0) kth = best;
  if (tid == 0 && cm == -INFINITY) kth = 0;
  // sum of exp(x - max) over the chunk
  double sum = 0.0;
  if (cm > -INFINITY) {
    float part = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int e = 0; e < kVec; ++e) part += __expf(x[s][e] - cm);
    sum = part;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) wsum[warp] = sum;
  const int have = __syncthreads_count(best != 0);  // threads with a logit
  const unsigned long long least = have < k ? 1ull : kth;
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      const unsigned long long key = make_key(x[s][e], chunk * kChunk + (s * kThreads + tid) * kVec + e);
      if (x[s][e] > -INFINITY && key >= least) {
        const int at = atomicAdd(&n_cand, 1);
        if (at < kMaxCand) cand[at] = key;
      }
    }
  __syncthreads();
  const long long out = row * a.chunks + chunk;
  const int n = n_cand;                            // only k threads have a key >= kth: at most 32 k
  for (int i = tid; i < n; i += kThreads) {
    const unsigned long long mine = cand[i];
    int r = 0;
    for (int j = 0; j < n && r < k; ++j) r += cand[j] > mine;
    if (r < k) keys[out * k + r] = mine;
  }
  for (int i = n + tid; i < k; i += kThreads) keys[out * k + i] = 0;
  if (tid == 0) {
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) t += wsum[w];
    stats[out].sum = t;
    stats[out].max = cm;
  }
}

// order-preserving map of a double (no NaN)
__device__ __forceinline__ unsigned long long ordered64(double x) {
  const long long u = __double_as_longlong(x + 0.0);
  return (unsigned long long)u ^ ((unsigned long long)(u >> 63) | 0x8000000000000000ull);
}

// candidates of a request, sorted by repeated choice of the best: beams_out
// rounds over a list in shared memory (64-bit score, flattened index)
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads)
    beam_join_kernel(Args a, const float* __restrict__ scores, const uint8_t* __restrict__ finished,
                     const Stat* __restrict__ stats, const unsigned long long* __restrict__ keys,
                     int32_t* __restrict__ parent, int32_t* __restrict__ token, float* __restrict__ scores_out,
                     uint8_t* __restrict__ finished_out) {
  __shared__ double lse[kMaxBeams];
  __shared__ unsigned long long key_s[kMaxBeams * kMaxBeams];
  __shared__ uint32_t key_i[kMaxBeams * kMaxBeams];
  __shared__ int n_list;
  const int b = blockIdx.x, tid = threadIdx.x, k = a.wout;
  if (tid == 0) n_list = 0;
  for (int i = tid; i < k; i += kJoinThreads) {
    parent[(long long)b * k + i] = -1;
    token[(long long)b * k + i] = -1;
    scores_out[(long long)b * k + i] = -INFINITY;
    if (finished_out) finished_out[(long long)b * k + i] = 0;
  }
  // log-sum-exp of each beam, the chunks in order
  for (int w = tid; w < a.win; w += kJoinThreads) {
    const long long row = (long long)b * a.win + w;
    const bool done = finished && finished[row];
    if (done || !(scores[row] > -INFINITY)) continue;
    const Stat* s = stats + row * a.chunks;
    float m = -INFINITY;
    for (int c = 0; c < a.chunks; ++c) m = fmaxf(m, s[c].max);
    double t = 0.0;
    for (int c = 0; c < a.chunks; ++c)
      if (s[c].max > -INFINITY) t += s[c].sum * exp((double)s[c].max - (double)m);
    lse[w] = m > -INFINITY ? (double)m + log(t) : 0.0;
  }
  __syncthreads();
  // one warp per beam: the best k of its chunks' sorted lists
  for (int w = tid >> 5; w < a.win; w += kJoinThreads / 32) {
    const int lane = tid & 31;
    const long long row = (long long)b * a.win + w;
    const float sc = scores[row];
    if (finished && finished[row]) {
      if (lane == 0 && sc > -INFINITY) {
        const int at = atomicAdd(&n_list, 1);
        key_s[at] = ordered64((double)sc);
        key_i[at] = (uint32_t)w * (uint32_t)a.vocab + (uint32_t)a.eos;
      }
      continue;
    }
    if (!(sc > -INFINITY)) continue;
    const unsigned long long* kr = keys + row * a.chunks * k;
    const int n = a.chunks * k;
    unsigned long long last = ~0ull;
    for (int r = 0; r < k; ++r) {                  // the largest key below the last one taken
      unsigned long long best = 0;
      for (int i = lane; i < n; i += 32) {
        const unsigned long long v = kr[i];
        if (v < last && v > best) best = v;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const unsigned long long v = __shfl_xor_sync(0xffffffffu, best, o);
        best = v > best ? v : best;
      }
      if (best == 0) break;
      last = best;
      if (lane == 0) {
        const int at = atomicAdd(&n_list, 1);
        key_s[at] = ordered64((double)sc + ((double)key_value(best) - lse[w]));
        key_i[at] = (uint32_t)w * (uint32_t)a.vocab + key_index(best);
      }
    }
  }
  __syncthreads();
  const int n = n_list;
  for (int i = tid; i < n; i += kJoinThreads) {
    const unsigned long long s = key_s[i];
    const uint32_t id = key_i[i];
    int r = 0;
    for (int j = 0; j < n && r < k; ++j) r += key_s[j] > s || (key_s[j] == s && key_i[j] < id);
    if (r >= k) continue;
    const int w = (int)(id / (uint32_t)a.vocab), v = (int)(id % (uint32_t)a.vocab);
    const long long o = (long long)b * k + r, row = (long long)b * a.win + w;
    const unsigned long long u = (s & 0x8000000000000000ull) ? s ^ 0x8000000000000000ull : ~s;
    parent[o] = (int32_t)row;
    token[o] = v;
    scores_out[o] = (float)__longlong_as_double((long long)u);
    if (finished_out) finished_out[o] = (finished && finished[row]) || v == a.eos;
  }
}

static int check(const dsa_beam* p, Args* a) {
  if (!p) return DSA_ERR_INVALID_ARG;
  if (p->dtype != DSA_BF16 && p->dtype != DSA_FP32) return DSA_ERR_UNSUPPORTED;
  if (p->n_batch < 1 || p->beams_in < 1 || p->beams_out < 1 || p->vocab < 1 || p->ld < p->vocab || p->eos < -1 ||
      p->eos >= p->vocab)
    return DSA_ERR_INVALID_ARG;
  if (p->beams_in > kMaxBeams || p->beams_out > kMaxBeams || p->vocab > (1 << 24) || p->ld > (1ll << 40) ||
      p->n_batch * p->beams_in * ((p->vocab + kChunk - 1) / kChunk) >= (1ll << 31))
    return DSA_ERR_UNSUPPORTED;
  a->n_batch = (int)p->n_batch;
  a->win = (int)p->beams_in;
  a->wout = (int)p->beams_out;
  a->vocab = (int)p->vocab;
  a->chunks = (int)((p->vocab + kChunk - 1) / kChunk);
  a->ld = p->ld;
  a->eos = (int)p->eos;
  return DSA_OK;
}
static size_t stat_bytes(const Args& a) { return (size_t)a.n_batch * a.win * a.chunks * sizeof(Stat); }

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
  if (((uintptr_t)logits & (esz - 1)) != 0) return DSA_ERR_INVALID_ARG;
  if (!workspace || ((uintptr_t)workspace & 15u) != 0) return DSA_ERR_WORKSPACE;
  DevCtx c;
  if (!ext_dev_ctx(&c)) return DSA_ERR_CUDA;
  Stat* stats = (Stat*)workspace;
  unsigned long long* keys = (unsigned long long*)((uint8_t*)workspace + stat_bytes(a));
  cudaStream_t st = (cudaStream_t)stream;
  const int vec = (((uintptr_t)logits | (uintptr_t)(p->ld * esz)) & 15u) == 0;
  const unsigned grid = (unsigned)(a.n_batch * a.win) * (unsigned)a.chunks;
  if (p->dtype == DSA_BF16)
    beam_part_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a, (const __nv_bfloat16*)logits, scores, finished, stats,
                                                               keys, vec);
  else
    beam_part_kernel<float><<<grid, kThreads, 0, st>>>(a, (const float*)logits, scores, finished, stats, keys, vec);
  if (cudaGetLastError() != cudaSuccess) return DSA_ERR_CUDA;
  beam_join_kernel<<<a.n_batch, kJoinThreads, 0, st>>>(a, scores, finished, stats, keys, parent, token, scores_out,
                                                       finished_out);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // extern "C"
