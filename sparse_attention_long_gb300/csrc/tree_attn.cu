// dsa_tree_attn_fwd: checks, dispatch, and the exact fp32 kernel.
#include <math.h>

#include "tree_attn.cuh"

namespace dsa {

bool ext_dev_ctx(DevCtx* c);
size_t tree_tc_workspace();
int launch_tree_attn_tc(const TreeArgs& a, const void* q, const void* pool, long long page_stride, const void* kv_new,
                        void* out, float* mx, float* sm, void* ws, DevCtx c, cudaStream_t st);

namespace tree_exact {

constexpr int kThreads = 128;
constexpr int kMaxCols = 1024 / kThreads;

__device__ __forceinline__ float block_reduce(float v, bool take_max, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, v, o);
    v = take_max ? fmaxf(v, y) : v + y;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return take_max ? fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])) : (red[0] + red[1]) + (red[2] + red[3]);
}

// One CTA per (token, head).  Keys in tiles of 128, one per thread for the
// logits (fp32 FMAs), then the tile's weighted sum with one thread per value
// column.  A key that the token does not see is not read.  Small shapes: its
// time is the latency of a few key tiles.
template <bool VEC>
__global__ void __launch_bounds__(kThreads)
    tree_exact_kernel(TreeArgs a, const float* __restrict__ qg, const uint8_t* __restrict__ pool, long long page_stride,
                      const float* __restrict__ kvn, float* __restrict__ out, float* __restrict__ mx,
                      float* __restrict__ sm_out, DevCtx c) {
  extern __shared__ float qs[];                    // [d_qk]
  __shared__ float p[kThreads], red[4];
  __shared__ const float* rows[kThreads];
  const int tid = threadIdx.x;
  const long long t = blockIdx.x / a.H;
  const int h = blockIdx.x % a.H;
  if (blockIdx.x == 0) {
    bool wrong = false;
    for (int b = tid; b < a.n_seqs; b += kThreads) tree_seq(a, b, &wrong);
    if (wrong) set_status(c, DSA_ERR_INDEX);
  }
  int lo = 0, hi = a.n_seqs;                       // the sequence of token t: last b with tok_start[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.tok_start[mid] <= t) lo = mid;
    else hi = mid;
  }
  bool wrong = false;
  const TreeSeq s = tree_seq(a, lo, &wrong);
  if (t < s.t0 || t >= (long long)s.t0 + s.T) return;
  const int tok = (int)(t - s.t0);
  const long long row = t * a.H + h;
  for (int d = tid; d < a.d_qk; d += kThreads) qs[d] = qg[row * a.d_qk + d];
  const int32_t* trow = a.table + (long long)lo * a.max_pages;
  const unsigned long long* mrow = a.mask ? a.mask + t * a.mask_words : nullptr;
  const long long keys = (long long)s.len + (a.mask ? s.T : tok + 1);
  float m_run = -INFINITY, l_run = 0.f;
  float o[kMaxCols];
#pragma unroll
  for (int u = 0; u < kMaxCols; ++u) o[u] = 0.f;
  for (long long k0 = 0; k0 < keys; k0 += kThreads) {
    const long long k = k0 + tid;
    const float* kr = nullptr;
    if (k < s.len) {
      const int page = trow[k / a.R];
      if (page >= 0 && page < a.n_pages)
        kr = reinterpret_cast<const float*>(pool + page * page_stride) + (k % a.R) * a.d_qk;
      else set_status(c, DSA_ERR_INDEX);
    } else if (k < keys) {
      const int j = (int)(k - s.len);
      if (!mrow || ((mrow[j >> 6] >> (j & 63)) & 1ull)) kr = kvn + (long long)(s.t0 + j) * a.d_qk;
    }
    __syncthreads();                               // qs written; the last tile's p and rows read
    float x = -INFINITY;
    if (kr) {
      float acc = 0.f;
      if (VEC) {
        for (int d = 0; d < a.d_qk; d += 4) {
          const float4 v = *reinterpret_cast<const float4*>(kr + d);
          acc = fmaf(qs[d], v.x, acc);
          acc = fmaf(qs[d + 1], v.y, acc);
          acc = fmaf(qs[d + 2], v.z, acc);
          acc = fmaf(qs[d + 3], v.w, acc);
        }
      } else {
        for (int d = 0; d < a.d_qk; ++d) acc = fmaf(qs[d], kr[d], acc);
      }
      x = acc * a.scale;
    }
    const float m_new = fmaxf(m_run, block_reduce(x, true, red));
    const float mu = m_new == -INFINITY ? 0.f : m_new;
    const float e = kr ? expf(x - mu) : 0.f;
    p[tid] = e;
    rows[tid] = kr;
    const float alpha = m_run == -INFINITY ? 0.f : expf(m_run - m_new);
    l_run = l_run * alpha + block_reduce(e, false, red);
    m_run = m_new;
    const int n = keys - k0 < kThreads ? (int)(keys - k0) : kThreads;
#pragma unroll
    for (int u = 0; u < kMaxCols; ++u) {
      const int d = tid + u * kThreads;
      if (d >= a.d_v) break;
      float acc = o[u] * alpha;
#pragma unroll 4
      for (int i = 0; i < n; ++i)
        if (rows[i]) acc = fmaf(p[i], rows[i][d], acc);
      o[u] = acc;
    }
  }
#pragma unroll
  for (int u = 0; u < kMaxCols; ++u) {
    const int d = tid + u * kThreads;
    if (d < a.d_v) out[row * a.d_v + d] = l_run == 0.f ? 0.f : o[u] / l_run;
  }
  if (tid == 0) {
    mx[row] = m_run;
    sm_out[row] = l_run;
  }
}

}  // namespace tree_exact

static int check_tree(const dsa_cache* p, const dsa_tree* t, TreeArgs* a) {
  if (!p || !t) return DSA_ERR_INVALID_ARG;
  if (t->dtype != DSA_BF16 && t->dtype != DSA_FP32) return DSA_ERR_UNSUPPORTED;
  if (p->n_seqs < 1 || p->n_pages < 1 || p->page_rows < 1 || p->max_pages < 1 || t->n_tok < 1 || t->H < 1 ||
      t->d_qk < 1 || t->d_v < 1 || t->d_v > t->d_qk || t->mask_words < 0)
    return DSA_ERR_INVALID_ARG;
  if (!(t->scale > 0.f) || !isfinite(t->scale)) return DSA_ERR_INVALID_ARG;
  if (p->n_seqs > (1ll << 20) || p->n_pages > (1ll << 30) || p->page_rows > (1ll << 30) || p->max_pages > (1ll << 30) ||
      p->n_pages * p->page_rows >= (1ll << 31) || p->max_pages * p->page_rows >= (1ll << 31) || t->H > 1024 ||
      t->n_tok > (1ll << 30) || t->n_tok * t->H >= (1ll << 31) || t->mask_words > (1 << 20))
    return DSA_ERR_UNSUPPORTED;
  if (t->dtype == DSA_BF16) {
    if (t->d_qk != 576 || t->d_v != 512 || p->page_rows % 16 != 0) return DSA_ERR_UNSUPPORTED;
  } else if (t->d_qk > 1024) {
    return DSA_ERR_UNSUPPORTED;
  }
  a->n_seqs = (int)p->n_seqs;
  a->n_pages = (int)p->n_pages;
  a->R = (int)p->page_rows;
  a->max_pages = (int)p->max_pages;
  a->n_tok = (int)t->n_tok;
  a->H = (int)t->H;
  a->d_qk = (int)t->d_qk;
  a->d_v = (int)t->d_v;
  a->mask_words = (int)t->mask_words;
  a->scale = t->scale;
  return DSA_OK;
}

}  // namespace dsa

using namespace dsa;

extern "C" {

size_t dsa_tree_workspace_size(const dsa_cache* p, const dsa_tree* t) {
  TreeArgs a;
  if (check_tree(p, t, &a) != DSA_OK) return 0;
  return t->dtype == DSA_BF16 ? tree_tc_workspace() : 0;
}

int dsa_tree_attn_fwd(const dsa_cache* p, const dsa_tree* t, const void* q, const dsa_pool* pool,
                      const int32_t* table, const int32_t* lens, const void* kv_new, const int32_t* tok_start,
                      const uint64_t* mask, void* out, float* softmax_max, float* softmax_sum, void* workspace,
                      dsa_stream_t stream) {
  TreeArgs a;
  int rc = check_tree(p, t, &a);
  if (rc) return rc;
  if (!q || !pool || !pool->base || !table || !lens || !kv_new || !tok_start || !out || !softmax_max || !softmax_sum)
    return DSA_ERR_INVALID_ARG;
  if ((mask != nullptr) != (t->mask_words > 0)) return DSA_ERR_INVALID_ARG;
  const bool bf16 = t->dtype == DSA_BF16;
  const long long row_bytes = t->d_qk * (bf16 ? 2 : 4);
  if (pool->n_layers != 1 || pool->row_bytes != row_bytes || pool->page_stride < p->page_rows * row_bytes)
    return DSA_ERR_INVALID_ARG;
  if (pool->page_stride >= (1ll << 38)) return DSA_ERR_UNSUPPORTED;
  const uintptr_t bits = (uintptr_t)q | (uintptr_t)pool->base | (uintptr_t)kv_new | (uintptr_t)out |
                         (uintptr_t)pool->page_stride;
  if ((bits & (bf16 ? 15u : 3u)) != 0) return DSA_ERR_INVALID_ARG;
  if (bf16 && (!workspace || ((uintptr_t)workspace & 15u) != 0)) return DSA_ERR_WORKSPACE;
  DevCtx c;
  if (!ext_dev_ctx(&c)) return DSA_ERR_CUDA;
  a.table = table;
  a.lens = lens;
  a.tok_start = tok_start;
  a.mask = reinterpret_cast<const unsigned long long*>(mask);
  cudaStream_t st = (cudaStream_t)stream;
  if (bf16)
    return launch_tree_attn_tc(a, q, pool->base, pool->page_stride, kv_new, out, softmax_max, softmax_sum, workspace, c,
                               st);
  using namespace tree_exact;
  const bool vec = (bits & 15u) == 0 && t->d_qk % 4 == 0;
  auto kernel = vec ? tree_exact_kernel<true> : tree_exact_kernel<false>;
  kernel<<<(unsigned)(t->n_tok * t->H), kThreads, t->d_qk * sizeof(float), st>>>(
      a, (const float*)q, (const uint8_t*)pool->base, pool->page_stride, (const float*)kv_new, (float*)out,
      softmax_max, softmax_sum, c);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // extern "C"
