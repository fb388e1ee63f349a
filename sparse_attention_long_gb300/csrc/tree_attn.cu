// dsa_tree_attn_fwd: checks, dispatch, and the exact fp32 kernel.
#include <math.h>

#include "tree_attn.cuh"

namespace dsa {

bool ext_dev_ctx(DevCtx* c);
size_t tree_tc_workspace();
int launch_tree_attn_tc(const TreeArgs& a, const void* q, const void* pool, long long page_stride, const void* kv_new,
                        void* out, float* mx, float* sm, void* ws, DevCtx c, cudaStream_t st);

namespace tree_exact {

constexpr int kHeads = 4, kPerHead = 128;          // heads per CTA, threads of each
constexpr int kThreads = kHeads * kPerHead, kWarps = kThreads / 32;
constexpr int kMaxCols = 1024 / kThreads;
constexpr int kMaxCluster = 4;                      // CTAs that share a token's keys
constexpr int kMaxKeys = 128;                      // keys per tile at most
constexpr int kStageFloats = 12 * 1024;            // 48 KB of keys
__host__ __device__ inline int row_pitch(int d_qk) { return (d_qk + 3) / 4 * 4 + 4; }  // 16-byte rows, spread over the banks
inline int tile_keys(int d_qk) {                   // 8 at least: d_qk <= 1024
  int k = kMaxKeys;
  while (k * row_pitch(d_qk) > kStageFloats) k /= 2;
  return k;
}

// over the four warps of a head
__device__ __forceinline__ float head_reduce(float v, bool take_max, float (*red)[4]) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, v, o);
    v = take_max ? fmaxf(v, y) : v + y;
  }
  const int head = threadIdx.x / kPerHead, w = (threadIdx.x % kPerHead) / 32;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[head][w] = v;
  __syncthreads();
  return take_max ? fmaxf(fmaxf(red[head][0], red[head][1]), fmaxf(red[head][2], red[head][3]))
                  : (red[head][0] + red[head][1]) + (red[head][2] + red[head][3]);
}

__device__ __forceinline__ float4 ld_peer4(const float4* local, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(mapa_shared(smem_u32(local), rank))
               : "memory");
  return v;
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// One CTA per (token, four heads), or a cluster of them that takes the tiles in turn
// and joins in rank order through distributed shared memory.  Keys in tiles of `kt`
// rows (a power of two that fits the shared memory), staged row by row, a warp
// reading a row's consecutive values, all of its rows in flight.  128 threads per
// head: one or more per key for the logits; for the weighted sum a thread takes a
// value column of the four heads and every G-th key, and the G groups are added at
// the end.  A key that the token does not see is not read.  Small shapes: the time is
// the latency of a few tiles, and issuing their instructions (one head per CTA,
// staging the keys for itself, took 39 us for the case that takes 18 now: five
// sequences of up to 700 rows, seven tokens, eight heads of 80 / 64 columns).
template <bool VEC>
__global__ void __launch_bounds__(kThreads, 2)
    tree_exact_kernel(TreeArgs a, const float* __restrict__ qg, const uint8_t* __restrict__ pool, long long page_stride,
                      const float* __restrict__ kvn, float* __restrict__ out, float* __restrict__ mx,
                      float* __restrict__ sm_out, int kt, int nc, DevCtx c) {
  extern __shared__ __align__(16) float sh[];
  const int pitch = row_pitch(a.d_qk);
  float* qs = sh;                                  // [kHeads][pitch]
  float* ks = sh + kHeads * pitch;                 // [kt][pitch]
  __shared__ __align__(16) float p[kMaxKeys][kHeads];
  __shared__ float4 sums[kThreads];
  __shared__ float red[kHeads][4], alpha_s[kHeads];
  __shared__ __align__(16) float l_s[kHeads], m_s[kHeads];
  __shared__ const float* rows[kMaxKeys];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  let_next_launch();
  wait_for_earlier();
  const int hgroups = (a.H + kHeads - 1) / kHeads;
  const uint32_t rank = cluster_ctarank();
  const unsigned item = blockIdx.x / nc;
  const long long t = item / hgroups;
  const int h0 = (item % hgroups) * kHeads, nh = a.H - h0 < kHeads ? a.H - h0 : kHeads;
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
  const long long row = t * a.H + h0;              // of the first head
  for (int h = 0; h < nh; ++h)
    for (int d = tid; d < a.d_qk; d += kThreads) qs[h * pitch + d] = qg[(row + h) * a.d_qk + d];
  const int32_t* trow = a.table + (long long)lo * a.max_pages;
  const unsigned long long* mrow = a.mask ? a.mask + t * a.mask_words : nullptr;
  const long long keys = (long long)s.len + (a.mask ? s.T : tok + 1);
  // address of key k, nullptr if the token does not see it
  auto key_row = [&](long long k) -> const float* {
    if (k < s.len) {                               // a length fits 32 bits
      const int page = trow[(int)k / a.R];
      if (page >= 0 && page < a.n_pages)
        return reinterpret_cast<const float*>(pool + page * page_stride) + (long long)((int)k % a.R) * a.d_qk;
      set_status(c, DSA_ERR_INDEX);
    } else if (k < keys) {
      const int j = (int)(k - s.len);
      if (!mrow || ((mrow[j >> 6] >> (j & 63)) & 1ull)) return kvn + (long long)(s.t0 + j) * a.d_qk;
    }
    return nullptr;
  };
  const int head = tid / kPerHead, th = tid % kPerHead;
  const int share = kPerHead / kt, key = th / share, piece = th % share;  // this thread's key and part of its logit
  int width = kThreads;                            // value column of this thread, its group among `groups`
  while (width / 2 >= a.d_v) width /= 2;
  const int groups = kThreads / width, group = tid / width, col = tid % width;
  float m_run = -INFINITY, l_run = 0.f;            // of this thread's head
  float4 o[kMaxCols];
#pragma unroll
  for (int u = 0; u < kMaxCols; ++u) o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
  const long long step = (long long)nc * kt;
  const float* mine = tid < kt ? key_row((long long)rank * kt + tid) : nullptr;
  for (long long k0 = (long long)rank * kt; k0 < keys; k0 += step) {
    const int n = keys - k0 < kt ? (int)(keys - k0) : kt;
    __syncthreads();                               // the last tile is read
    if (tid < kt) rows[tid] = mine;
    __syncthreads();
    for (int r = warp; r < n; r += kWarps) {
      const float* src = rows[r];
      const uint32_t dst = smem_u32(ks + r * pitch);
      if (VEC) {
        for (int d = 4 * lane; d < a.d_qk; d += 128) {
          if (src) cp_async16_cg(dst + 4 * d, src + d);
          else *reinterpret_cast<float4*>(ks + r * pitch + d) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      } else {
        for (int d = lane; d < a.d_qk; d += 32) {
          if (src) cp_async4(dst + 4 * d, src + d);
          else ks[r * pitch + d] = 0.f;
        }
      }
    }
    if (tid < kt) mine = key_row(k0 + step + tid);   // of the next tile, while this one is worked on
    cp_async_wait_all();
    __syncthreads();
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    const bool seen = head < nh && key < n && rows[key] != nullptr;
    if (seen) {
      const float *kr = ks + key * pitch, *qr = qs + head * pitch;
      int d = 4 * piece;
#pragma unroll 4
      for (; d + 3 < a.d_qk; d += 4 * share) {
        const float4 x = *reinterpret_cast<const float4*>(kr + d), y = *reinterpret_cast<const float4*>(qr + d);
        acc[0] = fmaf(y.x, x.x, acc[0]);
        acc[1] = fmaf(y.y, x.y, acc[1]);
        acc[2] = fmaf(y.z, x.z, acc[2]);
        acc[3] = fmaf(y.w, x.w, acc[3]);
      }
      for (; d < a.d_qk && d < (a.d_qk & ~3) + 4; ++d) acc[0] = fmaf(qr[d], kr[d], acc[0]);  // the last one to three
    }
    float dot = (acc[0] + acc[1]) + (acc[2] + acc[3]);
    for (int w = 1; w < share; w <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, w);
    const float x = seen ? dot * a.scale : -INFINITY;
    const float m_new = fmaxf(m_run, head_reduce(x, true, red));
    const float mu = m_new == -INFINITY ? 0.f : m_new;
    const float e = seen ? expf(x - mu) : 0.f;
    const float alpha = m_run == -INFINITY ? 0.f : expf(m_run - m_new);
    if (piece == 0) p[key][head] = e;
    if (th == 0) alpha_s[head] = alpha;
    l_run = l_run * alpha + head_reduce(piece == 0 ? e : 0.f, false, red);  // (its barriers also publish p)
    m_run = m_new;
    const float4 al = make_float4(alpha_s[0], alpha_s[1], alpha_s[2], alpha_s[3]);
#pragma unroll
    for (int u = 0; u < kMaxCols; ++u) {
      const int d = col + u * kThreads;
      if (d >= a.d_v) break;
      float4 sum = make_float4(o[u].x * al.x, o[u].y * al.y, o[u].z * al.z, o[u].w * al.w);
#pragma unroll 8
      for (int i = group; i < n; i += groups) {
        const float v = ks[i * pitch + d];
        const float4 w = *reinterpret_cast<const float4*>(p[i]);
        sum.x = fmaf(w.x, v, sum.x);
        sum.y = fmaf(w.y, v, sum.y);
        sum.z = fmaf(w.z, v, sum.z);
        sum.w = fmaf(w.w, v, sum.w);
      }
      o[u] = sum;
    }
  }
  if (th == 0) l_s[head] = l_run;
  if (groups > 1) sums[tid] = o[0];
  __syncthreads();
  if (groups > 1 && group == 0) {                  // the groups in order
    for (int i = 1; i < groups; ++i) {
      const float4 v = sums[i * width + col];
      o[0].x += v.x;
      o[0].y += v.y;
      o[0].z += v.z;
      o[0].w += v.w;
    }
  }
  if (nc > 1) {
    // every CTA's sums (columns of the four heads), maxima and denominators
    float4* part = reinterpret_cast<float4*>(ks);  // [d_v]
    if (group == 0)
      for (int u = 0; u < kMaxCols && col + u * kThreads < a.d_v; ++u) part[col + u * kThreads] = o[u];
    if (th == 0) m_s[head] = m_run;
    cluster_sync_all();
    if (rank == 0) {
      float M[kHeads], l[kHeads], w[kMaxCluster][kHeads];
#pragma unroll
      for (int h = 0; h < kHeads; ++h) M[h] = -INFINITY, l[h] = 0.f;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        if (r >= nc) break;
        const float4 m = ld_peer4(reinterpret_cast<const float4*>(m_s), r);
        w[r][0] = m.x, w[r][1] = m.y, w[r][2] = m.z, w[r][3] = m.w;
#pragma unroll
        for (int h = 0; h < kHeads; ++h) M[h] = fmaxf(M[h], w[r][h]);
      }
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        if (r >= nc) break;
        const float4 p4 = ld_peer4(reinterpret_cast<const float4*>(l_s), r);
        const float lr[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
          w[r][h] = expf(w[r][h] - (M[h] == -INFINITY ? 0.f : M[h]));  // no key: exp(-inf) = 0
          l[h] = fmaf(w[r][h], lr[h], l[h]);
        }
      }
      if (group == 0) {
#pragma unroll
        for (int u = 0; u < kMaxCols; ++u) {
          const int d = col + u * kThreads;
          if (d >= a.d_v) break;
          float v[kHeads] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int r = 0; r < kMaxCluster; ++r) {
            if (r >= nc) break;
            const float4 p4 = ld_peer4(part + d, r);
            v[0] = fmaf(w[r][0], p4.x, v[0]);
            v[1] = fmaf(w[r][1], p4.y, v[1]);
            v[2] = fmaf(w[r][2], p4.z, v[2]);
            v[3] = fmaf(w[r][3], p4.w, v[3]);
          }
#pragma unroll
          for (int h = 0; h < kHeads; ++h)
            if (h < nh) out[(row + h) * a.d_v + d] = l[h] == 0.f ? 0.f : v[h] / l[h];
        }
      }
      if (tid < nh) {
        mx[row + tid] = tid == 0 ? M[0] : tid == 1 ? M[1] : tid == 2 ? M[2] : M[3];
        sm_out[row + tid] = tid == 0 ? l[0] : tid == 1 ? l[1] : tid == 2 ? l[2] : l[3];
      }
    }
    cluster_sync_all();                            // rank 0 has read the others' memory
    return;
  }
  if (group == 0) {
#pragma unroll
    for (int u = 0; u < kMaxCols; ++u) {
      const int d = col + u * kThreads;
      if (d >= a.d_v) break;
      const float v[4] = {o[u].x, o[u].y, o[u].z, o[u].w};
#pragma unroll
      for (int h = 0; h < kHeads; ++h)
        if (h < nh) out[(row + h) * a.d_v + d] = l_s[h] == 0.f ? 0.f : v[h] / l_s[h];
    }
  }
  if (th == 0 && head < nh) {
    mx[row + head] = m_run;
    sm_out[row + head] = l_run;
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
  const uintptr_t words = (uintptr_t)table | (uintptr_t)lens | (uintptr_t)tok_start | (uintptr_t)softmax_max |
                          (uintptr_t)softmax_sum;
  if ((bits & (bf16 ? 15u : 3u)) != 0 || (words & 3u) != 0 || ((uintptr_t)mask & 7u) != 0) return DSA_ERR_INVALID_ARG;
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
  const int kt = tile_keys((int)t->d_qk);
  const size_t smem = (size_t)(kt + kHeads) * row_pitch((int)t->d_qk) * sizeof(float);
  const long long items = t->n_tok * ((t->H + kHeads - 1) / kHeads);
  // CTAs per item: as many as are resident at once, two per SM, if the cache can hold
  // more than a tile.  One CTA against several, d_qk 80: 2 items x 4000 rows 133 us
  // against 38 (4 CTAs), 72 x 700 rows 31 against 19 (4), 128 x 700 rows 37 against
  // 24 (2); one tile each 72 items 8.8 against 12 (4); with more CTAs than are
  // resident 160 x 700 rows 38 against 45 (4).
  int dev = 0, sms = 0;
  if (!cuda_ok(cudaGetDevice(&dev)) || !cuda_ok(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)))
    return DSA_ERR_CUDA;
  int nc = p->max_pages * p->page_rows > kt ? kMaxCluster : 1;
  while (nc > 1 && items * nc > 2ll * sms) nc /= 2;
  const unsigned grid = (unsigned)(items * nc);
  if (!cuda_ok(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)))
    return DSA_ERR_CUDA;
  return launch_programmatic(kernel, dim3(grid), dim3(kThreads), smem, st, nc, a,
                             (const float*)q, (const uint8_t*)pool->base, (long long)pool->page_stride,
                             (const float*)kv_new, (float*)out, softmax_max, softmax_sum, kt, nc, c)
             ? DSA_OK
             : DSA_ERR_CUDA;
}

}  // extern "C"
