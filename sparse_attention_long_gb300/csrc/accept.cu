// Acceptance of drafted tokens (dsa_tree_accept): one warp walks a sequence's tree from
// token 0 along the sampled tokens; when the counts of the sequences before it are known,
// it writes the kept rows.  Up to 64 tokens are read at once, two per lane, and walked by
// votes (a load per step took 11.8 us where this takes 5.1).
//
// Bound: latency.  One chain of 5 tokens 3.1 us, 256 trees of 17 to 64 tokens 5.1 us: launch, two
// dependent loads, the walk, and with more than 32 sequences the cluster's barrier.
#include <algorithm>

#include "dsa_common.cuh"

namespace dsa {

bool ext_dev_ctx(DevCtx* c);

namespace accept {

constexpr int kWarps = 32, kThreads = kWarps * 32;
constexpr int kCluster = 8;

struct Args {
  int n_seqs, n_tok, words, eos;
};

__device__ __forceinline__ void store_remote(uint32_t* local, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(local), rank)), "r"(v) : "memory");
}

// the last token before t that t sees, -1: none
__device__ __forceinline__ int parent_of(const uint64_t* __restrict__ mask, int words, int t) {
  if (words == 0) return t - 1;
  for (int w = t >> 6; w >= 0; --w) {
    uint64_t m = mask[w];
    if (w == t >> 6) m &= (1ull << (t & 63)) - 1;
    if (m) return 64 * w + 63 - __clzll((long long)m);
  }
  return -1;
}

// What a sequence keeps: up to 64 tokens as bits, more walked again when they are written.
struct Kept {
  int s0, T, n, last;                              // first token, tokens, kept ones, the last one's sampled token
  uint32_t low, high;                              // of up to 64 tokens: which
  int32_t sampled[2];                              // of tokens `lane` and 32 + lane
};

// Up to 64 tokens: two per lane, read at once; the walk is votes and shuffles.
__device__ __forceinline__ void walk_short(const Args& a, Kept& k, const uint64_t* __restrict__ mask,
                                           const int32_t* __restrict__ drafted, const int32_t* __restrict__ sampled,
                                           int lane) {
  int token[2], parent[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = 32 * i + lane, row = k.s0 + t;
    const bool there = t < k.T;
    token[i] = there ? drafted[row] : 0;
    k.sampled[i] = there ? sampled[row] : -1;
    const uint64_t before = a.words == 0 ? (t ? 1ull << (t - 1) : 0) : there ? mask[(long long)row * a.words] & ((1ull << t) - 1) : 0;
    parent[i] = there && before ? 63 - __clzll((long long)before) : -1;
  }
  int cur = 0;
  k.n = 0, k.last = -1, k.low = k.high = 0;
  while (cur < k.T) {                              // cur rises with every turn
    if (cur < 32) k.low |= 1u << cur;
    else k.high |= 1u << (cur - 32);
    ++k.n;
    const int s0 = __shfl_sync(0xFFFFFFFFu, k.sampled[0], cur & 31), s1 = __shfl_sync(0xFFFFFFFFu, k.sampled[1], cur & 31);
    k.last = cur < 32 ? s0 : s1;
    if (k.last < 0 || k.last == a.eos) break;
    const uint32_t h0 = __ballot_sync(0xFFFFFFFFu, parent[0] == cur && token[0] == k.last);
    const uint32_t h1 = __ballot_sync(0xFFFFFFFFu, parent[1] == cur && token[1] == k.last);
    cur = h0 ? __ffs(h0) - 1 : h1 ? 31 + __ffs(h1) : k.T;
  }
}

// Any number: f(row, i) for the i-th kept row.
template <typename F>
__device__ __forceinline__ void walk_long(const Args& a, Kept& k, const uint64_t* __restrict__ mask,
                                          const int32_t* __restrict__ drafted, const int32_t* __restrict__ sampled, int lane,
                                          F f) {
  int cur = 0;
  k.n = 0, k.last = -1;
  while (cur < k.T) {                              // cur rises with every turn
    f(k.s0 + cur, k.n++);
    k.last = sampled[k.s0 + cur];
    int next = k.T;
    if (k.last >= 0 && k.last != a.eos)
      for (int c = cur + 1; c < k.T && next == k.T; c += 32) {
        const int t = c + lane;
        const bool ok = t < k.T && drafted[k.s0 + t] == k.last &&
                        parent_of(mask + (long long)(k.s0 + t) * a.words, a.words, t) == cur;
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, ok);
        if (hit) next = c + __ffs(hit) - 1;
        if (a.words == 0) break;                   // a chain's only child is the next token
      }
    cur = next;
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    accept_kernel(Args a, const int32_t* __restrict__ tok_start, const uint64_t* __restrict__ mask,
                  const int32_t* __restrict__ drafted, const int32_t* __restrict__ sampled, int32_t* __restrict__ n_new,
                  int32_t* __restrict__ row_index, int32_t* __restrict__ tokens, int32_t* __restrict__ next, DevCtx c) {
  __shared__ uint32_t of_warp[kWarps], of_cta[kCluster];
  let_next_launch();
  if (gridDim.x > 1) cluster_arrive();             // no CTA writes to one that has not begun
  wait_for_earlier();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int nc = gridDim.x, rank = nc > 1 ? (int)cluster_ctarank() : 0;
  // consecutive sequences for each warp, so that their order is the warps'
  const int each = (a.n_seqs + nc * warps - 1) / (nc * warps);
  const int first = min((rank * warps + warp) * each, a.n_seqs), behind = min(first + each, a.n_seqs);
  // sequence b's kept tokens; false: its bounds are out of range
  const auto look_at = [&](int b, Kept& k) {
    const int s1 = tok_start[b + 1];
    k.s0 = tok_start[b], k.T = s1 - k.s0, k.n = 0, k.last = -1;
    if (k.s0 < 0 || k.s0 > s1 || s1 > a.n_tok || (a.words && k.T > 64ll * a.words)) {
      k.T = 0;
      return false;
    }
    if (k.T <= 64) walk_short(a, k, mask, drafted, sampled, lane);
    else walk_long(a, k, mask, drafted, sampled, lane, [](int, int) {});
    return true;
  };
  uint32_t mine = 0;
  Kept k{};
  for (int b = first; b < behind; ++b) {
    if (!look_at(b, k) && lane == 0) set_status(c, DSA_ERR_INDEX);
    if (lane == 0) n_new[b] = k.n, next[b] = k.last;
    mine += k.n;
  }
  if (lane == 0) of_warp[warp] = mine;
  __syncthreads();
  uint32_t sum = 0;
  for (int w = 0; w < warps; ++w) sum += of_warp[w];
  uint32_t place = 0, total = 0;
  if (nc > 1) {
    cluster_wait();
    if ((int)threadIdx.x < nc) store_remote(&of_cta[rank], threadIdx.x, sum);
    cluster_sync_all();
    for (int r = 0; r < nc; ++r) {
      if (r < rank) place += of_cta[r];
      total += of_cta[r];
    }
  } else {
    total = sum;
  }
  for (int w = 0; w < warp; ++w) place += of_warp[w];
  for (int b = first; b < behind; ++b) {
    if (each > 1) look_at(b, k);                   // (else it is still there)
    // (bounds that overlap name more tokens than there are)
    if (k.T <= 64) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t bits = i ? k.high : k.low;
        const uint32_t to = place + (i ? __popc(k.low) : 0) + __popc(bits & ((1u << lane) - 1));
        if (k.n && (bits >> lane & 1) && to < (uint32_t)a.n_tok)
          row_index[to] = k.s0 + 32 * i + lane, tokens[to] = k.sampled[i];
      }
    } else {
      walk_long(a, k, mask, drafted, sampled, lane, [&](int row, int i) {
        if (lane == 0 && place + i < (uint32_t)a.n_tok) row_index[place + i] = row, tokens[place + i] = sampled[row];
      });
    }
    place += k.n;
  }
  if (total > (uint32_t)a.n_tok && rank == 0 && threadIdx.x == 0) set_status(c, DSA_ERR_INDEX);
  for (long long i = (long long)total + rank * blockDim.x + threadIdx.x; i < a.n_tok; i += nc * (int)blockDim.x)
    row_index[i] = tokens[i] = -1;
}

static bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}

}  // namespace accept
}  // namespace dsa

using namespace dsa;
using namespace dsa::accept;

extern "C" int dsa_tree_accept(const dsa_cache* p, const dsa_tree* t, const int32_t* tok_start, const uint64_t* mask,
                               const int32_t* drafted, const int32_t* sampled, int64_t eos, int32_t* n_new,
                               int32_t* row_index, int32_t* tokens, int32_t* next, dsa_stream_t stream) {
  if (!p || !t || p->n_seqs < 1 || t->n_tok < 1 || t->mask_words < 0) return DSA_ERR_INVALID_ARG;
  if (p->n_seqs > 8192 || t->n_tok > (1ll << 30) || t->mask_words > (1 << 20)) return DSA_ERR_UNSUPPORTED;
  if ((mask != nullptr) != (t->mask_words > 0) || eos < -1 || eos >= (1ll << 31)) return DSA_ERR_INVALID_ARG;
  const int32_t* arrays[] = {tok_start, drafted, sampled, n_new, row_index, tokens, next};
  const size_t n = (size_t)t->n_tok * 4, b = (size_t)p->n_seqs * 4;
  const size_t sizes[] = {b + 4, n, n, b, n, n, b};
  for (const int32_t* a : arrays)
    if (!a || ((uintptr_t)a & 3u)) return DSA_ERR_INVALID_ARG;
  if ((uintptr_t)mask & 7u) return DSA_ERR_INVALID_ARG;
  for (int o = 3; o < 7; ++o) {
    for (int i = 0; i < o; ++i)
      if (overlap(arrays[o], sizes[o], arrays[i], sizes[i])) return DSA_ERR_INVALID_ARG;
    if (mask && overlap(arrays[o], sizes[o], mask, (size_t)t->n_tok * t->mask_words * 8)) return DSA_ERR_INVALID_ARG;
  }
  DevCtx c;
  if (!ext_dev_ctx(&c)) return DSA_ERR_CUDA;
  const Args a{(int)p->n_seqs, (int)t->n_tok, (int)t->mask_words, (int)eos};
  // a warp per sequence as long as eight CTAs have as many
  const int ctas = p->n_seqs <= kWarps ? 1 : kCluster;
  const int warps = ctas > 1 ? std::min(kWarps, (a.n_seqs + ctas - 1) / ctas) : std::max(4, a.n_seqs);
  return launch_programmatic(accept_kernel, dim3(ctas), dim3(32 * warps), 0, (cudaStream_t)stream, ctas, a, tok_start, mask,
                             drafted, sampled, n_new, row_index, tokens, next, c)
             ? DSA_OK
             : DSA_ERR_CUDA;
}
