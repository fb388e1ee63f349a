// Acceptance of drafted tokens (dsa_tree_accept): one warp walks a sequence's tree from
// token 0 along the sampled tokens, twice: once to count, and again, when the counts of
// the sequences before it are known, to write the kept rows.
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

// Walks sequence rows [s0, s0 + T): f(row) for each kept one in order; returns their
// number and the last sampled token.
template <typename F>
__device__ __forceinline__ int walk(const Args& a, int s0, int T, const uint64_t* __restrict__ mask,
                                    const int32_t* __restrict__ drafted, const int32_t* __restrict__ sampled, int lane,
                                    int& last, F f) {
  int cur = 0, n = 0;
  last = -1;
  while (cur < T) {                                // cur rises with every turn
    f(s0 + cur, n++);
    last = sampled[s0 + cur];
    int next = T;
    if (last >= 0 && last != a.eos)
      for (int c = cur + 1; c < T && next == T; c += 32) {
        const int t = c + lane;
        const bool ok = t < T && drafted[s0 + t] == last &&
                        parent_of(mask + (long long)(s0 + t) * a.words, a.words, t) == cur;
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, ok);
        if (hit) next = c + __ffs(hit) - 1;
        if (a.words == 0) break;                   // a chain's only child is the next token
      }
    cur = next;
  }
  return n;
}

__global__ void __launch_bounds__(kThreads)
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
  const auto bounds = [&](int b, int& s0, int& T) {
    s0 = tok_start[b];
    const int s1 = tok_start[b + 1];
    T = s1 - s0;
    return s0 >= 0 && s0 <= s1 && s1 <= a.n_tok && (a.words == 0 || T <= 64ll * a.words);
  };
  uint32_t mine = 0;
  for (int b = first; b < behind; ++b) {
    int s0, T, last = -1, n = 0;
    if (bounds(b, s0, T)) n = walk(a, s0, T, mask, drafted, sampled, lane, last, [](int, int) {});
    else if (lane == 0) set_status(c, DSA_ERR_INDEX);
    if (lane == 0) n_new[b] = n, next[b] = last;
    mine += n;
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
    int s0, T, last, n = 0;
    if (bounds(b, s0, T))
      n = walk(a, s0, T, mask, drafted, sampled, lane, last, [&](int row, int i) {
        // (bounds that overlap name more tokens than there are)
        if (lane == 0 && place + i < (uint32_t)a.n_tok) row_index[place + i] = row, tokens[place + i] = sampled[row];
      });
    place += n;
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
  const int ctas = p->n_seqs <= kWarps ? 1 : kCluster;
  return launch_programmatic(accept_kernel, dim3(ctas), dim3(kThreads), 0, (cudaStream_t)stream, ctas, a, tok_start, mask,
                             drafted, sampled, n_new, row_index, tokens, next, c)
             ? DSA_OK
             : DSA_ERR_CUDA;
}
