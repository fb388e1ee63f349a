// Arguments of the attention of drafted tokens over a paged cache, shared by
// its tensor-core and exact kernels.
#pragma once

#include "dsa_common.cuh"

namespace dsa {

struct TreeArgs {
  int n_seqs, n_pages, R, max_pages;     // cache
  int n_tok, H, d_qk, d_v, mask_words;
  float scale;
  const int32_t *table, *lens, *tok_start;
  const unsigned long long* mask;        // [n_tok][mask_words], nullptr: token t sees drafted tokens 0..t
};

struct TreeSeq {
  int len, t0, T;                        // cached rows, first drafted token, drafted tokens
};

// Sequence b; T = 0 (nothing to do, *bad set) when its numbers are out of range.
__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int b, bool* bad) {
  TreeSeq s;
  s.len = a.lens[b];
  s.t0 = a.tok_start[b];
  const int t1 = a.tok_start[b + 1];
  const bool wrong = s.len < 0 || s.len > (long long)a.max_pages * a.R || s.t0 < 0 || t1 < s.t0 || t1 > a.n_tok ||
                     (a.mask != nullptr && t1 - s.t0 > 64ll * a.mask_words);
  s.T = wrong ? 0 : t1 - s.t0;
  *bad |= wrong;
  return s;
}

}  // namespace dsa
