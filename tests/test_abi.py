"""The C-ABI library builds, loads without a GPU, and exports every entry
point include/dsa.h declares (no compute calls here)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dsa.h")


def _lib():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_attention_long_gb300 as dsa
    return dsa


def declared_symbols():
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(dsa_[a-z0-9_]+)\s*\(", text)))


def test_header_declares_the_path():
    names = declared_symbols()
    for n in ["dsa_indexer_scores", "dsa_topk", "dsa_sparse_attn_fwd", "dsa_sparse_attn_bwd",
              "dsa_forward", "dsa_indexer_kl_loss_bwd", "dsa_get_status", "dsa_workspace_size"]:
        assert n in names


def test_library_exports_every_declared_symbol():
    dsa = _lib()
    raw = ctypes.CDLL(dsa.LIB_PATH)
    for n in declared_symbols():
        assert hasattr(raw, n), n
    assert dsa.version() == 100


def test_params_struct_layout_matches_header():
    dsa = _lib()
    # 4 int32, 9 int64, float + int32, int64, pointer, int64
    assert ctypes.sizeof(dsa.dsa_params) == 16 + 9 * 8 + 8 + 8 + 8 + 8


def test_host_validation_without_gpu():
    # argument errors are found on the host before any CUDA call
    dsa = _lib()
    p = dsa.make_params(B=1, S_q=8, S_k=8, H=2, d_qk=8, d_v=4, H_I=2, d_I=4, topk=4, scale=0.5,
                        dtype="fp32")
    assert dsa.workspace_size(p, dsa.DSA_CALL_FORWARD) == 8 * 8 * 4
    bad = dsa.make_params(B=1, S_q=8, S_k=8, H=2, d_qk=8, d_v=16, H_I=2, d_I=4, topk=4, scale=0.5,
                          dtype="fp32")
    assert dsa.lib.dsa_sparse_attn_fwd(ctypes.byref(bad), 16, 16, 16, 16, 16, 16, None, None) == \
        dsa.DSA_ERR_INVALID_ARG
    uly = dsa.make_params(B=1, S_q=8, S_k=8, H=2, d_qk=8, d_v=4, H_I=2, d_I=4, topk=4, scale=0.5,
                          dtype="fp32", cp_mode="ulysses")
    assert dsa.lib.dsa_topk(ctypes.byref(uly), 16, 0, 1, 16, None) == dsa.DSA_ERR_UNSUPPORTED
    tnd = dsa.make_params(B=2, S_q=8, S_k=8, H=2, d_qk=8, d_v=4, H_I=2, d_I=4, topk=4, scale=0.5,
                          dtype="fp32", layout="TND")
    assert dsa.lib.dsa_topk(ctypes.byref(tnd), 16, 0, 1, 16, None) == dsa.DSA_ERR_INVALID_ARG
    off = dsa.make_params(B=1, S_q=8, S_k=8, H=2, d_qk=8, d_v=4, H_I=2, d_I=4, topk=4, scale=0.5,
                          dtype="fp32", q_row_offset=1)
    assert dsa.lib.dsa_topk(ctypes.byref(off), 16, 0, 1, 16, None) == dsa.DSA_ERR_INVALID_ARG
    assert dsa.lib.dsa_topk(ctypes.byref(p), 16, 0, 9, 16, None) == dsa.DSA_ERR_INVALID_ARG
    assert dsa.lib.dsa_topk(None, 16, 0, 1, 16, None) == dsa.DSA_ERR_INVALID_ARG
    bf = dsa.make_params(B=1, S_q=8, S_k=8, H=64, d_qk=576, d_v=512, H_I=64, d_I=128, topk=4,
                         scale=0.5, dtype="bf16")
    assert dsa.lib.dsa_sparse_attn_fwd(ctypes.byref(bf), 16, 16, 16, 16, 16, 16, None, None) == \
        dsa.DSA_ERR_UNSUPPORTED
    # the FP8 indexer flag adds the E4M3 operands and scales to the forward's
    # workspace; the scratch-free forward runs the bf16 indexer only
    f8 = dsa.make_params(B=1, S_q=64, S_k=64, H=128, d_qk=576, d_v=512, H_I=64, d_I=128, topk=16,
                         scale=0.5, dtype="bf16", flags=2)
    plain = dsa.make_params(B=1, S_q=64, S_k=64, H=128, d_qk=576, d_v=512, H_I=64, d_I=128, topk=16,
                            scale=0.5, dtype="bf16")
    assert dsa.workspace_size(f8, dsa.DSA_CALL_FORWARD) >= \
        dsa.workspace_size(plain, dsa.DSA_CALL_FORWARD) + 64 * 64 * 128 + 64 * 128 + 64 * 64 * 4 + 64 * 4
    assert dsa.lib.dsa_forward_static_ws(ctypes.byref(f8), *([16] * 9), None) == dsa.DSA_ERR_UNSUPPORTED
    fp32 = dsa.make_params(B=1, S_q=8, S_k=8, H=2, d_qk=8, d_v=4, H_I=2, d_I=4, topk=4, scale=0.5,
                           dtype="fp32")
    assert dsa.lib.dsa_indexer_scores_fp8(ctypes.byref(fp32), 16, 16, 16, 16, 16, 0, 1, 16, None) == \
        dsa.DSA_ERR_UNSUPPORTED
    # the bf16 path stores O with TMA: q, kv and out must be 16-byte aligned
    ds = dsa.make_params(B=1, S_q=8, S_k=8, H=128, d_qk=576, d_v=512, H_I=64, d_I=128, topk=4,
                         scale=0.5, dtype="bf16")
    assert dsa.lib.dsa_sparse_attn_fwd(ctypes.byref(ds), 16, 16, 16, 24, 16, 16, None, None) == \
        dsa.DSA_ERR_INVALID_ARG
    assert dsa.lib.dsa_sparse_attn_fwd(ctypes.byref(ds), 16, 8, 16, 16, 16, 16, None, None) == \
        dsa.DSA_ERR_INVALID_ARG


def test_backward_workspace_sizes():
    # bf16 tensor-core backward: P and scale*dS as bf16 hi/lo pairs
    # [rows*128][k] plus D [rows*128] fp32; the KL pass: head-summed P
    # [rows][k] fp32
    dsa = _lib()
    rows, k = 24, 2048
    p = dsa.make_params(B=1, S_q=rows, S_k=16384, H=128, d_qk=576, d_v=512, H_I=64, d_I=128,
                        topk=k, scale=0.5, dtype="bf16")
    rh = rows * 128
    assert dsa.workspace_size(p, dsa.DSA_CALL_ATTN_BWD) == 4 * rh * k * 2 + rh * 4 + 256
    assert dsa.workspace_size(p, dsa.DSA_CALL_KL_BWD) == rows * k * 4 + 256
    # the fused backward: the attention backward's workspace, then the KL target
    assert dsa.workspace_size(p, dsa.DSA_CALL_BACKWARD) == \
        (4 * rh * k * 2 + rh * 4 + 256) + (rows * k * 4 + 256)
    # row passes (0 < wave_rows < S_q): the workspace holds one pass of
    # wave_rows rows whatever B and S_q are; wave_rows >= S_q is one pass
    for B, S_q, W in ((1, 24, 10), (3, 24, 10), (2, 100, 7)):
        pw = dsa.make_params(B=B, S_q=S_q, S_k=16384, H=128, d_qk=576, d_v=512, H_I=64, d_I=128,
                             topk=k, scale=0.5, dtype="bf16", wave_rows=W)
        wh = W * 128
        assert dsa.workspace_size(pw, dsa.DSA_CALL_ATTN_BWD) == 4 * wh * k * 2 + wh * 4 + 256
        assert dsa.workspace_size(pw, dsa.DSA_CALL_KL_BWD) == W * k * 4 + 256
        assert dsa.workspace_size(pw, dsa.DSA_CALL_BACKWARD) == \
            (4 * wh * k * 2 + wh * 4 + 256) + (W * k * 4 + 256)
    whole = dsa.make_params(B=1, S_q=rows, S_k=16384, H=128, d_qk=576, d_v=512, H_I=64, d_I=128,
                            topk=k, scale=0.5, dtype="bf16", wave_rows=rows)
    assert dsa.workspace_size(whole, dsa.DSA_CALL_ATTN_BWD) == dsa.workspace_size(p, dsa.DSA_CALL_ATTN_BWD)
    # a k that is not a multiple of 8 has no tensor-core backward
    odd = dsa.make_params(B=1, S_q=rows, S_k=16384, H=128, d_qk=576, d_v=512, H_I=64, d_I=128,
                          topk=2047, scale=0.5, dtype="bf16")
    assert dsa.workspace_size(odd, dsa.DSA_CALL_ATTN_BWD) == 0
    assert dsa.lib.dsa_sparse_attn_bwd(ctypes.byref(odd), 16, 16, 16, 16, 16, 16, 16, 16, 16, 16,
                                       None) == dsa.DSA_ERR_UNSUPPORTED
    # the tensor-core backward needs its workspace
    assert dsa.lib.dsa_sparse_attn_bwd(ctypes.byref(p), 16, 16, 16, 16, 16, 16, 16, 16, 16, None,
                                       None) == dsa.DSA_ERR_WORKSPACE


def test_fused_indexer_topk_workspace_and_rejections():
    # dsa_indexer_topk (and dsa_forward with DSA_FLAG_FUSED_TOPK) keep one
    # wave's candidate lists: keys and positions (4 bytes each per key) and a
    # count per row; bf16 DeepSeek indexer shapes with S_k < 65536 only
    dsa = _lib()
    mk = lambda **kw: dsa.make_params(**dict(dict(B=1, S_q=64, S_k=64, H=128, d_qk=576, d_v=512,
                                                  H_I=64, d_I=128, topk=16, scale=0.5, dtype="bf16",
                                                  wave_rows=64), **kw))
    p = mk()
    W, S = 64, 64
    need = 2 * W * S * 4 + W * 4
    assert dsa.workspace_size(p, dsa.DSA_CALL_INDEXER_TOPK) >= need
    assert dsa.workspace_size(mk(flags=dsa.DSA_FLAG_FUSED_TOPK), dsa.DSA_CALL_FORWARD) >= need
    # the plain forward's ring is unchanged by the new call
    assert dsa.workspace_size(p, dsa.DSA_CALL_FORWARD) == W * S * 4
    # unsupported: fp32, other indexer shapes, S_k >= 65536, with the FP8 flag
    for bad in (mk(dtype="fp32"), mk(H_I=32), mk(S_k=65536, S_q=64),
                mk(flags=dsa.DSA_FLAG_FUSED_TOPK | dsa.DSA_FLAG_FP8_INDEXER)):
        assert dsa.workspace_size(bad, dsa.DSA_CALL_INDEXER_TOPK) == 0
        assert dsa.lib.dsa_indexer_topk(ctypes.byref(bad), 16, 16, 16, 0, 1, 16, 16, None) == \
            dsa.DSA_ERR_UNSUPPORTED
    # argument checks happen on the host, before any launch
    assert dsa.lib.dsa_indexer_topk(ctypes.byref(p), 16, 16, 16, 0, 65, 16, 16, None) == \
        dsa.DSA_ERR_INVALID_ARG
    assert dsa.lib.dsa_indexer_topk(ctypes.byref(p), 16, 16, 16, 0, 1, 16, None, None) == \
        dsa.DSA_ERR_WORKSPACE
    assert dsa.lib.dsa_forward_static_ws(ctypes.byref(mk(flags=dsa.DSA_FLAG_FUSED_TOPK)),
                                         *([16] * 9), None) == dsa.DSA_ERR_UNSUPPORTED


def test_cache_host_validation_without_gpu():
    dsa = _lib()
    assert ctypes.sizeof(dsa.dsa_cache) == 4 * 8 and ctypes.sizeof(dsa.dsa_pool) == 5 * 8
    mk = lambda **kw: dsa.make_cache(**dict(dict(n_seqs=2, n_pages=8, page_rows=4, max_pages=3), **kw))
    ref = ctypes.byref
    # distinct made-up addresses, far enough apart not to overlap
    A = [0x10000 * (i + 1) for i in range(10)]
    for bad, code in ((mk(n_seqs=0), dsa.DSA_ERR_INVALID_ARG), (mk(page_rows=0), dsa.DSA_ERR_INVALID_ARG),
                      (mk(n_seqs=8193), dsa.DSA_ERR_UNSUPPORTED),
                      (mk(n_pages=1 << 26, page_rows=64), dsa.DSA_ERR_UNSUPPORTED),
                      (mk(max_pages=1 << 26, page_rows=64), dsa.DSA_ERR_UNSUPPORTED)):
        assert dsa.lib.dsa_cache_fork(ref(bad), *A[:9], None) == code
        assert dsa.lib.dsa_cache_extend(ref(bad), *A[:7], 5, None) == code
        assert dsa.lib.dsa_cache_compact(ref(bad), *A[:8], None) == code
    c = mk()
    assert dsa.lib.dsa_cache_fork(None, *A[:9], None) == dsa.DSA_ERR_INVALID_ARG
    for i in range(9):
        assert dsa.lib.dsa_cache_fork(ref(c), *[None if j == i else A[j] for j in range(9)], None) == \
            dsa.DSA_ERR_INVALID_ARG
    # outputs over inputs: the whole table, and one entry of it
    for shift in (0, 4, -4):
        assert dsa.lib.dsa_cache_fork(ref(c), A[0], A[1], A[2], A[3], A[1] + shift, A[5], A[6], A[7], A[8], None) == \
            dsa.DSA_ERR_INVALID_ARG
        assert dsa.lib.dsa_cache_compact(ref(c), A[0], A[1], A[2], A[3], A[2] + shift, A[5], A[6], A[7], None) == \
            dsa.DSA_ERR_INVALID_ARG
    assert dsa.lib.dsa_cache_extend(ref(c), A[0], A[1], A[2], A[3], A[2] + 4, A[5], A[6], 5, None) == \
        dsa.DSA_ERR_INVALID_ARG
    assert dsa.lib.dsa_cache_extend(ref(c), *A[:7], 0, None) == dsa.DSA_ERR_INVALID_ARG
    assert dsa.lib.dsa_cache_extend(ref(c), *A[:7], (1 << 20) + 1, None) == dsa.DSA_ERR_UNSUPPORTED
    pool = lambda *a: ref(dsa.dsa_pool(*a))
    copy = lambda pl, n=4: dsa.lib.dsa_cache_copy_pages(ref(c), pl, A[0], A[1], n, None)
    assert copy(pool(None, 1, 0, 64, 16)) == dsa.DSA_ERR_INVALID_ARG
    assert copy(pool(A[2], 0, 0, 64, 16)) == dsa.DSA_ERR_INVALID_ARG
    assert copy(pool(A[2], 1, 0, 63, 16)) == dsa.DSA_ERR_INVALID_ARG      # pages closer than their rows
    assert copy(pool(A[2], 2, 64, 64, 16)) == dsa.DSA_ERR_INVALID_ARG     # layers and pages on each other
    assert copy(pool(A[2], 2, 511, 64, 16)) == dsa.DSA_ERR_INVALID_ARG
    assert copy(pool(A[2], 2, 512, 64, 16), -1) == dsa.DSA_ERR_INVALID_ARG
    assert copy(pool(A[2], 2, 512, 64, 16), 0) == dsa.DSA_OK              # nothing to do, nothing launched
    assert copy(pool(A[2], 2, 64, 128, 16), 0) == dsa.DSA_OK
    assert dsa.lib.dsa_cache_write(ref(c), pool(A[2], 1, 0, 64, 16), A[3], 0, 0, A[4], None, 3, None) == \
        dsa.DSA_ERR_INVALID_ARG
    assert dsa.lib.dsa_cache_write(ref(c), pool(A[2], 1, 0, 64, 16), None, 3, 0, A[4], None, 3, None) == \
        dsa.DSA_ERR_INVALID_ARG
    # the binding refuses tensors that are not on a GPU
    import torch
    with pytest.raises(ValueError):
        dsa.cache_copy_pages(c, torch.zeros(8, 4, 16), torch.zeros(3, dtype=torch.int32),
                             torch.zeros(1, dtype=torch.int32))


def test_tree_attention_host_validation_without_gpu():
    dsa = _lib()
    assert ctypes.sizeof(dsa.dsa_tree) == 8 + 5 * 8
    A = [0x10000 * (i + 1) for i in range(12)]
    cache = lambda **kw: dsa.make_cache(**dict(dict(n_seqs=2, n_pages=8, page_rows=64, max_pages=3), **kw))
    tree = lambda **kw: dsa.make_tree(**dict(dict(n_tok=5, H=16, d_qk=576, d_v=512, scale=0.1), **kw))

    def call(c, t, pool=None, mask=None, q=A[0], ws=A[11]):
        pool = pool or dsa.dsa_pool(A[1], 1, 0, 64 * 1152, 1152)
        return dsa.lib.dsa_tree_attn_fwd(ctypes.byref(c), ctypes.byref(t), q, ctypes.byref(pool), A[2], A[3], A[4],
                                         A[5], mask, A[6], A[7], A[8], ws, None)

    I, U = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED
    for c, t, code in ((cache(n_seqs=0), tree(), I), (cache(page_rows=24), tree(), U), (cache(), tree(n_tok=0), I),
                       (cache(), tree(H=0), I), (cache(), tree(H=1025), U), (cache(), tree(d_qk=512), U),
                       (cache(), tree(d_v=576), U), (cache(), tree(d_v=600), I), (cache(), tree(scale=-1.0), I),
                       (cache(), tree(scale=float("nan")), I), (cache(), tree(n_tok=1 << 30), U),
                       (cache(), tree(mask_words=-1), I), (cache(), tree(dtype="fp32", d_qk=1025), U)):
        assert call(c, t) == code
        assert dsa.tree_workspace_size(c, t) == 0
    assert call(cache(), tree(mask_words=1)) == I and call(cache(), tree(), mask=A[9]) == I
    assert call(cache(), tree(), q=None) == I and call(cache(), tree(), q=A[0] + 8) == I
    for pool in (dsa.dsa_pool(None, 1, 0, 64 * 1152, 1152), dsa.dsa_pool(A[1], 2, 1 << 20, 64 * 1152, 1152),
                 dsa.dsa_pool(A[1], 1, 0, 64 * 1152, 1024), dsa.dsa_pool(A[1], 1, 0, 64 * 1152 - 16, 1152),
                 dsa.dsa_pool(A[1], 1, 0, 64 * 1152 + 8, 1152)):
        assert call(cache(), tree(), pool=pool) == I
    assert call(cache(), tree(), ws=None) == dsa.DSA_ERR_WORKSPACE
    assert dsa.tree_workspace_size(cache(), tree()) > 0
    assert dsa.tree_workspace_size(cache(page_rows=5), tree(dtype="fp32", d_qk=80, d_v=64)) == 0


def test_beam_host_validation_without_gpu():
    dsa = _lib()
    assert ctypes.sizeof(dsa.dsa_beam) == 8 + 6 * 8
    mk = lambda **kw: dsa.make_beam(**dict(dict(n_batch=1, beams_in=2, beams_out=2, vocab=8, dtype="fp32"), **kw))
    A = [0x10000 * (i + 1) for i in range(8)]
    call = lambda b, fin=None, logits=A[0], ws=A[7]: dsa.lib.dsa_beam_select(
        ctypes.byref(b), logits, A[1], fin, A[3], A[4], A[5], A[6], ws, None)
    I, U = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED
    for b, code in ((mk(n_batch=0), I), (mk(beams_in=0), I), (mk(beams_out=0), I), (mk(vocab=0), I), (mk(ld=7), I),
                    (mk(eos=8), I), (mk(eos=-2), I), (mk(beams_in=33), U), (mk(beams_out=33), U),
                    (mk(vocab=(1 << 24) + 1), U), (mk(n_batch=1 << 31), U)):
        assert call(b) == code and dsa.beam_workspace_size(b) == 0
    assert call(mk(), fin=A[2]) == I and call(mk(), logits=None) == I and call(mk(), logits=A[0] + 2) == I
    assert call(mk(), ws=None) == dsa.DSA_ERR_WORKSPACE and call(mk(), ws=A[7] + 8) == dsa.DSA_ERR_WORKSPACE


def test_decoding_calls_refuse_misaligned_and_overlapping_arrays():
    dsa = _lib()
    I, U = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED
    ref = ctypes.byref
    A = [0x10000 * (i + 1) for i in range(13)]
    off = lambda k, n, by=2: [a + by if i == k else a for i, a in enumerate(A[:n])]
    c = dsa.make_cache(n_seqs=2, n_pages=8, page_rows=64, max_pages=3)
    pool = dsa.dsa_pool(A[11], 1, 0, 64 * 1152, 1152)
    for k in range(9):
        assert dsa.lib.dsa_cache_fork(ref(c), *off(k, 9), None) == I
    for k in range(7):
        assert dsa.lib.dsa_cache_extend(ref(c), *off(k, 7), 5, None) == I
    for k in range(8):
        assert dsa.lib.dsa_cache_compact(ref(c), *off(k, 8), None) == I
    for k in range(2):
        assert dsa.lib.dsa_cache_copy_pages(ref(c), ref(pool), *off(k, 2), 4, None) == I
    assert dsa.lib.dsa_cache_write(ref(c), ref(pool), A[0], 4, 0, A[1] + 1, None, 4, None) == I
    assert dsa.lib.dsa_cache_write(ref(c), ref(pool), A[0], 4, 0, A[1], A[2] + 2, 4, None) == I
    wide = dsa.make_cache(n_seqs=8192, n_pages=8, page_rows=1, max_pages=1 << 18)
    assert dsa.lib.dsa_cache_fork(ref(wide), *A[:9], None) == U

    def tree(t, a, mask):                 # q, table, lens, kv_new, tok_start, out, max, sum
        return dsa.lib.dsa_tree_attn_fwd(ref(c), ref(t), a[0], ref(pool), a[1], a[2], a[3], a[4], mask, a[5], a[6],
                                         a[7], A[12], None)

    t = dsa.make_tree(n_tok=5, H=16, d_qk=576, d_v=512, scale=0.1, mask_words=1)
    for k in range(8):
        assert tree(t, off(k, 8), A[8]) == I
    assert tree(t, A, A[8] + 4) == I

    def beam(b, a, fin, fin_out):         # logits, scores, parent, token, scores_out
        return dsa.lib.dsa_beam_select(ref(b), a[0], a[1], fin, a[2], a[3], a[4], fin_out, A[12], None)

    b = dsa.make_beam(n_batch=2, beams_in=2, beams_out=3, vocab=8, dtype="fp32", eos=0)
    for k in range(5):
        assert beam(b, off(k, 5), A[8], A[9]) == I
    a = list(A)
    for shift in (0, 12, -20):            # scores: 16 bytes, scores_out: 24
        a[4] = A[1] + shift
        assert beam(b, a, A[8], A[9]) == I
    for shift in (0, 3, -5):
        assert beam(b, A, A[8], A[8] + shift) == I
    for n in (1 << 31, 1 << 60):
        assert beam(dsa.make_beam(n_batch=n, beams_in=32, beams_out=3, vocab=8), A, None, None) == U
