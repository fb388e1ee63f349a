"""Refusals of rotary positions, sampling and acceptance: on the host, before any CUDA call."""
import ctypes
import math
from decimal import Decimal

import pytest
import torch

from oracle.rope import PI, frequencies
from test_abi import _lib

ref = ctypes.byref
A = [0x1000000 * (i + 1) for i in range(14)]               # made-up addresses, far apart


@pytest.fixture(scope="module")
def dsa():
    return _lib()


def test_structures_match_the_header(dsa):
    assert ctypes.sizeof(dsa.dsa_rope_part) == 32 and ctypes.sizeof(dsa.dsa_rope) == 16 + 4 * 32 + 128 * 8
    assert ctypes.sizeof(dsa.dsa_rope_rows) == 24 and ctypes.sizeof(dsa.dsa_sampler) == 8 + 4 * 8


def test_rope_steps_refuse(dsa):
    I, U = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED
    for rot, kw, code in ((0, {}, I), (3, {}, I), (-2, {}, I), (258, {}, U), (64, dict(base=1.0), I),
                          (64, dict(base=math.nan), I), (64, dict(base=math.inf), I),
                          (64, dict(scaling="linear", factor=0.5), I), (64, dict(scaling="ntk", factor=math.inf), I),
                          (64, dict(scaling="ntk", factor=1e300, base=1e300), I),
                          (64, dict(scaling="yarn", factor=4.0), I),
                          (64, dict(scaling="yarn", factor=4.0, original=4096, beta_slow=0.0), I),
                          (64, dict(scaling="yarn", factor=4.0, original=4096, beta_fast=0.5), I)):
        with pytest.raises(dsa.DSAError) as e:
            dsa.make_rope(rot_dim=rot, parts=[dsa.rope_part(heads=1, dim=64)], **kw)
        assert e.value.code == code
    assert dsa.lib.dsa_rope_steps(None, 1e4, 0, 1, 0, 32, 1) == I
    r = dsa.make_rope(rot_dim=64, parts=[dsa.rope_part(heads=1, dim=64)])
    assert dsa.lib.dsa_rope_steps(ref(r), 1e4, 4, 1, 0, 32, 1) == U
    for n in (0, 5):
        with pytest.raises(ValueError):
            dsa.make_rope(rot_dim=64, parts=[dsa.rope_part(heads=1, dim=64)] * n)


@pytest.mark.parametrize("base", [2.0, 12345.678, 10000.0, 500000.0, 1e6])
def test_rope_steps_are_good_to_what_the_header_states(dsa, base):
    """2^-20 radians at position 2^31.  Of a frequency f <= 1 in fp64: the power, the quotient by 2 pi and 2 pi itself are off
    by 2^-53 of it or less each, the exponent's rounding by 2^-53 / e at most; a scaling's steps fall on f / factor or
    on a mixture well below 1.  Together less than 2^-51."""
    for rot in (2, 26, 64, 128, 256):
        for kw in (dict(), dict(scaling="linear", factor=2.7), dict(scaling="ntk", factor=1.7),
                   dict(scaling="yarn", factor=40.0, original=4096), dict(scaling="yarn", factor=3.3, original=8192)):
            r = dsa.make_rope(rot_dim=rot, base=base, parts=[dsa.rope_part(heads=1, dim=256)], **kw)
            for i, f in enumerate(frequencies(rot, base=base, **kw)):
                angle = Decimal(int(r.step[i])) / Decimal(2) ** 64 * 2 * PI
                assert abs(angle - f) * 2 ** 31 <= Decimal(2) ** -20


def test_rope_apply_refuses(dsa):
    I, U = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED

    def call(n=5, pos=A[0], x=(A[1], 128, 32), out=(A[2], 128, 32), part=None, rot=16, **kw):
        r = dsa.make_rope(rot_dim=16, parts=[dsa.rope_part(**dict(dict(heads=4, dim=32, offset=8), **(part or {})))])
        r.rot_dim = rot
        for k, v in kw.items():
            setattr(r, k, v)
        rows = lambda a: None if a is None else ref(dsa.dsa_rope_rows(*a))
        return dsa.lib.dsa_rope_apply(ref(r), n, pos, rows(x), rows(out), 0, None)

    assert dsa.lib.dsa_rope_apply(None, 5, A[0], None, None, 0, None) == I
    for kw in (dict(n=0), dict(pos=None), dict(pos=A[0] + 2), dict(x=None), dict(out=None), dict(rot=15), dict(rot=0),
               dict(n_parts=0), dict(n_parts=5), dict(mscale=math.nan), dict(part=dict(heads=0)), dict(part=dict(dim=23)),
               dict(part=dict(offset=17)), dict(part=dict(offset=-1)), dict(x=(None, 128, 32)), dict(out=(None, 128, 32)),
               dict(x=(A[1] + 1, 128, 32)), dict(out=(A[2] + 1, 128, 32)), dict(x=(A[1], -128, 32)),
               dict(out=(A[2], 127, 32)), dict(out=(A[2], 128, 31)), dict(out=(A[2], 0, 32)), dict(out=(A[2], 32, 32)),
               # out meets x without being it
               dict(out=(A[1] + 2, 128, 32)), dict(out=(A[1] - 2, 128, 32)), dict(out=(A[1], 256, 32)),
               dict(out=(A[1] + 2 * (4 * 128 + 3 * 32 + 31), 128, 32))):
        assert call(**kw) == I, kw
    for kw in (dict(rot=258, part=dict(dim=512)), dict(part=dict(dim=(1 << 20) + 1), x=(A[1], 1 << 24, 1 << 22)),
               dict(n=1 << 30), dict(n=1 << 31, part=dict(heads=1)), dict(n=1, part=dict(heads=1 << 31))):
        assert call(**kw) == U, kw
    bad = dsa.make_rope(rot_dim=16, parts=[dsa.rope_part(heads=1, dim=16)])
    bad.part[0].dtype = 2
    assert dsa.lib.dsa_rope_apply(ref(bad), 1, A[0], ref(dsa.dsa_rope_rows(A[1], 16, 16)),
                                  ref(dsa.dsa_rope_rows(A[2], 16, 16)), 0, None) == U
    bad.part[0].dtype, bad.part[0].layout = 0, 2
    assert dsa.lib.dsa_rope_apply(ref(bad), 1, A[0], ref(dsa.dsa_rope_rows(A[1], 16, 16)),
                                  ref(dsa.dsa_rope_rows(A[2], 16, 16)), 0, None) == I


def test_sample_refuses(dsa):
    I, U = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED
    mk = lambda **kw: dsa.make_sampler(**dict(dict(rows=3, vocab=8, dtype="fp32"), **kw))
    # logits, u, temperature, top_k, top_p, min_p, index, token, prob
    call = lambda s, a=A: dsa.lib.dsa_sample(ref(s), *a[:9], None)
    at = lambda **kw: [kw.get(f"a{i}", a) for i, a in enumerate(A)]
    assert dsa.lib.dsa_sample(None, *A[:9], None) == I
    for s, code in ((mk(rows=0), I), (mk(vocab=0), I), (mk(ld=7), I), (mk(requests=0), I), (mk(vocab=(1 << 18) + 1), U),
                    (mk(rows=1 << 27), U), (mk(requests=1 << 31), U), (mk(ld=(1 << 40) + 1), U)):
        assert call(s) == code
    other = mk()
    other.dtype = 2
    assert call(other) == U
    for i in (0, 1, 7):
        assert call(mk(), at(**{f"a{i}": None})) == I
    assert call(mk(requests=2), at(a6=None)) == I           # settings of requests need an index
    for i in range(9):
        assert call(mk(), at(**{f"a{i}": A[i] + 2})) == I
    for i in range(7):
        assert call(mk(), at(a7=A[i])) == I and call(mk(), at(a8=A[i] + 8)) == I
    assert call(mk(), at(a8=A[7] - 8)) == I
    assert call(mk(ld=100), at(a7=A[0] + 4 * 207)) == I


def test_accept_refuses(dsa):
    I, U = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED
    cache = lambda n=2: dsa.make_cache(n_seqs=n, n_pages=1, page_rows=1, max_pages=1)
    tree = lambda n=6, w=1: dsa.make_tree(n_tok=n, H=1, d_qk=1, d_v=1, scale=1.0, mask_words=w)
    # tok_start, mask, drafted, sampled | n_new, row_index, tokens, next
    call = lambda c, t, a=A, eos=-1: dsa.lib.dsa_tree_accept(ref(c), ref(t), *a[:4], eos, *a[4:8], None)
    at = lambda i, v: [v if j == i else a for j, a in enumerate(A)]
    for c, t, code in ((cache(0), tree(), I), (cache(8193), tree(), U), (cache(), tree(0), I), (cache(), tree(w=-1), I),
                       (cache(), tree(w=0), I), (cache(), tree((1 << 30) + 1), U), (cache(), tree(w=(1 << 20) + 1), U)):
        assert call(c, t) == code
    assert call(cache(), tree(), eos=-2) == I and call(cache(), tree(), eos=1 << 31) == I
    for i in range(8):
        assert call(cache(), tree(), at(i, None)) == I and call(cache(), tree(), at(i, A[i] + 2)) == I
    for o in range(4, 8):
        for i in range(o):
            assert call(cache(), tree(), at(o, A[i] + 4)) == I
    assert call(cache(), tree(), at(4, A[1] + 44)) == I      # the mask's last word
    assert dsa.lib.dsa_tree_accept(None, ref(tree()), *A[:4], -1, *A[4:8], None) == I


def test_the_binding_refuses_tensors_off_the_gpu(dsa):
    i32 = torch.zeros(4, dtype=torch.int32)
    r = dsa.make_rope(rot_dim=8, parts=[dsa.rope_part(heads=1, dim=8)])
    with pytest.raises(ValueError):
        dsa.rope_apply(r, i32, (torch.zeros(4, 8, dtype=torch.bfloat16),))
    with pytest.raises(ValueError):
        dsa.sample(dsa.make_sampler(rows=4, vocab=8), torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4), None, None,
                   None, None, None, i32)
    c, t = dsa.make_cache(n_seqs=1, n_pages=1, page_rows=1, max_pages=1), dsa.make_tree(n_tok=4, H=1, d_qk=1, d_v=1, scale=1.0)
    with pytest.raises(ValueError):
        dsa.tree_accept(c, t, i32[:2], None, i32, i32, i32[:1], i32, i32, i32[:1])
