"""Argument checks of the rotation, the append and the cached attention (no GPU): status codes of the
C ABI before any device work, and the binding's own refusals."""
import ctypes
import math

import pytest
import torch

import block_sparse_attention_build_b200 as sa
from block_sparse_attention_build_b200 import cached as cc

OK_PTR = 1 << 12  # never followed: every call below is refused, or has nothing to do, before device work
INV, UNS, MIS, SMALL = sa.SA_ERR_INVALID_ARG, sa.SA_ERR_UNSUPPORTED, sa.SA_ERR_MISALIGNED, sa.SA_ERR_BUFFER_TOO_SMALL


def view(ptr=OK_PTR, b=64 * 8 * 10, h=64 * 10, t=64):
    return cc._View(ptr, b, h, t)


def rotary_call(q=None, k=None, pos=OK_PTR, spec=None, shape=(2, 4, 2, 10, 64), backward=0, qo=None, ko=None, pa=20,
                pb=10):
    spec = spec if spec is not None else sa.Rotary([1.0] * 32)._struct
    r = lambda x: None if x is None else ctypes.byref(x)
    q, qo = q or view(), qo or view()
    return sa.lib.sparse_attn_rotary(r(q), r(k), pos, pa, pb, r(spec), r(sa._Shape(*shape)), backward, r(qo), r(ko),
                                     None)


def test_rotary_refusals():
    assert rotary_call(k=view()) == INV                       # k without k_out
    assert rotary_call(backward=2) == INV
    assert rotary_call(pos=None) == INV
    assert rotary_call(pos=OK_PTR + 2) == MIS
    assert rotary_call(pa=-1) == INV
    assert rotary_call(shape=(2, 4, 2, 10, 96)) == UNS
    assert rotary_call(shape=(-1, 4, 2, 10, 64)) == INV
    assert rotary_call(q=view(ptr=None)) == INV
    assert rotary_call(q=view(ptr=OK_PTR + 8)) == MIS
    assert rotary_call(q=view(t=68)) == MIS
    assert rotary_call(q=view(h=-64)) == INV
    assert rotary_call(qo=view(h=0)) == INV                   # a written tensor repeats nothing
    assert rotary_call(shape=(0, 4, 2, 10, 64), pos=None) == sa.SA_OK
    assert rotary_call(shape=(2, 4, 2, 0, 64)) == sa.SA_OK
    assert rotary_call(shape=(2, 0, 2, 10, 64)) == sa.SA_OK   # no q heads, no k


@pytest.mark.parametrize("freq,axis,axes,inter,status", [
    ([1.0] * 33, None, 1, 0, INV), ([math.inf], None, 1, 0, INV), ([math.nan], None, 1, 0, INV),
    ([1.0], [1], 1, 0, INV), ([1.0], [-1], 1, 0, INV), ([1.0], None, 0, 0, INV), ([1.0], None, 5, 0, INV),
    ([1.0], None, 1, 2, INV)])
def test_rotary_spec_refusals(freq, axis, axes, inter, status):
    f = (ctypes.c_double * len(freq))(*freq)
    a = (ctypes.c_int32 * len(axis))(*axis) if axis else None
    s = cc._Rotary(len(freq), axes, inter, ctypes.addressof(f), ctypes.addressof(a) if a else None)
    assert rotary_call(spec=s) == status
    s = cc._Rotary(-1, 1, 0, None, None)
    assert rotary_call(spec=s) == INV
    s = cc._Rotary(1, 1, 0, None, None)
    assert rotary_call(spec=s) == INV


def cache_of(k=OK_PTR, v=OK_PTR, n=4, page=16, Hkv=2, D=64, strides=None):
    ps, hs, ts = strides or (Hkv * page * D, page * D, D)
    return cc._KVCache(k, v, n, page, Hkv, D, ps, hs, ts)


def batch_of(B=2, T=3, max_q=1, max_pages=4, stride=4, q=OK_PTR, kv=OK_PTR, table=OK_PTR):
    return cc._CacheBatch(B, T, max_q, max_pages, stride, q, kv, table)


BAD_CACHES = [(dict(page=8), UNS), (dict(page=48), UNS), (dict(page=512), UNS), (dict(page=0), UNS),
              (dict(D=80), UNS), (dict(D=0), INV), (dict(n=-1), INV), (dict(k=None), INV), (dict(v=None), INV),
              (dict(k=OK_PTR + 2), MIS), (dict(strides=(2048, 1024, 60)), MIS), (dict(strides=(2048, 0, 64)), INV),
              (dict(strides=(-2048, 1024, 64)), INV)]
BAD_BATCHES = [(dict(B=-1), INV), (dict(T=-1), INV), (dict(max_q=-1), INV), (dict(q=None), INV), (dict(kv=None), INV),
               (dict(table=None), INV), (dict(stride=3), INV), (dict(max_pages=1 << 27, stride=1 << 27), UNS)]


def append_call(cache=None, batch=None, k=None, v=None, spec=None, pos=None, off=0, q=None, qo=None, Hq=4, pa=3):
    r = lambda x: None if x is None else ctypes.byref(x)
    return sa.lib.sparse_attn_cache_append(r(k or view()), r(v or view()), r(cache or cache_of()),
                                           r(batch or batch_of()), r(spec), pos, pa, off, r(q), r(qo), Hq, None)


def test_append_refusals():
    spec = sa.Rotary([1.0] * 32)._struct
    for kw, status in BAD_CACHES:
        assert append_call(cache=cache_of(**kw)) == status, kw
    for kw, status in BAD_BATCHES:
        assert append_call(batch=batch_of(**kw)) == status, kw
    assert append_call(q=view(), qo=view()) == INV            # q without a rotation
    assert append_call(q=view(), spec=spec) == INV            # q without q_out
    assert append_call(pos=OK_PTR) == INV                     # positions without a rotation
    assert append_call(spec=spec, pos=OK_PTR + 1) == MIS
    assert append_call(spec=spec, off=-1) == INV
    assert append_call(spec=spec, pa=-1) == INV
    assert append_call(spec=sa.Rotary([1.0] * 33)._struct) == INV
    assert append_call(k=view(ptr=OK_PTR + 2)) == MIS
    assert append_call(v=view(t=3)) == MIS
    assert append_call(q=view(), qo=view(t=0), spec=spec) == INV
    assert append_call(batch=batch_of(B=0)) == sa.SA_OK
    assert append_call(batch=batch_of(T=0)) == sa.SA_OK


def attend_call(shared, cache=None, batch=None, pattern=None, Hq=4, scale=0.125, q=None, o=None, lse=OK_PTR,
                ws=OK_PTR, nbytes=1 << 40, prefix=0, ptable=None):
    r = ctypes.byref
    head = (r(q or view()), r(cache or cache_of()), r(batch or batch_of()))
    tail = (r((pattern or sa.Pattern(window=5))._c()), Hq, scale, r(o or view()), lse, ws, nbytes, None)
    if shared:
        return sa.lib.sparse_attn_fwd_shared(*head, ptable, prefix, *tail)
    return sa.lib.sparse_attn_fwd_cached(*head, *tail)


@pytest.mark.parametrize("shared", [False, True])
def test_attention_refusals(shared):
    call = lambda **kw: attend_call(shared, **kw)
    for kw, status in BAD_CACHES:
        assert call(cache=cache_of(**kw)) == status, kw
    for kw, status in BAD_BATCHES:
        assert call(batch=batch_of(**kw)) == status, kw
    for p in (sa.Pattern(window=5, causal=0), sa.Pattern(window=5, stride=3), sa.Pattern(area=16)):
        assert call(pattern=p) == UNS, p
    assert call(pattern=sa.Pattern(window=-2)) == INV
    assert call(pattern=sa.Pattern(sinks=-1)) == INV
    for s in (0.0, -1.0, math.inf, math.nan):
        assert call(scale=s) == INV
    assert call(Hq=3) == UNS
    assert call(Hq=-1) == INV
    assert call(cache=cache_of(Hkv=0)) == UNS
    assert call(batch=batch_of(T=2 ** 29)) == UNS             # rows are counted in 31 bits
    big = dict(B=1, T=2 ** 22, max_q=2 ** 22, max_pages=2 ** 25, stride=2 ** 25)
    assert call(batch=batch_of(**big)) == UNS                 # and so are units of rows and keys
    assert call(q=view(ptr=None)) == INV
    assert call(o=view(ptr=OK_PTR + 4)) == MIS
    assert call(o=view(t=0)) == INV
    assert call(lse=None) == INV
    assert call(lse=OK_PTR + 1) == MIS
    assert call(ws=None) == INV
    assert call(ws=OK_PTR + 16) == MIS
    assert call(nbytes=0) == SMALL
    assert call(batch=batch_of(B=0)) == sa.SA_OK
    assert call(batch=batch_of(T=0)) == sa.SA_OK
    assert call(Hq=0) == sa.SA_OK
    if shared:
        assert call(prefix=-1) == INV
        assert call(prefix=5) == INV                          # no table
        assert call(prefix=2 ** 31 - 1, ptable=OK_PTR) == UNS


def test_workspace_bytes():
    for f in (sa.fwd_cached_workspace_bytes, sa.fwd_shared_workspace_bytes):
        assert f(1, 8, 2, 128) > 0
        assert f(0, 0, 0, 64) >= 0
        for bad in ((-1, 8, 2, 128), (1, 8, 2, 0)):
            with pytest.raises(sa.SparseAttnError):
                f(*bad)
        for bad in ((1, 8, 3, 128), (1, 8, 2, 96), (1, 8, 0, 64)):
            with pytest.raises(sa.SparseAttnError):
                f(*bad)


def test_binding_refuses_host_and_wrong_tensors():
    x = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="bf16 CUDA"):
        sa.KVCache(x, x)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError, match="int32 CUDA"):
        sa.CacheBatch(i, i[:1], i[:1, None])
    with pytest.raises(ValueError, match="one axis"):
        sa.Rotary([1.0, 2.0], axis=[0])
    with pytest.raises(TypeError, match="bf16 CUDA"):
        sa.rotary(x, x, torch.zeros(1, 1, 16, dtype=torch.int32), sa.Rotary([1.0]))


def test_packed_structures_match_the_header():
    """The structures packed for every call lay their fields out as the ctypes ones do."""
    b = cc._CacheBatch(2, 3, 4, 5, 6, 7, 8, 9)
    assert bytes(b) == cc._pack_batch(2, 3, 4, 5, 6, 7, 8, 9)
    assert bytes(cc._View(1, 2, 3, 4)) == cc._pack_view(1, 2, 3, 4)
    assert bytes(sa._Shape(1, 2, 3, 4, 5)) == cc._pack_shape(1, 2, 3, 4, 5)
    p = sa.Pattern(window=5, sinks=2, n_global=3)
    assert bytes(p._c()) == cc._pack_pattern(p.causal, p.window, p.sinks, p.stride, p.n_global, p.area, p.summary)
