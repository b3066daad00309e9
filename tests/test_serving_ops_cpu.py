"""Refusals of the serving operators: every check comes before any launch, so
they are tested on the host alone (the pointers are never followed)."""
import ctypes

import pytest

ARG, SHAPE, CAPACITY = -1, -2, -3
P = 1 << 20  # a 16-byte aligned address that nothing reads


def _lib():
    from looped_transformer_self_b200 import build
    build.build()
    from looped_transformer_self_b200 import binding as B
    return B.lib()


def _prompt(**kw):
    a = dict(dtype=1, q=P, sq=512, k=P, sk=256, v=P, sv=256, o=P, so=512, qo=P, ko=None, n_seqs=2, n_q=10,
             n_kv=10, H=4, Hk=2, hd=128, scale=0.1, scratch=P, bytes=1 << 40, status=None, stream=None)
    a.update(kw)
    return _lib().lt_attn_prompt(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), ARG), (dict(n_q=-1), ARG), (dict(n_seqs=-1), ARG), (dict(n_kv=-1), ARG),
    (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG), (dict(scale=float("inf")), ARG),
    (dict(scale=float("nan")), ARG), (dict(hd=48), SHAPE), (dict(hd=256), SHAPE), (dict(Hk=3), SHAPE),
    (dict(Hk=0), SHAPE), (dict(H=130, Hk=2, sq=130 * 128, so=130 * 128), SHAPE), (dict(q=None), ARG),
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(o=None), ARG), (dict(qo=None), ARG),
    (dict(scratch=None), ARG), (dict(scratch=P + 16), SHAPE), (dict(sq=511), ARG), (dict(sk=255), ARG), (dict(sv=255), ARG),
    (dict(so=504), ARG), (dict(sq=516), SHAPE), (dict(sk=260), SHAPE), (dict(q=P + 8), SHAPE),
    (dict(v=P + 2), SHAPE), (dict(o=P + 4), SHAPE), (dict(bytes=0), CAPACITY),
    (dict(n_q=2**31 - 1, H=64, Hk=1, sq=64 * 128, so=64 * 128), SHAPE),
    (dict(n_seqs=0), 0), (dict(n_q=0), 0),
])
def test_prompt_refusals(kw, code):
    assert _prompt(**kw) == code


def _prefix(**kw):
    a = dict(dtype=1, q=P, sq=512, cache=P, n_slots=100, o=P, so=512, ro=P, n_groups=2, n_rows=5, prefix=P,
             po=P, n_prefix=50, tail=P, to=P, n_tail=9, H=4, Hk=2, hd=128, scale=0.1, scratch=P,
             bytes=1 << 40, status=None, stream=None)
    a.update(kw)
    return _lib().lt_attn_prefix(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=-1), ARG), (dict(n_rows=-1), ARG), (dict(n_groups=-1), ARG), (dict(n_slots=-1), ARG),
    (dict(n_prefix=-1), ARG), (dict(n_tail=-1), ARG), (dict(scale=0.0), ARG), (dict(hd=40), SHAPE),
    (dict(H=5), SHAPE), (dict(n_rows=65536), SHAPE), (dict(q=None), ARG), (dict(cache=None), ARG),
    (dict(o=None), ARG), (dict(ro=None), ARG), (dict(prefix=None), ARG), (dict(po=None), ARG),
    (dict(tail=None), ARG), (dict(to=None), ARG), (dict(scratch=None), ARG), (dict(sq=500), ARG),
    (dict(so=8), ARG), (dict(sq=513), SHAPE), (dict(cache=P + 8), SHAPE), (dict(o=P + 8), SHAPE),
    (dict(scratch=P + 4), SHAPE), (dict(scratch=P + 16), SHAPE), (dict(n_prefix=2**31 - 1, n_rows=4000), SHAPE), (dict(bytes=1000), CAPACITY), (dict(n_rows=0), 0), (dict(n_groups=0), 0),
])
def test_prefix_refusals(kw, code):
    assert _prefix(**kw) == code


def _verify(**kw):
    a = dict(p=P, sp=100, q=P, sq=100, x=P, off=P, n=2, k=5, V=100, ua=P, ud=P, acc=P, tok=P, status=None,
             stream=None)
    a.update(kw)
    return _lib().lt_verify_drafts(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), ARG), (dict(k=-1), ARG), (dict(V=0), ARG),
    (dict(V=2**30 + 1, sp=2**31, sq=2**31), ARG), (dict(p=None), ARG), (dict(sp=99), ARG),
    (dict(sq=99), ARG), (dict(x=None), ARG), (dict(off=None), ARG), (dict(ua=None), ARG),
    (dict(ud=None), ARG), (dict(acc=None), ARG), (dict(tok=None), ARG), (dict(n=0), 0),
])
def test_verify_refusals(kw, code):
    assert _verify(**kw) == code


def test_scratch_sizes():
    L, n = _lib(), ctypes.c_size_t()
    for f in (L.lt_attn_prompt_scratch_bytes, L.lt_attn_prefix_scratch_bytes):
        assert f(1, 8, 1, 16, 16, 128, ctypes.byref(n)) == 0 and n.value > 0
        assert f(1, 8, 1, 16, 16, 128, None) == ARG
        assert f(3, 8, 1, 16, 16, 128, ctypes.byref(n)) == ARG
        assert f(1, 8, 1, 16, 5, 128, ctypes.byref(n)) == SHAPE
        assert f(1, 0, 0, 16, 16, 128, ctypes.byref(n)) == 0
