"""CPU checks of what the calls on 4-bit caches, the read-back and the head norms refuse: fake
pointers, which a refused call never follows."""
import ctypes

import pytest

from speculative_decoding_draft_bf16_gb300 import dtree
from test_abi_cpu import _cache, _rope, _rows

ref = ctypes.byref


def _append4(cache=None, rope=None, batch=1, M=3, dtype=0, k=None, rows=None, N=3, len_out=None, status=0x7000, count=None,
             count_add=0):
    return dtree.lib().dt_kv_append4(ref(cache or _cache()), ref(rope) if rope else None, batch, M, dtype,
                                     ref(k or _rows()), ref(_rows()), rows, N, count, count_add, len_out, status, None)


def _attention4(cache=None, rope=None, batch=1, M=3, Hq=4, q=None, scale=1.0, out=0x8000, ws=0x9000, n=1 << 40,
                status=0x7000):
    return dtree.lib().dt_tree_attention4(ref(cache or _cache()), ref(rope) if rope else None, batch, M, Hq,
                                          ref(q or _rows()), ref(_rows()), ref(_rows()), None, None, None, scale, out,
                                          ws, n, status, None)


def _read(four, cache=None, batch=1, rows=None, N=3, start=None, count=None, count_add=0, dtype=0, k=None, v=None,
          status=0x7000):
    call = dtree.lib().dt_kv_read4 if four else dtree.lib().dt_kv_read
    return call(ref(cache or _cache()), batch, rows, N, start, count, count_add, dtype, ref(k or _rows()),
                ref(v or _rows(ptr=0x9000)), status, None)


def _norm(batch=1, M=3, Hq=4, Hk=2, D=64, dtype=0, q=None, k=None, qw=0x2000, qs=0, kw=0x3000, ks=0, eps=1e-6, rope=None,
          q_out=None, k_out=None, status=0x7000):
    return dtree.lib().dt_qk_norm(batch, M, Hq, Hk, D, dtype, ref(q or _rows()), ref(k or _rows()), qw, qs, kw, ks, eps,
                                  ref(rope) if rope else None, None, None, None, ref(q_out or _rows()),
                                  ref(k_out or _rows(ptr=0x9000)), status, None)


@pytest.mark.parametrize("call", [_append4, _attention4, lambda **kw: _read(True, **kw), lambda **kw: _read(False, **kw)])
@pytest.mark.parametrize("bad,rc", [
    (dict(page=48), -1), (dict(page=0), -1), (dict(n_pages=0), -1), (dict(max_pages=0), -1), (dict(Hkv=0), -1),
    (dict(D=0), -1), (dict(D=96), -2), (dict(max_pages=1 << 30), -2), (dict(k=None), -1), (dict(v=0x2008), -1),
    (dict(v_scale=None), -1), (dict(table=None), -1), (dict(len=None), -1), (dict(Hkv=65536), -2),
])
def test_invalid_caches(call, bad, rc):
    assert call(cache=_cache(**bad)) == rc


@pytest.mark.parametrize("call", [_append4, _attention4, lambda **kw: _read(True, **kw)])
def test_scale_bytes_start_on_16_bytes(call):
    assert call(cache=_cache(k_scale=0x3008)) == -1 and call(cache=_cache(v_scale=0x4004)) == -1


@pytest.mark.parametrize("call", [_append4, _attention4, _norm])
@pytest.mark.parametrize("bad", [dict(rot=0), dict(rot=8), dict(rot=40), dict(rot=80), dict(max_pos=0), dict(cos=None),
                                 dict(sin=0x2004), dict(interleaved=2)])
def test_invalid_rotations(call, bad):
    assert call(rope=_rope(**bad)) == -1


def test_append():
    for kw in (dict(batch=0), dict(M=0), dict(N=0), dict(N=4), dict(dtype=2), dict(status=None), dict(len_out=0x6000),
               dict(k=_rows(ptr=None)), dict(k=_rows(ptr=0x1002)), dict(k=_rows(stride_n=100)),
               dict(k=_rows(stride_b=-1024)), dict(count=0x8000, count_add=(1 << 30) + 1)):
        assert _append4(**kw) == -1, kw
    assert _append4(rows=0x8000, N=(1 << 30) + 1) == -2


def test_attention():
    nan, inf = float("nan"), float("inf")
    for kw in (dict(batch=0), dict(M=0), dict(Hq=0), dict(Hq=3), dict(scale=0.0), dict(scale=-1.0), dict(scale=nan),
               dict(scale=inf), dict(out=None), dict(out=0x8004), dict(status=None), dict(q=_rows(ptr=None)),
               dict(q=_rows(stride_h=60))):
        assert _attention4(**kw) == -1, kw
    assert _attention4(Hq=2 * 129) == -2
    need = dtree.lib().dt_tree_attention4_workspace(ref(_cache()), 1, 3, 4)
    assert need == dtree.lib().dt_tree_attention_workspace(ref(_cache()), 1, 3, 4)
    assert _attention4(ws=None) == -1 and _attention4(ws=0x9004) == -1 and _attention4(n=need - 1) == -1


@pytest.mark.parametrize("four", [False, True])
def test_read(four):
    for kw in (dict(batch=0), dict(N=0), dict(dtype=2), dict(status=None), dict(rows=0x8000, start=0x9000),
               dict(k=_rows(ptr=None)), dict(v=_rows(ptr=0x1008)), dict(v=_rows(stride_n=100)),
               dict(v=_rows()), dict(k=_rows(stride_n=0)), dict(v=_rows(stride_h=56)), dict(k=_rows(stride_b=0), batch=2),
               dict(count=0x8000, count_add=-(1 << 30) - 1)):
        assert _read(four, **kw) == -1, kw
    assert _read(four, N=(1 << 30) + 1) == -2 and _read(four, cache=_cache(Hkv=32768)) == -2


def test_norm():
    nan, inf = float("nan"), float("inf")
    for kw in (dict(batch=0), dict(M=0), dict(Hq=-1), dict(Hk=-1), dict(Hq=0, Hk=0), dict(D=0), dict(dtype=2),
               dict(eps=-1e-6), dict(eps=nan), dict(eps=inf), dict(status=None), dict(qw=0x2004), dict(qs=63), dict(ks=128),
               dict(q=_rows(ptr=None)), dict(k=_rows(ptr=0x1004)), dict(q_out=_rows(stride_h=60)),
               dict(k_out=_rows(ptr=None)), dict(k_out=_rows()), dict(q_out=_rows(stride_h=0)), dict(k_out=_rows(stride_n=32)),
               dict(q_out=_rows(stride_b=0), batch=2)):
        assert _norm(**kw) == -1, kw
    for kw in (dict(D=96), dict(D=256), dict(batch=65536), dict(M=(1 << 20) + 1), dict(Hq=65536), dict(batch=2048, M=1 << 20)):
        assert _norm(**kw) == -2, kw


def test_null_caches():
    L = dtree.lib()
    assert L.dt_kv_append4(None, None, 1, 1, 0, ref(_rows()), ref(_rows()), None, 1, None, 0, None, 0x7000, None) == -1
    assert L.dt_kv_read4(None, 1, None, 1, None, None, 0, 0, ref(_rows()), ref(_rows()), 0x7000, None) == -1
    assert L.dt_kv_read(None, 1, None, 1, None, None, 0, 0, ref(_rows()), ref(_rows()), 0x7000, None) == -1
    assert L.dt_tree_attention4_workspace(None, 1, 1, 1) == 0


def test_the_division_counts_each_form_with_its_own_weights():
    """Refused (-2) where a form's units would leave 32 bits and not before; `status` is left out, so that
    what passes is refused next (-1) and nothing is launched."""
    def eight(cache, M):
        return dtree.lib().dt_tree_attention(ref(cache), None, 65535, M, cache.Hkv, ref(_rows()), ref(_rows()), ref(_rows()),
                                             None, None, None, 1.0, 0x8000, 0x9000, 1 << 40, None, None)

    def four(cache, M):
        return _attention4(cache=cache, batch=65535, M=M, Hq=cache.Hkv, status=None)

    # two tiles and an eighth a unit at most: with 17 rows 42.75 (4 bits) and 30.625 a unit, with 3 rows 8.125
    for Hkv, M, rc4, rc8 in ((1400, 17, -1, -1), (1800, 17, -2, -1), (2200, 17, -2, -2), (6000, 3, -1, -1), (8000, 3, -2, -2)):
        cache = _cache(Hkv=Hkv, max_pages=1, page=16)
        assert (four(cache, M), eight(cache, M)) == (rc4, rc8)
