"""Cache scores, eviction and filtered draws without a GPU: the host's refusals
and the references' own small cases."""
import ctypes
import math

import numpy as np
import pytest
import torch

import serving_reference as sref
from memory_bound_transformer_decode_gb300 import build, ddl
from test_kv8_cpu import BAD_POOLS, _kv


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ddl.load()


def v(n):
    return ctypes.c_void_p(256 * n)


def needs_no_gpu():
    if torch.cuda.is_available():
        pytest.skip("host checks with fake pointers run without a GPU")


def test_score_refusals(lib):
    needs_no_gpu()

    def call(opts=(0.1, 0.0, 0, None), **kw):
        a = dict(kv=_kv(), Hq=8, Hkv=2, hd=64, dt=1, opts=None, R=2, T=2, rows=1, len=100, off=None, kl=v(1), tab=v(2),
                 per=7, q=v(3), qs=512, lse=v(4), decay=1.0, score=v(5), stride=100, bad=None)
        a.update(kw)
        a["opts"] = ddl.AttnOpts(*opts) if opts else None
        return lib.ddl_kv8_score(*a.values(), None)

    assert call() == 6  # past the host checks: no device here
    assert call(decay=0.0) == 6
    for kw, code in BAD_POOLS:
        assert call(kv=_kv(**kw)) == code, kw
    for kw, code in [(dict(Hq=7), 1), (dict(Hq=18, qs=2048), 1), (dict(Hq=0), 1), (dict(hd=32), 1), (dict(dt=-1), 5),
                     (dict(opts=None), 8), (dict(opts=(math.inf, 0.0, 0, None)), 8), (dict(opts=(0.1, -1.0, 0, None)), 8),
                     (dict(opts=(0.1, 0.0, -1, None)), 8), (dict(opts=(0.1, 0.0, 0, 258)), 3), (dict(R=0), 8),
                     (dict(R=4097, T=4097), 5), (dict(T=1), 8), (dict(rows=2), 8), (dict(rows=65, off=v(6)), 5),
                     (dict(len=0), 8), (dict(kl=None), 8), (dict(tab=None), 8), (dict(per=0), 8), (dict(per=1 << 28), 5),
                     (dict(q=None), 8), (dict(lse=None), 8), (dict(score=None), 8), (dict(qs=504), 8), (dict(qs=516), 8),
                     (dict(q=ctypes.c_void_p(264)), 3), (dict(lse=ctypes.c_void_p(258)), 3),
                     (dict(score=ctypes.c_void_p(258)), 3), (dict(stride=99), 8), (dict(decay=-0.1), 8),
                     (dict(decay=1.5), 8), (dict(decay=math.nan), 8)]:
        assert call(**kw) == code, kw


def test_evict_refusals(lib):
    needs_no_gpu()

    def call(**kw):
        a = dict(kv=_kv(), H=2, hd=64, R=2, len=100, score=v(1), stride=100, kl=v(2), keep=v(3), sinks=0, recent=0,
                 tab=v(4), per=7, new=v(5), nper=3, most=40, kept=v(6), out=v(7), bad=None)
        a.update(kw)
        return lib.ddl_kv8_evict(*a.values(), None)

    assert call() == 6
    for kw, code in BAD_POOLS:
        assert call(kv=_kv(**kw)) == code, kw
    for kw, code in [(dict(H=0), 1), (dict(hd=96), 1), (dict(R=0), 8), (dict(R=4097), 5), (dict(len=0), 8),
                     (dict(stride=99), 8), (dict(sinks=-1), 8), (dict(recent=-1), 8), (dict(per=0), 8), (dict(nper=0), 8),
                     (dict(per=1 << 28), 5), (dict(nper=1 << 28), 5), (dict(most=0), 8), (dict(most=101), 8),
                     (dict(score=None), 8), (dict(kl=None), 8), (dict(keep=None), 8), (dict(tab=None), 8),
                     (dict(new=None), 8), (dict(kept=None), 8), (dict(out=None), 8), (dict(out=v(1)), 8),
                     (dict(new=v(4)), 8), (dict(kept=ctypes.c_void_p(258)), 3), (dict(bad=ctypes.c_void_p(258)), 3)]:
        assert call(**kw) == code, kw


def test_sample_refusals(lib):
    needs_no_gpu()

    def call(**kw):
        a = dict(x=v(1), dt=0, stride=1000, B=3, V=1000, t=None, k=None, p=None, m=None, u=v(2), tok=v(3), lp=None)
        a.update(kw)
        return lib.ddl_sample(*a.values(), None)

    assert call() == 6
    assert call(x=ctypes.c_void_p(260)) == 6 and call(x=ctypes.c_void_p(258), dt=1) == 6
    for kw, code in [(dict(x=None), 8), (dict(u=None), 8), (dict(tok=None), 8), (dict(B=0), 8), (dict(V=0), 8),
                     (dict(stride=999), 8), (dict(dt=3), 5), (dict(B=65537), 5), (dict(V=2 ** 20 + 1, stride=2 ** 21), 5),
                     (dict(x=ctypes.c_void_p(258)), 3), (dict(x=ctypes.c_void_p(257), dt=2), 3),
                     (dict(t=ctypes.c_void_p(258)), 3), (dict(lp=ctypes.c_void_p(258)), 3)]:
        assert call(**kw) == code, kw


def test_bindings_refuse_host_tensors_and_wrong_shapes(lib):
    pool = (torch.zeros((2, 1, 16, 64), dtype=torch.int8), torch.zeros((2, 1, 16, 64), dtype=torch.int8),
            torch.zeros((2, 1, 1)), torch.zeros((2, 1, 1)))
    i, x, s = torch.zeros(1, dtype=torch.int32), torch.zeros((1, 1, 64)), torch.zeros((1, 1, 16))
    with pytest.raises(ValueError):
        ddl.ddl_kv8_score(pool, x, torch.zeros((1, 1)), i, i.view(1, 1), 16, s)
    with pytest.raises(ValueError):
        ddl.ddl_kv8_evict(pool, s, i, i, i.view(1, 1), i.view(1, 1), 16, kept=i.view(1, 1, 1), score_out=s)
    with pytest.raises(ValueError, match="logits"):
        ddl.ddl_sample(torch.zeros((1, 8)), torch.zeros(1), tokens=i)


def test_reference_draw():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    for u, tok in ((0.05, 0), (0.15, 1), (0.6, 2), (0.9, 3)):
        assert set(sref.draw(x, 1.0, 0, 1.0, 0.0, u)) == {tok}
    assert set(sref.draw(x, 1.0, 2, 1.0, 0.0, 0.5)) == {1} and set(sref.draw(x, 1.0, 2, 1.0, 0.0, 0.6)) == {3}
    assert set(sref.draw(x, 1.0, 0, 0.5, 0.0, 0.99)) == {3}   # 0.4, 0.7: two stay
    assert set(sref.draw(x, 1.0, 0, 1.0, 0.6, 0.99)) == {3} and set(sref.draw(x, 0.0, 0, 1.0, 0.0, 0.99)) == {1}


def test_reference_evict():
    score = np.array([[[5.0, 1.0, 3.0, 3.0, 0.0, 9.0, 2.0]]])
    codes = [np.arange(2 * 16 * 64, dtype=np.uint8).reshape(2, 1, 16, 64) % 100 for _ in range(2)]
    scales = [np.full((2, 1, 1), 0.5) for _ in range(2)]
    kept, out = np.full((1, 1, 4), -1), np.zeros((1, 1, 7))
    c, s, kept, out = sref.evict(codes, scales, score, [7], [4], np.array([[0]]), np.array([[1]]), 1, 1, 16, True, kept, out)
    assert kept.tolist() == [[[0, 2, 5, 6]]] and out[0, 0, :4].tolist() == [5, 3, 9, 2]
    x = codes[0][0, 0, [0, 2, 5, 6]].astype(float) * 0.5
    assert np.array_equal(c[0][1, 0, :4].astype(float) * s[0][1, 0, 0], x) and not c[0][1, 0, 4:].any()


def test_scored_stack_refusals(lib):
    needs_no_gpu()
    shape = ddl.Shape(512, 8, 2, 64, 1408, 1e-6, 1e4)
    lw = (ddl.LayerW * 2)(ddl.LayerW(256, 256, 256), ddl.LayerW(256, 256, 256))
    kv = (ddl.KV8 * 2)(_kv(), _kv())

    def call(scores=(2560, 2816), **kw):
        ptrs = (ctypes.c_void_p * 2)(*scores) if scores else None
        a = dict(kv=kv, L=2, opts=None, R=2, T=3, rows=2, len=64, off=v(1), kl=v(2), pos=v(3), slot=v(4), tab=v(5), per=4,
                 res=None, x=v(6), rout=None, out=v(7), score=ptrs, stride=64, decay=1.0, bad=None, ws=v(8), n=1 << 30)
        a.update(kw)
        return lib.ddl_stack_step_kv8_scored(ctypes.byref(shape), ddl.INT4, lw, *a.values(), None)

    assert call() == 6
    assert call(scores=None) == 8 and call(scores=(2560, None)) == 8 and call(scores=(2560, 2818)) == 3
    for kw, code in [(dict(stride=63), 8), (dict(decay=1.1), 8), (dict(decay=math.nan), 8), (dict(L=0), 8), (dict(T=65), 5),
                     (dict(ws=None), 4), (dict(slot=None), 8)]:
        assert call(**kw) == code, kw
    assert lib.ddl_stack_kv8_scored_workspace_bytes(ctypes.byref(shape), 0, 3, 2, 64) == 0
