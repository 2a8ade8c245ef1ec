"""The 8-bit paged KV cache without a GPU: the references the GPU tests compare
with against closed forms and brute force, and the entry points' refusals
(argument errors are found on the host, before any device work).
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import kv8_reference as ref
from memory_bound_transformer_decode_gb300 import build, ddl


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ddl.load()


# ------------------------------------------------------------------ references

def test_e4m3_codes_are_torchs():
    raw = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(raw, ref.E4M3, equal_nan=True)
    x = np.concatenate([np.random.RandomState(0).randn(20000) * 100, np.linspace(-460, 460, 40001),
                        ref.E4M3[:127], (ref.E4M3[1:127] + ref.E4M3[:126]) / 2, [0.0, -0.0, 2.0 ** -10, 1e-9]])
    x = x.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(np.clip(x, -448, 448)).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.encode_e4m3(x), want)


def test_append_reference_by_hand():
    codes, scale = np.zeros((1, 1, 16, 64), np.uint8), np.ones((1, 1, 1))
    x = np.zeros((2, 1, 64))
    x[0, 0, 0], x[1, 0, 0] = 7.0, 28.0          # 7 = 448 * 2^-6, 28 = 448 * 2^-4
    c1, s1 = ref.append(codes, scale, x[:1], np.array([0]), 16, False)
    assert s1[0, 0, 0] == 2.0 ** -6 and ref.E4M3[c1[0, 0, 0, 0]] == 448
    c2, s2 = ref.append(c1, s1, x[1:], np.array([1]), 16, False)   # the scale grows by 4, the old value stays
    assert s2[0, 0, 0] == 2.0 ** -4 and ref.E4M3[c2[0, 0, 0, 0]] == 112 and ref.E4M3[c2[0, 0, 1, 0]] == 448
    c3, s3 = ref.append(c1, s1, x[1:] * 0.5, np.array([0]), 16, True)  # a block's first token: no old scale
    assert s3[0, 0, 0] == 0.125 and c3[0, 0, 0, 0] == 112


def test_attention_reference_by_hand():
    """Two keys whose scores differ by ln 3: weights 3/4 and 1/4."""
    k = torch.zeros((1, 1, 16, 64), dtype=torch.int8)
    v = torch.zeros_like(k)
    k[0, 0, 0, 0], v[0, 0, 0], v[0, 0, 1] = 1, 4, 8
    sc = torch.ones((1, 1, 1))
    q = torch.zeros((1, 1, 64))
    q[0, 0, 0] = math.log(3.0)
    out, lse, tol, _ = ref.attention((k, v, sc, sc), q, [0, 1], [2], [[0]], 1.0)
    assert torch.allclose(out, torch.full_like(out, 5.0), atol=1e-6) and abs(float(lse) - math.log(4)) < 1e-6
    assert 0 < float(tol.max()) < 1e-3
    out, lse, _, _ = ref.attention((k, v, sc, sc), q, [0, 1], [0], [[0]], 1.0)
    assert (out == 0).all() and float(lse) == -math.inf
    out, _, _, _ = ref.attention((k, v, sc, sc), q, [0, 1], [2], [[0]], 1.0, window=1)
    assert (out == 8).all()


def test_plan_reference_by_hand():
    table, off, kl, pos, slot, used, st = ref.plan([15, 0, 3], [2, 20, 1], [7, 8], np.array([[1, -1], [-1, -1], [2, -1]]),
                                                   16, 6)
    assert st.tolist() == [0, 2, 3] or st.tolist() == [0, 2, 0]
    assert table.tolist() == [[1, 7], [-1, -1], [2, -1]] and used.tolist() == [1]
    assert kl[:2].tolist() == [17, 0] and pos[:2].tolist() == [15, 16] and slot[:2].tolist() == [31, 112]


# ------------------------------------------------------------------ refusals

def _kv(**kw):
    f = dict(k=256, v=256, k_scale=256, v_scale=256, pages=10, page_size=16, type=0)
    f.update(kw)
    return ddl.KV8(*[f[n] for n in ("k", "v", "k_scale", "v_scale", "pages", "page_size", "type")])


BAD_POOLS = [(dict(k=None), 8), (dict(v_scale=None), 8), (dict(pages=0), 8), (dict(page_size=24), 8),
             (dict(page_size=8), 8), (dict(page_size=1 << 21), 8), (dict(pages=1 << 27), 5), (dict(type=2), 5),
             (dict(v=264), 3), (dict(k_scale=260), 3)]


def test_append_refusals(lib):
    if torch.cuda.is_available():  # fake device pointers must never reach a GPU
        pytest.skip("host checks with fake pointers run without a GPU; tests/test_gpu_kv8.py has real buffers")
    p = ctypes.c_void_p(256)

    def call(kv=None, H=2, hd=64, dt=1, k=p, ks=128, v=p, vs=128, slot=p, T=3, bad=None):
        return lib.ddl_kv8_append(kv or _kv(), H, hd, dt, k, ks, v, vs, slot, T, bad, None)

    assert call() == 6  # past the host checks: no device here
    for kw, code in BAD_POOLS:
        assert call(_kv(**kw)) == code, kw
    for kw, code in [(dict(H=0), 2 - 1), (dict(H=1025), 1), (dict(hd=96), 1), (dict(dt=3), 5), (dict(k=None), 8),
                     (dict(slot=None), 8), (dict(T=0), 8), (dict(T=65537), 5), (dict(ks=120), 8),
                     (dict(vs=132), 8), (dict(k=ctypes.c_void_p(264)), 3), (dict(slot=ctypes.c_void_p(257)), 3),
                     (dict(bad=ctypes.c_void_p(258)), 3)]:
        assert call(**kw) == code, kw


def test_plan_refusals(lib):
    if torch.cuda.is_available():
        pytest.skip("host checks with fake pointers run without a GPU; tests/test_gpu_kv8.py has real buffers")
    v = lambda n: ctypes.c_void_p(256 * n)  # noqa: E731

    def call(**kw):
        a = dict(old=v(1), add=v(2), R=4, P=16, free=v(3), nf=9, tab=v(4), per=5, off=v(5), kl=v(6), pos=v(7),
                 slot=v(8), T=7, used=v(9), st=v(10))
        a.update(kw)
        return lib.ddl_page_plan(*a.values(), None)

    assert call() == 6
    assert call(free=None, nf=0) == 6 and call(pos=None, slot=None, T=0) == 6
    for kw, code in [(dict(old=None), 8), (dict(tab=None), 8), (dict(used=None), 8), (dict(R=0), 8), (dict(R=4097), 5),
                     (dict(P=17), 8), (dict(P=8), 8), (dict(nf=-1), 8), (dict(free=None), 8), (dict(T=-1), 8),
                     (dict(slot=None), 8), (dict(per=0), 8), (dict(per=1 << 28), 5), (dict(kl=v(1)), 8),
                     (dict(st=ctypes.c_void_p(257)), 3)]:
        assert call(**kw) == code, kw


def test_attention_refusals(lib):
    if torch.cuda.is_available():
        pytest.skip("host checks with fake pointers run without a GPU; tests/test_gpu_kv8.py has real buffers")
    v = lambda n: ctypes.c_void_p(256 * n)  # noqa: E731

    def call(opts=(0.1, 0.0, 0, None), **kw):
        a = dict(kv=_kv(), Hq=8, Hkv=2, hd=64, dt=1, opts=None, R=2, T=2, rows=1, len=100, off=None, kl=v(1), tab=v(2),
                 per=7, q=v(3), qs=512, out=v(4), os=512, lse=None, bad=None, ws=v(5), n=1 << 30)
        a.update(kw)
        a["opts"] = ddl.AttnOpts(*opts) if opts else None
        return lib.ddl_kv8_attention(*a.values(), None)

    assert call() == 6
    for kw, code in BAD_POOLS:
        assert call(kv=_kv(**kw)) == code, kw
    for kw, code in [(dict(Hq=7), 1), (dict(Hq=18, qs=2048, os=2048), 1), (dict(Hq=0), 1), (dict(hd=32), 1),
                     (dict(dt=-1), 5), (dict(opts=None), 8), (dict(opts=(math.inf, 0.0, 0, None)), 8),
                     (dict(opts=(0.1, -1.0, 0, None)), 8), (dict(opts=(0.1, math.nan, 0, None)), 8),
                     (dict(opts=(0.1, 0.0, -1, None)), 8), (dict(opts=(0.1, 0.0, 0, 258)), 3), (dict(R=0), 8),
                     (dict(R=4097, T=4097), 5), (dict(T=1), 8), (dict(rows=2), 8), (dict(rows=65, off=v(6)), 5),
                     (dict(len=0), 8), (dict(kl=None), 8), (dict(tab=None), 8), (dict(per=0), 8),
                     (dict(per=1 << 28), 5), (dict(q=None), 8), (dict(out=v(3)), 8), (dict(qs=504), 8),
                     (dict(os=516), 8), (dict(q=ctypes.c_void_p(264)), 3), (dict(lse=ctypes.c_void_p(258)), 3),
                     (dict(ws=None), 4)]:
        assert call(**kw) == code, kw
    assert lib.ddl_kv8_attention_workspace_bytes(8, 2, 96, 1, 1, 1, 100) == 0


def test_stack_step_refusals(lib):
    if torch.cuda.is_available():
        pytest.skip("host checks with fake pointers run without a GPU; tests/test_gpu_kv8_stack.py has real buffers")
    v = lambda n: ctypes.c_void_p(256 * n)  # noqa: E731
    shape = ddl.Shape(512, 8, 2, 64, 1408, 1e-6, 1e4)
    lw = (ddl.LayerW * 2)(ddl.LayerW(256, 256, 256), ddl.LayerW(256, 256, 256))

    def call(kv=None, opts=None, **kw):
        kv = (ddl.KV8 * 2)(*(kv or [_kv(), _kv()]))
        a = dict(kv=kv, L=2, opts=ddl.AttnOpts(*opts) if opts else None, R=2, T=3, rows=2, len=64, off=v(1), kl=v(2),
                 pos=v(3), slot=v(4), tab=v(5), per=4, res=None, x=v(6), rout=None, out=v(7), bad=None, ws=v(8),
                 n=1 << 30)
        a.update(kw)
        return lib.ddl_stack_step_kv8(ctypes.byref(shape), ddl.INT4, lw, *a.values(), None)

    assert call() == 6  # past the host checks: no device here
    for kw, code in BAD_POOLS:
        assert call(kv=[_kv(), _kv(**kw)]) == code, kw
    for kw, code in [(dict(kv=[_kv(), _kv(page_size=32)]), 8), (dict(kv=[_kv(), _kv(pages=11)]), 8), (dict(L=0), 8),
                     (dict(T=0), 5), (dict(T=65), 5), (dict(off=None), 8), (dict(slot=None), 8), (dict(R=0), 8),
                     (dict(rows=65), 5), (dict(rows=0), 8), (dict(len=0), 8), (dict(per=0), 8), (dict(per=1 << 28), 5),
                     (dict(pos=ctypes.c_void_p(258)), 3), (dict(ws=None), 4), (dict(ws=ctypes.c_void_p(264)), 3),
                     (dict(opts=(1.0, -1.0, 0, None)), 8), (dict(opts=(1.0, 0.0, 0, 258)), 3)]:
        assert call(**kw) == code, kw


def test_bindings_refuse_host_tensors(lib):
    pool = (torch.zeros((2, 1, 16, 64), dtype=torch.int8), torch.zeros((2, 1, 16, 64), dtype=torch.int8),
            torch.zeros((2, 1, 1)), torch.zeros((2, 1, 1)))
    x = torch.zeros((1, 1, 64))
    with pytest.raises(ValueError):
        ddl.ddl_kv8_append(pool, x, x, torch.zeros(1, dtype=torch.int32))
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        ddl.ddl_kv8_attention(pool, x, i, i.view(1, 1), 16, workspace=torch.empty(4096, dtype=torch.uint8))
