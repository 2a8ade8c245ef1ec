"""Rows of q that an offset list puts outside q: those inside are computed, at their positions; nothing else is
written, and the flag is set."""
import math

import numpy as np
import pytest
import torch

import kv8_reference as ref
from memory_bound_transformer_decode_gb300 import ddl
from test_gpu_kv8 import dev, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    ddl.load(build_if_missing=True)


@pytest.mark.parametrize("codes,hd,dtype,bound", [("e4m3", 128, "bf16", None), ("e4m3", 128, "f32", 60000),
                                                  ("int8", 64, "f32", None), ("int8", 128, "bf16", 60000)])
@pytest.mark.parametrize("offs,lens", [([-2, 1, 3], [50, 40]), ([0, 1, 5], [50, 40]), ([-3, 6], [300]), ([-9, -2], [70]),
                                       ([3, 7], [70]), ([2, 0], [70]), ([-40, 3], [20]), ([-2, 9], [0]),
                                       ([-1, 2, 3], [700, 1]), ([0, 1, 3, 64], [9, 20, 500])])
@pytest.mark.parametrize("window", [0, 9])
def test_rows_outside_are_left_out(codes, hd, dtype, bound, offs, lens, window):
    T, H_q, most = 3, 8, 64
    pool, q, _, lens, table = setup(len(lens), [1] * len(lens), H_q, 2, hd, 16, lens, codes, dtype, seed=41)
    g = torch.Generator(device="cuda").manual_seed(5)
    wide = torch.randn((200, H_q, hd), generator=g, device="cuda").to(q.dtype)  # row i of q is row 100 + i
    q = wide[100:100 + T].clone()
    out = torch.full_like(q, 7.0)
    lse = torch.full((T, H_q), 7.0, device="cuda")
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    ddl.ddl_kv8_attention(pool, q, dev(lens), dev(table), bound or int(max(1, lens.max())), q_off=dev(offs),
                          max_rows=most, window=window, out=out, lse=lse, bad=bad)
    assert int(bad) == 1
    for r in range(len(lens)):  # one request at a time, in a q that has all its rows
        a, b = offs[r], offs[r + 1]
        if b <= a:
            continue
        want, want_l, tol, tol_l = ref.attention(pool, wide[100 + a:100 + b], [0, b - a], lens[r:r + 1], table[r:r + 1],
                                                 1 / math.sqrt(hd), window=window)
        for i in range(max(a, 0), min(b, T)):
            assert ((out[i].double() - want[i - a]).abs() <= tol[i - a]).all(), (r, i)
            l, wl = lse[i].double(), want_l[i - a]
            assert torch.equal(l == -math.inf, wl == -math.inf)
            assert ((l - wl).abs()[wl > -math.inf] <= tol_l[i - a][wl > -math.inf]).all()
    mine = np.zeros(T, bool)
    for a, b in zip(offs, offs[1:]):
        mine[max(a, 0):max(0, min(b, T))] = True
    rest = torch.from_numpy(~mine).cuda()
    assert (out[rest] == 7).all() and (lse[rest] == 7).all()


@pytest.mark.parametrize("codes,hd", [("e4m3", 128), ("int8", 64)])
def test_offsets_as_far_apart_as_can_be(codes, hd):
    pool, q, _, lens, table = setup(1, [1], 8, 2, hd, 16, [50], codes, "bf16", seed=42)
    q = q.repeat(3, 1, 1)
    out, bad = torch.full_like(q, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    for offs in ([-2 ** 31, 2 ** 31 - 1], [0, 2 ** 31 - 1]):
        for window in (0, 5, 2 ** 31 - 2):
            ddl.ddl_kv8_attention(pool, q, dev(lens), dev(table), 2 ** 31 - 1, q_off=dev(offs), max_rows=64, window=window,
                                  out=out, bad=bad)
            assert int(bad) == 1 and (out == 0).all()  # (all rows there are lie before the first token)
            out.fill_(7.0)
    for offs in ([2 ** 31 - 1, -2 ** 31], [2 ** 31 - 1, 2 ** 31 - 1], [-2 ** 31, -2 ** 31], [-2 ** 31, 0]):
        bad.zero_()
        ddl.ddl_kv8_attention(pool, q, dev(lens), dev(table), 64, q_off=dev(offs), max_rows=64, out=out, bad=bad)
        assert int(bad) == 1 and (out == 7).all()
