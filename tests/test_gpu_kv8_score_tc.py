"""Attention weight drawn by cached tokens where a request brings many queries
(more than 8 tiles of 8 rows x heads, 4 of fp32 rows: the tensor-core kernel):
options, masks, decays, lengths, broken inputs and bounds against the 64-bit
reference, and the border to the kernel for fewer."""
import math

import numpy as np
import pytest
import torch

import serving_reference as sref
from memory_bound_transformer_decode_gb300 import ddl
from test_gpu_kv8 import dev
from test_gpu_kv8_score import case, check, lse_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ddl.load(build_if_missing=True)


OPTIONS = [dict(softcap=20.0), dict(softcap=0.5), dict(window=33), dict(window=300), dict(window=1), dict(slopes=1.0),
           dict(slopes=-0.02), dict(softcap=5.0, window=150, slopes=1.0)]


def with_slopes(opts, heads):
    if "slopes" not in opts:
        return opts
    return dict(opts, slopes=opts["slopes"] * torch.exp2(-8.0 * torch.arange(1, heads + 1, device="cuda") / heads))


@pytest.mark.parametrize("codes,dtype,hd", [("e4m3", "bf16", 128), ("int8", "f32", 128), ("e4m3", "f32", 64), ("int8", "f16", 64)])
@pytest.mark.parametrize("opts", OPTIONS, ids=str)
def test_options(codes, dtype, hd, opts):
    """Tiles with and without masks, tiles that only decay, queries in one group and (fp32, 512 of 128) in two."""
    lens, H = [700, 130, 385], 2
    for G, rows in ((8, [64, 33, 9]), (3, [64, 24, 40])):
        pool, table, q, off = case(lens, rows, H, G, hd, 64, codes, dtype, seed=G)
        for decay in (0.0, 0.5, 1.0):
            check(pool, table, q, off, lens, decay=decay, **with_slopes(opts, H * G))


@pytest.mark.parametrize("decay", [0.0, 0.9, 1.0])
@pytest.mark.parametrize("dtype,rows", [("f32", 64), ("bf16", 64), ("f16", 17)])
def test_lengths_and_decays(dtype, rows, decay):
    """Around tiles of 128 tokens, several tiles a CTA, more rows than tokens, requests without rows or tokens."""
    lens = [1, 127, 128, 129, 2049, 0, 300, 40]
    n = [1, rows, 5, rows, rows, 3, 0, rows]
    check(*case(lens, n, 1, 8, 128, 16, "e4m3", dtype, seed=rows), lens, decay=decay)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("queries", [32, 33, 40, 64, 65, 72, 256, 258, 264, 504, 512])
def test_numbers_of_queries(dtype, queries):
    """At the borders of the kernels, of a chunk and of a group of queries."""
    G = next(g for g in range(8, 0, -1) if queries % g == 0 and queries // g <= 64)
    check(*case([333], [queries // G], 2, G, 128, 32, "int8", dtype, seed=queries), [333], decay=0.5)


@pytest.mark.parametrize("max_len", [200, 4000, 100000])
def test_long_bounds_of_short_requests(max_len):
    lens = [200, 17]
    check(*case(lens, [40, 12], 2, 4, 64, 16, "int8", "bf16"), lens, max_len=max_len, decay=0.25)


def test_junk_outside_what_the_rows_see_has_no_effect():
    lens, rows = [300], 40
    pool, table, q, off = case(lens, [rows], 2, 4, 128, 64, "e4m3", "bf16")
    a, _ = check(pool, table, q, off, lens, window=20)       # tokens 241 .. 299 are seen
    raw = pool[0].view(torch.uint8)
    raw[table[0, :3].tolist()] = 127
    raw[table[0, 3], :, :49] = 127                           # up to token 240, in a block that is seen
    pool[2][table[0, :3].tolist()] = math.inf
    pool[2][table[0, 3], :, :3] = math.nan
    raw[table[0, 4], :, 44:] = 255                           # behind the last token
    pool[2][table[0, 4], :, 3] = -math.inf
    b, _ = check(pool, table, q, off, lens, window=20)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_nan_codes_and_broken_scales_stay_with_their_tokens(dtype):
    lens, rows, scale = [300, 260], 40, 128 ** -0.5
    pool, table, q, off = case(lens, [rows, rows], 2, 4, 128, 64, "e4m3", dtype)
    lse = lse_of(pool, q, off, lens, table, scale)
    old = torch.rand((2, 2, 300), device="cuda")
    want, tol = sref.score(pool, q, lse, off, lens, table, old, 0.5, scale)
    raw, nan = pool[0].view(torch.uint8), torch.zeros_like(old, dtype=torch.bool)
    raw[table[0, 1], 0, 13, 5] = 127
    nan[0, 0, 64 + 13] = True
    raw[table[1, 4], 1, 3, 127] = 255          # token 259: the newest row alone sees it
    nan[1, 1, 259] = True
    pool[2][table[0, 4], 1, 2] = math.inf      # tokens 288 .. 299
    nan[0, 1, 288:300] = True
    pool[2][table[1, 0], 0, 1] = math.nan
    nan[1, 0, 16:32] = True
    got = old.clone()
    ddl.ddl_kv8_score(pool, q, lse, dev(lens), dev(table), 300, got, q_off=dev(off), max_rows=rows, decay=0.5, scale=scale)
    assert torch.equal(got.isnan(), nan)
    assert float(torch.where(nan, 0, (got.double() - want).abs() - tol).max()) <= 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_log_sums_that_are_not_finite(dtype):
    lens, rows, scale = [200, 200], 40, 0.125
    pool, table, q, off = case(lens, [rows, rows], 1, 4, 64, 16, "e4m3", dtype)
    lse = lse_of(pool, q, off, lens, table, scale)
    lse[:20] = -math.inf
    lse[25, 1] = -math.inf
    lse[30, 2] = math.inf
    want, tol = sref.score(pool, q, lse, off, lens, table, torch.ones((2, 1, 200), device="cuda"), 1.0, scale)
    lse[rows + 5, 3] = math.nan                # sees tokens 0 .. 165
    got = torch.ones((2, 1, 200), device="cuda")
    ddl.ddl_kv8_score(pool, q, lse, dev(lens), dev(table), 200, got, q_off=dev(off), max_rows=rows, scale=scale)
    assert got[1, 0, :166].isnan().all() and int(got.isnan().sum()) == 166
    assert float(((got.double() - want).abs() - tol).nan_to_num(nan=0.0).max()) <= 0


def test_bounds_of_the_launch():
    """As the kernel for fewer queries: what lies outside is reported, the rest computed."""
    lens, rows = [300, 300], 32
    pool, table, q, off = case(lens, [rows, rows], 2, 4, 64, 16, "int8", "bf16")
    lse = lse_of(pool, q, off, lens, table, 0.125)

    def run(kv_len, tab, max_len=300, q_off=None, max_rows=rows, T=2 * rows):
        bad = torch.zeros(1, dtype=torch.int32, device="cuda")
        score = torch.ones((2, 2, 300), device="cuda")
        ddl.ddl_kv8_score(pool, q[:T], lse[:T], dev(kv_len), dev(tab), max_len, score, bad=bad, scale=0.125,
                          q_off=dev(off) if q_off is None else dev(q_off), max_rows=max_rows)
        return score, int(bad)

    good, b = run(lens, table)
    assert b == 0
    s, b = run([300, 999], table)
    assert b == 1 and torch.equal(s, good)
    s, b = run([300, -3], table)
    assert b == 1 and torch.equal(s[0], good[0]) and bool((s[1] == 1).all())
    holes = table.copy()
    holes[1, 1], holes[1, 2], holes[1, 9] = -1, pool[0].shape[0], 2 ** 30
    s, b = run(lens, holes)
    assert b == 1 and bool((s[1, :, 16:48] == 1).all()) and bool((s[1, :, 144:160] == 1).all())
    for a, e in ((0, 16), (48, 144), (160, 300)):
        assert torch.equal(s[1, :, a:e], good[1, :, a:e])
    assert torch.equal(s[0], good[0])
    s, b = run(lens, table, q_off=[0, rows, 3 * rows])
    assert b == 1 and torch.equal(s[0], good[0])
    s, b = run(lens, table, T=rows)            # request 1's rows lie outside: it is left as it was
    assert b == 1 and torch.equal(s[0], good[0]) and bool((s[1] == 1).all())
    # more rows than the bound: the first of them alone, at their own positions
    s, b = run(lens, table, max_rows=20)
    want, tol = sref.score(pool, q[:20], lse[:20], [0, 20], [288], table[:1], torch.ones((1, 2, 300), device="cuda"), 1.0, 0.125)
    assert b == 1 and float(((s[0, :, :268].double() - want[0, :, :268]).abs() - tol[0, :, :268]).max()) <= 0
    assert float(((s[0, :, 268:288].double() - want[0, :, 268:288]).abs() - tol[0, :, 268:288]).max()) <= 0
    assert bool((s[0, :, 288:] == 0).all())


def test_strided_rows_on_a_stream_of_their_own():
    lens = [150, 140]
    pool, table, q, off = case(lens, [20, 30], 2, 6, 128, 16, "e4m3", "f16", wide=True)
    assert q.stride(0) == 2 * q.shape[1] * q.shape[2]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        check(pool, table, q, off, lens, decay=0.5, softcap=30.0)
    torch.cuda.current_stream().wait_stream(side)


def test_the_same_step_by_both_kernels():
    """The rows of a chunk in one call (tensor cores), and one row a call, whose weights add up to the same."""
    L, rows, scale = 200, 40, 128 ** -0.5
    pool, table, q, off = case([L], [rows], 2, 4, 128, 32, "int8", "f32")
    lse = lse_of(pool, q, off, [L], table, scale)
    want, tol = sref.score(pool, q, lse, off, [L], table, torch.zeros((1, 2, L), device="cuda"), 1.0, scale)
    one = torch.zeros((1, 2, L), device="cuda")
    for i in range(rows):
        n = L - rows + i + 1
        ddl.ddl_kv8_score(pool, q[i:i + 1], lse[i:i + 1], dev([n]), dev(table), L, one, scale=scale)
    many = torch.zeros_like(one)
    ddl.ddl_kv8_score(pool, q, lse, dev([L]), dev(table), L, many, q_off=dev(off), max_rows=rows, scale=scale)
    for got, more in ((one, rows * 2.0 ** -23), (many, 0.0)):  # (row by row: a rounding of the sum each)
        assert float(((got.double() - want).abs() - tol - want * more).max()) <= 0
