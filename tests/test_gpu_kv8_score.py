"""Attention weight drawn by cached tokens (ddl_kv8_score) against a 64-bit
reference, where masks, lengths, placements and types can go wrong."""
import ctypes
import math
import threading

import numpy as np
import pytest
import torch

import kv8_reference as ref
import serving_reference as sref
from memory_bound_transformer_decode_gb300 import ddl
from test_gpu_kv8 import CODES, DTYPES, dev, make_pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ddl.load(build_if_missing=True)


def case(lens, rows, H, G, hd, page, codes, dtype, seed=0, tame=True, wide=False):
    """Pool, table, q, q_off, kv_len and the 64-bit lse's inputs of a step; rows: per request."""
    rng = np.random.RandomState(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [max(1, -(-n // page)) for n in lens]
    pages = sum(need) + 2
    pool = make_pool(pages, H, page, hd, codes, seed)
    if tame:  # keys of about N(0, 1), so that many tokens have weight
        for i in (2, 3):
            pool[i].fill_(2.0 ** (-9 if codes == "e4m3" else -7))
    ids = rng.permutation(pages)
    table = np.full((len(lens), max(need) + 1), -5, np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += n
    off = np.concatenate([[0], np.cumsum(rows)])
    T = int(off[-1])
    q = torch.randn((T, H * G * (2 if wide else 1), hd), generator=g, device="cuda").to(DTYPES[dtype])[:, :H * G]
    return pool, table, q, off


def lse_of(pool, q, off, lens, table, scale, **opts):
    lse = ref.attention(pool, q, off, lens, table, scale, **opts)[1]
    return lse.float().nan_to_num(nan=0.0, neginf=-math.inf, posinf=math.inf).contiguous()


def check(pool, table, q, off, lens, decay=1.0, scale=None, one_row=None, max_len=None, extra=5, seed=1, stream=None, **opts):
    H, hd = pool[0].shape[1], q.shape[2]
    scale = 1.0 / math.sqrt(hd) if scale is None else scale
    lse = lse_of(pool, q, off, lens, table, scale, **opts)
    R, most = len(lens), max(max(lens), 1)
    max_len = most if max_len is None else max_len
    g = torch.Generator(device="cuda").manual_seed(seed)
    old = torch.exp(2 * torch.randn((R, H, max_len + extra), generator=g, device="cuda"))
    want, tol = sref.score(pool, q, lse, off, lens, table, old, decay, scale, **opts)
    rows = int(np.diff(off).max())
    one_row = (np.diff(off) == 1).all() if one_row is None else one_row
    got = old.clone()
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dict(q_off=None if one_row else dev(off), max_rows=max(rows, 1), decay=decay, scale=scale, bad=bad, **opts)
    ddl.ddl_kv8_score(pool, q, lse, dev(lens), dev(table), max_len, got, **args)
    torch.cuda.synchronize()
    assert int(bad) == 0
    far = (got.double() - want).abs() - tol
    assert not torch.isnan(far).any() and float(far.max()) <= 0, (float(far.max()), torch.nonzero(far > 0)[:5])
    for r, n in enumerate(lens):  # what lies behind the tokens is as it was
        assert torch.equal(got[r, :, n:], old[r, :, n:])
    again = old.clone()
    ddl.ddl_kv8_score(pool, q, lse, dev(lens), dev(table), max_len, again, **args)
    assert torch.equal(got, again)
    return got, old


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("hd,H,G,page", [(64, 2, 4, 16), (128, 3, 7, 64), (128, 8, 8, 256), (64, 1, 1, 32)])
def test_one_row(codes, dtype, hd, H, G, page):
    lens = [1, 15, 16, 17, 700, 129, 257, 2]
    check(*case(lens, [1] * 8, H, G, hd, page, codes, dtype, seed=hd + G), lens, decay=0.9)


@pytest.mark.parametrize("codes,dtype,hd", [("e4m3", "bf16", 128), ("int8", "f32", 128), ("e4m3", "f32", 64), ("int8", "f16", 64)])
@pytest.mark.parametrize("rows", [[2, 1, 0, 3], [9, 8, 1, 7], [64, 33, 0, 17]])
def test_several_rows(codes, dtype, hd, rows):
    lens = [300, 40, 77, 1000]
    for G in (1, 3, 8):
        check(*case(lens, rows, 2, G, hd, 32, codes, dtype, seed=G), lens)


@pytest.mark.parametrize("rows", [[1, 1, 1], [5, 4, 1]])
@pytest.mark.parametrize("opts", [dict(softcap=20.0), dict(window=33), dict(slopes=True), dict(window=1),
                                  dict(softcap=5.0, window=100, slopes=True)])
def test_masks(rows, opts):
    lens = [90, 513, 16]
    pool, table, q, off = case(lens, rows, 2, 3, 128, 16, "e4m3", "bf16", seed=5)
    if "slopes" in opts:
        opts = dict(opts, slopes=torch.exp2(-torch.arange(1, 7, device="cuda").float()))
    check(pool, table, q, off, lens, decay=0.5, **opts)
    check(pool, table, q, off, lens, decay=1.0, **opts)


def test_more_rows_than_tokens_and_rows_strided():
    lens = [3, 0, 5]
    pool, table, q, off = case(lens, [6, 2, 5], 2, 4, 64, 16, "int8", "bf16", wide=True)
    assert q.stride(0) != q.shape[1] * q.shape[2]
    check(pool, table, q, off, lens)


def test_decay_zero_reads_nothing_and_new_tokens_begin_at_zero():
    lens = [100, 64]
    pool, table, q, off = case(lens, [1, 1], 2, 4, 128, 16, "e4m3", "bf16")
    lse = lse_of(pool, q, off, lens, table, 128 ** -0.5)
    score = torch.full((2, 2, 100), math.nan, device="cuda")
    ddl.ddl_kv8_score(pool, q, lse, dev(lens), dev(table), 100, score, decay=0.0)
    assert torch.isfinite(score[0]).all() and torch.isfinite(score[1, :, :64]).all() and score[1, :, 64:].isnan().all()
    # each query head's weights sum to 1: a group's to 4
    assert torch.allclose(score[0].sum(-1), torch.full((2,), 4.0, device="cuda"), rtol=1e-4)
    score = torch.full((2, 2, 100), 7.0, device="cuda")
    score[0, :, 99] = math.nan
    ddl.ddl_kv8_score(pool, q, lse, dev(lens), dev(table), 100, score)
    assert torch.isfinite(score).all() and float(score[0, :, 99].max()) <= 4.001


def test_nan_and_infinite_lse_stay_with_the_keys_concerned():
    lens = [40, 40]
    pool, table, q, off = case(lens, [2, 2], 1, 2, 64, 16, "e4m3", "f16")
    lse = lse_of(pool, q, off, lens, table, 0.125)
    want, _ = check(pool, table, q, off, lens, scale=0.125)
    lse[0] = -math.inf   # row 0 of request 0: no keys
    lse[2, 0] = math.nan  # row 0 of request 1 sees tokens 0 .. 38
    score = torch.ones((2, 1, 40), device="cuda")
    ddl.ddl_kv8_score(pool, q, lse, dev(lens), dev(table), 40, score, q_off=dev(off), max_rows=2, scale=0.125)
    assert torch.isfinite(score[0]).all() and score[1, 0, :39].isnan().all() and torch.isfinite(score[1, 0, 39])
    assert float(score[0].sum()) == pytest.approx(38 + 2, rel=1e-4)  # 38 old tokens of 1, row 1's two heads


def test_junk_codes_and_scales_outside_the_tokens_have_no_effect():
    lens = [37]
    pool, table, q, off = case(lens, [1], 2, 8, 128, 64, "e4m3", "bf16")
    a, _ = check(pool, table, q, off, lens, window=20)
    page = table[0, 0]
    raw = pool[0].view(torch.uint8)
    raw[page, :, 37:] = 127
    raw[page, :, :16] = 127         # whole blocks before the window
    pool[2][page, :, 3:] = math.inf  # blocks behind the last token
    pool[2][page, :, 0] = math.nan
    raw[page, :, 16] = 127          # a token before the window, in a block with tokens inside
    b, _ = check(pool, table, q, off, lens, window=20)
    assert torch.equal(a, b)
    raw[page, :, 30] = 127           # a seen token: NaN for it alone (lse is given)
    lse = torch.zeros((1, 16), device="cuda")
    score = torch.zeros((1, 2, 37), device="cuda")
    ddl.ddl_kv8_score(pool, q, lse, dev(lens), dev(table), 37, score, window=20)
    assert score[0, :, 30].isnan().all() and int(score.isnan().sum()) == 2


def test_bounds_of_the_launch():
    """Lengths, rows and pages outside the call's bounds are reported and computed on what lies inside."""
    lens = [64, 64]
    pool, table, q, off = case(lens, [1, 1], 2, 2, 64, 16, "int8", "bf16")
    lse = lse_of(pool, q, off, lens, table, 0.125)

    def run(kv_len, tab, max_len, T=2, q_off=None, max_rows=1):
        bad = torch.zeros(1, dtype=torch.int32, device="cuda")
        score = torch.ones((2, 2, 64), device="cuda")
        ddl.ddl_kv8_score(pool, q[:T], lse[:T], dev(kv_len), dev(tab), max_len, score, bad=bad, scale=0.125, q_off=q_off,
                          max_rows=max_rows)
        return score, int(bad)

    good, b = run(lens, table, 64)
    assert b == 0
    s, b = run([64, 999], table, 64)
    assert b == 1 and torch.equal(s, good)
    s, b = run([64, -3], table, 64)
    assert b == 1 and torch.equal(s[0], good[0]) and bool((s[1] == 1).all())
    holes = table.copy()
    holes[1, 1], holes[1, 2] = -1, pool[0].shape[0]
    s, b = run(lens, holes, 64)
    assert b == 1 and bool((s[1, :, 16:48] == 1).all())
    assert torch.equal(s[1, :, :16], good[1, :, :16]) and torch.equal(s[0], good[0])
    s, b = run(lens, table, 64, q_off=dev([0, 1, 7]), max_rows=4)
    assert b == 1 and torch.equal(s[0], good[0])


def test_a_request_without_rows_is_left_alone():
    lens = [50, 50, 50]
    pool, table, q, off = case(lens, [1, 0, 1], 2, 2, 64, 16, "e4m3", "bf16")
    got, old = check(pool, table, q, off, lens, decay=0.25)
    assert torch.equal(got[1], old[1])


def test_after_the_attention_on_a_stream_and_replayed():
    """Attention and scores in one captured step; a replay with other lengths."""
    lens = [300, 45]
    pool, table, q, off = case(lens, [1, 1], 4, 8, 128, 64, "e4m3", "bf16")
    kv_len, tab = dev(lens), dev(table)
    lse, out = torch.zeros((2, 32), device="cuda"), torch.zeros_like(q)
    ws = torch.empty(ddl.ddl_kv8_attention_workspace_bytes(32, 4, 128, 2, 2, 1, 320), dtype=torch.uint8, device="cuda")
    score = torch.zeros((2, 4, 320), device="cuda")

    def step():
        ddl.ddl_kv8_attention(pool, q, kv_len, tab, 320, out=out, lse=lse, workspace=ws)
        ddl.ddl_kv8_score(pool, q, lse, kv_len, tab, 320, score)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        score.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    graph.replay()
    kv_len.copy_(dev([299, 7]))
    score.zero_()
    graph.replay()
    torch.cuda.synchronize()
    want, tol = sref.score(pool, q, lse, off, [299, 7], table, torch.zeros_like(score), 1.0, 128 ** -0.5)
    assert float(((score.double() - want).abs() - tol).max()) <= 0
    assert torch.allclose(score[0].sum(-1), torch.full((4,), 8.0, device="cuda"), rtol=1e-4)


def test_a_long_cache():
    lens = [33000]
    check(*case(lens, [1], 2, 8, 128, 256, "int8", "f32"), lens, decay=0.99)


def test_no_scores_past_32_bits():
    """Rows of score and pages whose offsets pass 2^31 elements and 2^32 bytes."""
    H, S = 8, 2 ** 20
    R = 2 ** 31 // (H * S) + 2  # entries past 2^31
    page, hd = 2 ** 14, 128
    lens = [20] * R
    pool = make_pool(R, 1, 16, hd, "int8")
    del pool
    pages = 2 ** 32 // (H * page * hd) + 2
    raw = torch.zeros((pages, H, page, hd), dtype=torch.int8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    raw[-1, :, :32] = torch.randint(-127, 128, (H, 32, hd), generator=g, device="cuda", dtype=torch.int8)
    sc = torch.full((pages, H, page // 16), 2.0 ** -7, device="cuda")
    pool = (raw, raw, sc, sc)
    table = np.full((R, 1), pages - 1, np.int32)
    q = torch.randn((R, 8, hd), generator=g, device="cuda").bfloat16()
    off = np.arange(R + 1)
    lse = lse_of(pool, q, off, lens, table, 0.1)
    score = torch.zeros((R, H, S), device="cuda")
    ddl.ddl_kv8_score(pool, q, lse, dev(lens), dev(table), S, score, scale=0.1)
    small = torch.zeros((R, H, 20), device="cuda")
    want, tol = sref.score(pool, q, lse, off, lens, table, small, 1.0, 0.1)
    assert float(((score[..., :20].double() - want).abs() - tol).max()) <= 0
    assert float(score[-1, :, 20:].abs().max()) == 0


@pytest.mark.parametrize("dtype,rows", [("bf16", (2, 8)), ("f32", (2, 4)), ("bf16", (9, 64)), ("f32", (5, 32))])
def test_two_host_threads_with_other_numbers_of_rows(dtype, rows):
    """Calls of one kernel with unlike sizes of shared memory, from threads that do not wait for one another, are all
    launched and give what each gives alone."""
    lens, H, G, hd = [200], 1, 8, 128
    cases, lib = [], ddl.load()
    for n in rows:
        pool, table, q, off = case(lens, [n], H, G, hd, 16, "e4m3", dtype, seed=n)
        lse = lse_of(pool, q, off, lens, table, hd ** -0.5)
        keep = dict(pool=pool, q=q, lse=lse, off=dev(off), lens=dev(lens), table=dev(table), n=n)
        keep["kv"] = ddl._kv8(pool, 0, H, hd)
        keep["opts"] = ddl.AttnOpts(hd ** -0.5, 0.0, 0, None)
        cases.append(keep)
    wrong = []

    def call(c, score, stream):
        return lib.ddl_kv8_score(ctypes.byref(c["kv"]), H * G, H, hd, {"f32": 0, "bf16": 1}[dtype], ctypes.byref(c["opts"]),
                                 1, c["n"], c["n"], 200, c["off"].data_ptr(), c["lens"].data_ptr(), c["table"].data_ptr(),
                                 c["table"].shape[1], c["q"].data_ptr(), H * G * hd, c["lse"].data_ptr(), 0.0,
                                 score.data_ptr(), 200, None, stream.cuda_stream)

    torch.cuda.synchronize()
    alone = [torch.zeros((1, H, 200), device="cuda") for _ in cases]
    for c, s in zip(cases, alone):
        assert call(c, s, torch.cuda.current_stream()) == 0
    torch.cuda.synchronize()
    many = [torch.zeros((1, H, 200), device="cuda") for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]

    def loop(i):
        for _ in range(3000):
            st = call(cases[i], many[i], streams[i])
            if st:
                wrong.append((i, st, lib.ddl_last_cuda_error()))
                return

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong, wrong
    assert all(torch.equal(a, b) for a, b in zip(alone, many))


@pytest.mark.parametrize("dtype,rows", [("bf16", 1), ("f32", 3), ("f16", 8), ("bf16", 20), ("f32", 40)])
@pytest.mark.parametrize("opts", [dict(), dict(softcap=15.0)])
def test_rows_of_minus_infinite_lse_add_nothing_whatever_they_see(dtype, rows, opts):
    """Not even NaN: of codes and scales among their keys, or of their own q.  (One tile of queries, a few, many.)"""
    lens, H, G, hd, scale = [200, 200], 2, 4, 128, 128 ** -0.5
    pool, table, q, off = case(lens, [rows, rows], H, G, hd, 16, "e4m3", dtype, seed=rows)
    lse = lse_of(pool, q, off, lens, table, scale, **opts)
    last = 2 * rows - 1
    lse[:rows] = -math.inf                 # request 0: no row adds anything
    q[0] = math.nan
    lse[last, :G] = -math.inf              # request 1: the newest row's heads of K/V head 0
    clean = [t.clone() for t in pool]
    old = torch.rand((2, H, 200), device="cuda")
    want, tol = sref.score(clean, q.nan_to_num(nan=0.0), lse, off, lens, table, old, 0.5, scale, **opts)
    raw = pool[0].view(torch.uint8)
    raw[table[0, 3]] = 127
    pool[2][table[0, 5]] = math.inf
    pool[2][table[0, 6]] = math.nan
    if rows == 1:                          # (else other rows see it)
        raw[table[1, 4], 0, 7] = 255
    got = old.clone()
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    ddl.ddl_kv8_score(pool, q, lse, dev(lens), dev(table), 200, got, q_off=dev(off), max_rows=rows, decay=0.5, scale=scale,
                      bad=bad, **opts)
    assert int(bad) == 0 and float(((got.double() - want).abs() - tol).max()) <= 0
    assert torch.equal(got[0, :, :200 - rows], 0.5 * old[0, :, :200 - rows])
    if rows > 1:                           # a token that a row with weights sees
        raw[table[1, 4], 0, 7] = 255
        ddl.ddl_kv8_score(pool, q, lse, dev(lens), dev(table), 200, got, q_off=dev(off), max_rows=rows, decay=0.0, scale=scale,
                          **opts)
        assert got[1, 0, 71].isnan() and int(got.isnan().sum()) == 1


@pytest.mark.parametrize("rows", [1, 9])
def test_a_request_as_long_as_32_bits_allow(rows):
    """Every page of it the same one, by one tile of queries and by many (tiles of 128 tokens: the last one ends at 2^31)."""
    page, hd, H, G = 16, 64, 1, 8
    per = 2 ** 27 - 1
    L = per * page
    pool = make_pool(2, H, page, hd, "int8", 3)
    pool[2].fill_(2.0 ** -8)
    table = torch.ones((1, per), dtype=torch.int32, device="cuda")
    q = torch.randn((rows, G, hd), generator=torch.Generator(device="cuda").manual_seed(rows), device="cuda").bfloat16()
    lse = torch.zeros((rows, G), device="cuda")
    score = torch.full((1, H, L), -1.0, device="cuda")
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    ddl.ddl_kv8_score(pool, q, lse, dev([L]), table, L, score, q_off=dev([0, rows]), max_rows=rows, decay=0.0, scale=0.1, bad=bad)
    torch.cuda.synchronize()
    # the same keys in a request of four pages: its last page is that of this one, the others all alike
    small = torch.zeros((1, H, 64), device="cuda")
    want, tol = sref.score(pool, q, lse, [0, rows], [64], np.ones((1, 4), int), small, 0.0, 0.1)
    assert int(bad) == 0
    got = score.view(-1, page)
    assert bool((got[:-1] == got[0]).all())
    assert float(((got[0].double() - want[0, 0, :page]).abs() - tol[0, 0, :page]).max()) <= 0
    assert float(((got[-1].double() - want[0, 0, -page:]).abs() - tol[0, 0, -page:]).max()) <= 0
