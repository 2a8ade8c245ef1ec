"""The 8-bit paged KV cache on the GPU: page plans, quantizing appends and
attention against 64-bit references, at the sizes, masks and placements where
they can go wrong, and a serving loop of the three.
"""
import math

import numpy as np
import pytest
import torch

import kv8_reference as ref
from memory_bound_transformer_decode_gb300 import ddl

pytestmark = pytest.mark.gpu

CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ddl.load(build_if_missing=True)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


# ------------------------------------------------------------------ plan

def run_plan(old, add, free, table, page, T):
    R = len(old)
    t = {n: torch.full((k,), -7, dtype=torch.int32, device="cuda")
         for n, k in (("row_off", R + 1), ("kv_len", R), ("row_pos", T), ("slot", T), ("used", 1), ("status", R))}
    tab = dev(table)
    ddl.ddl_page_plan(dev(old), dev(add), dev(free), tab, page, **t)
    return [x.cpu().numpy() for x in (tab, t["row_off"], t["kv_len"], t["row_pos"], t["slot"], t["used"],
                                      t["status"])]


def check_plan(old, add, free, table, page, T):
    got, want = run_plan(old, add, free, table, page, T), ref.plan(old, add, free, table, page, T)
    for name, g, w in zip(("table", "row_off", "kv_len", "row_pos", "slot", "used", "status"), got, want):
        assert np.array_equal(g, w), name
    return want


@pytest.mark.parametrize("R", [1, 2, 31, 128, 129, 1000, 4096])
@pytest.mark.parametrize("page,most_add", [(16, 1), (64, 40), (256, 700)])
def test_plan(R, page, most_add):
    g = np.random.RandomState(R + page)
    per = 9
    old, add = g.randint(0, per * page, R), g.randint(0, most_add + 1, R)
    old[g.rand(R) < 0.2] = 0
    add[g.rand(R) < 0.2] = 0
    held = -(-old // page)
    ids = g.permutation(R * per + 3 * R + 8)
    table = np.where(np.arange(per)[None] < held[:, None], ids[:R * per].reshape(R, per), -1)
    free = ids[R * per:]
    if R > 2:  # bad lengths among them
        old[1], add[2] = -3, -1
    T = int(np.maximum(add, 0).sum()) + 5
    st = check_plan(old, add, free, table, page, T)[6]
    assert R == 1 or (st == 0).any()
    check_plan(old, add, free[:len(free) // 9], table, page, T)  # pages run out
    check_plan(old, add, free, table, page, T // 2)              # rows run out
    check_plan(old, add, free[:len(free) // 9], table, page, T // 3)


def test_plan_edges():
    table = np.full((3, 2), 9)
    z = np.zeros(0, int)
    check_plan([0, 5, 16], [0, 0, 0], z, table, 16, 0)               # nothing to do
    check_plan([0, 5, 16], [3, 1, 1], z, table, 16, 9)               # no free page: only the row that needs none
    check_plan([15, 16, 31], [1, 1, 1], [4, 5, 6], table, 16, 3)     # exact page ends, a full table row
    check_plan([32, 31, 33], [0, 2, 0], [4, 5, 6], table, 16, 3)     # past the table row
    check_plan([2 ** 31 - 1, 0, 0], [2 ** 31 - 1, 32, 33], [4, 5, 6], table, 16, 40)  # sums past 32 bits
    check_plan([0, 0, 0], [20, 20, 1], [4, 5, 6], table, 16, 21)     # a later small request does not overtake
    check_plan([0] * 4, [2 ** 20] * 4, np.arange(70000), np.full((4, 65536), -1), 64, 2 ** 20 + 7)


# ------------------------------------------------------------------ append

def make_pool(pages, H, page, hd, codes, seed=0, junk=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in range(2):
        raw = torch.randint(0, 256, (pages, H, page, hd), generator=g, device="cuda", dtype=torch.uint8)
        if codes == "int8":
            raw = torch.where(raw == 128, 0, raw)
        elif not junk:
            raw = torch.where((raw & 127) == 127, 0, raw)
        sc = torch.exp2(torch.randint(-9, -4, (pages, H, page // 16), generator=g, device="cuda").float())
        out.append((raw.view(CODES[codes]), sc))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def check_append(pool, k_new, v_new, slot, bad=None):
    page, int8 = pool[0].shape[2], pool[0].dtype == torch.int8
    before = [t.view(torch.uint8).cpu().numpy() if t.element_size() == 1 else t.cpu().numpy() for t in pool]
    ddl.ddl_kv8_append(pool, k_new, v_new, dev(slot), bad=bad)
    torch.cuda.synchronize()
    for i, x in ((0, k_new), (1, v_new)):
        codes, scale = ref.append(before[i], before[i + 2], x.double().cpu().numpy(), slot, page, int8)
        assert np.array_equal(pool[i + 2].cpu().numpy().astype(np.float64), scale)
        got = pool[i].view(torch.uint8).cpu().numpy()
        a, b = ref.decode(got, int8), ref.decode(codes, int8)
        assert np.array_equal(a, b, equal_nan=True)


def rows(T, H, hd, dtype, seed, mag=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    m = torch.exp2(torch.randint(-3, 4, (T, H, 1), generator=g, device="cuda").float()) * mag
    kv = (torch.randn((T, 2 * H, hd), generator=g, device="cuda") * torch.cat([m, m], 1)).to(DTYPES[dtype])
    return kv[:, :H], kv[:, H:]  # rows wider than the heads


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("hd,H", [(64, 3), (128, 1), (128, 8)])
def test_append_decode_rows(codes, dtype, hd, H):
    """One row for each of several sequences, every place in a block, growing scales."""
    pool = make_pool(40, H, 32, hd, codes, seed=hd + H)
    g = np.random.RandomState(3)
    blocks = g.permutation(80)[:48]
    for step, mag in enumerate((0.02, 1.0, 30.0)):
        slot = blocks * 16 + (np.arange(48) + step) % 16
        k, v = rows(48, H, hd, dtype, 11 + step, mag)
        check_append(pool, k, v, slot)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype,hd,H,page", [("bf16", 128, 2, 16), ("f32", 64, 4, 64), ("f16", 128, 3, 256)])
@pytest.mark.parametrize("start,T", [(0, 1), (5, 16), (15, 2), (3, 255), (0, 257), (9, 700)])
def test_append_prompt_rows(codes, dtype, hd, H, page, start, T):
    pages = -(-(start + T) // page) + 3
    pool = make_pool(pages, H, page, hd, codes, seed=T)
    table = np.random.RandomState(T).permutation(pages)
    pos = np.arange(start, start + T)
    k, v = rows(T, H, hd, dtype, T)
    check_append(pool, k, v, table[pos // page] * page + pos % page)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
def test_append_odd_values_and_slots(codes):
    H, hd, page = 2, 64, 32
    for dtype in ("f32", "bf16", "f16"):
        pool = make_pool(8, H, page, hd, codes, seed=5)
        k, v = (x.clone() for x in rows(40, H, hd, dtype, 9))
        k[3] = 0                                 # a block of zeros
        v[4, 0, 7], v[4, 1, 9] = math.inf, -math.inf
        k[5, 0, 1], k[5, 1] = math.nan, math.nan
        v[6] = torch.finfo(v.dtype).tiny         # the smallest normal values
        k[7] = torch.finfo(k.dtype).max
        k[8] *= 0 if dtype == "f16" else 1e-38
        slot = np.full(40, -1)
        slot[3], slot[4], slot[5], slot[6], slot[7], slot[8] = 16, 33, 64 + 5, 96, 112, 128 + 1
        slot[10:13] = [200, 201, 201]            # a slot twice in a run: the last row counts
        slot[13:17] = [214, 210, 212, 211]       # a run out of order
        slot[20], slot[21] = 8 * page, 2 ** 31 - 1
        slot[30:36] = np.arange(140, 146)        # over a block's end
        bad = torch.zeros(1, dtype=torch.int32, device="cuda")
        check_append(pool, k, v, slot, bad)
        assert int(bad) == 1
        bad.zero_()
        slot[20:22] = -1
        check_append(pool, k, v, slot, bad)
        assert int(bad) == 0


def test_append_long_run_of_one_slot():
    """More rows than a block has tokens, all in one block."""
    pool = make_pool(2, 2, 16, 128, "e4m3", seed=1)
    k, v = rows(70, 2, 128, "f32", 4)
    slot = np.concatenate([np.full(33, 3), np.arange(3, 16), np.full(24, 9)])
    check_append(pool, k, v, slot)
    assert not pool[0].float().isnan().any()


@pytest.mark.parametrize("T", [60, 1500])
@pytest.mark.parametrize("H", [1, 3, 8])
def test_append_blocks_met_again(T, H):
    """A page that two requests write to: separate runs of one block, in map order."""
    pool = make_pool(30, H, 32, 64, "e4m3", seed=T)
    slot = np.random.RandomState(H).randint(-40, 30 * 32, T)
    slot[T // 2:T // 2 + 20] = np.arange(100, 120)
    slot[T // 2 + 25:T // 2 + 30] = np.arange(98, 103)
    k, v = rows(T, H, 64, "bf16", 5, 4.0)
    check_append(pool, k, v, np.maximum(slot, -1))


@pytest.mark.parametrize("T", [256, 257, 512, 513, 4096, 4097, 9001])
@pytest.mark.parametrize("H,dtype", [(1, "f32"), (4, "bf16")])
def test_append_decode_rows_and_prompts_in_one_map(T, H, dtype):
    """Rows of many requests, most of them one and some up to 100, from any place of a block on, padding between."""
    g = np.random.RandomState(T)
    slot, block = [], 0
    while len(slot) < T:
        n, at = (1 if g.rand() < 0.8 else g.randint(1, 101)), g.randint(16)
        slot += [block * 16 + at + i for i in range(n)] + [-1] * (g.rand() < 0.1)
        block += (at + n + 15) // 16 + g.randint(2)
    pages = block // 2 + 2
    slot = np.array(slot[:T])
    slot = np.where(slot >= 0, g.permutation(2 * pages)[np.maximum(slot, 0) // 16] * 16 + slot % 16, -1)
    pool = make_pool(pages, H, 32, 64, "e4m3", seed=T)
    k, v = rows(T, H, 64, dtype, 5, 4.0)
    check_append(pool, k, v, slot)


def test_append_scale_steps_are_exact():
    """amax just at and past the largest code's multiples; ties of the rounding."""
    for codes, top in (("e4m3", 448.0), ("int8", 127.0)):
        pool = make_pool(4, 1, 16, 64, codes, seed=2)
        k = torch.zeros(4, 1, 64, device="cuda")
        k[0, 0, 0], k[1, 0, 0] = top * 2.0 ** -5, float(np.nextafter(np.float32(top * 2.0 ** -5), np.float32(1e9)))
        k[2, 0, :] = torch.arange(64, device="cuda") * 0.5 + 0.5   # ties of int8 (scale 2^-1) among them
        k[2, 0, 63] = top / 2
        k[3, 0, :] = (1 + torch.arange(64, device="cuda") / 16) * 2.0 ** -8
        check_append(pool, k, -k, np.array([0, 16, 32, 48]))


# ------------------------------------------------------------------ attention

def setup(R, n_rows, H_q, H_kv, hd, page, lens, codes, dtype, seed=0, spare=3, junk=True):
    """A pool whose pages hold random codes (slots behind the sequences and
    spare pages NaN codes where the type has them), q and the table."""
    lens, n_rows = np.asarray(lens), np.asarray(n_rows)
    g = np.random.RandomState(seed)
    need = -(-lens // page)
    per = int(max(1, need.max())) + 2
    pages = int(need.sum()) + spare
    pool = make_pool(pages, H_kv, page, hd, codes, seed)
    ids = g.permutation(pages)
    table = np.full((R, per), 2 ** 31 - 1)
    at = 0
    for r in range(R):
        table[r, :need[r]] = ids[at:at + need[r]]
        at += need[r]
    if junk and codes == "e4m3":
        for t in pool[:2]:
            raw = t.view(torch.uint8)
            raw[torch.from_numpy(ids[at:]).cuda()] = 127
            for r in range(R):
                if lens[r] % page:
                    raw[int(table[r, need[r] - 1]), :, int(lens[r] % page):] = 255
    q_off = np.concatenate([[0], np.cumsum(n_rows)])
    gg = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = (torch.randn((int(q_off[-1]), H_q, hd), generator=gg, device="cuda") * 0.5).to(DTYPES[dtype])
    return pool, q, q_off, lens, table


def check_attention(pool, q, q_off, lens, table, *, rows_given=None, max_len=None, expect_bad=0, **opts):
    R, (T, H_q, hd) = len(lens), q.shape
    n = np.diff(q_off)
    many = bool((n != 1).any()) if rows_given is None else rows_given
    out = torch.full_like(q, 7.0)
    lse = torch.full((T, H_q), 7.0, device="cuda")
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    scale = opts.pop("scale", 1 / math.sqrt(hd))
    for rep in range(2):  # the second run has to give the same bits
        got = ddl.ddl_kv8_attention(pool, q, dev(lens), dev(table), int(max_len or max(1, lens.max())),
                                    q_off=dev(q_off) if many else None, max_rows=int(max(1, n.max())) if many else 1,
                                    scale=scale, out=out if rep == 0 else torch.full_like(q, 7.0),
                                    lse=lse if rep == 0 else None, bad=bad, **opts)
        torch.cuda.synchronize()
        if rep:
            assert torch.equal(got.view(torch.uint8), out.view(torch.uint8))
    assert int(bad) == expect_bad
    want, want_l, tol, tol_l = ref.attention(pool, q, q_off, lens, table, scale, opts.get("softcap", 0.0),
                                             opts.get("window", 0), opts.get("slopes"))
    none = want.isnan().all(-1).all(-1)
    assert (out[none] == 7).all() and (lse[none] == 7).all()
    o, l = out.double()[~none], lse.double()[~none]
    assert not o.isnan().any()
    err = (o - want[~none]).abs() - tol[~none]
    assert (err <= 0).all(), f"out past its bound by {float(err.max()):.3g}"
    inf = want_l[~none] == -math.inf
    assert torch.equal(l == -math.inf, inf)
    assert ((l - want_l[~none]).abs()[~inf] <= tol_l[~none][~inf]).all()
    return out


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("H_q,H_kv,hd", [(8, 2, 64), (28, 4, 128), (16, 2, 128), (3, 3, 64), (5, 1, 128)])
def test_attention_decode(codes, dtype, H_q, H_kv, hd):
    lens = [1, 0, 15, 16, 17, 33, 129, 700, 64, 2]
    check_attention(*setup(10, [1] * 10, H_q, H_kv, hd, 32, lens, codes, dtype, seed=H_q))


@pytest.mark.parametrize("codes,dtype", [("e4m3", "bf16"), ("int8", "f32"), ("e4m3", "f32")])
@pytest.mark.parametrize("H_q,H_kv,hd,page", [(8, 1, 128, 16), (6, 2, 64, 64), (7, 1, 128, 256)])
@pytest.mark.parametrize("n_rows", [[2, 1, 0, 3], [9, 64, 17, 1], [64, 64, 64, 64]])
def test_attention_rows(codes, dtype, H_q, H_kv, hd, page, n_rows):
    """Several rows of a request, causal among themselves; a request without rows; more rows than tokens."""
    lens = [130, 64, 40, 1000]
    check_attention(*setup(4, n_rows, H_q, H_kv, hd, page, lens, codes, dtype, seed=3), rows_given=True)


@pytest.mark.parametrize("codes,dtype", [("e4m3", "f32"), ("int8", "bf16")])
@pytest.mark.parametrize("opts", [dict(softcap=30.0), dict(softcap=2.0, scale=0.7), dict(window=1), dict(window=40),
                                  dict(window=5000), dict(slopes=True), dict(scale=-0.3),
                                  dict(softcap=5.0, window=77, slopes=True), dict(scale=0.0)])
@pytest.mark.parametrize("n_rows", [[1] * 5, [4, 1, 33, 2, 0]])
def test_attention_options(codes, dtype, opts, n_rows):
    opts = dict(opts)
    if opts.get("slopes"):
        opts["slopes"] = torch.exp2(-torch.arange(12, device="cuda").float())
    check_attention(*setup(5, n_rows, 12, 2, 128, 16, [1, 37, 300, 16, 2100], codes, dtype, seed=6),
                    rows_given=True, **opts)


@pytest.mark.parametrize("R,L", [(1, 8193), (1, 33000), (3, 5000), (64, 1500), (300, 90)])
def test_attention_long_and_wide(R, L):
    lens = np.random.RandomState(L).randint(1, L + 1, R)
    lens[0] = L
    check_attention(*setup(R, [1] * R, 16, 2, 128, 64, lens, "e4m3", "f32", seed=R))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n_rows,opts", [([1] * 7, {}), ([1] * 7, dict(window=33, slopes=True)),
                                         ([4, 0, 1, 64, 3, 17, 2], {}),
                                         ([1, 33, 2, 9, 64, 0, 5], dict(softcap=4.0, window=100, slopes=True)),
                                         ([2] * 7, dict(softcap=20.0))])
@pytest.mark.parametrize("bound", [2000, 9000, 60000])
def test_attention_every_split(dtype, n_rows, opts, bound):
    """The bound on the lengths chooses kernel and split (clusters of several sizes, shares); the lengths stay
    short, empty and ragged."""
    opts = dict(opts)
    if opts.get("slopes"):
        opts["slopes"] = torch.exp2(-torch.arange(12, device="cuda").float() / 2)
    check_attention(*setup(7, n_rows, 12, 2, 128, 32, [1, 0, 40, 129, 16, 1900, 257], "e4m3", dtype, seed=12),
                    rows_given=max(n_rows) > 1, max_len=bound, **opts)


@pytest.mark.parametrize("codes,hd", [("int8", 128), ("e4m3", 64)])
@pytest.mark.parametrize("bound", [2000, 60000])
def test_attention_every_split_of_the_warp_kernel(codes, hd, bound):
    for n_rows in ([1] * 6, [3, 0, 1, 40, 2, 8]):
        check_attention(*setup(6, n_rows, 14, 2, hd, 16, [1, 0, 40, 129, 1700, 257], codes, "f32", seed=13),
                        rows_given=max(n_rows) > 1, max_len=bound)


def test_attention_one_request_in_clusters_of_every_size():
    for L, H in ((40, 1), (300, 1), (600, 2), (1100, 1), (5000, 1), (5000, 8), (20000, 4)):
        for codes in ("e4m3", "int8"):
            check_attention(*setup(1, [1], 4 * H, H, 128, 64, [L], codes, "bf16", seed=L))


@pytest.mark.parametrize("codes,dtype,hd", [("int8", "bf16", 128), ("e4m3", "f32", 64), ("int8", "f32", 128)])
@pytest.mark.parametrize("H_q,H_kv", [(32, 8), (12, 12), (18, 6), (64, 8)])
@pytest.mark.parametrize("R,most,rows", [(40, 60, 1), (150, 300, 1), (400, 16, 1), (70, 100, 3)])
def test_attention_many_short_requests(codes, dtype, hd, H_q, H_kv, R, most, rows):
    """Several K/V heads a CTA (1 to 8, by the sizes), with and without options, empty requests among them."""
    g = np.random.RandomState(R + H_q)
    n = g.randint(0, rows + 1, R) if rows > 1 else np.ones(R, int)
    s = setup(R, n, H_q, H_kv, hd, 16, g.randint(0, most + 1, R), codes, dtype, seed=R)
    check_attention(*s, max_len=most, rows_given=rows > 1)
    slopes = torch.exp2(-torch.arange(H_q, device="cuda").float() / 2)
    check_attention(*s, max_len=most, rows_given=rows > 1, window=19, slopes=slopes, softcap=9.0)


def test_attention_calls_on_three_streams_at_once():
    """Clusters, shares and many rows side by side, each with its own workspace: the bits of the calls alone."""
    cases = [(setup(1, [1], 16, 2, 128, 64, [9000], "e4m3", "f32", seed=1), 9000),
             (setup(20, [1] * 20, 32, 8, 128, 16, [40 + 90 * i for i in range(20)], "e4m3", "bf16", seed=2), 30000),
             (setup(2, [64, 33], 16, 2, 128, 32, [700, 1900], "e4m3", "bf16", seed=3), 2000)]
    calls = []
    for (pool, q, off, lens, table), bound in cases:
        kw = dict(q_off=dev(off), max_rows=int(np.diff(off).max()))
        n = ddl.ddl_kv8_attention_workspace_bytes(q.shape[1], pool[0].shape[1], 128, len(lens), q.shape[0],
                                                  kw["max_rows"], bound)
        args = (pool, q, dev(lens), dev(table), bound)
        calls.append((args, kw, torch.empty(n, dtype=torch.uint8, device="cuda"),
                      ddl.ddl_kv8_attention(*args, **kw), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for _ in range(15):
        for args, kw, ws, want, s in calls:
            outs.append((ddl.ddl_kv8_attention(*args, **kw, workspace=ws, stream=s), want))
    torch.cuda.synchronize()
    for got, want in outs:
        assert torch.equal(got, want)


def test_attention_bound_far_above_the_lengths():
    """max_len only sizes the launch."""
    s = setup(3, [1, 1, 1], 8, 2, 64, 16, [5, 100, 17], "int8", "f32")
    table = np.concatenate([s[4], np.full((3, 3000), 7)], 1)
    a = check_attention(s[0], s[1], s[2], s[3], table)
    b = check_attention(s[0], s[1], s[2], s[3], table, max_len=40000)
    assert (a - b).abs().max() < 1e-5


def test_attention_scales_of_any_size():
    """Blocks whose V scales differ by 2^20 and K scales that are no powers of two; a zero block."""
    pool, q, q_off, lens, table = setup(2, [1, 1], 8, 1, 128, 16, [200, 64], "e4m3", "f32", seed=8)
    k, v, ks, vs = pool
    n = vs.shape[0]
    vs.copy_(torch.exp2((torch.arange(n, device="cuda") % 5 * 5.0 - 18).view(n, 1, 1)))
    ks.mul_(1.2345)
    vs[int(table[0, 2])] = 0
    check_attention(pool, q, q_off, lens, table)
    vs.zero_()
    check_attention(pool, q, q_off, lens, table)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("codes,hd,H_kv,lens,bound", [
    ("e4m3", 128, 1, [200, 64], None), ("int8", 64, 1, [200, 64], None), ("e4m3", 128, 8, [4000, 300, 2100], None),
    ("int8", 128, 8, [4000, 300, 2100], 60000), ("e4m3", 128, 8, [4000, 300, 2100], 60000)])
def test_attention_smallest_v_scales(dtype, codes, hd, H_kv, lens, bound):
    """V scales at the smallest a call writes (2^-126), above it and, subnormal, below it."""
    pool, q, q_off, lens, table = setup(len(lens), [1] * len(lens), 4 * H_kv, H_kv, hd, 16, lens, codes, dtype, seed=9)
    vs = pool[3]
    small = torch.tensor([2.0 ** -126, 1.37 * 2.0 ** -125, 2.0 ** -130, 2.0 ** -119], device="cuda")
    for some in (small, small[2:3]):
        i = torch.arange(vs.numel(), device="cuda") * 7 % len(some)
        vs.copy_(some[i].view(vs.shape))
        check_attention(pool, q, q_off, lens, table, max_len=bound)


@pytest.mark.parametrize("scale", [math.inf, -math.inf, math.nan, -1.0])
@pytest.mark.parametrize("codes,hd,bound", [("e4m3", 128, 1000), ("int8", 128, 1000), ("e4m3", 64, 60000),
                                            ("e4m3", 128, 60000)])
def test_attention_bad_scale_reaches_only_the_rows_that_see_its_block(scale, codes, hd, bound):
    n, L, window = 40, 300, 64
    pool, q, q_off, lens, table = setup(2, [n, 1], 8, 1, hd, 16, [L, 90], codes, "bf16", seed=14)
    args = (q, dev(lens), dev(table), bound)
    kw = dict(q_off=dev(q_off), max_rows=n, window=window)
    want, _, tol, _ = ref.attention(pool, q, q_off, lens, table, hd ** -0.5, 0.0, window, None)
    for which in (2, 3):
        if which == 2 and scale == -1.0:
            continue  # (a factor of the scores like any other)
        for block in (12, 13, 17):  # tokens 16 b .. 16 b + 15; row i sees 197 + i .. 260 + i
            bad_pool = [t.clone() for t in pool]
            bad_pool[which][int(table[0, block]), 0, 0] = scale
            out = ddl.ddl_kv8_attention(tuple(bad_pool), *args, **kw)
            p = np.arange(L - n, L)
            sees = torch.from_numpy(np.concatenate([(p >= 16 * block) & (p - window + 1 <= 16 * block + 15), [False]]))
            assert 0 < int(sees.sum()) < n + 1
            assert out[sees.cuda()].isnan().all()
            # The others: not the clean run's bits (the running maximum and the unit of the weights' rounding
            # follow the tiles' scales, and the bad one counts as zero there), but within the same bound: it
            # holds for any running maximum, and a smaller largest V scale only lowers its floor.
            err = (out.double() - want).abs() - tol
            assert (err[~sees.cuda()] <= 0).all(), f"out past its bound by {float(err[~sees.cuda()].max()):.3g}"


def test_attention_window_as_long_as_can_be():
    s = setup(3, [4, 0, 7], 8, 2, 128, 16, [3, 20, 400], "e4m3", "bf16", seed=6)  # (a request with more rows than tokens)
    want = check_attention(*s)
    for window in (400, 401, 2 ** 31 - 1):
        assert torch.equal(check_attention(*s, window=window), want)


def test_attention_makes_its_tensors_on_the_stream_that_uses_them():
    pool, q, q_off, lens, table = setup(3, [1] * 3, 8, 2, 128, 16, [500, 40, 9], "e4m3", "bf16", seed=3)
    want = check_attention(pool, q, q_off, lens, table)
    kl, tb = dev(lens), dev(table)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # the current stream is busy: zeros made there would come too late
    out = ddl.ddl_kv8_attention(pool, q, kl, tb, 60000, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    ref_out = ddl.ddl_kv8_attention(pool, q, kl, tb, 60000)
    assert torch.equal(out, ref_out)
    assert (want.float() - out.float()).abs().max() < 0.1


def test_attention_q_of_any_size():
    s = setup(4, [1] * 4, 4, 2, 64, 16, [40, 70, 3, 100], "e4m3", "f32", seed=2)
    q = s[1]
    q[0] *= 1e30
    q[1] *= 1e-30
    q[2] = 0
    check_attention(s[0], q, *s[2:], scale=1e-30 / 8)
    q[0] *= 1e-30
    check_attention(s[0], q, *s[2:])


def test_attention_nan_reaches_only_the_rows_that_see_it():
    n, L, H_q = 6, 50, 4
    for page, where in ((16, 47), (64, 46)):
        for which in (0, 1):
            pool, q, q_off, lens, table = setup(1, [n], H_q, 1, 64, page, [L], "e4m3", "bf16", seed=4)
            clean = check_attention(pool, q, q_off, lens, table, rows_given=True)
            pool[which].view(torch.uint8)[int(table[0, where // page]), 0, where % page, 9] = 127
            out = ddl.ddl_kv8_attention(pool, q, dev(lens), dev(table), L, q_off=dev(q_off), max_rows=n)
            first = where - (L - n)
            assert torch.equal(out[:first], clean[:first])
            assert out[first:].isnan().any(-1).all()


def test_attention_strides_streams_and_spare_rows():
    pool, q, q_off, lens, table = setup(6, [1, 2, 0, 1, 5, 1], 8, 2, 128, 32, [20, 64, 9, 1, 300, 77], "e4m3", "bf16")
    want = check_attention(pool, q, q_off, lens, table, rows_given=True)
    T = q.shape[0]
    wide = torch.full((T + 4, 24, 128), 5.0, dtype=q.dtype, device="cuda")
    wide[:T, :8] = q
    wide[T:, :8] = math.nan
    out = torch.full((T + 4, 16, 128), 3.0, dtype=q.dtype, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    off, kl, tb = dev(q_off), dev(lens), dev(table)
    s.wait_stream(torch.cuda.current_stream())
    ddl.ddl_kv8_attention(pool, wide[:, :8], kl, tb, 300, q_off=off, max_rows=5, out=out[:, 8:], stream=s)
    s.synchronize()
    assert torch.equal(out[:T, 8:], want)
    assert (out[T:] == 3).all() and (out[:, :8] == 3).all()  # rows behind the last sequence, and beside the heads


def test_attention_reports_what_lies_outside():
    pool, q, q_off, lens, table = setup(3, [1] * 3, 8, 2, 64, 16, [60, 40, 33], "e4m3", "f32", junk=False)
    call = lambda **k: ddl.ddl_kv8_attention(  # noqa: E731
        pool, q, dev(k.get("lens", lens)), dev(k.get("table", table)), k.get("max_len", 64), bad=k["bad"],
        q_off=k.get("q_off"), max_rows=k.get("max_rows", 1))
    flag = lambda: torch.zeros(1, dtype=torch.int32, device="cuda")  # noqa: E731
    b = flag()
    good = call(bad=b)
    assert int(b) == 0
    for page_id in (-1, pool[0].shape[0], 2 ** 31 - 1):  # a page that is none: its keys are left out
        t2 = table.copy()
        t2[1, 1] = page_id
        b = flag()
        out = call(table=t2, bad=b)
        assert int(b) == 1 and torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
        # keys 0..15 and 32..39 of request 1
        keep = [p for j, p in enumerate(table[1, :3]) if j != 1]
        kk, vv = ref.gather(pool[0], pool[2], keep, 24), ref.gather(pool[1], pool[3], keep, 24)
        s = torch.einsum("hgd,hkd->hgk", q[1].double().view(2, 4, 64), kk) / 8
        o = torch.einsum("hgk,hkd->hgd", torch.softmax(s, -1), vv).reshape(8, 64)
        assert (out[1].double() - o).abs().max() < 1e-4 * vv.abs().max()
    for kw in (dict(max_len=50), dict(lens=[60, -1, 33]), dict(lens=[60, 40, 1000]),
               dict(q_off=dev([0, 1, 2, 9])), dict(q_off=dev([0, 2, 1, 3])), dict(q_off=dev([-1, 0, 1, 3]))):
        b = flag()
        call(bad=b, **kw)
        torch.cuda.synchronize()
        assert int(b) == 1, kw


def test_attention_offsets_past_32_bits():
    """A pool of more than 2^32 bytes of codes, the sequence at its end."""
    H, page, hd = 8, 64, 128
    pages = (1 << 32) // (H * page * hd) + 40
    k, v = (torch.zeros((pages, H, page, hd), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((pages, H, page // 16), device="cuda") for _ in range(2))
    pool = (k, v, ks, vs)
    L = 200
    table = np.array([[pages - 1, pages - 9, pages - 2, pages - 17]])
    pos = np.arange(L)
    slot = table[0, pos // page] * page + pos % page
    kn, vn = rows(L, H, hd, "bf16", 3)
    ddl.ddl_kv8_append(pool, kn, vn, dev(slot))
    q = torch.randn((1, 16, hd), device="cuda")
    check_attention(pool, q, np.array([0, 1]), np.array([L]), table)
    assert int((ks != 0).any(-1).any(-1).sum()) == 4
    got = ref.gather(k, ks, table[0], L)
    assert (got - kn.double().transpose(0, 1)).abs().max() <= float(ks.max()) / 2


# ------------------------------------------------------------------ as they are used

def serving_state(R, per, page, H_kv, hd, codes, T, seed=0):
    g = np.random.RandomState(seed)
    pages = R * per
    s = {"pool": make_pool(pages, H_kv, page, hd, codes, seed, junk=True), "table": dev(np.full((R, per), -1)),
         "free": dev(g.permutation(pages)), "old": dev(np.zeros(R)), "page": page}
    for n, k in (("row_off", R + 1), ("kv_len", R), ("row_pos", T), ("slot", T), ("used", 1), ("status", R)):
        s[n] = torch.zeros(k, dtype=torch.int32, device="cuda")
    return s


def plan_step(s, add, taken):
    ddl.ddl_page_plan(s["old"], add, s["free"][taken:], s["table"], s["page"],
                      **{n: s[n] for n in ("row_off", "kv_len", "row_pos", "slot", "used", "status")})


@pytest.mark.parametrize("codes,dtype", [("e4m3", "bf16"), ("int8", "f32")])
def test_serving_loop(codes, dtype):
    """Prompts of odd lengths, then decode steps: every step plans its pages,
    stores its rows and attends; against the 64-bit attention over what the
    64-bit append has stored, step by step from the same inputs."""
    R, page, H_q, H_kv, hd, T = 5, 16, 8, 2, 64, 64
    s = serving_state(R, 8, page, H_kv, hd, codes, T)
    int8 = codes == "int8"
    host = [[p.view(torch.uint8).cpu().numpy(), sc.cpu().numpy().astype(np.float64)]
            for p, sc in ((s["pool"][0], s["pool"][2]), (s["pool"][1], s["pool"][3]))]
    lens, taken = np.zeros(R, int), 0
    table_h = np.full((R, 8), -1)
    free_h = s["free"].cpu().numpy()
    for step, add in enumerate([[17, 1, 0, 30, 16], [1, 1, 12, 1, 1], [1, 4, 1, 0, 1], [1] * 5, [1, 0, 1, 1, 1]]):
        plan_step(s, dev(add), taken)
        q = torch.randn((T, H_q, hd), device="cuda", generator=torch.Generator("cuda").manual_seed(step)).to(
            DTYPES[dtype])
        k, v = rows(T, H_kv, hd, dtype, 50 + step)
        ddl.ddl_kv8_append(s["pool"], k, v, s["slot"])
        out = torch.full_like(q, 9)
        ddl.ddl_kv8_attention(s["pool"], q, s["kv_len"], s["table"], 8 * page, q_off=s["row_off"], max_rows=32,
                              out=out)
        table_h, row_off, kv_len, _, slot, used, status = ref.plan(lens, add, free_h[taken:], table_h, page, T)
        assert (status == 0).all() and np.array_equal(s["slot"].cpu().numpy(), slot)
        for i, x in enumerate((k, v)):
            host[i] = list(ref.append(host[i][0], host[i][1], x.double().cpu().numpy(), slot, page, int8))
        pool64 = [torch.from_numpy(h[0]).cuda().view(CODES[codes]) for h in host] + [
            torch.from_numpy(h[1]).cuda() for h in host]
        want, _, tol, _ = ref.attention(pool64, q, row_off, kv_len, table_h, 1 / math.sqrt(hd))
        n = int(row_off[-1])
        assert ((out.double() - want).abs()[:n] <= tol[:n]).all()
        assert (out[n:] == 9).all()
        lens, taken = kv_len, taken + int(used[0])
        s["old"] = dev(lens)


def test_captured_step_replays_with_new_lengths():
    """plan -> append -> attention in a graph: replays follow the lengths, tables and rows in device memory."""
    R, page, H_q, H_kv, hd = 4, 16, 8, 2, 128
    s = serving_state(R, 6, page, H_kv, hd, "e4m3", R)
    add = dev([1] * R)
    q = torch.randn((R, H_q, hd), device="cuda").bfloat16()
    k, v = (x.contiguous() for x in rows(R, H_kv, hd, "bf16", 1))
    out = torch.empty_like(q)
    ws = torch.empty(ddl.ddl_kv8_attention_workspace_bytes(H_q, H_kv, hd, R, R, 1, 6 * page), dtype=torch.uint8,
                     device="cuda")

    def step(o, pool):
        plan_step(s, add, 0)
        ddl.ddl_kv8_append(pool, k, v, s["slot"])
        ddl.ddl_kv8_attention(pool, q, s["kv_len"], s["table"], 6 * page, out=o, workspace=ws)

    pool2 = tuple(t.clone() for t in s["pool"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(out, s["pool"])
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(s["pool"], pool2):
        a.copy_(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out, s["pool"])
    free0 = s["free"].clone()
    taken = 0
    for i in range(40):
        q.copy_(torch.randn((R, H_q, hd), device="cuda", generator=torch.Generator("cuda").manual_seed(i)))
        kn, vn = rows(R, H_kv, hd, "bf16", 100 + i)
        k.copy_(kn)
        v.copy_(vn)
        graph.replay()
        torch.cuda.synchronize()
        mine = out.clone()
        eager = torch.empty_like(q)
        ddl.ddl_kv8_append(pool2, k, v, s["slot"])
        ddl.ddl_kv8_attention(pool2, q, s["kv_len"], s["table"], 6 * page, out=eager)
        assert torch.equal(mine, eager)
        assert (s["status"] == 0).all()
        taken += int(s["used"])
        s["free"].copy_(torch.roll(free0, -taken))  # used ids go to the end (never reached again here)
        s["old"].copy_(s["kv_len"])
    assert (s["kv_len"] == 40).all()


def test_refusals():
    """Argument errors before any launch, with real buffers."""
    pool, q, q_off, lens, table = setup(2, [1, 1], 8, 2, 64, 16, [20, 9], "e4m3", "bf16")
    kl, tb, slot = dev(lens), dev(table), dev([0, 16])
    k, v = rows(2, 2, 64, "bf16", 0)
    bad_calls = [
        lambda: ddl.ddl_kv8_append(pool, k[:1], v, slot),
        lambda: ddl.ddl_kv8_append(pool, k.float(), v, slot),
        lambda: ddl.ddl_kv8_append(pool, k, v, slot.long()),
        lambda: ddl.ddl_kv8_append(pool, k.cpu(), v.cpu(), slot),
        lambda: ddl.ddl_kv8_append(pool[:2] + (pool[2].double(), pool[3]), k, v, slot),
        lambda: ddl.ddl_kv8_append((pool[0].transpose(1, 2),) + pool[1:], k, v, slot),
        lambda: ddl.ddl_kv8_attention(pool, q[:, :7], kl, tb, 32),
        lambda: ddl.ddl_kv8_attention(pool, q, kl.long(), tb, 32),
        lambda: ddl.ddl_kv8_attention(pool, q, kl, tb[:1], 32),
        lambda: ddl.ddl_kv8_attention(pool, q, kl, tb, 0),
        lambda: ddl.ddl_kv8_attention(pool, q, kl, tb, 32, max_rows=2),
        lambda: ddl.ddl_kv8_attention(pool, q, kl, tb, 32, q_off=dev([0, 1, 2]), max_rows=65),
        lambda: ddl.ddl_kv8_attention(pool, q, kl, tb, 32, out=q),
        lambda: ddl.ddl_kv8_attention(pool, q, kl, tb, 32, softcap=-1.0),
        lambda: ddl.ddl_kv8_attention(pool, q, kl, tb, 32, window=-1),
        lambda: ddl.ddl_kv8_attention(pool, q, kl, tb, 32, scale=math.nan),
        lambda: ddl.ddl_kv8_attention(pool, q, kl, tb, 32, slopes=torch.zeros(3, device="cuda")),
        lambda: ddl.ddl_kv8_attention(pool, q, kl, tb, 32, workspace=torch.empty(16, dtype=torch.uint8).cuda()),
        lambda: ddl.ddl_kv8_attention(pool, torch.zeros((2, 20, 64), device="cuda"), kl, tb, 32),  # group of 10
        lambda: ddl.ddl_kv8_attention(pool, q[:1], kl, tb, 32),  # two requests, one row
    ]
    for i, call in enumerate(bad_calls):
        with pytest.raises((ValueError, ddl.DDLError)):
            call()
            pytest.fail(f"call {i} was accepted")
    torch.cuda.synchronize()
