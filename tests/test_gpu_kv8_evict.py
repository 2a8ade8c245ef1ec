"""Requests cut to their heaviest tokens (ddl_kv8_evict) against a 64-bit
reference: which tokens stay, their codes and scales on the new pages, and what
is left as it was."""
import math

import numpy as np
import pytest
import torch

import kv8_reference as ref
import serving_reference as sref
from memory_bound_transformer_decode_gb300 import ddl
from test_gpu_kv8 import dev, make_pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ddl.load(build_if_missing=True)


def tables(lens, keep, page, seed):
    rng = np.random.RandomState(seed)
    need = [max(0, -(-n // page)) for n in lens]
    new = [-(-k // page) if 0 <= k < n else 0 for n, k in zip(lens, keep)]
    pages = sum(need) + sum(new) + 3
    ids = rng.permutation(pages)
    a = np.full((len(lens), max(need) + 1), -9, np.int32)
    b = np.full((len(lens), max(new + [1])), -9, np.int32)
    at = 0
    for r, n in enumerate(need):
        a[r, :n] = ids[at:at + n]
        at += n
    for r, n in enumerate(new):
        b[r, :n] = ids[at:at + n]
        at += n
    return a, b, pages


def host(t):
    return (t.view(torch.uint8) if t.element_size() == 1 else t).cpu().numpy()


def check(lens, keep, H, hd, page, codes, sinks=0, recent=0, score=None, seed=0, max_keep=None, pool=None, table=None,
          new_table=None, want_bad=0, max_len=None):
    a, b, pages = tables(lens, keep, page, seed)
    table, new_table = a if table is None else table, b if new_table is None else new_table
    pool = make_pool(pages, H, page, hd, codes, seed) if pool is None else pool
    R, most = len(lens), max(max(lens), 1) if max_len is None else max_len
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    if score is None:
        score = torch.exp(3 * torch.randn((R, H, most + 3), generator=g, device="cuda"))
        score[torch.rand(score.shape, generator=g, device="cuda") < 0.2] = 0.0
    cut = [k for n, k in zip(lens, keep) if 0 <= k < n]
    max_keep = max(cut + [1]) if max_keep is None else max_keep
    kept = torch.full((R, H, max_keep), -3, dtype=torch.int32, device="cuda")
    out = torch.full_like(score, -1.0)
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    int8 = codes == "int8"
    want = sref.evict([host(pool[0]), host(pool[1])], [host(pool[i]).astype(np.float64) for i in (2, 3)],
                      score.cpu().numpy(), np.clip(lens, 0, most), [min(k, max_keep) if k < n else k for n, k in zip(lens, keep)],
                      table, new_table, sinks, recent, page, int8, kept.cpu().numpy(), out.cpu().numpy())
    ddl.ddl_kv8_evict(pool, score, dev(lens), dev(keep), dev(table), dev(new_table), most, kept=kept, score_out=out,
                      sinks=sinks, recent=recent, bad=bad)
    torch.cuda.synchronize()
    assert int(bad) == want_bad
    assert np.array_equal(kept.cpu().numpy(), want[2])
    assert np.array_equal(out.cpu().numpy(), want[3], equal_nan=True)
    for i in range(2):
        sc = host(pool[i + 2]).astype(np.float64)
        assert np.array_equal(sc, want[1][i], equal_nan=True)
        x, y = ref.decode(host(pool[i]), int8), ref.decode(want[0][i], int8)
        broken = np.isnan(sc).repeat(16, -1)[..., None]
        assert np.array_equal(np.where(broken, 0, x), np.where(broken, 0, y), equal_nan=True)
    return pool, kept, out


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("H,hd,page", [(1, 128, 16), (3, 64, 32), (2, 128, 256)])
@pytest.mark.parametrize("sinks,recent", [(0, 0), (4, 16), (1, 33), (100, 7)])
def test_cut(codes, H, hd, page, sinks, recent):
    lens = [200, 17, 1, 64, 90]
    keep = [77, 16, 0, 64, -1]
    check(lens, keep, H, hd, page, codes, sinks, recent, seed=hd + sinks)


@pytest.mark.parametrize("L,keep", [(2, 1), (16, 15), (17, 16), (33, 32), (513, 512), (700, 1), (1024, 1000), (5000, 2501)])
def test_lengths(L, keep):
    check([L, 3, 0], [keep, 1, 0], 2, 64, 64, "e4m3", 1, 5, seed=L)


@pytest.mark.parametrize("kind", ["equal", "zeros", "nan", "inf", "negative", "tiny"])
def test_scores(kind):
    """Ties go to the lower index, NaN comes last, both zeros are one."""
    g = torch.Generator(device="cuda").manual_seed(9)
    s = torch.rand((2, 2, 300), generator=g, device="cuda")
    hit = torch.rand(s.shape, generator=g, device="cuda") < 0.5
    if kind == "equal":
        s.fill_(0.5)
    elif kind == "zeros":
        s = torch.where(hit, 0.0, -0.0)
    elif kind == "nan":
        s[hit] = math.nan
        s[1] = math.nan
    elif kind == "inf":
        s[hit] = math.inf
        s[1][torch.rand((2, 300), generator=g, device="cuda") < 0.9] = -math.inf
    elif kind == "negative":
        s = torch.round(s * 20 - 10)
    else:
        s = s * 1e-44
    check([300, 280], [101, 150], 2, 64, 16, "int8", 3, 9, score=s)


def test_a_long_request():
    """Past the keys that fit shared memory."""
    check([60000], [700], 1, 64, 256, "e4m3", 4, 20)


@pytest.mark.parametrize("lens,keep,H", [([10001, 9], [6000, 3], 3), ([400001], [701], 1),
                                         ([60001, 300, 7] + [100] * 17, [123, 299, 7] + [50] * 17, 8)])
def test_clusters_of_four_and_scores_left_in_global_memory(lens, keep, H):
    """A cluster's shared memory holds 393216 scores, that of a CTA (many requests and heads) 49152."""
    check(lens, keep, H, 64, 256, "int8", 2, 11, seed=len(lens))


def test_extreme_scales():
    pool = make_pool(40, 1, 16, 64, "e4m3", 3)
    for i in (2, 3):
        e = torch.randint(-126, 115, pool[i].shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(i))
        pool[i].copy_(torch.exp2(e.float()))
        pool[i][::5] = 0.0
        pool[i][1::5] *= 1.37
    a, b, _ = tables([200, 150], [90, 60], 16, 5)
    check([200, 150], [90, 60], 1, 64, 16, "e4m3", pool=pool, table=a, new_table=b, seed=5)


def test_nan_codes_and_broken_scales():
    pool = make_pool(60, 2, 16, 128, "e4m3", 4, junk=True)
    a, b, _ = tables([200, 150], [90, 60], 16, 6)
    pool[2][a[0, 3], 1] = math.inf
    pool[3][a[1, 2], 0] = -1.0
    pool[2][a[1, 5], 0] = math.nan
    check([200, 150], [90, 60], 2, 128, 16, "e4m3", pool=pool, table=a, new_table=b, seed=6)


def test_outside_the_bounds():
    a, b, pages = tables([100, 80], [40, 30], 16, 7)
    holes = a.copy()
    holes[0, 2] = -1
    holes[1, 0] = pages + 4
    check([100, 80], [40, 30], 2, 64, 16, "int8", seed=7, table=holes, new_table=b, want_bad=1)
    lost = b.copy()
    lost[0, 1] = pages
    check([100, 80], [40, 30], 2, 64, 16, "int8", seed=7, table=a, new_table=lost, want_bad=1)
    check([100, 80], [40, 30], 2, 64, 16, "int8", seed=7, max_keep=25, want_bad=1)
    check([100, 80], [40, 30], 2, 64, 16, "int8", seed=7, max_len=96, want_bad=1)  # kv_len past max_len


def test_shared_pages_are_left_alone_and_a_cut_request_attends_as_before():
    """Two requests on one prefix, one of them cut: the other's attention keeps its bits, and the cut one's
    attention equals that over its kept tokens."""
    H, hd, page = 2, 64, 16
    pool = make_pool(30, H, page, hd, "e4m3", 8)
    for i in (2, 3):
        pool[i].fill_(2.0 ** -8)
    table = np.array([[3, 9, 4, 7], [3, 9, 12, -1]], np.int32)
    lens, keep = [60, 41], [-1, 20]
    q = torch.randn((2, H * 4, hd), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    before = ddl.ddl_kv8_attention(pool, q, dev(lens), dev(table), 64)
    score = torch.rand((2, H, 64), device="cuda")
    new = np.array([[-1, -1, -1, -1], [20, 21, -1, -1]], np.int32)
    kept = torch.zeros((2, H, 20), dtype=torch.int32, device="cuda")
    ddl.ddl_kv8_evict(pool, score, dev(lens), dev(keep), dev(table), dev(new), 64, kept=kept,
                      score_out=torch.zeros_like(score), sinks=2, recent=4)
    after = ddl.ddl_kv8_attention(pool, q, dev([60, 20]), dev([table[0].tolist(), new[1].tolist()]), 64)
    assert torch.equal(before[0], after[0])
    full = [ref.gather(pool[i], pool[i + 2], table[1, :3].tolist(), 41) for i in (0, 1)]
    for h in range(H):
        k, v = (x[h][kept[1, h].long()] for x in full)
        w = torch.softmax(q[1, 4 * h:4 * h + 4].double() @ k.T * hd ** -0.5, -1) @ v
        # (e4m3 codes move to the new scale exactly; bf16 outputs: half a step, and weights to 2^-11)
        assert float((after[1, 4 * h:4 * h + 4].double() - w).abs().max()) <= float(w.abs().max()) * (2 ** -8 + 2 ** -10)


def test_replayed_with_other_lengths():
    H, hd, page = 2, 128, 16
    lens, keep = [100, 90], [50, 40]
    a, b, pages = tables([128, 128], [64, 64], page, 1)
    pool = make_pool(pages, H, page, hd, "int8", 1)
    kv_len, keep_len, tab, new = dev(lens), dev(keep), dev(a), dev(b)
    score = torch.rand((2, H, 128), device="cuda")
    kept = torch.full((2, H, 64), -1, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(score)

    def call():
        ddl.ddl_kv8_evict(pool, score, kv_len, keep_len, tab, new, 128, kept=kept, score_out=out, sinks=1, recent=8)

    call()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        call()
    kv_len.copy_(dev([128, 33]))
    keep_len.copy_(dev([64, 33]))
    score.copy_(torch.rand_like(score))
    kept.fill_(-1)
    out.zero_()
    before = [t.clone() for t in pool]
    want = sref.evict([host(before[0]), host(before[1])], [host(before[i]).astype(np.float64) for i in (2, 3)],
                      score.cpu().numpy(), [128, 33], [64, 33], a, b, 1, 8, page, True, kept.cpu().numpy(), out.cpu().numpy())
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(kept.cpu().numpy(), want[2]) and np.array_equal(out.cpu().numpy(), want[3])
    for i in range(2):
        assert np.array_equal(host(pool[i]), want[0][i]) and np.array_equal(host(pool[i + 2]), want[1][i])


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("odd", [False, True])
def test_scales_up_to_the_largest_power_of_two(codes, odd):
    """Values past fp32: as those of scales 2^64 times smaller, whose products fit."""
    H, hd, page, lens, keep = 2, 64, 16, [200, 150], [90, 60]
    a, b, pages = tables(lens, keep, page, 11)
    pool = make_pool(pages, H, page, hd, codes, 11)
    for i in (2, 3):
        g = torch.Generator(device="cuda").manual_seed(i)
        e = torch.randint(80, 128, pool[i].shape, device="cuda", generator=g).float()
        pool[i].copy_(torch.exp2(e))
        if odd:
            pool[i].copy_(torch.exp2(e - 1) * (1 + torch.rand(e.shape, device="cuda", generator=g) * 0.9))
        pool[i][::7] = 0.0
    score = torch.rand((2, H, 200), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    kept = torch.full((2, H, 90), -1, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(score)
    want = sref.evict([host(pool[0]), host(pool[1])], [host(pool[i]).astype(np.float64) * 2.0 ** -64 for i in (2, 3)],
                      score.cpu().numpy(), lens, keep, a, b, 1, 2, page, codes == "int8", kept.cpu().numpy(), out.cpu().numpy())
    ddl.ddl_kv8_evict(pool, score, dev(lens), dev(keep), dev(a), dev(b), 200, kept=kept, score_out=out, sinks=1, recent=2)
    for i in range(2):
        sc = host(pool[i + 2]).astype(np.float64)
        assert np.isfinite(sc).all() and np.array_equal(sc, want[1][i] * 2.0 ** 64)
        assert np.array_equal(ref.decode(host(pool[i]), codes == "int8"), ref.decode(want[0][i], codes == "int8"))


def test_a_value_past_the_largest_code_of_the_largest_scale():
    pool = make_pool(4, 1, 16, 64, "e4m3", 2)
    for i in (2, 3):
        pool[i].fill_(1.5 * 2.0 ** 127)
    score = torch.arange(16, device="cuda").float().view(1, 1, 16)
    x = [ref.decode(host(pool[i]), False)[1, 0, 8:] * 1.5 for i in range(2)]
    kept = torch.zeros((1, 1, 8), dtype=torch.int32, device="cuda")
    assert max(np.abs(x[0]).max(), np.abs(x[1]).max()) > 448
    ddl.ddl_kv8_evict(pool, score, dev([16]), dev([8]), dev([[1]]), dev([[3]]), 16, kept=kept, score_out=torch.zeros_like(score))
    for i in range(2):
        assert float(pool[i + 2][3]) == 2.0 ** 127
        want = ref.decode(ref.encode_e4m3(np.clip(x[i], -448, 448)), False)
        assert np.array_equal(ref.decode(host(pool[i]), False)[3, 0, :8], want)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("e", [0, 112, 118, 124, 127])
def test_a_scale_of_minus_zero_is_zero(codes, e):
    """Its rows move as zeros beside rows of any scale."""
    pool = make_pool(4, 1, 16, 64, codes, 2)
    for i in (2, 3):
        pool[i].fill_(2.0 ** e)
        pool[i][2] = -0.0
    score = torch.zeros((1, 1, 32), device="cuda")
    score[0, 0, 10:24] = 1.0
    kept = torch.zeros((1, 1, 14), dtype=torch.int32, device="cuda")
    src = [ref.decode(host(pool[i]), codes == "int8")[1, 0, 10:16] for i in range(2)]
    ddl.ddl_kv8_evict(pool, score, dev([32]), dev([14]), dev([[1, 2]]), dev([[3]]), 32, kept=kept,
                      score_out=torch.zeros_like(score))
    assert kept[0, 0].tolist() == list(range(10, 24))
    for i in range(2):
        x = ref.decode(host(pool[i]), codes == "int8")[3, 0]
        assert np.array_equal(x[:6] * float(pool[i + 2][3]), src[i] * 2.0 ** e) and not x[6:].any()


def test_a_request_as_long_as_32_bits_allow():
    """Every page of it the same one; its last tokens lie nearer to 2^31 than a step of any loop."""
    page, hd, keep, sinks, recent = 1024, 64, 300, 3, 5
    per = 2 ** 21 - 1
    L = per * page
    pool = make_pool(3, 1, page, hd, "int8", 5)
    pool[2][0], pool[3][0] = 2.0 ** -7, 2.0 ** -8
    table = torch.zeros((1, per), dtype=torch.int32, device="cuda")
    score = torch.zeros((1, 1, L), device="cuda")
    at = np.unique(np.concatenate([np.random.RandomState(1).randint(0, L, 250), [sinks, 77, L - 900, L - recent - 1, L - 1]]))
    score[0, 0, torch.from_numpy(at).cuda()] = torch.rand(len(at), device="cuda") + 0.5
    out = torch.full_like(score, -1.0)
    kept = torch.full((1, 1, keep), -1, dtype=torch.int32, device="cuda")
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(k):
        ddl.ddl_kv8_evict(pool, score, dev([L]), dev([k]), table, dev([[2]]), L, kept=kept, score_out=out, sinks=sinks,
                          recent=recent, bad=bad)
        torch.cuda.synchronize()

    call(keep)
    edge = set(range(sinks)) | set(range(L - recent, L))
    mid = [i for i in at.tolist() if i not in edge]
    rest, zeros = keep - len(edge) - len(mid), []
    i = sinks
    while len(zeros) < rest:  # ties of zero: the lowest indices
        if i not in mid:
            zeros.append(i)
        i += 1
    want = np.array(sorted(edge | set(mid) | set(zeros)))
    assert int(bad) == 0 and np.array_equal(kept[0, 0].cpu().numpy(), want)
    assert torch.equal(out[0, 0, :keep], score[0, 0, torch.from_numpy(want).cuda()]) and float(out[0, 0, keep:].max()) == -1.0
    for i in range(2):
        src = ref.decode(host(pool[i]), True)[0, 0, want % page] * float(pool[i + 2][0, 0, 0])
        got = ref.decode(host(pool[i]), True)[2, 0, :keep]
        assert np.array_equal(got * host(pool[i + 2])[2, 0].repeat(16)[:keep, None], src)
    call(-1)
    assert torch.equal(out, score)
