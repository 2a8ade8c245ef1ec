"""Tokens drawn from logits (ddl_sample) against a 64-bit reference, over the
filters, types, sizes, ties and values where they can go wrong."""
import math

import numpy as np
import pytest
import torch

import serving_reference as sref
from memory_bound_transformer_decode_gb300 import ddl

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ddl.load(build_if_missing=True)


def logits(B, V, seed, spread=2.0, peaks=32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((B, V), generator=g, device="cuda") * spread
    n = min(V, peaks)
    at = torch.randint(0, V, (B, n), generator=g, device="cuda")
    return x.scatter_add_(1, at, torch.rand((B, n), generator=g, device="cuda") * 9)


def check(x, t=None, k=None, p=None, m=None, u=None, seed=0):
    B, V = x.shape
    g = torch.Generator(device="cuda").manual_seed(seed)
    f = lambda a: None if a is None else torch.as_tensor(a, dtype=torch.float32).expand(B).contiguous().cuda()  # noqa: E731
    t, p, m = f(t), f(p), f(m)
    k = None if k is None else torch.as_tensor(k, dtype=torch.int32).expand(B).contiguous().cuda()
    u = torch.rand(B, generator=g, device="cuda") if u is None else f(u)
    logp = torch.zeros(B, device="cuda")
    got = ddl.ddl_sample(x, u, temperature=t, top_k=k, top_p=p, min_p=m, logp=logp)
    again = ddl.ddl_sample(x, u, temperature=t, top_k=k, top_p=p, min_p=m)
    assert torch.equal(got, again)
    xs = x.double().cpu().numpy()
    one = lambda a, b, d: d if a is None else float(a[b])  # noqa: E731
    for b in range(B):
        ok = sref.draw(xs[b], one(t, b, 1.0), int(one(k, b, 0)), one(p, b, 1.0), one(m, b, 0.0), float(u[b]))
        tok = int(got[b])
        assert tok in ok, (b, tok, ok)
        have = float(logp[b])
        # one rounding to fp32 of a number that the weights' 2^-32 moves by as much
        assert any(have == w or abs(have - w) <= 2.0 ** -22 * (1 + abs(w)) for w in ok[tok]), (b, have, ok[tok])
    return got, logp


FILTERS = [dict(), dict(t=0.7), dict(k=1), dict(k=50), dict(k=4000), dict(p=0.5), dict(p=0.95), dict(p=0.999), dict(m=0.05),
           dict(t=1.4, k=300, p=0.9, m=0.01), dict(t=0.0), dict(k=40, m=0.3), dict(p=0.9, m=0.2)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("f", FILTERS, ids=str)
def test_filters(dtype, f):
    for B, V in ((3, 50257), (2, 1000)):
        check(logits(B, V, V).to(DTYPES[dtype]), seed=V, **f)


@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 31, 255, 2047, 4096, 4097, 16385, 152064, 2 ** 20])
def test_vocabularies(V):
    x = logits(2, V, V)
    check(x, p=0.8, k=[0, 7])
    check(x)


@pytest.mark.parametrize("B", [1, 2, 9, 10, 64, 151, 300])
def test_rows_with_settings_of_their_own(B):
    """Every cluster size; greedy, unfiltered and filtered rows in one call."""
    g = np.random.RandomState(B)
    x = logits(B, 33000, B).to(torch.bfloat16)
    check(x, t=g.choice([0.0, 0.5, 1.0, 2.0], B), k=g.choice([0, 1, 20, 999, 40000, -3], B), p=g.choice([1.0, 0.3, 0.9, 0.99], B),
          m=g.choice([0.0, 0.02, 1.0], B), seed=B)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V,lead", [(1001, 0), (1001, 3), (50257, 1)])
def test_rows_and_bases_off_16_bytes(dtype, V, lead):
    wide = logits(5, V + 9, 3).to(DTYPES[dtype])
    check(wide[:, lead:lead + V], p=0.9)
    check(wide[:, lead:lead + V].contiguous()[1:], k=20)


@pytest.mark.parametrize("value", [0.0, -0.0, 1e30, -1e30])
@pytest.mark.parametrize("V", [10, 5000, 152064])
def test_equal_logits(value, V):
    """Ties: the lower ids stay, whether the elements fit the list or not."""
    x = torch.full((4, V), value, device="cuda")
    if value == 0.0:
        x[:, ::3] = -0.0
    got, _ = check(x, k=[0, 1, 7, V - 1], u=[0.5, 0.99, 0.999, 0.25])
    assert int(got[1]) == 0 and int(got[2]) == 6 % V
    check(x, p=[0.5, 0.1, 1e-9, 0.999], u=[0.9999, 0.5, 0.5, 0.5])
    check(x, k=[V // 2, 3, 0, 1], p=[0.5, 0.5, 0.5, 0.0], m=[1.0, 0.0, 0.5, 0.0])


def test_two_values_and_coarse_logits():
    """Many ties at the borders, in the list (few) and past it (many)."""
    x = torch.zeros((3, 100000), device="cuda")
    x[:, 17::1000] = 3.0
    check(x, k=[100, 101, 5000], u=[0.3, 0.9999, 0.9])
    check(x, p=[0.01, 0.02, 0.9], u=[0.99, 0.9999, 0.9])
    y = torch.round(logits(4, 152064, 5))
    check(y, k=[60000, 200, 3000, 0], p=[0.99, 0.97, 0.5, 0.9])
    check(y, t=8.0, p=[0.99, 0.97, 0.5, 0.9999])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows_of_nearly_flat_logits(dtype):
    """A CTA a row, thousands of its elements within 1/50 octave: more than a bin of the histogram can hold, some with
    a part of the row above them, masked tokens, and a top-k of more than there are."""
    B, V = 160, 24000
    g = np.random.RandomState(3)
    x = logits(B, V, 5, spread=1.0, peaks=40)
    few = torch.arange(V, device="cuda") % 3 == 0
    x[1::2] = torch.where(few, x[1::2], x[1::2] * 1e-4)
    x[2::4] = torch.where(few, float("-inf"), x[2::4])
    t = np.where(np.arange(B) % 2 == 0, 1e4, 1.0)
    check(x.to(DTYPES[dtype]), t=t, k=g.choice([0, 7, 5000, 13000, 17000, 24000], B), p=g.choice([0.2, 0.9, 1.0], B),
          m=g.choice([0.0, 0.5], B), seed=B)
    check(x.to(DTYPES[dtype]), t=t, p=0.6, seed=V)


@pytest.mark.parametrize("t", [1e-18, 1e-6, 1e6, 1e30, math.inf, math.nan, -1.0, 2.0 ** -60, 2.0 ** -61])
def test_temperatures(t):
    x = logits(2, 3000, 2)
    x[1] = torch.round(x[1])  # several largest
    check(x, t=t)
    check(x, t=t, k=10, p=0.7)


def test_settings_at_their_ends():
    x = logits(8, 2500, 4)
    nan, inf = math.nan, math.inf
    check(x, p=[0.0, -1.0, 1.0, 2.0, nan, inf, 1 - 2.0 ** -24, 1e-30])
    check(x, m=[0.0, -1.0, 1.0, 2.0, nan, inf, 1e-38, 1 - 2.0 ** -24])
    check(x, k=[0, -1, 1, 2500, 2501, 2499, 2 ** 31 - 1, -2 ** 31])
    check(x, u=[0.0, 1.0, -1.0, 2.0, nan, inf, 1 - 2.0 ** -24, 2.0 ** -40])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_infinities_and_nan(dtype):
    x = logits(6, 3001, 6).to(DTYPES[dtype])
    inf = math.inf
    low = float(torch.finfo(DTYPES[dtype]).min)
    x[0, ::2] = -inf
    x[1, :] = -inf          # nothing to draw
    x[2, :] = math.nan      # nothing to draw
    x[3, 5::7] = math.nan
    x[4, [3, 70, 2999]] = inf
    x[5, 1:] = low          # a mask of the type's lowest value: one token left
    for kw in (dict(), dict(k=50), dict(p=0.9), dict(t=0.0), dict(t=math.inf, p=0.5), dict(m=0.1)):
        got, logp = check(x, **kw)
        assert got[1:3].tolist() == [-1, -1] and logp[1:3].tolist() == [-inf, -inf]
        assert int(got[5]) == 0 or kw.get("t") == math.inf


def test_a_mask_leaves_one_token():
    x = torch.full((3, 20000), -math.inf, device="cuda")
    x[0, 0], x[1, 19999], x[2, 7777] = -5.0, 0.0, 3.0
    got, logp = check(x, k=5, p=0.5, u=[0.999, 0.0, 0.5])
    assert got.tolist() == [0, 19999, 7777] and logp.tolist() == [0.0, 0.0, 0.0]


def test_draws_follow_the_distribution():
    """The share of each token over evenly spaced numbers is its probability, to one number."""
    x = logits(1, 12, 8)
    n = 20000
    u = (torch.arange(n, device="cuda") + 0.5) / n
    got = ddl.ddl_sample(x.expand(n, 12).contiguous(), u)
    share = torch.bincount(got.long(), minlength=12).double() / n
    assert float((share - torch.softmax(x[0].double(), 0)).abs().max()) <= 1.0 / n + 2e-7


def test_a_stream_of_its_own_and_a_replay():
    x, u = logits(4, 5000, 1), torch.rand(4, device="cuda")
    t, k, tok = torch.ones(4, device="cuda"), torch.full((4,), 30, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ddl.ddl_sample(x, u, temperature=t, top_k=k, tokens=tok)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ddl.ddl_sample(x, u, temperature=t, top_k=k, tokens=tok)
    t.fill_(0.5)
    k.fill_(0)
    u.copy_(torch.rand(4, device="cuda"))
    x.copy_(logits(4, 5000, 2))
    graph.replay()
    torch.cuda.synchronize()
    for b in range(4):
        assert int(tok[b]) in sref.draw(x[b].double().cpu().numpy(), 0.5, 0, 1.0, 0.0, float(u[b]))


def test_logits_past_32_bits():
    V = 2 ** 20
    B = 2 ** 32 // (2 * V) + 2  # elements past 2^31, bytes past 2^32
    x = torch.zeros((B, V), dtype=torch.bfloat16, device="cuda")
    x[-1, V - 3] = 30.0
    x[-2, 5] = 30.0
    got = ddl.ddl_sample(x, torch.full((B,), 0.5, device="cuda"), top_k=torch.full((B,), 3, dtype=torch.int32, device="cuda"))
    assert int(got[-1]) == V - 3 and int(got[-2]) == 5 and int(got[0]) == 1


def test_after_the_lm_head():
    """The head's logits and a filtered draw: a token step with settings per row."""
    from memory_bound_transformer_decode_gb300 import synth  # noqa: F401

    D, V, B = 128, 3000, 4
    g = torch.Generator(device="cuda").manual_seed(0)
    w = (torch.randn((V, D), generator=g, device="cuda") * 0.3).bfloat16()
    head = ddl.ddl_pack_head(w, D, V, ddl.BF16)
    h = torch.randn((B, D), generator=g, device="cuda")
    out = torch.zeros((B, V), device="cuda")
    best = ddl.ddl_lm_head(D, V, ddl.BF16, head, h, logits=out)
    got, _ = check(out, t=[0.0, 0.8, 1.0, 1.0], k=[0, 20, 0, 50], p=[1.0, 1.0, 0.9, 0.9])
    assert int(got[0]) == int(best[0])


def test_the_most_rows_and_one_more():
    B, V = 65536, 5
    x = logits(B, V, 1, peaks=2)
    u = torch.rand(B, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    got = ddl.ddl_sample(x, u)
    w = torch.softmax(x.double(), -1).cumsum(-1)
    want = (w <= u.double()[:, None] * w[:, -1:]).sum(-1)
    # (a draw within 2^-30 of a border may go either way: softmax's sums are rounded, 5 * 2^-53, the weights to 2^-33)
    near = ((w - u.double()[:, None] * w[:, -1:]).abs() < 2.0 ** -30).any(-1)
    assert torch.equal(got[~near].long(), want[~near]) and int(near.sum()) < 10
    with pytest.raises(Exception):
        ddl.ddl_sample(logits(B + 1, V, 1, peaks=2), torch.rand(B + 1, device="cuda"))


def test_two_streams_at_once():
    """No state is shared: calls that run side by side give what each gives alone."""
    xs = [logits(b, 60000, b) for b in (3, 20)]
    us = [torch.rand(len(x), device="cuda") for x in xs]
    kw = [dict(top_p=torch.full((3,), 0.9, device="cuda")), dict(top_k=torch.full((20,), 3000, dtype=torch.int32, device="cuda"))]
    alone = [ddl.ddl_sample(x, u, **k) for x, u, k in zip(xs, us, kw)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(ddl.ddl_sample(xs[i], us[i], **kw[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, alone[i]) for o in outs[i])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [2, 40, 9000, 152064])
def test_a_min_p_above_one_leaves_the_first_candidate(dtype, V):
    """No weight reaches it, so of several largest logits the lowest id alone stays; a min-p of 1 keeps them all."""
    inf = math.inf
    x = torch.round(logits(9, V, V)).clamp(max=3).to(DTYPES[dtype])  # many largest ones
    x[6, V // 2:] = inf
    x[7, :] = -inf
    m = [2.0, inf, 1.0, 1 + 2.0 ** -23, 2.0, 1.0, 2.0, 2.0, 1.0]
    t = [1.0, 1.0, 1.0, 0.5, inf, inf, 1.0, 1.0, 1e-3]
    for kw in (dict(), dict(k=7), dict(p=0.6)):
        got, logp = check(x, t=t, m=m, u=0.9, **kw)
        first = torch.where(x == x.amax(-1, keepdim=True), torch.arange(V, device="cuda"), V).amin(-1)
        for b in (0, 1, 3, 4, 6):
            assert int(got[b]) == int(first[b]) and float(logp[b]) == 0.0
        assert int(got[7]) == -1
    check(torch.zeros((3, V), device="cuda").to(DTYPES[dtype]), m=[2.0, 1.0, 1.5], u=0.9)
