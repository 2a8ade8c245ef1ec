"""V scales that lie far apart: what a row does not see, or sees with next to no
weight, costs its output no bits. Against 64 bits, with a bound from each row's
own keys (kv8_bounds)."""
import math

import numpy as np
import pytest
import torch

import kv8_bounds
from memory_bound_transformer_decode_gb300 import ddl
from test_gpu_kv8 import dev, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    ddl.load(build_if_missing=True)


def check(pool, q, q_off, lens, table, *, max_len=None, **opts):
    n = np.diff(q_off)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    got = ddl.ddl_kv8_attention(pool, q, dev(lens), dev(table), int(max_len or lens.max()), q_off=dev(q_off),
                                max_rows=int(n.max()), lse=lse, **opts)
    opts.setdefault("scale", 1 / math.sqrt(q.shape[2]))
    want, want_l, tol, tol_l = kv8_bounds.attention(pool, q, q_off, lens, table, **opts)
    # (past float16's range: both sides clamped to it are no further apart)
    top = torch.finfo(q.dtype).max
    over = (got.double().clamp(-top, top) - want.clamp(-top, top)).abs() - tol
    row = int(over.amax((1, 2)).argmax())
    assert not got.isnan().any()
    assert (over <= 0).all(), f"row {row}: past its bound by {float(over.max()):.3g} (bound {float(tol[row].max()):.3g})"
    inf = want_l == -math.inf
    assert torch.equal(lse == -math.inf, inf) and ((lse - want_l).abs()[~inf] <= tol_l[~inf]).all()
    return got, want


# kernels: tensor memory (e4m3, head_dim 128), warp MMAs; bounds on the length that choose clusters or shares
KERNELS = [("e4m3", 128, None), ("e4m3", 128, 60000), ("int8", 128, None), ("e4m3", 64, 60000)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("codes,hd,bound", KERNELS)
@pytest.mark.parametrize("far", [2.0 ** 12, 2.0 ** 30, 2.0 ** 70])
def test_a_later_rows_scale_does_not_reach_earlier_rows(dtype, codes, hd, bound, far):
    """A chunk of 40 rows on 300 tokens, causal: the block of its last 12 tokens has a V scale far above the others."""
    pool, q, off, lens, table = setup(2, [40, 1], 8, 1, hd, 16, [300, 90], codes, dtype, seed=21)
    pool[3][int(table[0, 18])] *= far
    got, want = check(pool, q, off, lens, table, max_len=bound)
    assert want[:28].abs().max() < 1e3 and got[:28].abs().amax((1, 2)).min() > 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("codes,hd,bound", KERNELS)
@pytest.mark.parametrize("H_q", [8, 2])
def test_a_scale_before_the_window_does_not_reach_later_rows(dtype, codes, hd, bound, H_q):
    """Windows of 64 tokens: the first rows of a chunk still see the block of the far scale, the others do not; blocks
    that no row sees, before and behind, have one above all float16 values."""
    pool, q, off, lens, table = setup(2, [40, 3], H_q, 1, hd, 16, [300, 200], codes, dtype, seed=22)
    pool[3][int(table[0, 12])] *= 2.0 ** 40   # tokens 192 .. 207: rows 0 .. 10 see some
    pool[3][int(table[0, 3])] *= 2.0 ** 100   # seen by none
    pool[3][int(table[1, 1])] *= 2.0 ** 100
    got, want = check(pool, q, off, lens, table, max_len=bound, window=64)
    assert want[11:].abs().max() < 1e3 and got[11:].abs().amax((1, 2)).min() > 0


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("codes,hd,bound", KERNELS)
@pytest.mark.parametrize("far,block", [(2.0 ** 20, 0), (2.0 ** 20, 9), (2.0 ** 36, 18), (2.0 ** -40, 5)])
def test_a_scale_of_next_to_no_weight_costs_no_bits(dtype, codes, hd, bound, far, block):
    """One block's keys score 40 below the others (e^-40 = 2^-57.7): with a far V scale their products stay below."""
    pool, q, off, lens, table = setup(1, [3], 4, 1, hd, 16, [301], codes, dtype, seed=23)
    k, ks = pool[0], pool[2]
    q.fill_(1.0)
    ks.fill_(0.01)
    k[int(table[0, block])] = torch.full_like(k[0], -40).to(k.dtype)
    pool[3][int(table[0, block])] *= far
    check(pool, q, off, lens, table, max_len=bound, scale=1.0 / hd * 2.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("codes,hd,bound", KERNELS)
def test_scales_that_rise_and_fall_along_the_tokens(dtype, codes, hd, bound):
    """Scales from 2^-60 to 2^60 up, down and at random, blocks of zeros among them, several rows and requests."""
    for seed, order in enumerate((1, -1, 0)):
        pool, q, off, lens, table = setup(3, [1, 5, 33], 8, 1, hd, 16, [700, 400, 333], codes, dtype, seed=24 + seed)
        g = np.random.RandomState(seed)
        for r in range(3):
            nb = -(-int(lens[r]) // 16)
            e = np.linspace(-60, 60, nb)[::order or 1]
            if not order:
                e = g.permutation(e)
            for j in range(nb):
                pool[3][int(table[r, j])] = 0.0 if j % 11 == 3 else float(2.0 ** round(e[j]) * (1 + 0.3 * (j % 2)))
        check(pool, q, off, lens, table, max_len=bound)


def test_bound_by_hand():
    """Two keys of equal score, V 1 and 2^20: the bound of the row that sees the first alone knows nothing of the other."""
    k = torch.zeros((2, 1, 16, 64), dtype=torch.int8, device="cuda")
    v = torch.ones_like(k)
    vs = torch.tensor([1.0, 2.0 ** 20], device="cuda").view(2, 1, 1)
    q = torch.zeros((2, 1, 64), device="cuda", dtype=torch.bfloat16)
    out, _, tol, _ = kv8_bounds.attention((k, v, torch.ones_like(vs), vs), q, [0, 2], [17], [[0, 1]], 1.0)
    assert torch.allclose(out[0], torch.ones_like(out[0])) and float(tol[0].max()) < 2.0 ** -7
    assert torch.allclose(out[1], torch.full_like(out[1], (16 + 2.0 ** 20) / 17))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("codes,hd,bound", KERNELS)
@pytest.mark.parametrize("cap", [30.0, 1e3, 1e4, 1e6, 1e12, 3e38])
def test_a_cap_far_above_the_scores_changes_nothing(dtype, codes, hd, bound, cap):
    pool, q, off, lens, table = setup(2, [3, 1], 8, 2, hd, 16, [300, 900], codes, dtype, seed=27)
    got, _ = check(pool, q, off, lens, table, max_len=bound, softcap=cap, scale=1.0 / hd)
    if cap >= 1e6:
        plain, want = check(pool, q, off, lens, table, max_len=bound, scale=1.0 / hd)
        assert (got.double() - plain.double()).abs().max() <= 4 * torch.finfo(q.dtype).eps * want.abs().max()


@pytest.mark.parametrize("codes,hd", [("e4m3", 128), ("int8", 64)])
def test_the_longest_window_of_rows_before_the_first_token(codes, hd):
    """More rows than tokens and a window that reaches 2^31 back from a negative position hide nothing."""
    for n, L in ((7, 3), (64, 40)):
        pool, q, off, lens, table = setup(2, [n, 1], 8, 2, hd, 16, [L, 90], codes, "bf16", seed=28)
        for window in (2 ** 31 - 2, 2 ** 31 - 5):
            got, _ = check(pool, q, off, lens, table, max_len=2 ** 31 - 1, window=window)
            plain, _ = check(pool, q, off, lens, table, max_len=2 ** 31 - 1)
            assert torch.equal(got, plain)
