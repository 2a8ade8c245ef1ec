"""The 8-bit cache at the ends of its ranges: the longest slot map, and shares whose weights pass 2^22 (64-bit
arithmetic) beside the most requests; and ordinary calls within the bound from each row's own keys."""
import numpy as np
import pytest
import torch

import kv8_bounds
from memory_bound_transformer_decode_gb300 import ddl
from test_gpu_kv8 import check_append, dev, make_pool, rows, setup
from test_gpu_kv8_scales import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    ddl.load(build_if_missing=True)


@pytest.mark.parametrize("T", [65535, 65536])
@pytest.mark.parametrize("codes,dtype", [("e4m3", "bf16"), ("int8", "f32")])
def test_append_of_the_most_rows(T, codes, dtype):
    """Prompts of up to 1200 rows from any place of a block on, padding between them, and blocks met again far behind."""
    g = np.random.RandomState(T)
    slot, block = [], 0
    while len(slot) < T:
        n, at = g.randint(1, 1201), g.randint(16)
        slot += [block * 16 + at + i for i in range(n)] + [-1] * g.randint(3)
        block += (at + n + 15) // 16
    slot = np.array(slot[:T])
    pages = block // 2 + 2
    slot = np.where(slot >= 0, g.permutation(2 * pages)[np.maximum(slot, 0) // 16] * 16 + slot % 16, -1)
    slot[60000:60040] = slot[100:140]
    slot[-5:] = slot[3:8]
    pool = make_pool(pages, 1, 32, 64, codes, seed=T)
    k, v = rows(T, 1, 64, dtype, 5, 4.0)
    check_append(pool, k, v, slot)


@pytest.mark.parametrize("R,H_q,H_kv,hd,codes,dtype,shortest,longest,bound,shares", [
    (4096, 8, 8, 128, "e4m3", "bf16", 1400, 1700, 40000, False),     # (whole units)
    (900, 16, 16, 128, "e4m3", "bf16", 4200, 4600, 40000, True),     # 14400 units of about 275 + 48 blocks: 4.6 million
    (31, 10, 10, 64, "int8", "f32", 220000, 224000, 224000, True)])  # 310 units of about 13900 blocks: 4.3 million
def test_shares_of_the_most_weight(R, H_q, H_kv, hd, codes, dtype, shortest, longest, bound, shares):
    """All requests' pages come from one small pool."""
    page, g = 64, np.random.RandomState(R)
    pool = make_pool(300, H_kv, page, hd, codes, seed=R)
    lens = g.randint(shortest, longest + 1, R)
    lens[0], lens[R // 2] = 0, 5
    table = g.randint(0, 300, (R, -(-longest // page)))
    q = (torch.randn((R, H_q, hd), generator=torch.Generator("cuda").manual_seed(R), device="cuda") * 0.5).to(
        torch.bfloat16 if dtype == "bf16" else torch.float32)
    lse = torch.zeros((R, H_q), device="cuda")
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ddl.ddl_kv8_attention(pool, q, dev(lens), dev(table), bound, lse=lse, bad=bad)
    assert int(bad) == 0
    if shares:  # (only they have records to keep)
        with pytest.raises(ddl.DDLError, match="workspace"):
            ddl.ddl_kv8_attention(pool, q, dev(lens), dev(table), bound, out=out,
                                  workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    for r in (0, 1, 2, R // 2 - 1, R // 2, R // 2 + 1, R - 2, R - 1):
        want, want_l, tol, tol_l = kv8_bounds.attention(pool, q[r:r + 1], [0, 1], lens[r:r + 1], table[r:r + 1], hd ** -0.5)
        assert ((out[r].double() - want[0]).abs() <= tol[0]).all(), r
        assert lens[r] == 0 or ((lse[r] - want_l[0]).abs() <= tol_l[0]).all(), r
    assert not out.isnan().any()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("codes,hd", [("e4m3", 128), ("int8", 128), ("e4m3", 64)])
@pytest.mark.parametrize("n_rows", [[1] * 6, [4, 1, 33, 2, 0, 64]])
@pytest.mark.parametrize("opts", [{}, dict(softcap=30.0), dict(window=77), dict(slopes=True, window=300),
                                  dict(softcap=3.0, window=40, slopes=True)])
@pytest.mark.parametrize("bound", [None, 60000])
def test_calls_are_within_the_bound_of_their_own_keys(dtype, codes, hd, n_rows, opts, bound):
    opts = dict(opts)
    if opts.get("slopes"):
        opts["slopes"] = torch.exp2(-torch.arange(12, device="cuda").float())
    check(*setup(6, n_rows, 12, 2, hd, 16, [1, 37, 300, 16, 2100, 64], codes, dtype, seed=51), max_len=bound, **opts)
