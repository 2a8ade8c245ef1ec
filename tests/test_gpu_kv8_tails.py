"""Long tails of small weights: fp32 rows count in O what they count in the sum."""
import pytest
import torch

import kv8_bounds
from memory_bound_transformer_decode_gb300 import ddl
from test_gpu_kv8 import dev, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    ddl.load(build_if_missing=True)


@pytest.mark.parametrize("codes,hd", [("e4m3", 128), ("int8", 128), ("e4m3", 64)])
@pytest.mark.parametrize("H_q,n", [(8, 1), (64, 1), (64, 2), (64, 4)])
@pytest.mark.parametrize("drop", [18.8, 20.5])
def test_a_tail_beside_one_sharp_key(codes, hd, H_q, n, drop):
    """One key of score 0 whose V row is 0, and 32000 of score -18.8 or -20.5 (weights 2^-27.1, 2^-29.6 of the largest)
    whose V is near 1: the output is the tail's 2^-12 or 2^-15, and all of it where weights that small are dropped.
    38 requests of 8 heads, so that a CTA has a whole request (they share the pages)."""
    L, R = 32000, 38
    pool, q, _, lens, table = setup(1, [n], H_q, 8, hd, 64, [L], codes, "f32", seed=31)
    k, v, ks, vs = pool
    q = torch.ones((R * n, H_q, hd), device="cuda")
    ks.fill_(1.0)
    k.copy_(torch.full_like(k, -1).to(k.dtype))
    vs.fill_(2.0 ** -7)
    v.copy_((torch.rand(v.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(3)) * 24 + 100).to(v.dtype))
    j = 17005
    for t in (k, v):
        t[int(table[0, j // 64]), :, j % 64] = torch.zeros((8, hd), device="cuda").to(t.dtype)
    got = ddl.ddl_kv8_attention(pool, q, dev([L] * R), dev(table.repeat(R, 0)), L, q_off=dev([n * r for r in range(R + 1)]),
                                max_rows=n, scale=drop / hd)
    want, _, tol, _ = kv8_bounds.attention(pool, q[:n], [0, n], [L], table, drop / hd)
    assert float(want.min()) > 0 and float((tol / want).max()) < 0.1
    err = (got.double().view(R, n, H_q, hd) - want).abs()
    assert (err <= tol).all(), f"off by {float((err / want).max()):.3g} of the value (bound {float((tol / want).max()):.3g})"
