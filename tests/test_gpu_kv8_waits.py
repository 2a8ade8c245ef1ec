"""What the attention over the 8-bit cache waits for: its lengths, written by the
launch before it."""
import numpy as np
import pytest
import torch

from memory_bound_transformer_decode_gb300 import ddl
from test_gpu_kv8 import dev, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    ddl.load(build_if_missing=True)


def test_replayed_shares_follow_the_lengths():
    """plan and attention in one graph, its blocks cut into shares and joined: every replay with other lengths has the
    bits of the call alone."""
    page, per = 64, 160
    pool, q, _, _, ids = setup(1, [1], 16, 2, 128, page, [per * page], "e4m3", "bf16", seed=7)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    old, add = i32(1), dev([1])
    table = dev(ids[:, :per])  # (the pool's other pages hold NaN codes)
    free = table[0].clone()
    p = dict(row_off=i32(2), kv_len=i32(1), row_pos=i32(1), slot=i32(1), used=i32(1), status=i32(1))
    bound = 60000
    ws = torch.empty(ddl.ddl_kv8_attention_workspace_bytes(16, 2, 128, 1, 1, 1, bound), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)

    def step():
        ddl.ddl_page_plan(old, add, free, table.clone(), page, **p)
        ddl.ddl_kv8_attention(pool, q, p["kv_len"], table, bound, out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in np.random.RandomState(0).randint(0, per * page, 60):
        old.fill_(int(n))
        graph.replay()
        mine = out.clone()
        assert int(p["kv_len"]) == n + 1
        assert torch.equal(mine, ddl.ddl_kv8_attention(pool, q, dev([n + 1]), table, bound))
