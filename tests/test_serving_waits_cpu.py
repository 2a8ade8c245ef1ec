"""What the kernels of scores, eviction and draws read, and when, from their sources: under a dependent launch a
grid runs beside its predecessors, and only its own wait makes what they wrote visible to it.  And the bounded
wait of the tensor-core score kernel."""
import os
import re

import pytest

from memory_bound_transformer_decode_gb300 import build

FILES = ("ddl_kv8_score.cu", "ddl_kv8_score_tc.cu", "ddl_kv8_evict.cu", "ddl_sample.cu")
# the launch's arguments that are device memory, and the helpers that read it
READS = re.compile(r"load_req\s*\(|load_cut\s*\(|part\.load\s*\(|column_of\s*<|load_elem4\s*<|Row<DT> row\(|"
                   r"\bA\.(score|score_out|kept|kv_len|keep_len|table|new_table|temperature|top_k|top_p|min_p|u|scale|code|ks|lse)\b")


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(build.CSRC, name)).read())


def kernels():
    for name in FILES:
        src = source(name)
        for m in re.finditer(r"__global__[^;{]*?(\w+)\(const __grid_constant__", src):
            at = src.index("{", src.index(")", m.end()))
            depth, end = 0, at
            for end in range(at, len(src)):
                depth += {"{": 1, "}": -1}.get(src[end], 0)
                if depth == 0:
                    break
            yield name, m.group(1), src[at:end]


def test_the_kernels_are_found():
    assert sorted(k for _, k, _ in kernels()) == ["kv8_move_kernel", "kv8_score_few_kernel", "kv8_score_tc_kernel",
                                                  "kv8_select_kernel", "sample_kernel"]


@pytest.mark.parametrize("name,kernel,body", [pytest.param(*k, id=k[1]) for k in kernels()])
def test_nothing_is_read_ahead_of_the_wait(name, kernel, body):
    before, wait, after = body.partition("pdl_wait();")
    assert wait, f"{kernel} ({name}) has no wait"
    assert not READS.search(before), f"{kernel} ({name}) reads ahead of its wait: {READS.search(before).group(0)}"
    assert READS.search(after)


def test_a_wait_that_gives_up_is_seen_and_its_mmas_are_drained():
    """The one spin of these kernels counts the time; where it gives up the tile's sums become NaN and bad_out's bit 1
    is set, and MMAs on their way are waited for by a limit of their own before the memory goes to another."""
    src = source("ddl_kv8_score_tc.cu")
    assert src.count("mbar_try_wait") == 1 and "now - since > S.wait_ns" in src
    assert re.search(r"late \|\| !ok \? __uint_as_float\(0x7fffffffu\)", src)
    assert "if (!ok && A.bad && tid == 0) atomicOr(A.bad, 2);" in src
    drain = src.index("mbar_wait_thread(bar + 8 * x, phase >> x & 1, DRAIN_NS)")
    assert drain < src.index("tmem_dealloc(")
    assert int(re.search(r"DRAIN_NS = (\d+)ull", src).group(1)) >= 2 * 10 ** 9
    for name in FILES:
        if name != "ddl_kv8_score_tc.cu":
            assert "mbar" not in source(name)


def test_clusters_end_together():
    """No CTA of a cluster leaves while another may still read its shared memory: each kernel that reads it ends its
    last reads with a barrier of the cluster."""
    for name in ("ddl_kv8_evict.cu", "ddl_sample.cu"):
        body = next(b for n, k, b in kernels() if n == name and k in ("kv8_select_kernel", "sample_kernel"))
        last = max(m.start() for m in re.finditer(r"ld[ul]4?_cluster\(|ld_cluster\(|cluster_add\(", body))
        assert "cluster_sync();" in body[last:]
