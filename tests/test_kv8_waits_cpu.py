"""What the kernels of the 8-bit cache read, and when, from their sources: under
a dependent launch a grid runs beside its predecessors, and only its own wait
makes what they wrote visible to it."""
import os
import re

import pytest

from memory_bound_transformer_decode_gb300 import build

FILES = ("ddl_kv8.cu", "ddl_kv8_attn.cu", "ddl_kv8_tc.cu")
# the launch's arguments that are device memory, and the helpers that read it
READS = re.compile(r"load_req\s*\(|req_weight\s*\(|unit_prefix\s*<|load_elem4\s*<|"
                   r"\bA\.(old_len|add_len|free_pages|q_off|kv_len|table|prefix|slot|scale|slopes|rec_o|rec_ml|ks|vs)\s*\[")


def kernels():
    for name in FILES:
        src = re.sub(r"//[^\n]*", "", open(os.path.join(build.CSRC, name)).read())
        for m in re.finditer(r"__global__[^;{]*?(\w+)\(const __grid_constant__", src):
            at = src.index("{", src.index(")", m.end()))
            depth, end = 0, at
            for end in range(at, len(src)):
                depth += {"{": 1, "}": -1}.get(src[end], 0)
                if depth == 0:
                    break
            yield name, m.group(1), src[at:end]


def test_the_kernels_are_found():
    assert sorted(k for _, k, _ in kernels()) == ["kv8_append_kernel", "kv8_attention_kernel", "kv8_join_kernel",
                                                  "kv8_tc_kernel", "page_plan_kernel"]


@pytest.mark.parametrize("name,kernel,body", [pytest.param(*k, id=k[1]) for k in kernels()])
def test_nothing_is_read_ahead_of_the_wait(name, kernel, body):
    before, wait, after = body.partition("pdl_wait();")
    assert wait, f"{kernel} ({name}) has no wait"
    assert not READS.search(before), f"{kernel} ({name}) reads ahead of its wait: {READS.search(before).group(0)}"
    assert READS.search(after)


def test_a_leaving_cta_waits_for_its_copies_whatever_the_limit():
    """ddl_set_wait_limit_ns may be a nanosecond: what is in flight (tensor copies, MMAs) is waited for by a limit
    of its own before the CTA's shared and tensor memory goes to another."""
    src = open(os.path.join(build.CSRC, "ddl_kv8_tc.cu")).read()
    limits = re.findall(r"mbar_wait_thread\(.*, (?:[^,]*& 1|0), ([\w.]+)\)", src)
    assert limits == ["DRAIN_NS"] * 3
    assert int(re.search(r"DRAIN_NS = (\d+)ull", src).group(1)) >= 2 * 10 ** 9


def test_a_wait_that_gives_up_makes_the_results_nan():
    """Without bad_out nothing else tells the caller: the softmax warps that gave up still reach the segment's end,
    and sum and factor of its queries (output, record, and the record in a cluster) are NaN there."""
    src = open(os.path.join(build.CSRC, "ddl_kv8_tc.cu")).read()
    end = src[src.index("// the result: thread = head dimension"):src.index("template <int DT, int EX>\nconst void* tc_fn")]
    assert "break;" not in end
    assert "ok = !ssync_or(3, NS, !ok);" in end
    nan = re.search(r"const float (\w+) = ok \? 1\.f : __uint_as_float\(0x7fffffffu\);", end).group(1)
    assert re.search(rf"lq = \(.*\) \* {nan}, m", end) and re.search(rf"float f = .* \* {nan};", end)
    assert "S.al[x] = f;" in end and "S.ml[x] = make_float2(m, lq);" in end and "make_float2(m, lq);" in end
