"""Numbers that do not fit the C interface of the 8-bit cache are refused, not cut down to 32 bits."""
import pytest
import torch

from memory_bound_transformer_decode_gb300 import build, configs, ddl

BIG = 2 ** 32 + 64  # (64 in its low 32 bits)


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return ddl.load()


@pytest.mark.parametrize("name", ["H_q", "H_kv", "hd", "R", "T", "max_rows", "max_len"])
def test_attention_sizes(name):
    sizes = dict(H_q=8, H_kv=2, hd=64, R=1, T=1, max_rows=1, max_len=64)
    with pytest.raises(ValueError, match=f"^{name}: a 32-bit integer"):
        ddl.ddl_kv8_attention_workspace_bytes(**{**sizes, name: BIG})


@pytest.mark.parametrize("name", ["R", "T", "max_rows", "max_len"])
def test_stack_sizes(name):
    sizes = dict(R=1, T=1, max_rows=1, max_len=64)
    with pytest.raises(ValueError, match=f"^{name}: a 32-bit integer"):
        ddl.ddl_stack_kv8_workspace_bytes(ddl.make_shape(configs.SMALL_LAYER), **{**sizes, name: BIG})


@pytest.mark.parametrize("name,value", [("max_rows", BIG), ("max_len", BIG), ("window", BIG), ("window", -2 ** 31 - 1)])
def test_stack_step(name, value):
    t = torch.zeros(1, dtype=torch.int32)
    kw = dict(row_off=t, kv_len=t, row_pos=t, slot=t, page_table=t.view(1, 1), max_rows=1, max_len=64, workspace=t,
              x_bf16=torch.zeros((1, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match=f"^{name}: a 32-bit integer"):
        ddl.ddl_stack_step_kv8(ddl.make_shape(configs.SMALL_LAYER), ddl.INT4, [], [], **{**kw, name: value})


def test_the_header_states_the_precision_of_the_weights():
    """The tests' bounds take the roundings that the header gives, and it claims no more than the kernels hold."""
    import os

    import kv8_bounds

    text = " ".join(open(os.path.join(build.HERE, "..", "include", "ddl.h")).read().replace("*", " ").split())
    assert "Scores, softmax and sums are fp32" not in text
    assert ("times its V scale to 2^-11 of itself for 16-bit rows, 2^-22 for fp32 rows, no finer than 2^-30 (fp32 2^-36) of "
            "the row's largest such product") in text
    for t, step, floor in ((torch.bfloat16, -11, -30), (torch.float16, -11, -30), (torch.float32, -22, -36)):
        assert kv8_bounds.STEP[t] == 2.0 ** step and kv8_bounds.FLOOR[t] == 2.0 ** (floor + 1)
