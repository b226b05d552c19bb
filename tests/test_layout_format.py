"""Which KV format a Layout names, by kv_format or, where that is not given, by fp8."""
import dataclasses

import pytest

import sparse_attention_decode_indexer_gb300 as ssa


def _layout(fp8, **kw):
    return ssa.Layout(64, 8, 2, 128, fp8, 1, 8, 8, 1, 4, 2, **kw)


def test_fp8_alone_can_change():
    a = _layout(False)
    assert (a.c().kv_dtype, a.scale_floats) == (ssa.SSA_KV_BF16, 0)
    b = dataclasses.replace(a, fp8=True)
    assert (b.c().kv_dtype, b.scale_floats) == (ssa.SSA_KV_FP8_E4M3, 64)
    b.fp8 = False
    assert (b.c().kv_dtype, b.scale_floats) == (ssa.SSA_KV_BF16, 0)
    assert a == b


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name,scales", [("bf16", 0), ("fp8", 64), ("e4m3_page_head", 2), ("int8_page_head", 2)])
def test_a_format_by_name(fp8, name, scales):
    a = _layout(fp8, kv_format=name)
    assert (a.c().kv_dtype, a.fp8, a.scale_floats) == (ssa.KV_FORMATS[name], name != "bf16", scales)


def test_other_names_are_refused():
    with pytest.raises(ValueError):
        _layout(True, kv_format="int4")
