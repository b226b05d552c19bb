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


@pytest.mark.parametrize("first", [None, "bf16", "fp8", "int8_page_head"])
@pytest.mark.parametrize("name,scales", [("bf16", 0), ("fp8", 64), ("e4m3_page_head", 2), ("int8_page_head", 2)])
def test_a_format_assigned_later_sizes_the_cache(first, name, scales):
    """What the library writes by the format has its place: bf16 values two bytes, 8-bit codes their scales."""
    a = _layout(first != "bf16", kv_format=first)
    a.kv_format = name
    assert (a.c().kv_dtype, a.fp8, a.scale_floats) == (ssa.KV_FORMATS[name], name != "bf16", scales)
    c = ssa.KVCache(a, False, device="cpu")
    assert c.k_pool.shape[-1] == c.v_pool.shape[-1] == 2 * 64 * 128 * (2 if name == "bf16" else 1)
    assert (c.k_scale is None) == (name == "bf16") and (c.k_scale is None or c.k_scale.shape[-1] == scales)
    a.kv_format = None                           # fp8 decides again, and says what it said last
    assert a.c().kv_dtype == (ssa.SSA_KV_BF16 if name == "bf16" else ssa.SSA_KV_FP8_E4M3)


def test_fp8_does_not_contradict_the_format():
    a, b = _layout(True, kv_format="bf16"), _layout(False, kv_format="int8_page_head")
    assert not a.fp8 and b.fp8
    for x, fp8 in ((a, True), (b, False)):
        with pytest.raises(ValueError):
            x.fp8 = fp8
        x.fp8 = not fp8
    with pytest.raises(ValueError):
        a.kv_format = "int4"
    assert a.kv_format == "bf16" and not a.fp8
    assert dataclasses.replace(b, page_size=16).fp8
