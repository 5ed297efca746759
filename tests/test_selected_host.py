"""Key bounds, page selection and attention over selected pages refuse bad arguments on the host, before any launch."""
import ctypes

import pytest
import torch

B, H, HKV, D, PAGES = 2, 4, 2, 64, 3


@pytest.fixture(scope="module")
def ops():
    from paged_decode_attention_cache_gb300 import build, ops
    build.build()
    ops.lib()
    return ops


def structs(ops, a):
    c = ops._Cache(a["kind"], a["num_blocks"], a["block"], 8, a["head_dim"], 32, a["k"], 0x20000, 0x50000, 0x60000, 0x70000)
    s = ops._Seqs(0x30000, 0x40000, a["num_seqs"], a["max_blocks"], a["q_len"], a["window"])
    return ctypes.byref(c), ctypes.byref(s)


BASE = dict(kind=1, num_blocks=64, block=16, head_dim=128, k=0x10000, num_seqs=4, max_blocks=8, q_len=1, window=0, heads=32, rows=4,
            q=0x80000, q_dtype=1, bounds=0x90000, cu=None, lists=0xa0000, counts=0xb0000, pages=5, first=1, last=2, out=0xc0000,
            out_dtype=1, scale=0.1)


def call_bounds(ops, **change):
    a = dict(BASE, **change)
    c, s = structs(ops, a)
    return ops.lib().pkv_key_bounds(ops._P(a["bounds"]), c, a["cu"], s, None, None)


def call_select(ops, **change):
    a = dict(BASE, **change)
    c, s = structs(ops, a)
    return ops.lib().pkv_select_pages(ops._P(a["lists"]), ops._P(a["counts"]), a["pages"], a["first"], a["last"], ops._P(a["q"]),
                                      a["q_dtype"], a["heads"], a["rows"], ops._P(a["bounds"]), c, ops._P(a["cu"]), s, None, None)


def call_attention(ops, **change):
    a = dict(BASE, **change)
    c, s = structs(ops, a)
    return ops.lib().pkv_paged_attention_selected(ops._P(a["out"]), a["out_dtype"], ops._P(a["q"]), a["q_dtype"], a["heads"], a["rows"],
                                                  ctypes.c_float(a["scale"]), c, ops._P(a["cu"]), s, ops._P(a["lists"]),
                                                  ops._P(a["counts"]), a["pages"], None, None)


def refused(ops, st):
    assert st in (ops.PKV_ERR_INVALID_ARG, ops.PKV_ERR_UNSUPPORTED)
    assert ops.lib().pkv_last_error()


@pytest.mark.parametrize("change", [dict(kind=5), dict(block=32), dict(head_dim=96), dict(num_blocks=0), dict(k=None), dict(k=0x10008),
                                    dict(bounds=None), dict(bounds=0x90008), dict(num_seqs=-1), dict(q_len=0), dict(max_blocks=0),
                                    dict(num_seqs=70000)])
def test_bounds_refusals(ops, change):
    refused(ops, call_bounds(ops, **change))


SHARED = [dict(kind=-1), dict(q_dtype=0), dict(q_dtype=2), dict(heads=24), dict(heads=12), dict(heads=128), dict(window=4), dict(window=-1),
          dict(pages=0), dict(rows=3), dict(rows=-1), dict(q_len=2), dict(q=None), dict(q=0x80002), dict(lists=None), dict(counts=None),
          dict(rows=2 ** 30, cu=0x30000), dict(kind=3, q_dtype=2), dict(max_blocks=2 ** 27)]


@pytest.mark.parametrize("change", SHARED + [dict(first=-1), dict(last=-1), dict(first=4), dict(pages=2), dict(bounds=None),
                                             dict(first=2 ** 31 - 1, last=2 ** 31 - 1), dict(bounds=0x90004), dict(max_blocks=327681)])
def test_selection_refusals(ops, change):
    refused(ops, call_select(ops, **change))


@pytest.mark.parametrize("change", SHARED + [dict(out=None), dict(out=0xc0008), dict(out_dtype=3), dict(scale=float("nan")),
                                             dict(pages=131073)])
def test_attention_refusals(ops, change):
    refused(ops, call_attention(ops, **change))


def test_nothing_to_do_is_a_no_op(ops):
    assert call_bounds(ops, num_seqs=0) == ops.PKV_OK
    for call in (call_select, call_attention):
        assert call(ops, num_seqs=0, rows=0, q=None, lists=None, counts=None) == ops.PKV_OK
        assert call(ops, num_seqs=0, rows=7, cu=0x30000) == ops.PKV_OK


def tensors(ops, kind="bf16"):
    c = ops.Cache.empty(kind, 4, HKV, D, device="cpu")
    dt = torch.float16 if kind == "f16" else torch.bfloat16
    s = ops.Seqs(torch.zeros(B, 1, dtype=torch.int32), torch.ones(B, dtype=torch.int32))
    return dict(bounds=ops.key_bounds(c), cache=c, seqs=s, q=torch.zeros(B, H, D, dtype=dt), out=torch.zeros(B, H, D),
                lists=torch.zeros(B, HKV, PAGES, dtype=torch.int32), counts=torch.zeros(B, HKV, dtype=torch.int32),
                cu=torch.zeros(B + 1, dtype=torch.int32))


@pytest.mark.parametrize("kind", ["f16", "bf16", "i8", "e4m3", "k8v4"])
def test_the_bounds_have_the_keys_type(ops, kind):
    t = tensors(ops, kind)
    want = {"f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8, "e4m3": torch.float8_e4m3fn, "k8v4": torch.float16}[kind]
    assert t["bounds"].dtype == want and t["bounds"].shape == (4, HKV, 2, D)
    # everything fits; host tensors are refused last
    with pytest.raises(ValueError, match="CUDA device"):
        ops.pkv_key_bounds(t["bounds"], t["cache"], t["seqs"], t["cu"])
    with pytest.raises(ValueError, match="CUDA device"):
        ops.pkv_select_pages(t["lists"], t["counts"], t["q"], t["bounds"], t["cache"], t["seqs"])
    with pytest.raises(ValueError, match="CUDA device"):
        ops.pkv_paged_attention_selected(t["out"], t["q"], 0.1, t["cache"], t["seqs"], t["lists"], t["counts"])
    with pytest.raises(ValueError, match="bounds must be"):
        ops.pkv_key_bounds(t["bounds"].float(), t["cache"], t["seqs"])


@pytest.mark.parametrize("name,bad,text", [
    ("bounds", torch.zeros(4, HKV, 2, D // 2, dtype=torch.bfloat16), "bounds must be"),
    ("bounds", torch.zeros(5, HKV, 2, D, dtype=torch.bfloat16), "bounds must be"),
    ("lists", torch.zeros(B, HKV, PAGES, dtype=torch.int64), "int32"),
    ("lists", torch.zeros(B, PAGES, dtype=torch.int32), "page_lists must be"),
    ("lists", torch.zeros(B + 1, HKV, PAGES, dtype=torch.int32), "page_lists must be"),
    ("counts", torch.zeros(B, HKV + 1, dtype=torch.int32), "page_lists must be"),
    ("counts", torch.zeros(B * HKV, dtype=torch.int32), "page_lists must be"),
    ("q", torch.zeros(B, H, D), "q must be float16 or bfloat16"),
    ("q", torch.zeros(B, H, 2 * D, dtype=torch.bfloat16), "head_dim"),
    ("q", torch.zeros(B, H * D, dtype=torch.bfloat16), "head_dim"),
    ("out", torch.zeros(B, H, 2 * D), "q and out"),
    ("out", torch.zeros(B, H, D, dtype=torch.float64), "out must be"),
])
def test_wrong_tensors(ops, name, bad, text):
    t = tensors(ops)
    t[name] = bad
    if name != "out":
        with pytest.raises(ValueError, match=text):
            ops.pkv_select_pages(t["lists"], t["counts"], t["q"], t["bounds"], t["cache"], t["seqs"])
    if name != "bounds":
        with pytest.raises(ValueError, match=text):
            ops.pkv_paged_attention_selected(t["out"], t["q"], 0.1, t["cache"], t["seqs"], t["lists"], t["counts"])


@pytest.mark.parametrize("kind,want", [("f16", torch.float16), ("bf16", torch.bfloat16)])
def test_bounds_of_a_cache_that_holds_16_bits_under_another_name(ops, kind, want):
    c = ops.Cache(kind, *(torch.zeros(4, 16, HKV, D, dtype=torch.int16) for _ in "kv"))
    b = ops.key_bounds(c)
    assert b.dtype == want
    with pytest.raises(ValueError, match="CUDA device"):
        ops.pkv_key_bounds(b, c, ops.Seqs(torch.zeros(B, 1, dtype=torch.int32), torch.ones(B, dtype=torch.int32)))
