"""pkv_paged_attention_scored refuses bad arguments on the host, before any launch."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def ops():
    from paged_decode_attention_cache_gb300 import build, ops
    build.build()
    ops.lib()
    return ops


def call(ops, **change):
    a = dict(kind=1, cap=30.0, slopes=0x1000, starts=0x2000, prefix=0x3000, scores=True, q_len=1, heads=32, q_dtype=1, out=0x4000,
             out_dtype=1, ws=0x100000, ws_bytes=1 << 30, window=0, num_seqs=4)
    a.update(change)
    c = ops._Cache(a["kind"], 64, 16, 8, 128, 32, 0x10000, 0x20000, 0x50000, 0x60000, 0x70000)
    s = ops._Seqs(0x30000, 0x40000, a["num_seqs"], 8, a["q_len"], a["window"])
    x = ops._Scores(a["cap"], a["slopes"], a["starts"], a["prefix"])
    return ops.lib().pkv_paged_attention_scored(a["out"], a["out_dtype"], 0x80000, a["q_dtype"], a["heads"],
                                                ctypes.c_float(0.1), ctypes.byref(c), ctypes.byref(s),
                                                ctypes.byref(x) if a["scores"] else None, a["ws"], a["ws_bytes"], None, None)


@pytest.mark.parametrize("change", [
    dict(kind=5), dict(kind=-1), dict(scores=False), dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf")),
    dict(cap=1e-31), dict(q_len=0), dict(q_len=5), dict(heads=24), dict(heads=12), dict(q_dtype=0), dict(q_dtype=2),
    dict(out=None), dict(out=0x4008), dict(out_dtype=3), dict(ws=None), dict(ws=0x100010), dict(ws_bytes=1024),
    dict(window=-1), dict(num_seqs=-1)])
def test_refusals(ops, change):
    assert call(ops, **change) in (ops.PKV_ERR_INVALID_ARG, ops.PKV_ERR_UNSUPPORTED), change
    assert ops.lib().pkv_last_error()


def test_no_sequences_is_a_no_op(ops):
    assert call(ops, num_seqs=0, slopes=None, starts=None, prefix=None, cap=0.0) == ops.PKV_OK
