"""Host-side checks of the 8-bit caches with block scales, no GPU needed: the
entry points refuse bad arguments before touching the device, and the reference
the GPU tests compare with has the properties it is derived from."""
import ctypes

import numpy as np
import pytest
import torch

from tests import blocks_reference as R


@pytest.fixture(scope="module")
def lib():
    from paged_decode_attention_cache_gb300 import build, ops
    build.build()
    return ops.lib()


def structs(kind=3, scales=(0x50000, 0x60000), q_len=1, num_seqs=4):
    from paged_decode_attention_cache_gb300 import ops
    c = ops._Cache(kind, 64, 16, 8, 128, 0, 0x10000, 0x20000, *scales, None)
    return c, ops._Seqs(0x30000, 0x40000, num_seqs, 8, q_len, 0)


def append(lib, c, s, dtype=1, tokens=4, cu=None, k=0x70000, v=0x80000, ks=1024, vs=1024):
    return lib.pkv_quantize_kv_blocks(ctypes.byref(c), k, ks, v, vs, dtype, tokens, cu, ctypes.byref(s), None, None)


def test_append_arguments_checked_on_the_host(lib):
    from paged_decode_attention_cache_gb300 import ops
    bad = ops.PKV_ERR_INVALID_ARG
    for kind in (0, 1, 2, 5):   # only the two 8-bit kinds (K8V4: refused for its v_group already)
        c, s = structs(kind)
        assert append(lib, c, s) == (ops.PKV_ERR_UNSUPPORTED if kind == 2 else bad)
    c, s = structs(scales=(None, 0x60000))
    assert append(lib, c, s) == bad and "k_scale" in lib.pkv_last_error().decode()
    c, s = structs(scales=(0x50000, 0x60008))
    assert append(lib, c, s) == bad and "aligned" in lib.pkv_last_error().decode()
    c, s = structs()
    assert append(lib, c, s, dtype=2) == bad
    assert append(lib, c, s, tokens=-1) == bad
    assert append(lib, c, s, tokens=5) == bad and "q_len" in lib.pkv_last_error().decode()
    assert append(lib, c, s, tokens=2 ** 31 - 1, cu=0x90000) == bad
    assert append(lib, c, s, ks=1016) == bad and append(lib, c, s, vs=1028) == bad and append(lib, c, s, ks=0) == bad
    assert append(lib, c, s, k=None) == bad and append(lib, c, s, v=0x80008) == bad
    assert append(lib, c, s, tokens=0, cu=0x90000) == ops.PKV_OK      # nothing to append: no launch
    c, s = structs(num_seqs=0)
    assert append(lib, c, s, tokens=0) == ops.PKV_OK
    c.head_dim = 96
    assert append(lib, c, s) == ops.PKV_ERR_UNSUPPORTED
    c, s = structs()
    c.num_blocks = 2 ** 27 + 1
    assert append(lib, c, s) == bad


def test_other_entry_points_on_the_new_kinds(lib):
    from paged_decode_attention_cache_gb300 import ops
    c, s = structs()
    byte = ctypes.byref
    assert lib.pkv_reshape_and_cache(byte(c), 0x70000, 0x80000, 0x90000, 4, None, None) == ops.PKV_ERR_INVALID_ARG
    assert lib.pkv_quantize_kv(byte(c), 0x70000, 0x80000, 1, 0x90000, 4, None, None) == ops.PKV_ERR_INVALID_ARG
    assert lib.pkv_gather_kv_cache(0x70000, 0x80000, 0x90000, byte(c), byte(s), None, None) == ops.PKV_ERR_INVALID_ARG
    assert lib.pkv_decode_step_balanced(0x70000, 1, 0x80000, 1, 32, ctypes.c_float(0.1), byte(c), byte(s), 0xa0000, 0xb0000,
                                        1, 0xc0000, 4, 0x100000, 1 << 30, None, None) == ops.PKV_ERR_UNSUPPORTED
    assert "pkv_quantize_kv_blocks" in lib.pkv_last_error().decode()
    s.q_len = 5      # 4 heads per kv head x 5 rows > 16
    assert lib.pkv_paged_attention(0x70000, 1, 0x80000, 1, 32, ctypes.c_float(0.1), byte(c), byte(s), None,
                                   None) == ops.PKV_ERR_UNSUPPORTED


def test_reference_e4m3_is_the_type(lib):
    # every finite e4m3 number maps to itself, and the reference rounds as torch's conversion does
    b = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    b = b[np.isfinite(b)]
    assert np.array_equal(R.to_e4m3(b), b)
    x = np.random.default_rng(0).uniform(-448, 448, 100000) * np.exp2(np.random.default_rng(1).integers(-18, 1, 100000))
    x = x.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).float().double().numpy()
    assert np.array_equal(R.to_e4m3(x), want)


@pytest.mark.parametrize("kind,worst", [("i8", 0.25 + 2 ** -20), ("e4m3", 1.0)])
def test_reference_scale_covers_and_wastes_little(kind, worst):
    rng = np.random.default_rng(2)
    for a in np.exp(rng.uniform(-60, 60, 2000)).astype(np.float32):
        s = R.scale_for(a, kind)
        t = np.float32(a) / np.float32(R.QMAX[kind])
        assert t <= s < t * (1 + worst) * (1 + 2.0 ** -22)
    # the smallest: t = 2^-149 / qmax rounds to zero; a t that does not is held up to 2^-126
    assert R.scale_for(0.0, kind) == 0 and R.scale_for(1e-45, kind) == 0
    assert R.scale_for(1e-40, kind) == np.float32(2.0 ** -126)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_reference_append_error(kind):
    """Token by token or all at once, a stored value is within a few half-steps of what was given: half a step of its
    own rounding, and at most as much again for all the times its block's scale grew (each growth is by a quarter or
    more, so the roundings' errors shrink in units of the last step: 1 + 4/5 + 16/25 + ... = 5 halves; e4m3's
    power-of-two growth rounds again only where codes turn subnormal, half of 2^-9 each time, 2 in all)."""
    rng = np.random.default_rng(3)
    H, D, n = 1, 64, 40
    x = rng.standard_normal((n, H, D)) * np.exp(rng.uniform(-2, 2, (n, H, 1)))
    x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    tables = np.array([[2, 0, 1]], np.int32)
    for sizes in ([n], [1] * n, [7, 13, 20]):
        kc, vc = np.zeros((3, 16, H, D)), np.zeros((3, 16, H, D))
        ks, vs = np.zeros((3, H), np.float32), np.zeros((3, H), np.float32)
        at = 0
        for m in sizes:
            R.append(kc, vc, ks, vs, kind, x[at:at + m], -x[at:at + m], tables, [at + m], [m])
            at += m
        got, scale = R.stored(kc, ks, tables, 0, n), ks[tables[0]].repeat(16, 0)[:n, :, None].astype(np.float64)
        if kind == "i8":
            allowed = 0.5 * scale * (1 if len(sizes) == 1 else 5) * (1 + 2.0 ** -20)
        else:
            allowed = 2.0 ** -4 * np.abs(x) + 2 * 2.0 ** -10 * scale
        assert (np.abs(got - x) <= allowed * (1 + 1e-6)).all()
        assert np.array_equal(R.stored(vc, vs, tables, 0, n), -got)
