"""Host-side checks of the rotary entry points: the frequency table against its
formulas, and the refusals, without a GPU."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def ops():
    from paged_decode_attention_cache_gb300 import build, ops
    build.build()
    ops.lib()
    return ops


def formula(r, base, kind, factor=1.0, low=1.0, high=32.0, original=0.0):
    """Radians a position."""
    if kind == "ntk" and r > 2:
        base = base * factor ** (r / (r - 2))
    out = []
    for i in range(r // 2):
        f = base ** (-2.0 * i / r)
        if kind == "linear":
            f /= factor
        if kind == "by_parts":
            n = original * f / (2 * math.pi)
            m = 0.0 if n <= low else 1.0 if n >= high else (n - low) / (high - low)
            f = (1 - m) * f / factor + m * f
        out.append(f)
    return out


@pytest.mark.parametrize("r", [2, 6, 20, 64, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
@pytest.mark.parametrize("kind", ["none", "linear", "ntk", "by_parts"])
def test_frequencies(ops, r, base, kind):
    got = ops.pkv_rope_frequencies(r, base, kind, factor=8.0, low_rotations=1.0, high_rotations=4.0, original_context=8192)
    want = formula(r, base, kind, 8.0, 1.0, 4.0, 8192)
    assert got.dtype == torch.int64 and got.numel() == r // 2
    for g, w in zip(got.tolist(), want):
        turns = (g % 2 ** 64) / 2.0 ** 64
        # pow, the mixing and the division by 2 pi: a few roundings of 2^-53 each, and 2^-64 absolute
        assert abs(turns * 2 * math.pi - w) <= 8 * 2.0 ** -53 * max(w, 1e-3) + 2.0 ** -60


def test_frequency_refusals(ops):
    for args in ((0, 1e4), (3, 1e4), (-2, 1e4), (64, 0.0), (64, -1.0), (64, float("inf")), (64, float("nan"))):
        with pytest.raises(ops.PkvError):
            ops.pkv_rope_frequencies(*args)
    for more in (dict(scaling="linear", factor=0.0), dict(scaling="ntk", factor=float("nan")),
                 dict(scaling="by_parts", factor=2.0, low_rotations=4.0, high_rotations=4.0, original_context=100),
                 dict(scaling="by_parts", factor=2.0)):
        with pytest.raises(ops.PkvError):
            ops.pkv_rope_frequencies(64, 1e4, **more)
    with pytest.raises(ValueError):
        ops.pkv_rope_frequencies(64, 1e4, "other")
    assert ops.lib().pkv_rope_frequencies(None, 64, 1e4, None) == ops.PKV_ERR_INVALID_ARG


def call(ops, **change):
    a = dict(kind=1, rotary=128, layout=0, mscale=1.0, freq=0x1000, q_out=0x10000, qos=4096, q=0x20000, qs=4096, H=32,
             k_out=None, kos=0, k=0x30000, ks=1024, v=0x40000, vs=1024, Hkv=8, D=128, dtype=1, pos=0x50000, slots=0x60000,
             T=4, cache=True)
    a.update(change)
    c = ops._Cache(a["kind"], 64, 16, 8, 128, 32, 0x70000, 0x80000, None, None, None)
    r = ops._Rope(a["freq"], a["rotary"], a["layout"], a["mscale"])
    return ops.lib().pkv_rope_and_cache(ctypes.byref(c) if a["cache"] else None, ctypes.byref(r), a["q_out"], a["qos"], a["q"],
                                        a["qs"], a["H"], a["k_out"], a["kos"], a["k"], a["ks"], a["v"], a["vs"], a["Hkv"],
                                        a["D"], a["dtype"], a["pos"], a["slots"], a["T"], None, None)


@pytest.mark.parametrize("change", [
    dict(kind=2), dict(kind=3), dict(dtype=0), dict(dtype=2), dict(Hkv=4, ks=512, vs=512), dict(D=64),
    dict(rotary=0), dict(rotary=3), dict(rotary=130), dict(layout=2), dict(layout=-1), dict(mscale=float("nan")),
    dict(H=0), dict(H=70000), dict(T=-1), dict(qs=4088), dict(qos=4100), dict(ks=0), dict(vs=1020),
    dict(k_out=0x90000, kos=1000), dict(q=None), dict(q=0x20008), dict(q_out=None), dict(k=None), dict(k=0x30002),
    dict(v=None), dict(k_out=0x90008, kos=1024), dict(slots=None), dict(pos=None), dict(freq=None), dict(cache=False)])
def test_refusals(ops, change):
    assert call(ops, **change) in (ops.PKV_ERR_INVALID_ARG, ops.PKV_ERR_UNSUPPORTED), change
    assert ops.lib().pkv_last_error()


def test_no_tokens_is_a_no_op(ops):
    assert call(ops, T=0, q=None, q_out=None, k=None, v=None) == ops.PKV_OK
    assert call(ops, D=96, cache=False) == ops.PKV_ERR_UNSUPPORTED


def test_frequencies_are_within_what_the_header_says(ops):
    """The table against the formulas in 60 digits: an entry is off by at most 2^-53 turns.  In units of 2^-53 / (2 pi) turns,
    theta = base^(-x) <= 1 with x = 2i/R: the exponent's rounding x ln(base) base^-x <= 1/e, pow 1, a scaled base's
    2 x base^-x <= 2 / (e ln(base)) < 0.1, the factor 1, 2 pi's own 1/2, the division 1: 4.  By parts mixes only where
    theta <= 2 pi high / original, far below 1, so its dozen roundings add nothing that counts.  4 / (2 pi) < 1."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")

    def exact(r, base, kind, factor, low, high, original):
        base, factor = Decimal(base), Decimal(factor)
        if kind == "ntk" and r > 2:
            base *= (factor.ln() * r / (r - 2)).exp()
        step, f0 = (base.ln() * -2 / r).exp(), Decimal(1)
        for _ in range(r // 2):
            f, f0 = f0, f0 * step
            if kind == "linear":
                f /= factor
            if kind == "by_parts":
                n = Decimal(original) * f / two_pi
                m = min(Decimal(1), max(Decimal(0), (n - Decimal(low)) / (Decimal(high) - Decimal(low))))
                f = f / factor * (1 - m) + f * m
            yield f / two_pi

    worst = Decimal(0)
    for r in (2, 6, 20, 50, 64, 96, 128):
        for base in (10000.0, 150000.0, 500000.0, 1e7):
            for kind, factor, high in (("none", 1.0, 4.0), ("linear", 3.0, 4.0), ("ntk", 2.5, 4.0), ("ntk", 8.0, 4.0),
                                       ("by_parts", 8.0, 4.0), ("by_parts", 40.0, 32.0)):
                got = ops.pkv_rope_frequencies(r, base, kind, factor, 1.0, high, 8192.0).tolist()
                for g, w in zip(got, exact(r, base, kind, factor, 1.0, high, 8192.0)):
                    worst = max(worst, abs(Decimal(g % 2 ** 64) / Decimal(2) ** 64 - w))
    assert worst <= Decimal(2) ** -53, math.log2(worst)


def test_the_header_states_the_angle_by_the_table():
    import os
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "pkv.h")).read()
    flat = " ".join(text.replace(" * ", " ").split())
    assert "exact to 2^-25 of a half-turn at every position" not in flat
    assert "2^-53 of a turn" in flat and "up to position 2^26" in flat
