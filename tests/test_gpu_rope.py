"""Rotary positions with the cache write, against the formula in 64 bits (angles
in extended precision): both layouts, whole and part of the head, packed views,
in place, far and negative positions, padding and bad slots."""
import numpy as np
import pytest
import torch

from paged_decode_attention_cache_gb300 import ops
from tests.helpers import GuardedOut

pytestmark = pytest.mark.gpu
SRC = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_decode_attention_cache_gb300 import build
    build.build()
    ops.lib()
    torch.cuda.set_device(0)


def turned(x, positions, freq, r, layout, mscale):
    """x float64 [T, heads, D] turned; freq int64 fractions of a turn.  Also |a| + |b| of each element's pair."""
    phase = np.array([[(int(p) * (int(f) % 2 ** 64)) % 2 ** 64 for f in freq] for p in positions], dtype=object)
    angle = (phase / 2 ** 64).astype(np.float64) * 2 * np.pi   # each quotient is rounded once, to 53 bits
    c, s = (f(angle)[:, None, :] * mscale for f in (np.cos, np.sin))
    ia = np.arange(r // 2) * (1 if layout == "half" else 2)
    ib = ia + (r // 2 if layout == "half" else 1)
    y, size = x.copy(), np.abs(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    return y, size * abs(mscale)


def check(got, want, size, r, dt):
    """Angle: 2^-25 of a half-turn (1e-7 rad) and 2^-31; cosine and sine 2 ulp; three fp32 roundings: under 2^-20 of
    |a| + |b|.  Then half a step of the output (of the smallest normal below it).  Dims past r are bit-exact."""
    got = got.double().cpu().numpy()
    f = torch.finfo(SRC[dt])
    allowed = 2.0 ** -20 * size + f.eps / 2 * np.maximum(np.abs(want), f.tiny) * (1 + 2.0 ** -10)
    err = np.abs(got - want)
    assert (err <= allowed).all(), f"max err {err.max():.3e}"
    assert np.array_equal(got[..., r:], want[..., r:])


def data(gen, T, H, Hkv, D, dt, packed):
    if packed:   # one projection's rows, a few unused columns at the end
        x = torch.randn(T, (H + 2 * Hkv) * D + 8, generator=gen).to(SRC[dt]).cuda()
        cut = [x[:, a * D:b * D].view(T, b - a, D) if T == 1 else x[:, a * D:b * D].unflatten(1, (b - a, D))
               for a, b in ((0, H), (H, H + Hkv), (H + Hkv, H + 2 * Hkv))]
        return cut
    return [torch.randn(T, h, D, generator=gen).to(SRC[dt]).cuda() for h in (H, Hkv, Hkv)]


CASES = [("half", 128, 128), ("half", 64, 64), ("half", 128, 64), ("half", 64, 16), ("half", 128, 20), ("half", 64, 2),
         ("interleaved", 128, 128), ("interleaved", 64, 32), ("interleaved", 128, 8), ("interleaved", 64, 6),
         ("interleaved", 128, 50)]


@pytest.mark.parametrize("layout,D,r", CASES)
@pytest.mark.parametrize("dt,T,H,Hkv,packed", [("bf16", 1, 32, 8, False), ("f16", 7, 4, 4, True), ("bf16", 65, 3, 1, True),
                                               ("f16", 300, 8, 2, False)])
def test_rotate_and_write(layout, D, r, dt, T, H, Hkv, packed):
    gen = torch.Generator().manual_seed(T + r)
    q, k, v = data(gen, T, H, Hkv, D, dt, packed)
    nb = T // 16 + 3
    pools = [GuardedOut((nb, 16, Hkv, D), SRC[dt], "cuda") for _ in "kv"]
    for p in pools:
        p.out.copy_(torch.randn(p.out.shape, generator=gen))
    before = [p.out.clone() for p in pools]
    slots = torch.randperm(nb * 16, generator=gen)[:T]
    positions = torch.randint(0, 200000, (T,), generator=gen)
    if T > 4:
        slots[1], slots[3] = -1, -7
        positions[:4] = torch.tensor([0, 2 ** 31 + 5, -3, 2 ** 40 + 1])
    freq = ops.pkv_rope_frequencies(r, 500000.0, "by_parts", 8.0, 1.0, 4.0, 8192)
    rope = ops.Rope(freq.cuda(), r, layout, 1.25)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = ops.Cache(dt, pools[0].out, pools[1].out)
    qo, ko = GuardedOut(q.shape, SRC[dt], "cuda"), GuardedOut(k.shape, SRC[dt], "cuda")
    ops.pkv_rope_and_cache(qo.out, q, k, v, rope, positions.cuda(), cache, slots.cuda(), ko.out, err)
    for g in (qo, ko, *pools):
        g.check()
    assert int(err.item()) == 0
    check(qo.out, *turned(q.double().cpu().numpy(), positions, freq.tolist(), r, layout, 1.25), r, dt)
    check(ko.out, *turned(k.double().cpu().numpy(), positions, freq.tolist(), r, layout, 1.25), r, dt)
    # the slots hold the rotated keys and the values; nothing else in the pools has changed
    for pool, old, rows in ((pools[0].out, before[0], ko.out), (pools[1].out, before[1], v)):
        want = old.clone().view(nb * 16, Hkv, D)
        there = slots >= 0
        want[slots[there].cuda()] = rows[there.cuda()]
        assert torch.equal(pool.view(nb * 16, Hkv, D).view(torch.int16), want.view(torch.int16))
    # the cache alone, and rows alone, give the same bits
    again = GuardedOut(q.shape, SRC[dt], "cuda")
    ops.pkv_rope_and_cache(again.out, q, k, v, rope, positions.cuda(), cache, slots.cuda(), None, err)
    assert torch.equal(again.out, qo.out)
    alone = torch.empty_like(ko.out)
    ops.pkv_rope_and_cache(again.out, q, k, None, rope, positions.cuda(), None, None, alone, err)
    assert torch.equal(alone, ko.out) and torch.equal(again.out, qo.out)
    # in place, in the packed rows too
    ops.pkv_rope_and_cache(q, q, k, v, rope, positions.cuda(), None, None, k, err)
    assert torch.equal(q, qo.out) and torch.equal(k, ko.out)


def test_many_heads_one_token_and_bad_slots():
    T, H, Hkv, D = 5, 128, 16, 128
    gen = torch.Generator().manual_seed(1)
    q, k, v = data(gen, T, H, Hkv, D, "bf16", False)
    cache = ops.Cache.empty("bf16", 2, Hkv, D)
    slots = torch.tensor([0, 32, 31, 2 ** 40, -1], device="cuda")
    positions = torch.arange(T, device="cuda")
    rope = ops.Rope(ops.pkv_rope_frequencies(D, 10000.0).cuda(), D)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    ops.pkv_rope_and_cache(out, q, k, v, rope, positions, cache, slots, None, err)
    assert int(err.item()) == ops.DEVERR_OOB_SLOT
    assert torch.equal(cache.v.view(32, Hkv, D)[[0, 31]], v[[0, 2]])
    assert int((cache.v.view(32, Hkv, D)[1:31] != 0).sum()) == 0
    assert torch.equal(out[0], q[0])     # position 0 turns nothing
    # the other outputs are as without bad slots
    good = torch.empty_like(q)
    ops.pkv_rope_and_cache(good, q, k, v, rope, positions, None, None, torch.empty_like(k))
    assert torch.equal(out, good)


def test_nothing_is_lost_or_read_across_rows_with_inf_and_nan():
    # a non-finite value spoils its own pair only
    T, H, D, r = 3, 2, 64, 32
    gen = torch.Generator().manual_seed(2)
    q, k, v = data(gen, T, H, H, D, "f16", False)
    for layout in ("half", "interleaved"):
        x = q.clone()
        x[1, 0, 5], x[2, 1, 40] = float("nan"), float("inf")
        rope = ops.Rope(ops.pkv_rope_frequencies(r, 10000.0).cuda(), r, layout)
        clean, dirty = torch.empty_like(q), torch.empty_like(q)
        pos = torch.tensor([9, 10, 11], device="cuda")
        ops.pkv_rope_and_cache(clean, q, k, v, rope, pos, None, None, torch.empty_like(k))
        ops.pkv_rope_and_cache(dirty, x, k, v, rope, pos, None, None, torch.empty_like(k))
        differs = torch.zeros(q.shape, dtype=torch.bool)
        differs[1, 0, [5, 21] if layout == "half" else [4, 5]] = True
        differs[2, 1, 40] = True
        assert torch.equal((clean != dirty).cpu() | dirty.isnan().cpu(), differs)


def test_no_tokens_and_other_streams():
    D, H = 64, 4
    rope = ops.Rope(ops.pkv_rope_frequencies(D, 10000.0).cuda(), D)
    e = torch.empty((0, H, D), dtype=torch.float16, device="cuda")
    ops.pkv_rope_and_cache(e, e, e, e, rope, torch.empty(0, dtype=torch.int64, device="cuda"), None, None, e)
    gen = torch.Generator().manual_seed(3)
    q, k, v = data(gen, 40, H, H, D, "f16", False)
    pos = torch.arange(40, device="cuda")
    want, got = torch.empty_like(q), torch.empty_like(q)
    ops.pkv_rope_and_cache(want, q, k, v, rope, pos, None, None, torch.empty_like(k))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ops.pkv_rope_and_cache(got, q, k, v, rope, pos, None, None, torch.empty_like(k))
    side.synchronize()
    assert torch.equal(got, want)
    ops.pkv_rope_and_cache(got.zero_(), q, k, v, rope, pos, None, None, torch.empty_like(k), stream=torch.cuda.current_stream())
    assert torch.equal(got, want)
    # captured and replayed
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.pkv_rope_and_cache(got, q, k, v, rope, pos, None, None, k)
    k0 = k.clone()
    got.zero_()
    graph.replay()
    assert torch.equal(got, want) and not torch.equal(k, k0)


def test_binding_refuses():
    D, H = 64, 4
    rope = ops.Rope(ops.pkv_rope_frequencies(D, 10000.0).cuda(), D)
    x = torch.zeros((3, H, D), dtype=torch.float16, device="cuda")
    pos = torch.zeros(3, dtype=torch.int64, device="cuda")
    cache = ops.Cache.empty("f16", 2, H, D)
    args = lambda **c: {**dict(q_out=x, q=x, k=x, v=x, rope=rope, positions=pos, cache=cache, slot_mapping=pos), **c}  # noqa: E731
    for change in (dict(positions=pos.int()), dict(positions=pos[:2]), dict(slot_mapping=None), dict(v=None),
                   dict(slot_mapping=pos[:1]), dict(k=x[:2]), dict(v=x.bfloat16()), dict(q_out=x[:, :2]),
                   dict(q=x.transpose(1, 2).contiguous().transpose(1, 2)), dict(q=x.float(), q_out=x.float()),
                   dict(positions=pos.cpu()), dict(rope=ops.Rope(rope.freq, 32)), dict(rope=ops.Rope(rope.freq, D, "other"))):
        with pytest.raises(ValueError):
            ops.pkv_rope_and_cache(**args(**change))
    for change in (dict(cache=ops.Cache.empty("bf16", 2, H, D)), dict(cache=ops.Cache.empty("i8", 2, H, D)),
                   dict(cache=None), dict(q=torch.zeros((3, H * D + 4), dtype=torch.float16, device="cuda")[:, :H * D].unflatten(1, (H, D))),
                   dict(q=x.new_zeros(1, H, D).expand(3, H, D))):
        with pytest.raises(ops.PkvError):
            ops.pkv_rope_and_cache(**args(**change))
