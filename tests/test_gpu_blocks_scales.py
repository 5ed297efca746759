"""Attention over 8-bit caches whose V scales are zero or tiny: a cache straight from
Cache.empty, heads and blocks of zeros as the append leaves them, and scales down to
the smallest fp32 numbers, under every schedule and the scored call."""
import numpy as np
import pytest
import torch

from paged_decode_attention_cache_gb300 import ops
from tests import blocks_reference as R
from tests.helpers import GuardedOut
from tests.test_gpu_blocks import State, attend, rows, tables_for, want_attention

pytestmark = pytest.mark.gpu
H, HKV = 8, 2
CTX = [1, 16, 17, 40, 100, 301, 0, 700]
SCHEDULES = ["single", "split", "balanced", "noalloc", "cascade", "sparse", "scored"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_decode_attention_cache_gb300 import build
    build.build()
    ops.lib()
    torch.cuda.set_device(0)


def tables_seqs(rng, ctx):
    """Tables whose last two sequences of more than 64 tokens share four blocks (for the cascade)."""
    tables, nb = tables_for(rng, ctx)
    long_ones = [s for s, c in enumerate(ctx) if c > 80]
    tables[long_ones[1], :4] = tables[long_ones[0], :4]
    return tables, nb, ops.Seqs(torch.from_numpy(tables).cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"))


def run(schedule, st, seqs, q, out):
    B, D = seqs.block_tables.shape[0], st.cache.head_dim
    scale = D ** -0.5
    if schedule == "cascade":
        members, blocks = ops.pkv_cascade_plan(seqs.block_tables, seqs.context_lens, 4, min_shared_blocks=1)
        assert members.shape[0] >= 1
        ops.pkv_paged_attention_cascade(out, q, scale, st.cache, seqs, members.cuda(), blocks.cuda(),
                                        ops.cascade_workspace(B, H, HKV, D, members.shape[0], 4), st.err)
    elif schedule == "sparse":     # every page listed: the same result
        mb = seqs.block_tables.shape[1]
        lists = torch.arange(mb, dtype=torch.int32, device="cuda").repeat(B, 1)
        counts = ((seqs.context_lens + 15) // 16).to(torch.int32)
        ops.pkv_paged_attention_sparse(out, q, scale, st.cache, seqs, lists, counts,
                                       ops.sparse_workspace(B, HKV, D, mb), st.err)
    elif schedule == "scored":     # a cap far above every score
        ops.pkv_paged_attention_scored(out, q, scale, st.cache, seqs, ops.Scores(1e6), ops.balanced_workspace(B, HKV, D), st.err)
    else:
        attend(st, seqs, q, out, schedule, scale)
    assert int(st.err.item()) == 0


def check(schedule, st, seqs, ctx, q, qr):
    g = GuardedOut(q.shape, torch.float32, "cuda")
    run(schedule, st, seqs, q, g.out)
    g.check()
    want, biggest, vmax = want_attention(st, qr, ctx, 1, st.cache.head_dim ** -0.5)
    # below fp32's normal numbers a rounding is half of 2^-149 whatever the value: one as the partials leave the MMA's
    # unit, two for each of up to 24 warps and 8 pieces that a sum goes through, one at the division: under 2^7 of them
    allowed = R.tolerance(biggest, vmax)[0] + 2.0 ** -24 * np.abs(want) + 2.0 ** -143
    got = g.out.double().cpu().numpy()
    assert np.isfinite(got).all()
    err = np.abs(got - want)
    assert (err <= allowed).all(), f"max err {err.max():.3e}, vmax {vmax:.3e}"


@pytest.mark.parametrize("schedule", SCHEDULES)
@pytest.mark.parametrize("kind,D", [("i8", 128), ("i8", 64), ("e4m3", 128), ("e4m3", 64)])
def test_a_fresh_cache_attends_to_zeros(schedule, kind, D):
    rng = np.random.default_rng(51)
    tables, nb, seqs = tables_seqs(rng, CTX)
    st = State(rng, kind, nb, HKV, D)
    st.cache = ops.Cache.empty(kind, nb, HKV, D)
    q, _ = rows(rng, len(CTX), H, D, "bf16", 1.0)
    g = GuardedOut(q.shape, torch.bfloat16, "cuda")
    run(schedule, st, seqs, q, g.out)
    g.check()
    assert torch.equal(g.out, torch.zeros_like(g.out))


@pytest.mark.parametrize("schedule", SCHEDULES)
@pytest.mark.parametrize("kind,D", [("i8", 128), ("e4m3", 64)])
@pytest.mark.parametrize("zero", ["one head", "first 32 tokens", "first 16 tokens", "last block", "all"])
def test_appended_zeros_are_attended(schedule, kind, D, zero):
    rng = np.random.default_rng(52)
    ctx = CTX
    tables, nb, seqs = tables_seqs(rng, ctx)
    st = State(rng, kind, nb, HKV, D)
    st.tables = tables
    n = sum(ctx)
    cu = np.concatenate([[0], np.cumsum(ctx)])
    k, (v, vr) = rows(rng, n, HKV, D, "bf16", 1.0), rows(rng, n, HKV, D, "bf16", 1.0)
    if zero == "one head":
        v[:, 1], vr[:, 1] = 0, 0
    for s, c in enumerate(ctx):
        a, b = {"first 32 tokens": (0, 32), "first 16 tokens": (0, 16), "last block": ((c - 1) // 16 * 16, c),
                "all": (0, c)}.get(zero, (0, 0))
        v[cu[s]:cu[s + 1]][a:b] = 0
        vr[cu[s]:cu[s + 1]][a:b] = 0
    # sequence by sequence: the two that share blocks write them one after the other
    whole = seqs
    for s, c in enumerate(ctx):
        if c:
            st.append((k[0][cu[s]:cu[s + 1]], k[1][cu[s]:cu[s + 1]]), (v[cu[s]:cu[s + 1]], vr[cu[s]:cu[s + 1]]),
                      tables[s:s + 1], [c], [c], cu=[0, c])
    st.same()
    q, qr = rows(rng, len(ctx), H, D, "bf16", 1.0)
    check(schedule, st, whole, ctx, q, qr)


@pytest.mark.parametrize("schedule", SCHEDULES)
@pytest.mark.parametrize("kind,D", [("i8", 128), ("e4m3", 64)])
@pytest.mark.parametrize("low,high", [(-149, -149), (-126, -126), (-126, -110), (-114, -114), (-126, 0), (-100, 60)])
def test_v_scales_of_any_size(schedule, kind, D, low, high):
    rng = np.random.default_rng(53)
    ctx = CTX
    tables, nb, seqs = tables_seqs(rng, ctx)
    st = State(rng, kind, nb, HKV, D)
    st.tables = tables
    st.ks[:] = np.float32(0.02)
    st.vs[:] = np.ldexp(1.0, rng.integers(low, high + 1, st.vs.shape)).astype(np.float32)
    st.vs *= np.where(rng.random(st.vs.shape) < 0.3, -1, 1).astype(np.float32)
    st.cache.k_scale.copy_(torch.from_numpy(st.ks))
    st.cache.v_scale.copy_(torch.from_numpy(st.vs))
    q, qr = rows(rng, len(ctx), H, D, "bf16", 1.0)
    check(schedule, st, seqs, ctx, q, qr)


@pytest.mark.parametrize("schedule", ["single", "split", "balanced", "scored"])
@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_zeros_under_verify_blocks(schedule, kind):
    # 16 query rows a kv head: the wider instantiation
    rng = np.random.default_rng(54)
    ctx, D, ql = [4, 33, 64, 200], 128, 4
    tables, nb = tables_for(rng, ctx)
    st = State(rng, kind, nb, HKV, D)
    st.tables = tables
    st.ks[:] = np.float32(0.02)
    st.vs[:] = np.float32(0.0)
    st.vs[tables[3, 2:5]] = np.float32(0.5)      # one sequence has three blocks of something, behind two of zeros
    st.cache.k_scale.copy_(torch.from_numpy(st.ks))
    st.cache.v_scale.copy_(torch.from_numpy(st.vs))
    seqs = ops.Seqs(torch.from_numpy(tables).cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"), ql)
    q, qr = rows(rng, len(ctx) * ql, H, D, "f16", 1.0)
    g = GuardedOut(q.shape, torch.float32, "cuda")
    if schedule == "scored":
        ops.pkv_paged_attention_scored(g.out, q, D ** -0.5, st.cache, seqs, ops.Scores(1e6),
                                       ops.balanced_workspace(len(ctx), HKV, D), st.err)
    else:
        attend(st, seqs, q, g.out, schedule, D ** -0.5)
    g.check()
    want, biggest, vmax = want_attention(st, qr, ctx, ql, D ** -0.5)
    got = g.out.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= R.tolerance(biggest, vmax)[0] + 2.0 ** -24 * np.abs(want)).all()


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("scale", [2.0 ** -149, 1e-40, 2.0 ** -127, 2.0 ** -126])
def test_zeros_appended_behind_a_subnormal_scale(kind, scale):
    # the block's scale stays, so do the older codes, and the new ones are zeros
    rng = np.random.default_rng(55)
    D, c = 64, 7
    st = State(rng, kind, 1, HKV, D)
    for t in (st.cache.k_scale, st.cache.v_scale):
        t.fill_(scale)
    before = [t.view(torch.uint8).clone() for t in (st.cache.k, st.cache.v)]
    held = st.cache.k_scale.clone()
    new = torch.zeros((1, HKV, D), dtype=torch.bfloat16, device="cuda")
    seqs = ops.Seqs(torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.tensor([c + 1], dtype=torch.int32, device="cuda"))
    ops.pkv_quantize_kv_blocks(st.cache, new, -new, seqs, None, st.err)
    for was, t in zip(before, (st.cache.k, st.cache.v)):
        got = t.view(torch.uint8)
        assert torch.equal(got[:, :c], was[:, :c]) and torch.equal(got[:, c + 1:], was[:, c + 1:])
        assert ((got[:, c] & 0x7f) == 0).all()
    assert torch.equal(st.cache.k_scale, held) and torch.equal(st.cache.v_scale, held)
    # something to hold: the scale grows to the grid and the older codes shrink with it
    k, v = rows(rng, 1, HKV, D, "bf16"), rows(rng, 1, HKV, D, "bf16")
    st.kc, st.vc = (R.values(t, kind) for t in (st.cache.k, st.cache.v))
    st.ks, st.vs = (t.cpu().numpy().copy() for t in (st.cache.k_scale, st.cache.v_scale))
    st.append(k, v, np.zeros((1, 1), np.int32), [c + 2], [1])
    st.same()
