"""The 8-bit caches with one scale per (16-token block, kv head): append, read-back
and attention over them, against a plain 64-bit restatement.  Codes and scales
are compared bit for bit; every pool block that no sequence owns has NaN scales."""
import numpy as np
import pytest
import torch

from paged_decode_attention_cache_gb300 import ops
from tests import blocks_reference as R
from tests.helpers import GuardedOut

pytestmark = pytest.mark.gpu
SRC = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_decode_attention_cache_gb300 import build
    build.build()
    ops.lib()
    torch.cuda.set_device(0)


def tables_for(rng, ctx, spare=3, extra_cols=1):
    used = [-(-max(int(c), 0) // 16) for c in ctx]
    nb = sum(used) + spare
    perm = rng.permutation(nb).astype(np.int32)
    t = np.full((len(ctx), max(used + [0]) + extra_cols), -1, np.int32)
    at = 0
    for s, n in enumerate(used):
        t[s, :n] = perm[at:at + n]
        at += n
    return t, nb


def rows(rng, n, H, D, dt, spread=3.0):
    """Values whose tokens differ in size by up to e^spread, as device tensor and float64."""
    x = rng.standard_normal((n, H, D)) * np.exp(rng.uniform(-spread, spread, (n, H, 1)))
    t = torch.from_numpy(x).to(SRC[dt])
    return t.cuda(), t.double().numpy()


class State:
    """A device cache of garbage codes and NaN scales, and the same held by the reference."""

    def __init__(self, rng, kind, nb, H, D):
        self.kind = kind
        self.cache = ops.Cache.empty(kind, nb, H, D)
        for t in (self.cache.k, self.cache.v):
            b = rng.integers(0, 256, t.shape, dtype=np.uint8)
            b[(b & 0x7f) == 0x7f] ^= 1
            b[b == 0x80] = 0
            t.view(torch.uint8).copy_(torch.from_numpy(b))
        self.cache.k_scale.fill_(float("nan"))
        self.cache.v_scale.fill_(float("nan"))
        self.kc, self.vc = (R.values(t, kind) for t in (self.cache.k, self.cache.v))
        self.ks, self.vs = (t.cpu().numpy().copy() for t in (self.cache.k_scale, self.cache.v_scale))
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def append(self, k, v, tables, ctx, new, cu=None, expect=0):
        kd, kr = k
        vd, vr = v
        seqs = ops.Seqs(torch.from_numpy(tables).cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                        1 if cu is not None else new[0])
        cu = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
        ops.pkv_quantize_kv_blocks(self.cache, kd, vd, seqs, cu, self.err)
        R.append(self.kc, self.vc, self.ks, self.vs, self.kind, kr, vr, tables, ctx, new)
        assert int(self.err.item()) == expect
        return seqs

    def same(self):
        for t, want in ((self.cache.k, self.kc), (self.cache.v, self.vc)):
            got = R.values(t, self.kind)
            assert np.array_equal(got, want), f"{(got != want).sum()} codes differ"
        for t, want in ((self.cache.k_scale, self.ks), (self.cache.v_scale, self.vs)):
            assert np.array_equal(t.cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("dt,H,D", [("bf16", 2, 128), ("f16", 1, 64), ("bf16", 3, 64), ("f16", 8, 128)])
def test_prompts_then_tokens_bit_exact(kind, dt, H, D):
    # ragged prompts (one of none), then single tokens, then blocks of three: scales grow inside blocks
    rng = np.random.default_rng(H * 1000 + D + len(kind))
    final = [60, 1, 16, 33, 90, 17, 40]
    new = [35, 0, 15, 16, 70, 1, 17]
    tables, nb = tables_for(rng, final)
    st = State(rng, kind, nb, H, D)
    cu = np.concatenate([[0], np.cumsum(new)])
    n = int(cu[-1])
    st.append(rows(rng, n, H, D, dt), rows(rng, n, H, D, dt), tables, new, new, cu=cu)
    st.same()
    ctx = list(new)
    for step in (1, 1, 1, 1, 1, 3, 3, 3):
        ctx = [min(c + step, f) for c, f in zip(ctx, final)]
        B = len(ctx)
        st.append(rows(rng, B * step, H, D, dt), rows(rng, B * step, H, D, dt), tables, ctx, [step] * B)
        st.same()


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_append_edges(kind):
    rng = np.random.default_rng(5)
    H, D = 2, 64
    # lengths 0 and below are padding; a context shorter than its new tokens; exactly one block; a table's last slot
    ctx = [0, -3, 2, 16, 32, 47]
    tables, nb = tables_for(rng, ctx, extra_cols=0)
    st = State(rng, kind, nb, H, D)
    st.append(rows(rng, 6 * 4, H, D, "bf16"), rows(rng, 6 * 4, H, D, "bf16"), tables, ctx, [4] * 6)
    st.same()
    # zeros: scale 0 and code 0, and what follows them in the block takes over
    k, v = rows(rng, 6 * 1, H, D, "bf16"), rows(rng, 6 * 1, H, D, "bf16")
    k[0].zero_()
    k[1][:] = 0
    ctx = [1, 0, 3, 17, 33, 48]
    tables, nb = tables_for(rng, ctx, extra_cols=0)
    st = State(rng, kind, nb, H, D)
    st.append(k, v, tables, [c - 1 if c > 1 else c for c in ctx], [1] * 6)
    st.append(rows(rng, 6, H, D, "bf16"), rows(rng, 6, H, D, "bf16"), tables, ctx, [1] * 6)
    st.same()
    # very small and very large values
    for size in (1e-38, 1e-30, 3e38):
        st = State(rng, kind, nb, H, D)
        x = torch.rand(6, H, D, generator=torch.Generator().manual_seed(3)).mul(size).to(torch.bfloat16)
        st.append((x.cuda(), x.double().numpy()), (x.cuda(), x.double().numpy()), tables, ctx, [1] * 6)
        st.same()


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_append_bad_tables_and_lengths(kind):
    rng = np.random.default_rng(6)
    H, D = 2, 64
    ctx = [20, 40, 60]
    tables, nb = tables_for(rng, ctx, extra_cols=0)
    tables[0, 1] = nb           # out of range: its tokens are skipped
    tables[1, 1] = -1
    st = State(rng, kind, nb, H, D)
    new = [20, 30, 10]
    cu = [0, 20, 50, 60]
    st.append(rows(rng, 60, H, D, "f16"), rows(rng, 60, H, D, "f16"), tables, ctx, new, cu=cu, expect=0x1)
    st.same()
    # longer than the table: the tokens past it are skipped
    st = State(rng, kind, nb, H, D)
    tables, nb = tables_for(rng, ctx, extra_cols=0)
    st = State(rng, kind, nb, H, D)
    st.append(rows(rng, 60, H, D, "f16"), rows(rng, 60, H, D, "f16"), tables, [20, 40, 70], [0, 40, 20], cu=[0, 0, 40, 60],
              expect=0x4)
    st.same()
    # row offsets that overrun num_tokens or fall: bounded by num_tokens, nothing written outside it
    st = State(rng, kind, nb, H, D)
    k = rows(rng, 10, H, D, "f16")
    st.append(k, k, tables, [20, 40, 60], [4, 6, 0], cu=[0, 4, 30, 2])
    st.same()


def test_append_many_sequences():
    # more sequences than a warp has lanes, most without a new token: the unit search
    rng = np.random.default_rng(7)
    H, D, B = 1, 64, 1500
    new = [int(x) for x in rng.choice([0, 0, 1, 2, 17, 40], B)]
    ctx = [n + int(rng.integers(0, 20)) if n else 0 for n in new]
    tables, nb = tables_for(rng, ctx)
    st = State(rng, "i8", nb, H, D)
    for t, want in ((st.cache.k_scale, st.ks), (st.cache.v_scale, st.vs)):
        t.fill_(0.01)
        want[:] = np.float32(0.01)
    n = sum(new)
    st.append(rows(rng, n, H, D, "bf16", 1.0), rows(rng, n, H, D, "bf16", 1.0), tables, ctx, new,
              cu=np.concatenate([[0], np.cumsum(new)]))
    st.same()


def test_append_rows_of_a_packed_projection():
    # k and v as views of one [tokens, (heads + 2 kv heads) * head_dim] tensor: the same codes as from copies
    rng = np.random.default_rng(9)
    H, D, ctx = 2, 64, [5, 18, 1, 33]
    tables, nb = tables_for(rng, ctx)
    n = sum(ctx)
    cu = np.concatenate([[0], np.cumsum(ctx)])
    x = torch.from_numpy(rng.standard_normal((n, 7 * D))).to(torch.bfloat16).cuda()
    k, v = x[:, 3 * D:5 * D].unflatten(1, (H, D)), x[:, 5 * D:].unflatten(1, (H, D))
    st = State(rng, "i8", nb, H, D)
    st.append((k, k.double().cpu().numpy()), (v, v.double().cpu().numpy()), tables, ctx, ctx, cu=cu)
    st.same()
    # one token: any stride
    st = State(rng, "e4m3", nb, H, D)
    one = (k[:1], k[:1].double().cpu().numpy())
    st.append(one, one, tables[:1], [1], [1])
    st.same()


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_gather_dequant(kind, dt):
    rng = np.random.default_rng(8)
    H, D = 3, 128
    ctx = [1, 0, 16, 17, 130]
    tables, nb = tables_for(rng, ctx)
    st = State(rng, kind, nb, H, D)
    n = sum(ctx)
    cu = np.concatenate([[0], np.cumsum(ctx)])
    seqs = st.append(rows(rng, n, H, D, dt, 1.0), rows(rng, n, H, D, dt, 1.0), tables, ctx, ctx, cu=cu)
    k, v = GuardedOut((n, H, D), SRC[dt], "cuda"), GuardedOut((n, H, D), SRC[dt], "cuda")
    ops.pkv_gather_kv_cache_dequant(k.out, v.out, torch.tensor(cu, dtype=torch.int32, device="cuda"), st.cache, seqs, st.err)
    assert int(st.err.item()) == 0
    for g, codes, scale in ((k, st.kc, st.ks), (v, st.vc, st.vs)):
        g.check()
        want = np.concatenate([R.stored(codes, scale, tables, s, c) for s, c in enumerate(ctx)])
        # code * scale has at most 10 significant bits, so fp32 holds it exactly and one rounding is left
        assert torch.equal(g.out.cpu(), torch.from_numpy(want).float().to(SRC[dt]))


@pytest.mark.parametrize("H,D", [(1, 64), (3, 64), (8, 64), (17, 128), (40, 128)])
@pytest.mark.parametrize("offset", [0, 8])
def test_gather_dequant_rows_of_all_widths_and_alignments(H, D, offset):
    """Blocks of a part, of one and of several CTAs; outputs on a 32-byte boundary and 16 bytes off it."""
    rng = np.random.default_rng(9)
    ctx = [33, 16, 5]
    tables, nb = tables_for(rng, ctx)
    st = State(rng, "i8", nb, H, D)
    n = sum(ctx)
    cu = np.concatenate([[0], np.cumsum(ctx)])
    seqs = st.append(rows(rng, n, H, D, "bf16", 1.0), rows(rng, n, H, D, "bf16", 1.0), tables, ctx, ctx, cu=cu)
    held = [torch.full((n * H * D + 64,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    k, v = (x[offset:offset + n * H * D].view(n, H, D) for x in held)
    ops.pkv_gather_kv_cache_dequant(k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), st.cache, seqs, st.err)
    assert int(st.err.item()) == 0
    for got, whole, codes, scale in ((k, held[0], st.kc, st.ks), (v, held[1], st.vc, st.vs)):
        want = np.concatenate([R.stored(codes, scale, tables, s, c) for s, c in enumerate(ctx)])
        assert torch.equal(got.cpu(), torch.from_numpy(want).float().to(torch.bfloat16))
        assert (whole[:offset] == 7.0).all() and (whole[offset + n * H * D:] == 7.0).all()


# ---------------------------------------------------------------- attention

CTX = [1, 15, 16, 17, 40, 100, 301, 0, 64]


def filled(rng, kind, ctx, H, D, dt="bf16"):
    tables, nb = tables_for(rng, ctx)
    st = State(rng, kind, nb, H, D)
    n = int(sum(max(c, 0) for c in ctx))
    cu = np.concatenate([[0], np.cumsum([max(c, 0) for c in ctx])])
    seqs = st.append(rows(rng, n, H, D, dt, 1.0), rows(rng, n, H, D, dt, 1.0), tables, ctx, [max(c, 0) for c in ctx], cu=cu)
    st.tables = tables
    return st, seqs


def want_attention(st, qr, ctx, q_len, scale, **more):
    k = [R.stored(st.kc, st.ks, st.tables, s, max(int(c), 0)) for s, c in enumerate(ctx)]
    v = [R.stored(st.vc, st.vs, st.tables, s, max(int(c), 0)) for s, c in enumerate(ctx)]
    out, biggest = R.attention(qr, k, v, ctx, q_len, scale, **more)
    return out, biggest, max([1e-30] + [np.abs(x).max() for x in v if x.size])


def close(got, want, biggest, vmax, dtype=torch.float32, p_bits=None):
    # the 8-bit caches' weights: one fp16 operand (half a step: 2^-11) for a bf16 output, hi + lo for the others
    p_bits = p_bits or (11 if dtype == torch.bfloat16 else 22)
    a, r = R.tolerance(biggest, vmax, dtype, p_bits)
    got = got.double().cpu().numpy()
    err = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (err <= a + r * np.abs(want)).all(), f"max err {err.max():.3e}, allowed {a:.3e}"


def attend(st, seqs, q, out, schedule, scale):
    B, Hkv, D = seqs.block_tables.shape[0], st.cache.num_kv_heads, st.cache.head_dim
    if schedule == "single":
        ops.pkv_paged_attention(out, q, scale, st.cache, seqs, st.err)
    elif schedule == "split":
        n = -(-seqs.block_tables.shape[1] * 16 // 48)
        ws = ops.split_workspace(q.shape[0], q.shape[1], D, n)
        ops.pkv_paged_attention_split(*ws, 48, q, scale, st.cache, seqs, st.err)
        ops.pkv_reduce(out, *ws, seqs, 48)
    elif schedule == "noalloc":
        ops.pkv_paged_attention_balanced_noalloc(out, q, scale, st.cache, seqs, st.err)
    else:
        ops.pkv_paged_attention_balanced(out, q, scale, st.cache, seqs, ops.balanced_workspace(B, Hkv, D), st.err)


@pytest.mark.parametrize("schedule", ["single", "split", "balanced", "noalloc"])
@pytest.mark.parametrize("kind,dt,H,Hkv,D,ql", [
    ("i8", "bf16", 8, 2, 128, 1), ("i8", "f16", 4, 4, 64, 1), ("e4m3", "bf16", 16, 2, 64, 1), ("e4m3", "f16", 2, 1, 128, 1),
    ("i8", "bf16", 8, 2, 128, 4), ("e4m3", "bf16", 8, 8, 64, 16), ("i8", "f16", 8, 1, 128, 2), ("e4m3", "f16", 6, 3, 128, 3)])
def test_attention(schedule, kind, dt, H, Hkv, D, ql):
    rng = np.random.default_rng(H * 100 + D + ql)
    ctx = [c if c == 0 else max(c, ql) for c in CTX]
    st, seqs = filled(rng, kind, ctx, Hkv, D)
    seqs.q_len = ql
    q, qr = rows(rng, len(ctx) * ql, H, D, dt, 1.0)
    for odt in (torch.float32, SRC[dt]):
        g = GuardedOut(q.shape, odt, "cuda")
        attend(st, seqs, q, g.out, schedule, D ** -0.5)
        g.check()
        assert int(st.err.item()) == 0
        close(g.out, *want_attention(st, qr, ctx, ql, D ** -0.5), odt)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_attention_window(kind):
    rng = np.random.default_rng(11)
    ctx, D = [5, 16, 100, 300], 128
    st, seqs = filled(rng, kind, ctx, 2, D)
    q, qr = rows(rng, len(ctx), 8, D, "bf16", 1.0)
    for window in (1, 16, 17, 77):
        seqs.sliding_window = window
        for schedule in ("single", "split", "balanced"):
            g = GuardedOut(q.shape, torch.float32, "cuda")
            attend(st, seqs, q, g.out, schedule, D ** -0.5)
            g.check()
            close(g.out, *want_attention(st, qr, ctx, 1, D ** -0.5, window=window))


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_attention_cascade_and_sparse(kind):
    rng = np.random.default_rng(12)
    D, Hkv, H = 128, 2, 8
    ctx = [70, 90, 130, 20]
    st, seqs = filled(rng, kind, ctx, Hkv, D)
    st.tables[1, :4] = st.tables[0, :4]     # the first two share four whole blocks
    seqs.block_tables.copy_(torch.from_numpy(st.tables))
    q, qr = rows(rng, 4, H, D, "bf16", 1.0)
    want = want_attention(st, qr, ctx, 1, D ** -0.5)
    members, blocks = ops.pkv_cascade_plan(seqs.block_tables, seqs.context_lens, 4, min_shared_blocks=1)
    assert members.shape[0] == 1
    g = GuardedOut(q.shape, torch.float32, "cuda")
    ops.pkv_paged_attention_cascade(g.out, q, D ** -0.5, st.cache, seqs, members.cuda(), blocks.cuda(),
                                    ops.cascade_workspace(4, H, Hkv, D, 1, 4), st.err)
    g.check()
    close(g.out, *want)
    lists = torch.tensor([[0, 2, 4, -1], [1, 5, -1, -1], [0, 3, 8, -1], [-1] * 4], dtype=torch.int32)
    counts = torch.tensor([3, 2, 3, 0], dtype=torch.int32)
    g = GuardedOut(q.shape, torch.float32, "cuda")
    ops.pkv_paged_attention_sparse(g.out, q, D ** -0.5, st.cache, seqs, lists.cuda(), counts.cuda(),
                                   ops.sparse_workspace(4, Hkv, D, 4), st.err)
    g.check()
    assert int(st.err.item()) == 0
    k = [R.stored(st.kc, st.ks, st.tables, s, c) for s, c in enumerate(ctx)]
    v = [R.stored(st.vc, st.vs, st.tables, s, c) for s, c in enumerate(ctx)]
    for x in (k, v):
        for s in range(4):
            keep = [t for t in range(ctx[s]) if t // 16 in set(lists[s, :counts[s]].tolist())]
            x[s] = x[s][keep]
    out, biggest = R.attention(qr, k, v, [len(x) for x in k], 1, D ** -0.5)
    close(g.out, out, biggest, want[2])


@pytest.mark.parametrize("size", [1e-36, 1e-6, 1.0, 1e5, 1e30])
def test_queries_of_any_bf16_size(size):
    # the fp16 operand holds a query row scaled by a power of two: the result scales with it
    rng = np.random.default_rng(13)
    ctx, D = [40, 100], 128
    st, seqs = filled(rng, "i8", ctx, 2, D)
    x = rng.standard_normal((2, 4, D))
    t = torch.from_numpy(x * size).to(torch.bfloat16)
    out = torch.empty((2, 4, D), device="cuda")
    attend(st, seqs, t.cuda(), out, "balanced", D ** -0.5 / size)
    close(out, *want_attention(st, t.double().numpy(), ctx, 1, float(np.float32(D ** -0.5 / size))))


def test_long_cache_and_extreme_scales():
    # weights far below fp16's range times a large scale, and scales of very different sizes from block to block
    rng = np.random.default_rng(14)
    ctx, D = [5000], 64
    st, seqs = filled(rng, "e4m3", ctx, 1, D)
    f = 2.0 ** rng.integers(-20, 20, st.vs.shape)
    st.vs = np.where(np.isnan(st.vs), st.vs, (st.vs * f)).astype(np.float32)
    st.cache.v_scale.copy_(torch.from_numpy(st.vs))
    q, qr = rows(rng, 1, 4, D, "f16", 1.0)
    for schedule in ("single", "balanced"):
        out = torch.empty(q.shape, device="cuda")
        attend(st, seqs, q, out, schedule, D ** -0.5)
        close(out, *want_attention(st, qr, ctx, 1, D ** -0.5))


def test_append_and_attention_captured_and_replayed():
    # one graph holds a step's append and attention; each replay takes new contents of the same buffers
    rng = np.random.default_rng(15)
    ctx, D, H, Hkv = [31, 5, 100], 128, 8, 2
    final = [c + 4 for c in ctx]
    tables, nb = tables_for(rng, final)
    st = State(rng, "i8", nb, Hkv, D)
    st.tables = tables
    cu = np.concatenate([[0], np.cumsum(ctx)])
    n = sum(ctx)
    seqs = st.append(rows(rng, n, Hkv, D, "bf16", 1.0), rows(rng, n, Hkv, D, "bf16", 1.0), tables, ctx, ctx, cu=cu)
    kb, vb = (torch.empty((3, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    qb = torch.empty((3, H, D), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((3, H, D), device="cuda")
    ws = ops.balanced_workspace(3, Hkv, D)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        ops.pkv_quantize_kv_blocks(st.cache, kb, vb, seqs, None, st.err)
        ops.pkv_paged_attention_balanced(out, qb, D ** -0.5, st.cache, seqs, ws, st.err)
    for step in range(4):
        ctx = [c + 1 for c in ctx]
        k, v, q = rows(rng, 3, Hkv, D, "bf16"), rows(rng, 3, Hkv, D, "bf16"), rows(rng, 3, H, D, "bf16", 1.0)
        kb.copy_(k[0]); vb.copy_(v[0]); qb.copy_(q[0])
        seqs.context_lens.copy_(torch.tensor(ctx, dtype=torch.int32))
        graph.replay()
        R.append(st.kc, st.vc, st.ks, st.vs, "i8", k[1], v[1], tables, ctx, [1] * 3)
        st.same()
        assert int(st.err.item()) == 0
        close(out, *want_attention(st, q[1], ctx, 1, D ** -0.5))


def test_binding_refuses():
    cache = ops.Cache.empty("i8", 4, 2, 64)
    seqs = ops.Seqs(torch.zeros((2, 1), dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda"), 1)
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        ops.pkv_quantize_kv_blocks(cache, x, x.half(), seqs)
    with pytest.raises(ValueError):
        ops.pkv_quantize_kv_blocks(cache, x[:, :1].contiguous(), x[:, :1].contiguous(), seqs)
    with pytest.raises(ValueError):
        ops.pkv_quantize_kv_blocks(cache, x, x, seqs, torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        ops.pkv_quantize_kv_blocks(cache, x, x.cpu(), seqs)
    with pytest.raises(ValueError):
        ops.pkv_quantize_kv_blocks(cache, x.float(), x.float(), seqs)
    with pytest.raises(ops.PkvError):   # three rows for two sequences of one token
        y = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
        ops.pkv_quantize_kv_blocks(cache, y, y, seqs)
    with pytest.raises(ValueError):
        ops.Cache("i8", cache.k, cache.v, cache.k_scale[:, :1].contiguous(), cache.v_scale).c_struct()
    with pytest.raises(ValueError):
        ops.Cache("e4m3", cache.k, cache.v, cache.k_scale, cache.v_scale).c_struct()
    ws = ops.balanced_workspace(2, 2, 64)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ops.PkvError) as e:
        ops.pkv_decode_step_balanced(torch.empty_like(q), q, 0.125, cache, seqs, x, x,
                                     torch.zeros(2, dtype=torch.int64, device="cuda"), ws)
    assert e.value.status == ops.PKV_ERR_UNSUPPORTED
    for call in (lambda: ops.pkv_reshape_and_cache(cache, x, x, torch.zeros(2, dtype=torch.int64, device="cuda")),
                 lambda: ops.pkv_quantize_kv(cache, x, x, torch.zeros(2, dtype=torch.int64, device="cuda"))):
        with pytest.raises(ops.PkvError):
            call()
