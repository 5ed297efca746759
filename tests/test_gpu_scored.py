"""Attention with capped and distance-biased scores and document / prefix masks,
over every cache kind, against a plain 64-bit restatement.  Tokens that a mask
leaves out hold NaN and infinities (their scales, in the quantised caches), and so
does every slot past a context."""
import numpy as np
import pytest
import torch

from paged_decode_attention_cache_gb300 import ops
from tests import blocks_reference as R
from tests.helpers import GuardedOut
from tests.test_gpu_blocks import State, close, rows, tables_for

pytestmark = pytest.mark.gpu
SRC = {"bf16": torch.bfloat16, "f16": torch.float16}
P_BITS = {"bf16": 17, "f16": 22}   # 8-bit caches: close() goes by the output type
K8V4_ABS = 2e-2


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_decode_attention_cache_gb300 import build
    build.build()
    ops.lib()
    torch.cuda.set_device(0)


def masked_out(ctx, window, starts, prefix):
    """Per sequence, which stored tokens no row may see."""
    out = []
    for s, c in enumerate(ctx):
        at = np.arange(max(c, 0))
        lo = max(0, c - window) if window else 0
        if starts is not None:
            lo = max(lo, min(max(int(starts[s]), 0), max(c, 0)))
        out.append((at < lo) & ~(at < (0 if prefix is None else int(prefix[s]))))
    return out


def make(rng, kind, ctx, Hkv, D, hidden, dt):
    """(cache, block tables, per-sequence K, V in float64); what `hidden` names is poisoned in the device cache."""
    tables, nb = tables_for(rng, ctx)
    n = int(sum(max(c, 0) for c in ctx))
    cu = np.concatenate([[0], np.cumsum([max(c, 0) for c in ctx])])
    if kind in ("i8", "e4m3"):
        st = State(rng, kind, nb, Hkv, D)
        st.append(rows(rng, n, Hkv, D, dt, 1.0), rows(rng, n, Hkv, D, dt, 1.0), tables, ctx, [max(c, 0) for c in ctx], cu=cu)
        k, v = ([R.stored(c, x, tables, s, max(ctx[s], 0)) for s in range(len(ctx))] for c, x in ((st.kc, st.ks), (st.vc, st.vs)))
        for s, h in enumerate(hidden):
            for b in range(-(-len(h) // 16)):
                if h[16 * b:16 * b + 16].all():   # the block is never read
                    st.cache.k_scale[tables[s, b]] = float("nan")
                    st.cache.v_scale[tables[s, b]] = float("inf")
        return st.cache, tables, k, v
    x = [rng.standard_normal((n, Hkv, D)) * (2 if i == 0 else 1) for i in range(2)]
    x = [torch.from_numpy(y).to(SRC[dt] if kind == "k8v4" else SRC[kind]) for y in x]
    slots = np.concatenate([[int(tables[s, t // 16]) * 16 + t % 16 for t in range(max(c, 0))] for s, c in enumerate(ctx)] or [[]])
    slots = torch.from_numpy(slots.astype(np.int64)).cuda()
    cache = ops.Cache.empty(kind, nb, Hkv, D)
    bad = torch.from_numpy(np.concatenate([np.zeros(0, bool)] + list(hidden))).cuda()
    if kind == "k8v4":
        for t in (cache.k_scale, cache.v_scale, cache.v_zero):
            t.fill_(float("nan"))
        ops.pkv_quantize_kv(cache, x[0].cuda(), x[1].cuda(), slots)
        k, v = (torch.empty((n, Hkv, D), dtype=torch.float16, device="cuda") for _ in "kv")
        seqs = ops.Seqs(torch.from_numpy(tables).cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"))
        ops.pkv_gather_kv_cache_dequant(k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), cache, seqs)
        x = [k.cpu(), v.cpu()]
        b, o = slots[bad] // 16, slots[bad] % 16
        cache.k_scale.transpose(1, 2)[b, o] = float("nan")
        cache.v_scale.transpose(1, 2)[b, o] = float("inf")
        cache.v_zero.transpose(1, 2)[b, o] = float("nan")
    else:
        for t, y in ((cache.k, x[0]), (cache.v, x[1])):
            t.fill_(float("nan"))
            flat = t.view(nb * 16, Hkv, D)
            flat[slots] = y.cuda()
            flat[slots[bad]] = float("inf") if t is cache.v else float("nan")
    cut = [[y[cu[s]:cu[s + 1]].double().numpy() for s in range(len(ctx))] for y in x]
    return cache, tables, cut[0], cut[1]


def run(rng, kind, dt, ctx, H, Hkv, D, ql, window=0, cap=0.0, slopes=None, starts=None, prefix=None, loud=3.0, out_dtypes=None):
    hidden = masked_out(ctx, window, starts, prefix)
    cache, tables, k, v = make(rng, kind, ctx, Hkv, D, hidden, dt)
    for x in (k, v):
        for s, h in enumerate(hidden):
            x[s][h] = 0.0     # the reference masks them too; no NaN arithmetic there
    B = len(ctx)
    q, qr = rows(rng, B * ql, H, D, dt, 0.5)
    q, qr = q * loud, (q * loud).double().cpu().numpy()
    as_int = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    scores = ops.Scores(cap, None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device="cuda"),
                        as_int(starts), as_int(prefix))
    seqs = ops.Seqs(torch.from_numpy(tables).cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"), ql, window)
    ws = ops.balanced_workspace(B, Hkv, D)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    scale = D ** -0.5
    want, biggest = R.attention(qr, k, v, ctx, ql, scale, window, float(np.float32(cap)), slopes, starts, prefix)
    vmax = max([1e-30] + [np.abs(x).max() for x in v if x.size])
    for odt in out_dtypes or (torch.float32, SRC[dt]):
        g = GuardedOut(q.shape, odt, "cuda")
        for _ in range(2):      # the workspace comes back ready
            ops.pkv_paged_attention_scored(g.out, q, scale, cache, seqs, scores, ws, err)
        g.check()
        assert int(err.item()) == 0
        if kind == "k8v4":
            got = g.out.double().cpu().numpy()
            assert np.isfinite(got).all() and np.abs(got - want).max() <= K8V4_ABS
        else:
            close(g.out, want, biggest, vmax, odt, P_BITS.get(kind))
    return g.out, (q, cache, seqs, ws)


CTX = [1, 15, 16, 17, 40, 100, 301, 0, 64, 700]
SHAPES = [("bf16", "bf16", 8, 2, 128, 1), ("f16", "f16", 4, 4, 64, 1), ("f16", "f16", 2, 1, 128, 1), ("bf16", "bf16", 16, 2, 64, 2),
          ("f16", "f16", 8, 2, 128, 2), ("k8v4", "bf16", 8, 2, 128, 1), ("k8v4", "f16", 8, 1, 64, 2), ("i8", "bf16", 8, 2, 128, 1),
          ("e4m3", "f16", 8, 8, 64, 1), ("i8", "f16", 8, 1, 64, 2), ("e4m3", "bf16", 6, 3, 128, 5)]


def slopes_of(H):
    return [float(np.float32(2.0 ** (-8.0 * (h + 1) / H))) for h in range(H)]


@pytest.mark.parametrize("kind,dt,H,Hkv,D,ql", SHAPES)
def test_cap(kind, dt, H, Hkv, D, ql):
    ctx = [c if c == 0 else max(c, ql) for c in CTX]
    for cap in (0.5, 20.0, 50.0, 1e6):     # nearly all capped, some, few, none
        run(np.random.default_rng(H + D + ql), kind, dt, ctx, H, Hkv, D, ql, cap=cap)


@pytest.mark.parametrize("kind,dt,H,Hkv,D,ql", SHAPES)
def test_distance_bias(kind, dt, H, Hkv, D, ql):
    ctx = [c if c == 0 else max(c, ql) for c in CTX]
    s = slopes_of(H)
    run(np.random.default_rng(H + D + ql + 1), kind, dt, ctx, H, Hkv, D, ql, slopes=s, loud=1.0)
    s[0], s[-1] = 0.0, -0.01     # a head without a bias, one that favours far tokens
    run(np.random.default_rng(H + D + ql + 2), kind, dt, ctx, H, Hkv, D, ql, slopes=s, cap=30.0, loud=1.0)


@pytest.mark.parametrize("kind,dt,H,Hkv,D,ql", SHAPES)
@pytest.mark.parametrize("window", [0, 1, 33])
def test_masks(kind, dt, H, Hkv, D, ql, window):
    rng = np.random.default_rng(H + D + ql + window)
    ctx = [c if c == 0 else max(c, ql) for c in CTX]
    # a document that begins at the start, inside a block, at a block's edge, at the last token, past the end, before 0
    starts = [0, 7, 16, 16, 25, 96, 300, 3, 64, -5]
    prefix = [0, 3, 16, 1, 17, 40, 33, 5, 2, 16]
    run(rng, kind, dt, ctx, H, Hkv, D, ql, window=window, starts=starts)
    run(rng, kind, dt, ctx, H, Hkv, D, ql, window=window, prefix=prefix)
    run(rng, kind, dt, ctx, H, Hkv, D, ql, window=window, starts=starts, prefix=prefix, cap=25.0, slopes=slopes_of(H), loud=1.0)


@pytest.mark.parametrize("kind", ["bf16", "f16", "i8", "e4m3", "k8v4"])
def test_nothing_visible_and_everything_prefix(kind):
    rng = np.random.default_rng(20)
    ctx = [5, 33, 64, 0]
    out, _ = run(rng, kind, "f16" if kind == "f16" else "bf16", ctx, 8, 2, 64, 1, starts=[5, 40, 64, 1])
    assert int((out != 0).sum()) == 0
    run(rng, kind, "f16" if kind == "f16" else "bf16", ctx, 8, 2, 64, 1, starts=[5, 40, 64, 1], prefix=[9, 33, 1, 4])
    run(rng, kind, "f16" if kind == "f16" else "bf16", ctx, 8, 2, 64, 1, window=4, prefix=[100, 100, 100, 100])


@pytest.mark.parametrize("kind", ["bf16", "i8"])
def test_long_and_split_over_many_ctas(kind):
    rng = np.random.default_rng(21)
    ctx = [20000, 3]
    run(rng, kind, "bf16", ctx, 8, 2, 128, 1, cap=50.0, window=5000, prefix=[100, 1])
    run(rng, kind, "bf16", ctx, 8, 2, 128, 1, starts=[11111, 0], slopes=slopes_of(8), loud=1.0)
    run(rng, kind, "bf16", ctx, 8, 2, 128, 1, cap=30.0)


def test_many_sequences_of_all_kinds():
    # more sequences than a CTA has threads, most of them short, empty or hidden
    rng = np.random.default_rng(22)
    ctx = [int(x) for x in rng.choice([0, 1, 5, 16, 30, 80], 700)]
    starts = [int(x) for x in rng.integers(0, 40, 700)]
    prefix = [int(x) for x in rng.choice([0, 0, 1, 20], 700)]
    run(rng, "bf16", "bf16", ctx, 4, 1, 64, 1, window=50, starts=starts, prefix=prefix, cap=20.0, slopes=slopes_of(4), loud=1.0)


@pytest.mark.parametrize("D,ql", [(64, 1), (128, 1), (128, 4)])
def test_nan_codes_of_masked_tokens_beside_visible_ones(D, ql):
    """e4m3: a block holds masked and visible tokens; the masked ones' codes turn to NaN and nothing changes."""
    rng = np.random.default_rng(41 + ql)
    ctx, starts, prefix, H, Hkv = [100, 37, 64, 5, 333], [41, 36, 3, 2, 300], [5, 20, 1, 0, 17], 8, 2
    hidden = masked_out(ctx, 0, starts, prefix)
    cache, tables, _, _ = make(rng, "e4m3", ctx, Hkv, D, [np.zeros_like(h) for h in hidden], "bf16")
    q, _ = rows(rng, len(ctx) * ql, H, D, "bf16", 0.5)
    as_int = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    seqs = ops.Seqs(torch.from_numpy(tables).cuda(), as_int(ctx), ql, 0)
    scores, ws = ops.Scores(30.0, None, as_int(starts), as_int(prefix)), ops.balanced_workspace(len(ctx), Hkv, D)
    outs = [torch.full_like(q, float("nan")) for _ in range(2)]
    ops.pkv_paged_attention_scored(outs[0], q, D ** -0.5, cache, seqs, scores, ws)
    for t in (cache.k, cache.v):
        codes = t.view(torch.uint8)
        for s, h in enumerate(hidden):
            for at in np.nonzero(h)[0]:
                codes[int(tables[s, at // 16]), int(at % 16)] = 0x7f
    ops.pkv_paged_attention_scored(outs[1], q, D ** -0.5, cache, seqs, scores, ws)
    assert torch.isfinite(outs[0]).all() and torch.equal(*outs)


def test_without_scores_it_is_the_balanced_attention():
    rng = np.random.default_rng(23)
    for kind in ("bf16", "i8"):
        out, (q, cache, seqs, ws) = run(rng, kind, "bf16", CTX, 8, 2, 128, 1, out_dtypes=(torch.float32,))
        plain = torch.empty_like(out)
        ops.pkv_paged_attention_balanced(plain, q, 128 ** -0.5, cache, seqs, ws)
        assert torch.equal(out, plain)


def test_infinite_keys_are_capped():
    # a cap makes an infinite score finite: the token's weight is the cap's
    ctx, D = [20], 64
    k = torch.zeros((2, 16, 1, D), dtype=torch.float16, device="cuda")
    v = torch.randn((2, 16, 1, D), device="cuda").half()
    k[0, 3, 0, 0] = float("inf")
    k[0, 5, 0, 0] = float("-inf")
    q = torch.zeros((1, 4, D), dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    out = torch.empty((1, 4, D), device="cuda")
    seqs = ops.Seqs(torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), torch.tensor(ctx, dtype=torch.int32, device="cuda"))
    ops.pkv_paged_attention_scored(out, q, 1.0, ops.Cache("f16", k, v), seqs, ops.Scores(2.0), ops.balanced_workspace(1, 1, D))
    w = torch.ones(20, dtype=torch.float64)
    w[3], w[5] = np.exp(2.0), np.exp(-2.0)
    want = (w / w.sum()) @ v.cpu().double().view(32, D)[:20]
    assert (out[0].double().cpu() - want).abs().max() <= 2.0 ** -18 * float(v.abs().max())


def test_capture_and_new_masks():
    # the masks' values are read on the device: a replay takes the buffers' new contents
    rng = np.random.default_rng(24)
    ctx, H, Hkv, D = [40, 100, 64], 8, 2, 128
    none = [np.zeros(c, bool) for c in ctx]
    cache, tables, k, v = make(rng, "bf16", ctx, Hkv, D, none, "bf16")
    q, qr = rows(rng, 3, H, D, "bf16", 0.5)
    starts, prefix = (torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2))
    seqs = ops.Seqs(torch.from_numpy(tables).cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"))
    out, ws = torch.empty((3, H, D), device="cuda"), ops.balanced_workspace(3, Hkv, D)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.pkv_paged_attention_scored(out, q, D ** -0.5, cache, seqs, ops.Scores(20.0, None, starts, prefix), ws)
    for a, b in (([0, 0, 0], [0, 0, 0]), ([39, 50, 64], [0, 3, 0]), ([5, 200, 1], [1, 1, 1])):
        starts.copy_(torch.tensor(a, dtype=torch.int32))
        prefix.copy_(torch.tensor(b, dtype=torch.int32))
        graph.replay()
        want, biggest = R.attention(qr, k, v, ctx, 1, D ** -0.5, 0, 20.0, None, a, b)
        close(out, want, biggest, max(np.abs(x).max() for x in v), p_bits=17)


def test_bad_blocks_and_long_contexts_are_flagged():
    rng = np.random.default_rng(25)
    ctx, D = [40, 40], 64
    cache, tables, k, v = make(rng, "f16", ctx, 1, D, [np.zeros(c, bool) for c in ctx], "f16")
    tables[0, 1] = 10 ** 6
    q, qr = rows(rng, 2, 4, D, "f16", 0.5)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, ws = torch.empty((2, 4, D), device="cuda"), ops.balanced_workspace(2, 1, D)
    seqs = ops.Seqs(torch.from_numpy(tables).cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"))
    ops.pkv_paged_attention_scored(out, q, 0.125, cache, seqs, ops.Scores(20.0), ws, err)
    assert int(err.item()) == ops.DEVERR_OOB_BLOCK
    want, biggest = R.attention(qr[1:], k[1:], v[1:], ctx[1:], 1, 0.125, 0, 20.0)
    close(out[1:], want, biggest, np.abs(v[1]).max())


def test_binding_refuses():
    H, Hkv, D, B = 8, 2, 64, 3
    cache = ops.Cache.empty("f16", 4, Hkv, D)
    seqs = ops.Seqs(torch.zeros((B, 1), dtype=torch.int32, device="cuda"), torch.ones(B, dtype=torch.int32, device="cuda"))
    q = torch.zeros((B, H, D), dtype=torch.float16, device="cuda")
    ws = ops.balanced_workspace(B, Hkv, D)
    call = lambda scores, **c: ops.pkv_paged_attention_scored(**{**dict(out=q.clone(), q=q, scale=1.0, cache=cache, seqs=seqs,  # noqa: E731
                                                                        scores=scores, workspace=ws), **c})
    ints = torch.zeros(B, dtype=torch.int32, device="cuda")
    call(ops.Scores(1.0, torch.zeros(H, device="cuda"), ints, ints))
    for bad in (ops.Scores(1.0, torch.zeros(H - 1, device="cuda")), ops.Scores(1.0, torch.zeros(H, device="cuda").half()),
                ops.Scores(1.0, None, ints[:2]), ops.Scores(1.0, None, ints.long()), ops.Scores(1.0, None, None, ints[:1]),
                ops.Scores(1.0, None, ints.cpu())):
        with pytest.raises(ValueError):
            call(bad)
    for cap in (-1.0, float("nan"), float("inf"), 1e-35):
        with pytest.raises(ops.PkvError):
            call(ops.Scores(cap))
    for change in (dict(q=q[:2]), dict(out=q[:, :4].contiguous()), dict(out=q.cpu()),
                   dict(seqs=ops.Seqs(seqs.block_tables, seqs.context_lens, 2))):
        with pytest.raises(ValueError):
            call(ops.Scores(1.0), **change)
    with pytest.raises(ops.PkvError):
        call(ops.Scores(1.0), workspace=ws[:256])
