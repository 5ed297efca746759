"""The decode step's operators together, as a model's layer calls them: rotary
positions straight from a packed projection, the cache write (in place for bf16,
the append for the 8-bit caches) and the scored attention, over prompts and then
steps replayed from one graph; calls side by side on two streams; caches whose
offsets pass 32 bits."""
import numpy as np
import pytest
import torch

from paged_decode_attention_cache_gb300 import ops
from tests import blocks_reference as R
from tests.test_gpu_blocks import State, close, rows, tables_for
from tests.test_gpu_rope import turned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_decode_attention_cache_gb300 import build
    build.build()
    ops.lib()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3"])
def test_prompts_then_graph_steps(kind):
    rng = np.random.default_rng(31)
    H, Hkv, D, r = 8, 2, 128, 64
    prompts, steps = [37, 1, 16, 90], 5
    final = [c + steps for c in prompts]
    tables, nb = tables_for(rng, final)
    B, dt = len(prompts), torch.bfloat16
    freq = ops.pkv_rope_frequencies(r, 500000.0, "linear", 4.0)
    rope = ops.Rope(freq.cuda(), r, "half")
    byte = kind != "bf16"
    st = State(rng, kind if byte else "i8", nb, Hkv, D)
    cache = st.cache if byte else ops.Cache("bf16", *(torch.full((nb, 16, Hkv, D), float("nan"), dtype=dt, device="cuda") for _ in "kv"))
    slopes = torch.tensor([2.0 ** -(h + 1) for h in range(H)], device="cuda")
    prefix = torch.tensor([2, 1, 0, 20], dtype=torch.int32, device="cuda")
    scores = ops.Scores(25.0, slopes, None, prefix)
    seqs = ops.Seqs(torch.from_numpy(tables).cuda(), torch.tensor(prompts, dtype=torch.int32, device="cuda"), 1, 48)

    def packed(n):
        x = torch.from_numpy(rng.standard_normal((n, (H + 2 * Hkv) * D)) * 1.5).to(dt).cuda()
        return x, [x[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, H), (H, H + Hkv), (H + Hkv, H + 2 * Hkv))]

    def slot(s, t):
        return int(tables[s, t // 16]) * 16 + t % 16

    # ---- prompts
    n = sum(prompts)
    cu = np.concatenate([[0], np.cumsum(prompts)])
    pos = np.concatenate([np.arange(c) for c in prompts])
    _, (q, k, v) = packed(n)
    q_rot, k_rot = torch.empty(n, H, D, dtype=dt, device="cuda"), torch.empty(n, Hkv, D, dtype=dt, device="cuda")
    slots = torch.tensor([slot(s, t) for s, c in enumerate(prompts) for t in range(c)], device="cuda")
    where = dict(cache=None, slot_mapping=None) if byte else dict(cache=cache, slot_mapping=slots)
    ops.pkv_rope_and_cache(q_rot, q, k, v, rope, torch.from_numpy(pos).cuda(), k_out=k_rot, err_flags=st.err, **where)
    want, size = turned(k.double().cpu().numpy(), pos, freq.tolist(), r, "half", 1.0)
    assert (np.abs(k_rot.double().cpu().numpy() - want) <= 2.0 ** -20 * size + 2.0 ** -8 * np.abs(want)).all()
    history = [([k_rot[cu[s]:cu[s + 1]].double().cpu().numpy()], [v[cu[s]:cu[s + 1]].double().cpu().numpy()]) for s in range(B)]
    if byte:
        ops.pkv_quantize_kv_blocks(cache, k_rot, v, seqs, torch.tensor(cu, dtype=torch.int32, device="cuda"), st.err)
        R.append(st.kc, st.vc, st.ks, st.vs, kind, k_rot.double().cpu().numpy(), v.double().cpu().numpy(), tables, prompts, prompts)
        st.same()

    # ---- steps: one graph, new contents of its buffers each time
    x, (q, k, v) = packed(B)
    pos_d, slot_d = torch.zeros(B, dtype=torch.int64, device="cuda"), torch.zeros(B, dtype=torch.int64, device="cuda")
    k_out, out = torch.empty(B, Hkv, D, dtype=dt, device="cuda"), torch.empty(B, H, D, device="cuda")
    q_out = torch.empty(B, H, D, dtype=dt, device="cuda")   # the attention takes contiguous queries
    ws = ops.balanced_workspace(B, Hkv, D)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if byte:
            ops.pkv_rope_and_cache(q_out, q, k, v, rope, pos_d, None, None, k_out, st.err)
            ops.pkv_quantize_kv_blocks(cache, k_out, v, seqs, None, st.err)
        else:
            ops.pkv_rope_and_cache(q_out, q, k, v, rope, pos_d, cache, slot_d, k_out, st.err)
        ops.pkv_paged_attention_scored(out, q_out, D ** -0.5, cache, seqs, scores, ws, st.err)
    ctx = list(prompts)
    for _ in range(steps):
        x.copy_(packed(B)[0])
        pos_d.copy_(torch.tensor(ctx))
        slot_d.copy_(torch.tensor([slot(s, c) for s, c in enumerate(ctx)]))
        ctx = [c + 1 for c in ctx]
        seqs.context_lens.copy_(torch.tensor(ctx, dtype=torch.int32))
        graph.replay()
        assert int(st.err.item()) == 0
        for s in range(B):
            history[s][0].append(k_out[s:s + 1].double().cpu().numpy())
            history[s][1].append(v[s:s + 1].double().cpu().numpy())
        if byte:
            R.append(st.kc, st.vc, st.ks, st.vs, kind, k_out.double().cpu().numpy(), v.double().cpu().numpy(), tables, ctx, [1] * B)
            st.same()
            K = [R.stored(st.kc, st.ks, tables, s, c) for s, c in enumerate(ctx)]
            V = [R.stored(st.vc, st.vs, tables, s, c) for s, c in enumerate(ctx)]
        else:
            K, V = ([np.concatenate(h[i]) for h in history] for i in (0, 1))
        want, biggest = R.attention(q_out.double().cpu().numpy(), K, V, ctx, 1, D ** -0.5, 48, 25.0, slopes.tolist(), None, prefix.tolist())
        close(out, want, biggest, max(np.abs(y).max() for y in V), p_bits=22 if byte else 17)


def test_two_streams_at_once():
    # calls with workspaces of their own may overlap; a cache may be read by both
    rng = np.random.default_rng(32)
    H, Hkv, D, ctx = 8, 2, 128, [900, 30, 2000, 1]
    tables, nb = tables_for(rng, ctx)
    st = State(rng, "e4m3", nb, Hkv, D)
    n = sum(ctx)
    seqs = st.append(rows(rng, n, Hkv, D, "bf16", 1.0), rows(rng, n, Hkv, D, "bf16", 1.0), tables, ctx, ctx,
                     cu=np.concatenate([[0], np.cumsum(ctx)]))
    qs = [rows(rng, len(ctx), H, D, "bf16", 1.0)[0] for _ in range(2)]
    outs = [[torch.empty((len(ctx), H, D), device="cuda") for _ in range(2)] for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [ops.balanced_workspace(len(ctx), Hkv, D) for _ in range(2)]
    for i in range(2):
        ops.pkv_paged_attention_scored(outs[0][i], qs[i], D ** -0.5, st.cache, seqs, ops.Scores(20.0 * i), ws[i])
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                ops.pkv_paged_attention_scored(outs[1][i], qs[i], D ** -0.5, st.cache, seqs, ops.Scores(20.0 * i), ws[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[0][i], outs[1][i])


@pytest.mark.parametrize("kind", ["i8", "bf16"])
def test_offsets_past_32_bits(kind):
    # a pool of more than 2^32 bytes for K and for V, the sequence's blocks at both of its ends
    H, Hkv, D, c = 8, 8, 128, 40
    nb = 2 ** 32 // (16 * Hkv * D * (1 if kind == "i8" else 2)) + 16
    cache = ops.Cache.empty(kind, nb, Hkv, D)
    tables = torch.tensor([[nb - 1, 0, nb - 2, 5]], dtype=torch.int32, device="cuda")
    seqs = ops.Seqs(tables, torch.tensor([c], dtype=torch.int32, device="cuda"))
    rng = np.random.default_rng(33)
    (k, kr), (v, vr), (q, qr) = (rows(rng, n, Hkv, D, "bf16", 1.0) for n in (c, c, 1))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if kind == "i8":
        ops.pkv_quantize_kv_blocks(cache, k, v, seqs, torch.tensor([0, c], dtype=torch.int32, device="cuda"), err)
        local = np.arange(3)[None, :]
        kc, vc = np.zeros((3, 16, Hkv, D)), np.zeros((3, 16, Hkv, D))
        ks, vs = np.zeros((3, Hkv), np.float32), np.zeros((3, Hkv), np.float32)
        R.append(kc, vc, ks, vs, kind, kr, vr, local, [c], [c])
        used = tables[0, :3].long()
        assert np.array_equal(R.values(cache.k[used], kind), kc) and np.array_equal(R.values(cache.v[used], kind), vc)
        K, V = R.stored(kc, ks, local, 0, c), R.stored(vc, vs, local, 0, c)
        ko, vo = (torch.empty((c, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
        ops.pkv_gather_kv_cache_dequant(ko, vo, torch.tensor([0, c], dtype=torch.int32, device="cuda"), cache, seqs, err)
        assert torch.equal(ko.cpu(), torch.from_numpy(K).float().bfloat16()) and torch.equal(vo.cpu(), torch.from_numpy(V).float().bfloat16())
    else:
        rope = ops.Rope(ops.pkv_rope_frequencies(D, 10000.0).cuda(), D)
        slots = torch.tensor([int(tables[0, t // 16]) * 16 + t % 16 for t in range(c)], device="cuda")
        k_out = torch.empty_like(k)
        ops.pkv_rope_and_cache(torch.empty((c, 1, D), dtype=torch.bfloat16, device="cuda"), k[:, :1], k, v, rope,
                               torch.arange(c, device="cuda"), cache, slots, k_out, err)
        assert torch.equal(cache.k.view(-1, Hkv, D)[slots], k_out) and torch.equal(cache.v.view(-1, Hkv, D)[slots], v)
        K, V = k_out.double().cpu().numpy(), vr
    out = torch.empty((1, H, D), device="cuda")
    ops.pkv_paged_attention_scored(out, q, D ** -0.5, cache, seqs, ops.Scores(30.0), ops.balanced_workspace(1, Hkv, D), err)
    assert int(err.item()) == 0
    want, biggest = R.attention(qr, [K], [V], [c], 1, D ** -0.5, 0, 30.0)
    close(out, want, biggest, np.abs(V).max(), p_bits=22 if kind == "i8" else 17)
