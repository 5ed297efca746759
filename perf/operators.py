"""Cases of the operators around a decode step's attention: rotary positions
with the cache write, the 8-bit cache with one scale per block and kv head
(append, attention, read-back), and attention whose scores are capped, biased
by distance or masked by document and prefix.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, angles in 64) or, where ``own`` is true, through the library's entry
points.  Sequence lengths follow from the case alone, values from the seed.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
QMAX = {"i8": 127.0, "e4m3": 448.0}


# ---------------------------------------------------------------- the cases


def listed():
    return [
        # one user's next token in an 8B-like model: nothing but latency
        rope("rope_decode_1", 1, 32, 8, 128, 128, "half", "bf16", "none", 8192, False),
        # a wide decode batch of a small model that rotates half of each head, pairs side by side
        rope("rope_decode_256_part", 256, 16, 4, 64, 32, "interleaved", "f16", "linear", 32768, True),
        # a chunk of prompts far into a long context, straight from a packed q/k/v projection
        rope("rope_prompt_8192_far", 8192, 32, 8, 128, 128, "half", "bf16", "by_parts", 131072, True),
        # one short chat on an int8 cache
        attend("blocks_short_1", "i8", "bf16", 1, 300, 8, 2, 64, 1),
        # a serving batch of mixed lengths on an e4m3 cache
        attend("blocks_batch_32", "e4m3", "bf16", 32, 4096, 32, 8, 128, 1),
        # a few long documents, two drafted tokens each to verify
        attend("blocks_long_8_verify", "i8", "f16", 8, 65536, 32, 8, 128, 2),
        # the next chunk of prompts stored behind what the sequences hold, then read back for the chunk's own attention
        store("blocks_store_prompts", "i8", "bf16", 7, 2500, 777, 8, 128),
        # one decode step on an e4m3 cache: the new tokens' append, then the attention over everything
        step("blocks_step_64", "e4m3", "bf16", 64, 1500, 32, 8, 128),
        # the library's batch of 8 with capped scores
        scored("scored_cap_8", "bf16", "bf16", 8, 4096, 32, 8, 128, 1, 50.0, False, 0, 0, False),
        # verify blocks of 4 drafts with a bias that falls with distance (every head its own K/V)
        scored("scored_distance_verify_16", "f16", "f16", 16, 1024, 8, 8, 64, 4, 0.0, True, 0, 0, False),
        # long sequences that keep a prefix and the last window
        scored("scored_prefix_window_32k", "bf16", "bf16", 4, 32768, 32, 8, 128, 1, 30.0, False, 4096, 40, False),
        # packed documents on an int8 cache, capped and biased; one sequence's document has not begun
        scored("scored_documents_i8_32", "i8", "bf16", 32, 6000, 16, 4, 128, 1, 30.0, True, 0, 0, True),
    ]


def rope(name, tokens, heads, kv_heads, head_dim, rotary, layout, dtype, scaling, far, packed):
    return dict(name=name, op="rope", tokens=tokens, heads=heads, kv_heads=kv_heads, head_dim=head_dim, rotary=rotary,
                layout=layout, dtype=dtype, scaling=scaling, far=far, packed=packed)


def attend(name, cache, dtype, seqs, ctx, heads, kv_heads, head_dim, q_len):
    return dict(name=name, op="attend", cache=cache, dtype=dtype, seqs=seqs, ctx=ctx, heads=heads, kv_heads=kv_heads,
                head_dim=head_dim, q_len=q_len)


def store(name, cache, dtype, seqs, ctx, new, kv_heads, head_dim):
    return dict(name=name, op="store", cache=cache, dtype=dtype, seqs=seqs, ctx=ctx, new=new, kv_heads=kv_heads,
                head_dim=head_dim)


def step(name, cache, dtype, seqs, ctx, heads, kv_heads, head_dim):
    return dict(name=name, op="step", cache=cache, dtype=dtype, seqs=seqs, ctx=ctx, heads=heads, kv_heads=kv_heads,
                head_dim=head_dim, q_len=1)


def scored(name, cache, dtype, seqs, ctx, heads, kv_heads, head_dim, q_len, cap, bias, window, prefix, documents):
    return dict(name=name, op="scored", cache=cache, dtype=dtype, seqs=seqs, ctx=ctx, heads=heads, kv_heads=kv_heads,
                head_dim=head_dim, q_len=q_len, cap=cap, bias=bias, window=window, prefix=prefix, documents=documents)


def draw(rng):
    def spread(lo, hi):   # over the logarithm, odd sizes among them
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "rope", "attend", "attend", "store", "step", "scored", "scored", "scored"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 8])
    if hkv * g > 32:
        g = 32 // hkv
    dt = rng.choice(["bf16", "f16"])
    if op == "rope":
        c = rope("", spread(1, 8192), hkv * g, hkv, d, rng.choice([d, d, d // 2, d // 4, 20, 6]),
                 rng.choice(["half", "interleaved"]), dt, rng.choice(["none", "linear", "ntk", "by_parts"]),
                 spread(2048, 1000000), rng.choice([True, False]))
    else:
        seqs = spread(1, 128)
        tokens = 8 * 65536 * 8 * 128 // (hkv * d) // 8   # an eighth of the largest listed case's cache, at most
        ctx = spread(1, min(65536, max(64, tokens // seqs)))
        q_len = rng.choice([1, 1, 1, 2, 3, 4])
        while q_len > 1 and (g * q_len > 16 or ctx < q_len):
            q_len -= 1
        if op == "attend":
            c = attend("", rng.choice(["i8", "e4m3"]), dt, seqs, ctx, hkv * g, hkv, d, q_len)
        elif op == "store":
            seqs = min(seqs, 32)
            new = spread(1, min(4000, 24000 // seqs + 1))
            c = store("", rng.choice(["i8", "e4m3"]), dt, seqs, min(ctx, 16384 // seqs) + new, new, hkv, d)
        elif op == "step":
            c = step("", "e4m3", dt, seqs, ctx, hkv * g, hkv, d)
        else:
            c = scored("", rng.choice([dt, dt, "i8", "e4m3"]), dt, seqs, ctx, hkv * g, hkv, d, q_len,
                       rng.choice([0.0, 20.0, 50.0]), rng.choice([True, False]), rng.choice([0, 0, 100, 1024]),
                       rng.choice([0, 0, 5, 64]), rng.choice([True, False]))
    del c["name"]
    return c


# ---------------------------------------------------------------- lengths and masks: from the case alone


def lengths(case):
    """Stored tokens of each sequence, the new ones among them: the first holds `ctx`, the others a quarter to all of it."""
    lo = max(1, case.get("q_len", 1), case.get("new", 0))
    return [max(lo, int(case["ctx"] * (0.25 + 0.75 * ((1.0 + i * 0.6180339887) % 1.0)))) if i else max(lo, case["ctx"])
            for i in range(case["seqs"])]


def new_lengths(case):
    """New tokens of each sequence of a store: the first all of `new`, the others down to one."""
    return [max(1, case["new"] - i * case["new"] // case["seqs"]) for i in range(case["seqs"])]


def first_visible(case, ctx):
    """(first token of each sequence's document, its prefix tokens)."""
    starts = [(c * (3 * i % 7)) // 10 if case.get("documents") else 0 for i, c in enumerate(ctx)]
    if case.get("documents") and len(ctx) > 2:
        starts[2] = ctx[2]   # its document has not begun: nothing to see
    return starts, [min(c, case.get("prefix", 0) + (i % 3 if case.get("prefix") else 0)) for i, c in enumerate(ctx)]


def slopes(heads):
    return [2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)]


def frequencies(case):
    """Radians a position, in 64 bits."""
    r, base, kind = case["rotary"], 500000.0, case["scaling"]
    factor, low, high, original = 8.0, 1.0, 4.0, 8192.0
    if kind == "ntk" and r > 2:
        base *= factor ** (r / (r - 2))
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if kind == "linear":
        f = [x / factor for x in f]
    if kind == "by_parts":
        for i, x in enumerate(f):
            turns = original * x / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - low) / (high - low)))
            f[i] = x / factor * (1 - keep) + x * keep
    return f


def mscale(case):
    return 1.1386 if case["scaling"] == "by_parts" else 1.0


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    st = {"case": case}
    if case["op"] == "rope":
        prepare_rope(case, gen, st)
    else:
        prepare_cache(case, gen, st)
    if own:   # what a user's program sets up once: the library's handles and scratch
        from paged_decode_attention_cache_gb300 import ops
        if case["op"] == "rope":
            r = ops.pkv_rope_frequencies(case["rotary"], 500000.0, case["scaling"], factor=8.0, low_rotations=1.0,
                                         high_rotations=4.0, original_context=8192)
            st["rope"] = ops.Rope(r.cuda(), case["rotary"], case["layout"], mscale(case))
            st["cache"] = ops.Cache(case["dtype"], st["kc"], st["vc"])
        else:
            st["cache"] = ops.Cache(case["cache"], st["kc"], st["vc"], st["ks"], st["vs"])
            st["seqs"] = ops.Seqs(st["tables"], st["ctx"], case.get("q_len", 1), case.get("window", 0))
            if "q" in st:
                st["ws"] = ops.balanced_workspace(case["seqs"], case["kv_heads"], case["head_dim"])
            if case["op"] == "scored":
                st["scores"] = ops.Scores(case["cap"], st["slopes"], st["starts"], st["prefix"])
    return st


def prepare_rope(case, gen, st):
    T, H, Hk, D, dt = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"], DT[case["dtype"]]
    rows = torch.randn(T, H + 2 * Hk, D, generator=gen, device="cuda").to(dt)
    q, k, v = rows[:, :H], rows[:, H:H + Hk], rows[:, H + Hk:]
    st["q"], st["k"], st["v"] = (q, k, v) if case["packed"] else (q.contiguous(), k.contiguous(), v.contiguous())
    nb = -(-T // 16) + 2
    st["kc"] = torch.randn(nb, 16, Hk, D, generator=gen, device="cuda").to(dt)
    st["vc"] = torch.randn(nb, 16, Hk, D, generator=gen, device="cuda").to(dt)
    slots = torch.randperm(nb, generator=gen, device="cuda")[:, None] * 16 + torch.arange(16, device="cuda")
    st["slots"] = slots.flatten()[:T].contiguous()
    if T > 4:   # a batch padded to a round size: rows without a slot
        st["slots"][T - T // 16 - 1:] = -1
    if T > 512:   # prompts: runs of positions
        st["positions"] = case["far"] - 1 - torch.arange(T, device="cuda") % min(T, case["far"])
    else:
        st["positions"] = torch.randint(0, case["far"], (T,), generator=gen, device="cuda")
    st["freq"] = torch.tensor(frequencies(case), dtype=torch.float64, device="cuda")


def prepare_cache(case, gen, st):
    B, Hk, D, dt = case["seqs"], case["kv_heads"], case["head_dim"], DT[case["dtype"]]
    ctx = lengths(case)
    mb = -(-max(ctx) // 16) + 1
    used = [-(-c // 16) for c in ctx]
    nb = sum(used) + 3
    perm = torch.randperm(nb, generator=gen, device="cuda").to(torch.int32)
    tables = torch.zeros(B, mb, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(used):
        tables[s, :n] = perm[at:at + n]
        at += n
    st["tables"], st["ctx"] = tables, torch.tensor(ctx, dtype=torch.int32, device="cuda")
    st["ks"] = st["vs"] = None
    for key in ("k", "v"):
        x = torch.randn(nb, 16, Hk, D, generator=gen, device="cuda")
        if key == "k":   # a few loud channels, as keys have
            x[..., ::17] *= 4.0
        if case["cache"] in QMAX:
            scale = grid_up(x.abs().amax(dim=(1, 3)), case["cache"])
            st[key + "s"] = scale
            st[key + "c"] = to_codes(x / scale[:, None, :, None], case["cache"])
        else:
            st[key + "c"] = x.to(DT[case["cache"]])
        del x
    rows = sum(new_lengths(case)) if case["op"] == "store" else B * case["q_len"]
    if case["op"] != "store":
        st["q"] = torch.randn(rows, case["heads"], D, generator=gen, device="cuda").to(dt)
        if case["op"] == "scored" and case["cap"]:
            st["q"] *= 6.0   # scores that reach the cap
    if case["op"] in ("store", "step"):
        # some tokens louder than what the block holds: its scale grows
        loud = 1.0 + 3.0 * (torch.rand(rows, Hk, 1, generator=gen, device="cuda") > 0.7)
        st["kn"] = (torch.randn(rows, Hk, D, generator=gen, device="cuda") * 2 * loud).to(dt)
        st["vn"] = (torch.randn(rows, Hk, D, generator=gen, device="cuda") * loud).to(dt)
        new = new_lengths(case) if case["op"] == "store" else [1] * B
        st["cu_new"] = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
        st["cu"] = torch.tensor([0] + ctx, device="cuda").cumsum(0).to(torch.int32)
        st["total"] = sum(ctx)
    if case["op"] == "scored":
        starts, prefix = first_visible(case, ctx)
        as_int = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        st["starts"] = as_int(starts) if case["documents"] else None
        st["prefix"] = as_int(prefix) if case["prefix"] else None
        st["slopes"] = torch.tensor(slopes(case["heads"]), device="cuda") if case["bias"] else None


def grid_up(amax, kind):
    """amax / qmax rounded up: to three significant bits (i8), to a power of two (e4m3); zero stays zero."""
    t = amax / torch.full_like(amax, QMAX[kind])
    drop = 21 if kind == "i8" else 23
    up = ((t.view(torch.int32) + ((1 << drop) - 1)) >> drop << drop).view(torch.float32)
    return torch.where(t > 0, up.clamp_min(2.0 ** -126), torch.zeros_like(up))


def to_codes(y, kind):
    if kind == "i8":
        return y.round().clamp(-127, 127).to(torch.int8)
    return y.clamp(-448, 448).to(torch.float8_e4m3fn)


# ---------------------------------------------------------------- one pass


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        from paged_decode_attention_cache_gb300 import ops
        if op == "rope":
            q_out = torch.empty(st["q"].shape, dtype=st["q"].dtype, device="cuda")
            ops.pkv_rope_and_cache(q_out, st["q"], st["k"], st["v"], st["rope"], st["positions"], st["cache"], st["slots"])
            return {"q": q_out, "k_cache": st["kc"], "v_cache": st["vc"]}
        if op == "store":
            ops.pkv_quantize_kv_blocks(st["cache"], st["kn"], st["vn"], st["seqs"], st["cu_new"])
            k = torch.empty(st["total"], case["kv_heads"], case["head_dim"], dtype=st["kn"].dtype, device="cuda")
            v = torch.empty_like(k)
            ops.pkv_gather_kv_cache_dequant(k, v, st["cu"], st["cache"], st["seqs"])
            return {"k": k, "v": v, "k_scale": st["ks"], "v_scale": st["vs"]}
        out = torch.empty_like(st["q"])
        if op == "scored":
            ops.pkv_paged_attention_scored(out, st["q"], case["head_dim"] ** -0.5, st["cache"], st["seqs"], st["scores"], st["ws"])
            return out
        if op == "step":
            ops.pkv_quantize_kv_blocks(st["cache"], st["kn"], st["vn"], st["seqs"])
        ops.pkv_paged_attention_balanced(out, st["q"], case["head_dim"] ** -0.5, st["cache"], st["seqs"], st["ws"])
        return with_state(st, out) if op == "step" else out
    if op == "rope":
        return plain_rope(st, case)
    if op == "store":
        plain_append(st, case)
        k, v = plain_read(st, case)
        L = torch.arange(k.shape[1], device="cuda")
        keep = L[None, :] < st["ctx"][:, None]
        return {"k": k[keep].to(st["kn"].dtype), "v": v[keep].to(st["kn"].dtype), "k_scale": st["ks"], "v_scale": st["vs"]}
    if op == "step":
        plain_append(st, case)
        return with_state(st, plain_attention(st, case))
    return plain_attention(st, case)


def with_state(st, out):
    """The output and the cache after the step: e4m3 numbers and the scales that multiply them."""
    return {"out": out, "k": st["kc"], "v": st["vc"], "k_scale": st["ks"], "v_scale": st["vs"]}


# ---------------------------------------------------------------- plain forms


def plain_rope(st, case):
    r = case["rotary"]
    a = st["positions"].double()[:, None] * st["freq"]
    c, s = ((x * mscale(case)).float()[:, None, :] for x in (a.cos(), a.sin()))

    def turn(x):
        y = x.float()
        if case["layout"] == "half":
            u, w = y[..., :r // 2], y[..., r // 2:r]
            y = torch.cat([u * c - w * s, w * c + u * s, y[..., r:]], dim=-1)
        else:
            u, w = y[..., 0:r:2], y[..., 1:r:2]
            y = torch.cat([torch.stack([u * c - w * s, w * c + u * s], dim=-1).flatten(-2), y[..., r:]], dim=-1)
        return y.to(x.dtype)

    q, k = turn(st["q"]), turn(st["k"])
    there = st["slots"] >= 0
    rows = st["slots"][there]
    st["kc"].view(-1, *st["kc"].shape[2:])[rows] = k[there]
    st["vc"].view(-1, *st["vc"].shape[2:])[rows] = st["v"][there]
    return {"q": q, "k_cache": st["kc"], "v_cache": st["vc"]}


def plain_append(st, case):
    """New tokens behind each sequence's others: the block's scale first, then what it held, then the new rows."""
    kind = case["cache"]
    cu, ctx, tables = st["cu_new"].long(), st["ctx"].long(), st["tables"].long()
    rows = st["kn"].shape[0]
    seq = torch.searchsorted(cu[1:], torch.arange(rows, device="cuda"), right=True)
    first = ctx - (cu[1:] - cu[:-1])   # position of each sequence's first new token
    pos = first[seq] + torch.arange(rows, device="cuda") - cu[seq]
    blk, off = tables[seq, pos // 16], pos % 16
    held = first % 16                  # old rows of the block that the new tokens begin in
    old = tables[torch.arange(len(first), device="cuda"), first // 16]
    below = torch.arange(16, device="cuda")[None, :, None, None] < held[:, None, None, None]
    for key, x in (("k", st["kn"].float()), ("v", st["vn"].float())):
        codes, scale = st[key + "c"], st[key + "s"]
        amax = torch.zeros_like(scale).index_reduce_(0, blk, x.abs().amax(-1), "amax")
        need = grid_up(amax, kind)
        kept = torch.zeros_like(scale)
        kept[old] = torch.where(held[:, None] > 0, scale[old], torch.zeros_like(scale[old]))
        new = torch.maximum(kept, need)
        share = torch.where(new > 0, kept / new, torch.zeros_like(new))
        had = codes.view(torch.uint8)[old].view(codes.dtype)
        again = to_codes(had.float() * share[old][:, None, :, None], kind)
        codes.view(torch.uint8)[old] = torch.where(below, again.view(torch.uint8), had.view(torch.uint8))
        inv = torch.where(new > 0, torch.ones_like(new) / new, torch.zeros_like(new))
        codes.view(torch.uint8)[blk, off] = to_codes(x * inv[blk][..., None], kind).view(torch.uint8)
        scale[blk] = new[blk]


def plain_read(st, case):
    """K and V of every stored token in 32 bits, [sequences, longest, kv heads, head_dim]; zero past each sequence's tokens."""
    t = st["tables"].long()
    there = torch.arange(t.shape[1] * 16, device="cuda")[None, :] < st["ctx"][:, None]
    got = []
    for key in ("k", "v"):
        c, scale = st[key + "c"], st[key + "s"]
        x = c.view(torch.uint8)[t].view(c.dtype).float() if scale is not None else c[t].float()
        if scale is not None:
            x = x * scale[t][:, :, None, :, None]
        got.append(torch.where(there[..., None, None], x.flatten(1, 2), 0.0))
    return got


def plain_attention(st, case):
    B, ql, Hk, D = case["seqs"], case["q_len"], case["kv_heads"], case["head_dim"]
    g = case["heads"] // Hk
    k, v = plain_read(st, case)
    q = st["q"].float().view(B, ql, Hk, g, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, g * ql, D)
    x = (q @ k.permute(0, 2, 3, 1)).view(B, Hk, g, ql, -1) * D ** -0.5
    if case.get("cap"):
        x = case["cap"] * torch.tanh(x / case["cap"])
    ctx, pos = st["ctx"].long(), torch.arange(k.shape[1], device="cuda")
    mine = ctx[:, None] - ql + torch.arange(ql, device="cuda")   # position of each query
    if case.get("bias"):
        x = x + st["slopes"].view(1, Hk, g, 1, 1) * (pos[None, None, :] - mine[..., None])[:, None, None].float()
    lo = (ctx - case["window"]).clamp_min(0) if case.get("window") else torch.zeros_like(ctx)
    if st.get("starts") is not None:
        lo = torch.maximum(lo, st["starts"].long())
    seen = pos[None, :] >= lo[:, None]
    if st.get("prefix") is not None:
        seen = seen | (pos[None, :] < st["prefix"][:, None])
    seen = seen[:, None, :] & (pos[None, None, :] <= mine[..., None])
    x = torch.where(seen[:, None, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
    o = p.reshape(B, Hk, g * ql, -1) @ v.permute(0, 2, 1, 3)
    l = p.sum(-1).reshape(B, Hk, g * ql, 1)
    o = torch.where(l > 0, o / l, 0.0).view(B, Hk, g, ql, D).permute(0, 3, 1, 2, 4)
    return o.reshape(B * ql, Hk * g, D).to(st["q"].dtype)


# ---------------------------------------------------------------- work


def visible(case):
    """(tokens whose K/V are read, blocks they lie in)."""
    ctx = lengths(case)
    starts, prefix = first_visible(case, ctx)
    tokens = blocks = 0
    for c, a, p in zip(ctx, starts, prefix):
        if case.get("window"):
            a = max(a, c - case["window"])
        a = min(a, c)
        p = min(p, a) if case.get("prefix") else 0
        tokens += c - a + p
        blocks += -(-c // 16) - a // 16 + -(-p // 16)
    return tokens, blocks


def work(case):
    D, Hk = case["head_dim"], case["kv_heads"]
    if case["op"] == "rope":
        T, H, r = case["tokens"], case["heads"], case["rotary"]
        stored = T - (T // 16 + 1 if T > 4 else 0)
        return {"bytes": 2 * D * (2 * T * H + 4 * stored * Hk) + 16 * T, "flops": 3 * r * T * H + 3 * r * stored * Hk}
    if case["op"] == "store":
        rows, all_ = sum(new_lengths(case)), sum(lengths(case))
        blocks = sum(-(-c // 16) for c in lengths(case))
        # new rows read, the whole cache's codes read or written once, its values written
        return {"bytes": Hk * D * (4 * rows + 2 * all_ + 4 * all_) + 8 * Hk * blocks, "flops": 6 * Hk * D * rows + 2 * Hk * D * all_}
    tokens, blocks = visible(case)
    rows = case["seqs"] * case["q_len"]
    small = case["cache"] in QMAX
    moved = tokens * Hk * D * (2 if small else 4) + (blocks * Hk * 8 if small else 0) + rows * case["heads"] * D * 4
    if case["op"] == "step":
        moved += rows * Hk * D * 4
    return {"bytes": moved, "flops": 4 * case["q_len"] * case["heads"] * D * tokens}


# ---------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return exact_rope(st, case)
    ctx = lengths(case)
    state = {}
    if case["op"] in ("store", "step"):
        state = exact_append(st, case, ctx)
    if case["op"] == "store":
        got = {}
        for key in ("k", "v"):
            got[key] = torch.cat([stored(st, case, key, s, c) for s, c in enumerate(ctx)])
        return {**got, "k_scale": st["ks"].double(), "v_scale": st["vs"].double()}
    ql, Hk, D = case["q_len"], case["kv_heads"], case["head_dim"]
    g = case["heads"] // Hk
    starts, prefix = first_visible(case, ctx)
    out = torch.zeros(case["seqs"] * ql, Hk * g, D, dtype=torch.float64, device="cuda")
    for s, c in enumerate(ctx):
        K, V = stored(st, case, "k", s, c), stored(st, case, "v", s, c)
        at = torch.arange(c, device="cuda")
        lo = max(starts[s], c - case["window"]) if case.get("window") else starts[s]
        for j in range(ql):
            me = c - ql + j
            see = ((at >= lo) | (at < prefix[s])) & (at <= me)
            if not bool(see.any()):
                continue
            for h in range(Hk):
                q = st["q"][s * ql + j, h * g:(h + 1) * g].double()
                x = q @ K[see, h].T / math.sqrt(D)
                if case.get("cap"):
                    x = case["cap"] * torch.tanh(x / case["cap"])
                if case.get("bias"):
                    x = x + torch.tensor(slopes(case["heads"]), device="cuda").double()[h * g:(h + 1) * g, None] * (at[see] - me)
                out[s * ql + j, h * g:(h + 1) * g] = torch.softmax(x, dim=-1) @ V[see, h]
    return {"out": out, **state} if case["op"] == "step" else out


def stored(st, case, key, s, c):
    """[c, kv heads, head_dim]: what sequence s holds, as the numbers that it stands for."""
    t = st["tables"][s, :-(-c // 16)].long()
    x = st[key + "c"]
    x = (x.view(torch.uint8)[t].view(x.dtype).float() if x.element_size() == 1 else x[t]).double()
    if st[key + "s"] is not None:
        x = x * st[key + "s"][t].double()[:, None, :, None]
    return x.flatten(0, 1)[:c]


def exact_append(st, case, ctx):
    """Block by block, in 64 bits; the state is changed in place."""
    new = new_lengths(case) if case["op"] == "store" else [1] * case["seqs"]
    row = 0
    todo = {}   # (first row of a block, how many) -> the blocks and rows that have them: one pass for each
    for s, (c, n) in enumerate(zip(ctx, new)):
        p = c - n
        while p < c:
            a, m = p % 16, min(16 - p % 16, c - p)
            todo.setdefault((a, m), []).append((s, p // 16, row))
            p, row = p + m, row + m
    for (a, m), where in todo.items():
        w = torch.tensor(where, device="cuda")
        b = st["tables"][w[:, 0], w[:, 1]].long()
        for key, x in (("k", st["kn"]), ("v", st["vn"])):
            y = x[w[:, 2:3] + torch.arange(m, device="cuda")].double()          # [blocks, m, heads, dims]
            t = y.abs().amax(dim=(1, 3)) / QMAX[case["cache"]]
            e = torch.floor(torch.log2(t.clamp_min(1e-300)))
            e = e + (t >= torch.exp2(e + 1)).double() - (t < torch.exp2(e)).double()
            unit = torch.exp2(e - 2) if case["cache"] == "i8" else torch.exp2(e)
            need = torch.where(t > 0, torch.ceil(t / unit) * unit, 0.0)
            had = st[key + "s"][b].double() if a else torch.zeros_like(need)
            s_new = torch.maximum(need, had)
            code = st[key + "c"].view(torch.uint8)[b].view(st[key + "c"].dtype).float().double()
            code[:, :a] *= (had / s_new)[:, None, :, None]
            code[:, a:a + m] = y / s_new[:, None, :, None]
            part = to_codes(code[:, :a + m].float(), case["cache"]).view(torch.uint8)
            whole = st[key + "c"].view(torch.uint8)[b]
            whole[:, :a + m] = part
            st[key + "c"].view(torch.uint8)[b] = whole
            st[key + "s"][b] = s_new.float()
    return {"k": st["kc"].float().double(), "v": st["vc"].float().double(), "k_scale": st["ks"].double(),
            "v_scale": st["vs"].double()}


def exact_rope(st, case):
    r = case["rotary"]
    f = torch.tensor(frequencies(case), dtype=torch.float64, device="cuda")
    z = torch.polar(torch.full_like(f, mscale(case)).expand(case["tokens"], -1), st["positions"].double()[:, None] * f)[:, None]

    def turn(x):
        y = x.double().clone()
        if case["layout"] == "half":
            w = torch.complex(y[..., :r // 2].contiguous(), y[..., r // 2:r].contiguous()) * z
            y[..., :r // 2], y[..., r // 2:r] = w.real, w.imag
        else:
            w = torch.view_as_complex(y[..., :r].reshape(*y.shape[:-1], r // 2, 2).contiguous()) * z
            y[..., :r] = torch.view_as_real(w).flatten(-2)
        return y

    kc, vc, k = st["kc"].double(), st["vc"].double(), turn(st["k"])
    for name, pool, x in (("k", kc, k), ("v", vc, st["v"].double())):
        there = torch.nonzero(st["slots"] >= 0).flatten()
        pool.view(-1, *pool.shape[2:]).index_copy_(0, st["slots"][there], x[there])
    return {"q": turn(st["q"]), "k_cache": kc, "v_cache": vc}
