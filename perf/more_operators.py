"""Cases of attention over the pages that a cheap score selects for each query:
the elementwise bounds of each page's keys, kept as the cache grows; the
selection of the pages whose bounds promise the largest scores, for every query
token and kv head; and the attention over each one's own list of pages.

A page is a cache block of 16 tokens.  With lo and hi the bounds of its keys, its
score for a query token and a kv head is the sum over the kv head's query heads h and
the dims d of max(q[h, d] lo[d], q[h, d] hi[d]): no key of the page has a larger product
with those queries, summed over them.  The first and the last visible pages are always
taken, the others by score, the lower page where two are equal.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, the scores in 64, as pages next to the border differ by little) or, where
``own`` is true, through the library's entry points.  Sequence lengths follow
from the case alone, values from the seed.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8, "e4m3": torch.float8_e4m3fn}


# ---------------------------------------------------------------- the cases


def listed():
    return [
        # a decode step's keys join their pages' bounds
        bounds("bounds_step_64", "bf16", 64, 4096, 1, 8, 128),
        # prompts of mixed lengths stored behind what the sequences hold, on an e4m3 cache
        bounds("bounds_prompts_e4m3", "e4m3", 7, 16384, 4000, 8, 128),
        # one user's next token over a long chat: nothing but latency
        select("select_1_8k", "bf16", "bf16", 1, 8192, 1, False, 32, 8, 128, 64),
        # a serving batch of long contexts
        select("select_batch_32_32k", "bf16", "bf16", 32, 32768, 1, False, 32, 8, 128, 128),
        # very long contexts on an int8 cache, two drafted tokens each to verify
        select("select_verify_4_128k_i8", "i8", "bf16", 4, 131072, 2, False, 32, 8, 128, 256),
        # chunks of prompts far into their contexts: every token its own pages
        select("select_prompts", "bf16", "bf16", 3, 16384, 700, True, 32, 8, 128, 64),
        # one user's next token over the pages selected for it
        attend("attend_1_8k", "bf16", "bf16", 1, 8192, 1, False, 32, 8, 128, 64),
        # a serving batch of long contexts, 2048 tokens of each
        attend("attend_batch_32_32k", "bf16", "bf16", 32, 32768, 1, False, 32, 8, 128, 128),
        # drafts to verify on an e4m3 cache, an odd number of pages
        attend("attend_verify_16_e4m3", "e4m3", "f16", 16, 6000, 3, False, 16, 4, 128, 101),
        # chunks of prompts, neighbouring tokens with much of their lists in common
        attend("attend_prompts", "bf16", "bf16", 3, 16384, 500, True, 32, 8, 128, 64),
        # the library's batch of 8, one whole step: cache write, bounds, selection, attention
        step("step_8", "bf16", 8, 4096, 32, 8, 128, 64),
        # a wide batch of a small model, every head its own K/V
        step("step_64_f16", "f16", 64, 2000, 8, 8, 64, 33),
    ]


def bounds(name, cache, seqs, ctx, new, kv_heads, head_dim):
    return dict(name=name, op="bounds", cache=cache, seqs=seqs, ctx=ctx, new=new, ragged=new > 1, kv_heads=kv_heads,
                head_dim=head_dim)


def select(name, cache, dtype, seqs, ctx, new, ragged, heads, kv_heads, head_dim, pages):
    return dict(name=name, op="select", cache=cache, dtype=dtype, seqs=seqs, ctx=ctx, new=new, ragged=ragged, heads=heads,
                kv_heads=kv_heads, head_dim=head_dim, pages=pages, first=1, last=2)


def attend(name, cache, dtype, seqs, ctx, new, ragged, heads, kv_heads, head_dim, pages):
    return dict(select(name, cache, dtype, seqs, ctx, new, ragged, heads, kv_heads, head_dim, pages), op="attend")


def step(name, cache, seqs, ctx, heads, kv_heads, head_dim, pages):
    return dict(select(name, cache, cache, seqs, ctx, 1, False, heads, kv_heads, head_dim, pages), op="step")


def draw(rng):
    def spread(lo, hi):   # over the logarithm, odd sizes among them
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))

    op = rng.choice(["bounds", "select", "select", "select", "attend", "attend", "attend", "step"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 8])
    if hkv * g > 32:
        g = 32 // hkv
    half = rng.choice(["bf16", "f16"])
    kind = rng.choice([half, half, "i8", "e4m3"])
    seqs = spread(1, 64)
    tokens = 32 * 32768 * 8 * 128 // (hkv * d)   # the largest listed pool, at most
    if op == "bounds":
        ctx = spread(1, min(32768, tokens // 4 // seqs))
        c = bounds("", half if kind == "i8" else kind, seqs, ctx, rng.choice([1, spread(1, min(4000, ctx))]), hkv, d)
    elif op == "step":
        ctx = spread(200, min(8192, tokens // 8 // seqs))
        c = step("", half, seqs, ctx, hkv * g, hkv, d, min(ctx // 32, spread(4, 128)))
    else:
        kind_of = {"select": select, "attend": attend}[op]
        ragged = rng.choice([False, False, True])
        if ragged:
            seqs = min(seqs, 8)
            ctx = spread(200 if op == "select" else 16, 16384)
            new = spread(2, min(ctx, 1200 // seqs))
        else:
            ctx = spread(200 if op == "select" else 1, min(131072, tokens // 2 // seqs))
            new = min(ctx, rng.choice([1, 1, 1, 2, 3, 4]))
        pages = spread(4, 256 if new == 1 else 64)
        if op == "select":   # the longest sequence has more pages than it may take
            pages = min(pages, ctx // 32)
        c = kind_of("", kind, half, seqs, ctx, new, ragged, hkv * g, hkv, d, pages)
        c["first"], c["last"] = rng.choice([(1, 2), (0, 1), (1, 1), (2, 0)])
    del c["name"]
    return c


# ---------------------------------------------------------------- lengths: from the case alone


def lengths(case):
    """Stored tokens of each sequence, the new ones among them: the first holds `ctx`, the others a quarter to all of it."""
    new = new_lengths(case)
    return [max(n, int(case["ctx"] * (0.25 + 0.75 * ((1.0 + i * 0.6180339887) % 1.0)))) if i else max(n, case["ctx"])
            for i, n in enumerate(new)]


def new_lengths(case):
    """New tokens of each sequence: `new`, or, ragged, from `new` down to one."""
    return [max(1, case["new"] - i * case["new"] // case["seqs"]) if case["ragged"] else case["new"] for i in range(case["seqs"])]


def visible(case):
    """Visible tokens of each query token."""
    return [c - n + j + 1 for c, n in zip(lengths(case), new_lengths(case)) for j in range(n)]


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    B, Hk, D = case["seqs"], case["kv_heads"], case["head_dim"]
    ctx, new = lengths(case), new_lengths(case)
    used = [-(-c // 16) for c in ctx]
    nb, mb = sum(used) + 3, max(used) + 1
    perm = torch.randperm(nb, generator=gen, device="cuda").to(torch.int32)
    slot = torch.arange(mb, device="cuda")[None, :]
    n = torch.tensor(used, device="cuda")
    tables = torch.zeros(B, mb, dtype=torch.int32, device="cuda")
    tables[slot < n[:, None]] = perm[:sum(used)]
    st = {"case": case, "tables": tables, "ctx": torch.tensor(ctx, dtype=torch.int32, device="cuda"),
          "cu": torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32) if case["ragged"] else None, "ks": None, "vs": None}
    if case["op"] == "select":   # keys of a page lie around a centre of their own
        at = torch.randn(nb, Hk, D, generator=gen, device="cuda")
        wide = 0.5 + torch.rand(nb, Hk, D, generator=gen, device="cuda")
        both = torch.stack([at - wide, at + wide], dim=2)
        both[..., ::17] *= 4.0   # a few loud channels, as keys have
        st["bounds"] = store(st, "k", both, (2, 3), case["cache"])
        st["kc"] = st["vc"] = None
        if own:   # the pools whose bounds these are
            st["kc"] = st["vc"] = torch.zeros(nb, 16, Hk, D, dtype=torch.uint8 if case["cache"] == "e4m3" else DT[case["cache"]], device="cuda")
            st["vs"] = st["ks"]
    else:
        for key in ("k", "v"):
            x = torch.randn(nb, 16, Hk, D, generator=gen, device="cuda")
            if key == "k":
                x += torch.randn(nb, 1, Hk, D, generator=gen, device="cuda")
                x[..., ::17] *= 4.0
            st[key + "c"] = store(st, key, x, (1, 3), case["cache"])
            del x
        st["bounds"] = torch.zeros(nb, Hk, 2, D, dtype=torch.uint8 if case["cache"] == "e4m3" else DT[case["cache"]],
                                   device="cuda").view(DT[case["cache"]])
    rows = sum(new)
    if "heads" in case:
        st["q"] = torch.randn(rows, case["heads"], D, generator=gen, device="cuda").to(DT[case["dtype"]])
    if case["op"] == "attend":
        st["lists"], st["counts"] = coherent_lists(case, gen)
    if case["op"] == "step":
        st["kn"], st["vn"] = (torch.randn(rows, Hk, D, generator=gen, device="cuda").to(DT[case["cache"]]) for _ in "kv")
        last = st["ctx"].long() - 1
        st["slots"] = tables[torch.arange(B, device="cuda"), last // 16].long() * 16 + last % 16
        every = bounds_of(st, case, torch.arange(nb, device="cuda"), torch.full((nb,), 16, device="cuda"))
        st["bounds"].copy_(every)   # of what earlier steps stored
    if own:   # what a user's program sets up once: the library's handles
        from paged_decode_attention_cache_gb300 import ops
        st["cache"] = ops.Cache(case["cache"], st["kc"], st["vc"], st["ks"], st["vs"])
        st["seqs"] = ops.Seqs(st["tables"], st["ctx"], 1 if case["ragged"] else case["new"])
    return st


def store(st, key, x, dims, kind):
    """x as the cache holds it; 8-bit caches have one scale per (block, kv head), on their grid."""
    if kind not in ("i8", "e4m3"):
        return x.to(DT[kind])
    t = x.abs().amax(dim=dims) / (127.0 if kind == "i8" else 448.0)
    drop = 21 if kind == "i8" else 23
    scale = ((t.view(torch.int32) + ((1 << drop) - 1)) >> drop << drop).view(torch.float32)
    st[key + "s"] = scale
    at = (slice(None), slice(None), None, None) if dims == (2, 3) else (slice(None), None, slice(None), None)
    y = x / scale[at]
    return y.round().clamp(-127, 127).to(torch.int8) if kind == "i8" else y.clamp(-448, 448).to(torch.float8_e4m3fn)


def coherent_lists(case, gen):
    """Lists as a selection gives them: neighbouring query tokens of a sequence share much of theirs."""
    vis, new = visible(case), new_lengths(case)
    n = -(-max(lengths(case)) // 16)
    of = torch.tensor([s for s, k in enumerate(new) for _ in range(k)], device="cuda")
    near = torch.tensor([i for k in new for i in range(k)], device="cuda") // 16 + of * (case["new"] // 16 + 1)
    Hk, R = case["kv_heads"], len(vis)
    x = torch.rand(case["seqs"], Hk, n, generator=gen, device="cuda")[of]
    x += 0.5 * torch.rand(int(near.max()) + 1, Hk, n, generator=gen, device="cuda")[near]
    x += 0.2 * torch.rand(R, Hk, n, generator=gen, device="cuda")
    return take(x.double(), torch.tensor(vis, device="cuda"), case)


def take(score, vis, case):
    """(lists [rows, kv heads, pages], counts [rows, kv heads]) of scores [rows, kv heads, n]: the first and last pages
    always, the others by score and then by index; in rising order, -1 behind the last."""
    n, k = score.shape[-1], case["pages"]
    have = (vis + 15) // 16
    page = torch.arange(n, device="cuda")
    seen = page < have[:, None]
    kept = seen & ((page < case["first"]) | (page >= have[:, None] - case["last"]))
    x = torch.where(kept[:, None], math.inf, torch.where(seen[:, None], score, -math.inf))
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :k]
    counts = have.clamp(max=k)[:, None].expand(-1, score.shape[1]).to(torch.int32).contiguous()
    if order.shape[-1] < k:
        order = torch.nn.functional.pad(order, (0, k - order.shape[-1]))
    there = torch.arange(k, device="cuda") < counts[..., None]
    lists = torch.where(there, order, n).sort(dim=-1).values
    return torch.where(there, lists, -1).to(torch.int32), counts


# ---------------------------------------------------------------- one pass


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        from paged_decode_attention_cache_gb300 import ops
        if op == "step":
            ops.pkv_reshape_and_cache(st["cache"], st["kn"], st["vn"], st["slots"])
        if op in ("bounds", "step"):
            ops.pkv_key_bounds(st["bounds"], st["cache"], st["seqs"], st["cu"])
        if op == "bounds":
            return st["bounds"]
        lists, counts = st.get("lists"), st.get("counts")
        if op in ("select", "step"):
            R, Hk = st["q"].shape[0], case["kv_heads"]
            lists = torch.empty(R, Hk, case["pages"], dtype=torch.int32, device="cuda")
            counts = torch.empty(R, Hk, dtype=torch.int32, device="cuda")
            ops.pkv_select_pages(lists, counts, st["q"], st["bounds"], st["cache"], st["seqs"], st["cu"],
                                 keep_first=case["first"], keep_last=case["last"])
        if op == "select":
            return {"lists": lists, "counts": counts}
        out = torch.empty_like(st["q"])
        ops.pkv_paged_attention_selected(out, st["q"], case["head_dim"] ** -0.5, st["cache"], st["seqs"], lists, counts, st["cu"])
    else:
        if op == "step":
            for_slot = st["slots"]
            st["kc"].view(-1, *st["kc"].shape[2:])[for_slot] = st["kn"]
            st["vc"].view(-1, *st["vc"].shape[2:])[for_slot] = st["vn"]
        if op in ("bounds", "step"):
            plain_bounds(st, case)
        if op == "bounds":
            return st["bounds"]
        lists, counts = st.get("lists"), st.get("counts")
        if op in ("select", "step"):
            lists, counts = plain_select(st, case)
        if op == "select":
            return {"lists": lists, "counts": counts}
        out = plain_attention(st, case, lists)
    if op == "attend":
        return out
    return {"out": out, "lists": lists, "counts": counts, "bounds": st["bounds"], "k": st["kc"], "v": st["vc"]}


# ---------------------------------------------------------------- plain forms


def rows_of(st, case):
    """(sequence, visible tokens) of each query token, or new token."""
    B, ctx = case["seqs"], st["ctx"].long()
    if st["cu"] is None:
        n = case["new"]
        of = torch.arange(B, device="cuda").repeat_interleave(n)
        return of, ctx[of] - n + torch.arange(n, device="cuda").repeat(B) + 1
    cu = st["cu"].long()
    row = torch.arange(sum(new_lengths(case)), device="cuda")
    of = torch.searchsorted(cu[1:], row, right=True)
    return of, ctx[of] - (cu[of + 1] - cu[of]) + (row - cu[of]) + 1


def at_bytes(x, index):
    """x[index] for the types that have no indexing of their own."""
    return x.view(torch.uint8)[index].view(x.dtype) if x.element_size() == 1 else x[index]


def bounds_of(st, case, block, tokens):
    """The bounds of the first `tokens` rows of each block, as the cache's numbers (8 bits: its codes)."""
    x = at_bytes(st["kc"], block).float()
    there = (torch.arange(16, device="cuda") < tokens[:, None])[:, :, None, None]
    lo, hi = torch.where(there, x, math.inf).amin(1), torch.where(there, x, -math.inf).amax(1)
    return torch.stack([lo, hi], dim=2).to(st["kc"].dtype)


def plain_bounds(st, case):
    """The pages that hold new tokens, over all that they store."""
    of, vis = rows_of(st, case)
    pos = vis - 1
    first = torch.ones_like(of, dtype=torch.bool)
    first[1:] = of[1:] != of[:-1]
    one = first | (pos % 16 == 0)   # a row of each page
    of, page = of[one], pos[one] // 16
    block = st["tables"].long()[of, page]
    new = bounds_of(st, case, block, (st["ctx"].long()[of] - page * 16).clamp(max=16))
    if new.element_size() == 1:
        st["bounds"].view(torch.uint8)[block] = new.view(torch.uint8)
    else:
        st["bounds"][block] = new


def plain_select(st, case):
    B, Hk, D = case["seqs"], case["kv_heads"], case["head_dim"]
    of, vis = rows_of(st, case)
    n = -(-max(lengths(case)) // 16)
    table = st["tables"][:, :n].long()
    x = at_bytes(st["bounds"], table).double()                                # [B, n, Hk, 2, D]
    if st["ks"] is not None:
        x = x * st["ks"][table].double()[..., None, None]
    q = st["q"].double().view(-1, Hk, case["heads"] // Hk, D)
    w = torch.cat([q.clamp(max=0).sum(2), q.clamp(min=0).sum(2)], dim=-1)     # what lo and hi are multiplied by
    # the rows of a sequence side by side: one product for each
    new = new_lengths(case)
    beside = torch.zeros(B, max(new), Hk, 2 * D, dtype=torch.float64, device="cuda")
    first = torch.tensor([0] + new, device="cuda").cumsum(0)
    j = torch.arange(len(of), device="cuda") - first[of]
    beside[of, j] = w
    score = beside.transpose(1, 2) @ x.flatten(3).permute(0, 2, 3, 1)          # [B, Hk, rows, n]
    return take(score[of, :, j], vis, case)


def plain_attention(st, case, lists):
    Hk, D = case["kv_heads"], case["head_dim"]
    g = case["heads"] // Hk
    of, vis = rows_of(st, case)
    page = lists.long().clamp(min=0)                                           # [R, Hk, P]
    block = st["tables"].long()[of[:, None, None], page]
    head = torch.arange(Hk, device="cuda")[None, :, None]
    pos = page[..., None] * 16 + torch.arange(16, device="cuda")
    seen = ((lists >= 0)[..., None] & (pos < vis[:, None, None, None])).flatten(2)
    got = {}
    for key in ("k", "v"):
        c = st[key + "c"].transpose(1, 2)                                      # [nb, Hk, 16, D]
        x = at_bytes(c, (block, head)).float()
        if st[key + "s"] is not None:
            x = x * st[key + "s"][block, head][..., None, None]
        got[key] = x.flatten(2, 3)
    x = st["q"].float().view(-1, Hk, g, D) @ got["k"].transpose(2, 3) * D ** -0.5
    x = torch.where(seen[:, :, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
    l = p.sum(-1, keepdim=True)
    o = p @ got["v"]
    o = torch.where(l > 0, o / l, 0.0)
    return o.reshape(-1, Hk * g, D).to(st["q"].dtype)


# ---------------------------------------------------------------- work


def work(case):
    D, Hk = case["head_dim"], case["kv_heads"]
    e = 1 if case["cache"] in ("i8", "e4m3") else 2
    ctx, new, vis = lengths(case), new_lengths(case), visible(case)
    bytes_ = flops = 0
    if case["op"] in ("bounds", "step"):   # the touched pages' keys, their bounds
        for c, n in zip(ctx, new):
            p = (c - n) // 16
            bytes_ += Hk * D * e * (c - 16 * p + 2 * (-(-c // 16) - p))
            flops += 2 * Hk * D * (c - 16 * p)
    if case["op"] in ("select", "step"):   # every page's bounds once a sequence, the queries, the lists
        pages = sum(-(-c // 16) for c in ctx)
        bytes_ += pages * Hk * (2 * D * e + (4 if e == 1 else 0)) + len(vis) * (case["heads"] * D * 2 + Hk * (case["pages"] + 1) * 4)
        flops += sum(4 * D * Hk * (-(-v // 16)) for v in vis) + len(vis) * case["heads"] * D
    if case["op"] in ("attend", "step"):   # at least one token's pages of each sequence, each row's list, queries and outputs
        k = case["pages"]
        for c in ctx:
            p = min(k, -(-c // 16))
            bytes_ += Hk * min(c, 16 * p) * 2 * D * e + (8 * Hk * p if e == 1 else 0)
        bytes_ += len(vis) * (case["heads"] * D * 4 + Hk * (k + 1) * 4)
        flops += sum(4 * case["heads"] * D * min(v, 16 * k) for v in vis)
    if case["op"] == "step":
        bytes_ += case["seqs"] * Hk * D * 8
    return {"bytes": bytes_, "flops": flops}


# ---------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    B, Hk, D = case["seqs"], case["kv_heads"], case["head_dim"]
    ctx, new = lengths(case), new_lengths(case)
    first = [sum(new[:s]) for s in range(B)]
    state = {}
    if op == "step":
        for s in range(B):
            b, o = int(st["tables"][s, (ctx[s] - 1) // 16]), (ctx[s] - 1) % 16
            st["kc"][b, o], st["vc"][b, o] = st["kn"][s], st["vn"][s]
    if op in ("bounds", "step"):
        table = st["tables"].tolist()
        todo = {}   # stored tokens of a touched page -> the pages that have as many: one pass for each
        for s in range(B):
            for p in range((ctx[s] - new[s]) // 16, -(-ctx[s] // 16)):
                todo.setdefault(min(16, ctx[s] - 16 * p), []).append(table[s][p])
        kv = number(st["kc"])
        full = number(st["bounds"])
        for n, blocks in todo.items():
            b = torch.tensor(blocks, device="cuda")
            full[b] = torch.stack([kv[b, :n].min(1).values, kv[b, :n].max(1).values], dim=2)
        state = {"bounds": full}
        if op == "bounds":
            return full
        state["k"], state["v"] = kv, number(st["vc"])
    if op in ("select", "step"):
        R = sum(new)
        lists = torch.full((R, Hk, case["pages"]), -1, dtype=torch.int32, device="cuda")
        counts = torch.zeros(R, Hk, dtype=torch.int32, device="cuda")
        for s in range(B):
            exact_select(st, case, state, s, range(first[s], first[s] + new[s]), lists, counts)
        state.update(lists=lists, counts=counts)
        if op == "select":
            return {"lists": lists, "counts": counts}
    out = exact_attention(st, case, state.get("lists", st.get("lists")), first)
    return out if op == "attend" else {"out": out, "lists": state["lists"], "counts": state["counts"], "bounds": state["bounds"],
                                       "k": state["k"], "v": state["v"]}


def number(x):
    return (x.float() if x.element_size() == 1 else x).double()


def exact_select(st, case, state, s, rows, lists, counts):
    """One sequence: the definition's maximum for every query head, its sums and a sort by (score, page)."""
    Hk, D, k = case["kv_heads"], case["head_dim"], case["pages"]
    g = case["heads"] // Hk
    c = lengths(case)[s]
    blocks = st["tables"][s, :-(-c // 16)].long()
    x = state["bounds"][blocks] if state else number(at_bytes(st["bounds"], blocks))
    if st["ks"] is not None:
        x = x * st["ks"][blocks].double()[:, :, None, None]
    lo, hi = x[:, :, 0], x[:, :, 1]
    mid, wide = (lo + hi) / 2, (hi - lo) / 2       # max(q lo, q hi) = q mid + |q| wide
    for r in rows:
        n = -(-(c - len(rows) + (r - rows[0]) + 1) // 16)
        q = st["q"][r].double().view(Hk, g, D)
        score = torch.einsum("hgd,nhd->hn", q, mid[:n]) + torch.einsum("hgd,nhd->hn", q.abs(), wide[:n])
        score[:, :min(case["first"], n)] = math.inf
        if case["last"]:
            score[:, max(0, n - case["last"]):] = math.inf
        m = min(k, n)
        best = torch.sort(-score, dim=1, stable=True).indices[:, :m].sort(dim=1).values
        lists[r, :, :m] = best.to(torch.int32)
        counts[r] = m


def exact_attention(st, case, lists, first):
    Hk, D = case["kv_heads"], case["head_dim"]
    g = case["heads"] // Hk
    ctx, new = lengths(case), new_lengths(case)
    out = torch.zeros(sum(new), Hk * g, D, dtype=torch.float64, device="cuda")
    kinds = {key: st[key + "c"].transpose(1, 2) for key in ("k", "v")}
    head = torch.arange(Hk, device="cuda")[:, None]
    for s in range(case["seqs"]):
        for r in range(first[s], first[s] + new[s]):
            vis = ctx[s] - new[s] + (r - first[s]) + 1
            page = lists[r]                                    # [Hk, P]
            ok = (page >= 0)[..., None] & (page.long()[..., None] * 16 + torch.arange(16, device="cuda") < vis)
            block = st["tables"][s].long()[page.long().clamp(min=0)]
            K, V = (number(at_bytes(kinds[key], (block, head))) for key in ("k", "v"))
            if st["ks"] is not None:
                K, V = K * st["ks"][block, head].double()[..., None, None], V * st["vs"][block, head].double()[..., None, None]
            x = torch.einsum("hgd,hptd->hgpt", st["q"][r].double().view(Hk, g, D), K) / math.sqrt(D)
            x = x.masked_fill(~ok[:, None], -math.inf).flatten(2)
            out[r] = (torch.softmax(x, dim=-1) @ V.flatten(1, 2)).reshape(Hk * g, D)
    return out
