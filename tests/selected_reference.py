"""What key bounds, page selection and attention over selected pages are, in 64 bits on the CPU, and caches to
try them on.  Written from the definitions in include/pkv.h; nothing here calls the library."""
import math

import torch

from paged_decode_attention_cache_gb300 import ops

SRC = {"bf16": torch.bfloat16, "f16": torch.float16}


class World:
    """A cache of `kind` with random contents, the sequences' tables, and the numbers that it stands for.  What lies
    behind a sequence's last token, and in blocks of no sequence, is not a number where the kind has such values."""

    def __init__(self, kind, ctx, hkv, d, seed=0, q_dtype=None, spare=2, extra_cols=1):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.ctx, self.hkv, self.d = kind, list(ctx), hkv, d
        self.q_dtype = SRC.get(kind) or q_dtype or torch.bfloat16
        used = [-(-c // 16) for c in ctx]
        nb = sum(used) + spare
        perm = torch.randperm(nb, generator=g)
        self.tables = torch.full((len(ctx), max(used + [1]) + extra_cols), 2 ** 30, dtype=torch.int32)   # not read past the context
        at = 0
        for s, n in enumerate(used):
            self.tables[s, :n] = perm[at:at + n].to(torch.int32)
            at += n
        stored = torch.zeros(nb, 16, dtype=torch.bool)
        for s, c in enumerate(ctx):
            for p in range(used[s]):
                stored[self.tables[s, p], :min(16, c - 16 * p)] = True
        shape = (nb, 16, hkv, d)
        nan = float("nan")
        if kind in SRC:
            k, v = (torch.randn(shape, generator=g) for _ in "kv")
            k[..., ::13] *= 3.0
            k, v = (torch.where(stored[:, :, None, None], x, nan).to(SRC[kind]) for x in (k, v))
            self.cache = ops.Cache(kind, k, v)
            self.k64, self.v64 = k.double(), v.double()
        elif kind == "i8":
            k, v = (torch.randint(-127, 128, shape, generator=g).to(torch.int8) for _ in "kv")
            ks, vs = (2.0 ** torch.randint(-8, -4, (nb, hkv), generator=g).float() * 1.25 for _ in "kv")
            ks[0], vs[0] = 0.0, 0.0
            self.cache = ops.Cache(kind, k, v, ks, vs)
            self.k64, self.v64 = k.double() * ks[:, None, :, None].double(), v.double() * vs[:, None, :, None].double()
        elif kind == "e4m3":
            k, v = (torch.randn(shape, generator=g).to(torch.float8_e4m3fn).view(torch.uint8) for _ in "kv")
            k[~stored], v[~stored] = 0x7f, 0xff
            ks, vs = (2.0 ** torch.randint(-3, 3, (nb, hkv), generator=g).float() for _ in "kv")
            self.cache = ops.Cache(kind, k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), ks, vs)
            self.k64 = k.view(torch.float8_e4m3fn).float().double() * ks[:, None, :, None].double()
            self.v64 = v.view(torch.float8_e4m3fn).float().double() * vs[:, None, :, None].double()
        else:
            k = torch.randint(-127, 128, shape, generator=g).to(torch.int8)
            codes = torch.randint(0, 16, shape, generator=g)
            v = (codes[..., 0::2] + 16 * codes[..., 1::2]).to(torch.uint8)
            there = stored[:, None, :].expand(nb, hkv, 16)
            ks = torch.where(there, 0.01 + 0.02 * torch.rand(nb, hkv, 16, generator=g), nan).half()
            vs = torch.where(there[..., None], 0.05 + 0.1 * torch.rand(nb, hkv, 16, d // 32, generator=g), nan).half()
            vz = torch.where(there[..., None], -1.0 + 0.5 * torch.rand(nb, hkv, 16, d // 32, generator=g), nan).half()
            self.cache = ops.Cache(kind, k, v, ks, vs, vz)
            self.k64 = k.double() * ks.permute(0, 2, 1)[..., None].double()
            wide = lambda x: x.permute(0, 2, 1, 3).repeat_interleave(32, dim=-1).double()  # noqa: E731
            self.v64 = codes.double() * wide(vs) + wide(vz)

    def on_gpu(self):
        c = self.cache
        move = lambda x: None if x is None else x.cuda()  # noqa: E731
        return ops.Cache(c.kind, c.k.cuda(), c.v.cuda(), move(c.k_scale), move(c.v_scale), move(c.v_zero))

    def seqs(self, q_len=1, ctx=None):
        return ops.Seqs(self.tables.cuda(), torch.tensor(self.ctx if ctx is None else ctx, dtype=torch.int32).cuda(), q_len)


def rows_of(ctx, q_lens):
    """(sequence, visible tokens) of each query token."""
    return [(s, max(0, c - n + j + 1)) for s, (c, n) in enumerate(zip(ctx, q_lens)) for j in range(n)]


def bounds(w, before, new_lens):
    """The bounds tensor (as the library's, on the CPU) after the call; blocks that it does not touch as `before`."""
    out = before.clone()
    raw = out.view(torch.uint8) if out.element_size() == 1 else out
    for s, (c, n) in enumerate(zip(w.ctx, new_lens)):
        for p in range(max(0, c - n) // 16, -(-c // 16)):
            if n <= 0:
                continue
            b, m = int(w.tables[s, p]), min(16, c - 16 * p)
            if w.kind == "k8v4":
                x = w.k64[b, :m]
                lo, hi = x.min(0).values, x.max(0).values
                h_lo, h_hi = lo.half(), hi.half()
                h_lo = torch.where(h_lo.double() > lo, torch.nextafter(h_lo, torch.tensor(-math.inf).half()), h_lo)
                h_hi = torch.where(h_hi.double() < hi, torch.nextafter(h_hi, torch.tensor(math.inf).half()), h_hi)
                raw[b] = torch.stack([h_lo, h_hi], dim=1)
                continue
            x = w.cache.k[b, :m].float()
            y = torch.stack([x.min(0).values, x.max(0).values], dim=1).to(w.cache.k.dtype)
            raw[b] = y.view(torch.uint8) if y.element_size() == 1 else y
    return out


def page_scores(q, x, blocks, scale, hkv):
    """[hkv, pages]: the definition's sum, every query head and dim by itself, in 64 bits.  x: the bounds of all blocks."""
    g = q.shape[0] // hkv
    b = torch.as_tensor(blocks, dtype=torch.long)
    y = (x.float() if x.element_size() == 1 else x)[b].double()                     # [n, hkv, 2, d]
    if scale is not None:
        y = y * scale[b].double()[..., None, None]
    qq = q.double().view(hkv, g, 1, -1)
    lo, hi = (y[:, :, i].permute(1, 0, 2)[:, None] for i in (0, 1))                 # [hkv, 1, n, d]
    return torch.maximum(qq * lo, qq * hi).sum(-1).sum(1)


def select(w, q, x, q_lens, max_pages, keep_first, keep_last, tables=None, num_blocks=None):
    """(lists, counts) as nested python lists, per row and kv head."""
    tables = w.tables if tables is None else tables
    scale = w.cache.k_scale if w.kind in ("i8", "e4m3") else None
    lists = []
    for r, (s, vis) in enumerate(rows_of(w.ctx, q_lens)):
        n = -(-vis // 16)
        if n <= max_pages:
            lists.append([list(range(n))] * w.hkv)
            continue
        blocks = tables[s, :n].tolist()
        ok = [0 <= b < x.shape[0] for b in blocks]
        sc = page_scores(q[r], x, [b if o else 0 for b, o in zip(blocks, ok)], scale, w.hkv)
        sc = torch.where(torch.isnan(sc), -math.inf, sc)
        sc[:, [i for i, o in enumerate(ok) if not o]] = -math.inf
        mine = []
        for h in range(w.hkv):
            mid = range(keep_first, n - keep_last)
            best = sorted(mid, key=lambda i: (-float(sc[h, i]), i))[:max_pages - keep_first - keep_last]
            mine.append(sorted([*range(keep_first), *best, *range(n - keep_last, n)]))
        lists.append(mine)
    return lists


def attention(w, q, scale, q_lens, lists):
    """(out [rows, H, D], weight-sum of magnitudes [rows, H, D], largest sum of |q k| [rows, H])."""
    R, H, d = q.shape
    g = H // w.hkv
    out, mag, big = torch.zeros(R, H, d, dtype=torch.float64), torch.zeros(R, H, d, dtype=torch.float64), torch.zeros(R, H, dtype=torch.float64)
    for r, (s, vis) in enumerate(rows_of(w.ctx, q_lens)):
        for h in range(w.hkv):
            pos = [p * 16 + t for p in lists[r][h] for t in range(16) if p * 16 + t < vis]
            if not pos:
                continue
            pos = torch.tensor(pos)
            b = w.tables[s, pos // 16].long()
            K, V = w.k64[b, pos % 16, h], w.v64[b, pos % 16, h]
            qq = q[r, h * g:(h + 1) * g].double()
            p = torch.softmax(scale * qq @ K.T, dim=-1)
            out[r, h * g:(h + 1) * g] = p @ V
            mag[r, h * g:(h + 1) * g] = p @ V.abs()
            big[r, h * g:(h + 1) * g] = (qq.abs() @ K.abs().T).amax(-1) * abs(scale)
    return out, mag, big
