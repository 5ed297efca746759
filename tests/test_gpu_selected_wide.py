"""Page selection and attention over selected pages for batches with enough query tokens that several go to a CTA: 16 for
the selection, those that fill an MMA's 16 rows or, for prompts over 16-bit caches, its 128 for the attention.  A batch is
a small one's sequences many times over, each time with the same queries and lists: every copy has to come out as the
reference does for the first (the tolerances are tests/test_gpu_selected.py's)."""
import numpy as np
import pytest
import torch

from paged_decode_attention_cache_gb300 import ops
from tests import selected_reference as ref
from tests.helpers import GuardedOut
from tests.test_gpu_selected import (CAPACITY, KINDS, OOB_BLOCK, PAGE_LIST, as_tensors, check_lists, check_out, cu, err, full_bounds,
                                     grid, queries, random_lists)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_decode_attention_cache_gb300 import build
    build.build()
    ops.lib()
    torch.cuda.set_device(0)


def copies(need, rows, hkv):
    """Copies of a batch of `rows` query tokens for `need` (query token, kv head) pairs and one more."""
    return need // (rows * hkv) + 1


SELECT_16 = 4 * 912     # from more pairs on, 16 tokens to a CTA of the selection


def together(width):    # from more on, neighbouring tokens of the attention together
    return 96 * 152 // width


def prompt_pairs(H, hkv):
    return 608 * min(8, 16 * hkv // H)


def many(w, n, q_len=1):
    return ops.Seqs(w.tables.repeat(n, 1).cuda(), torch.tensor(w.ctx * n, dtype=torch.int32).cuda(), q_len)


def wide_select(w, q, b, q_lens, n, pages, first, last, ragged=True, e=None, seqs=None):
    rows, extra = q.shape[0] * n, 3 if ragged else 0
    qq = torch.cat([q.repeat(n, 1, 1), torch.zeros(extra, *q.shape[1:], dtype=q.dtype)]).cuda()
    lists = torch.full((rows + extra, w.hkv, pages), 77, dtype=torch.int32, device="cuda")
    counts = torch.full((rows + extra, w.hkv), 78, dtype=torch.int32, device="cuda")
    ops.pkv_select_pages(lists, counts, qq, b, w.on_gpu(), seqs or many(w, n, 1 if ragged else q_lens[0]),
                         cu(q_lens * n) if ragged else None, keep_first=first, keep_last=last, err_flags=e)
    lists, counts = lists.cpu(), counts.cpu()
    assert (lists[rows:] == 77).all() and (counts[rows:] == 78).all()
    lists, counts = lists[:rows].view(n, -1, w.hkv, pages), counts[:rows].view(n, -1, w.hkv)
    assert (lists == lists[0]).all() and (counts == counts[0]).all()
    return lists[0], counts[0]


def wide_attention(w, q, q_lens, lists, n, width, dtype, ragged=True, extra=4, e=None, scale=0.15):
    extra = extra if ragged else 0
    t, c = as_tensors(lists, w.hkv, width)
    t, c = (torch.cat([x.repeat(n, *[1] * (x.dim() - 1)), torch.zeros_like(x[:1]).expand(extra, *x.shape[1:])]).contiguous() for x in (t, c))
    rows = q.shape[0] * n
    qq = torch.cat([q.repeat(n, 1, 1), torch.ones(extra, *q.shape[1:], dtype=q.dtype)]).cuda()
    guard = GuardedOut((rows + extra, *q.shape[1:]), dtype, "cuda")
    ops.pkv_paged_attention_selected(guard.out, qq, scale, w.on_gpu(), many(w, n, 1 if ragged else q_lens[0]), t, c,
                                     cu(q_lens * n) if ragged else None, err_flags=e)
    torch.cuda.synchronize()
    guard.check()
    assert torch.isnan(guard.out[rows:].float()).all()
    out = guard.out[:rows].view(n, *q.shape)
    assert torch.equal(torch.nan_to_num(out, 12345.0), torch.nan_to_num(out[:1], 12345.0).expand_as(out))
    return out[0]


# ---------------------------------------------------------------- selection


@pytest.mark.parametrize("kind,qd", [("bf16", None), ("f16", None), ("i8", torch.float16), ("e4m3", torch.bfloat16), ("k8v4", torch.float16)])
@pytest.mark.parametrize("H,hkv,d", [(8, 2, 64), (8, 1, 128)])
@pytest.mark.parametrize("q_lens,ragged", [([17] * 4, False), ([40, 1, 0, 17], True), ([300, 0, 0, 5], True)])
@pytest.mark.parametrize("pages,first,last", [(6, 1, 1), (20, 0, 0), (1, 0, 1)])
def test_selection(kind, qd, H, hkv, d, q_lens, ragged, pages, first, last):
    w = ref.World(kind, [500, 20, 64, 1260], hkv, d, seed=7, q_dtype=qd)
    q = queries(w, sum(q_lens), H)
    b = full_bounds(w)
    lists, counts = wide_select(w, q, b.cuda(), q_lens, copies(SELECT_16, sum(q_lens), hkv), pages, first, last, ragged)
    check_lists(lists, counts, ref.select(w, q, b, q_lens, pages, first, last), pages)


@pytest.mark.parametrize("same", [1, 3, 40, 1000])
def test_equal_scores_go_to_the_lower_page(same):
    w = ref.World("f16", [3000], 2, 64, seed=same)
    n = -(-3000 // 16)
    b = full_bounds(w)
    lo = grid((-(-n // same), 2, 64), 2.0 ** -6, 4.0, 5)
    for p in range(n):
        b[int(w.tables[0, p])] = torch.stack([lo[p // same], lo[p // same] + 1.0], dim=1).half()
    q = grid((19, 8, 64), 2.0 ** -6, 2.0, 6).half()
    q[4] = 0.0   # every score 0
    for pages in (4, 21):
        lists, counts = wide_select(w, q, b.cuda(), [19], copies(SELECT_16, 19, 2), pages, 1, 1)
        check_lists(lists, counts, ref.select(w, q, b, [19], pages, 1, 1), pages)


def test_bounds_that_are_not_finite():
    w = ref.World("bf16", [1000], 1, 64, seed=4)
    b = full_bounds(w)
    b[int(w.tables[0, 7]), 0, 1, 3] = float("inf")
    b[int(w.tables[0, 9]), 0, 0, 3] = float("nan")
    b[int(w.tables[0, 11]), 0, :, 5] = -float("inf")
    q = queries(w, 18, 4).abs() + 0.5
    for pages in (3, 10, 60, 61):
        lists, counts = wide_select(w, q, b.cuda(), [18], copies(SELECT_16, 18, 1), pages, 1, 1)
        check_lists(lists, counts, ref.select(w, q, b, [18], pages, 1, 1), pages)


@pytest.mark.parametrize("wide", [False, True])
def test_queries_of_far_apart_sizes(wide):
    # pages that only fp64 can rank, under folded queries whose exact sum needs more than two fp32 numbers
    w = ref.World("bf16", [1600], 1, 64, seed=31)
    b = full_bounds(w)
    base = grid((64,), 2.0 ** -3, 4.0, 32)
    base[3] = 0.0
    step = torch.randperm(100, generator=torch.Generator().manual_seed(33)).float()
    for p in range(100):
        x = base.clone()
        x[5] = step[p]
        b[int(w.tables[0, p])] = torch.stack([x, x])[None].bfloat16()
    q = torch.ones(18, 8, 64)
    q[:, :, 3] = torch.tensor([2.0 ** 100, 1.0, -2.0 ** 100, 2.0 ** -60, 3.0, -2.0 ** -70, -1.0, 0.0])
    q[:, :, 5] = 2.0 ** -20
    q = q.bfloat16()
    for pages in (3, 30, 64):
        if wide:
            lists, counts = wide_select(w, q, b.cuda(), [18], copies(SELECT_16, 18, 1), pages, 1, 0)
            check_lists(lists, counts, ref.select(w, q, b, [18], pages, 1, 0), pages)
        else:
            lists, counts = wide_select(w, q[:1], b.cuda(), [1], 1, pages, 1, 0, ragged=False)
            check_lists(lists, counts, ref.select(w, q[:1], b, [1], pages, 1, 0), pages)


@pytest.mark.parametrize("kind", ["bf16", "f16", "i8"])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_queries_that_are_not_finite(kind, value):
    # their scores are not numbers, so the lower pages go first; the other tokens and kv heads are as ever
    w = ref.World(kind, [1000], 2, 64, seed=34)
    b = full_bounds(w)
    q = queries(w, 18, 8)
    good = ref.select(w, q, b, [18], 9, 1, 2)
    q[5, 6, 11] = value   # kv head 1
    n = -(-(1000 - 17 + 5) // 16)
    good[5][1] = list(range(7)) + [n - 2, n - 1]
    for copies_ in (1, copies(SELECT_16, 18, 2)):
        lists, counts = wide_select(w, q, b.cuda(), [18], copies_, 9, 1, 2)
        check_lists(lists, counts, good, 9)


def test_selection_flags_bad_tables():
    w = ref.World("f16", [600, 600], 1, 64, seed=8)
    q_lens, n = [20, 9], copies(SELECT_16, 29, 1)
    q = queries(w, 29, 4)
    b = full_bounds(w)
    t = w.tables.clone()
    t[0, 3], t[0, 5], t[1, 20] = -1, 5000, 2 ** 30
    e = err()
    ctx = torch.tensor([600, 600] * n, dtype=torch.int32).cuda()
    lists, counts = wide_select(w, q, b.cuda(), q_lens, n, 10, 1, 1, seqs=ops.Seqs(t.repeat(n, 1).cuda(), ctx), e=e)
    check_lists(lists, counts, ref.select(w, q, b, q_lens, 10, 1, 1, tables=t), 10)
    assert int(e) == OOB_BLOCK
    e.zero_()
    wide_select(w, q, b.cuda(), q_lens, n, 6, 1, 1, seqs=ops.Seqs(w.tables[:, :20].repeat(n, 1).cuda(), ctx), e=e)
    assert int(e) == CAPACITY


# ---------------------------------------------------------------- attention, several tokens


@pytest.mark.parametrize("kind,qd", [("bf16", None), ("f16", None), ("i8", torch.float16), ("e4m3", torch.bfloat16), ("k8v4", torch.float16)])
@pytest.mark.parametrize("H,hkv,d", [(8, 2, 128), (4, 2, 64), (2, 2, 128), (8, 1, 64)])
@pytest.mark.parametrize("q_lens,ragged", [([4] * 3, False), ([2] * 3, False), ([9, 0, 7], True)])
def test_neighbouring_tokens(kind, qd, H, hkv, d, q_lens, ragged):
    w = ref.World(kind, [300, 20, 101], hkv, d, seed=5, q_dtype=qd)
    q = queries(w, sum(q_lens), H)
    lists = random_lists(w.ctx, q_lens, hkv, 9, 4)
    want = ref.attention(w, q, 0.15, q_lens, lists)
    e = err()
    for n in (copies(together(9), sum(q_lens), hkv), copies(4000, sum(q_lens), hkv)):
        check_out(wide_attention(w, q, q_lens, lists, n, 9, torch.float32, ragged, e=e), *want, kind, torch.float32)
    assert int(e) == 0


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("f16", 64), ("k8v4", 128)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_what_one_token_lists_reaches_no_other(kind, d, value):
    w = ref.World(kind, [200, 100], 2, d, seed=21)
    q_lens = [5, 3]
    q = queries(w, 8, 8)
    lists = [[[0, 3, 5], [12]], [[3, 5, 12], [1, 12]], [[2, 3], [2]], [[3, 11, 12], [12]], [[7, 12], [0, 12]],
             [[6], [6]], [[1, 6], [0, 6]], [[6], [3]]]
    spots = [(int(w.tables[0, 5]), 3, 0), (int(w.tables[0, 2]), 1, 1), (int(w.tables[0, 12]), 198 % 16, slice(None)),
             (int(w.tables[1, 6]), 99 % 16, 1)]
    for at in spots:
        if kind == "k8v4":
            w.cache.v_zero[at[0], at[2], at[1], 0] = value   # a token's first group of 32 dims
            w.v64[at[0], at[1], at[2], :32] = value
        else:
            w.cache.v[at] = value
            w.v64[at] = value
    want, mag, big = ref.attention(w, q, 0.2, q_lens, lists)
    got = wide_attention(w, q, q_lens, lists, copies(together(4), 8, 2), 4, torch.float32, scale=0.2).double().cpu()
    fine = torch.isfinite(want)
    assert 0 < int((~fine).sum()) < fine.numel() / 2
    assert torch.equal(torch.isfinite(got), fine)
    tol = mag * (2.0 ** -15 + (2.0 ** -11 if kind == "k8v4" else 0.0) + big[..., None] * 2.0 ** -18)
    assert ((got - want).abs()[fine] <= tol[fine] + want.abs()[fine] * 2.0 ** -24).all()


@pytest.mark.parametrize("kind", ["f16", "i8"])
def test_bad_entries_and_tables(kind):
    w = ref.World(kind, [400, 300], 2, 64, seed=23)
    q_lens = [6, 5]
    n = copies(together(6), 11, 2)
    q = queries(w, 11, 8)
    given, taken = [], []
    for _, vis in ref.rows_of(w.ctx, q_lens):
        m = -(-vis // 16)
        given.append([[0, m + 3, 2, 2, 1, m - 1], [-1, 5, 4, m]])
        taken.append([[0, 2, m - 1], [5]])
    e = err()
    got = wide_attention(w, q, q_lens, given, n, 6, torch.float32, e=e)
    assert int(e) == PAGE_LIST
    check_out(got, *ref.attention(w, q, 0.15, q_lens, taken), kind, torch.float32)
    good = w.tables.clone()
    w.tables[0, 2], w.tables[1, 5] = -1, 10 ** 6
    e.zero_()
    got = wide_attention(w, q, q_lens, taken, n, 6, torch.float32, e=e)
    assert int(e) == OOB_BLOCK
    w.tables = good
    left = [[[p for p in h if p != (2 if r < 6 else 5)] for h in heads] for r, heads in enumerate(taken)]
    check_out(got, *ref.attention(w, q, 0.15, q_lens, left), kind, torch.float32)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_scales_of_every_size(kind):
    w = ref.World(kind, [160], 1, 128, seed=14)
    vs = w.cache.v_scale
    for p, x in enumerate([2.0 ** -120, 0.0, 1e-30, 2.0 ** -126, 1.0, 3.0, 0.0, 1e10, 2.0 ** -10, 1e20]):
        vs[int(w.tables[0, p])] = x
    w.v64 = w.cache.v.float().double() * vs[:, None, :, None].double()
    q = queries(w, 4, 4)
    for pages in ([0], [1], [1, 2, 3], [0, 1, 2, 3, 4, 5], list(range(10)), [7, 8]):
        lists = [[[p for p in pages if p < 9]]] * 3 + [[pages]]
        want = ref.attention(w, q, 0.01, [4], lists)
        got = wide_attention(w, q, [4], lists, copies(together(10), 4, 1), 10, torch.float32, scale=0.01)
        # below 2^-126 fp32 itself rounds by 2^-149
        assert ((got.double().cpu() - want[0]).abs() <= want[1] * 2.0 ** -14 + 2.0 ** -130).all(), pages


# ---------------------------------------------------------------- attention, chunks of prompts


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("H,hkv,d", [(8, 2, 128), (4, 2, 64), (8, 1, 128), (2, 2, 64), (2, 2, 128), (8, 1, 64)])
@pytest.mark.parametrize("ctx,q_lens,width", [([300, 150, 101], [130, 129, 64], 9), ([1000], [200], 40), ([90, 16, 400], [90, 0, 300], 3),
                                              ([5, 2000], [70, 260], 64), ([700, 20], [33, 20], 12)])
def test_chunks_of_prompts(kind, H, hkv, d, ctx, q_lens, width):
    # the first tokens of a sequence shorter than its query tokens see nothing
    w = ref.World(kind, ctx, hkv, d, seed=d + H)
    q = queries(w, sum(q_lens), H)
    lists = random_lists(ctx, q_lens, hkv, width, 4)
    want = ref.attention(w, q, 0.15, q_lens, lists)
    e = err()
    for dtype in (torch.float32, w.q_dtype):
        got = wide_attention(w, q, q_lens, lists, copies(prompt_pairs(H, hkv), sum(q_lens), hkv), width, dtype, e=e)
        check_out(got, *want, kind, dtype)
    assert int(e) == 0


@pytest.mark.parametrize("q_len", [16, 33])
def test_chunks_of_prompts_of_one_length(q_len):
    w = ref.World("bf16", [300, 90, 8], 2, 64, seed=26)
    q_lens = [q_len] * 3
    q = queries(w, 3 * q_len, 8)
    lists = random_lists(w.ctx, q_lens, 2, 7, 9)
    got = wide_attention(w, q, q_lens, lists, copies(prompt_pairs(8, 2), 3 * q_len, 2), 7, torch.float32, ragged=False)
    check_out(got, *ref.attention(w, q, 0.15, q_lens, lists), "bf16", torch.float32)


def test_chunks_of_prompts_with_bad_entries_and_tables():
    w = ref.World("bf16", [400, 300], 2, 64, seed=23)
    q_lens = [64, 64]
    n = copies(prompt_pairs(8, 2), 128, 2)
    q = queries(w, 128, 8)
    given, taken = [], []
    for _, vis in ref.rows_of(w.ctx, q_lens):
        m = -(-vis // 16)
        given.append([[0, m + 3, 2, 2, 1, m - 1], [-1, 5, 4, m]])
        taken.append([[0, 2, m - 1], [5]])
    e = err()
    got = wide_attention(w, q, q_lens, given, n, 6, torch.float32, e=e)
    assert int(e) == PAGE_LIST
    check_out(got, *ref.attention(w, q, 0.15, q_lens, taken), "bf16", torch.float32)
    good = w.tables.clone()
    w.tables[0, 2], w.tables[1, 5] = -1, 10 ** 6
    e.zero_()
    got = wide_attention(w, q, q_lens, taken, n, 6, torch.float32, e=e)
    assert int(e) == OOB_BLOCK
    w.tables = good
    left = [[[p for p in h if p != (2 if r < 64 else 5)] for h in heads] for r, heads in enumerate(taken)]
    check_out(got, *ref.attention(w, q, 0.15, q_lens, left), "bf16", torch.float32)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_chunks_of_prompts_keep_what_they_do_not_see(value):
    w = ref.World("bf16", [200, 330], 2, 128, seed=24)
    q_lens = [60, 40]
    q = queries(w, 100, 8)
    lists = random_lists(w.ctx, q_lens, 2, 6, 8)
    lists[3][0] = sorted(set(lists[3][0][:4]) | {2})
    w.cache.v[int(w.tables[0, 2]), 5, 0, 77] = value    # kv head 0, page 2: the rows that list it
    w.cache.v[int(w.tables[0, 12]), 199 % 16] = value   # the last token of sequence 0
    w.v64 = w.cache.v.double()
    want, mag, big = ref.attention(w, q, 0.15, q_lens, lists)
    got = wide_attention(w, q, q_lens, lists, copies(prompt_pairs(8, 2), 100, 2), 6, torch.float32).double().cpu()
    fine = torch.isfinite(want)
    assert 0 < int((~fine).sum()) < fine.numel() / 2
    assert torch.equal(torch.isfinite(got), fine)
    tol = mag * (2.0 ** -15 + big[..., None] * 2.0 ** -18)
    assert ((got - want).abs()[fine] <= tol[fine] + want.abs()[fine] * 2.0 ** -24).all()


# ---------------------------------------------------------------- single tokens of many sequences


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [40, 300])
def test_single_tokens_of_many_sequences(kind, n):
    w = ref.World(kind, [700, 16, 33], 2, 64, seed=27)
    q = queries(w, 3, 4)
    b = full_bounds(w)
    lists, counts = wide_select(w, q, b.cuda(), [1] * 3, n, 9, 1, 2, ragged=False)
    want = ref.select(w, q, b, [1] * 3, 9, 1, 2)
    check_lists(lists, counts, want, 9)
    got = wide_attention(w, q, [1] * 3, want, n, 9, torch.float32, ragged=False)
    check_out(got, *ref.attention(w, q, 0.15, [1] * 3, want), kind, torch.float32)


# ---------------------------------------------------------------- tables much wider than the sequences


@pytest.mark.parametrize("cols", [12000, 30000, 140000])
@pytest.mark.parametrize("H,hkv,d", [(8, 2, 128), (2, 2, 64)])
def test_wide_tables(cols, H, hkv, d):
    # what a CTA has room for then has fewer query tokens to a tile, or more CTAs to a cluster
    w = ref.World("bf16", [400, 35], hkv, d, seed=28, extra_cols=cols)
    q_lens = [60, 13]
    q = queries(w, 73, H)
    b = full_bounds(w)
    want = ref.select(w, q, b, q_lens, 6, 1, 1)
    out, mag, big = ref.attention(w, q, 0.15, q_lens, want)
    for pairs in (1, SELECT_16, prompt_pairs(H, hkv)):
        n = copies(pairs, 73, hkv)
        check_lists(*wide_select(w, q, b.cuda(), q_lens, n, 6, 1, 1), want, 6)
        check_out(wide_attention(w, q, q_lens, want, n, 6, torch.float32), out, mag, big, "bf16", torch.float32)


def test_bounds_of_more_new_tokens_than_any_sequence_has():
    w = ref.World("bf16", [400, 35], 2, 64, seed=29)
    b = ops.key_bounds(w.on_gpu())
    ops.pkv_key_bounds(b, w.on_gpu(), w.seqs(2 ** 31 - 1))
    assert torch.equal(b.cpu(), ref.bounds(w, torch.zeros_like(b.cpu()), [400, 35]))


# ---------------------------------------------------------------- a selection for the sparse attention


@pytest.mark.parametrize("ctx", [[4000, 700, 33, 2000], [60000]])
def test_lists_for_the_sparse_attention(ctx):
    # with one kv head a selection's lists are the sparse attention's: the next call on the stream may read them
    w = ref.World("bf16", ctx, 1, 64, seed=30)
    B, pages, n = len(ctx), 16, 12
    cache, seqs, b = w.on_gpu(), w.seqs(), full_bounds(w).cuda()
    qs = [queries(w, B, 4, seed=i).cuda() for i in range(n)]
    lists, counts = torch.empty(B, 1, pages, dtype=torch.int32, device="cuda"), torch.empty(B, 1, dtype=torch.int32, device="cuda")
    ws = ops.sparse_workspace(B, 1, 64, pages)

    def one(i, wait):
        out = torch.empty_like(qs[i])
        ops.pkv_select_pages(lists, counts, qs[i], b, cache, seqs)
        if wait:
            torch.cuda.synchronize()
        return ops.pkv_paged_attention_sparse(out, qs[i], 0.125, cache, seqs, lists.view(B, pages), counts.view(B), ws)

    want = [one(i, True).clone() for i in range(n)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = [one(i, False) for i in range(n)]
    for _ in range(3):
        got = [one(i, False) for i in range(n)]
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(captured, want))
