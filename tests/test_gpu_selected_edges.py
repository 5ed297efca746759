"""Page selection and attention over selected pages where numbers leave the usual range: scales, bounds and queries of very
different sizes, infinities beside finite numbers (against tests/selected_reference.py; the attention's tolerances are
tests/test_gpu_selected.py's)."""
import math

import pytest
import torch

from paged_decode_attention_cache_gb300 import ops
from tests import selected_reference as ref
from tests.test_gpu_selected import check_lists, cu, full_bounds, queries, random_lists
from tests.test_gpu_selected_wide import SELECT_16, copies, prompt_pairs, together, wide_attention, wide_select

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_decode_attention_cache_gb300 import build
    build.build()
    ops.lib()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("kind,d", [("i8", 128), ("e4m3", 128), ("i8", 64), ("e4m3", 64)])
@pytest.mark.parametrize("value", [math.inf, 2.0 ** 40, 2.0 ** 26, math.nan])
def test_a_v_scale_reaches_the_rows_that_list_its_page(kind, d, value):
    # neighbouring tokens share a pass over the union of their lists, 20 pages and more, five to a warp: what a page's V scale
    # does to the weights of the pages behind it is for the rows that list it alone
    w = ref.World(kind, [600, 330], 2, d, seed=41)
    q_lens = [4, 4]
    q = queries(w, 8, 8)
    lists = [[sorted(set(h) | {0, 9, 12, 15, 18}) for h in heads] for heads in random_lists(w.ctx, q_lens, 2, 14, 42)]
    only = [(0, 0, 1), (2, 1, 3), (5, 0, 2)]   # row, kv head, page
    for r, h, p in only:
        for i, heads in enumerate(lists):
            heads[h] = sorted((set(heads[h]) - {p}) | ({p} if i == r else set()))
        w.cache.v_scale[int(w.tables[r // 4, p]), h] = value
    w.v64 = w.cache.v.float().double() * w.cache.v_scale[:, None, :, None].double()
    want, mag, big = ref.attention(w, q, 0.15, q_lens, lists)
    got = wide_attention(w, q, q_lens, lists, copies(together(19), 8, 2), 19, torch.float32).double().cpu()
    fine = torch.isfinite(want)
    if not math.isfinite(value):
        assert sorted({(r, h // 4) for r, h, _ in (~fine).nonzero().tolist()}) == [(r, h) for r, h, _ in only]
    assert torch.equal(torch.isfinite(got), fine)
    tol = mag * (2.0 ** -15 + big[..., None] * 2.0 ** -18) + want.abs() * 2.0 ** -24
    assert ((got - want).abs()[fine] <= tol[fine]).all()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("wide", [False, True])
def test_infinite_bounds_beside_queries_of_the_other_sign(kind, wide):
    # max(q lo, q hi) is finite where q is negative and hi infinite, or q positive and lo -infinite
    w = ref.World(kind, [1000], 2, 64, seed=43)
    b = full_bounds(w)
    q = queries(w, 18, 8)
    q[:, :4, 3], q[:, :4, 5] = -q[:, :4, 3].abs() - 0.25, q[:, :4, 5].abs() + 0.25   # kv head 0: every query head alike
    for page in (7, 20, 33, 50):
        b[int(w.tables[0, page]), :, 1, 3] = math.inf
    for page in (9, 20, 41):
        b[int(w.tables[0, page]), :, 0, 5] = -math.inf
    assert torch.isfinite(ref.page_scores(q[0], b, w.tables[0, :62].tolist(), None, 2)[0]).all()
    assert (q != 0).all()
    for pages in (3, 10, 40, 60):
        want = ref.select(w, q, b, [18], pages, 1, 1)
        if wide:
            check_lists(*wide_select(w, q, b.cuda(), [18], copies(SELECT_16, 18, 2), pages, 1, 1), want, pages)
        else:
            check_lists(*wide_select(w, q, b.cuda(), [18], 1, pages, 1, 1), want, pages)


@pytest.mark.parametrize("ctx", [600, 12000])
def test_k8v4_keys_past_fp16(ctx):
    # codes times scales of up to 127 * 700 are finite keys, and their bounds, rounded outwards to fp16, infinite
    w = ref.World("k8v4", [ctx], 1, 64, seed=44, q_dtype=torch.bfloat16)
    for page in (3, 8, 21, 30):
        w.cache.k_scale[int(w.tables[0, page]), 0, page % 16] = 700.0
    w.k64 = w.cache.k.double() * w.cache.k_scale.permute(0, 2, 1)[..., None].double()
    b = torch.zeros(w.cache.num_blocks, 1, 2, 64, dtype=torch.float16)
    got = b.cuda()
    ops.pkv_key_bounds(got, w.on_gpu(), w.seqs(), cu([ctx]))
    b = ref.bounds(w, b, [ctx])
    assert torch.isinf(b).any() and torch.equal(got.cpu(), b)
    q = queries(w, 2, 4)
    q[0, :, :] = q[0, :1, :]   # all heads alike: a bound is taken or not
    assert (q != 0).all()
    for pages in (4, 12):
        lists, counts = wide_select(w, q, got, [2], 1, pages, 1, 1)
        check_lists(lists, counts, ref.select(w, q, b, [2], pages, 1, 1), pages)


@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("ctx,wide", [(1000, False), (1000, True), (20000, False)])
def test_scores_that_underflow_fp32(kind, ctx, wide):
    # products of 2^-155 and less, which fp64 tells apart
    w = ref.World(kind, [ctx], 1, 64, seed=45, q_dtype=torch.bfloat16)
    b = full_bounds(w)
    if kind == "bf16":
        b = (b.float() * 2.0 ** -75).bfloat16()
    else:
        w.cache.k_scale *= 2.0 ** -80
    rows = 18 if wide else 2
    q = (queries(w, rows, 8, dtype=torch.float32) * 2.0 ** -85).bfloat16()
    q[0, 1:] = 0.0   # one query head left
    n = copies(SELECT_16, rows, 1) if wide else 1
    for pages in (5, 30, 60):
        lists, counts = wide_select(w, q, b.cuda(), [rows], n, pages, 1, 1)
        check_lists(lists, counts, ref.select(w, q, b, [rows], pages, 1, 1), pages)


@pytest.mark.parametrize("kind", ["bf16", "f16", "i8"])
@pytest.mark.parametrize("ctx", [1000, 20000])
def test_bounds_of_zeros(kind, ctx):
    # every score is 0 whatever the queries; a block id out of range goes behind them
    w = ref.World(kind, [ctx], 2, 64, seed=46)
    b = torch.zeros_like(full_bounds(w))
    q = queries(w, 3, 8)
    t = w.tables.clone()
    t[0, 3], t[0, 5] = -1, 2 ** 30
    seqs = ops.Seqs(t.cuda(), torch.tensor([ctx], dtype=torch.int32).cuda())
    for pages in (5, 60):
        lists, counts = wide_select(w, q, b.cuda(), [3], 1, pages, 1, 1, seqs=seqs)
        check_lists(lists, counts, ref.select(w, q, b, [3], pages, 1, 1, tables=t), pages)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("ctx,wide", [(1600, False), (1600, True), (16000, False)])
def test_errors_that_line_up(kind, ctx, wide):
    # folded queries that two 16-bit terms miss by as much as they can, upwards in even dims and downwards in odd ones, and
    # pages of either: their exact scores differ by 2^-20 and less of themselves
    w = ref.World(kind, [ctx], 1, 128, seed=47)
    u = 8 if kind == "bf16" else 11   # bits of a number
    parts = [1.0, 2.0 ** -u - 2.0 ** (-2 * u), 2.0 ** (-2 * u - 1) * (1 - 2.0 ** (1 - u)), 0.0]
    q = torch.zeros(18 if wide else 2, 8, 128, dtype=torch.float64)
    for h, x in enumerate(parts):
        q[:, h] = x
    q[:, 3, 1::2] = 2.0 ** (-2 * u)   # past the half: rounded up
    if kind == "f16":
        q[:, 2:] *= 0.0               # below fp16's smallest number beside 1
    q[:, :, 0], q[:, 4, 0] = 0.0, 2.0 ** -12
    assert torch.equal(q, q.to(w.q_dtype).double())
    n, g = -(-ctx // 16), torch.Generator().manual_seed(48)
    b = full_bounds(w)
    hi = torch.zeros(n, 128)
    odd = torch.randint(0, 2, (n,), generator=g).bool()
    hi[~odd, 2::2] = 1.0
    hi[odd, 1::2] = 1.0
    hi[odd, 1] = 0.0                  # 63 dims each
    hi[:, 0] = torch.randint(0, 64, (n,), generator=g).float() / 8
    b[w.tables[0, :n].long(), 0] = torch.stack([torch.zeros_like(hi), hi], dim=1).to(b.dtype)
    q = q.to(w.q_dtype)
    copies_ = copies(SELECT_16, q.shape[0], 1) if wide else 1
    for pages in (9, 50):
        lists, counts = wide_select(w, q, b.cuda(), [q.shape[0]], copies_, pages, 1, 1)
        check_lists(lists, counts, ref.select(w, q, b, [q.shape[0]], pages, 1, 1), pages)


@pytest.mark.parametrize("kind,up", [("i8", True), ("e4m3", True), ("e4m3", False)])   # sums of int8 codes do not get that small
@pytest.mark.parametrize("wide", [False, True])
def test_queries_that_the_scales_bring_back(kind, up, wide):
    # queries times codes leave fp32 in some pages, upwards or downwards; times the scales all are ordinary numbers
    w = ref.World(kind, [1600], 1, 64, seed=49, q_dtype=torch.bfloat16)
    g = torch.Generator().manual_seed(50)
    large = torch.rand(w.cache.num_blocks, generator=g) < 0.5   # pages of large codes
    code = torch.where(large[:, None, None, None], torch.randint(90, 128, (w.cache.num_blocks, 1, 2, 64), generator=g),
                       torch.randint(0, 5, (w.cache.num_blocks, 1, 2, 64), generator=g))
    if kind == "i8":
        code[:, :, 0] *= -1
        b, back, more = code.to(torch.int8), -124, 5
    else:   # the codes 0 .. 4 stand for 2^-9 each, 80 .. 117 for 8 to 208
        code = torch.where(large[:, None, None, None], code - 10, code)
        code[:, :, 0] += 128
        b, back, more = code.to(torch.uint8).view(torch.float8_e4m3fn), -124 if up else 105, 14
    w.cache.k_scale[:, 0] = torch.where(large, 2.0 ** back, 2.0 ** (back + more))
    rows = 18 if wide else 2
    q = (queries(w, rows, 8, dtype=torch.float32) * 2.0 ** (115 if up else -131)).bfloat16()
    for pages in (5, 30, 70):
        lists, counts = wide_select(w, q, b.cuda(), [rows], copies(SELECT_16, rows, 1) if wide else 1, pages, 1, 1)
        check_lists(lists, counts, ref.select(w, q, b, [rows], pages, 1, 1), pages)


def chunk_of_a_prompt(kind, seed):
    """65 query tokens of one sequence, every one of which lists page 0 and some others; dim 0 of the queries is 4, of the keys 0."""
    w = ref.World(kind, [400], 2, 64, seed=seed)
    q = queries(w, 65, 8)
    q[:, :, 0] = 4.0
    w.cache.k[..., 0] = 0.0
    w.k64 = w.cache.k.double()
    lists = [[sorted(set(h) | {0}) for h in heads] for heads in random_lists(w.ctx, [65], 2, 7, seed)]
    return w, q, lists


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_chunks_of_prompts_keep_an_infinity_of_little_weight(kind, value):
    # the first token of each list weighs 2^-34 of the others
    w, q, lists = chunk_of_a_prompt(kind, 51)
    first = int(w.tables[0, 0])
    w.cache.k[first, 0, :, 0] = -40.0
    w.cache.v[first, 0, 0, 7] = value
    w.k64, w.v64 = w.cache.k.double(), w.cache.v.double()
    want, mag, big = ref.attention(w, q, 0.15, [65], lists)
    got = wide_attention(w, q, [65], lists, copies(prompt_pairs(8, 2), 65, 2), 8, torch.float32).double().cpu()
    fine = torch.isfinite(want)
    assert torch.equal(~fine, torch.zeros_like(fine).index_fill_(2, torch.tensor([7]), True) & (torch.arange(8) < 4)[None, :, None])
    assert torch.equal(torch.isfinite(got), fine)
    tol = mag * (2.0 ** -15 + big[..., None] * 2.0 ** -18) + want.abs() * 2.0 ** -24
    assert ((got - want).abs()[fine] <= tol[fine]).all()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_chunks_of_prompts_whose_first_scores_are_minus_infinity(kind, value):
    # three tokens that weigh nothing, and an infinity or NaN in the V of a page that another token lists
    w, q, lists = chunk_of_a_prompt(kind, 52)
    lists = [[sorted((set(h) - {9}) | ({9} if r == 30 else set())) for h in heads] for r, heads in enumerate(lists)]
    _, _, big = ref.attention(w, q, 0.15, [65], lists)
    first = int(w.tables[0, 0])
    w.k64[first, :3, :, 0] = -1e6   # as good as
    w.v64[int(w.tables[0, 9])] = value
    want, mag, _ = ref.attention(w, q, 0.15, [65], lists)
    w.cache.k[first, :3, :, 0] = -math.inf
    w.cache.v[int(w.tables[0, 9])] = value
    got = wide_attention(w, q, [65], lists, copies(prompt_pairs(8, 2), 65, 2), 9, torch.float32).double().cpu()
    fine = torch.isfinite(want)
    assert torch.equal(~fine, (torch.arange(65) == 30)[:, None, None].expand_as(fine))
    assert torch.equal(torch.isfinite(got), fine)
    tol = mag * (2.0 ** -15 + big[..., None] * 2.0 ** -18) + want.abs() * 2.0 ** -24
    assert ((got - want).abs()[fine] <= tol[fine]).all()


@pytest.mark.parametrize("kind", ["bf16", "f16", "k8v4"])
@pytest.mark.parametrize("q_lens,width", [([1, 1], 9), ([1, 1], 64), ([4, 4], 9)])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_partial_sums_keep_an_infinity_of_little_weight(kind, q_lens, width, value):
    # page 1's tokens weigh some 2^-200 of the others and less: nothing, in the fp32 weights of one warp's or CTA's sums beside another's
    w = ref.World(kind, [1100, 200], 2, 64, seed=53, q_dtype=torch.float16)
    q = queries(w, sum(q_lens), 8)
    q[:, :, 0] = 8.0
    if kind == "k8v4":
        w.cache.k[..., 0], w.cache.k_scale[...] = 0, 1 / 32   # codes of -127: scores 8 * -4 * 5.5
    else:
        w.cache.k[..., 0] = 0.0
    lists = [[sorted(set(h) | {1, 2, 3}) for h in heads] for heads in random_lists(w.ctx, q_lens, 2, width - 3, 54)]
    for s in range(2):
        b = int(w.tables[s, 1])
        w.cache.k[b, :, :, 0] = -127 if kind == "k8v4" else -4.0
        if kind == "k8v4":
            w.cache.v_zero[b, :, 5, 0] = value
        else:
            w.cache.v[b, 5, :, :32] = value
    if kind == "k8v4":
        w.k64 = w.cache.k.double() / 32
        for s in range(2):
            w.v64[int(w.tables[s, 1]), 5, :, :32] = value
    else:
        w.k64, w.v64 = w.cache.k.double(), w.cache.v.double()
    want, _, _ = ref.attention(w, q, 5.5, q_lens, lists)
    fine = torch.isfinite(want)
    assert torch.equal(~fine, (torch.arange(64) < 32)[None, None].expand_as(fine))
    n = copies(together(width), sum(q_lens), 2) if q_lens[0] > 1 else 1
    got = wide_attention(w, q, q_lens, lists, n, width, torch.float32, ragged=False, scale=5.5).cpu()
    assert torch.equal(torch.isfinite(got), fine)


def test_long_lists_for_the_sparse_attention():
    # lists of more than one round of the sparse attention's set-up, which reads the first ones ahead, and counts that change
    w = ref.World("bf16", [60000, 30000, 9000], 1, 64, seed=55)
    B, pages, n = 3, 1500, 6
    cache, b = w.on_gpu(), full_bounds(w).cuda()
    qs = [queries(w, B, 4, seed=i).cuda() for i in range(n)]
    seqs = [w.seqs(ctx=[60000, 30000 - 3000 * i, 9000]) for i in range(n)]
    lists, counts = torch.empty(B, 1, pages, dtype=torch.int32, device="cuda"), torch.empty(B, 1, dtype=torch.int32, device="cuda")
    ws = ops.sparse_workspace(B, 1, 64, pages)

    def one(i, wait):
        out = torch.empty_like(qs[i])
        ops.pkv_select_pages(lists, counts, qs[i], b, cache, seqs[i])
        if wait:
            torch.cuda.synchronize()
        return ops.pkv_paged_attention_sparse(out, qs[i], 0.125, cache, seqs[i], lists.view(B, pages), counts.view(B), ws)

    want = [one(i, True).clone() for i in range(n)]
    assert int(counts[1]) < pages
    for _ in range(3):
        got = [one(i, False) for i in range(n)]
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("kind", ["bf16", "f16", "i8"])
@pytest.mark.parametrize("ctx,wide", [(6400, False), (6400, True), (30000, False)])
def test_many_pages_that_the_last_bits_of_fp64_tell_apart(kind, ctx, wide):
    # hundreds of scores that differ by 2^-36 of themselves and less, some of them equal, and a few far from them
    w = ref.World(kind, [ctx], 1, 64, seed=56, q_dtype=torch.float16 if kind == "f16" else torch.bfloat16)
    n, g = -(-ctx // 16), torch.Generator().manual_seed(57)
    x = torch.full((n, 64), 1.0 if kind == "i8" else 1.5)
    x[:, 5] = torch.randint(0, 120, (n,), generator=g).float()
    x[7], x[100], x[200] = 3.0, -2.0, 4.0
    b = full_bounds(w)
    b[w.tables[0, :n].long(), 0] = torch.stack([x, x], dim=1).to(b.dtype)
    if kind == "i8":
        w.cache.k_scale[:] = 0.75
    q = torch.ones(18 if wide else 2, 2, 64)
    q[:, 0] = 128.0
    q[:, :, 5] = 2.0 ** (-24 if kind == "f16" else -28)
    q = q.to(w.q_dtype)
    for pages in (3, 30, 64):
        lists, counts = wide_select(w, q, b.cuda(), [q.shape[0]], copies(SELECT_16, q.shape[0], 1) if wide else 1, pages, 1, 1)
        check_lists(lists, counts, ref.select(w, q, b, [q.shape[0]], pages, 1, 1), pages)
