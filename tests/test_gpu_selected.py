"""Key bounds, page selection and attention over selected pages on the GPU, against their definitions in 64 bits
(tests/selected_reference.py).  Bounds and lists have to be equal.

Attention's tolerance, for an output of magnitude sum mag = sum_t p_t |v_t| and the largest sum of |scale q k| of a
token, big.  A score is a sum of fp32 multiply-adds, D / 16 in a row in the tensor core, each rounded (or truncated) to
2^-23 of at most big, and multiplied once or twice: 2^-19 big covers 16 of them; a weight's relative error is that of its
score's difference to the maximum's, twice as much, and 2^-21 of the exponential.  In the operand a weight is split in two
16-bit halves: 2^-17 of it for bf16 (8 + 8 bits and the second's rounding), less for fp16.  Sums of up to 2^7 pages a warp in
fp32 are off by 2^-16 of mag at most, the merge by less.  K8/V4's values are rounded once to fp16, 2^-11 of a value: mag.
Then the output's own rounding, half a step."""
import numpy as np
import pytest
import torch

from paged_decode_attention_cache_gb300 import ops
from tests import selected_reference as ref
from tests.helpers import GuardedOut

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "f16", "i8", "e4m3", "k8v4"]
OOB_BLOCK, CAPACITY, PAGE_LIST = 0x1, 0x4, 0x20


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_decode_attention_cache_gb300 import build
    build.build()
    ops.lib()
    torch.cuda.set_device(0)


def err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def cu(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32).cuda()


def queries(w, rows, heads, seed=1, dtype=None):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, heads, w.d, generator=g).to(dtype or w.q_dtype)


def same_bytes(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---------------------------------------------------------------- bounds


def numbers(x):
    return x.float() if x.element_size() == 1 else x


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hkv,d", [(2, 64), (8, 128), (1, 64), (3, 128)])
@pytest.mark.parametrize("ctx,new", [([1, 15, 16, 17, 40, 0, 300], 1), ([5, 64, 33], 3), ([20, 16, 400, 7], [20, 1, 333, 0])])
def test_bounds(kind, hkv, d, ctx, new):
    w = ref.World(kind, ctx, hkv, d, seed=d + hkv)
    cache = w.on_gpu()
    b = ops.key_bounds(cache)
    b.view(torch.uint8).fill_(0x3c)   # what earlier steps left
    want = ref.bounds(w, b.cpu(), [new] * len(ctx) if isinstance(new, int) else new)
    e = err()
    if isinstance(new, int):
        ops.pkv_key_bounds(b, cache, w.seqs(new), err_flags=e)
    else:
        ops.pkv_key_bounds(b, cache, w.seqs(), cu(new), err_flags=e)
    assert int(e) == 0
    got = b.cpu()
    assert torch.equal(numbers(got), numbers(want))
    # the blocks of no new token keep every bit
    touched = {int(w.tables[s, p]) for s, (c, n) in enumerate(zip(ctx, [new] * len(ctx) if isinstance(new, int) else new))
               for p in range(max(0, c - n) // 16, -(-c // 16)) if n > 0}
    rest = [i for i in range(got.shape[0]) if i not in touched]
    assert same_bytes(got.view(torch.uint8)[rest], want.view(torch.uint8)[rest])


def test_bounds_of_signs_and_extremes():
    # the largest codes and values of both signs, one token and sixteen
    for kind, top in (("i8", 127), ("e4m3", 448.0), ("bf16", 3.0e38), ("f16", 65504.0)):
        w = ref.World(kind, [16, 1, 2], 1, 64)
        k = w.cache.k
        vals = torch.tensor([-top, top, -1.0, 1.0, 0.0, -0.0, top, -top])
        pattern = vals[torch.randint(0, 8, k.shape, generator=torch.Generator().manual_seed(3))]
        w.cache.k = pattern.to(k.dtype)
        cache = w.on_gpu()
        b = ops.key_bounds(cache)
        want = ref.bounds(w, b.cpu(), [16, 16, 16])
        ops.pkv_key_bounds(b, cache, w.seqs(16))
        assert torch.equal(numbers(b.cpu()), numbers(want)), kind


def test_bounds_flags():
    w = ref.World("bf16", [40, 20], 2, 64)
    cache = w.on_gpu()
    b = ops.key_bounds(cache)
    e = err()
    t = w.tables.clone()
    t[0, 2] = 1000
    t[1, 1] = -1
    ops.pkv_key_bounds(b, cache, ops.Seqs(t.cuda(), torch.tensor([40, 20], dtype=torch.int32).cuda()), err_flags=e)
    assert int(e) == OOB_BLOCK and not b.any()
    e.zero_()
    # a context past its table: what the table holds is done
    ops.pkv_key_bounds(b, cache, ops.Seqs(w.tables[:, :1].contiguous().cuda(), torch.tensor([40, 16], dtype=torch.int32).cuda(), 40),
                       err_flags=e)
    assert int(e) == CAPACITY
    w.ctx = [16, 16]
    assert torch.equal(b.cpu(), ref.bounds(w, torch.zeros_like(b.cpu()), [16, 16]))


# ---------------------------------------------------------------- selection


def run_select(w, q, b, q_lens, pages, first, last, ragged=False, extra_rows=0, seqs=None, e=None):
    rows = q.shape[0] + extra_rows
    qq = torch.cat([q, torch.zeros(extra_rows, *q.shape[1:], dtype=q.dtype)]).cuda()
    lists = torch.full((rows, w.hkv, pages), 77, dtype=torch.int32, device="cuda")
    counts = torch.full((rows, w.hkv), 78, dtype=torch.int32, device="cuda")
    ops.pkv_select_pages(lists, counts, qq, b, w.on_gpu(), seqs or w.seqs(1 if ragged else q_lens[0]), cu(q_lens) if ragged else None,
                         keep_first=first, keep_last=last, err_flags=e)
    return lists.cpu(), counts.cpu()


def check_lists(lists, counts, want, pages):
    for r, heads in enumerate(want):
        for h, x in enumerate(heads):
            assert int(counts[r, h]) == len(x), (r, h)
            assert lists[r, h].tolist() == x + [-1] * (pages - len(x)), (r, h)
    assert (lists[len(want):] == 77).all() and (counts[len(want):] == 78).all()   # rows behind the last sequence


def full_bounds(w):
    b = ops.key_bounds(w.cache)
    return ref.bounds(w, b, [c for c in w.ctx])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H,hkv,d", [(4, 1, 64), (8, 8, 128), (16, 2, 128), (6, 3, 64)])
@pytest.mark.parametrize("pages,first,last", [(8, 1, 2), (5, 0, 0), (3, 1, 2), (20, 4, 1), (1, 0, 1)])
def test_selection(kind, H, hkv, d, pages, first, last):
    w = ref.World(kind, [0, 1, 129, 700, 1500, 320, 16 * pages, 16 * pages + 1], hkv, d, seed=H + d)
    q = queries(w, len(w.ctx), H)
    b = full_bounds(w)
    lists, counts = run_select(w, q, b.cuda(), [1] * len(w.ctx), pages, first, last)
    check_lists(lists, counts, ref.select(w, q, b, [1] * len(w.ctx), pages, first, last), pages)


@pytest.mark.parametrize("kind,qd", [("bf16", None), ("i8", torch.float16), ("e4m3", torch.bfloat16), ("k8v4", torch.float16)])
@pytest.mark.parametrize("q_lens,ragged", [([3] * 4, False), ([40, 1, 0, 17], True), ([300, 0, 0, 5], True)])
def test_selection_of_several_tokens(kind, qd, q_lens, ragged):
    w = ref.World(kind, [500, 20, 64, 260], 2, 64, seed=7, q_dtype=qd)
    q = queries(w, sum(q_lens), 8)
    b = full_bounds(w)
    lists, counts = run_select(w, q, b.cuda(), q_lens, 6, 1, 1, ragged, extra_rows=3 if ragged else 0)
    check_lists(lists, counts, ref.select(w, q, b, q_lens, 6, 1, 1), 6)


def test_a_sequence_shorter_than_its_query_tokens():
    # the first tokens of the chunk see nothing
    w = ref.World("bf16", [2, 40], 1, 64, seed=3)
    q = queries(w, 10, 2)
    b = full_bounds(w)
    lists, counts = run_select(w, q, b.cuda(), [5, 5], 2, 0, 1)
    want = ref.select(w, q, b, [5, 5], 2, 0, 1)
    assert [len(x[0]) for x in want[:5]] == [0, 0, 0, 1, 1]
    check_lists(lists, counts, want, 2)


def grid(shape, step, top, seed):
    """Multiples of `step` up to `top`: the scores' sums are exact in 64 bits whatever their order."""
    return (torch.randint(-int(top / step), int(top / step) + 1, shape, generator=torch.Generator().manual_seed(seed)) * step)


@pytest.mark.parametrize("ctx", [400, 5000])
@pytest.mark.parametrize("same", [1, 2, 40, 1000])
def test_equal_scores_go_to_the_lower_page(ctx, same):
    # runs of `same` pages have the same keys, so there are ties at the border, few or hundreds of them
    w = ref.World("f16", [ctx], 2, 64, seed=same)
    n = -(-ctx // 16)
    b = full_bounds(w)
    lo = grid((-(-n // same), 2, 64), 2.0 ** -6, 4.0, 5)
    for p in range(n):
        b[int(w.tables[0, p])] = torch.stack([lo[p // same], lo[p // same] + 1.0], dim=1).half()
    q = grid((1, 8, 64), 2.0 ** -6, 2.0, 6).half()
    for pages in (4, 21):
        lists, counts = run_select(w, q, b.cuda(), [1], pages, 1, 1)
        check_lists(lists, counts, ref.select(w, q, b, [1], pages, 1, 1), pages)


def test_a_query_dim_that_outweighs_the_others():
    # its keys are zero everywhere: the scores lie 2^25 below the largest weight, where the other weights' fp16 terms run out of
    # bits, and differ by less than those are worth
    w = ref.World("f16", [2000], 1, 64, seed=22)
    b = torch.zeros_like(full_bounds(w))
    q = torch.zeros(1, 8, 64).half()
    q[:, :, 3] = 2.0 ** 14
    q[:, :, 4:] = grid((1, 8, 60), 2.0 ** -22, 2.0 ** -12, 23).half()
    base = grid((60,), 2.0 ** -6, 4.0, 24)
    for p in range(125):
        x = torch.cat([torch.zeros(4), base + grid((60,), 2.0 ** -6, 0.125, 25 + p)]).half()
        b[int(w.tables[0, p]), 0] = torch.stack([x, x])
    for pages in (3, 40):
        lists, counts = run_select(w, q, b.cuda(), [1], pages, 1, 0)
        check_lists(lists, counts, ref.select(w, q, b, [1], pages, 1, 0), pages)


@pytest.mark.parametrize("pages", [3, 30, 64])
def test_scores_closer_than_fp32_tells(pages):
    # every page the same but for one dim, whose 2^-14 steps leave scores of about 2^11 apart by less than fp32's error
    w = ref.World("f16", [1600], 1, 128, seed=2)
    b = full_bounds(w)
    base = grid((128,), 2.0 ** -4, 8.0, 8).half()
    g = torch.Generator().manual_seed(9)
    step = torch.randperm(100, generator=g).half() * 2.0 ** -14
    q = torch.full((1, 8, 128), 2.0).half()
    q[0, :, 5] = 2.0 ** -10
    for p in range(100):
        x = base.clone()
        x[5] = step[p]
        b[int(w.tables[0, p])] = torch.stack([x, x], dim=0)[None]
    lists, counts = run_select(w, q, b.cuda(), [1], pages, 1, 0)
    check_lists(lists, counts, ref.select(w, q, b, [1], pages, 1, 0), pages)


def test_queries_and_keys_of_zeros():
    w = ref.World("bf16", [1000, 900], 1, 64, seed=2)
    b = full_bounds(w)
    q = torch.zeros(2, 4, 64).bfloat16()
    q[1] = 1.0
    for p in range(-(-900 // 16)):
        b[int(w.tables[1, p])] = 0.0
    lists, counts = run_select(w, q, b.cuda(), [1, 1], 9, 2, 3)
    check_lists(lists, counts, ref.select(w, q, b, [1, 1], 9, 2, 3), 9)
    assert lists[0, 0].tolist() == [0, 1, 2, 3, 4, 5, 60, 61, 62]


def test_bounds_that_are_not_finite():
    w = ref.World("f16", [1000], 1, 64, seed=4)
    b = full_bounds(w)
    b[int(w.tables[0, 7]), 0, 1, 3] = float("inf")     # the largest score
    b[int(w.tables[0, 9]), 0, 0, 3] = float("nan")     # not a number: goes last
    b[int(w.tables[0, 11]), 0, :, 5] = -float("inf")   # the smallest
    q = queries(w, 1, 4).abs() + 0.5
    for pages in (3, 10, 60, 61, 62):
        lists, counts = run_select(w, q, b.cuda(), [1], pages, 1, 1)
        want = ref.select(w, q, b, [1], pages, 1, 1)
        check_lists(lists, counts, want, pages)


def test_long_sequences_by_clusters():
    w = ref.World("bf16", [70000, 33], 1, 64, seed=6)
    q = queries(w, 2, 8)
    b = full_bounds(w)
    for pages, first, last in ((512, 1, 2), (64, 0, 1), (4000, 10, 0)):
        lists, counts = run_select(w, q, b.cuda(), [1, 1], pages, first, last)
        check_lists(lists, counts, ref.select(w, q, b, [1, 1], pages, first, last), pages)


def test_selection_flags_bad_tables():
    w = ref.World("f16", [600, 600], 1, 64, seed=8)
    q = queries(w, 2, 4)
    b = full_bounds(w)
    t = w.tables.clone()
    t[0, 3], t[0, 5], t[1, 20] = -1, 5000, 2 ** 30
    e = err()
    for pages in (10, 37):
        seqs = ops.Seqs(t.cuda(), torch.tensor([600, 600], dtype=torch.int32).cuda())
        lists, counts = run_select(w, q, b.cuda(), [1, 1], pages, 1, 1, seqs=seqs, e=e)
        check_lists(lists, counts, ref.select(w, q, b, [1, 1], pages, 1, 1, tables=t), pages)
        assert int(e) == OOB_BLOCK
    # a context past its table: the table's pages
    e.zero_()
    seqs = ops.Seqs(w.tables[:, :20].contiguous().cuda(), torch.tensor([600, 320], dtype=torch.int32).cuda())
    lists, counts = run_select(w, q, b.cuda(), [1, 1], 6, 1, 1, seqs=seqs, e=e)
    assert int(e) == CAPACITY
    w.ctx = [320, 320]
    check_lists(lists, counts, ref.select(w, q, b, [1, 1], 6, 1, 1), 6)


# ---------------------------------------------------------------- attention


def random_lists(ctx, q_lens, hkv, width, seed):
    g = np.random.default_rng(seed)
    lists = []
    for i, (_, vis) in enumerate(ref.rows_of(ctx, q_lens)):
        n = -(-vis // 16)
        lists.append([sorted(g.choice(n, size=min(n, int(g.integers(0, width + 1)) if (i + h) % 3 else width), replace=False).tolist())
                      for h in range(hkv)])
    return lists


def as_tensors(lists, hkv, width, extra=0):
    t = torch.full((len(lists) + extra, hkv, width), 2 ** 31 - 1, dtype=torch.int32)
    c = torch.full((len(lists) + extra, hkv), 5, dtype=torch.int32)
    for r, heads in enumerate(lists):
        for h, x in enumerate(heads):
            t[r, h, :len(x)] = torch.tensor(x, dtype=torch.int32)
            c[r, h] = len(x)
    return t.cuda(), c.cuda()


def check_out(got, want, mag, big, kind, dtype):
    tol = mag * (2.0 ** -15 + (2.0 ** -11 if kind == "k8v4" else 0.0) + big[..., None] * 2.0 ** -18)
    tol = tol + (want.abs() + tol) * (torch.finfo(dtype).eps / 2) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    bad = (got.double().cpu() - want).abs() > tol
    assert torch.isfinite(got).all()
    assert not bad.any(), f"{int(bad.sum())} outputs off, worst {float(((got.double().cpu() - want).abs() / tol).max())} of the tolerance"


def run_attention(w, q, q_lens, lists, width, dtype, ragged=False, extra=0, e=None, scale=None, cache=None):
    t, c = as_tensors(lists, w.hkv, width, extra)
    rows = q.shape[0] + extra
    qq = torch.cat([q, torch.ones(extra, *q.shape[1:], dtype=q.dtype)]).cuda()
    guard = GuardedOut((rows, *q.shape[1:]), dtype, "cuda")
    ops.pkv_paged_attention_selected(guard.out, qq, scale or w.d ** -0.5, cache or w.on_gpu(), w.seqs(1 if ragged else q_lens[0]), t, c,
                                     cu(q_lens) if ragged else None, err_flags=e)
    torch.cuda.synchronize()
    guard.check()
    if extra:   # rows behind the last sequence keep what they held
        assert torch.isnan(guard.out[q.shape[0]:].float()).all()
    return guard.out[:q.shape[0]]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H,hkv,d", [(4, 1, 64), (8, 8, 128), (16, 2, 128), (6, 3, 64), (32, 8, 128)])
@pytest.mark.parametrize("width", [1, 5, 40])
def test_attention(kind, H, hkv, d, width):
    w = ref.World(kind, [0, 1, 15, 16, 17, 40, 300, 700], hkv, d, seed=H + width)
    q_lens = [1] * len(w.ctx)
    q = queries(w, len(w.ctx), H)
    lists = random_lists(w.ctx, q_lens, hkv, width, H)
    e = err()
    want = ref.attention(w, q, d ** -0.5, q_lens, lists)
    for dtype in (torch.float32, w.q_dtype):
        check_out(run_attention(w, q, q_lens, lists, width, dtype, e=e), *want, kind, dtype)
    assert int(e) == 0


@pytest.mark.parametrize("kind,qd", [("bf16", None), ("f16", None), ("i8", torch.float16), ("e4m3", torch.bfloat16), ("k8v4", torch.float16)])
@pytest.mark.parametrize("q_lens,ragged", [([4] * 3, False), ([30, 0, 7], True), ([1, 20, 7], True)])
def test_attention_of_several_tokens(kind, qd, q_lens, ragged):
    w = ref.World(kind, [300, 20, 101], 2, 128, seed=5, q_dtype=qd)
    q = queries(w, sum(q_lens), 8)
    lists = random_lists(w.ctx, q_lens, 2, 9, 4)
    want = ref.attention(w, q, 0.2, q_lens, lists)
    got = run_attention(w, q, q_lens, lists, 9, torch.float32, ragged, extra=4 if ragged else 0, scale=0.2)
    check_out(got, *want, kind, torch.float32)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("H,hkv,d", [(8, 2, 128), (4, 2, 64), (8, 1, 128), (2, 2, 64), (2, 2, 128), (8, 1, 64)])
@pytest.mark.parametrize("ctx,q_lens,width", [([300, 150, 101], [130, 129, 64], 9), ([1000], [200], 40), ([90, 16, 400], [90, 0, 300], 3),
                                              ([5, 2000], [70, 260], 64)])
def test_chunks_of_prompts(kind, H, hkv, d, ctx, q_lens, width):
    # the first tokens of a sequence shorter than its query tokens see nothing
    w = ref.World(kind, ctx, hkv, d, seed=d + H)
    q = queries(w, sum(q_lens), H)
    lists = random_lists(ctx, q_lens, hkv, width, 4)
    want = ref.attention(w, q, 0.15, q_lens, lists)
    e = err()
    for dtype in (torch.float32, w.q_dtype):
        got = run_attention(w, q, q_lens, lists, width, dtype, ragged=True, extra=5, scale=0.15, e=e)
        check_out(got, *want, kind, dtype)
    assert int(e) == 0


def test_chunks_of_prompts_with_bad_entries_and_tables():
    w = ref.World("bf16", [400, 300], 2, 64, seed=23)
    q_lens = [64, 64]
    q = queries(w, 128, 8)
    given, taken = [], []
    for _, vis in ref.rows_of(w.ctx, q_lens):
        n = -(-vis // 16)
        given.append([[0, n + 3, 2, 2, 1, n - 1], [-1, 5, 4, n]])
        taken.append([[0, 2, n - 1], [5]])
    e = err()
    got = run_attention(w, q, q_lens, given, 6, torch.float32, ragged=True, scale=0.15, e=e)
    assert int(e) == PAGE_LIST
    check_out(got, *ref.attention(w, q, 0.15, q_lens, taken), "bf16", torch.float32)
    good = w.tables.clone()
    w.tables[0, 2], w.tables[1, 5] = -1, 10 ** 6
    e.zero_()
    got = run_attention(w, q, q_lens, taken, 6, torch.float32, ragged=True, scale=0.15, e=e)
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
    got = run_attention(w, q, q_lens, lists, 6, torch.float32, ragged=True, scale=0.15).double().cpu()
    fine = torch.isfinite(want)
    assert 0 < int((~fine).sum()) < fine.numel() / 2
    assert torch.equal(torch.isfinite(got), fine)
    tol = mag * (2.0 ** -15 + big[..., None] * 2.0 ** -18)
    assert ((got - want).abs()[fine] <= tol[fine] + want.abs()[fine] * 2.0 ** -24).all()


@pytest.mark.parametrize("kind", KINDS)
def test_long_lists_by_clusters(kind):
    w = ref.World(kind, [20000], 1, 64, seed=9)
    q = queries(w, 1, 8)
    lists = [[sorted(np.random.default_rng(1).choice(1250, size=1003, replace=False).tolist())]]
    want = ref.attention(w, q, 0.125, [1], lists)
    check_out(run_attention(w, q, [1], lists, 1100, torch.float32), *want, kind, torch.float32)


def test_unlisted_pages_are_not_read():
    w = ref.World("bf16", [200, 330], 2, 64, seed=11)
    q = queries(w, 2, 4)
    lists = [[[0, 3, 12], [1]], [[], [2, 20]]]
    want = ref.attention(w, q, 0.125, [1, 1], lists)
    for s, n in enumerate((13, 21)):
        for p in range(n):
            for h in range(2):
                if p not in lists[s][h]:
                    w.cache.k[int(w.tables[s, p]), :, h] = float("nan")
                    w.cache.v[int(w.tables[s, p]), :, h] = float("inf")
    got = run_attention(w, q, [1, 1], lists, 4, torch.float32)
    check_out(got, *want, "bf16", torch.float32)
    assert not got[1, :2].any()


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_what_one_token_lists_reaches_no_other(kind, d, value):
    # neighbouring tokens share a pass over the union of their lists; an infinity or NaN in the V of a page that one of them
    # lists, or of a token that only the later ones see, reaches their rows alone
    w = ref.World(kind, [200, 100], 2, d, seed=21)
    q_lens = [5, 3]
    q = queries(w, 8, 8)
    lists = [[[0, 3, 5], [12]], [[3, 5, 12], [1, 12]], [[2, 3], [2]], [[3, 11, 12], [12]], [[7, 12], [0, 12]],
             [[6], [6]], [[1, 6], [0, 6]], [[6], [3]]]
    w.cache.v[int(w.tables[0, 5]), 3, 0] = value           # sequence 0, kv head 0: tokens 0 and 1 list page 5
    w.cache.v[int(w.tables[0, 2]), 1, 1, 7] = value        # kv head 1, one dim: token 2
    w.cache.v[int(w.tables[0, 12]), 198 % 16] = value      # position 198, seen by the last two tokens
    w.cache.v[int(w.tables[1, 6]), 99 % 16, 1] = value     # the last position of sequence 1
    w.v64 = w.cache.v.double()
    want, mag, big = ref.attention(w, q, 0.2, q_lens, lists)
    got = run_attention(w, q, q_lens, lists, 4, torch.float32, ragged=True, scale=0.2).double().cpu()
    fine = torch.isfinite(want)
    assert 0 < int((~fine).sum()) < fine.numel() / 2
    assert torch.equal(torch.isfinite(got), fine)
    tol = mag * (2.0 ** -15 + big[..., None] * 2.0 ** -18)
    assert ((got - want).abs()[fine] <= tol[fine] + want.abs()[fine] * 2.0 ** -24).all()


def test_bad_entries_are_skipped_and_flagged():
    w = ref.World("f16", [100, 64, 40, 600], 1, 64, seed=12)
    q = queries(w, 4, 4)
    given = [[[0, 3, 3, 2, 6, 7, 99, -1]], [[5, 1, 2, 4, 0]], [[-2, 0, 2, 1, 9]], [list(range(30, 0, -1)) + [31, 37, 36] + [20, 50, 37]]]
    taken = [[[0, 3, 6]], [[1, 2]], [[0, 2]], [[30, 31, 37]]]
    want = ref.attention(w, q, 0.125, [1] * 4, taken)
    e = err()
    got = run_attention(w, q, [1] * 4, given, 40, torch.float32, e=e)
    assert int(e) == PAGE_LIST
    check_out(got, *want, "f16", torch.float32)
    # counts outside [0, max_pages] are cut to it
    t, c = as_tensors(taken, 1, 3)
    c[0], c[1] = 1000, -7
    t[0, 0] = torch.tensor([0, 3, 6])
    out = torch.empty(4, 4, 64, device="cuda")
    ops.pkv_paged_attention_selected(out, q.cuda(), 0.125, w.on_gpu(), w.seqs(), t, c)
    taken[1] = [[]]
    check_out(out, *ref.attention(w, q, 0.125, [1] * 4, taken), "f16", torch.float32)


def test_attention_flags_bad_tables():
    w = ref.World("i8", [100, 100], 1, 64, seed=13)
    q = queries(w, 2, 4)
    e = err()
    good = w.tables.clone()
    w.tables[0, 2], w.tables[1, 5] = -1, 10 ** 6
    got = run_attention(w, q, [1, 1], [[[0, 2, 4]], [[5]]], 3, torch.float32, e=e)
    assert int(e) == OOB_BLOCK
    w.tables = good
    check_out(got, *ref.attention(w, q, 0.125, [1, 1], [[[0, 4]], [[]]]), "i8", torch.float32)
    e.zero_()
    w.tables = good[:, :5].contiguous()   # tables shorter than the context
    got = run_attention(w, q, [1, 1], [[[0, 4]], [[1, 2, 6]]], 3, torch.float32, e=e)
    assert int(e) == CAPACITY | PAGE_LIST
    check_out(got, *ref.attention(w, q, 0.125, [1, 1], [[[0, 4]], [[1, 2]]]), "i8", torch.float32)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_scales_of_every_size(kind):
    w = ref.World(kind, [160], 1, 128, seed=14)
    vs = w.cache.v_scale
    for p, x in enumerate([2.0 ** -120, 0.0, 1e-30, 2.0 ** -126, 1.0, 3.0, 0.0, 1e10, 2.0 ** -10, 1e20]):
        vs[int(w.tables[0, p])] = x
    codes = w.cache.v.float().double()
    w.v64 = codes * vs[:, None, :, None].double()
    q = queries(w, 1, 4)
    for pages in ([0], [1], [1, 2, 3], [0, 1, 2, 3, 4, 5], list(range(10)), [7, 8]):
        want = ref.attention(w, q, 0.01, [1], [[pages]])
        got = run_attention(w, q, [1], [[pages]], 10, torch.float32, scale=0.01)
        # below 2^-126 fp32 itself rounds by 2^-149
        tol = want[1] * 2.0 ** -14 + 2.0 ** -130
        assert ((got.double().cpu() - want[0]).abs() <= tol).all(), pages


# ---------------------------------------------------------------- the three together


@pytest.mark.parametrize("kind", ["bf16", "f16", "k8v4"])
@pytest.mark.parametrize("q_len", [1, 2])
def test_a_decode_step_that_selects(kind, q_len):
    """DecodeStep's schedule: with room for every page the oracle's whole attention, else that of the selected ones."""
    from paged_decode_attention_cache_gb300 import workloads as W
    from paged_decode_attention_cache_gb300.runner import DecodeStep
    from tests.helpers import oracle_attention
    w = W.build(name="t", seed=31, context_lens=[40, 17, 260, 129], num_heads=8, num_kv_heads=2, head_dim=64, cache=kind, q_len=q_len)
    st = DecodeStep(w, "cuda", out_dtype=torch.float32, schedule="selected", max_pages=17)
    st.step()
    assert st.error_flags() == 0 and st.launches_per_step() == 4
    assert np.abs(st.out.double().cpu().numpy() - oracle_attention(w, threads=8)).max() <= (2e-2 if kind == "k8v4" else 2e-3)
    few = DecodeStep(w, "cuda", out_dtype=torch.float32, schedule="selected", max_pages=5, keep_first=0, keep_last=2)
    few.step()
    assert few.error_flags() == 0
    n = [-(-(c - q_len + j + 1) // 16) for c in w.context_lens.tolist() for j in range(q_len)]
    assert few.page_counts.tolist() == [[min(5, k)] * 2 for k in n]
    for r, k in enumerate(n):
        assert {k - 1, max(k - 2, 0)} <= set(few.page_lists[r, 0].tolist())
    # the lists' attention by the framework's other call, where that has one list for all kv heads
    if q_len == 1:
        one = few.page_lists[:, :1].expand(-1, 2, -1).contiguous()
        a, b = torch.empty_like(few.out), torch.empty_like(few.out)
        ops.pkv_paged_attention_selected(a, few.q, w.scale, few.cache, few.seqs, one, few.page_counts, None, few.err)
        ws = ops.sparse_workspace(w.num_seqs, 2, 64, 5)
        ops.pkv_paged_attention_sparse(b, few.q, w.scale, few.cache, few.seqs, one[:, 0].contiguous(), few.page_counts[:, 0].contiguous(),
                                       ws, few.err)
        assert few.error_flags() == 0
        assert (a - b).abs().max() <= (2e-2 if kind == "k8v4" else 2e-3)


def test_all_pages_is_the_whole_attention():
    # a list that leaves nothing out gives what the framework's own attention gives
    w = ref.World("bf16", [100, 333, 16], 2, 128, seed=15)
    q = queries(w, 3, 8).cuda()
    cache, seqs = w.on_gpu(), w.seqs()
    b = ops.key_bounds(cache)
    ops.pkv_key_bounds(b, cache, seqs, cu(w.ctx))
    lists = torch.empty(3, 2, 32, dtype=torch.int32, device="cuda")
    counts = torch.empty(3, 2, dtype=torch.int32, device="cuda")
    ops.pkv_select_pages(lists, counts, q, b, cache, seqs)
    one, all_ = torch.empty(3, 8, 128, device="cuda"), torch.empty(3, 8, 128, device="cuda")
    ops.pkv_paged_attention_selected(one, q, 0.1, cache, seqs, lists, counts)
    ops.pkv_paged_attention(all_, q, 0.1, cache, seqs)
    # both within check_out's tolerance of the same numbers
    _, mag, big = ref.attention(w, q.cpu(), 0.1, [1] * 3, [[list(range(-(-c // 16)))] * 2 for c in w.ctx])
    tol = 2 * mag * (2.0 ** -15 + big[..., None] * 2.0 ** -18)
    assert ((one - all_).double().cpu().abs() <= tol).all()


@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3", "k8v4"])
def test_steps_on_a_stream_and_in_a_graph(kind):
    """Prompts in chunks, then decode steps: append, bounds, selection, attention; the steps captured once and replayed
    with other tokens, on a stream of their own, against the definitions over the cache that results."""
    hkv, H, d, B, pages = 2, 8, 64, 3, 6
    w = ref.World(kind, [16 * 12] * B, hkv, d, seed=16, extra_cols=0)
    cache = ops.Cache.empty(kind, w.cache.num_blocks, hkv, d)
    tables = w.tables.cuda()
    dt = ref.SRC.get(kind, torch.bfloat16)
    g = torch.Generator().manual_seed(17)
    ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
    b = ops.key_bounds(cache)
    lists = torch.empty(B, hkv, pages, dtype=torch.int32, device="cuda")
    counts = torch.empty(B, hkv, dtype=torch.int32, device="cuda")
    q, out = torch.empty(B, H, d, dtype=dt, device="cuda"), torch.empty(B, H, d, device="cuda")
    kn, vn = (torch.empty(B, hkv, d, dtype=dt, device="cuda") for _ in "kv")
    slots = torch.empty(B, dtype=torch.int64, device="cuda")

    def append(k, v, seqs, c, sl):
        if kind in ("i8", "e4m3"):
            ops.pkv_quantize_kv_blocks(cache, k, v, seqs, c)
        elif kind == "k8v4":
            ops.pkv_quantize_kv(cache, k, v, sl)
        else:
            ops.pkv_reshape_and_cache(cache, k, v, sl)
        ops.pkv_key_bounds(b, cache, seqs, c)

    def step():
        append(kn, vn, ops.Seqs(tables, ctx), None, slots)
        ops.pkv_select_pages(lists, counts, q, b, cache, ops.Seqs(tables, ctx), keep_first=1, keep_last=1)
        ops.pkv_paged_attention_selected(out, q, 0.15, cache, ops.Seqs(tables, ctx), lists, counts)

    def slots_of(first, n):
        return torch.tensor([int(w.tables[s, (f + i) // 16]) * 16 + (f + i) % 16 for s, (f, m) in enumerate(zip(first, n)) for i in range(m)],
                            dtype=torch.int64, device="cuda")

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        have = [0] * B
        for chunk in ([50, 1, 33], [90, 120, 16]):
            T = sum(chunk)
            k, v = (torch.randn(T, hkv, d, generator=g).to(dt).cuda() for _ in "kv")
            sl = slots_of(have, chunk)
            have = [a + c for a, c in zip(have, chunk)]
            ctx.copy_(torch.tensor(have, dtype=torch.int32))
            append(k, v, ops.Seqs(tables, ctx), cu(chunk), sl)

        def feed():
            for x in (q, kn, vn):
                x.copy_(torch.randn(x.shape, generator=g).to(x.dtype))
            slots.copy_(slots_of(have, [1] * B))
            for s in range(B):
                have[s] += 1
            ctx.copy_(torch.tensor(have, dtype=torch.int32))

        graph = None
        for i in range(20):
            feed()
            if i == 1:
                side.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    step()
            if graph is None:
                step()
            else:
                graph.replay()
            side.synchronize()
            check_step(w, kind, cache, b, have, q, out, lists, counts, pages)


def check_step(w, kind, cache, b, have, q, out, lists, counts, pages):
    got = ref.World.__new__(ref.World)
    move = lambda x: None if x is None else x.cpu()  # noqa: E731
    got.kind, got.ctx, got.hkv, got.d, got.tables = kind, list(have), w.hkv, w.d, w.tables
    got.cache = ops.Cache(kind, cache.k.cpu(), cache.v.cpu(), move(cache.k_scale), move(cache.v_scale), move(cache.v_zero))
    c = got.cache
    if kind in ref.SRC:
        got.k64, got.v64 = c.k.double(), c.v.double()
    elif kind in ("i8", "e4m3"):
        got.k64, got.v64 = c.k.float().double() * c.k_scale[:, None, :, None].double(), c.v.float().double() * c.v_scale[:, None, :, None].double()
    else:
        wide = lambda x: x.permute(0, 2, 1, 3).repeat_interleave(32, dim=-1).double()  # noqa: E731
        codes = torch.stack([c.v & 15, c.v >> 4], dim=-1).flatten(-2)
        got.k64 = c.k.double() * c.k_scale.permute(0, 2, 1)[..., None].double()
        got.v64 = codes.double() * wide(c.v_scale) + wide(c.v_zero)
    want_b = ref.bounds(got, torch.zeros_like(b.cpu().view(torch.uint8)).view(b.dtype) if b.element_size() == 1 else torch.zeros_like(b.cpu()),
                        list(have))
    used = torch.cat([w.tables[s, :-(-n // 16)] for s, n in enumerate(have)]).long()
    assert torch.equal(numbers(b.cpu())[used], numbers(want_b)[used])
    want = ref.select(got, q.cpu(), want_b, [1] * len(have), pages, 1, 1)
    check_lists(lists.cpu(), counts.cpu(), want, pages)
    check_out(out, *ref.attention(got, q.cpu(), 0.15, [1] * len(have), want), kind, torch.float32)


def test_two_streams_at_once():
    # no workspace: calls on two streams do not disturb one another
    w = ref.World("bf16", [3000] * 4, 2, 128, seed=18)
    cache, seqs, b = w.on_gpu(), w.seqs(), full_bounds(w).cuda()
    q = [queries(w, 4, 8, seed=i).cuda() for i in (1, 2)]
    lists = [torch.empty(4, 2, 40, dtype=torch.int32, device="cuda") for _ in q]
    counts = [torch.empty(4, 2, dtype=torch.int32, device="cuda") for _ in q]
    out = [torch.empty(4, 8, 128, device="cuda") for _ in q]

    def go(i):
        ops.pkv_select_pages(lists[i], counts[i], q[i], b, cache, seqs)
        ops.pkv_paged_attention_selected(out[i], q[i], 0.1, cache, seqs, lists[i], counts[i])

    alone = []
    for i in (0, 1):
        go(i)
        torch.cuda.synchronize()
        alone.append((lists[i].clone(), out[i].clone()))
    streams = [torch.cuda.Stream() for _ in q]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                go(i)
    torch.cuda.synchronize()
    for i in (0, 1):
        assert torch.equal(lists[i], alone[i][0]) and torch.equal(out[i], alone[i][1])


def test_blocks_past_32_bit_offsets():
    # 2^31 bytes of keys into the pool and beyond
    hkv, d = 8, 128
    nb = (2 ** 31) // (16 * hkv * d * 2) + 3000
    k, v = (torch.zeros(nb, 16, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    cache = ops.Cache("bf16", k, v)
    g = torch.Generator().manual_seed(19)
    ids = torch.randperm(2900, generator=g)[:30] + nb - 2950
    for x in (k, v):
        x[ids.cuda()] = torch.randn(30, 16, hkv, d, generator=g).bfloat16().cuda()
    tables = ids.to(torch.int32)[None].contiguous().cuda()
    seqs = ops.Seqs(tables, torch.tensor([470], dtype=torch.int32).cuda())
    b = ops.key_bounds(cache)
    ops.pkv_key_bounds(b, cache, seqs, cu([470]))
    q = torch.randn(1, 16, d, generator=g).bfloat16()
    lists = torch.empty(1, hkv, 7, dtype=torch.int32, device="cuda")
    counts = torch.empty(1, hkv, dtype=torch.int32, device="cuda")
    out = torch.empty(1, 16, d, device="cuda")
    ops.pkv_select_pages(lists, counts, q.cuda(), b, cache, seqs)
    ops.pkv_paged_attention_selected(out, q.cuda(), 0.1, cache, seqs, lists, counts)
    w = ref.World.__new__(ref.World)
    w.kind, w.ctx, w.hkv, w.d = "bf16", [470], hkv, d
    w.tables = torch.arange(30, dtype=torch.int32)[None]
    kk, vv = k[ids.cuda()].cpu(), v[ids.cuda()].cpu()
    w.cache, w.k64, w.v64 = ops.Cache("bf16", kk, vv), kk.double(), vv.double()
    want_b = ref.bounds(w, torch.zeros(30, hkv, 2, d).bfloat16(), [470])
    assert torch.equal(b[ids.cuda()].cpu(), want_b)
    want = ref.select(w, q, want_b, [1], 7, 1, 1)
    check_lists(lists.cpu(), counts.cpu(), want, 7)
    check_out(out, *ref.attention(w, q, 0.1, [1], want), "bf16", torch.float32)
