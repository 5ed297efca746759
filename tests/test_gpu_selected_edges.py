"""Page selection and attention over selected pages where numbers leave the usual range: scales, bounds and queries of very
different sizes, infinities beside finite numbers (against tests/selected_reference.py; the attention's tolerances are
tests/test_gpu_selected.py's)."""
import math

import pytest
import torch

from paged_decode_attention_cache_gb300 import ops
from tests import selected_reference as ref
from tests.test_gpu_selected import queries, random_lists
from tests.test_gpu_selected_wide import copies, together, wide_attention

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
