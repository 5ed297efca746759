"""Steps without a token: every call of the decode chain takes them, whatever strides the empty tensors have."""
import pytest
import torch

from paged_decode_attention_cache_gb300 import ops

pytestmark = pytest.mark.gpu
H, HKV, D = 4, 2, 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_decode_attention_cache_gb300 import build
    build.build()
    ops.lib()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("strides", [None, (1, 1, 1), (0, 0, 0)])
def test_no_tokens(strides):
    def none(heads):
        t = torch.empty((0, heads, D), dtype=torch.bfloat16, device="cuda")
        return t if strides is None else t.as_strided((0, heads, D), strides)

    seqs = ops.Seqs(torch.zeros((3, 1), dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda"))
    cache = ops.Cache.empty("i8", 2, HKV, D)
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    ops.pkv_quantize_kv_blocks(cache, none(HKV), none(HKV), seqs, torch.zeros(4, dtype=torch.int32, device="cuda"))
    rope = ops.Rope(ops.pkv_rope_frequencies(D, 1e4).cuda(), D)
    empty = torch.empty(0, dtype=torch.int64, device="cuda")
    ops.pkv_rope_and_cache(none(H), none(H), none(HKV), None, rope, empty, k_out=none(HKV))
    half = ops.Cache.empty("bf16", 2, HKV, D)
    ops.pkv_rope_and_cache(none(H), none(H), none(HKV), none(HKV), rope, empty, half, empty)
    torch.cuda.synchronize()
    for t, was in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), before):
        assert torch.equal(t, was)
    assert not half.k.any() and not half.v.any()


def test_no_visible_tokens_in_a_cache_of_one_block():
    # all contexts zero: every attention call writes zeros and reads no block
    seqs = ops.Seqs(torch.full((3, 1), -1, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"))
    cache = ops.Cache.empty("e4m3", 1, HKV, D)
    q = torch.ones((3, H, D), dtype=torch.bfloat16, device="cuda")
    ws, err = ops.balanced_workspace(3, HKV, D), torch.zeros(1, dtype=torch.int32, device="cuda")
    for call in (lambda o: ops.pkv_paged_attention(o, q, 0.125, cache, seqs, err),
                 lambda o: ops.pkv_paged_attention_balanced(o, q, 0.125, cache, seqs, ws, err),
                 lambda o: ops.pkv_paged_attention_scored(o, q, 0.125, cache, seqs, ops.Scores(1.0), ws, err)):
        out = torch.full_like(q, float("nan"))
        call(out)
        assert int(err.item()) == 0 and not out.any()
