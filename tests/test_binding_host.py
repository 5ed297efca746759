"""What the Python module of the decode step's calls refuses before it asks for a GPU."""
import pytest
import torch

from paged_decode_attention_cache_gb300 import ops

B, H, HKV, D = 2, 4, 2, 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_decode_attention_cache_gb300 import build
    build.build()


def cache(kind="i8"):
    return ops.Cache.empty(kind, 4, HKV, D, device="cpu")


def seqs(n=B, q_len=1):
    return ops.Seqs(torch.zeros((n, 1), dtype=torch.int32), torch.ones(n, dtype=torch.int32), q_len)


def zeros(*shape, dtype=torch.float16):
    return torch.zeros(shape, dtype=dtype)


def test_host_tensors_are_refused_by_every_call():
    q, k, ints = zeros(B, H, D), zeros(B, HKV, D), torch.zeros(B + 1, dtype=torch.int32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    rope = ops.Rope(torch.zeros(D // 2, dtype=torch.int64), D)
    for call in (lambda: ops.pkv_paged_attention_balanced(q.clone(), q, 0.125, cache(), seqs(), ws),
                 lambda: ops.pkv_paged_attention_scored(q.clone(), q, 0.125, cache(), seqs(), ops.Scores(), ws),
                 lambda: ops.pkv_gather_kv_cache_dequant(k.clone(), k.clone(), ints, cache(), seqs()),
                 lambda: ops.pkv_quantize_kv_blocks(cache(), k, k, seqs()),
                 lambda: ops.pkv_rope_and_cache(q.clone(), q, k, None, rope, torch.zeros(B, dtype=torch.int64), k_out=k.clone())):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


def refused(text, call):
    with pytest.raises(ValueError, match=text):
        call()


@pytest.mark.parametrize("kind", ["f16", "k8v4", "i8"])
def test_the_balanced_call_refuses_buffers_that_are_too_small(kind):
    q, ws = zeros(B, H, D), torch.zeros(1 << 20, dtype=torch.uint8)
    call = lambda out, q, s=seqs(), c=None: ops.pkv_paged_attention_balanced(out, q, 0.125, c or cache(kind), s, ws)  # noqa: E731
    refused("q and out", lambda: call(zeros(B, H, D), q[:1]))                       # a row too few
    refused("q and out", lambda: call(zeros(B, H - 1, D), q))
    refused("q and out", lambda: call(zeros(B, H, D), zeros(B, H, D // 2)))         # another head_dim
    refused("q and out", lambda: call(q.clone(), q, seqs(q_len=2)))
    refused("q must be", lambda: call(q.clone(), q.flatten()))
    refused("context_lens", lambda: call(q.clone(), q, ops.Seqs(torch.zeros((B, 1), dtype=torch.int32), torch.ones(1, dtype=torch.int32))))
    # as large, or larger (a buffer of the largest batch): not refused for its size
    refused("CUDA device", lambda: call(q.clone(), q))
    refused("CUDA device", lambda: call(zeros(B + 3, H, D), zeros(B + 1, H, D)))


def test_the_read_back_refuses_outputs_and_offsets_that_do_not_fit():
    k, ints = zeros(5, HKV, D), torch.zeros(B + 1, dtype=torch.int32)
    call = lambda k, v, cu=ints: ops.pkv_gather_kv_cache_dequant(k, v, cu, cache(), seqs())  # noqa: E731
    refused("k_out and v_out", lambda: call(k, zeros(4, HKV, D)))
    refused("k_out and v_out", lambda: call(zeros(5, D - 1), zeros(5, D - 1)))
    refused("cu_seq_lens", lambda: call(k, k.clone(), ints[:B]))
    refused("CUDA device", lambda: call(k, k.clone()))


def test_a_cache_whose_tensors_disagree_is_refused():
    q, ws = zeros(B, H, D), torch.zeros(1 << 20, dtype=torch.uint8)
    call = lambda c: ops.pkv_paged_attention_balanced(q.clone(), q, 0.125, c, seqs(), ws)  # noqa: E731
    half, packed = cache("f16"), cache("k8v4")
    refused("v is smaller", lambda: call(ops.Cache("f16", half.k, half.v[:3])))
    refused("k is smaller", lambda: call(ops.Cache("f16", half.k.to(torch.int8), half.v)))
    for name in ("v", "k_scale", "v_scale", "v_zero"):
        c = cache("k8v4")
        setattr(c, name, getattr(c, name)[:3])
        refused(name + " is smaller", lambda: call(c))
    refused("v_zero is smaller", lambda: call(ops.Cache("k8v4", packed.k, packed.v, packed.k_scale, packed.v_scale)))


def test_lengths_are_whatever_int_takes():
    # a q_len or a window that comes out of a division or a tensor, as the other calls take them
    q, k, ws = zeros(B, H, D), zeros(B, HKV, D), torch.zeros(1 << 20, dtype=torch.uint8)
    for one, window in ((1.0, 32.0), (torch.tensor(1), torch.tensor(32.0)), (True, 32)):
        s = ops.Seqs(torch.zeros((B, 1), dtype=torch.int32), torch.ones(B, dtype=torch.int32), one, window)
        refused("CUDA device", lambda: ops.pkv_paged_attention_balanced(q.clone(), q, 0.125, cache(), s, ws))
        refused("CUDA device", lambda: ops.pkv_gather_kv_cache_dequant(k, k.clone(), torch.zeros(B + 1, dtype=torch.int32), cache(), s))
    s = ops.Seqs(torch.zeros((B, 1), dtype=torch.int32), torch.ones(B, dtype=torch.int32), None)
    with pytest.raises(TypeError):
        ops.pkv_paged_attention_balanced(q.clone(), q, 0.125, cache(), s, ws)
