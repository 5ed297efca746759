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
