"""What the cache writes by slot refuse before they ask for a GPU."""
import pytest
import torch

from paged_decode_attention_cache_gb300 import ops

HKV, D = 2, 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_decode_attention_cache_gb300 import build
    build.build()


@pytest.mark.parametrize("call,kind", [(ops.pkv_reshape_and_cache, "f16"), (ops.pkv_quantize_kv, "k8v4")])
def test_writes_by_slot(call, kind):
    cache = ops.Cache.empty(kind, 4, HKV, D, device="cpu")
    x, slots = torch.zeros(3, HKV, D, dtype=torch.float16), torch.zeros(3, dtype=torch.int64)
    for bad in ((cache, x[:2], x, slots), (cache, x, x[:2], slots), (cache, x, x, slots.int())):
        with pytest.raises(ValueError, match="k_new / v_new|slot_mapping"):
            call(*bad)
    with pytest.raises(ValueError, match="CUDA device"):
        call(cache, x, x, slots)
    with pytest.raises(ValueError, match="torch tensor"):
        call(cache, None, x, slots) if kind == "f16" else call(cache, x, None, slots)


def test_a_quantised_write_of_another_type():
    x = torch.zeros(3, HKV, D, dtype=torch.float64)
    with pytest.raises(KeyError):
        ops.pkv_quantize_kv(ops.Cache.empty("k8v4", 4, HKV, D, device="cpu"), x, x, torch.zeros(3, dtype=torch.int64))
