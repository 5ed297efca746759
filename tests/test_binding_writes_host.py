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


@pytest.mark.parametrize("kind,good", [("f16", torch.float16), ("bf16", torch.bfloat16)])
@pytest.mark.parametrize("bad", [torch.float32, torch.float64, torch.float16, torch.bfloat16, torch.int8, torch.uint8, torch.int32])
def test_a_write_of_another_type_than_the_caches(kind, good, bad):
    # its bits would be stored as the cache's numbers, and of a narrower type more read than there is
    cache = ops.Cache.empty(kind, 4, HKV, D, device="cpu")
    x, y, slots = torch.zeros(3, HKV, D, dtype=good), torch.zeros(3, HKV, D, dtype=bad), torch.zeros(3, dtype=torch.int64)
    for k, v in ((x, y), (y, x), (y, y)):
        with pytest.raises(ValueError, match="CUDA device" if bad == good else "k_new / v_new must be"):
            ops.pkv_reshape_and_cache(cache, k, v, slots)


def test_a_write_of_16_bits_under_the_caches_own_name_for_them():
    cache = ops.Cache("bf16", torch.zeros(4, 16, HKV, D, dtype=torch.int16), torch.zeros(4, 16, HKV, D, dtype=torch.int16))
    x = torch.zeros(3, HKV, D, dtype=torch.int16)
    with pytest.raises(ValueError, match="CUDA device"):
        ops.pkv_reshape_and_cache(cache, x, x, torch.zeros(3, dtype=torch.int64))


@pytest.mark.parametrize("other", [torch.bfloat16, torch.float32, torch.uint8, torch.float64])
def test_a_quantised_write_of_two_types(other):
    cache = ops.Cache.empty("k8v4", 4, HKV, D, device="cpu")
    x, y, slots = torch.zeros(3, HKV, D, dtype=torch.float16), torch.zeros(3, HKV, D, dtype=other), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="k_new / v_new must be"):
        ops.pkv_quantize_kv(cache, x, y, slots)
    with pytest.raises((ValueError, KeyError)):
        ops.pkv_quantize_kv(cache, y, x, slots)
