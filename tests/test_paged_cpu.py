"""Checks of the paged caches' Python side that need no GPU."""
import re

import pytest

torch = pytest.importorskip("torch")

from speculative_decoding_exact_gb300 import abi, runtime  # noqa: E402


def test_caches_say_what_their_pool_holds():
    text = open(abi.HEADER).read()
    for name, cls in (("ANY", runtime.PagedKV), ("BF16", runtime.DeviceKV), ("4BIT", runtime.DeviceKV4)):
        value = int(re.search(rf"#define SPEC_KV_{name}\s+(\d)", text).group(1))
        assert getattr(abi, f"KV_{name}") == cls.KIND == value
    assert abi.spec_kv().kind == abi.KV_ANY


def test_a_4bit_cache_has_no_bf16_rows():
    assert not issubclass(runtime.DeviceKV4, runtime.DeviceKV)
    for name in ("write_rows", "write_rows_bulk", "write_ring_rows", "ring_rows"):
        assert hasattr(runtime.DeviceKV, name) and not hasattr(runtime.DeviceKV4, name)


@pytest.mark.parametrize("k,v", [
    (torch.zeros(2, 256, dtype=torch.bfloat16), torch.zeros(2, 256, dtype=torch.bfloat16)),   # read past their end
    (torch.zeros(2, 128), torch.zeros(2, 128)),                                              # too narrow
    (torch.zeros(2, 512), torch.zeros(2, 512)),
    (torch.zeros(512), torch.zeros(512)),
    (torch.zeros(2, 256), torch.zeros(2, 256)),                                              # not on the GPU
])
def test_append_refuses_rows_of_another_shape_or_type(k, v):
    kv = runtime.DeviceKV4.__new__(runtime.DeviceKV4)
    kv.cfg = runtime.ModelConfig(hidden=512, n_layers=1, n_q_heads=4, n_kv_heads=2, head_dim=128, ffn=512, vocab=512)
    with pytest.raises(ValueError):
        kv.append(None, 0, k, v)
