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
