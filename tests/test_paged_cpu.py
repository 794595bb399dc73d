"""Checks of the paged caches' Python side that need no GPU."""
import re

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from speculative_decoding_exact_gb300 import abi, runtime  # noqa: E402
from tests import kv4_util as u, paged_util as pu  # noqa: E402


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


@pytest.mark.parametrize("kind", ["kv4", "bf16"])
@pytest.mark.parametrize("nq,M,length", [(2, 3, 1000), (26, 16, 700)])
def test_the_accuracy_bound_notices_a_lost_part(kind, nq, M, length):
    """With all parts of q and p an exact sum lies far below the bound that the GPU tests
    assert; without one of either it lies above."""
    rng = np.random.default_rng(4)
    k, v = (rng.standard_normal((length, 256)).astype(np.float32) for _ in range(2))
    if kind == "kv4":
        k, v = (u.from_pages(u.to_pages(*(np.concatenate([a, np.zeros((-length % 16,) + a.shape[1:], a.dtype)])
                                          for a in u.quantise_rows(x, 2)))) for x in (k, v))
    else:
        k, v = (pu.parts_bf16(x, 1).reshape(length, 2, 128) for x in (k, v))
    q = rng.standard_normal((M, nq, 128)).astype(np.float32)
    want = pu.attention64(q, k, v, nq, 0, 0, length)[0]
    parts, n = (pu.parts_binary16, 2) if kind == "kv4" else (pu.parts_bf16, 3)
    err = {(a, b): pu.rel_l2(pu.attention_in_parts(q, k, v, nq, length, parts, a, b), want)
           for a, b in ((n, n), (n - 1, n), (n, n - 1), (n - 1, n - 1))}
    assert err[n, n] < pu.ACCURACY / 8
    assert min(err[n - 1, n], err[n, n - 1], err[n - 1, n - 1]) > 1.5 * pu.ACCURACY
