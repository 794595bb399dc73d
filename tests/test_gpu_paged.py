"""Attention over the paged caches where a call is easily right for one block and
wrong for another: a row's bits when a window starts in another chunk of keys,
scores far past a softmax's usual range, infinite values, windows that limit the
chunks, the operands' precision, and calls that follow each other.

One-hot rows: where the largest score leads by more than 2^8 (base 2) and more than
the products' rounding, every other weight is 0 in fp32 and the row's output is
that key's V row, off by the roundings of one product, one sum and one quotient.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from speculative_decoding_exact_gb300 import abi, runtime  # noqa: E402
from tests import kv4_util as u  # noqa: E402
from tests import test_gpu_kv4 as base  # noqa: E402

EPS = 2.0 ** -24
KINDS = base.KINDS
attend, cache, context, status, sync = base.attend, base.cache, base.context, base.status, base.sync


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    for c in base._CTX.values():
        c.close()
    base._CTX.clear()


def same_bits(a, b):
    return np.array_equal(a.view(np.uint32), b.view(np.uint32))


# ---------------------------------------------------------------------------
# a row's bits
# ---------------------------------------------------------------------------
# (query heads, KV heads, rows, window, row whose window starts a chunk, smaller
# blocks).  More than 32 chunks each, of 1 to 7 tiles of 128 keys.
WIDE = {"few": (4, 4, 16, 8192, 8, ((8, 8), (8, 1), (15, 1), (9, 4))),
        "few_one_head": (8, 1, 2, 8192, 1, ((1, 1),)),
        "few_sinks": (16, 4, 4, 12000, 2, ((2, 2), (2, 1), (3, 1))),
        "tile": (52, 4, 8, 32768, 4, ((4, 4), (5, 2), (6, 2))),
        "tile_one_head": (12, 1, 9, 8192, 5, ((5, 4), (7, 2))),
        "two_tiles": (12, 1, 16, 8192, 5, ((5, 11),))}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", sorted(WIDE))
def test_a_window_that_starts_in_another_chunk_leaves_a_rows_bits(kind, case):
    """The block's first row sees one chunk of keys that its later rows do not."""
    nq, nkv, M, window, row, parts = WIDE[case]
    ctx = context(nq, nkv, max_ctx=65536)
    sinks = 300 if case == "few_sinks" else 0
    # row `row` sees from a multiple of 84 tiles on, which starts a chunk of 1, 2, 3,
    # 4, 6 or 7 tiles
    n_past = 84 * 128 + window - 1 - row
    kv, _, _, _ = cache(ctx, kind, n_past + M, 31)
    q = np.random.default_rng(5).standard_normal((M, nq, 128)).astype(np.float32) * 3
    whole = attend(ctx, kv, kind, q, window, sinks)
    for i, m in parts:
        kv.seq_len[0] = n_past + i + m
        part = attend(ctx, kv, kind, q[i:i + m], window, sinks)
        assert same_bits(part, whole[i:i + m]), (i, m)
    assert status(ctx) == 0
