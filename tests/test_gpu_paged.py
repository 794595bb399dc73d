"""Attention over the paged caches where a call is easily right for one block and
wrong for another: a row's bits when a window starts in another chunk of keys,
scores far past a softmax's usual range, infinite values, windows that limit the
chunks, the operands' precision, and calls that follow each other.

One-hot rows: where the largest score leads by more than 2^8 (base 2) and more than
the products' rounding, every other weight is 0 in fp32 and the row's output is
that key's V row, off by the roundings of one product, one sum and one quotient.
"""
import time

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from speculative_decoding_exact_gb300 import abi, runtime  # noqa: E402
from tests import kv4_util as u  # noqa: E402
from tests import paged_util as pu  # noqa: E402
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


# ---------------------------------------------------------------------------
# scores far past a softmax's usual range
# ---------------------------------------------------------------------------
def one_hot(q, k, v, nq, length):
    """Rows' V of the key with the largest score (causal), and which rows have one."""
    M, nkv = q.shape[0], k.shape[1]
    o, sure = np.zeros((M, nq, 128)), np.zeros((M, nq), dtype=bool)
    for h in range(nq):
        at = h // (nq // nkv)
        kh, vh, qh = k[:length, at], v[:length, at], q[:, h].astype(np.float64)
        s, size = kh @ qh.T, np.abs(kh) @ np.abs(qh).T                    # [length][M]
        for i in range(M):
            n = length - M + i + 1
            top = s[:n, i].argmax()
            rest = np.delete(s[:n, i], top)
            # split, 256 products' sums and the scaling (kv4_util), and 2^8 in base 2
            lead = (s[top, i] - rest.max()) if n > 1 else np.inf
            o[i, h] = vh[top]
            sure[i, h] = lead > 4 * 520 * EPS * size[:n, i].max() + 2.0 ** 12
    return o, sure


@pytest.mark.parametrize("nq,M", [(2, 3), (26, 3), (26, 16)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q_exp,k_exp", [(8, 8), (16, 12), (20, 12), (24, 12), (40, 12), (98, 0), (110, 0)])
def test_scores_of_any_size_that_fp32_holds(kind, q_exp, k_exp, nq, M):
    check_one_hot(kind, 2.0 ** q_exp, 2.0 ** k_exp, nq, M)


def check_one_hot(kind, q_scale, spread, nq, M):
    ctx = context(nq, 2)
    length = 700
    kv, k, v, _ = cache(ctx, kind, length, 17, spread=spread)
    q = (np.random.default_rng(3).standard_normal((M, nq, 128)) * q_scale).astype(np.float32)
    assert np.isfinite(q).all()
    got = attend(ctx, kv, kind, q, 0, 0).reshape(M, nq, 128)
    want, sure = one_hot(q, k, v, nq, length)
    assert sure.mean() > 0.8
    assert np.isfinite(got[sure]).all()
    assert (np.abs(got - want)[sure] <= 4 * EPS * np.abs(want[sure])).all()
    assert status(ctx) == 0


@pytest.mark.parametrize("nq,M", [(64, 3), (128, 9)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("exponent", [23, 25, 26, 27, 30])
def test_large_scores_that_rise_a_little(kind, exponent, nq, M):
    """The largest score of a chunk's later tiles lies a little above that of its first
    ones, both near 2^exponent, where fp32 scores are that far apart: finite, and
    between V's smallest and largest values.  (64 KV heads: four chunks of four tiles.)"""
    ctx = context(nq, 64)
    length = 2048
    kv, k, v, ids = cache(ctx, kind, length, 19)
    for rise in (7.0, 8.0, 9.0, 12.0, 15.0, 16.0, 17.0):
        rows = np.zeros((length, 64, 128), dtype=np.float32)
        rows[:, :, 0] = 48.0
        rows[np.arange(length) % 512 >= 256, :, 17] = 1.0  # another group of the 4-bit format
        if kind == "kv4":
            pg = u.to_pages(*u.quantise_rows(rows.reshape(length, 64 * 128), 64))
            kv.pool[torch.from_numpy(ids.astype(np.int64)).cuda(), 1, 0] = torch.from_numpy(pg).cuda()
            k = u.from_pages(pg)
            assert k[0, 0, 0] == 48 and k[300, 0, 17] > 0.9
        else:
            b = torch.from_numpy(rows).bfloat16().reshape(-1, 16, 64, 128)
            kv.pool[torch.from_numpy(ids.astype(np.int64)).cuda(), 1, 0] = b.permute(0, 2, 1, 3).cuda()
        unit = np.log2(np.e) / np.sqrt(128.0)              # base-2 score of a product
        q = np.zeros((M, nq, 128), dtype=np.float32)
        q[:, :, 0] = 2.0 ** exponent / unit / 48
        q[:, :, 17] = rise / unit
        sync()
        got = attend(ctx, kv, kind, q, 0, 0).reshape(M, 64, nq // 64, 128)
        top = np.abs(v[:length]).max(0)[None, :, None]
        assert np.isfinite(got).all(), rise
        # 512 products in up to three parts, 2 eps an addition
        assert (np.abs(got) <= top * (1 + 3 * 512 * 2 * EPS)).all()
    assert status(ctx) == 0


@pytest.mark.parametrize("nq,M", [(2, 3), (26, 3), (26, 16)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q_exp", [116, 120, 124])
def test_queries_of_any_size_that_fp32_holds(kind, q_exp, nq, M):
    check_one_hot(kind, 2.0 ** q_exp, 2.0 ** -10, nq, M)


@pytest.mark.parametrize("nq,M", [(2, 3), (26, 3), (26, 16)])
@pytest.mark.parametrize("kind", KINDS)
def test_queries_next_to_the_largest_fp32_number(kind, nq, M):
    """Elements that would round to infinity in bf16."""
    ctx = context(nq, 2)
    length = 700
    kv, k, v, _ = cache(ctx, kind, length, 17, spread=2.0 ** -12)
    rng = np.random.default_rng(3)
    q = (rng.standard_normal((M, nq, 128)) * 2.0 ** 120).astype(np.float32)
    q[:, :, ::16] = np.where(rng.random((M, nq, 8)) < 0.5, -1, 1) * np.finfo(np.float32).max
    got = attend(ctx, kv, kind, q, 0, 0).reshape(M, nq, 128)
    want, sure = one_hot(q, k, v, nq, length)
    assert sure.mean() > 0.8
    assert (np.abs(got - want)[sure] <= 4 * EPS * np.abs(want[sure])).all()
    assert status(ctx) == 0

# ---------------------------------------------------------------------------
# infinite values
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 20)])
@pytest.mark.parametrize("nq,M", [(2, 16), (4, 4), (26, 16), (26, 9)])
def test_infinite_v_elements_reach_the_rows_that_see_them_alike(nq, M, window, sinks):
    """An infinite V element makes that output element of every row that sees it
    infinite, of its sign, NaN where signs meet; the row's other elements keep their
    bits; and the rows have the same bits in a smaller block."""
    ctx = context(nq, 2)
    length = 700
    kv, _, _, ids = cache(ctx, "bf16", length, 81)
    q = np.random.default_rng(8).standard_normal((M, nq, 128)).astype(np.float32)
    clean = attend(ctx, kv, "bf16", q, window, sinks).reshape(M, nq, 128)
    see = u.visible(M, length, window, sinks)
    inf, nan = float("inf"), float("nan")
    low = length - M - window + 1 if window else 300                       # the first row's first key
    spots = [[(length - M - 3, 5, inf)],                                   # seen by every row
             [(length - M - 3, 5, -inf), (low + 40, 127, inf)],
             [(length - 2, 64, -inf)],                                     # by the last two
             [(low + 1, 0, inf), (3, 17, -inf)],                           # by the first two (of a window); a sink
             [(length - M - 3, 9, inf), (length - 5, 9, -inf)],            # signs that meet in some rows
             [(length - M - 9, 77, nan), (length - 1, 78, inf)]]
    for spot in spots:
        saved = kv.pool.clone()
        want = np.zeros((M, 128))
        for t, d, val in spot:
            kv.pool[int(ids[t // 16]), 1, 1, :, t % 16, d] = val
            with np.errstate(invalid="ignore"):
                want[:, d] += np.where(see[:, t], val, 0.0)
        got = attend(ctx, kv, "bf16", q, window, sinks).reshape(M, nq, 128)
        odd = np.broadcast_to((want != 0)[:, None], got.shape)             # NaN too
        assert same_bits(np.where(odd, np.float32(0), got), np.where(odd, np.float32(0), clean)), spot
        assert np.array_equal(got[odd], np.broadcast_to(want[:, None], got.shape)[odd], equal_nan=True), spot
        for i, m in ((M - 1, 1), (M // 2, 2)) if nq < 26 else ((M - 2, 2), (M - 8, 8)) if M <= 9 else ((6, 10),):
            kv.seq_len[0] = length - M + i + m
            part = attend(ctx, kv, "bf16", q[i:i + m], window, sinks).reshape(m, nq, 128)
            assert np.array_equal(part, got[i:i + m], equal_nan=True), (spot, i, m)
        kv.seq_len[0] = length
        kv.pool.copy_(saved)
    assert status(ctx) == 0


# ---------------------------------------------------------------------------
# the plan of the chunks
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", KINDS)
def test_a_window_without_an_end_is_planned_at_once(kind):
    """Windows and sinks of 2^31 - 1 (no limit): the result without a window, and no
    search of millions of steps on the host (73 ms a call with four chunks)."""
    ctx = context(64, 64)
    kv, _, _, _ = cache(ctx, kind, 600, 13)
    q = np.random.default_rng(5).standard_normal((2, 64, 128)).astype(np.float32)
    want = attend(ctx, kv, kind, q, 0, 0)
    most = 2 ** 31 - 1
    for window, sinks in ((most, 0), (most, most), (600, most)):
        assert same_bits(attend(ctx, kv, kind, q, window, sinks), want)
    qd, out, st = torch.from_numpy(q).cuda(), torch.empty(2, 64 * 128, device="cuda"), kv.struct()
    f = abi.spec_attention_kv4 if kind == "kv4" else abi.spec_attention_window
    sync()
    t0 = time.perf_counter()
    for _ in range(20):
        abi.check("attention", f(ctx.h, st, 1, qd.data_ptr(), 2, most, most, out.data_ptr()))
    assert time.perf_counter() - t0 < 0.2
    sync()
    assert status(ctx) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nq,M", [(64, 4), (128, 16)])
@pytest.mark.parametrize("window,sinks", [(600, 0), (600, 300), (1000, 128), (2000, 5), (700, 2000)])
def test_windows_that_limit_the_chunks(kind, nq, M, window, sinks):
    """Few chunks (64 KV heads: four), lengths around every step of the chunks' length
    and far behind the last: chunks of several tiles for sinks and window, chunks that
    hold both, blocks on both sides of a step."""
    ctx = context(nq, 64)
    longest = 3000
    kv, k, v, _ = cache(ctx, kind, longest, 43)
    q = np.random.default_rng(5).standard_normal((M, nq, 128)).astype(np.float32)
    for length in (512 + M // 2, 1024, 1024 + M // 2, 1536 + M, 2048 + M // 2, 2049, longest):
        kv.seq_len[0] = length
        whole = attend(ctx, kv, kind, q, window, sinks)
        want, bound = pu.attention64(q, k, v, nq, window, sinks, length, split=base.SPLIT[kind])
        assert (np.abs(whole - want) <= bound).all(), length
        assert pu.rel_l2(whole, want) < pu.ACCURACY, length
        for i, m in ((M - 1, 1), (M // 2, M - M // 2)) if nq < 128 else ((7, 9), (3, 11), (0, 10)):
            kv.seq_len[0] = length - M + i + m
            assert same_bits(attend(ctx, kv, kind, q[i:i + m], window, sinks), whole[i:i + m]), (length, i, m)
    assert status(ctx) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (6000, 300), (3000, 5000)])
def test_two_row_tiles_across_a_step(kind, window, sinks):
    """16 rows of 13 heads on each of two KV heads, 38 chunks: around the position where
    chunks become two tiles long."""
    nq, M = 26, 16
    ctx = context(nq, 2, max_ctx=40000)
    kv, k, v, _ = cache(ctx, kind, 9800, 47)
    q = np.random.default_rng(5).standard_normal((M, nq, 128)).astype(np.float32)
    for length in (38 * 128 + 9, 2 * 38 * 128 + 5, 9800):
        kv.seq_len[0] = length
        whole = attend(ctx, kv, kind, q, window, sinks)
        want, bound = pu.attention64(q, k, v, nq, window, sinks, length, split=base.SPLIT[kind])
        assert (np.abs(whole - want) <= bound).all(), length
        assert pu.rel_l2(whole, want) < pu.ACCURACY, length
        for i, m in ((6, 10), (1, 12), (4, 11)):
            kv.seq_len[0] = length - M + i + m
            assert same_bits(attend(ctx, kv, kind, q[i:i + m], window, sinks), whole[i:i + m]), (length, i, m)
    assert status(ctx) == 0


# ---------------------------------------------------------------------------
# precision
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nq,M", [(2, 1), (2, 16), (26, 1), (26, 4), (26, 9), (26, 16)])
@pytest.mark.parametrize("length", [300, 5000, 33000])
def test_accuracy(kind, nq, M, length):
    """Every kernel (few rows, one tile, two tiles) and every part of its operands: far
    below what a lost part would cost."""
    ctx = context(nq, 2, max_ctx=40000)
    kv, k, v, _ = cache(ctx, kind, length, 53)
    q = np.random.default_rng(11).standard_normal((M, nq, 128)).astype(np.float32)
    got = attend(ctx, kv, kind, q, 0, 0)
    want = pu.attention64(q, k, v, nq, 0, 0, length)[0]
    err = pu.rel_l2(got, want)
    print(f"{kind} {nq} heads, {M} rows, {length} keys: {err:.2e}")
    assert err < pu.ACCURACY
    assert status(ctx) == 0


# ---------------------------------------------------------------------------
# calls that follow each other
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("nq,M", [(2, 1), (2, 3), (26, 1), (26, 9), (26, 16)])
def test_4bit_calls_next_to_each_other(nq, M):
    """No other launch between the calls, so that each may start while the one before
    ends: append and attention over its rows, append and read, norm with rotation and
    attention with its q (one row: q is the row's first columns), attention with the
    output before as q.  The same bits as with a pause after every call."""
    ctx = context(nq, 2, max_ctx=1024, rope_theta=1e4)
    rounds, n, length = 24, 200, 700
    kv, _, _, _ = cache(ctx, "kv4", length, 5)
    start = kv.pool.clone()
    gen = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.randn(rounds, 2, n, 512, generator=gen, device="cuda")
    q = torch.randn(rounds, M, nq * 128, generator=gen, device="cuda")
    x = torch.randn(rounds, M, (nq + 2) * 128, generator=gen, device="cuda")
    pos = torch.arange(length - M, length, dtype=torch.int32, device="cuda")
    # two views of the cache: the pages in two orders
    tables = [kv.page_table.clone(), torch.cat((torch.flip(kv.page_table[:length // 16], (0,)), kv.page_table[length // 16:]))]
    views = [kv.struct() for _ in tables]
    for s, t in zip(views, tables):
        s.page_table = t.data_ptr()
    h, p = ctx.h, lambda t: t.data_ptr()

    def run(pause):
        kv.pool.copy_(start)
        held = torch.zeros(rounds, 2, n, 512, device="cuda")
        qk = torch.zeros_like(x)
        out = torch.zeros(rounds, 4, M, nq * 128, device="cuda")
        sync()

        def call(name, *args):
            abi.check(name, getattr(abi, name)(h, *args))
            if pause:
                sync()
        for i in range(rounds):
            st = views[i % 2]
            a, b, r, s = p(rows[i, 0]), p(rows[i, 1]), p(held[i, 0]), p(held[i, 1])
            call("spec_kv4_append", st, 1, a, a + 1024, 512, n)
            call("spec_attention_kv4", st, 1, p(q[i]), M, 300, 7, p(out[i, 0]))
            call("spec_attention_kv4", st, 1, p(out[i, 0]), M, 0, 0, p(out[i, 1]))
            call("spec_kv4_read", st, 1, length - n, n, r, r + 1024, 512)
            call("spec_kv4_append", st, 1, b, b + 1024, 512, n)
            call("spec_kv4_read", st, 1, length - n, n, s, s + 1024, 512)
            call("spec_qk_norm_rope", p(x[i]), x.shape[2], M, p(pos), None, None, p(qk[i]), x.shape[2])
            # (for more rows than one, M rows of nq heads are what lies there)
            call("spec_attention_kv4", st, 1, p(qk[i]), M, 64, 0, p(out[i, 2]))
            call("spec_attention_kv4", views[1 - i % 2], 1, p(out[i, 2]), M, 300, 7, p(out[i, 3]))
        sync()
        return held, qk, out
    want = run(True)
    assert all(torch.isfinite(t).all() and t.abs().max() > 0 for t in want)
    for _ in range(3):
        got = run(False)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert status(ctx) == 0


@pytest.mark.parametrize("nq,M", [(2, 1), (2, 3), (26, 1), (26, 9), (26, 16)])
def test_bf16_calls_next_to_each_other(nq, M):
    """Attention whose q is the output of the call before, over two orders of the pages,
    and after norm with rotation."""
    ctx = context(nq, 2, max_ctx=1024, rope_theta=1e4)
    rounds, length = 30, 700
    kv, _, _, _ = cache(ctx, "bf16", length, 5)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rounds, M, (nq + 2) * 128, generator=gen, device="cuda")
    pos = torch.arange(length - M, length, dtype=torch.int32, device="cuda")
    tables = [kv.page_table.clone(), torch.cat((torch.flip(kv.page_table[:length // 16], (0,)), kv.page_table[length // 16:]))]
    views = [kv.struct() for _ in tables]
    for s, t in zip(views, tables):
        s.page_table = t.data_ptr()
    h, p = ctx.h, lambda t: t.data_ptr()

    def run(pause):
        qk = torch.zeros_like(x)
        out = torch.zeros(rounds, 4, M, nq * 128, device="cuda")
        sync()

        def call(name, *args):
            abi.check(name, getattr(abi, name)(h, *args))
            if pause:
                sync()
        for i in range(rounds):
            call("spec_qk_norm_rope", p(x[i]), x.shape[2], M, p(pos), None, None, p(qk[i]), x.shape[2])
            src = qk[i]
            for j, (window, sinks) in enumerate(((0, 0), (300, 7), (64, 0), (0, 0))):
                call("spec_attention_window", views[(i + j) % 2], 1, p(src), M, window, sinks, p(out[i, j]))
                src = out[i, j]
        sync()
        return qk, out
    want = run(True)
    assert all(torch.isfinite(t).all() and t.abs().max() > 0 for t in want)
    for _ in range(3):
        got = run(False)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert status(ctx) == 0


# ---------------------------------------------------------------------------
# queries that are not finite, and a captured layer
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nq,M", [(2, 4), (2, 16), (26, 9), (26, 16)])
def test_a_query_that_is_not_finite_spoils_its_own_row(kind, nq, M):
    ctx = context(nq, 2)
    kv, _, _, _ = cache(ctx, kind, 900, 61)
    q = np.random.default_rng(5).standard_normal((M, nq, 128)).astype(np.float32)
    clean = attend(ctx, kv, kind, q, 0, 0).reshape(M, nq, 128)
    for val in (np.nan, np.inf, -np.inf):
        bad = q.copy()
        bad[1, 0, 77] = bad[M - 1, nq - 1, 0] = val
        bad[2] = 0                                          # a row of zeros: the mean of V
        got = attend(ctx, kv, kind, bad, 0, 0).reshape(M, nq, 128)
        spoilt = np.zeros((M, nq), dtype=bool)
        spoilt[1, 0] = spoilt[M - 1, nq - 1] = True
        assert not np.isfinite(got[spoilt]).any()
        keep = ~spoilt
        keep[2] = False
        assert same_bits(got[keep], clean[keep])
        assert np.isfinite(got[2][~spoilt[2]]).all()
    assert status(ctx) == 0


@pytest.mark.parametrize("nq,M", [(2, 1), (26, 5)])
def test_a_captured_layer_replayed(nq, M):
    """Norm with rotation, extend, append, attention and read, captured on a stream of
    their own and replayed with new inputs: the bits of eager calls."""
    nkv, length, steps = 2, 400, 4
    cfg = base.config(nq, nkv, rope_theta=1e4)
    width = (nq + 2 * nkv) * 128
    gen = torch.Generator(device="cuda").manual_seed(2)
    xs = torch.randn(steps, M, width, generator=gen, device="cuda")
    qs = torch.randn(steps, M, nq * 128, generator=gen, device="cuda")
    prompt = torch.randn(length, 2 * nkv * 128, generator=gen, device="cuda")
    sync()

    def run(captured):
        stream = torch.cuda.Stream()
        results = []
        with torch.cuda.stream(stream):
            ctx = runtime.Context(cfg, max_ctx=1024, stream=stream)
            kv = runtime.DeviceKV4(cfg, 64, 64)
            kv.reset(ctx)
            kv.extend(ctx, length)
            kv.append(ctx, 1, prompt[:, :nkv * 128], prompt[:, nkv * 128:])
            x, q = torch.zeros(M, width, device="cuda"), torch.zeros(M, nq * 128, device="cuda")
            pos = torch.zeros(M, dtype=torch.int32, device="cuda")
            out, back = torch.zeros(M, nq * 128, device="cuda"), torch.zeros(2, length, nkv * 128, device="cuda")
            st, h, p = kv.struct(), ctx.h, lambda t: t.data_ptr()
            k, v = p(x) + 4 * nq * 128, p(x) + 4 * (nq + nkv) * 128

            def layer():
                abi.check("qk", abi.spec_qk_norm_rope(h, p(x), width, M, p(pos), None, None, p(x), width))
                abi.check("extend", abi.spec_kv_extend(h, st, M))
                abi.check("append", abi.spec_kv4_append(h, st, 1, k, v, width, M))
                abi.check("attention", abi.spec_attention_kv4(h, st, 1, p(q), M, 300, 5, p(out)))
                abi.check("read", abi.spec_kv4_read(h, st, 1, 20, length, p(back[0]), p(back[1]), nkv * 128))
            graph = None
            for i in range(steps):
                x.copy_(xs[i])
                q.copy_(qs[i])
                pos.copy_(torch.arange(length + i * M, length + (i + 1) * M, dtype=torch.int32))
                if not captured:
                    layer()
                else:
                    if graph is None:
                        stream.synchronize()
                        graph = torch.cuda.CUDAGraph()
                        with torch.cuda.graph(graph, stream=stream):
                            layer()
                    graph.replay()
                stream.synchronize()
                results.append((x.clone(), out.clone(), back.clone(), int(kv.seq_len[0])))
            stream.synchronize()
            assert status(ctx) == 0
            ctx.close()
        return results
    for a, b in zip(run(False), run(True)):
        assert a[3] == b[3] and all(torch.equal(s, t) for s, t in zip(a[:3], b[:3]))
        assert all(torch.isfinite(t).all() and t.abs().max() > 0 for t in a[:3])
