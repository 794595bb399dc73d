"""The 4-bit KV cache, attention with a window and sinks over both paged caches,
and QK-norm with RoPE as building blocks, against 64-bit numpy (kv4_util).

Tolerances: what the 4-bit cache holds is compared bit for bit; attention
elementwise against the bound that kv4_util.attention_bound derives from the
operand split and the number of additions; QK-norm + RoPE against the count of
its fp32 roundings.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from speculative_decoding_exact_gb300 import abi, runtime, synth  # noqa: E402
from tests import kv4_util as u  # noqa: E402

EPS = 2.0 ** -24


def config(nq, nkv, layers=2, **kw):
    return runtime.ModelConfig(hidden=512, n_layers=layers, n_q_heads=nq, n_kv_heads=nkv, head_dim=128, ffn=512,
                               vocab=512, **kw)


_CTX = {}


def context(nq, nkv, max_ctx=4096, layers=2, **kw):
    """One context per geometry for the whole module."""
    key = (nq, nkv, max_ctx, layers, tuple(sorted(kw.items())))
    if key not in _CTX:
        _CTX[key] = runtime.Context(config(nq, nkv, layers, **kw), max_ctx=max_ctx)
    return _CTX[key]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    for c in _CTX.values():
        c.close()
    _CTX.clear()


def sync():
    torch.cuda.synchronize()


def status(ctx):
    return abi.spec_last_status(ctx.h)


def shuffled(kv, ctx, length, seed):
    """Map `length` positions, then give the sequence scattered physical pages."""
    kv.reset(ctx)
    kv.extend(ctx, length)
    sync()
    n = -(-length // 16)
    ids = np.random.default_rng(seed).permutation(kv.num_pages)[:n].astype(np.int32)
    kv.page_table[:n] = torch.from_numpy(ids).cuda()
    return ids


def cache(ctx, kind, length, seed, spread=1.0, extra=3):
    """A filled cache and its float64 K, V [16*pages][nkv][128] (tail rows included)."""
    cfg = ctx.cfg
    pages = max(1, -(-length // 16))
    kv = (runtime.DeviceKV4 if kind == "kv4" else runtime.DeviceKV)(cfg, pages + extra, pages + 1)
    ids = shuffled(kv, ctx, length, seed)
    rng = np.random.default_rng(seed + 1)
    out = []
    for which in range(2):
        x = (rng.standard_normal((pages * 16, cfg.n_kv_heads * 128)) * (spread if which == 0 else 1)).astype(np.float32)
        if kind == "kv4":
            code, byte = u.quantise_rows(x, cfg.n_kv_heads)
            pg = u.to_pages(code, byte)
            kv.pool[torch.from_numpy(ids[:pages].astype(np.int64)).cuda(), 1, which] = \
                torch.from_numpy(pg[:len(ids)]).cuda()
            out.append(u.from_pages(pg))
        else:
            b = torch.from_numpy(x).bfloat16().reshape(pages, 16, cfg.n_kv_heads, 128)
            kv.pool[torch.from_numpy(ids[:pages].astype(np.int64)).cuda(), 1, which] = \
                b.permute(0, 2, 1, 3)[:len(ids)].cuda()
            out.append(b.double().numpy().reshape(-1, cfg.n_kv_heads, 128))
    sync()
    return kv, out[0], out[1], ids


def attend(ctx, kv, kind, q, window, sinks, layer=1):
    M = q.shape[0]
    qd = torch.from_numpy(np.ascontiguousarray(q, dtype=np.float32)).cuda()
    out = torch.full((M, ctx.cfg.n_q_heads * 128), float("nan"), device="cuda")
    f = abi.spec_attention_kv4 if kind == "kv4" else abi.spec_attention_window
    abi.check("attention", f(ctx.h, kv.struct(), layer, qd.data_ptr(), M, window, sinks, out.data_ptr()))
    sync()
    return out.cpu().numpy()


# what q and p lose as MMA operands (kv4_util): two binary16 parts against 4-bit
# values, three bf16 parts, 24 bits, against bf16 ones
SPLIT = {"kv4": 2.0 ** -22, "bf16": 2.0 ** -24}


def check_attention(ctx, kind, M, length, window, sinks, seed=0, spread=1.0, q_scale=1.0):
    kv, k, v, _ = cache(ctx, kind, length, seed, spread)
    q = (np.random.default_rng(seed + 7).standard_normal((M, ctx.cfg.n_q_heads, 128)) * q_scale).astype(np.float32)
    got = attend(ctx, kv, kind, q, window, sinks)
    want, bound = u.attention(q, k, v, ctx.cfg.n_q_heads, window, sinks, length, split=SPLIT[kind])
    err = np.abs(got - want)
    assert np.isfinite(got).all()
    worst = float((err / np.maximum(bound, 1e-30)).max())
    assert (err <= bound).all(), f"error {err.max():.3e}, {worst:.2f} of the bound"
    assert status(ctx) == 0
    return got


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------
def rows_of(kind, n, w, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, w)).astype(np.float32)
    if kind == "wide":
        x *= (10.0 ** rng.integers(-7, 7, (n, w // 16)).repeat(16, 1)).astype(np.float32)
    elif kind == "ties":
        # midpoints of neighbouring codes under scales with all 8 fractions, and
        # their neighbours in fp32
        s = ((8 + rng.integers(0, 8, (n, w // 16))) * 2.0 ** rng.integers(-6, 6, (n, w // 16))).repeat(16, 1)
        x = (rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], (n, w)) * s).astype(np.float32)
        x[:, ::16] = (6 * s[:, ::16]).astype(np.float32)
        step = rng.integers(-1, 2, (n, w))
        x = np.where(step > 0, np.nextafter(x, np.float32(np.inf)), np.where(step < 0, np.nextafter(x, np.float32(0)), x))
        x = (x * rng.choice([-1, 1], (n, w))).astype(np.float32)
    elif kind == "scales":
        # largest magnitudes on, just below and just above 6 times every scale
        top = 6 * u.scale_values()[rng.integers(1, 0xE3, (n, w // 16))].astype(np.float32)
        top = np.where(rng.random(top.shape) < 0.3, np.nextafter(top, np.float32(np.inf)), top)
        top = np.where(rng.random(top.shape) < 0.3, np.nextafter(top, np.float32(0)), top)
        x = (x.reshape(n, -1, 16) / 8 * top[..., None]).astype(np.float32)
        x[..., 3] = -top
        x = x.reshape(n, w)
    elif kind == "zeros":
        x[:, :32] = 0
        x[::2] = 0
        x[1, 5] = -0.0
        x[:, 40:56] *= np.float32(1e-44)
    return x


@pytest.mark.parametrize("kind", ["normal", "wide", "ties", "scales", "zeros"])
@pytest.mark.parametrize("n,start,nkv", [(1, 0, 1), (16, 5, 4), (37, 16, 2)])
def test_append_and_read_are_exact(kind, n, start, nkv):
    ctx = context(4 * nkv if nkv > 1 else 4, nkv)
    cfg, w = ctx.cfg, nkv * 128
    kv = runtime.DeviceKV4(cfg, 12, 8)
    ids = shuffled(kv, ctx, start + n, seed=n)
    kv.pool.random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(5))
    before = kv.pool.cpu().numpy()
    # k and v as columns of a wider matrix
    ld = 3 * w + 8
    x = np.stack([rows_of(kind, max(n, 2), w, 10 + i)[:n] for i in range(2)])
    mat = torch.full((n, ld), 7.0)
    mat[:, 4:4 + w] = torch.from_numpy(x[0])
    mat[:, 4 + 2 * w:4 + 3 * w] = torch.from_numpy(x[1])
    mat = mat.cuda()
    kv.append(ctx, 1, mat[:, 4:4 + w], mat[:, 4 + 2 * w:4 + 3 * w])
    sync()
    after = kv.pool.cpu().numpy()
    # every byte that belongs to the rows, and no other
    want = before.copy()
    for which in range(2):
        code, byte = u.quantise_rows(x[which], nkv)
        packed = (code[..., 0::2] | (code[..., 1::2] << 4)).reshape(n, nkv, 4, 16)
        for i in range(n):
            pg, t = ids[(start + i) // 16], (start + i) % 16
            for c in range(4):
                want[pg, 1, which, :, 256 * c + 16 * t:256 * c + 16 * t + 16] = packed[i, :, c]
            want[pg, 1, which, :, 1024 + 8 * t:1032 + 8 * t] = byte[i]
    assert np.array_equal(after, want)
    k, v = kv.read(ctx, 1, start, n)
    sync()
    for which, got in enumerate((k, v)):
        code, byte = u.quantise_rows(x[which], nkv)
        val = u.code_values()[code] * u.scale_values()[byte].repeat(16, -1)
        assert np.array_equal(got.cpu().numpy(), val.reshape(n, w).astype(np.float32))
    assert status(ctx) == 0


def test_append_of_nonfinite_and_saturating_values():
    ctx = context(4, 1)
    kv = runtime.DeviceKV4(ctx.cfg, 2, 2)
    kv.reset(ctx)
    kv.extend(ctx, 3)
    x = np.ones((3, 128), dtype=np.float32)
    x[0, 0], x[0, 17], x[1, 33], x[2, 50] = np.nan, np.inf, -np.inf, 1e30
    t = torch.from_numpy(x).cuda()
    kv.append(ctx, 0, t, t)
    k, _ = kv.read(ctx, 0, 0, 3)
    sync()
    assert status(ctx) == abi.ST_NONFINITE
    k = k.cpu().numpy()
    code, byte = u.quantise_rows(x, 1)
    assert np.array_equal(k, (u.code_values()[code] * u.scale_values()[byte].repeat(16, -1)).reshape(3, 128))
    assert k[0, 0] == 0 and k[0, 17] == 61440 and k[1, 33] == -61440 and k[2, 50] == 61440
    # a group of ones: 1/6 lies between the scales 10/64 and 11/64, so 6 * 11/64
    assert k[0, 1] == 6 * 11 / 64


def test_append_leaves_out_rows_without_a_place():
    ctx = context(4, 1)
    kv = runtime.DeviceKV4(ctx.cfg, 4, 4)
    kv.reset(ctx)
    kv.extend(ctx, 20)
    x = torch.randn(24, 128, device="cuda")
    kv.append(ctx, 1, x, x)                                   # positions -4 .. 19
    sync()
    assert status(ctx) == abi.ST_CTX_FULL
    k, _ = kv.read(ctx, 1, 0, 24)
    code, byte = u.quantise_rows(x.cpu().numpy()[4:], 1)
    want = (u.code_values()[code] * u.scale_values()[byte].repeat(16, -1)).reshape(20, 128)
    k = k.cpu().numpy()
    assert np.array_equal(k[:20], want.astype(np.float32)) and not k[20:].any()   # past seq_len: zeros
    # a bad page id: the row is left out, the pool is untouched, reads are zeros
    kv.page_table[1] = 4
    before = kv.pool.clone()
    kv.append(ctx, 1, x[:2], x[:2])
    k, _ = kv.read(ctx, 1, 15, 3)
    sync()
    assert status(ctx) == abi.ST_CTX_FULL and torch.equal(before, kv.pool)
    assert np.array_equal(k.cpu().numpy()[0], want[15]) and not k[1:].any()


def test_read_of_every_byte_value():
    ctx = context(4, 1)
    kv = runtime.DeviceKV4(ctx.cfg, 3, 3)
    kv.reset(ctx)
    kv.extend(ctx, 48)
    pool = np.arange(3 * 2 * 2 * 1152, dtype=np.int64).reshape(3, 2, 2, 1, 1152) * 7 % 256
    kv.pool.copy_(torch.from_numpy(pool.astype(np.uint8)))
    k, v = kv.read(ctx, 1, 0, 48)
    sync()
    for which, got in enumerate((k, v)):
        want = u.from_pages(pool[:, 1, which].astype(np.uint8))
        assert np.array_equal(got.cpu().numpy().reshape(48, 1, 128), want.astype(np.float32))


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
KINDS = ["kv4", "bf16"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,length", [(1, 1), (1, 2), (16, 16), (1, 16), (3, 17), (1, 127), (16, 128), (5, 129),
                                      (16, 143), (8, 255), (2, 257), (13, 1000), (16, 2071)])
def test_attention_causal(kind, M, length):
    check_attention(context(26, 2), kind, M, length, 0, 0, seed=M + length)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nq,nkv", [(52, 4), (48, 4), (8, 1), (16, 16), (32, 8), (2, 1), (2, 2), (64, 64)])
def test_attention_head_layouts(kind, nq, nkv):
    ctx = context(nq, nkv)
    check_attention(ctx, kind, 16, 300, 0, 0, seed=1)
    check_attention(ctx, kind, 1, 130, 100, 4, seed=2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,length,window,sinks", [
    (1, 500, 1, 0), (16, 500, 1, 0), (16, 500, 1, 1), (1, 500, 1, 4), (4, 500, 16, 0), (16, 500, 17, 3),
    (16, 1000, 128, 16), (16, 1000, 127, 33), (7, 1000, 300, 128), (16, 1000, 64, 200), (16, 1000, 500, 600),
    (16, 1000, 984, 0), (16, 1000, 985, 1), (16, 1000, 1000, 0), (16, 1000, 100000, 7), (3, 10, 4, 100),
    (16, 16, 4, 2), (1, 1, 1, 1), (5, 2500, 2 ** 31 - 1, 2 ** 31 - 1), (5, 2500, 40, 2 ** 31 - 1),
    (16, 2500, 1024, 4)])
def test_attention_window_and_sinks(kind, M, length, window, sinks):
    check_attention(context(26, 2), kind, M, length, window, sinks, seed=length + window % 97)


@pytest.mark.parametrize("nq,M", [(4, 2), (26, 9)])
@pytest.mark.parametrize("kind", KINDS)
def test_attention_long_and_peaked(kind, nq, M):
    """Many tiles in one chunk, scores far apart (the running maximum moves) and
    keys sorted so that it moves often; large and small queries."""
    ctx = context(nq, 2, max_ctx=40000)
    for q_scale, spread in ((1.0, 1.0), (8.0, 4.0), (1e-3, 1.0)):
        check_attention(ctx, kind, M, 33000, 0, 0, seed=5, spread=spread, q_scale=q_scale)
    cfg = ctx.cfg
    kv, k, v, ids = cache(ctx, kind, 20000, 9)
    # one direction grows along the sequence
    q = np.zeros((M - 1, cfg.n_q_heads, 128), dtype=np.float32)
    q[:, :, 3] = 60.0
    ramp = (np.arange(k.shape[0]) // 16 * 0.05).astype(np.float32)
    if kind == "kv4":
        code, byte = u.quantise_rows(np.repeat(ramp[:, None], 256, 1), 2)
        pg = u.to_pages(code, byte)
        kv.pool[torch.from_numpy(ids.astype(np.int64)).cuda(), 1, 0] = torch.from_numpy(pg).cuda()
        k = u.from_pages(pg)
    else:
        b = torch.from_numpy(np.repeat(ramp[:, None], 256, 1)).bfloat16().reshape(-1, 16, 2, 128)
        kv.pool[torch.from_numpy(ids.astype(np.int64)).cuda(), 1, 0] = b.permute(0, 2, 1, 3).cuda()
        k = b.double().numpy().reshape(-1, 2, 128)
    sync()
    got = attend(ctx, kv, kind, q, 0, 0)
    want, bound = u.attention(q, k, v, cfg.n_q_heads, 0, 0, 20000, split=SPLIT[kind])
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("nq", [26, 2])
@pytest.mark.parametrize("kind", KINDS)
def test_attention_rows_without_keys(kind, nq):
    """seq_len below M: the rows before position 0 see nothing and are zero."""
    ctx = context(nq, 2)
    for M, length in ((16, 5), (4, 0), (16, 1)):
        kv, k, v, _ = cache(ctx, kind, length, 3)
        q = np.random.default_rng(4).standard_normal((M, nq, 128)).astype(np.float32)
        got = attend(ctx, kv, kind, q, 0, 0)
        want, bound = u.attention(q, k, v, nq, 0, 0, length, split=SPLIT[kind])
        assert not got[:M - length].any()
        assert (np.abs(got - want) <= bound).all()
    assert status(ctx) == 0


@pytest.mark.parametrize("nq", [26, 2])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 20)])
def test_attention_unmapped_pages_are_not_seen(kind, window, sinks, nq):
    ctx = context(nq, 2)
    kv, k, v, ids = cache(ctx, kind, 700, 11)
    bad = {1: -1, 8: -1, 15: kv.num_pages, 16: 2 ** 30, 39: -5, 43: -1}
    mapped = np.ones(700, dtype=bool)
    for lp, val in bad.items():
        kv.page_table[lp] = val
        mapped[16 * lp:16 * lp + 16] = False
    q = np.random.default_rng(4).standard_normal((16, nq, 128)).astype(np.float32)
    got = attend(ctx, kv, kind, q, window, sinks)
    want, bound = u.attention(q, k, v, nq, window, sinks, 700, mapped=mapped, split=SPLIT[kind])
    assert (np.abs(got - want) <= bound).all()
    # no page at all: every row is empty
    kv.page_table.fill_(-1)
    assert not attend(ctx, kv, kind, q, window, sinks).any()


@pytest.mark.parametrize("nq", [26, 2])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5)])
def test_attention_is_untouched_by_what_rows_do_not_see(kind, window, sinks, nq):
    """NaN, infinities and the largest numbers behind the sequence, in other
    pages, outside the window, and in block rows that an earlier row does not
    see: every row equals the clean run bit for bit where it does not see them."""
    ctx = context(nq, 2)
    M, length = 16, 439
    kv, _, _, ids = cache(ctx, kind, length, 21)
    q = np.random.default_rng(8).standard_normal((M, nq, 128)).astype(np.float32)
    clean = attend(ctx, kv, kind, q, window, sinks)
    hidden = np.zeros((kv.num_pages, 16), dtype=bool)
    hidden[:] = True
    see = u.visible(M, length, window, sinks)
    for t in np.nonzero(see.any(0))[0]:
        hidden[ids[t // 16], t % 16] = False
    mask = torch.from_numpy(hidden).cuda()
    fills = [0xFF, 0x7F, 0x80] if kind == "kv4" else [float("nan"), float("inf"), -float("inf"), 3e38]
    for fill in fills:
        saved = kv.pool.clone()
        if kind == "kv4":
            codes = kv.pool[:, 1, :, :, :1024].view(kv.num_pages, 2, 2, 4, 16, 16)
            codes[mask[:, None, None, None, :].expand(-1, 2, 2, 4, -1)] = fill
            scales = kv.pool[:, 1, :, :, 1024:].view(kv.num_pages, 2, 2, 16, 8)
            scales[mask[:, None, None, :].expand(-1, 2, 2, -1)] = fill
        else:
            kv.pool[:, 1][mask[:, None, None, :].expand(-1, 2, 2, -1)] = fill
        got = attend(ctx, kv, kind, q, window, sinks)
        assert np.array_equal(got.view(np.uint32), clean.view(np.uint32)), fill
        kv.pool.copy_(saved)
    if kind == "kv4":
        return                                      # a 4-bit value is always finite
    # a non-finite V element and a non-finite K row at positions that only some
    # rows see: those rows turn non-finite there, the others stay as they were
    spots = [length - 6] + ([length - M - window + 4] if window else [])
    for t in spots:
        for which in (0, 1):
            for val in (float("nan"), float("inf")):
                saved = kv.pool.clone()
                kv.pool[int(ids[t // 16]), 1, which, :, t % 16, 77] = val
                got = attend(ctx, kv, kind, q, window, sinks)
                sees = see[:, t]
                same = (got.view(np.uint32) == clean.view(np.uint32)).all(-1)
                assert same[~sees].all()
                g = got.reshape(M, nq, 128)[sees]
                if which == 1:
                    assert not np.isfinite(g[:, :, 77]).any()
                    rest = np.delete(g, 77, -1)
                    assert np.array_equal(rest, np.delete(clean.reshape(M, nq, 128)[sees], 77, -1))
                elif math.isnan(val):
                    assert not np.isfinite(g).any()
                kv.pool.copy_(saved)


@pytest.mark.parametrize("nq", [26, 2])
@pytest.mark.parametrize("M,window,sinks", [(1, 0, 0), (16, 0, 0), (16, 100, 5), (5, 40, 200)])
def test_attention_bf16_values_past_binary16(M, window, sinks, nq):
    """bf16 elements from 2^15 up to the type's largest, and whole tiny rows, which
    binary16 operands could not hold."""
    ctx = context(nq, 2)
    length = 400
    kv, k, v, ids = cache(ctx, "bf16", length, 71)
    rng = np.random.default_rng(9)
    q = rng.standard_normal((M, nq, 128)).astype(np.float32)
    for n, (t, which, d, val) in enumerate([(3, 1, 5, 40000.0), (3, 1, 6, -1e9), (200, 1, 0, 32768.0), (390, 1, 127, 7e4),
                                            (length - 1, 1, 64, 1e30), (130, 0, 9, 70000.0), (length - 2, 0, 8, -1e5),
                                            (131, 0, slice(None), 1e-7), (132, 1, slice(None), 1e-7),
                                            (300, 1, slice(None), -65536.0)]):
        x = torch.full((2, 128), val).bfloat16() if isinstance(d, slice) else torch.tensor(val).bfloat16()
        kv.pool[int(ids[t // 16]), 1, which, :, t % 16, d] = x.cuda()
        (k, v)[which][t, :, d] = x.double().numpy()
    q[:, :, 8:10] *= 1e-4          # so that the large K elements do not decide every row
    sync()
    got = attend(ctx, kv, "bf16", q, window, sinks)
    want, bound = u.attention(q, k, v, nq, window, sinks, length, split=SPLIT["bf16"])
    assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())
    assert status(ctx) == 0


# the kinds of calls within which a row has the same bits: at most 16 query rows
# per KV head, one tile of 128 of them, two; each with blocks (first row, rows)
BLOCKS = {"few": (16, 16, 16, ((0, 1), (0, 4), (7, 1), (15, 1), (8, 8), (5, 7))),
          "few_grouped": (4, 8, 2, ((0, 1), (3, 1), (1, 2), (1, 3))),
          "tile": (9, 26, 2, ((0, 2), (0, 4), (7, 2), (1, 8), (5, 3))),
          "two_tiles": (16, 26, 2, ((0, 10), (0, 13), (6, 10), (1, 15), (2, 12)))}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("blocks", sorted(BLOCKS))
@pytest.mark.parametrize("n_past,window,sinks", [(45, 0, 0), (1000, 0, 0), (1000, 200, 9), (120, 121, 2)])
def test_attention_batch_height_invariance(kind, n_past, window, sinks, blocks):
    """A row has the same bits in every block of a kind that places it there."""
    M, nq, nkv, parts = BLOCKS[blocks]
    ctx = context(nq, nkv)
    kv, _, _, _ = cache(ctx, kind, n_past + M, 31)
    q = np.random.default_rng(5).standard_normal((M, nq, 128)).astype(np.float32) * 3
    whole = attend(ctx, kv, kind, q, window, sinks)
    for i, m in parts:
        kv.seq_len[0] = n_past + i + m
        part = attend(ctx, kv, kind, q[i:i + m], window, sinks)
        assert np.array_equal(part.view(np.uint32), whole[i:i + m].view(np.uint32)), (i, m)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nq,m", [(64, 1), (128, 9)])
def test_attention_across_a_chunk_size_step(kind, nq, m):
    """Blocks around every length at which the kernels change their split of the
    keys: right, and the same bits in a smaller block."""
    ctx = context(nq, 64, max_ctx=4096)
    kv, k, v, _ = cache(ctx, kind, 1100, 41)
    q = np.random.default_rng(5).standard_normal((16, nq, 128)).astype(np.float32)
    for boundary in (256, 512, 768, 1024):
        for length in (boundary + 5, boundary + 16, boundary):
            kv.seq_len[0] = length
            whole = attend(ctx, kv, kind, q, 0, 0)
            want, bound = u.attention(q, k, v, nq, 0, 0, length, split=SPLIT[kind])
            assert (np.abs(whole - want) <= bound).all()
            for i in (0, 1, 4, 6, 7, 9, 10, 11, 15):
                if i + m > 16:
                    continue
                kv.seq_len[0] = length - 16 + i + m
                part = attend(ctx, kv, kind, q[i:i + m], 0, 0)
                assert np.array_equal(part.view(np.uint32), whole[i:i + m].view(np.uint32)), (length, i)


@pytest.mark.parametrize("kind", KINDS)
def test_attention_offsets_past_32_bits(kind):
    """Pages whose byte offset in the pool passes 2^32 (and whose element offset
    passes 2^31)."""
    ctx = context(8, 4, layers=52, max_ctx=512)
    cfg = ctx.cfg
    length, per = 150, 52 * 2 * 4 * (1152 if kind == "kv4" else 4096)
    num = (1 << 32) // per + 40
    small, k, v, ids = cache(ctx, kind, length, 51)
    rows = [small.pool[int(i), 1].clone() for i in ids]
    cls = runtime.DeviceKV4 if kind == "kv4" else runtime.DeviceKV
    kv = cls.__new__(cls)
    kv.cfg = cfg
    kv.pool = torch.empty((num,) + tuple(small.pool.shape[1:]), dtype=small.pool.dtype, device="cuda")
    kv._init_metadata(num, 16)
    kv.reset(ctx)
    kv.extend(ctx, length)
    sync()
    high = [num - 1 - 3 * j for j in range(len(ids))]
    kv.page_table[:len(ids)] = torch.tensor(high, dtype=torch.int32)
    for lp, pg in enumerate(high):
        kv.pool[pg, 1] = rows[lp]
    q = np.random.default_rng(6).standard_normal((5, 8, 128)).astype(np.float32)
    got = attend(ctx, kv, kind, q, 0, 0)
    want, bound = u.attention(q, k, v, 8, 0, 0, length, split=SPLIT[kind])
    assert (np.abs(got - want) <= bound).all()
    if kind == "kv4":
        x = torch.randn(20, 512, device="cuda")
        kv.append(ctx, 51, x, x)
        r, _ = kv.read(ctx, 51, length - 20, 20)
        sync()
        code, byte = u.quantise_rows(x.cpu().numpy(), 4)
        want = (u.code_values()[code] * u.scale_values()[byte].repeat(16, -1)).reshape(20, 512)
        assert np.array_equal(r.cpu().numpy(), want.astype(np.float32))


# ---------------------------------------------------------------------------
# QK-norm + RoPE
# ---------------------------------------------------------------------------
def qk_reference(x, nq, nkv, pos, gq, gk, eps, theta):
    n = x.shape[0]
    y = x[:, :(nq + nkv) * 128].astype(np.float64).reshape(n, nq + nkv, 128)
    for sl, g in ((slice(0, nq), gq), (slice(nq, nq + nkv), gk)):
        if g is not None:
            z = y[:, sl]
            y[:, sl] = z / np.sqrt((z * z).mean(-1, keepdims=True) + eps) * g.astype(np.float64)
    if theta:
        ang = pos[:, None].astype(np.float64) * theta ** (-np.arange(64) / 64)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        a, b = y[..., :64].copy(), y[..., 64:].copy()
        y = np.concatenate([a * c - b * s, b * c + a * s], -1)
        mag = np.concatenate([np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)], -1)
    else:
        mag = np.abs(y)
    return y.reshape(n, -1), mag.reshape(n, -1)


@pytest.mark.parametrize("nq,nkv", [(52, 4), (2, 1), (2, 2)])
@pytest.mark.parametrize("n", [1, 2, 16, 129])
@pytest.mark.parametrize("norm,theta", [("qk", 5e5), ("q", 1e4), ("k", 0.0), ("", 1e4), ("", 0.0)])
def test_qk_norm_rope(nq, nkv, n, norm, theta):
    ctx = context(nq, nkv, max_ctx=4096, rope_theta=theta)
    w = (nq + nkv) * 128
    rng = np.random.default_rng(n)
    ldx, ldo = (nq + 2 * nkv) * 128 + 4, w + 8
    x = (rng.standard_normal((n, ldx)) * 3).astype(np.float32)
    pos = rng.integers(0, 4096, n).astype(np.int32)
    pos[0] = 4095
    g = [(1 + 0.2 * rng.standard_normal(128)).astype(np.float32) if c in norm else None for c in "qk"]
    xd, pd = torch.from_numpy(x).cuda(), torch.from_numpy(pos).cuda()
    gd = [None if t is None else torch.from_numpy(t).cuda() for t in g]
    out = torch.full((n, ldo), 5.0, device="cuda")
    abi.check("spec_qk_norm_rope", abi.spec_qk_norm_rope(
        ctx.h, xd.data_ptr(), ldx, n, pd.data_ptr() if theta else None, runtime.ptr(gd[0]), runtime.ptr(gd[1]),
        out.data_ptr(), ldo))
    sync()
    want, mag = qk_reference(x, nq, nkv, pos, g[0], g[1], 1e-6, theta)
    got = out.cpu().numpy()
    assert (got[:, w:] == 5.0).all()
    # sum of 128 squares (8 rounded adds and products deep), mean, eps, root,
    # reciprocal, two products; table, product and sum of the rotation
    assert (np.abs(got[:, :w] - want) <= 24 * EPS * mag + 1e-38).all()
    assert status(ctx) == 0
    # in place: the same bits, V columns untouched
    abi.check("spec_qk_norm_rope", abi.spec_qk_norm_rope(
        ctx.h, xd.data_ptr(), ldx, n, pd.data_ptr() if theta else None, runtime.ptr(gd[0]), runtime.ptr(gd[1]),
        xd.data_ptr(), ldx))
    sync()
    inplace = xd.cpu().numpy()
    assert np.array_equal(inplace[:, :w], got[:, :w]) and np.array_equal(inplace[:, w:], x[:, w:])


def test_qk_norm_rope_refuses_positions_without_an_angle():
    ctx = context(4, 2, max_ctx=64, rope_theta=1e4)
    x = torch.randn(4, 768, device="cuda")
    out = torch.full((4, 768), 5.0, device="cuda")
    pos = torch.tensor([0, 64, -1, 63], dtype=torch.int32, device="cuda")
    abi.check("spec_qk_norm_rope", abi.spec_qk_norm_rope(ctx.h, x.data_ptr(), 768, 4, pos.data_ptr(), None, None,
                                                         out.data_ptr(), 768))
    sync()
    assert status(ctx) == abi.ST_CTX_FULL
    o = out.cpu().numpy()
    assert not o[1:3].any() and o[0].any() and o[3].any()


# ---------------------------------------------------------------------------
# refusals: nothing is enqueued
# ---------------------------------------------------------------------------
def test_refusals():
    ctx = context(4, 2, max_ctx=64, rope_theta=1e4)
    kv = runtime.DeviceKV4(ctx.cfg, 4, 4)
    kv.reset(ctx)
    t = torch.zeros(1 << 16, device="cuda")
    a, s = t.data_ptr(), kv.struct()
    far = a + 4 * 32768
    E, N, G = abi.SPEC_EINVAL, abi.SPEC_ENULL, abi.SPEC_EALIGN
    for f in (abi.spec_attention_kv4, abi.spec_attention_window):
        ok = (ctx.h, s, 1, a, 2, 0, 0, far)
        for at, val, rc in ((3, None, N), (7, None, N), (2, -1, E), (2, 2, E), (4, 0, E), (4, 17, E), (5, -1, E),
                            (6, -1, E), (3, a + 4, G), (7, far + 8, G), (7, a, E), (7, a + 16, E)):
            args = list(ok)
            args[at] = val
            assert f(*args) == rc, (f.__name__, at, val)
    ok = (ctx.h, a, 1024, 2, a, None, None, far, 1024)
    for at, val, rc in ((1, None, N), (7, None, N), (4, None, N), (2, 767, E), (2, 764, E), (2, 1026, E), (3, -1, E),
                        (8, 764, E), (8, 770, E), (1, a + 4, G), (7, far + 4, G), (5, a + 4, G), (6, a + 4, G),
                        (7, a + 16, E)):
        args = list(ok)
        args[at] = val
        assert abi.spec_qk_norm_rope(*args) == rc, (at, val)
    assert abi.spec_qk_norm_rope(ctx.h, a, 1024, 2, a, None, None, a, 768) == E       # in place, another stride
    assert abi.spec_qk_norm_rope(ctx.h, a, 1024, 0, a, None, None, far, 1024) == abi.SPEC_OK
    ok = (ctx.h, s, 1, a, far, 256, 2)
    for at, val, rc in ((3, None, N), (4, None, N), (2, 2, E), (2, -1, E), (5, 252, E), (5, 258, E), (6, -1, E),
                        (3, a + 4, G), (4, far + 8, G)):
        args = list(ok)
        args[at] = val
        assert abi.spec_kv4_append(*args) == rc, (at, val)
    ok = (ctx.h, s, 1, 0, 2, a, far, 256)
    for at, val, rc in ((5, None, N), (6, None, N), (2, 2, E), (3, -1, E), (3, 2 ** 31 - 2, E), (4, -1, E), (7, 252, E),
                        (7, 258, E), (5, a + 4, G), (6, a, E), (6, a + 16, E), (6, a + 1024 - 16, E)):
        args = list(ok)
        args[at] = val
        assert abi.spec_kv4_read(*args) == rc, (at, val)
    bad = abi.spec_kv(*[getattr(s, n) for n, _ in s._fields_])
    bad.pool = None
    assert abi.spec_kv4_append(ctx.h, bad, 1, a, far, 256, 2) == N
    assert abi.spec_attention_kv4(ctx.h, bad, 1, a, 2, 0, 0, far) == N
    bad.pool = s.pool + 8
    assert abi.spec_kv4_read(ctx.h, bad, 1, 0, 2, a, far, 256) == G
    sync()
    assert not t.any() and status(ctx) == 0
    # K and V as columns of one matrix are not an overlap
    kv.extend(ctx, 2)
    assert abi.spec_kv4_read(ctx.h, s, 1, 0, 2, a, a + 4 * 256, 512) == abi.SPEC_OK


def test_window_attention_refuses_ring_layers():
    ctx = context(4, 1, max_ctx=256, swa_window=64, swa_period=2)
    kv = runtime.DeviceKV(ctx.cfg, 8, 8)
    kv.reset(ctx)
    kv.extend(ctx, 40)
    q = torch.randn(1, 512, device="cuda")
    out = torch.zeros(1, 512, device="cuda")
    assert abi.spec_attention_window(ctx.h, kv.struct(), 1, q.data_ptr(), 1, 8, 1, out.data_ptr()) == abi.SPEC_EINVAL
    assert abi.spec_attention_window(ctx.h, kv.struct(), 0, q.data_ptr(), 1, 8, 1, out.data_ptr()) == abi.SPEC_OK
    sync()


# ---------------------------------------------------------------------------
# together, and under graphs and streams
# ---------------------------------------------------------------------------
def test_a_draft_layer_end_to_end():
    """Two blocks of one attention layer as a draft runs it: QKV GEMM, QK-norm +
    RoPE, extend, append, attention with a window and sinks, O projection; the
    second block after a rollback.  Every stage against its definition on the
    stage's own inputs."""
    nq, nkv, theta = 4, 2, 1e4
    ctx = context(nq, nkv, max_ctx=512, rope_theta=theta)
    cfg = ctx.cfg
    H, nqkv, w = cfg.hidden, cfg.n_qkv, nkv * 128
    w_qkv = runtime.upload_tiled(ctx, synth.q4k_matrix(nqkv, H, 0, 1), nqkv, H)
    w_o = runtime.upload_tiled(ctx, synth.q4k_matrix(H, nq * 128, 0, 2), H, nq * 128)
    kv = runtime.DeviceKV4(cfg, 40, 32)
    kv.reset(ctx)
    rng = np.random.default_rng(0)
    gq, gk = ((1 + 0.1 * rng.standard_normal(128)).astype(np.float32) for _ in range(2))
    gqd, gkd = torch.from_numpy(gq).cuda(), torch.from_numpy(gk).cuda()
    # a prompt of 300 rows, already rotated
    prompt = rng.standard_normal((300, 2 * w)).astype(np.float32)
    pd = torch.from_numpy(prompt).cuda()
    kv.extend(ctx, 300)
    kv.append(ctx, 1, pd[:, :w], pd[:, w:])
    held = [u.code_values()[c] * u.scale_values()[b].repeat(16, -1)
            for c, b in (u.quantise_rows(prompt[:, i * w:(i + 1) * w], nkv) for i in range(2))]
    length = 300
    for M in (16, 1, 7):
        x = torch.from_numpy(rng.standard_normal((M, H)).astype(np.float32)).cuda()
        y = torch.empty((M, nqkv), device="cuda")
        abi.check("gemm", abi.spec_gemm_q4k(ctx.h, w_qkv.data_ptr(), nqkv, H, x.data_ptr(), M, y.data_ptr()))
        raw = y.cpu().numpy()
        pos = torch.arange(length, length + M, dtype=torch.int32, device="cuda")
        abi.check("qk", abi.spec_qk_norm_rope(ctx.h, y.data_ptr(), nqkv, M, pos.data_ptr(), gqd.data_ptr(),
                                              gkd.data_ptr(), y.data_ptr(), nqkv))
        kv.extend(ctx, M)
        kv.append(ctx, 1, y[:, nq * 128:nq * 128 + w], y[:, nq * 128 + w:])
        q = y[:, :nq * 128].contiguous()
        o = torch.empty((M, nq * 128), device="cuda")
        abi.check("attn", abi.spec_attention_kv4(ctx.h, kv.struct(), 1, q.data_ptr(), M, 128, 4, o.data_ptr()))
        z = torch.empty((M, H), device="cuda")
        abi.check("gemm", abi.spec_gemm_q4k(ctx.h, w_o.data_ptr(), H, nq * 128, o.data_ptr(), M, z.data_ptr()))
        sync()
        got = y.cpu().numpy()
        want, mag = qk_reference(raw, nq, nkv, np.arange(length, length + M), gq, gk, cfg.rms_eps, theta)
        assert (np.abs(got[:, :want.shape[1]] - want) <= 24 * EPS * mag + 1e-38).all()
        for i in range(2):
            code, byte = u.quantise_rows(got[:, nq * 128 + i * w:nq * 128 + (i + 1) * w], nkv)
            held[i] = np.concatenate([held[i][:length], u.code_values()[code] * u.scale_values()[byte].repeat(16, -1)])
        length += M
        ref, bound = u.attention(q.cpu().numpy().reshape(M, nq, 128), held[0], held[1], nq, 128, 4, length,
                                 split=SPLIT["kv4"])
        assert (np.abs(o.cpu().numpy() - ref) <= bound).all()
        assert torch.isfinite(z).all() and z.abs().max() > 0
        # the block is rejected but for its first row
        kv.rollback(ctx, length - M + 1)
        length -= M - 1
    assert status(ctx) == 0


@pytest.mark.parametrize("kind", KINDS)
def test_captured_calls_follow_the_device_length(kind):
    """Extend, (append,) attention captured once and replayed as the sequence
    grows, on a stream of its own, between two eager calls of the same context."""
    stream = torch.cuda.Stream()
    cfg = config(8, 2)
    kv, k, v, ids = None, None, None, None
    with torch.cuda.stream(stream):
        ctx = runtime.Context(cfg, max_ctx=1024, stream=stream)
        kv, k, v, ids = cache(ctx, kind, 400, 61)
        kv.seq_len[0] = 200
        q = torch.randn(3, 8, 128, device="cuda")
        out = torch.empty(3, 1024, device="cuda")
        f = abi.spec_attention_kv4 if kind == "kv4" else abi.spec_attention_window
        st = kv.struct()

        def call():
            abi.check("extend", abi.spec_kv_extend(ctx.h, st, 7))
            abi.check("attention", f(ctx.h, st, 1, q.data_ptr(), 3, 150, 6, out.data_ptr()))
        call()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call()
        for step in range(5):
            graph.replay()
            stream.synchronize()
            length = int(kv.seq_len[0])
            assert length == 207 + 7 * (step + 1)
            want, bound = u.attention(q.cpu().numpy(), k, v, 8, 150, 6, length, split=SPLIT[kind])
            assert (np.abs(out.cpu().numpy() - want) <= bound).all()
        assert status(ctx) == 0
        ctx.close()


def test_two_contexts_on_two_streams():
    """Calls of two contexts in flight at once (small blocks, larger ones and the
    bf16 cache): the same bits as one after the other."""
    jobs = []
    for seed in (1, 2):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            ctx = runtime.Context(config(26, 2), max_ctx=2048, stream=stream)
            for kind in KINDS:
                kv, _, _, _ = cache(ctx, kind, 1500, seed)
                for M in (1, 16):
                    q = torch.randn(M, 26, 128, device="cuda")
                    jobs.append((ctx, kind, kv, q, [torch.empty(M, 26 * 128, device="cuda") for _ in range(2)]))
    sync()

    def call(job, which):
        ctx, kind, kv, q, out = job
        f = abi.spec_attention_kv4 if kind == "kv4" else abi.spec_attention_window
        abi.check("attention", f(ctx.h, kv.struct(), 1, q.data_ptr(), q.shape[0], 700, 3, out[which].data_ptr()))
    for job in jobs:
        call(job, 0)
        sync()
    half = len(jobs) // 2
    for _ in range(5):
        for a, b in zip(jobs[:half], jobs[half:]):
            call(a, 1)
            call(b, 1)
    sync()
    for ctx, _, _, _, out in jobs:
        assert torch.equal(out[0], out[1])
        assert status(ctx) == 0
    for ctx in {id(j[0]): j[0] for j in jobs}.values():
        ctx.close()


@pytest.mark.parametrize("nq,M", [(2, 3), (26, 9)])
def test_calls_back_to_back_see_what_the_call_before_wrote(nq, M):
    """Reading, appending over the same positions, norm and rotation of q, attention,
    again and again without a pause (each kernel may start while the one before
    ends): the same bits as with a pause after every call."""
    ctx = context(nq, 2, max_ctx=1024, rope_theta=1e4)
    rounds, n, length = 24, 200, 700
    kv, _, _, _ = cache(ctx, "kv4", length, 5)
    start = kv.pool.clone()
    gen = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.randn(rounds, n, 512, generator=gen, device="cuda")
    x = torch.randn(rounds, M, (nq + 2) * 128, generator=gen, device="cuda")
    pos = torch.arange(length - M, length, dtype=torch.int32, device="cuda")
    table = kv.page_table.clone()
    other = torch.flip(table[:length // 16].clone(), (0,))
    st = kv.struct()

    def run(pause):
        kv.pool.copy_(start)
        held = torch.empty(rounds, n, 512, device="cuda")
        qk = torch.empty_like(x)
        q = torch.empty(rounds, M, nq * 128, device="cuda")
        out = torch.empty(rounds, M, nq * 128, device="cuda")
        sync()
        rest = sync if pause else (lambda: None)
        for i in range(rounds):
            # the pages change places every other round
            kv.page_table[:length // 16].copy_(other if i % 2 else table[:length // 16])
            rest()
            r, h = rows[i].data_ptr(), held[i].data_ptr()
            abi.check("read", abi.spec_kv4_read(ctx.h, st, 1, length - n, n, h, h + 1024, 512))
            rest()
            abi.check("append", abi.spec_kv4_append(ctx.h, st, 1, r, r + 1024, 512, n))
            rest()
            abi.check("qk", abi.spec_qk_norm_rope(ctx.h, x[i].data_ptr(), x.shape[2], M, pos.data_ptr(), None, None,
                                                  qk[i].data_ptr(), x.shape[2]))
            rest()
            q[i].copy_(qk[i, :, :nq * 128])
            rest()
            abi.check("attention", abi.spec_attention_kv4(ctx.h, st, 1, q[i].data_ptr(), M, 300, 7, out[i].data_ptr()))
            rest()
        sync()
        return held, out
    want = run(True)
    for _ in range(3):
        got = run(False)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    kv.page_table.copy_(table)
    assert status(ctx) == 0
