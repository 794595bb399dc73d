"""What the entry points and runtime classes refuse and allow around the two paged
caches."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from speculative_decoding_exact_gb300 import abi, runtime, synth  # noqa: E402
from tests import kv4_util as u  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def config(nq=4, nkv=2, **kw):
    return runtime.ModelConfig(hidden=512, n_layers=2, n_q_heads=nq, n_kv_heads=nkv, head_dim=128, ffn=512, vocab=512,
                               **kw)


def sync():
    torch.cuda.synchronize()


def weights(ctx):
    cfg = ctx.cfg
    w = runtime.DeviceWeights(cfg)
    for i in range(cfg.n_layers):
        for j, (name, N, K) in enumerate(cfg.matrices()):
            getattr(w, name).append(runtime.upload_tiled(ctx, synth.q4k_matrix(N, K, i, j), N, K))
    w.w_head = runtime.upload_tiled(ctx, synth.q4k_matrix(cfg.vocab, cfg.hidden, 9, 9), cfg.vocab, cfg.hidden)
    return w


def test_a_cache_of_the_other_kind_is_refused():
    """A 4-bit pool has smaller pages than a bf16 one: a call that took it for bf16 rows
    would reach past it.  (Large enough here that nothing would.)"""
    cfg = config()
    ctx = runtime.Context(cfg, max_ctx=128)
    w = weights(ctx)
    big = torch.zeros(8 * 2 * 2 * 2 * 4096, dtype=torch.uint8, device="cuda")
    kv = {abi.KV_BF16: runtime.DeviceKV(cfg, 8, 8), abi.KV_4BIT: runtime.DeviceKV4(cfg, 8, 8)}
    kv[abi.KV_4BIT].pool = big
    hidden, q, out, k, v = (torch.zeros(16, 512, device="cuda") for _ in range(5))
    draft = torch.zeros(15, dtype=torch.int32, device="cuda")
    parent = torch.tensor([-1, 0, 0], dtype=torch.int32, device="cuda")
    probs = torch.full((3, cfg.vocab), 1.0 / cfg.vocab, device="cuda")
    mt = torch.zeros(abi.MT_WORDS + 3, dtype=torch.int32, device="cuda")
    res = torch.zeros(4, dtype=torch.int32, device="cuda")
    hh, dh, rh = torch.zeros(4, 512), torch.zeros(3, dtype=torch.int32), abi.spec_result()
    h, p = ctx.h, lambda t: t.data_ptr()
    calls = {
        "step": (abi.KV_BF16, lambda s: abi.spec_verify_step(h, w.struct(), s, p(hidden), p(draft), 3, p(res))),
        "step_ex": (abi.KV_BF16, lambda s: abi.spec_verify_step_ex(h, w.struct(), s, p(hidden), p(draft), 3, p(res), None)),
        "step_host": (abi.KV_BF16, lambda s: abi.spec_verify_step_host(h, w.struct(), s, p(hh), p(dh), 3, rh)),
        "sampled": (abi.KV_BF16, lambda s: abi.spec_verify_step_sampled(h, w.struct(), s, p(hidden), p(draft), p(probs), 3,
                                                                        p(mt), p(res), None)),
        "tree": (abi.KV_BF16, lambda s: abi.spec_verify_tree(h, w.struct(), s, p(hidden), p(draft), p(parent), 3, p(res),
                                                             None, None)),
        "attention": (abi.KV_BF16, lambda s: abi.spec_attention(h, s, 1, p(q), 2, p(out))),
        "window": (abi.KV_BF16, lambda s: abi.spec_attention_window(h, s, 1, p(q), 2, 0, 0, p(out))),
        "kv4": (abi.KV_4BIT, lambda s: abi.spec_attention_kv4(h, s, 1, p(q), 2, 0, 0, p(out))),
        "append": (abi.KV_4BIT, lambda s: abi.spec_kv4_append(h, s, 1, p(k), p(v), 512, 2)),
        "read": (abi.KV_4BIT, lambda s: abi.spec_kv4_read(h, s, 1, 0, 2, p(k), p(v), 512)),
    }
    for c in kv.values():
        c.reset(ctx)
        c.extend(ctx, 5)                                   # the metadata calls take either
        c.rollback(ctx, 4)
    for name, (takes, call) in calls.items():
        for kind, c in kv.items():
            before, lengths = c.pool.clone(), c.seq_len.clone()
            s = c.struct()
            assert s.kind == kind
            if kind == takes:
                assert call(s) == abi.SPEC_OK, name
                sync()
                c.rollback(ctx, 4)
                sync()
                abi.spec_last_status(ctx.h)
            else:
                assert call(s) == abi.SPEC_EINVAL, name
                sync()
                assert torch.equal(before, c.pool) and torch.equal(lengths, c.seq_len)
    ctx.close()


def test_a_4bit_cache_beside_sliding_window_layers():
    """On a context with sliding-window layers a 4-bit cache needs no rings: reset,
    extend, append, attention on a ring layer and rollback, which reaches any length."""
    nq, nkv = 4, 2
    ctx = runtime.Context(config(nq, nkv, swa_window=32, swa_period=2), max_ctx=256)
    kv = runtime.DeviceKV4(ctx.cfg, 16, 16)
    assert kv.swa_ring is None and kv.swa_state is None
    kv.reset(ctx)
    kv.extend(ctx, 100)
    rows = np.random.default_rng(1).standard_normal((100, 2 * nkv * 128)).astype(np.float32)
    x = torch.from_numpy(rows).cuda()
    kv.append(ctx, 1, x[:, :nkv * 128], x[:, nkv * 128:])
    held = [u.code_values()[c] * u.scale_values()[b].repeat(16, -1)
            for c, b in (u.quantise_rows(rows[:, i * nkv * 128:(i + 1) * nkv * 128], nkv) for i in range(2))]
    q = np.random.default_rng(2).standard_normal((3, nq, 128)).astype(np.float32)
    qd = torch.from_numpy(q).cuda()
    out = torch.empty((3, nq * 128), device="cuda")
    for length in (100, 90, 20, 100):                      # back, further back, and forward again
        if length < 100 or int(kv.seq_len[0]) == 100:
            kv.rollback(ctx, length)
        else:
            kv.extend(ctx, length - int(kv.seq_len[0]))
        abi.check("attention", abi.spec_attention_kv4(ctx.h, kv.struct(), 1, qd.data_ptr(), 3, 40, 4, out.data_ptr()))
        sync()
        assert int(kv.seq_len[0]) == length
        want, bound = u.attention(q, held[0], held[1], nq, 40, 4, length)
        assert (np.abs(out.cpu().numpy() - want) <= bound).all()
    assert abi.spec_last_status(ctx.h) == 0
    # bf16: the metadata calls go without rings too, half of them or a step do not
    bf = runtime.DeviceKV(ctx.cfg, 16, 16)
    s = bf.struct()
    w = weights(ctx)
    hidden, draft = torch.zeros(4, 512, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    res = torch.zeros(4, dtype=torch.int32, device="cuda")
    for ring, state in ((None, s.swa_state), (s.swa_ring, None)):
        half = bf.struct()
        half.swa_ring, half.swa_state = ring, state
        assert abi.spec_kv_reset(ctx.h, half) == abi.spec_kv_extend(ctx.h, half, 1) == abi.SPEC_ENULL
        assert abi.spec_kv_rollback(ctx.h, half, 0) == abi.SPEC_ENULL
    s.swa_ring = s.swa_state = None
    assert abi.spec_kv_reset(ctx.h, s) == abi.spec_kv_extend(ctx.h, s, 8) == abi.SPEC_OK
    assert abi.spec_verify_step(ctx.h, w.struct(), s, hidden.data_ptr(), draft.data_ptr(), 3, res.data_ptr()) == abi.SPEC_ENULL
    assert abi.spec_attention(ctx.h, s, 1, hidden.data_ptr(), 2, hidden.data_ptr()) == abi.SPEC_ENULL
    sync()
    # a cache with rings keeps its limit: no rollback below an extend
    bf.reset(ctx)
    bf.extend(ctx, 60)
    bf.rollback(ctx, 59)
    assert abi.spec_last_status(ctx.h) == abi.ST_ROLLBACK and int(bf.seq_len[0]) == 60
    ctx.close()


def test_append_and_read_of_rows_on_another_stream():
    """Rows written on the current stream, a context on a stream of its own, results
    used on the current stream at once: every call waits for what it needs."""
    own = torch.cuda.Stream()
    ctx = runtime.Context(config(), max_ctx=128, stream=own)
    kv = runtime.DeviceKV4(ctx.cfg, 8, 8)
    sync()
    kv.reset(ctx)
    kv.extend(ctx, 100)
    sync()
    rng = np.random.default_rng(1)
    for i in range(3):
        rows = rng.standard_normal((100, 512)).astype(np.float32)
        src = torch.from_numpy(rows).cuda()
        sync()
        x = torch.zeros(100, 512, device="cuda")
        torch.cuda._sleep(20_000_000)                       # some 10 ms: x is written late
        x.copy_(src)
        kv.append(ctx, 1, x[:, :256], x[:, 256:])
        del x
        junk = torch.full((100, 512), 7.0, device="cuda")   # may take x's memory
        with torch.cuda.stream(own):
            torch.cuda._sleep(20_000_000)                   # k and v are written late
        k, v = kv.read(ctx, 1, 0, 100)
        got = torch.cat((k, v), 1).clone()
        sync()
        want = np.concatenate([(u.code_values()[c] * u.scale_values()[b].repeat(16, -1)).reshape(100, 256)
                               for c, b in (u.quantise_rows(rows[:, j * 256:j * 256 + 256], 2) for j in range(2))], 1)
        assert np.array_equal(got.cpu().numpy(), want.astype(np.float32)), i
        del junk
    assert abi.spec_last_status(ctx.h) == 0
    ctx.close()


def test_append_of_single_rows_and_other_strides():
    ctx = runtime.Context(config(), max_ctx=128)
    kv = runtime.DeviceKV4(ctx.cfg, 8, 8)
    kv.reset(ctx)
    kv.extend(ctx, 1)
    x = torch.randn(1, 256, device="cuda")
    y = torch.randn(1, 1024, device="cuda")[:, 512:768]     # one row: its stride says nothing
    kv.append(ctx, 1, x, y)
    kv.append(ctx, 1, x[:0], y[:0])
    k, v = kv.read(ctx, 1, 0, 1)
    for got, rows in ((k, x), (v, y)):
        c, b = u.quantise_rows(rows.cpu().numpy(), 2)
        want = (u.code_values()[c] * u.scale_values()[b].repeat(16, -1)).reshape(1, 256)
        assert np.array_equal(got.cpu().numpy(), want.astype(np.float32))
    assert kv.read(ctx, 1, 0, 0)[0].shape == (0, 256)
    two = torch.randn(2, 512, device="cuda")
    for bad in ((two[:, :256], torch.randn(2, 256, device="cuda")), (two[:, ::2], two[:, ::2]), (two[:, :256], two[:1, :256])):
        with pytest.raises(ValueError):
            kv.append(ctx, 1, *bad)
    assert abi.spec_last_status(ctx.h) == 0
    ctx.close()
