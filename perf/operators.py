"""Cases and plain forms of the building blocks around a 4-bit KV cache.

Four operators, each for one layer of one sequence:

  qk_norm_rope      RMS norm of every q and k head with its gain, then the
                    rotary embedding at the row's position
  kv4_store         K and V rows quantised into the pages of a 4-bit cache, and
                    the same rows read back as the values that they stand for
  attention_kv4     the last M positions' queries against a 4-bit paged cache
  attention_window  the same against the bf16 paged cache, every row seeing a
                    window of the last W positions and a few first ones (sinks)

`run` computes them with elementary torch operations in 32 bits (angles in 64)
where `own` is false, and calls the library where it is true.

A 4-bit page of one (layer, K or V, KV head) is 1,152 bytes for 16 positions:
  byte 256*c + 16*t + j   codes of elements 32c + 2j (low nibble) and
                          32c + 2j + 1 (high) of position t, c < 4, j < 16
  byte 1024 + 8*t + g     scale of elements 16g .. 16g + 15 of position t
A code is e2m1: sign, then one of 0, .5, 1, 1.5, 2, 3, 4, 6.  A scale byte b
stands for the binary16 number of bits b << 7, at most 10240 (b = 0xE2).
Quantising: the smallest scale s with 6 s >= the group's largest magnitude (at
most 10240), then the nearest code to x / s, ties to the even code.
"""
import math

import torch

own = False

DH = 128
PAGE = 16
LAYERS = 2            # the pools hold two layers, the calls work on the second
LAYER = 1
MAG = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TOP_SCALE = 0xE2      # the byte of 10240, the largest scale
EPS = 1e-6
THETA = 500000.0      # base of the rotary angles

# (query heads, KV heads): the 52-block target, its draft, the half-width test
# model, and generic grouped, single-KV-head and ungrouped attention
HEADS = ((52, 4), (48, 4), (26, 2), (32, 8), (8, 1), (16, 16))


def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoded token, a k + 1 = 16 verify block, a long prompt of odd length
        dict(name="qk_norm_rope_1", op="qk_norm_rope", n=1, nq=52, nkv=4, start=2055),
        dict(name="qk_norm_rope_16", op="qk_norm_rope", n=16, nq=52, nkv=4, start=32768),
        dict(name="qk_norm_rope_8191", op="qk_norm_rope", n=8191, nq=52, nkv=4, start=0),
        # the rows of a verify block; a prompt laid down behind a short context
        dict(name="kv4_store_16", op="kv4_store", n=16, nq=52, nkv=4, start=2055),
        dict(name="kv4_store_32761", op="kv4_store", n=32761, nq=52, nkv=4, start=7),
        # decoding and verifying at the benchmark's 2k context, verifying at
        # 32k, decoding behind a 128k context
        dict(name="attention_kv4_1_2k", op="attention_kv4", m=1, length=2056, nq=52, nkv=4, window=0, sinks=0),
        dict(name="attention_kv4_16_2k", op="attention_kv4", m=16, length=2071, nq=52, nkv=4, window=0, sinks=0),
        dict(name="attention_kv4_16_32k", op="attention_kv4", m=16, length=32784, nq=52, nkv=4, window=0, sinks=0),
        dict(name="attention_kv4_1_128k", op="attention_kv4", m=1, length=131071, nq=52, nkv=4, window=0, sinks=0),
        # a draft's token with a small window, a verify block with a larger one,
        # eight rows over most of a long context
        dict(name="attention_window_1_1k", op="attention_window", m=1, length=32769, nq=48, nkv=4, window=1024, sinks=4),
        dict(name="attention_window_16_4k", op="attention_window", m=16, length=16400, nq=52, nkv=4, window=4096,
             sinks=16),
        dict(name="attention_window_8_32k", op="attention_window", m=8, length=131072, nq=52, nkv=4, window=32768,
             sinks=100),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("qk_norm_rope", "kv4_store", "attention_kv4", "attention_window"))
    nq, nkv = rng.choice(HEADS)
    if op == "qk_norm_rope":
        return dict(op=op, n=_log(rng, 1, 8191), nq=nq, nkv=nkv, start=rng.randrange(0, 120000))
    if op == "kv4_store":
        return dict(op=op, n=_log(rng, 1, 32761 * 4 // max(4, nkv)), nq=nq, nkv=nkv, start=rng.randrange(0, 3000))
    m = rng.randint(1, 16)
    longest = min(131072 * 4 // max(4, nkv), 32784 * 16 // m)
    length = max(m, _log(rng, 1, longest))
    if op == "attention_kv4" and rng.random() < 0.6:
        return dict(op=op, m=m, length=length, nq=nq, nkv=nkv, window=0, sinks=0)
    window = _log(rng, 1, min(length, 262144 // m // max(1, nkv // 4)))
    return dict(op=op, m=m, length=length, nq=nq, nkv=nkv, window=window, sinks=rng.choice((0, 1, 4, 16, 33, 100)))


def _seen(case):
    """Keys that some row sees, and the (row, key) pairs that are seen, of an attention case."""
    m, length, w, sinks = case["m"], case["length"], case["window"], case["sinks"]
    past = length - m
    lo = max(0, past - w + 1) if w else 0
    keys = length - lo + min(sinks if w else 0, lo)
    pairs = 0
    for i in range(m):
        p = past + i
        first = max(0, p - w + 1) if w else 0
        pairs += p + 1 - first + min(sinks if w else 0, first)
    return keys, pairs


def work(case):
    nq, nkv = case["nq"], case["nkv"]
    if case["op"] == "qk_norm_rope":
        cols = (nq + nkv) * DH
        return dict(bytes=case["n"] * (8 * cols + 8 * (DH // 2) + 4), flops=case["n"] * cols * 8)
    if case["op"] == "kv4_store":
        values = 2 * case["n"] * nkv * DH
        return dict(bytes=values * (4 + 4) + 2 * values * 9 // 16, flops=values * 4)
    keys, pairs = _seen(case)
    per_value = 9 / 16 if case["op"] == "attention_kv4" else 2
    return dict(bytes=int(2 * keys * nkv * DH * per_value) + 2 * 4 * case["m"] * nq * DH, flops=4 * DH * nq * pairs)


# ---------------------------------------------------------------------------
# the 4-bit format, in elementary operations
# ---------------------------------------------------------------------------
def _scale_values(device):
    return (torch.arange(TOP_SCALE + 1, dtype=torch.int16, device=device) << 7).view(torch.float16).float()


def _quantise(x):
    """fp32 [..., 128] -> codes uint8 [..., 128] and scale bytes uint8 [..., 8]."""
    vals = _scale_values(x.device)
    g = x.reshape(*x.shape[:-1], 8, 16)
    byte = torch.searchsorted(6 * vals, g.abs().amax(-1).contiguous()).clamp_(max=TOP_SCALE)
    s = vals[byte][..., None]
    a = g.abs()
    mag = torch.zeros(g.shape, dtype=torch.uint8, device=x.device)
    # midpoints between neighbouring magnitudes; exact products in fp32
    for t, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        mag += (a >= t * s) if up else (a > t * s)
    mag[(s == 0).expand_as(mag)] = 0
    code = mag | (torch.signbit(g).to(torch.uint8) << 3)
    return code.reshape(x.shape), byte.to(torch.uint8)


def _to_pages(code, byte):
    """Codes [t, nkv, 128] and scale bytes [t, nkv, 8], t a multiple of 16 -> pages [t / 16, nkv, 1152]."""
    t, nkv = code.shape[0], code.shape[1]
    packed = code[..., 0::2] | (code[..., 1::2] << 4)                         # [t, nkv, 64]
    packed = packed.reshape(t // PAGE, PAGE, nkv, 4, 16).permute(0, 2, 3, 1, 4).reshape(t // PAGE, nkv, 1024)
    scales = byte.reshape(t // PAGE, PAGE, nkv, 8).permute(0, 2, 1, 3).reshape(t // PAGE, nkv, 128)
    return torch.cat((packed, scales), -1)


def _from_pages(pages):
    """Pages [p, nkv, 1152] -> fp32 values [16 p, nkv, 128]."""
    p, nkv = pages.shape[0], pages.shape[1]
    lut = torch.tensor(MAG + tuple(-m for m in MAG), dtype=torch.float32, device=pages.device)
    packed = pages[..., :1024].reshape(p, nkv, 4, PAGE, 16).permute(0, 3, 1, 2, 4).reshape(p * PAGE, nkv, 64)
    code = torch.stack((packed & 15, packed >> 4), -1).reshape(p * PAGE, nkv, DH)
    byte = pages[..., 1024:].reshape(p, nkv, PAGE, 8).permute(0, 2, 1, 3).reshape(p * PAGE, nkv, 8)
    s = _scale_values(pages.device)[byte.long().clamp_(max=TOP_SCALE)]
    return (lut[code.long()].reshape(p * PAGE, nkv, 8, 16) * s[..., None]).reshape(p * PAGE, nkv, DH)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _inputs(case, seed):
    """Everything that `run` reads, made from the seed alone."""
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def perm(n):
        return torch.randperm(n, generator=gen, device=dev).to(torch.int32)

    nq, nkv = case["nq"], case["nkv"]
    if case["op"] == "qk_norm_rope":
        return dict(x=normal(case["n"], (nq + 2 * nkv) * DH) * 3,
                    pos=torch.arange(case["start"], case["start"] + case["n"], dtype=torch.int32, device=dev),
                    gq=1 + 0.2 * normal(DH), gk=1 + 0.2 * normal(DH))
    # keys have channels of unlike size: every 32nd is four times as wide
    wide = 1 + 3 * (torch.arange(DH, device=dev) % 32 == 5).float()
    if case["op"] == "kv4_store":
        # rows of a QKV projection: q, then k, then v columns
        length = case["start"] + case["n"]
        pages = -(-length // PAGE)
        rows = normal(case["n"], (nq + 2 * nkv) * DH)
        rows[:, nq * DH:(nq + nkv) * DH] *= wide.repeat(nkv)
        return dict(rows=rows, table=perm(pages + 3)[:pages].contiguous(), length=length,
                    pool=torch.zeros((pages + 3, LAYERS, 2, nkv, 1152), dtype=torch.uint8, device=dev))
    length = case["length"]
    pages = -(-length // PAGE)
    table = perm(pages + 3)[:pages].contiguous()
    q = normal(case["m"], nq, DH)
    kv = [normal(pages * PAGE, nkv, DH) * wide, normal(pages * PAGE, nkv, DH)]
    if case["op"] == "attention_kv4":
        pool = torch.zeros((pages + 3, LAYERS, 2, nkv, 1152), dtype=torch.uint8, device=dev)
        for which in range(2):
            pool[table.long(), LAYER, which] = _to_pages(*_quantise(kv[which]))
    else:
        pool = torch.zeros((pages + 3, LAYERS, 2, nkv, PAGE, DH), dtype=torch.bfloat16, device=dev)
        for which in range(2):
            rows = kv[which].to(torch.bfloat16).reshape(pages, PAGE, nkv, DH)
            pool[table.long(), LAYER, which] = rows.permute(0, 2, 1, 3)
    return dict(q=q, table=table, length=length, pool=pool)


def prepare(case, seed):
    s = dict(case=dict(case), **_inputs(case, seed))
    dev = _device()
    nq, nkv = case["nq"], case["nkv"]
    if case["op"] == "qk_norm_rope":
        s["out"] = torch.empty((case["n"], (nq + nkv) * DH), device=dev)
    elif case["op"] == "kv4_store":
        s["k"], s["v"] = (torch.empty((case["n"], nkv * DH), device=dev) for _ in range(2))
    else:
        s["out"] = torch.empty((case["m"], nq * DH), device=dev)
    if own:
        s["abi"], s["ctx"], s["kv"] = _handles(s)
    return s


def _handles(s):
    """The library's context and, for a cache, its view of the paged cache."""
    from speculative_decoding_exact_gb300 import abi, runtime
    case = s["case"]
    rope = case["op"] == "qk_norm_rope"
    span = case["start"] + case["n"] if rope else s["length"] + 16
    cfg = runtime.ModelConfig(hidden=256, n_layers=LAYERS, n_q_heads=case["nq"], n_kv_heads=case["nkv"], head_dim=DH,
                              ffn=256, vocab=16, rms_eps=EPS, rope_theta=THETA if rope else 0.0)
    ctx = runtime.Context(cfg, max_ctx=max(16, span))
    if rope:
        return abi, ctx, None
    s["seq_len"] = torch.tensor([s["length"]], dtype=torch.int32, device=s["pool"].device)
    s["free"] = torch.zeros(s["pool"].shape[0], dtype=torch.int32, device=s["pool"].device)
    s["top"] = torch.zeros(1, dtype=torch.int32, device=s["pool"].device)
    kv = abi.spec_kv(s["pool"].data_ptr(), s["pool"].shape[0], s["table"].numel(), s["table"].data_ptr(),
                     s["seq_len"].data_ptr(), s["free"].data_ptr(), s["top"].data_ptr(), None, None)
    return abi, ctx, kv


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _own_qk(s):
    c, a = s["case"], s["abi"]
    a.check("spec_qk_norm_rope", a.spec_qk_norm_rope(
        s["ctx"].h, s["x"].data_ptr(), s["x"].stride(0), c["n"], s["pos"].data_ptr(), s["gq"].data_ptr(),
        s["gk"].data_ptr(), s["out"].data_ptr(), s["out"].stride(0)))
    return s["out"]


def _own_store(s):
    c, a, h = s["case"], s["abi"], s["ctx"].h
    rows = s["rows"].data_ptr()
    k = rows + 4 * c["nq"] * DH
    a.check("spec_kv4_append", a.spec_kv4_append(h, s["kv"], LAYER, k, k + 4 * c["nkv"] * DH, s["rows"].stride(0),
                                                 c["n"]))
    a.check("spec_kv4_read", a.spec_kv4_read(h, s["kv"], LAYER, c["start"], c["n"], s["k"].data_ptr(),
                                             s["v"].data_ptr(), s["k"].stride(0)))
    return s["k"], s["v"]


def _own_kv4(s):
    c, a = s["case"], s["abi"]
    a.check("spec_attention_kv4", a.spec_attention_kv4(s["ctx"].h, s["kv"], LAYER, s["q"].data_ptr(), c["m"],
                                                       c["window"], c["sinks"], s["out"].data_ptr()))
    return s["out"]


def _own_window(s):
    c, a = s["case"], s["abi"]
    a.check("spec_attention_window", a.spec_attention_window(s["ctx"].h, s["kv"], LAYER, s["q"].data_ptr(), c["m"],
                                                             c["window"], c["sinks"], s["out"].data_ptr()))
    return s["out"]


def _plain_qk(s):
    c = s["case"]
    nq, nkv, n = c["nq"], c["nkv"], c["n"]
    x = s["x"][:, :(nq + nkv) * DH].reshape(n, nq + nkv, DH)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    y = torch.cat((y[:, :nq] * s["gq"], y[:, nq:] * s["gk"]), 1)
    freq = THETA ** (-torch.arange(DH // 2, dtype=torch.float64, device=x.device) / (DH // 2))
    ang = s["pos"].double()[:, None] * freq
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    a, b = y[..., :DH // 2], y[..., DH // 2:]
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1).reshape(n, (nq + nkv) * DH)


def _plain_store(s):
    c = s["case"]
    nq, nkv, n, start = c["nq"], c["nkv"], c["n"], c["start"]
    at = torch.arange(start, start + n, device=s["rows"].device)
    page, slot = s["table"].long()[at // PAGE], at % PAGE
    out = []
    for which in range(2):
        first = (nq + which * nkv) * DH
        code, byte = _quantise(s["rows"][:, first:first + nkv * DH].reshape(n, nkv, DH))
        half = s["pool"][:, LAYER, which]                                     # [pages, nkv, 1152], a view
        packed = (code[..., 0::2] | (code[..., 1::2] << 4)).reshape(n, nkv, 4, 16)
        half[..., :1024].view(-1, nkv, 4, PAGE, 16)[page, :, :, slot] = packed
        half[..., 1024:].view(-1, nkv, PAGE, 8)[page, :, slot] = byte
        lo, hi = start // PAGE, -(-(start + n) // PAGE)
        rows = _from_pages(half[s["table"].long()[lo:hi]])
        out.append(rows[start - lo * PAGE:][:n].reshape(n, nkv * DH))
    return tuple(out)


def _plain_attention(s):
    c = s["case"]
    m, nq, nkv, w = c["m"], c["nq"], c["nkv"], c["window"]
    length, dev = s["length"], s["q"].device
    past = length - m
    # the pages that hold a visible key
    lo = max(0, past - w + 1) // PAGE if w else 0
    first = min(lo, -(-c["sinks"] // PAGE)) if w else 0
    pages = torch.cat((torch.arange(first, device=dev), torch.arange(lo, -(-length // PAGE), device=dev)))
    at = (pages[:, None] * PAGE + torch.arange(PAGE, device=dev)).reshape(-1)
    held = s["pool"][s["table"].long()[pages], LAYER]
    if c["op"] == "attention_kv4":
        k, v = _from_pages(held[:, 0]), _from_pages(held[:, 1])
    else:
        k, v = (held[:, i].permute(0, 2, 1, 3).reshape(-1, nkv, DH).float() for i in range(2))
    row = past + torch.arange(m, device=dev)[:, None]
    see = at <= row
    if w:
        see &= (at > row - w) | (at < c["sinks"])
    g = nq // nkv
    q = s["q"].reshape(m, nkv, g, DH).permute(1, 2, 0, 3).reshape(nkv, g * m, DH)
    score = torch.matmul(q, k.permute(1, 2, 0)) / math.sqrt(DH)
    score = score.reshape(nkv, g, m, -1).masked_fill(~see, float("-inf"))
    p = torch.exp(score - score.amax(-1, keepdim=True))
    o = torch.matmul(p.reshape(nkv, g * m, -1), v.permute(1, 0, 2)).reshape(nkv, g, m, DH) / p.sum(-1, keepdim=True)
    return o.permute(2, 0, 1, 3).reshape(m, nq * DH)


_OWN = dict(qk_norm_rope=_own_qk, kv4_store=_own_store, attention_kv4=_own_kv4, attention_window=_own_window)
_PLAIN = dict(qk_norm_rope=_plain_qk, kv4_store=_plain_store, attention_kv4=_plain_attention,
              attention_window=_plain_attention)


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_page_values(pages):
    """Pages uint8 [p, nkv, 1152] -> float64 [16 p, nkv, 128], element by element from the byte positions."""
    p, nkv = pages.shape[0], pages.shape[1]
    dev = pages.device
    d = torch.arange(DH, device=dev)
    t = torch.arange(PAGE, device=dev)[:, None]
    byte = pages[:, :, 256 * (d // 32) + 16 * t + (d % 32) // 2].int()        # [p, nkv, 16, 128]
    code = torch.where(d % 2 == 0, byte % 16, byte // 16)
    e, f = (code % 8) // 2, code % 2
    mag = torch.where(e == 0, 0.5 * f.double(), (1 + 0.5 * f.double()) * torch.pow(2.0, (e - 1).double()))
    b = pages[:, :, 1024 + 8 * t + d // 16].int().clamp(max=TOP_SCALE)
    be, bf = b // 8, (b % 8).double()
    s = torch.where(be == 0, bf / 8 * 2.0 ** -14, (1 + bf / 8) * torch.pow(2.0, (be - 15).double()))
    val = torch.where(code >= 8, -mag, mag) * s
    return val.permute(0, 2, 1, 3).reshape(p * PAGE, nkv, DH)


def _exact_store(x):
    """fp32 [n, w] -> float64 values after quantising groups of 16."""
    g = x.double().reshape(x.shape[0], -1, 16)
    b = torch.arange(TOP_SCALE + 1, device=x.device)
    be, bf = b // 8, (b % 8).double()
    vals = torch.where(be == 0, bf * 2.0 ** -17, (8 + bf) * torch.pow(2.0, (be - 18).double()))
    top = g.abs().amax(-1, keepdim=True)
    enough = torch.searchsorted(vals * 6, top.contiguous()).clamp(max=TOP_SCALE)
    s = vals[enough]
    mags = torch.tensor(MAG, dtype=torch.float64, device=x.device)
    out = torch.empty_like(g)
    step = max(1, (1 << 24) // g[0].numel())
    for i in range(0, g.shape[0], step):                                      # bounded memory
        part, sp = g[i:i + step], s[i:i + step]
        off = (part.abs()[..., None] - mags * sp[..., None]).abs()
        # nearest magnitude; of two equally near ones the even one comes first in this order
        order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device=x.device)
        pick = order[off[..., order].argmin(-1)]
        val = mags[pick] * sp
        out[i:i + step] = torch.where(part < 0, -val, val)
    return out.reshape(x.shape)


def exact(case, seed):
    s = _inputs(case, seed)
    nq, nkv = case["nq"], case["nkv"]
    if case["op"] == "qk_norm_rope":
        x = s["x"].double()[:, :(nq + nkv) * DH].reshape(case["n"], nq + nkv, DH)
        gain = torch.cat((s["gq"].double().expand(nq, DH), s["gk"].double().expand(nkv, DH)))
        y = x * gain / (x.square().sum(-1, keepdim=True) / DH + EPS).sqrt()
        i = torch.arange(DH // 2, device=x.device).double()
        turn = torch.polar(torch.ones(1, dtype=torch.float64, device=x.device),
                           s["pos"].double()[:, None, None] * torch.exp(-i / (DH // 2) * math.log(THETA)))
        z = torch.complex(y[..., :DH // 2].contiguous(), y[..., DH // 2:].contiguous()) * turn
        return torch.cat((z.real, z.imag), -1).reshape(case["n"], -1)
    if case["op"] == "kv4_store":
        k = s["rows"][:, nq * DH:(nq + nkv) * DH]
        return _exact_store(k), _exact_store(s["rows"][:, (nq + nkv) * DH:])
    m, length, w = case["m"], case["length"], case["window"]
    q = s["q"].double()
    out = torch.empty((m, nq, DH), dtype=torch.float64, device=q.device)
    table = s["table"].long()
    t = torch.arange(length, device=q.device)
    for h in range(nkv):
        held = s["pool"][table, LAYER, :, h:h + 1]
        if case["op"] == "attention_kv4":
            k, v = (_exact_page_values(held[:, i])[:length, 0] for i in range(2))
        else:
            k, v = (held[:, i, 0].reshape(-1, DH)[:length].double() for i in range(2))
        g = slice(h * (nq // nkv), (h + 1) * (nq // nkv))
        for i in range(m):
            p = length - m + i
            see = t <= p
            if w:
                see = see & ((t >= p - w + 1) | (t < case["sinks"]))
            at = see.nonzero()[:, 0]
            weight = torch.softmax(q[i, g] @ k[at].T / DH ** 0.5, -1)
            out[i, g] = weight @ v[at]
    return out.reshape(m, nq * DH)
