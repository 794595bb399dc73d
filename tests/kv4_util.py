"""The 4-bit page format, the cache view and attention with a window and sinks,
restated in 64-bit numpy for the tests."""
import numpy as np

MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TOP = 0xE2


def code_values():
    return np.concatenate([MAG, -MAG])


def scale_values():
    b = np.arange(TOP + 1)
    return np.where(b < 8, b * 2.0 ** -17, (8 + b % 8) * 2.0 ** (b // 8 - 18.0))


def quantise(x):
    """Groups [..., 16] of fp32 -> codes [..., 16], scale bytes [..., 1] (NaN as 0)."""
    x = np.asarray(x, dtype=np.float64)
    neg = np.signbit(np.where(np.isnan(x), 0.0, x))
    a = np.abs(np.where(np.isnan(x), 0.0, x))
    vals = scale_values()
    byte = np.minimum(np.searchsorted(6 * vals, a.max(-1, keepdims=True)), TOP)
    s = vals[byte]
    m = np.zeros(x.shape, dtype=np.uint8)
    for t, up in ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5.0, 0)):
        m += (a >= t * s) if up else (a > t * s)
    m = np.where(s == 0, 0, m).astype(np.uint8)
    return m | (neg.astype(np.uint8) << 3), byte.astype(np.uint8)


def quantise_rows(x, nkv):
    """fp32 [n][nkv*128] -> codes [n][nkv][128], scale bytes [n][nkv][8]."""
    code, byte = quantise(np.asarray(x).reshape(-1, nkv, 8, 16))
    return code.reshape(-1, nkv, 128), byte[..., 0]


def to_pages(code, byte):
    """codes [16p][nkv][128], bytes [16p][nkv][8] -> uint8 [p][nkv][1152]."""
    t, nkv = code.shape[:2]
    packed = code[..., 0::2] | (code[..., 1::2] << 4)
    packed = packed.reshape(t // 16, 16, nkv, 4, 16).transpose(0, 2, 3, 1, 4).reshape(t // 16, nkv, 1024)
    return np.concatenate([packed, byte.reshape(t // 16, 16, nkv, 8).transpose(0, 2, 1, 3).reshape(t // 16, nkv, 128)],
                          -1)


def from_pages(pages):
    """uint8 [p][nkv][1152] -> float64 [16p][nkv][128]."""
    p, nkv = pages.shape[:2]
    packed = pages[..., :1024].reshape(p, nkv, 4, 16, 16).transpose(0, 3, 1, 2, 4).reshape(p * 16, nkv, 64)
    code = np.stack([packed & 15, packed >> 4], -1).reshape(p * 16, nkv, 128)
    byte = pages[..., 1024:].reshape(p, nkv, 16, 8).transpose(0, 2, 1, 3).reshape(p * 16, nkv, 8)
    return code_values()[code] * scale_values()[np.minimum(byte, TOP)].repeat(16, -1)


def visible(M, length, window, sinks, mapped=None):
    """bool [M][max(length, 0)]: the keys that each row sees."""
    t = np.arange(max(length, 0))
    p = length - M + np.arange(M)[:, None]
    see = t <= p
    if window:
        see = see & ((t > p - window) | (t < sinks))
    return see if mapped is None else see & mapped


# Error bound of the attention kernels, relative per weight.  With eps = 2^-24:
#  - q and p are split into two binary16 parts, each rounded to nearest with 11
#    significant bits: off by at most half a step of the second, 2^-22 relative
#    (`split`), plus 2^-31 of a row's largest weight where binary16 leaves its
#    normal range;
#  - the score is a sum of 256 products (two parts), each add off by at most
#    2 eps (the tensor core may truncate): 512 eps of sum |q k|; scaled by
#    log2(e) / sqrt(128) (3 eps) and subtracted from the maximum, exp2 is off by
#    2^-22 relative;
#  - weights and outputs are summed over n keys: 2 eps per add, two parts.
# A weight's relative error e turns into at most 2 e of sum w |v|: numerator and
# denominator.
def attention_bound(q, k, v, w, see, split):
    """elementwise bound for o [M][128] of one head, from float64 inputs."""
    eps = 2.0 ** -24
    qk = (np.abs(q) @ np.abs(k).T) / np.sqrt(128.0)
    big = np.where(see, qk, 0.0).max(-1, keepdims=True)                  # [M][1]
    score = big * (split + 512 * eps + 4 * eps)
    n = see.sum(-1, keepdims=True)
    rel = 2 * (2 * score + split + 2.0 ** -22 + 4 * eps * np.minimum(n, 4096) + 64 * eps)
    mean = w @ np.abs(v)
    return rel * mean + n * 2.0 ** -31 * np.abs(np.where(see.any(0)[:, None], v, 0)).max() + 1e-30


def attention(q, k, v, nq, window, sinks, length, mapped=None, split=2.0 ** -22):
    """q [M][nq][128], k, v float64 [>= length][nkv][128] -> (o, bound) [M][nq*128]."""
    M, nkv = q.shape[0], k.shape[1]
    see = visible(M, length, window, sinks, mapped)
    o, bnd = np.zeros((M, nq, 128)), np.zeros((M, nq, 128))
    for h in range(nq):
        kvh = h // (nq // nkv)
        kh, vh, qh = k[:max(length, 0), kvh], v[:max(length, 0), kvh], q[:, h].astype(np.float64)
        kh = np.where(see.any(0)[:, None], kh, 0.0)
        for i in range(M):
            at = np.nonzero(see[i])[0]
            if len(at) == 0:
                continue
            s = kh[at] @ qh[i] / np.sqrt(128.0)
            w = np.exp(s - s.max())
            w /= w.sum()
            o[i, h] = w @ vh[at]
            bnd[i, h] = attention_bound(qh[i:i + 1], kh[at], vh[at], w[None], np.ones((1, len(at)), bool), split)
    return o.reshape(M, -1), bnd.reshape(M, -1)
