"""Attention with operands in parts, in numpy: what the kernels' precision rests on,
and the bound that a lost part breaks."""
import numpy as np

from tests import kv4_util as u

# Relative L2 error of the output against 64 bits, for rows whose scores are a few
# units.  With eps = 2^-24: an operand split (rms below eps a product, random over the
# 128 products of a score), 16 additions in a tensor core that truncates (2 eps each at
# most, of partial sums that grow to the score: 16 eps of it on average), log2(e) /
# sqrt(d), exp2 (4 eps) and the additions over keys, a tile at a time (as many again):
# at most about 34 eps, of which random signs leave a part.  Without one part of q or p
# an otherwise exact sum is off by 1.7e-4 (binary16, 11 bits) or 8e-6 (bf16, 16 bits).
ACCURACY = 2.0 ** -19      # 1.9e-6


def rel_l2(got, want):
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    return float(np.sqrt(((got - want) ** 2).sum() / (want ** 2).sum()))


def parts_binary16(x, n):
    """x [rows][cols] as the sum of n binary16 parts, rows scaled by a power of two."""
    x = np.asarray(x, dtype=np.float64)
    scale = 2.0 ** np.floor(np.log2(np.abs(x).max(-1, keepdims=True) + 1e-300))
    left, out = x / scale, np.zeros_like(x)
    for _ in range(n):
        h = left.astype(np.float16).astype(np.float64)
        out, left = out + h, left - h
    return out * scale


def parts_bf16(x, n):
    """x as the sum of n bf16 parts by truncation."""
    left, out = np.asarray(x, dtype=np.float32), np.zeros(np.shape(x))
    for _ in range(n):
        h = (left.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
        out, left = out + h, left - h
    return out


def attention64(q, k, v, nq, window, sinks, length, split=2.0 ** -22):
    """As kv4_util.attention, a head at a time: (o, bound) [M][nq*128]."""
    M, nkv = q.shape[0], k.shape[1]
    see = u.visible(M, length, window, sinks)
    keys = np.nonzero(see.any(0))[0]
    see = see[:, keys]
    o, bound = np.zeros((M, nq, 128)), np.zeros((M, nq, 128))
    for h in range(nq):
        kh, vh, qh = k[keys, h // (nq // nkv)], v[keys, h // (nq // nkv)], q[:, h].astype(np.float64)
        s = np.where(see, qh @ kh.T / np.sqrt(128.0), -np.inf)
        w = np.exp(s - s.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        o[:, h] = w @ vh
        bound[:, h] = u.attention_bound(qh, kh, vh, w, see, split)
    return o.reshape(M, -1), bound.reshape(M, -1)


def attention_in_parts(q, k, v, nq, length, parts, q_parts, p_parts):
    """Causal attention with q and p in that many parts and everything else exact."""
    M, nkv = q.shape[0], k.shape[1]
    see = u.visible(M, length, 0, 0)
    o = np.zeros((M, nq, 128))
    for h in range(nq):
        kh, vh = k[:length, h // (nq // nkv)], v[:length, h // (nq // nkv)]
        s = np.where(see, parts(q[:, h], q_parts) @ kh.T / np.sqrt(128.0), -np.inf)
        p = np.exp(s - s.max(-1, keepdims=True))
        o[:, h] = parts(p, p_parts) @ vh / p.sum(-1, keepdims=True)
    return o.reshape(M, -1)
