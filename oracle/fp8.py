"""The 8-bit (E4M3, block-scaled) path from its definitions, numpy only.

E4M3: sign, 4 exponent bits (bias 7), 3 mantissa bits, largest value 448, no
infinity.  Quantizer, per block: s = f32(max|v| / 448), at least 2^-126, 1 for
a block of zeros; code = the E4M3 value nearest to f32(v * f32(1/s)).
Products and sums are float64.
"""
import numpy as np

BLOCK = 128
E4M3_MAX = 448.0


def blocks(n):
    return -(-n // BLOCK)


def e4m3_round(v):
    """nearest E4M3 value (ties to even mantissa), saturating; float64"""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    e = np.where(a >= 2.0 ** (e + 1), e + 1, e)  # log2 that rounded down
    step = 2.0 ** (np.maximum(e, -6) - 3)
    r = np.minimum(np.round(a / step) * step, E4M3_MAX)  # np.round: ties to even
    return np.copysign(r, v)


def block_scale(amax):
    amax = np.asarray(amax, np.float32)
    s = np.maximum((amax / np.float32(E4M3_MAX)).astype(np.float32), np.float32(2.0 ** -126))
    return np.where(amax > 0, s, np.float32(1.0)).astype(np.float32)


def expand(s, n, axis):
    """one value per 128 -> one per element"""
    return np.take(np.repeat(s, BLOCK, axis=axis), np.arange(n), axis=axis)


def quant(v):
    """float32 [T, K] -> (E4M3 values float64 [T, K], scales float32 [T, K/128]), bit for bit"""
    v = np.asarray(v, np.float32)
    T, K = v.shape
    kb = blocks(K)
    pad = np.zeros((T, kb * BLOCK), np.float32)
    pad[:, :K] = np.abs(v)
    s = block_scale(pad.reshape(T, kb, BLOCK).max(-1))
    inv = (np.float32(1.0) / s).astype(np.float32)
    return e4m3_round((v * expand(inv, K, 1)).astype(np.float32)), s


def pack(W):
    """bf16 values float32 [K, D] -> (E4M3 values [D, K], scales [D/128, K/128]), bit for bit"""
    w = np.ascontiguousarray(np.asarray(W, np.float32).T)
    D, K = w.shape
    db, kb = blocks(D), blocks(K)
    pad = np.zeros((db * BLOCK, kb * BLOCK), np.float32)
    pad[:D, :K] = np.abs(w)
    s = block_scale(pad.reshape(db, BLOCK, kb, BLOCK).max((1, 3)))
    inv = (np.float32(1.0) / s).astype(np.float32)
    return e4m3_round((w * expand(expand(inv, D, 0), K, 1)).astype(np.float32)), s


def dequant_act(codes, s):
    return np.asarray(codes, np.float64) * expand(np.asarray(s, np.float64), codes.shape[1], 1)


def dequant_weight(codes, s):
    return np.asarray(codes, np.float64) * expand(expand(np.asarray(s, np.float64), codes.shape[-2], -2),
                                                  codes.shape[-1], -1)


def rms_norm(x, gamma, eps):
    x = np.asarray(x, np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(gamma, np.float64)


def silu(g):
    g = np.asarray(g, np.float64)
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, g, g * e) / (1 + e)


def route(logits, topk, renormalize=True):
    """chosen experts (equal logits by the lower index, NaN last) and their weights"""
    lg = np.asarray(logits, np.float64)
    T, E = lg.shape
    key = np.where(np.isnan(lg), -np.inf, lg)
    # NaN sorts below -inf: order by (is NaN, -logit, index)
    ids = np.stack([np.lexsort((np.arange(E), -key[t], np.isnan(lg[t])))[:topk] for t in range(T)]) if T else \
        np.zeros((0, topk), np.int64)
    p = np.zeros((T, topk))
    for t in range(T):
        mx = key[t].max()
        ex = np.where(key[t] > -np.inf, np.where(key[t] == mx, 1.0, np.exp(np.minimum(key[t] - mx, 0)
                                                                          if np.isfinite(mx) else -np.inf)), 0.0)
        chosen = ex[ids[t]]
        total = chosen.sum() if renormalize else ex.sum()
        p[t] = chosen / total if total > 0 else 0.0
    return ids, p


def moe(x, logits, w13, w2, topk, renormalize=True):
    """x [T, H]; w13 [E, 2 I, H] and w2 [E, H, I] dequantized.  Returns y, ids,
    p and a bound of a float32 evaluation's error per output:
      - x as two E4M3 terms, the block's largest scaled to [128, 256): exact, or
        off by half the spacing of the second term's smallest numbers, 2^-10
        2^-4 of the scaled value = 2^-21 of the block's largest (at least 2^-107)
      - h as three terms: 2^-12 of itself, or 2^-10 2^-8 = 2^-25 of the largest
      - float32 sums of 128 products a block and then over blocks and terms"""
    x = np.asarray(x, np.float64)
    T, H = x.shape
    inner = w2.shape[-1]
    ids, p = route(logits, topk, renormalize)
    y = np.zeros((T, H))
    bound = np.zeros((T, H))

    def block_max(v):
        pad = np.zeros(blocks(v.size) * BLOCK)
        pad[:v.size] = np.abs(v)
        return expand(np.maximum(pad.reshape(-1, BLOCK).max(-1), 2.0 ** -107), v.size, 0)

    for t in range(T):
        dx = 2.0 ** -21 * block_max(x[t])
        for j in range(topk):
            e = ids[t, j]
            gu = w13[e] @ x[t]
            a13, a2 = np.abs(w13[e]), np.abs(w2[e])
            g, u = gu[:inner], gu[inner:]
            h = silu(g) * u
            d = (2 * 128 + blocks(H) + 16) * 2.0 ** -23 * (a13 @ np.abs(x[t])) + a13 @ dx
            dh = 1.1 * np.abs(u) * d[:inner] + np.abs(silu(g)) * d[inner:] + 2.0 ** -16 * np.abs(h)
            dh = dh + 2.0 ** -12 * np.abs(h) + 2.0 ** -25 * block_max(h)
            y[t] += p[t, j] * (w2[e] @ h)
            bound[t] += p[t, j] * (a2 @ dh + (3 * 128 + blocks(inner) + topk + 16) * 2.0 ** -23 * (a2 @ np.abs(h)))
    return y, ids, p, bound
