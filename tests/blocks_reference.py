"""Plain restatement, in 64 bits on the CPU, of the 8-bit caches with one scale
per (block, kv head) and of paged attention with score caps, distance biases and
document / prefix masks.  Nothing here calls the library."""
import math

import numpy as np
import torch

QMAX = {"i8": 127.0, "e4m3": 448.0}


def to_e4m3(x):
    """The e4m3 number nearest x (ties to even), at most 448 in magnitude; float64 in and out."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    _, e = np.frexp(np.where(a > 0, a, 1.0))
    unit = np.exp2(np.maximum(e - 1, -6) - 3.0)   # three mantissa bits; subnormals below 2^-6
    return np.copysign(np.minimum(np.rint(a / unit) * unit, 448.0), x)


def to_code(y, kind):
    """The number a code stands for (before the scale) for y = value / scale."""
    return np.clip(np.rint(np.asarray(y, np.float64)), -127, 127) if kind == "i8" else to_e4m3(y)


def scale_for(amax, kind):
    """amax / qmax in fp32, rounded up to three significant bits (i8) or a power of two (e4m3)."""
    t = float(np.float32(amax) / np.float32(QMAX[kind]))
    if t == 0.0:
        return np.float32(0.0)
    m, e = math.frexp(t)             # m in [1/2, 1)
    keep = 8.0 if kind == "i8" else 2.0
    up = math.ldexp(math.ceil(m * keep) / keep, e) if kind == "i8" else math.ldexp(1.0 if m > 0.5 else 0.5, e)
    return np.float32(max(up, 2.0 ** -126))


def values(codes, kind):
    """Code tensor -> float64 numbers."""
    if kind == "i8":
        return codes.cpu().numpy().astype(np.float64)
    return codes.cpu().view(torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)


def append(kc, vc, ks, vs, kind, k_new, v_new, tables, ctx, new):
    """Append in place: kc, vc float64 code values [NB, 16, H, D]; ks, vs float32 [NB, H]; k_new, v_new float64
    rows; `new` the sequences' new-token counts, rows one after another."""
    row = 0
    NB, mb = kc.shape[0], tables.shape[1]
    for s, n in enumerate(new):
        c = int(ctx[s])
        first, last = max(c - n, 0), min(c, mb * 16)
        p = first
        while c > 0 and p < last:
            a, m = p % 16, min(16 - p % 16, last - p)
            pb = int(tables[s, p // 16])
            r = row + p - (c - n)
            p += m
            if not 0 <= pb < NB:
                continue
            for codes, scale, x in ((kc, ks, k_new), (vc, vs, v_new)):
                for h in range(codes.shape[2]):
                    y = x[r:r + m, h]
                    old = np.float32(scale[pb, h]) if a else np.float32(0)
                    old = old if 0 < old < np.inf else np.float32(0)
                    s_new = max(old, scale_for(np.abs(y).max(), kind))
                    if a and s_new > old:
                        share = np.float32(old / s_new)
                        codes[pb, :a, h] = to_code(codes[pb, :a, h].astype(np.float32) * share, kind)
                    inv = np.float32(1) / s_new if s_new > 0 else np.float32(0)
                    codes[pb, a:a + m, h] = to_code(y.astype(np.float32) * inv, kind)
                    scale[pb, h] = s_new
        row += n


def stored(codes, scale, tables, s, c):
    """[c, H, D] float64: the tokens of sequence s of a cache given as code values and scales (None: plain values)."""
    t = np.asarray(tables[s, :-(-c // 16)], np.int64)
    x = codes[t]
    if scale is not None:
        x = x * scale[t].astype(np.float64)[:, None, :, None]
    return x.reshape(-1, *codes.shape[2:])[:c]


def attention(q, k, v, ctx, q_len, scale, window=0, cap=0.0, slopes=None, starts=None, prefix=None):
    """q float64 [B * q_len, H, D]; k, v lists of float64 [ctx, Hkv, D].  Returns (out, the largest magnitude that
    goes into a score that counts: sum |q||k| scale, and the bias)."""
    out = np.zeros_like(q)
    biggest = 0.0
    for s, c in enumerate(ctx):
        c = int(c)
        if c <= 0:
            continue
        g = q.shape[1] // k[s].shape[1]
        lo = max(0, c - window) if window else 0
        if starts is not None:
            lo = max(lo, min(max(int(starts[s]), 0), c))
        pre = 0 if prefix is None else min(max(int(prefix[s]), 0), c)
        at = np.arange(c)
        for j in range(q_len):
            me = c - q_len + j
            see = ((at >= lo) | (at < pre)) & (at <= me)
            if not see.any():
                continue
            for h in range(q.shape[1]):
                K, V, row = k[s][see, h // g], v[s][see, h // g], q[s * q_len + j, h]
                x = K @ row * scale
                size = np.abs(K) @ np.abs(row) * abs(scale)
                if cap:
                    x = cap * np.tanh(x / cap)
                if slopes is not None:
                    x = x + float(slopes[h]) * (at[see] - me)
                    size = size + np.abs(float(slopes[h]) * (at[see] - me))
                w = np.exp(x - x.max())
                biggest = max(biggest, float(size[w > 2.0 ** -40].max()))   # the others weigh nothing
                out[s * q_len + j, h] = w @ V / w.sum()
    return out, biggest


def tolerance(biggest, vmax, dtype=torch.float32, p_bits=22):
    """Largest error of an attention output, absolute part: a score is a sum of D <= 128 products in fp32 with a few
    roundings after it (scale, cap, bias): at most 2^-19 of the sum of the products' magnitudes; a weight is off by as
    much, relatively (times ln 2 ... 1), in numerator and denominator: twice; 2^-20 covers the hardware's 2^x and the
    fp32 sums; a weight held in the MMA's operand to p_bits bits adds 2^-p_bits.  The output type adds half a step."""
    return vmax * (2 * 2.0 ** -19 * (biggest + 1.0) + 2.0 ** -20 + 2.0 ** -p_bits), torch.finfo(dtype).eps / 2
