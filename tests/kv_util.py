"""Plain numpy forms of the paged 8-bit cache's operators (not collected)."""
import numpy as np

# values of the e4m3 codes 0 .. 126 (code 127 is NaN)
MAGNITUDES = np.array([m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                       for e in range(16) for m in range(8)][:127])


def e4m3_decode(code):
    code = np.asarray(code, np.uint8)
    mag = np.append(MAGNITUDES, np.nan)[code & 127]
    return np.where(code & 128, -mag, mag)


def e4m3_encode(x):
    """Nearest code, ties to even, saturating; NaN to 0x7F."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(MAGNITUDES, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = MAGNITUDES[hi] - a, a - MAGNITUDES[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(np.isnan(x), 127, code).astype(np.uint8)
    return code | (np.signbit(x).astype(np.uint8) << 7) * ~np.isnan(x)


def needed_scale(amax):
    e = -40
    while e < 40 and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(x, slot, cache, scale, block):
    """x [T, H, D] into codes cache [pages, H, block, D], scale [pages, H]."""
    cache, scale = cache.copy(), scale.astype(np.float64).copy()
    t = 0
    while t < len(slot):
        if slot[t] < 0:
            t += 1
            continue
        n = 1
        while t + n < len(slot) and slot[t + n] == slot[t] + n and slot[t + n] % block:
            n += 1
        page, off = divmod(int(slot[t]), block)
        for h in range(x.shape[1]):
            v = x[t:t + n, h].astype(np.float64)
            a = np.abs(v[~np.isnan(v)])
            s = needed_scale(a.max() if a.size else 0.0)
            if off and scale[page, h] >= s:
                s = scale[page, h]
            elif off:
                cache[page, h, :off] = e4m3_encode(
                    e4m3_decode(cache[page, h, :off]) * (scale[page, h] / s))
            scale[page, h] = s
            cache[page, h, off:off + n] = e4m3_encode(v / s)
        t += n
    return cache, scale


def sees(i, n, ctx, L, bits=None):
    """Which of L positions new token i of n sees."""
    p = np.arange(L)
    if bits is None:
        return p <= ctx + i
    ok = p < ctx
    for j in range(n):
        if (int(bits[j // 32]) >> (j % 32)) & 1:
            ok[ctx + j] = True
    return ok


def attend(q, codes, scales, table, kv_len, cu, block, mask=None, softmax_scale=None):
    """fp64 (out, lse, absolute), where absolute = sum w |v| / sum w, and the
    largest sum |q||k| * scale of a row (for the error of its scores)."""
    T, Hq, D = q.shape
    H = codes[0].shape[1]
    G = Hq // H
    c = D ** -0.5 if softmax_scale is None else softmax_scale
    out, mag = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, size = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for b in range(len(kv_len)):
        L, n = int(kv_len[b]), int(cu[b + 1] - cu[b])
        pages = table[b, :-(-L // block)]
        K, V = (
            (e4m3_decode(x[pages]) * s[pages].astype(np.float64)[:, :, None, None])
            .transpose(1, 0, 2, 3).reshape(H, -1, D)[:, :L] for x, s in zip(codes, scales))
        for i in range(n):
            t = int(cu[b]) + i
            ok = sees(i, n, L - n, L, None if mask is None else mask[t])
            if not ok.any():
                continue
            for g in range(Hq):
                k, v = K[g // G][ok], V[g // G][ok]
                z = (k @ q[t, g]) * c
                size[t, g] = (np.abs(k) @ np.abs(q[t, g])).max() * abs(c)
                m = z.max()
                w = np.exp(z - m)
                out[t, g] = w @ v / w.sum()
                mag[t, g] = w @ np.abs(v) / w.sum()
                lse[t, g] = m + np.log(w.sum())
    return out, lse, mag, size
