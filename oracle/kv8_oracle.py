"""fp64 oracle of the 8-bit KV cache operators: store, block attention, attention weight, eviction.

Plain numpy from the definitions (OCP E4M3: one sign, four exponent bits of bias 7, three mantissa bits, largest value
448, the all-ones pattern NaN). Shares nothing with the CUDA path.
"""
import numpy as np

MIN_EXP, MAX_EXP = -64, 120


def e4m3_values():
    """The 256 codes' values."""
    c = np.arange(256)
    s, e, m = np.where(c & 0x80, -1.0, 1.0), (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    return np.where((c & 0x7F) == 0x7F, np.nan, s * v)


def round_e4m3(x):
    """x (fp64) to the nearest E4M3 value, ties to even mantissas; beyond +-448 saturates, NaN stays."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        a = np.abs(np.where(np.isfinite(x), x, 448.0))
        e = np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -30))), -6.0)
        step = 2.0 ** (e - 3.0)
        r = np.minimum(np.rint(a / step) * step, 448.0)
        return np.where(np.isnan(x), np.nan, np.copysign(r, x))


def run_scale(x):
    """Scale of one run [rows, d]: 2^k, k the least integer with the largest finite magnitude <= 448 * 2^k."""
    a = np.abs(x[np.isfinite(x)])
    amax = a.max() if a.size else 0.0
    if amax == 0.0:
        return 2.0 ** MIN_EXP
    k = int(np.floor(np.log2(amax / 448.0))) - 1
    while amax > 448.0 * 2.0 ** k:
        k += 1
    return 2.0 ** min(max(k, MIN_EXP), MAX_EXP)


def store(x, S):
    """Values in codes [..., n, d] (not multiplied by the scale) and scales [..., ceil(n / S)] of x [..., n, d]."""
    x = np.asarray(x, dtype=np.float64)
    n = x.shape[-2]
    flat = x.reshape(-1, n, x.shape[-1])
    codes = np.empty_like(flat)
    scale = np.empty((flat.shape[0], -(-n // S)))
    for i in range(flat.shape[0]):
        for r in range(scale.shape[1]):
            part = flat[i, r * S: (r + 1) * S]
            scale[i, r] = run_scale(part)
            codes[i, r * S: (r + 1) * S] = round_e4m3(part / scale[i, r])
    return codes.reshape(x.shape), scale.reshape(*x.shape[:-2], -1)


def values(codes, scale, S):
    n = codes.shape[-2]
    return codes * np.repeat(scale, S, axis=-1)[..., :n, None]


def attention(q, k, v, lens, k_own, v_own, blk_len, scale=None):
    """q [B, Lq, Hq, d]; k, v [B, Hkv, P, d] cache values; k_own, v_own [B, Hkv, Lq, d] or None. Returns o [B, Lq, Hq,
    d], lse [B, Lq, Hq] and, for error bounds, sum p |v| (same shape as o) and the largest |score| term sum
    scale * max|q| * sum|k| of each row."""
    B, Lq, Hq, d = q.shape
    Hkv = k.shape[1]
    scale = scale or 1.0 / np.sqrt(d)
    o, oa = np.zeros(q.shape), np.zeros(q.shape)
    lse, big = np.full((B, Lq, Hq), -np.inf), np.zeros((B, Lq, Hq))
    for b in range(B):
        n = int(lens[b])
        for h in range(Hq):
            g = h // (Hq // Hkv)
            for i in range(Lq):
                ks, vs = [k[b, g, :n]], [v[b, g, :n]]
                if k_own is not None:
                    lim = min(Lq, (i // blk_len + 1) * blk_len)
                    ks.append(k_own[b, g, :lim])
                    vs.append(v_own[b, g, :lim])
                kk, vv = np.concatenate(ks), np.concatenate(vs)
                if len(kk) == 0:
                    continue
                s = kk @ q[b, i, h] * scale
                m = s.max()
                p = np.exp(s - m)
                lse[b, i, h] = m + np.log(p.sum())
                p = p / p.sum()
                o[b, i, h] = p @ vv
                oa[b, i, h] = p @ np.abs(vv)
                big[b, i, h] = scale * np.abs(q[b, i, h]).max() * np.abs(kk).sum(1).max()
    return o, lse, oa, big


def mass(q, k, lens, lse, mass_in, mass_out, decay=1.0, scale=None):
    """The accumulators [B, Hkv, cap] after the call (mass_in None: zeros; rows past a prefix as in mass_out)."""
    B, Lq, Hq, d = q.shape
    Hkv = k.shape[1]
    scale = scale or 1.0 / np.sqrt(d)
    out = np.array(mass_out, dtype=np.float64)
    for b in range(B):
        n = int(lens[b])
        for g in range(Hkv):
            t = np.zeros(n) if mass_in is None else decay * np.asarray(mass_in, dtype=np.float64)[b, g, :n]
            for h in range(g * (Hq // Hkv), (g + 1) * (Hq // Hkv)):
                for i in range(Lq):
                    if lse[b, i, h] != -np.inf:
                        t = t + np.exp(k[b, g, :n] @ q[b, i, h] * scale - lse[b, i, h])
            out[b, g, :n] = t
    return out


def select(mass_rows, n, n_keep, n_first, n_last):
    """Kept rows of one selection, increasing: mass_rows [heads, >= n] are summed."""
    key = np.asarray(mass_rows, dtype=np.float64)[:, :n].sum(0).astype(np.float32)
    key = np.where(key > 0, key, np.float32(0))          # NaN and negative weights count as 0
    must = np.zeros(n, dtype=bool)
    must[:n_first] = True
    must[max(0, n - n_last):] = True
    order = sorted(range(n), key=lambda j: (not must[j], -key[j], j))
    return np.array(sorted(order[:n_keep]), dtype=np.int64)


def evict_rows(codes, scale, rows, S):
    """Codes and scales of the kept rows of one kv head ([cap, d], [runs])."""
    old = scale[rows // S]
    out = np.empty((len(rows), codes.shape[1]))
    new = np.empty(-(-len(rows) // S))
    for r in range(len(new)):
        new[r] = old[r * S: (r + 1) * S].max()
        ratio = (old[r * S: (r + 1) * S] / new[r]) if new[r] > 0 else np.zeros(len(old[r * S: (r + 1) * S]))
        out[r * S: (r + 1) * S] = round_e4m3(codes[rows[r * S: (r + 1) * S]] * ratio[:, None])
    return out, new
