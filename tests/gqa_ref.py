"""64-bit definitions for the grouped-query cache: the append (rotation, page scales, e4m3
rounding) and attention over the cache, with the error each result may carry."""
import math

import numpy as np
import torch


def round_e4m3(y):
    """Float64 values to the nearest e4m3 value, ties to even, saturating at 448."""
    a = np.abs(y)
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return np.sign(y) * np.minimum(np.rint(a / step) * step, 448.0)


def page_scale(amax):
    """Smallest power of two s >= 2^-60 with amax <= 448 s."""
    s = 2.0 ** -60
    if amax > 448 * s:
        s = 2.0 ** math.ceil(math.log2(amax / 448.0))
        while amax > 448 * s:
            s *= 2
        while amax <= 448 * (s / 2):
            s /= 2
    return s


def rotate32(x, cs):
    """Rotate-half in fp32, every product and sum rounded on its own. x [n, heads, d] fp32,
    cs [n, d/2, 2]."""
    h = x.shape[-1] // 2
    a, b = x[..., :h].astype(np.float32), x[..., h:].astype(np.float32)
    c, s = cs[:, None, :, 0].astype(np.float32), cs[:, None, :, 1].astype(np.float32)
    return np.concatenate([a * c - b * s, a * s + b * c], -1)


def append(q, k, v, k_cache, v_cache, k_scale, v_scale, tables, past, cu, cos_sin, page_size):
    """Values of the caches after the append: caches as float64 arrays [pages, h, ps, d] of the
    stored numbers (codes for e4m3, scales fp64 or None). Rotation in fp32 (exactly the
    documented roundings), quantization exact. Returns q_rot, k_rot (fp32), the caches and
    scales."""
    f8 = k_scale is not None
    kc, vc = k_cache.copy(), v_cache.copy()
    ks = None if not f8 else k_scale.astype(np.float64).copy()
    vs = None if not f8 else v_scale.astype(np.float64).copy()
    n_tok = k.shape[0]
    pos = np.zeros(n_tok, np.int64)
    for r, p in enumerate(past):
        pos[cu[r]:cu[r + 1]] = p + np.arange(cu[r + 1] - cu[r])
    if cos_sin is not None:
        qr = None if q is None else rotate32(q, cos_sin[pos])
        kr = rotate32(k, cos_sin[pos])
    else:
        qr, kr = q, k
    for r, p in enumerate(past):
        n = int(cu[r + 1] - cu[r])
        if n == 0:
            continue
        for a in range(p // page_size, (p + n - 1) // page_size + 1):
            lo, hi = max(p, a * page_size), min(p + n, (a + 1) * page_size)
            f, t0 = lo - a * page_size, cu[r] + lo - p
            pg = int(tables[r, a])
            for x, c, sc in ((kr, kc, ks), (v, vc, vs)):
                for h in range(x.shape[1]):
                    rows = x[t0:t0 + hi - lo, h].astype(np.float64)
                    if not f8:
                        c[pg, h, f:f + hi - lo] = rows
                        continue
                    s = page_scale(np.abs(rows).max())
                    if f > 0:
                        s = max(s, sc[pg, h])
                        if s != sc[pg, h]:
                            c[pg, h, :f] = round_e4m3(c[pg, h, :f] * (sc[pg, h] / s))
                    c[pg, h, f:f + hi - lo] = round_e4m3(rows / s)
                    sc[pg, h] = s
    return qr, kr, kc, vc, ks, vs


def visible(pos, L, window, sinks):
    j = np.arange(L)
    see = j <= pos
    if window > 0:
        see &= (j > pos - window) | (j < sinks)
    return see


def attend(q, k_cache, v_cache, k_scale, v_scale, tables, kv_lens, cu, scale, window, sinks,
           w_half, bad_page=lambda pg: False):
    """out, lse in 64 bits, and how far an implementation may be from them that rounds its
    softmax weights with relative error w_half and sums in fp32."""
    T, hq, d = q.shape
    hkv, ps = k_cache.shape[1], k_cache.shape[2]
    G = hq // hkv
    out = np.zeros((T, hq, d))
    lse = np.full((T, hq), -np.inf)
    tol, tol_l = np.zeros((T, hq, d)), np.full((T, hq), 1e-6)
    for r, L in enumerate(kv_lens):
        n = int(cu[r + 1] - cu[r])
        L = int(L)
        if L <= 0 or n == 0:
            continue
        j = np.arange(L)
        lo = max(0, L - n + 1 - window) if window > 0 else 0
        need = (j >= lo) | (j < sinks)
        pg = np.where(need, tables[r, j // ps], 0)
        gone = np.array([bad_page(x) for x in pg])
        pg = np.where(gone, 0, pg)
        K = k_cache[pg, :, j % ps].astype(np.float64)  # [L, hkv, d]
        V = v_cache[pg, :, j % ps].astype(np.float64)
        if k_scale is not None:
            K = K * k_scale[pg].astype(np.float64)[:, :, None]
            V = V * v_scale[pg].astype(np.float64)[:, :, None]
        K[~need | gone] = 0
        V[~need | gone] = 0
        for i in range(n):
            see = visible(L - n + i, L, window, sinks) & ~gone
            if not see.any():
                continue
            for h in range(hq):
                kk, vv = K[see, h // G], V[see, h // G]
                x = scale * (kk @ q[cu[r] + i, h].astype(np.float64))
                m = x.max()
                p = np.exp(x - m)
                l = p.sum()
                t = cu[r] + i
                out[t, h] = p @ vv / l
                lse[t, h] = m + math.log(l)
                # scores: d products summed in fp32, then scale factors and the shift by the
                # running reference, each rounded (2^-24 of what passes through)
                size = scale * (np.abs(kk) @ np.abs(q[cu[r] + i, h].astype(np.float64))).max()
                dx = (d + 16) * 2.0 ** -24 * size + 2.0 ** -18
                pv = p @ np.abs(vv) / l
                # weights: rounding, score error in numerator and denominator, sums in fp32
                tol[t, h] = pv * (w_half * 1.01 + 2.5 * dx) + 2.0 ** -34 * np.abs(vv).sum(0) / l
                tol_l[t, h] = 2 * dx + 2.0 ** -22 * abs(lse[t, h])
    return out, lse, tol, tol_l


def codes_of(t):
    """Stored numbers of a cache tensor as float64: codes' values for e4m3, the values for bf16."""
    t = t.cpu()
    if t.dtype == torch.uint8:
        t = t.view(torch.float8_e4m3fn)
    return t.float().double().numpy()


def rope_table(max_pos, d):
    a = np.arange(max_pos, dtype=np.float64)[:, None] * 10000.0 ** (
        -np.arange(0, d, 2, dtype=np.float64) / d)
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


def attend_packed(q, k, v, cu_q, cu_k, scale, window, sinks, w_half):
    """Windowed causal attention over packed sequences in 64 bits (bottom-right aligned), with
    the bounds of attend()."""
    T, hq, d = q.shape
    G = hq // k.shape[1]
    out = np.zeros((T, hq, d))
    lse = np.full((T, hq), -np.inf)
    tol, tol_l = np.zeros((T, hq, d)), np.full((T, hq), 1e-6)
    for r in range(len(cu_q) - 1):
        n, L = int(cu_q[r + 1] - cu_q[r]), int(cu_k[r + 1] - cu_k[r])
        if n == 0 or L == 0:
            continue
        pos = np.arange(n)[:, None] + L - n
        j = np.arange(L)[None]
        see = (j <= pos) & ((j > pos - window) | (j < sinks))
        some = see.any(1)
        rows = slice(cu_q[r], cu_q[r + 1])
        for h in range(hq):
            qq = q[rows, h].astype(np.float64)
            kk = k[cu_k[r]:cu_k[r + 1], h // G].astype(np.float64)
            vv = v[cu_k[r]:cu_k[r + 1], h // G].astype(np.float64)
            x = np.where(see, scale * (qq @ kk.T), -np.inf)
            size = np.where(see, scale * (np.abs(qq) @ np.abs(kk).T), 0).max(1)
            m = np.where(some, x.max(1), 0)
            p = np.exp(x - m[:, None])
            l = np.where(some, p.sum(1), 1)
            dx = (d + 16) * 2.0 ** -24 * size + 2.0 ** -18
            out[rows, h] = p @ vv / l[:, None]
            lse[rows, h] = np.where(some, m + np.log(l), -np.inf)
            tol[rows, h] = (p @ np.abs(vv) / l[:, None]) * (w_half * 1.01 + 2.5 * dx)[:, None]
            tol_l[rows, h] = 2 * dx + 2.0 ** -22 * np.abs(np.where(some, lse[rows, h], 0))
    return out, lse, tol, tol_l
