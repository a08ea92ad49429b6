"""64-bit definitions of the drafted-tree operators: attention under the tokens' masks with the error
a result may carry, the compaction of accepted paths, and forked requests."""
import numpy as np

import gqa_ref as ref


def random_tree(rng, n, wide=3):
    """Parents of n tokens, the first the root (-1), each behind its parent."""
    return [-1] + [int(rng.integers(max(0, i - 1 - wide * 2), i)) for i in range(1, n)]


def masks_of(parents):
    """Every token's ancestors and itself, as Python ints."""
    out = []
    for i, p in enumerate(parents):
        out.append((out[p] if p >= 0 else 0) | 1 << i)
    return out


def signed(m):
    return m - (1 << 64) if m >> 63 else m


def sees(mask, n, L, window, sinks):
    """Which of L keys a token with this mask sees; its request's new tokens are the last n."""
    base = L - n
    bits = [m for m in range(n) if mask >> m & 1]
    pos = base + max(len(bits) - 1, 0)
    j = np.arange(max(L, 0))
    see = j < base
    if window > 0:
        see &= (j > pos - window) | (j < sinks)
    for m in bits:
        if base + m >= 0:
            see[base + m] = True
    return see


def attend_tree(q, k_cache, v_cache, k_scale, v_scale, tables, kv_lens, cu, masks, scale, window,
                sinks, gone=lambda page, head: False):
    """out, lse in 64 bits, and how far an implementation may be from them. Caches are the stored
    numbers in float64, masks one Python int per token. gone: a page's keys are skipped.

    Scores: d products summed in fp32, scale factors and the shift by a reference (2^-24 of what
    passes through, as in gqa_ref). e4m3 caches: q is held to 2^-17 of its row's largest value, so
    a score moves by at most scale sum_i |k_i| 2^-17 max|q|; weights are rounded to fp16, relative
    2^-11, and end at 2^-25 of the largest. bf16 caches: weights are rounded to bf16, relative 2^-8."""
    T, hq, d = q.shape
    hkv, ps = k_cache.shape[1], k_cache.shape[2]
    G = hq // hkv
    f8 = k_scale is not None
    w_half = 2.0 ** -11 if f8 else 2.0 ** -8
    out, lse = np.zeros((T, hq, d)), np.full((T, hq), -np.inf)
    tol, tol_l = np.zeros((T, hq, d)), np.full((T, hq), 1e-6)
    for r, L in enumerate(kv_lens):
        n, L = int(cu[r + 1] - cu[r]), int(L)
        if n == 0 or L <= 0:
            continue
        see_all = np.stack([sees(masks[cu[r] + i], n, L, window, sinks) for i in range(n)])
        some = see_all.any(0)
        j = np.arange(L)
        pg = np.where(some, tables[r, j // ps], 0)
        for h in range(hkv):
            skip = np.array([bool(s) and gone(int(p), h) for p, s in zip(pg, some)])
            use = some & ~skip
            at = np.where(use, pg, 0)
            K, V = k_cache[at, h, j % ps].astype(np.float64), v_cache[at, h, j % ps].astype(np.float64)
            if f8:
                K = K * k_scale[at, h].astype(np.float64)[:, None]
                V = V * v_scale[at, h].astype(np.float64)[:, None]
            K[~use] = 0
            V[~use] = 0
            Q = q[cu[r]:cu[r + 1], h * G:(h + 1) * G].astype(np.float64)  # [n, G, d]
            see = (see_all & use)[:, None, :]
            x = np.where(see, scale * (Q @ K.T), -np.inf)
            ok = see.any(-1)
            ok = np.broadcast_to(ok, x.shape[:2])
            m = np.where(ok, x.max(-1, initial=-np.inf), 0)
            p = np.exp(x - m[..., None])
            l = np.where(ok, p.sum(-1), 1)
            size = np.where(see, scale * (np.abs(Q) @ np.abs(K).T), 0).max(-1)
            dx = (d + 16) * 2.0 ** -24 * size + 2.0 ** -18
            if f8:
                dx = dx + 2.0 ** -17 * scale * np.abs(Q).max(-1) * np.abs(K).sum(-1).max()
            rows, heads = slice(cu[r], cu[r + 1]), slice(h * G, (h + 1) * G)
            out[rows, heads] = p @ V / l[..., None]
            with np.errstate(divide="ignore"):
                lse[rows, heads] = np.where(ok, m + np.log(l), -np.inf)
            tol[rows, heads] = (p @ np.abs(V) / l[..., None]) * (w_half * 1.01 + 2.5 * dx)[..., None] + \
                2.0 ** -34 * (see @ np.abs(V)) / l[..., None]
            tol_l[rows, heads] = 2 * dx + 2.0 ** -22 * np.abs(m + np.log(l))
    return out, lse, tol, tol_l


def compact(k_cache, v_cache, k_scale, v_scale, tables, past, path, path_lens):
    """Stored numbers and scales after the accepted paths were moved (float64)."""
    ps = k_cache.shape[2]
    res = []
    for c, s in ((k_cache, k_scale), (v_cache, v_scale)):
        before, c = c, c.copy()
        sb = None if s is None else s.astype(np.float64)
        s = None if s is None else sb.copy()
        for r, p in enumerate(past):
            to = {}
            for i in range(path_lens[r]):
                a, b = p + path[r][i], p + i
                if a != b:
                    to.setdefault(int(tables[r, b // ps]), []).append(
                        (b % ps, int(tables[r, a // ps]), a % ps))
            for pg, moves in to.items():
                for h in range(c.shape[1]):
                    rows = np.stack([before[a, h, t] for _, a, t in moves])
                    if s is not None:
                        rows = rows * np.array([sb[a, h] for _, a, _ in moves])[:, None]
                        fin = np.abs(rows[np.isfinite(rows)])
                        t = sb[pg, h]
                        if fin.size and fin.max() > 448 * t:
                            t = ref.page_scale(fin.max())
                            c[pg, h] = ref.round_e4m3(before[pg, h] * (sb[pg, h] / t))
                        rows = ref.round_e4m3(rows / t)
                        s[pg, h] = t
                    for (b, _, _), row in zip(moves, rows):
                        c[pg, h, b] = row
        res += [c, s]
    return res[0], res[2], res[1], res[3], [p + m for p, m in zip(past, path_lens)]


def fork(k_cache, v_cache, k_scale, v_scale, tables, kv_lens, parents, new_pages):
    ps, width = k_cache.shape[2], tables.shape[1]
    t = np.full((len(parents), width), -1, np.int64)
    caches = [c.copy() for c in (k_cache, v_cache)]
    scales = [None if s is None else s.copy() for s in (k_scale, v_scale)]
    lens = []
    for i, p in enumerate(parents):
        L = int(kv_lens[p])
        full, used = divmod(L, ps)
        lens.append(L)
        if new_pages[i] < 0:
            t[i] = tables[p]
            continue
        t[i, :full] = tables[p, :full]
        if full < width:
            t[i, full] = new_pages[i]
        if used:
            src = int(tables[p, full])
            for c in caches:
                c[new_pages[i], :, :used] = c[src, :, :used]
            for s in scales:
                if s is not None:
                    s[new_pages[i]] = s[src]
    return caches[0], caches[1], scales[0], scales[1], t, lens


def turns(cos_sin, positions, pair_axis):
    """cos / sin of every token's pairs [tokens, pairs, 2]."""
    pos = np.stack([positions[a] for a in pair_axis], 1)
    return cos_sin[pos, np.arange(len(pair_axis))]
