"""Measured cases of the grouped-query serving operators: the append to a paged cache with the
position rotation (`rope_kv_append`), attention of a few new tokens over that cache held in
e4m3 or bf16 (`attn_decode_paged`), and prefill attention with a sliding window and first
tokens that stay visible (`attn_fwd_varlen_window`).

`run` computes an operator in its plain form (elementary torch operations in 32 bits) or,
where `own` is true, makes the calls a serving loop makes.
"""
import math
import random

import torch

own = False

HEADS_Q, HEADS_KV = 32, 8  # the varlen prefill workload's heads


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # -- append: K / V of new tokens into the paged cache, q and k rotated on the way
        # one decode step of a small batch: the smallest call of a serving loop
        dict(name="append step 8 requests", op="append", batch=8, new_min=1, new_max=1, past_min=100,
             past_max=2590, hq=32, hkv=8, d=128, page=64, cache="e4m3", shape=1),
        # one decode step of 64 long requests
        dict(name="append step 64 requests", op="append", batch=64, new_min=1, new_max=1, past_min=1,
             past_max=4095, hq=32, hkv=8, d=128, page=64, cache="e4m3", shape=2),
        # a prompt batch of ragged lengths written behind short cached prefixes
        dict(name="append prompts e4m3", op="append", batch=8, new_min=512, new_max=7100, past_min=0,
             past_max=323, hq=32, hkv=8, d=128, page=64, cache="e4m3", shape=3),
        # a bf16 cache of small pages, heads of 64, odd lengths
        dict(name="append prompts bf16", op="append", batch=5, new_min=77, new_max=1601, past_min=0,
             past_max=77, hq=16, hkv=4, d=64, page=16, cache="bf16", shape=4),
        # -- attention of the newest tokens over the paged cache
        # one request: latency
        dict(name="decode 1 x 2590", op="decode", batch=1, new_min=1, new_max=1, kv_min=2590,
             kv_max=2590, hq=32, hkv=8, d=128, page=64, cache="e4m3", window=0, sinks=0, shape=5),
        # a full decode batch at the longest context
        dict(name="decode 64 x 32768", op="decode", batch=64, new_min=1, new_max=1, kv_min=32768,
             kv_max=32768, hq=32, hkv=8, d=128, page=64, cache="e4m3", window=0, sinks=0, shape=6),
        # a ragged batch with a sliding window; pages behind the window have been freed
        dict(name="decode window ragged", op="decode", batch=33, new_min=1, new_max=1, kv_min=63,
             kv_max=40000, hq=32, hkv=8, d=128, page=32, cache="e4m3", window=4096, sinks=4,
             shape=7),
        # verifying a few drafted tokens per request, bf16 cache
        dict(name="decode drafts bf16", op="decode", batch=16, new_min=1, new_max=4, kv_min=700,
             kv_max=9001, hq=32, hkv=8, d=128, page=64, cache="bf16", window=0, sinks=0, shape=8),
        # -- prefill attention with a sliding window and sinks
        # one short prompt, heads of 64
        dict(name="window prefill short", op="window", batch=1, len_min=700, len_max=700, hq=8,
             hkv=2, d=64, window=256, sinks=4, shape=9),
        # a ragged prompt batch
        dict(name="window prefill ragged", op="window", batch=4, len_min=520, len_max=4000, hq=32,
             hkv=8, d=128, window=1024, sinks=4, shape=10),
        # a long prompt
        dict(name="window prefill long", op="window", batch=1, len_min=16000, len_max=16000, hq=16,
             hkv=4, d=128, window=4096, sinks=128, shape=11),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "decode", "window"))
    c = dict(op=op, shape=rng.randrange(100, 1 << 20))
    c["hkv"] = rng.choice((1, 2, 4, 8))
    c["hq"] = c["hkv"] * rng.choice((1, 2, 4, 5, 8))
    if op == "append":
        c.update(d=rng.choice((64, 128)), page=rng.choice((16, 32, 64, 128)),
                 cache=rng.choice(("e4m3", "bf16")), batch=_log(rng, 1, 64))
        if rng.random() < 0.5:
            c.update(new_min=1, new_max=rng.choice((1, 1, 4)), past_min=0, past_max=_log(rng, 10, 5000))
        else:
            c["batch"] = min(c["batch"], 8)
            c["new_max"] = _log(rng, 30, 4000)
            c.update(new_min=max(1, c["new_max"] // 8), past_min=0, past_max=_log(rng, 2, 1000))
    elif op == "decode":
        c.update(d=rng.choice((64, 128)), page=rng.choice((16, 32, 64, 128)),
                 cache=rng.choice(("e4m3", "bf16")), batch=_log(rng, 1, 64),
                 new_min=1, new_max=rng.choice((1, 1, 1, 3, 6)))
        c["kv_max"] = min(_log(rng, 20, 60000), 1500000 // c["batch"])
        c["kv_min"] = max(1, int(c["kv_max"] * rng.choice((0.02, 0.3, 1.0))))
        c["window"], c["sinks"] = rng.choice(((0, 0), (0, 0), (1024, 4), (_log(rng, 10, 5000), 0)))
    else:
        c.update(d=rng.choice((64, 80, 128)), batch=rng.choice((1, 2, 3)),
                 len_max=_log(rng, 100, 5000), window=_log(rng, 16, 3000),
                 sinks=rng.choice((0, 1, 4, 130)))
        c["len_min"] = max(1, c["len_max"] // rng.choice((1, 4)))
    return c


def _lens(case, salt, lo, hi):
    r = random.Random(case["shape"] * 1000003 + salt)
    return [r.randint(lo, hi) for _ in range(case["batch"])]


def _shape(case):
    """The lengths a case stands for (they are the case's own, whatever the seed)."""
    if case["op"] == "append":
        return dict(new=_lens(case, 1, case["new_min"], case["new_max"]),
                    past=_lens(case, 2, case["past_min"], case["past_max"]))
    if case["op"] == "decode":
        kv = _lens(case, 1, case["kv_min"], case["kv_max"])
        new = [min(n, k) for n, k in zip(_lens(case, 2, case["new_min"], case["new_max"]), kv)]
        return dict(new=new, kv=kv)
    return dict(len=_lens(case, 1, case["len_min"], case["len_max"]))


def _visible(pos, window, sinks):
    """Keys that the token at position pos sees."""
    if window <= 0:
        return pos + 1
    lo = max(0, pos + 1 - window)
    return pos + 1 - lo + min(sinks, lo)


# ------------------------------------------------------------------------------ inputs
def _cum(lens, dev):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(dev)


def _quantize(x):
    """e4m3 codes of x [..., tokens, d] and one power-of-two scale per block [...]."""
    m, e = torch.frexp(x.abs().amax((-1, -2)))  # amax = m 2^e, m in [0.5, 1): 448 = 0.875 2^9
    s = torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875).to(e.dtype))
    return (x / s[..., None, None]).to(torch.float8_e4m3fn), s


def _pool(g, pages, case, dev):
    """A cache pool whose rows hold standard normal values (keys a little larger)."""
    hkv, ps, d = case["hkv"], case["page"], case["d"]
    out = {}
    for n, gain in (("k", 1.25), ("v", 1.0)):
        if case["cache"] == "bf16":
            out[n + "_cache"] = torch.randn((pages, hkv, ps, d), generator=g, device=dev,
                                            dtype=torch.bfloat16) * gain
            out[n + "_scale"] = None
            continue
        codes = torch.empty((pages, hkv, ps, d), dtype=torch.uint8, device=dev)
        scale = torch.empty((pages, hkv), dtype=torch.float32, device=dev)
        for a in range(0, pages, 4096):
            x = torch.randn((min(4096, pages - a), hkv, ps, d), generator=g, device=dev)
            # heads and pages of different magnitudes, so that the scales differ
            x *= gain * torch.exp2(torch.randn(x.shape[:2], generator=g, device=dev))[..., None, None] \
                if n == "v" else gain
            c, s = _quantize(x)
            codes[a:a + 4096] = c.view(torch.uint8)
            scale[a:a + 4096] = s
        out[n + "_cache"], out[n + "_scale"] = codes, scale
    return out


def _tables(g, lens, ps, dev, extra=3):
    """Shuffled pages for every request: tables [batch, max_pages] (-1 behind the last) and
    the pool's size."""
    need = [-(-n // ps) for n in lens]
    total = sum(need) + extra
    perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    width = max(need) + 1
    col = torch.arange(width, device=dev)
    n = torch.tensor(need, device=dev)
    start = n.cumsum(0) - n
    at = (start[:, None] + col).clamp(max=total - 1)
    t = torch.where(col < n[:, None], perm[at], torch.full_like(at, -1, dtype=torch.int32))
    return t.to(torch.int32).contiguous(), total


def _rope_table(max_pos, d, dev):
    a = torch.arange(max_pos, dtype=torch.float64, device=dev)[:, None] * torch.pow(
        torch.tensor(10000.0, dtype=torch.float64, device=dev),
        -torch.arange(0, d, 2, dtype=torch.float64, device=dev) / d)
    return torch.stack((a.cos(), a.sin()), -1).float().contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    sh = _shape(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]

    def rnd(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(torch.bfloat16)

    s = dict(op=case["op"], case=dict(case), scale=1.0 / math.sqrt(d))
    if case["op"] == "append":
        total = sum(sh["new"])
        ends = [a + b for a, b in zip(sh["past"], sh["new"])]
        s["page_tables"], pages = _tables(g, ends, case["page"], dev)
        s.update(_pool(g, pages, case, dev))
        # q, k and v as the projection leaves them: one packed row per token
        qkv = rnd(total, hq + 2 * hkv, d)
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:],
                 past=torch.tensor(sh["past"], dtype=torch.int32, device=dev),
                 cu=_cum(sh["new"], dev), max_new=max(sh["new"]),
                 cos_sin=_rope_table(max(ends), d, dev))
        s["q_out"] = torch.empty((total, hq, d), dtype=torch.bfloat16, device=dev)
        s["k_out"] = torch.empty((total, hkv, d), dtype=torch.bfloat16, device=dev)
    elif case["op"] == "decode":
        total, ps, w = sum(sh["new"]), case["page"], case["window"]
        s["page_tables"], pages = _tables(g, sh["kv"], ps, dev)
        s["kv_lens"] = torch.tensor(sh["kv"], dtype=torch.int32, device=dev)
        if w > 0:  # pages that no new token of the request can see any more were given back
            n = torch.tensor(sh["new"], device=dev)
            lo = (s["kv_lens"] - n + 1 - w)[:, None]
            first = torch.arange(s["page_tables"].shape[1], device=dev) * ps
            gone = (first + ps <= lo) & (first >= case["sinks"])
            s["page_tables"] = s["page_tables"].masked_fill(gone, -1).contiguous()
        s.update(_pool(g, pages, case, dev))
        s.update(q=rnd(total, hq, d), cu=_cum(sh["new"], dev), max_new=max(sh["new"]),
                 window=w, sinks=case["sinks"])
        s["one"] = case["new_max"] == 1
    else:
        total = sum(sh["len"])
        s.update(q=rnd(total, hq, d), k=rnd(total, hkv, d), v=rnd(total, hkv, d),
                 cu=_cum(sh["len"], dev), max_new=max(sh["len"]), window=case["window"],
                 sinks=case["sinks"])
    if case["op"] != "append":
        s["out"] = torch.empty((total, hq, d), dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty((total, hq), dtype=torch.float32, device=dev)
        s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=dev)
    return s


# -------------------------------------------------------------------------- plain forms
def _owner(cu, total):
    """Which sequence each token belongs to, and its place there."""
    t = torch.arange(total, device=cu.device)
    r = torch.searchsorted(cu[1:].long(), t, right=True)
    return r, t - cu[r]


def _rotate(x, cs):
    x = x.float()
    a, b = x.chunk(2, -1)
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    return torch.cat((a * c - b * s, a * s + b * c), -1)


def _append_plain(s):
    total, ps = s["q"].shape[0], s["k_cache"].shape[2]
    r, i = _owner(s["cu"], total)
    pos = s["past"][r] + i
    cs = s["cos_sin"][pos]
    q, k, v = _rotate(s["q"], cs), _rotate(s["k"], cs), s["v"].float()
    page, slot = s["page_tables"][r, pos // ps].long(), pos % ps
    for x, n in ((k, "k"), (v, "v")):
        cache, scale = s[n + "_cache"], s[n + "_scale"]
        if scale is None:
            cache[page, :, slot] = x.to(torch.bfloat16)
            continue
        # scale each (page, head) needs: the smallest power of two that keeps the new values
        # within 448; a page that is begun in this call forgets its old scale
        amax = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax")
        m, e = torch.frexp(amax)
        need = torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875).to(e.dtype))
        need = need.clamp(min=2.0 ** -60)
        touched = torch.zeros(scale.shape[0], dtype=torch.bool, device=scale.device)
        touched[page] = True
        begun = torch.zeros_like(touched)
        begun[page[slot == 0]] = True
        new = torch.where(begun[:, None], need, torch.maximum(need, scale))
        new = torch.where(touched[:, None], new, scale)
        # codes of the page's earlier tokens move to the grown scale
        codes = cache.view(torch.float8_e4m3fn)
        first = torch.full((scale.shape[0],), ps, device=scale.device)
        first = first.index_reduce(0, page, slot, "amin")
        kept = torch.arange(ps, device=scale.device)[None, :] < first[:, None]
        move = (kept & touched[:, None] & ~begun[:, None])[:, None, :, None]
        old = codes.float()
        moved = old * (scale / new)[:, :, None, None]
        codes.copy_(torch.where(move, moved, old).to(torch.float8_e4m3fn))
        y = x / new[page][..., None]
        cache[page, :, slot] = y.to(torch.float8_e4m3fn).view(torch.uint8)
        scale.copy_(new)
    return q.to(torch.bfloat16), k.to(torch.bfloat16)


def _values(s, n):
    """The cache rows of every request in 32 bits: [batch, hkv, tokens, d]."""
    pt = s["page_tables"].clamp(min=0).long()
    x = s[n + "_cache"][pt]
    if s[n + "_scale"] is not None:
        x = x.view(torch.float8_e4m3fn).float() * s[n + "_scale"][pt][..., None, None]
    b, p, h, ps, d = x.shape
    return x.float().transpose(1, 2).reshape(b, h, p * ps, d)


def _softmax_plain(q, k, v, pos, window, sinks, scale):
    """q [b, h, g * n, d] with positions pos [b, 1, g * n] over k, v [b, h, L, d]."""
    key = torch.arange(k.shape[2], device=k.device)
    see = key <= pos[..., None]
    if window > 0:
        see &= (key > pos[..., None] - window) | (key < sinks)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    x.masked_fill_(~see, -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x, v) / total.clamp(min=1e-30)
    lse = (top + total.log()).squeeze(-1)
    return out, lse


def _spread(q, r, i, b, n, hkv):
    """Packed q [tokens, hq, d] to [b, hkv, g * n, d]."""
    t, hq, d = q.shape
    x = torch.zeros((b, n, hq, d), dtype=torch.float32, device=q.device)
    x[r, i] = q.float()
    return x.view(b, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)


def _gather(x, r, i, n):
    """[b, hkv, g * n, ...] back to packed [tokens, hq, ...]."""
    b, h, gn = x.shape[:3]
    x = x.reshape(b, h, gn // n, n, *x.shape[3:])
    x = x.movedim(3, 1)
    return x.reshape(b, n, h * (gn // n), *x.shape[4:])[r, i]


def _attend_plain(s, k, v, ends):
    """ends [batch]: tokens of each sequence; its last new ones are the queries."""
    total, hq = s["q"].shape[:2]
    b, hkv = k.shape[:2]
    n = s["max_new"]
    r, i = _owner(s["cu"], total)
    count = s["cu"][1:] - s["cu"][:-1]
    pos = (ends - count)[:, None] + torch.arange(n, device=k.device)
    pos = pos.repeat(1, hq // hkv)[:, None]
    out, lse = _softmax_plain(_spread(s["q"], r, i, b, n, hkv), k, v, pos, s["window"],
                              s["sinks"], s["scale"])
    return _gather(out, r, i, n).to(torch.bfloat16), _gather(lse, r, i, n)


def _decode_plain(s):
    return _attend_plain(s, _values(s, "k"), _values(s, "v"), s["kv_lens"])


def _window_plain(s):
    total, hkv, d = s["k"].shape
    b, n = s["cu"].numel() - 1, s["max_new"]
    r, i = _owner(s["cu"], total)
    return _attend_plain(s, _spread(s["k"], r, i, b, n, hkv), _spread(s["v"], r, i, b, n, hkv),
                         s["cu"][1:] - s["cu"][:-1])


# ---------------------------------------------------------------------------- one pass
def _cache_out(s, n):
    c = s[n + "_cache"]
    return c if s[n + "_scale"] is None else c.view(torch.float8_e4m3fn)


def run(s):
    if own:
        import tiled_top_sparse_gb300 as tts
        if s["op"] == "append":
            q, k = tts.rope_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_tables"],
                                      s["past"], s["cu"], s["max_new"], k_scale=s["k_scale"],
                                      v_scale=s["v_scale"], cos_sin=s["cos_sin"], q=s["q"],
                                      q_out=s["q_out"], k_out=s["k_out"])
        elif s["op"] == "decode":
            out, lse = tts.attn_decode_paged(
                s["q"], s["k_cache"], s["v_cache"], s["page_tables"], s["kv_lens"], s["scale"],
                cu_seqlens_q=None if s["one"] else s["cu"], max_seqlen_q=s["max_new"],
                k_scale=s["k_scale"], v_scale=s["v_scale"], window=s["window"],
                sinks=s["sinks"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
        else:
            out, lse = tts.attn_fwd_varlen_window(
                s["q"], s["k"], s["v"], s["cu"], s["cu"], s["max_new"], s["max_new"], s["window"],
                s["sinks"], s["scale"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
    elif s["op"] == "append":
        q, k = _append_plain(s)
    elif s["op"] == "decode":
        out, lse = _decode_plain(s)
    else:
        out, lse = _window_plain(s)
    if s["op"] == "append":
        return dict(q=q, k=k, k_cache=_cache_out(s, "k"), v_cache=_cache_out(s, "v"),
                    k_scale=s["k_scale"], v_scale=s["v_scale"])
    return dict(out=out, lse=lse)


def work(case):
    sh, hq, hkv, d = _shape(case), case["hq"], case["hkv"], case["d"]
    row = hkv * d * (1 if case.get("cache") == "e4m3" else 2)  # one token's keys in the cache
    if case["op"] == "append":
        t = sum(sh["new"])
        # q, k, v in, rotated q and k out, cache rows out, the tokens' cos / sin rows
        distinct = len({p for a, n in zip(sh["past"], sh["new"]) for p in range(a, a + n)})
        return dict(bytes=t * (4 * hq * d + 6 * hkv * d + 2 * row) + distinct * d * 4,
                    flops=t * (hq + hkv) * d * 3)
    w, sk = case["window"], case["sinks"]
    if case["op"] == "decode":
        t, rows, pairs = sum(sh["new"]), 0, 0
        for n, L in zip(sh["new"], sh["kv"]):
            pairs += sum(_visible(L - n + i, w, sk) for i in range(n))
            lo = max(0, L - n + 1 - w) if w > 0 else 0
            rows += L - lo + min(sk, lo)
        return dict(bytes=rows * row * 2 + t * hq * (d * 4 + 4), flops=4 * d * hq * pairs)
    t = sum(sh["len"])
    pairs = sum(_visible(p, w, sk) for L in sh["len"] for p in range(L))
    return dict(bytes=t * (hq * (d * 4 + 4) + hkv * d * 4), flops=4 * d * hq * pairs)


# ------------------------------------------------------------------- the definition, 64 bits
def _exact_append(s):
    dev = s["q"].device
    ps = s["k_cache"].shape[2]
    cu, past = s["cu"].tolist(), s["past"].tolist()
    table = s["page_tables"].cpu()
    d = s["q"].shape[2]
    pos = torch.cat([torch.arange(p, p + cu[r + 1] - cu[r]) for r, p in enumerate(past)]).to(dev)
    z = torch.complex(s["cos_sin"][pos, :, 0].double(), s["cos_sin"][pos, :, 1].double())[:, None]

    def turn(x):
        y = torch.complex(x[..., :d // 2].double(), x[..., d // 2:].double()) * z
        return torch.cat((y.real, y.imag), -1)

    q, k, v = turn(s["q"]), turn(s["k"]), s["v"].double()
    out = dict(q=q, k=k)
    for x, n in ((k, "k"), (v, "v")):
        if s[n + "_scale"] is None:
            c = s[n + "_cache"].double()
            for r, p in enumerate(past):
                for a in range(p // ps, (p + cu[r + 1] - cu[r] - 1) // ps + 1):
                    lo, hi = max(p, a * ps), min(p + cu[r + 1] - cu[r], (a + 1) * ps)
                    rows = x[cu[r] + lo - p:cu[r] + hi - p].transpose(0, 1)
                    c[int(table[r, a]), :, lo - a * ps:hi - a * ps] = rows
            out[n + "_cache"], out[n + "_scale"] = c, None
            continue
        c = s[n + "_cache"].view(torch.float8_e4m3fn).double()
        sc = s[n + "_scale"].double()

        def code(y):  # to the e4m3 grid, nearest even: 3 mantissa bits, steps of 2^-9 below 2^-6
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            return (torch.round(y / step) * step).clamp(-448, 448)

        for r, p in enumerate(past):
            for a in range(p // ps, (p + cu[r + 1] - cu[r] - 1) // ps + 1):
                lo, hi = max(p, a * ps), min(p + cu[r + 1] - cu[r], (a + 1) * ps)
                rows = x[cu[r] + lo - p:cu[r] + hi - p].transpose(0, 1)
                pg, f = int(table[r, a]), lo - a * ps
                t = torch.exp2(torch.ceil(torch.log2(rows.abs().amax((1, 2)) / 448)))
                t = t.clamp(min=2.0 ** -60)
                if f > 0:
                    t = torch.maximum(t, sc[pg])
                    c[pg, :, :f] = code(c[pg, :, :f] * (sc[pg] / t)[:, None, None])
                c[pg, :, f:f + hi - lo] = code(rows / t[:, None, None])
                sc[pg] = t
        out[n + "_cache"], out[n + "_scale"] = c, sc
    return out


def _exact_rows(q, k, v, pos, key, window, sinks, scale):
    """q [n, hq, d] at positions pos [n] over k, v [hkv, keys, d] at positions key [keys]."""
    n, hq, d = q.shape
    hkv = k.shape[0]
    x = torch.einsum("nhgd,hkd->nhgk", q.double().view(n, hkv, hq // hkv, d), k) * scale
    see = key[None] <= pos[:, None]
    if window > 0:
        see &= (key[None] > pos[:, None] - window) | (key[None] < sinks)
    x = x.masked_fill(~see[:, None, None], -math.inf)
    lse = torch.logsumexp(x, -1)
    return torch.einsum("nhgk,hkd->nhgd", torch.exp(x - lse[..., None]), v).reshape(n, hq, d), \
        lse.reshape(n, hq)


def _exact_attend(s, case):
    dev, cu = s["q"].device, s["cu"].tolist()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=dev)
    w, sk = s["window"], s["sinks"]
    ends = s["kv_lens"].tolist() if s["op"] == "decode" else [b - a for a, b in zip(cu, cu[1:])]
    for r, L in enumerate(ends):
        n = cu[r + 1] - cu[r]
        for a in range(0, n, 512):
            e = min(n, a + 512)
            pos = torch.arange(L - n + a, L - n + e, device=dev)
            lo = max(0, L - n + a + 1 - w) if w > 0 else 0
            key = torch.arange(L - n + e, device=dev)
            key = key[(key >= lo) | (key < sk)] if w > 0 else key
            if s["op"] == "decode":
                ps = case["page"]
                pg, sl = s["page_tables"][r][key // ps].long(), key % ps
                kv = []
                for m in ("k", "v"):
                    x = s[m + "_cache"][pg, :, sl]
                    if s[m + "_scale"] is not None:
                        x = x.view(torch.float8_e4m3fn).double() * s[m + "_scale"][pg].double()[..., None]
                    kv.append(x.double().transpose(0, 1))
            else:
                kv = [s[m][cu[r] + key].double().transpose(0, 1) for m in ("k", "v")]
            out[cu[r] + a:cu[r] + e], lse[cu[r] + a:cu[r] + e] = _exact_rows(
                s["q"][cu[r] + a:cu[r] + e], kv[0], kv[1], pos, key, w, sk, s["scale"])
    return dict(out=out, lse=lse)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s, case)
