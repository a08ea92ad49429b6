"""Measured cases of the operators for drafted trees, several position axes and moved cache rows:
attention of a tree of new tokens over the paged grouped-query cache (`attn_decode_tree`), the
append with explicit positions on one or several axes (`rope_kv_append_axes`), the accepted path of
a tree moved together in the cache (`kv_compact`), requests forked with a copy of their last page
(`kv_fork`), and the vision projection with positions on several axes (`qkv_rope_axes`).

`run` computes an operator in its plain form (elementary torch operations in 32 bits) or,
where `own` is true, makes the calls a serving loop makes.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # -- attention of drafted trees over the paged cache
        # one request, a small tree: latency
        dict(name="tree 1 x 2590", op="tree", batch=1, new_min=16, new_max=16, kv_min=2590,
             kv_max=2590, hq=32, hkv=8, d=128, page=64, cache="e4m3", window=0, sinks=0, wide=3,
             shape=1),
        # a batch verifying large trees: 200 to 256 q rows for each KV head
        dict(name="tree 16 large trees e4m3", op="tree", batch=16, new_min=50, new_max=64,
             kv_min=4000, kv_max=9001, hq=32, hkv=8, d=128, page=64, cache="e4m3", window=0,
             sinks=0, wide=4, shape=2),
        # the largest: long contexts in bf16, trees of a dozen tokens
        dict(name="tree 32 x 32768 bf16", op="tree", batch=32, new_min=8, new_max=16,
             kv_min=32768, kv_max=32768, hq=32, hkv=8, d=128, page=128, cache="bf16", window=0,
             sinks=0, wide=2, shape=3),
        # ragged lengths, a sliding window whose pages have been freed, heads of 64
        dict(name="tree window ragged", op="tree", batch=33, new_min=1, new_max=31, kv_min=63,
             kv_max=40000, hq=20, hkv=4, d=64, page=32, cache="e4m3", window=4096, sinks=4, wide=3,
             shape=4),
        # -- append with explicit positions
        # drafted trees: a token's position is its depth behind the cached ones
        dict(name="append trees", op="append", batch=16, new_min=25, new_max=64, past_min=100,
             past_max=4000, hq=32, hkv=8, d=128, page=64, cache="bf16", axes=1, mix=0, shape=5),
        # prompts with images and video: positions in time, height and width
        dict(name="append image prompts", op="append", batch=8, new_min=512, new_max=7100,
             past_min=0, past_max=323, hq=32, hkv=8, d=128, page=64, cache="e4m3", axes=3, mix=0,
             shape=6),
        # -- the accepted path of each request's tree moved together
        # the smallest step of a serving loop
        dict(name="compact 8 requests", op="compact", batch=8, new_min=16, new_max=32, keep_max=6,
             past_min=100, past_max=2590, hkv=8, d=128, page=64, cache="e4m3", shape=7),
        # a large batch
        dict(name="compact 256 requests", op="compact", batch=256, new_min=40, new_max=64,
             keep_max=14, past_min=1, past_max=1500, hkv=8, d=128, page=32, cache="bf16", shape=8),
        # -- requests forked
        # one prompt answered by four samples
        dict(name="fork 4 samples", op="fork", batch=1, children=4, kv_min=2590, kv_max=2590,
             hkv=8, d=128, page=64, cache="e4m3", shape=9),
        # beams of a large batch, long tables
        dict(name="fork 512 beams", op="fork", batch=64, children=512, kv_min=5000, kv_max=32768,
             hkv=8, d=128, page=64, cache="bf16", shape=10),
        # -- vision projection with row and column positions
        # a small image
        dict(name="vision 333 patches", op="vision", tokens=333, grid=37, frames=1, hidden=512,
             heads=8, d=64, axes=2, shape=11),
        # the vision workload's image (111 x 77 patches)
        dict(name="vision 8547 patches", op="vision", tokens=8547, grid=77, frames=1, hidden=1280,
             heads=16, d=80, axes=2, shape=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("tree", "tree", "append", "append", "compact", "fork", "vision"))
    c = dict(op=op, shape=rng.randrange(100, 1 << 20))
    if op == "vision":
        d = rng.choice((64, 80, 128))
        c.update(d=d, heads=rng.choice((12, 24) if d == 80 else (4, 8, 20)), frames=rng.choice((1, 1, 4)))
        c.update(grid=rng.randint(5, 90), tokens=_log(rng, 100, 8000), hidden=8 * rng.randint(16, 160))
        c["axes"] = 3 if c["frames"] > 1 else 2
        return c
    c.update(hkv=rng.choice((1, 2, 4, 8)), d=rng.choice((64, 128)),
             page=rng.choice((16, 32, 64, 128)), cache=rng.choice(("e4m3", "bf16")))
    c["hq"] = c["hkv"] * rng.choice((1, 2, 4, 5, 8))
    if op == "tree":
        c.update(batch=_log(rng, 1, 64), new_max=_log(rng, 2, 64), wide=rng.choice((1, 2, 4, 9)))
        c["new_min"] = rng.choice((1, c["new_max"]))
        most = 1000000 * min(1.0, 384 / (c["hq"] * c["new_max"]))  # keys of all requests
        c["kv_max"] = max(c["new_max"], min(_log(rng, 70, 60000), int(most / c["batch"])))
        c["kv_min"] = max(c["new_max"], int(c["kv_max"] * rng.choice((0.02, 0.3, 1.0))))
        c["window"], c["sinks"] = rng.choice(((0, 0), (0, 0), (1024, 4), (_log(rng, 64, 5000), 0)))
    elif op == "append":
        c.update(axes=rng.choice((1, 2, 3, 3, 4)), mix=rng.choice((0, 1)))
        if rng.random() < 0.5:
            c.update(batch=_log(rng, 1, 64), new_min=1, new_max=rng.choice((1, 4, 20, 64)),
                     past_min=0, past_max=_log(rng, 10, 5000))
        else:
            c.update(batch=_log(rng, 1, 8), new_max=_log(rng, 30, 4000), past_min=0,
                     past_max=_log(rng, 2, 1000))
            c["new_min"] = max(1, c["new_max"] // 8)
    elif op == "compact":
        c.update(batch=_log(rng, 1, 256), new_max=_log(rng, 4, 64), past_min=0,
                 past_max=_log(rng, 2, 1500))
        c.update(new_min=2, keep_max=max(1, c["new_max"] // rng.choice((2, 4))))
    else:
        c.update(batch=_log(rng, 1, 64), children=_log(rng, 1, 400), kv_min=1,
                 kv_max=_log(rng, 20, 10000))
    return c


def _lens(case, salt, lo, hi):
    r = random.Random(case["shape"] * 1000003 + salt)
    return [r.randint(lo, hi) for _ in range(case["batch"])]


def _tree(r, n, wide):
    """Parents of n nodes (the first is the root): each hangs at one of the last few before it."""
    return [-1] + [r.randint(max(0, i - 1 - wide * 3), i - 1) // max(1, wide // 2) for i in range(1, n)]


def _shape(case):
    """What a case stands for whatever the seed: lengths, trees, accepted paths, parents."""
    r = random.Random(case["shape"] * 7919 + 5)
    op = case["op"]
    if op == "tree":
        kv = _lens(case, 1, case["kv_min"], case["kv_max"])
        new = _lens(case, 2, case["new_min"], case["new_max"])
        return dict(kv=kv, new=new, parents=[_tree(r, n, case["wide"]) for n in new])
    if op == "append":
        new = _lens(case, 1, case["new_min"], case["new_max"])
        return dict(new=new, past=_lens(case, 2, case["past_min"], case["past_max"]),
                    parents=[_tree(r, n, 3) for n in new] if case["axes"] == 1 else None)
    if op == "compact":
        new, path = _lens(case, 1, case["new_min"], case["new_max"]), []
        for n in new:
            # the root, then accepted tokens of ever deeper levels, which lie behind the places
            # that the path is moved to
            m = r.randint(1, min(case["keep_max"], (n + 1) // 2))
            path.append([0] + sorted(r.sample(range(m, n), min(m - 1, n - m))))
        return dict(new=new, past=_lens(case, 2, case["past_min"], case["past_max"]), path=path)
    if op == "fork":
        kv = _lens(case, 1, case["kv_min"], case["kv_max"])
        return dict(kv=kv, parent=[r.randrange(case["batch"]) for _ in range(case["children"])])
    return dict()


def _masks(parents):
    """The ancestors' bits of every node, its own among them."""
    out = []
    for i, p in enumerate(parents):
        out.append((out[p] if p >= 0 else 0) | 1 << i)
    return out


def _depths(parents):
    out = []
    for p in parents:
        out.append(out[p] + 1 if p >= 0 else 0)
    return out


def _signed(m):
    return m - (1 << 64) if m >> 63 else m


# ------------------------------------------------------------------------------ inputs
def _cum(lens, dev):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(dev)


def _int(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _scale_for(amax):
    """The smallest power of two s >= 2^-60 with amax <= 448 s."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1): 448 = 0.875 2^9
    return torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875).to(e.dtype)).clamp(min=2.0 ** -60)


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
            s = _scale_for(x.abs().amax((-1, -2)))
            codes[a:a + 4096] = (x / s[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            scale[a:a + 4096] = s
        out[n + "_cache"], out[n + "_scale"] = codes, scale
    return out


def _tables(g, lens, ps, dev, extra=3):
    """Shuffled pages for every request: tables [batch, max_pages] (-1 behind the last), the
    pool's size and `extra` pages that no request has."""
    need = [-(-n // ps) for n in lens]
    total = sum(need) + extra
    perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    width = max(need) + 1
    col = torch.arange(width, device=dev)
    n = torch.tensor(need, device=dev)
    at = ((n.cumsum(0) - n)[:, None] + col).clamp(max=total - 1)
    t = torch.where(col < n[:, None], perm[at], torch.full_like(at, -1, dtype=torch.int32))
    return t.to(torch.int32).contiguous(), total, perm[total - extra:].contiguous()


def _rope_table(max_pos, d, dev):
    a = torch.arange(max_pos, dtype=torch.float64, device=dev)[:, None] * torch.pow(
        torch.tensor(10000.0, dtype=torch.float64, device=dev),
        -torch.arange(0, d, 2, dtype=torch.float64, device=dev) / d)
    return torch.stack((a.cos(), a.sin()), -1).float().contiguous()


def _pair_axis(pairs, axes, mix):
    """The axis of every rotation pair: consecutive sections (the first the smallest), or the
    axes in turn."""
    if mix:
        return bytes(j % axes for j in range(pairs))
    first = pairs if axes == 1 else pairs // (axes + 1)
    rest = pairs - first
    return bytes([0] * first) + bytes(1 + i * (axes - 1) // rest for i in range(rest))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    sh, op, d = _shape(case), case["op"], case["d"]

    def rnd(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(torch.bfloat16)

    s = dict(op=op, case=dict(case))
    if op == "vision":
        n, H, axes = case["tokens"], case["heads"], case["axes"]
        t = torch.arange(n, device=dev)
        per = -(-n // case["frames"])
        place = (t // per, t % per // case["grid"], t % per % case["grid"])[3 - axes:]
        s["positions"] = torch.stack(place).to(torch.int32).contiguous()
        # every axis has its own run of frequencies over its part of the head
        s["pair_axis"] = bytes(j * axes // (d // 2) for j in range(d // 2))
        sizes = [s["pair_axis"].count(a) for a in range(axes)]
        s["cos_sin"] = torch.cat([_rope_table(8192, 2 * m, dev) for m in sizes], 1).contiguous()
        s["x"] = rnd(n, case["hidden"])
        s["w"] = (torch.randn((3 * H * d, case["hidden"]), generator=g, device=dev)
                  / math.sqrt(case["hidden"])).to(torch.bfloat16)
        s["bias"] = 0.1 * torch.randn(3 * H * d, generator=g, device=dev)
        for m in ("q", "k", "v"):
            s[m] = torch.empty((n, H, d), dtype=torch.bfloat16, device=dev)
        return s
    hkv, ps = case["hkv"], case["page"]
    if op == "tree":
        hq, total, w = case["hq"], sum(sh["new"]), case["window"]
        s["page_tables"], pages, _ = _tables(g, sh["kv"], ps, dev)
        s["kv_lens"] = _int(sh["kv"], dev)
        if w > 0:  # pages that no new token of the request can see any more were given back
            n = torch.tensor(sh["new"], device=dev)
            lo = (s["kv_lens"] - n + 1 - w)[:, None]
            first = torch.arange(s["page_tables"].shape[1], device=dev) * ps
            gone = (first + ps <= lo) & (first >= case["sinks"])
            s["page_tables"] = s["page_tables"].masked_fill(gone, -1).contiguous()
        s.update(_pool(g, pages, case, dev))
        s["mask"] = torch.tensor([_signed(m) for p in sh["parents"] for m in _masks(p)],
                                 dtype=torch.int64, device=dev)
        s.update(q=rnd(total, hq, d), cu=_cum(sh["new"], dev), max_new=max(sh["new"]), window=w,
                 sinks=case["sinks"], scale=1.0 / math.sqrt(d))
        s["out"] = torch.empty((total, hq, d), dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty((total, hq), dtype=torch.float32, device=dev)
        s["workspace"] = torch.empty(256 << 20, dtype=torch.uint8, device=dev)
    elif op == "append":
        hq, total, axes = case["hq"], sum(sh["new"]), case["axes"]
        ends = [a + b for a, b in zip(sh["past"], sh["new"])]
        s["page_tables"], pages, _ = _tables(g, ends, ps, dev)
        s.update(_pool(g, pages, case, dev))
        qkv = rnd(total, hq + 2 * hkv, d)  # as the projection leaves them, a packed row per token
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:],
                 past=_int(sh["past"], dev), cu=_cum(sh["new"], dev), max_new=max(sh["new"]))
        if axes == 1:  # the depth in the tree, behind the cached tokens
            at = [p + x for p, t in zip(sh["past"], sh["parents"]) for x in _depths(t)]
            s["positions"] = _int([at], dev)
        else:  # text and images in turn: patches of a grid, all axes alike in between
            i = torch.cat([torch.arange(n) for n in sh["new"]]).to(dev)
            base = torch.repeat_interleave(s["past"].long(), torch.tensor(sh["new"], device=dev))
            side = torch.tensor([1, 23, 31, 17][:axes], device=dev)[:, None]
            image = (i // 300) % 2 == 1
            s["positions"] = torch.where(image, base + i // 300 * 40 + i % side, base + i).to(
                torch.int32).contiguous()
        s["pair_axis"] = _pair_axis(d // 2, axes, case["mix"])
        s["cos_sin"] = _rope_table(max(ends) + 8192, d, dev)
        s["q_out"] = torch.empty((total, hq, d), dtype=torch.bfloat16, device=dev)
        s["k_out"] = torch.empty((total, hkv, d), dtype=torch.bfloat16, device=dev)
    elif op == "compact":
        ends = [a + b for a, b in zip(sh["past"], sh["new"])]
        s["page_tables"], pages, _ = _tables(g, ends, ps, dev)
        s.update(_pool(g, pages, case, dev))
        width = max(sh["new"])
        s["path"] = _int([p + [-1] * (width - len(p)) for p in sh["path"]], dev)
        s["path_lens"] = _int([len(p) for p in sh["path"]], dev)
        s["past"] = _int(sh["past"], dev)
        s["lens"] = torch.empty(case["batch"], dtype=torch.int32, device=dev)
    else:
        n = case["children"]
        s["page_tables"], pages, s["new_pages"] = _tables(g, sh["kv"], ps, dev, extra=n)
        s.update(_pool(g, pages, case, dev))
        s["kv_lens"], s["parent"] = _int(sh["kv"], dev), _int(sh["parent"], dev)
        s["tables_out"] = torch.empty((n, s["page_tables"].shape[1]), dtype=torch.int32, device=dev)
        s["lens_out"] = torch.empty(n, dtype=torch.int32, device=dev)
    return s


# -------------------------------------------------------------------------- plain forms
def _owner(cu, total):
    """Which sequence each token belongs to, and its place there."""
    t = torch.arange(total, device=cu.device)
    r = torch.searchsorted(cu[1:].long(), t, right=True)
    return r, t - cu[r]


def _axis_index(s, dev):
    return torch.tensor(list(s["pair_axis"]), device=dev)


def _angles(s):
    """cos / sin of every token's pairs [tokens, d/2, 2]: the pair's axis chooses the position."""
    pairs = s["cos_sin"].shape[1]
    pos = s["positions"].long()[_axis_index(s, s["positions"].device)].t()
    return s["cos_sin"][pos, torch.arange(pairs, device=pos.device)]


def _rotate(x, cs):
    x = x.float()
    a, b = x.chunk(2, -1)
    c, sn = cs[:, None, :, 0], cs[:, None, :, 1]
    return torch.cat((a * c - b * sn, a * sn + b * c), -1)


def _append_plain(s):
    total, ps = s["q"].shape[0], s["k_cache"].shape[2]
    r, i = _owner(s["cu"], total)
    slot_at = s["past"][r] + i
    cs = _angles(s)
    q, k, v = _rotate(s["q"], cs), _rotate(s["k"], cs), s["v"].float()
    page, slot = s["page_tables"][r, slot_at // ps].long(), slot_at % ps
    for x, n in ((k, "k"), (v, "v")):
        cache, scale = s[n + "_cache"], s[n + "_scale"]
        if scale is None:
            cache[page, :, slot] = x.to(torch.bfloat16)
            continue
        # scale each (page, head) needs; a page that is begun in this call forgets its old one
        need = _scale_for(torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax"))
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
        codes.copy_(torch.where(move, old * (scale / new)[:, :, None, None], old).to(
            torch.float8_e4m3fn))
        cache[page, :, slot] = (x / new[page][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
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


def _tree_plain(s):
    """q rows spread to [batch, hkv, group * n, d] against every key of the request."""
    total, hq, d = s["q"].shape
    k, v = _values(s, "k"), _values(s, "v")
    b, hkv, keys, _ = k.shape
    n, dev = s["max_new"], k.device
    r, i = _owner(s["cu"], total)
    count = (s["cu"][1:] - s["cu"][:-1]).long()
    base = s["kv_lens"].long() - count
    q = torch.zeros((b, n, hq, d), dtype=torch.float32, device=dev)
    q[r, i] = s["q"].float()
    q = q.view(b, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    mask = torch.zeros((b, n), dtype=torch.int64, device=dev)
    mask[r, i] = s["mask"]
    key = torch.arange(keys, device=dev)
    bits = (mask[:, :, None] >> torch.arange(64, device=dev)) & 1
    bits = bits * (torch.arange(64, device=dev) < count[:, None])[:, None]
    see = key < base[:, None, None]
    if s["window"] > 0:
        pos = base[:, None] + (bits.sum(-1) - 1).clamp(min=0)
        see = see & ((key > pos[..., None] - s["window"]) | (key < s["sinks"]))
    m = key - base[:, None]  # which new token a key is
    own_bit = torch.gather(bits, 2, m.clamp(0, 63)[:, None].expand(b, n, keys)) == 1
    see = see | (own_bit & ((m >= 0) & (m < count[:, None]))[:, None])
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    x = x.view(b, hkv, -1, n, keys).masked_fill_(~see[:, None, None], -math.inf).view(b, hkv, -1, keys)
    top = x.amax(-1, keepdim=True)
    x.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    sums = x.sum(-1, keepdim=True)
    out = torch.matmul(x, v) / sums.clamp(min=1e-30)
    lse = (top + sums.log()).squeeze(-1)
    back = lambda y: y.reshape(b, hkv, hq // hkv, n, *y.shape[3:]).movedim(3, 1).reshape(  # noqa: E731
        b, n, hq, *y.shape[3:])[r, i]
    return back(out).to(torch.bfloat16), back(lse)


def _compact_plain(s):
    ps, width = s["k_cache"].shape[2], s["path"].shape[1]
    past, m = s["past"].long(), s["path_lens"].long()
    i = torch.arange(width, device=past.device)
    moved = (i < m[:, None]) & (s["path"] != i)
    r, i = moved.nonzero(as_tuple=True)
    src, dst = past[r] + s["path"][r, i], past[r] + i
    ps_, pd = s["page_tables"][r, src // ps].long(), s["page_tables"][r, dst // ps].long()
    ss, sd = src % ps, dst % ps
    for n in ("k", "v"):
        cache, scale = s[n + "_cache"], s[n + "_scale"]
        rows = cache[ps_, :, ss]
        if scale is None:
            cache[pd, :, sd] = rows
            continue
        x = rows.view(torch.float8_e4m3fn).float() * scale[ps_][..., None]
        need = torch.zeros_like(scale).index_reduce_(0, pd, x.abs().amax(-1), "amax")
        new = torch.where(need > 448 * scale, _scale_for(need), scale)
        codes = cache.view(torch.float8_e4m3fn)  # a page whose scale grows: all of its codes
        grown = (new > scale).any(1).nonzero().squeeze(1)
        codes[grown] = (codes[grown].float() * (scale / new)[grown][..., None, None]).to(
            torch.float8_e4m3fn)
        cache[pd, :, sd] = (x / new[pd][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scale.copy_(new)
    return (past + m).to(torch.int32)


def _fork_plain(s):
    ps = s["k_cache"].shape[2]
    parent = s["parent"].long()
    lens = s["kv_lens"][parent].long()
    full, used = lens // ps, lens % ps
    col = torch.arange(s["page_tables"].shape[1], device=lens.device)
    old = s["page_tables"][parent]
    t = torch.where(col < full[:, None], old, torch.full_like(old, -1))
    t = torch.where(col == full[:, None], s["new_pages"][:, None], t)
    at = full.clamp(max=t.shape[1] - 1)
    src = torch.gather(old, 1, at[:, None]).squeeze(1).clamp(min=0).long()
    dst = s["new_pages"].long()
    kept = (torch.arange(ps, device=lens.device) < used[:, None])[:, None, :, None]
    for n in ("k", "v"):
        cache, scale = s[n + "_cache"], s[n + "_scale"]
        cache[dst] = torch.where(kept, cache[src], cache[dst])
        if scale is not None:
            scale[dst] = torch.where((used > 0)[:, None], scale[src], scale[dst])
    return t, lens.to(torch.int32)


def _vision_plain(s):
    n, H, d = s["q"].shape
    y = (s["x"].float() @ s["w"].float().t() + s["bias"]).view(n, 3, H, d)
    cs = _angles(s)
    return tuple(t.to(torch.bfloat16) for t in (_rotate(y[:, 0], cs), _rotate(y[:, 1], cs), y[:, 2]))


# ---------------------------------------------------------------------------- one pass
def _caches(s):
    out = {}
    for n in ("k", "v"):
        c = s[n + "_cache"]
        out[n + "_cache"] = c if s[n + "_scale"] is None else c.view(torch.float8_e4m3fn)
        out[n + "_scale"] = s[n + "_scale"]
    return out


def run(s):
    op = s["op"]
    if own:
        import tiled_top_sparse_gb300 as tts
        if op == "tree":
            out, lse = tts.attn_decode_tree(
                s["q"], s["k_cache"], s["v_cache"], s["page_tables"], s["kv_lens"], s["mask"],
                s["scale"], s["cu"], s["max_new"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                window=s["window"], sinks=s["sinks"], out=s["out"], lse=s["lse"],
                workspace=s["workspace"])
        elif op == "append":
            q, k = tts.rope_kv_append_axes(
                s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_tables"], s["past"], s["cu"],
                s["max_new"], s["positions"], s["pair_axis"], s["cos_sin"], k_scale=s["k_scale"],
                v_scale=s["v_scale"], q=s["q"], q_out=s["q_out"], k_out=s["k_out"])
        elif op == "compact":
            lens = tts.kv_compact(s["k_cache"], s["v_cache"], s["page_tables"], s["past"],
                                  s["path"], s["path_lens"], k_scale=s["k_scale"],
                                  v_scale=s["v_scale"], kv_lens=s["lens"])
        elif op == "fork":
            tables, lens = tts.kv_fork(s["k_cache"], s["v_cache"], s["page_tables"], s["kv_lens"],
                                       s["parent"], s["new_pages"], k_scale=s["k_scale"],
                                       v_scale=s["v_scale"], tables_out=s["tables_out"],
                                       lens_out=s["lens_out"])
        else:
            q, k, v = tts.qkv_rope_axes(s["x"], s["w"], s["bias"], s["positions"], s["pair_axis"],
                                        s["cos_sin"], s["q"].shape[1], q=s["q"], k=s["k"],
                                        v=s["v"])
    elif op == "tree":
        out, lse = _tree_plain(s)
    elif op == "append":
        q, k = _append_plain(s)
    elif op == "compact":
        lens = _compact_plain(s)
    elif op == "fork":
        tables, lens = _fork_plain(s)
    else:
        q, k, v = _vision_plain(s)
    if op == "tree":
        return dict(out=out, lse=lse)
    if op == "append":
        return dict(q=q, k=k, **_caches(s))
    if op == "compact":
        return dict(lens=lens, **_caches(s))
    if op == "fork":
        return dict(tables=tables, lens=lens, **_caches(s))
    return dict(q=q, k=k, v=v)


def work(case):
    sh, d, op = _shape(case), case["d"], case["op"]
    if op == "vision":
        n, hid, H = case["tokens"], case["hidden"], case["heads"]
        return dict(bytes=2 * n * hid + 6 * H * d * hid + 6 * n * H * d + 12 * H * d
                    + 4 * n * case["axes"], flops=2 * n * hid * 3 * H * d)
    hkv = case["hkv"]
    row = hkv * d * (1 if case["cache"] == "e4m3" else 2)  # one token's keys in the cache
    if op == "append":
        hq, t = case["hq"], sum(sh["new"])
        # q, k, v in, rotated q and k out, cache rows out, positions; the table's rows are few
        return dict(bytes=t * (4 * hq * d + 6 * hkv * d + 2 * row + 4 * case["axes"]),
                    flops=t * (hq + hkv) * d * 3)
    if op == "tree":
        hq, w, sk, t = case["hq"], case["window"], case["sinks"], sum(sh["new"])
        rows = pairs = 0
        for n, L, par in zip(sh["new"], sh["kv"], sh["parents"]):
            for m in _masks(par):
                c = m.bit_count()
                lo = max(0, L - n + c - w) if w > 0 else 0
                pairs += c + max(0, L - n - lo) + min(sk, lo, L - n)
            lo = max(0, L - n + 1 - w) if w > 0 else 0
            rows += L - lo + min(sk, lo)
        return dict(bytes=rows * row * 2 + t * (hq * (d * 4 + 4) + 8), flops=4 * d * hq * pairs)
    if op == "compact":
        moved = sum(1 for p in sh["path"] for i, x in enumerate(p) if x != i)
        return dict(bytes=moved * row * 4 + 8 * case["batch"] + 4 * sum(map(len, sh["path"])), flops=0)
    ps = case["page"]
    pages = sum(sh["kv"][p] // ps + 1 for p in sh["parent"])
    distinct = sum(sh["kv"][p] % ps for p in set(sh["parent"]))
    return dict(bytes=2 * row * (distinct + sum(sh["kv"][p] % ps for p in sh["parent"])) + 8 * pages,
                flops=0)


# ------------------------------------------------------------------- the definition, 64 bits
def _code(y):
    """To the e4m3 grid, nearest even: 3 mantissa bits, steps of 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def _need(amax):
    return torch.exp2(torch.ceil(torch.log2(amax / 448))).clamp(min=2.0 ** -60)


def _turn(x, z):
    h = x.shape[-1] // 2
    y = torch.complex(x[..., :h].double(), x[..., h:].double()) * z[:, None]
    return torch.cat((y.real, y.imag), -1)


def _exact_turns(s):
    """The rotation of every token's pairs as complex numbers, pair by pair."""
    out = []
    for j, a in enumerate(s["pair_axis"]):
        c = s["cos_sin"][s["positions"][a].long(), j].double()
        out.append(torch.complex(c[:, 0], c[:, 1]))
    return torch.stack(out, 1)


def _stored(s, n):
    c = s[n + "_cache"]
    if s[n + "_scale"] is None:
        return c.double(), None
    return c.view(torch.float8_e4m3fn).double(), s[n + "_scale"].double()


def _exact_append(s):
    ps = s["k_cache"].shape[2]
    cu, past, table = s["cu"].tolist(), s["past"].tolist(), s["page_tables"].cpu()
    z = _exact_turns(s)
    q, k, v = _turn(s["q"], z), _turn(s["k"], z), s["v"].double()
    out = dict(q=q, k=k)
    for x, n in ((k, "k"), (v, "v")):
        c, sc = _stored(s, n)
        for r, p in enumerate(past):
            e = p + cu[r + 1] - cu[r]
            for a in range(p // ps, (e - 1) // ps + 1):
                lo, hi = max(p, a * ps), min(e, (a + 1) * ps)
                rows = x[cu[r] + lo - p:cu[r] + hi - p].transpose(0, 1)
                pg, f = int(table[r, a]), lo - a * ps
                if sc is None:
                    c[pg, :, f:f + hi - lo] = rows
                    continue
                t = _need(rows.abs().amax((1, 2)))
                if f > 0:
                    t = torch.maximum(t, sc[pg])
                    c[pg, :, :f] = _code(c[pg, :, :f] * (sc[pg] / t)[:, None, None])
                c[pg, :, f:f + hi - lo] = _code(rows / t[:, None, None])
                sc[pg] = t
        out[n + "_cache"], out[n + "_scale"] = c, sc
    return out


def _exact_tree(s, case):
    dev, cu, w, sk = s["q"].device, s["cu"].tolist(), s["window"], s["sinks"]
    hq, hkv, ps, d = case["hq"], case["hkv"], case["page"], case["d"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=dev)
    for r, L in enumerate(s["kv_lens"].tolist()):
        a, e = cu[r], cu[r + 1]
        n = e - a
        base = L - n
        masks = [m & ((1 << n) - 1) for m in s["mask"][a:e].tolist()]
        lo = max(0, base + 1 - w) if w > 0 else 0
        key = torch.arange(L, device=dev)
        key = key[(key >= lo) | (key < sk)]
        pg, sl = s["page_tables"][r][key // ps].long(), key % ps
        kv = []
        for m in ("k", "v"):
            x = s[m + "_cache"][pg, :, sl]
            if s[m + "_scale"] is not None:
                x = x.view(torch.float8_e4m3fn).double() * s[m + "_scale"][pg].double()[..., None]
            kv.append(x.double().transpose(0, 1))
        see = torch.zeros((n, key.numel()), dtype=torch.bool, device=dev)
        for i, m in enumerate(masks):
            pos = base + max(m.bit_count() - 1, 0)
            see[i] = (key < base) & ((key > pos - w) | (key < sk) | (w == 0))
            for b in range(n):
                if m >> b & 1:
                    see[i] |= key == base + b
        x = torch.einsum("nhgd,hkd->nhgk", s["q"][a:e].double().view(n, hkv, hq // hkv, d), kv[0])
        x = (x * s["scale"]).masked_fill(~see[:, None, None], -math.inf)
        ls = torch.logsumexp(x, -1)
        out[a:e] = torch.einsum("nhgk,hkd->nhgd", torch.exp(x - ls[..., None]), kv[1]).reshape(n, hq, d)
        lse[a:e] = ls.reshape(n, hq)
    return dict(out=out, lse=lse)


def _exact_compact(s):
    ps, table = s["k_cache"].shape[2], s["page_tables"].cpu()
    past, path, m = s["past"].tolist(), s["path"].tolist(), s["path_lens"].tolist()
    out = dict(lens=torch.tensor([a + b for a, b in zip(past, m)], dtype=torch.int32))
    for n in ("k", "v"):
        c, sc = _stored(s, n)
        before, sb = c.clone(), None if sc is None else sc.clone()
        for r, p in enumerate(past):
            to = {}
            for i in range(m[r]):
                if path[r][i] != i:
                    a, b = p + path[r][i], p + i
                    to.setdefault(int(table[r, b // ps]), []).append(
                        (b % ps, int(table[r, a // ps]), a % ps))
            for pg, moves in to.items():
                rows = torch.stack([before[a, :, t] for _, a, t in moves], 1)
                at = [b for b, _, _ in moves]
                if sc is None:
                    c[pg][:, at] = rows
                    continue
                rows = rows * torch.stack([sb[a] for _, a, _ in moves], 1)[..., None]
                amax = rows.abs().amax((1, 2))
                t = torch.where(amax > 448 * sb[pg], _need(amax), sb[pg])
                c[pg] = _code(before[pg] * (sb[pg] / t)[:, None, None])
                c[pg][:, at] = _code(rows / t[:, None, None])
                sc[pg] = t
        out[n + "_cache"], out[n + "_scale"] = c, sc
    return out


def _exact_fork(s):
    ps, old = s["k_cache"].shape[2], s["page_tables"].cpu()
    t = torch.full((s["parent"].numel(), old.shape[1]), -1, dtype=torch.int32)
    kv, parent, new = s["kv_lens"].tolist(), s["parent"].tolist(), s["new_pages"].tolist()
    out = dict(tables=t, lens=torch.tensor([kv[p] for p in parent], dtype=torch.int32))
    for n in ("k", "v"):
        c, sc = _stored(s, n)
        for i, p in enumerate(parent):
            full, used = divmod(kv[p], ps)
            t[i, :full] = old[p, :full]
            if full < old.shape[1]:
                t[i, full] = new[i]
            if used:
                c[new[i], :, :used] = c[int(old[p, full]), :, :used]
                if sc is not None:
                    sc[new[i]] = sc[int(old[p, full])]
        out[n + "_cache"], out[n + "_scale"] = c, sc
    return out


def _exact_vision(s):
    n, H, d = s["q"].shape
    y = torch.einsum("nc,oc->no", s["x"].double(), s["w"].double()) + s["bias"].double()
    y, z = y.view(n, 3, H, d), _exact_turns(s)
    return dict(q=_turn(y[:, 0], z), k=_turn(y[:, 1], z), v=y[:, 2])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_tree(s, case)
    return {"append": _exact_append, "compact": _exact_compact, "fork": _exact_fork,
            "vision": _exact_vision}[case["op"]](s)
