"""The operators of drafted trees used together, as a serving loop does: prompts with image positions
appended, requests forked, trees appended at their depths, attended and compacted; calls on streams,
in graphs, in caches beyond 32 bits."""
import numpy as np
import pytest
import torch

import gqa_ref as ref
import tree_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tts():
    import tiled_top_sparse_gb300 as m
    m.lib()
    return m


def cuda(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x)).to(dtype).cuda()


def masks_tensor(masks):
    return torch.tensor([tree_ref.signed(m) for m in masks], dtype=torch.int64, device="cuda")


def cache(pages, hkv, ps, d, f8):
    if f8:
        return [torch.zeros(pages, hkv, ps, d, dtype=torch.uint8, device="cuda") for _ in range(2)] + \
            [torch.zeros(pages, hkv, device="cuda") for _ in range(2)]
    return [torch.zeros(pages, hkv, ps, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)] + \
        [None, None]


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("f8", [True, False])
def test_a_serving_loop(tts, f8):
    """What the cache holds after every step is what the tokens that were kept would have put there;
    attention over it agrees with 64-bit attention over those tokens."""
    rng = np.random.default_rng(1)
    hq, hkv, d, ps, scale = 8, 2, 64, 16, 64 ** -0.5
    c = cache(40, hkv, ps, d, f8)
    free = list(rng.permutation(40))
    cs = torch.tensor(ref.rope_table(300, d)).cuda()
    axis = tts.rope_axes([8, 12, 12])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def tokens(n):
        return torch.tensor(rng.standard_normal((n, hq + 2 * hkv, d))).to(torch.bfloat16).cuda()

    def rotated(x, pos):  # as the cache should hold it, in 64 bits
        t = tree_ref.turns(cs.cpu().numpy(), pos, axis)
        return torch.tensor(ref.rotate32(x.float().cpu().numpy(), t)).double()

    def append(x, past, cu, pos):
        q, _ = tts.rope_kv_append_axes(x[:, hq:hq + hkv], x[:, hq + hkv:], c[0], c[1], tables, cuda(past),
                                       cuda(cu), int(np.diff(cu).max()), cuda(pos), axis, cs,
                                       k_scale=c[2], v_scale=c[3], q=x[:, :hq], status=st)
        return q

    # two prompts, one with an image: (time, row, column) positions
    lens, width = [50, 23], 10
    tables = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    for r, n in enumerate(lens):
        for a in range(-(-(n + 16) // ps)):
            tables[r, a] = int(free.pop())
    pos = np.zeros((3, 73), np.int64)
    pos[:, :50], pos[:, 50:] = np.arange(50), np.arange(23)
    pos[0, 10:35], pos[1, 10:35], pos[2, 10:35] = 10, 10 + np.arange(25) // 5, 10 + np.arange(25) % 5
    x = tokens(73)
    append(x, [0, 0], [0, 50, 73], pos)
    held = [(rotated(x[a:b, hq:hq + hkv], pos[:, a:b]), x[a:b, hq + hkv:].double().cpu())
            for a, b in ((0, 50), (50, 73))]

    # the first one is answered twice: requests 0, 1 and the fork of 0
    tables, kv = tts.kv_fork(c[0], c[1], tables, cuda(lens), cuda([0, 1, 0]),
                             cuda([-1, -1, int(free.pop())]), k_scale=c[2], v_scale=c[3], status=st)
    for a in range(50 // ps + 1, 6):
        tables[2, a] = int(free.pop())
    held = [held[0], held[1], held[0]]
    lens = kv.tolist()
    assert lens == [50, 23, 50]

    for step in range(4):
        n = [5 + step, 9, 12]
        trees = [tree_ref.random_tree(rng, m) for m in n]
        masks = [m for t in trees for m in tree_ref.masks_of(t)]
        cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        depth = np.array([bin(m).count("1") - 1 for m in masks])
        p = np.concatenate([np.full(m, L) for m, L in zip(n, lens)]) + depth
        pos = np.stack([p, p, p])
        x = tokens(sum(n))
        for r in range(3):  # pages for the tokens to come
            for a in range(-(-(lens[r] + n[r]) // ps)):
                if int(tables[r, a]) < 0:
                    tables[r, a] = int(free.pop())
        q = append(x, lens, cu, pos)
        out, lse = tts.attn_decode_tree(q, c[0], c[1], tables,
                                        cuda([a + b for a, b in zip(lens, n)]), masks_tensor(masks),
                                        scale, cuda(cu), max(n), k_scale=c[2], v_scale=c[3], status=st)
        new = (rotated(x[:, hq:hq + hkv], pos), x[:, hq + hkv:].double().cpu())
        path = []
        for r in range(3):
            k = torch.cat([held[r][0], new[0][cu[r]:cu[r + 1]]])
            v = torch.cat([held[r][1], new[1][cu[r]:cu[r + 1]]])
            see = torch.tensor(np.stack([tree_ref.sees(m, n[r], lens[r] + n[r], 0, 0)
                                         for m in masks[cu[r]:cu[r + 1]]]))
            qq = q[cu[r]:cu[r + 1]].double().cpu().view(n[r], hkv, hq // hkv, d)
            s = torch.einsum("nhgd,jhd->nhgj", qq, k) * scale
            w = s.masked_fill(~see[:, None, None], float("-inf")).softmax(-1)
            want = torch.einsum("nhgj,jhd->nhgd", w, v).reshape(n[r], hq, d)
            # e4m3: keys and values each off by up to 2^-4; bf16: by 2^-8
            assert rel(out[cu[r]:cu[r + 1]].cpu(), want) < (0.06 if f8 else 6e-3)
            leaf = int(rng.integers(0, n[r]))
            path.append([i for i in range(n[r]) if masks[cu[r] + leaf] >> i & 1])
        wide = max(map(len, path))
        kv = tts.kv_compact(c[0], c[1], tables, cuda(lens),
                            cuda([p + [-1] * (wide - len(p)) for p in path]),
                            cuda([len(p) for p in path]), k_scale=c[2], v_scale=c[3], status=st)
        held = [tuple(torch.cat([h, t[cu[r]:cu[r + 1]][path[r]]]) for h, t in zip(held[r], new))
                for r in range(3)]
        lens = kv.tolist()
        assert lens == [h[0].shape[0] for h in held]
        tts.check_status(st)
        for r in range(3):  # the cache's rows are the kept tokens'
            j = torch.arange(lens[r])
            pg, sl = tables[r].cpu()[j // ps].long(), j % ps
            for i in range(2):
                got = torch.tensor(ref.codes_of(c[i]))[pg, :, sl]
                if f8:  # two roundings of relative 2^-4 at most, in the end a page's scale to 2^-10 of it
                    sc = c[2 + i].cpu()[pg].double()[..., None]
                    tol = held[r][i].abs() * (2.0 ** -3 + 2.0 ** -8) + 2.0 ** -9 * sc
                    got = got * sc
                else:
                    tol = held[r][i].abs() * 2.0 ** -8 + 1e-30
                assert bool(((got - held[r][i]).abs() <= tol).all())
    # plain decoding goes on over what the trees left
    x = tokens(3)
    p = np.stack([np.array(lens)] * 3)
    for r in range(3):
        if int(tables[r, lens[r] // ps]) < 0:
            tables[r, lens[r] // ps] = int(free.pop())
    q = append(x, lens, [0, 1, 2, 3], p)
    one = cuda([a + 1 for a in lens])
    a, la = tts.attn_decode_paged(q, c[0], c[1], tables, one, scale, k_scale=c[2], v_scale=c[3])
    b, lb = tts.attn_decode_tree(q, c[0], c[1], tables, one, masks_tensor([1, 1, 1]), scale,
                                 k_scale=c[2], v_scale=c[3])
    assert rel(b, a.double()) < 4e-3 and float((la - lb).abs().max()) < 1e-3


def setup(seed, new, past, hq, hkv, d, ps, f8, extra=2):
    rng = np.random.default_rng(seed)
    ends = [a + b for a, b in zip(past, new)]
    need = [-(-n // ps) for n in ends]
    perm = rng.permutation(sum(need) + extra)
    tables = np.full((len(new), max(need) + 1), -1, np.int32)
    at = 0
    for r, n in enumerate(need):
        tables[r, :n] = perm[at:at + n]
        at += n
    c = []
    for _ in range(2):
        x = torch.tensor(rng.standard_normal((sum(need) + extra, hkv, ps, d)), dtype=torch.float32)
        c.append((x * 60).to(torch.float8_e4m3fn).view(torch.uint8).cuda() if f8
                 else x.to(torch.bfloat16).cuda())
    s = [torch.full((sum(need) + extra, hkv), 2.0 ** -6, device="cuda") if f8 else None for _ in range(2)]
    masks = [m for n in new for m in tree_ref.masks_of(tree_ref.random_tree(rng, n))]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.tensor(rng.standard_normal((sum(new), hq, d))).to(torch.bfloat16).cuda()
    return dict(c=c, s=s, tables=cuda(tables), masks=masks_tensor(masks), cu=cuda(cu), q=q,
                kv=cuda(ends), past=cuda(past), rng=rng, max_new=max(new), scale=d ** -0.5)


def attend(tts, z, q=None, **kw):
    return tts.attn_decode_tree(z["q"] if q is None else q, *z["c"], z["tables"], z["kv"], z["masks"],
                                z["scale"], z["cu"], z["max_new"], k_scale=z["s"][0],
                                v_scale=z["s"][1], **kw)


@pytest.mark.parametrize("f8", [True, False])
def test_a_captured_step(tts, f8):
    """Append, attention and compaction captured once (twice: two graphs with workspaces of their
    own) and replayed over other tokens, trees, lengths and paths: the bits of eager calls."""
    new, past, hq, hkv, d, ps = [30, 12], [100, 70], 8, 2, 128, 32
    rng = np.random.default_rng(5)
    cs = torch.tensor(ref.rope_table(400, d)).cuda()
    axis = tts.rope_axes([d // 2])

    def state():
        z = setup(6, new, [a + 40 for a in past], hq, hkv, d, ps, f8)
        z.update(past=cuda(past), kv=torch.zeros(2, dtype=torch.int32, device="cuda"), n=cuda(new),
                 x=torch.zeros(42, hq + 2 * hkv, d, dtype=torch.bfloat16, device="cuda"),
                 pos=torch.zeros(1, 42, dtype=torch.int32, device="cuda"),
                 path=torch.zeros(2, 8, dtype=torch.int32, device="cuda"), m=cuda([0, 0]),
                 lens=cuda([0, 0]), out=torch.zeros(42, hq, d, device="cuda"),
                 lse=torch.zeros(42, hq, device="cuda"),
                 qo=torch.zeros(42, hq, d, dtype=torch.bfloat16, device="cuda"))
        z["ws"] = torch.empty(tts.attn_decode_tree_workspace_bytes(30, hq, hkv, d), dtype=torch.uint8,
                              device="cuda")
        return z

    def step(z):
        tts.rope_kv_append_axes(z["x"][:, hq:hq + hkv], z["x"][:, hq + hkv:], *z["c"], z["tables"],
                                z["past"], z["cu"], 30, z["pos"], axis, cs, k_scale=z["s"][0],
                                v_scale=z["s"][1], q=z["x"][:, :hq], q_out=z["qo"])
        torch.add(z["past"], z["n"], out=z["kv"])
        attend(tts, z, z["qo"], out=z["out"], lse=z["lse"], workspace=z["ws"])
        tts.kv_compact(*z["c"], z["tables"], z["past"], z["path"], z["m"], k_scale=z["s"][0],
                       v_scale=z["s"][1], kv_lens=z["lens"])
        z["past"].copy_(z["lens"])

    feeds = []
    for _ in range(4):
        trees = [tree_ref.random_tree(rng, n) for n in new]
        masks = [tree_ref.masks_of(t) for t in trees]
        path = [[i for i in range(n) if m[int(rng.integers(0, n))] >> i & 1][:8]
                for n, m in zip(new, masks)]
        path = [sorted(set(p) | {0}) for p in path]
        feeds.append(dict(
            x=torch.tensor(rng.standard_normal((42, hq + 2 * hkv, d))).to(torch.bfloat16).cuda(),
            pos=cuda(rng.integers(0, 400, (1, 42))), masks=masks_tensor(sum(masks, [])),
            path=cuda([p[:8] + [0] * (8 - len(p)) for p in path]), m=cuda([min(len(p), 8) for p in path])))

    def feed(z, f):
        for k, v in f.items():
            z[k].copy_(v)

    plain, want = state(), []
    for f in feeds:
        feed(plain, f)
        step(plain)
        want.append((plain["out"].clone(), plain["lse"].clone(), plain["lens"].clone()))
    held, graphs = [state(), state()], []
    torch.cuda.synchronize()
    for z in held:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(z)
        graphs.append(g)
    for f, w in zip(feeds, want):
        for z, g in zip(held, graphs):
            feed(z, f)
            g.replay()
        for z in held:
            assert torch.equal(z["out"], w[0]) and torch.equal(z["lse"], w[1])
            assert torch.equal(z["lens"], w[2])
    for z in held:
        assert all(torch.equal(a, b) for a, b in zip(z["c"], plain["c"]))


def test_calls_on_two_streams(tts):
    """Calls in flight at once, each with a workspace of its own."""
    z = setup(7, [40, 16, 64], [5000, 300, 9], 16, 4, 128, 64, True)
    qs = [torch.randn_like(z["q"].float()).to(torch.bfloat16) for _ in range(2)]
    need = tts.attn_decode_tree_workspace_bytes(64, 16, 4, 128)
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    want = [tuple(t.clone() for t in attend(tts, z, q, workspace=w)) for q, w in zip(qs, ws)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(attend(tts, z, qs[i], workspace=ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


def test_calls_one_behind_another(tts):
    """Launches set up while the call before still runs: the same bits with and without a
    synchronisation in between, also where one call reads what the one before wrote."""
    z = setup(8, [20, 5], [200, 77], 8, 2, 128, 64, True)
    first = [t.clone() for t in (*z["c"], *z["s"])]
    path, m = cuda([[3, 7, 11], [0, 2, 4]]), cuda([3, 3])

    def run(sync):
        for t, f in zip((*z["c"], *z["s"]), first):
            t.copy_(f)
        res = []
        for _ in range(6):
            res.append(attend(tts, z))
            if sync:
                torch.cuda.synchronize()
            tts.kv_compact(*z["c"], z["tables"], z["past"], path, m, k_scale=z["s"][0], v_scale=z["s"][1])
            if sync:
                torch.cuda.synchronize()
        return res

    a, b = run(True), run(False)
    for (o, l), (o2, l2) in zip(a, b):
        assert torch.equal(o, o2) and torch.equal(l, l2)


def test_workspace_is_found_or_made(tts):
    z = setup(9, [9], [300], 4, 2, 128, 64, True)
    a = attend(tts, z)
    b = attend(tts, z, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_no_more_written_than_the_workspace(tts):
    """Bytes behind the workspace that was asked for stay as they are, at every number of rows."""
    for new, hq, hkv, d in (([3, 64], 2, 1, 64), ([64, 64], 16, 2, 128), ([1], 1, 1, 128)):
        z = setup(10, new, [3000] * len(new), hq, hkv, d, 64, False)
        need = tts.attn_decode_tree_workspace_bytes(max(new), hq, hkv, d)
        ws = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
        attend(tts, z, workspace=ws[:need])
        assert bool((ws[need:] == 77).all())


def test_caches_beyond_32_bits(tts):
    """Pages whose rows lie behind 2^32 bytes (and values) of the cache."""
    hq, hkv, d, ps = 8, 8, 128, 128
    pages = (1 << 32) // (hkv * ps * d) + 40  # e4m3: over 4 GB each
    c = [torch.zeros(pages, hkv, ps, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    s = [torch.ones(pages, hkv, device="cuda") for _ in range(2)]
    rng = np.random.default_rng(11)
    T = np.array([[pages - 1, 3, pages - 5], [pages - 30, pages - 2, 1]], np.int32)
    new, past = [20, 30], [200, 300]
    x = torch.tensor(rng.standard_normal((50, hq + 2 * hkv, d))).to(torch.bfloat16).cuda()
    fill = torch.tensor(rng.standard_normal((500, hq + 2 * hkv, d))).to(torch.bfloat16).cuda()
    cs, axis = torch.tensor(ref.rope_table(600, d)).cuda(), tts.rope_axes([16, 24, 24])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    small = [torch.zeros(8, hkv, ps, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    small_s = [torch.ones(8, hkv, device="cuda") for _ in range(2)]
    T2 = np.array([[0, 1, 2], [3, 4, 5]], np.int32)
    res = []
    for cc, ss, t, fresh in ((c, s, T, pages - 9), (small, small_s, T2, 6)):
        for rows, p, cu in ((fill, [0, 0], [0, 200, 500]), (x, past, [0, 20, 50])):
            pos = cuda(np.arange(3 * rows.shape[0]).reshape(3, -1) % 600)
            q, _ = tts.rope_kv_append_axes(rows[:, hq:hq + hkv], rows[:, hq + hkv:], *cc, cuda(t), cuda(p),
                                           cuda(cu), 300, pos, axis, cs, k_scale=ss[0], v_scale=ss[1],
                                           q=rows[:, :hq], status=st)
        masks = masks_tensor([m for n in new for m in tree_ref.masks_of([-1] + list(range(n - 1)))])
        o, l = tts.attn_decode_tree(q, *cc, cuda(t), cuda([220, 330]), masks, 0.09, cuda([0, 20, 50]), 30,
                                    k_scale=ss[0], v_scale=ss[1], status=st)
        lens = tts.kv_compact(*cc, cuda(t), cuda(past), cuda([[2, 9, 19], [0, 5, 29]]), cuda([3, 3]),
                              k_scale=ss[0], v_scale=ss[1], status=st)
        tt, ln = tts.kv_fork(*cc, cuda(t), lens, cuda([1]), cuda([fresh]), k_scale=ss[0], v_scale=ss[1],
                             status=st)
        o2, _ = tts.attn_decode_tree(q[:1], *cc, tt, ln, masks_tensor([1]), 0.09, k_scale=ss[0],
                                     v_scale=ss[1], status=st)
        res.append((o, l, lens, ln, o2))
    tts.check_status(st)
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_binding_refuses_tensors_that_do_not_fit(tts):
    z = setup(12, [4, 3], [30, 60], 4, 2, 64, 16, True)
    good = dict(q=z["q"], k_cache=z["c"][0], v_cache=z["c"][1], page_tables=z["tables"], kv_lens=z["kv"],
                tree_mask=z["masks"], scale=0.1, cu_seqlens_q=z["cu"], max_seqlen_q=4, k_scale=z["s"][0],
                v_scale=z["s"][1])
    tts.attn_decode_tree(**good)
    m = z["masks"]
    for bad in (dict(tree_mask=m[:-1]), dict(tree_mask=m.int()), dict(tree_mask=m.cpu()),
                dict(tree_mask=torch.stack([m, m], 1)[:, 0]), dict(tree_mask=None),
                dict(q=z["q"].float()), dict(k_scale=None), dict(kv_lens=z["kv"][:1])):
        with pytest.raises(ValueError):
            tts.attn_decode_tree(**{**good, **bad})
    for bad in (dict(scale=-1.0), dict(window=-1), dict(max_seqlen_q=65), dict(max_seqlen_q=0)):
        with pytest.raises(tts.TTSError):
            tts.attn_decode_tree(**{**good, **bad})
    path, n = cuda([[0, 2], [1, 2]]), cuda([2, 2])
    good = dict(k_cache=z["c"][0], v_cache=z["c"][1], page_tables=z["tables"], past_lens=z["past"],
                path=path, path_lens=n, k_scale=z["s"][0], v_scale=z["s"][1])
    tts.kv_compact(**good)
    for bad in (dict(path=path.t()), dict(path=path.long()), dict(path=path[:1]), dict(path_lens=n.cpu()),
                dict(v_scale=None), dict(kv_lens=n.long())):
        with pytest.raises(ValueError):
            tts.kv_compact(**{**good, **bad})
    with pytest.raises(tts.TTSError):
        tts.kv_compact(**{**good, "kv_lens": z["past"]})
    with pytest.raises(tts.TTSError):
        tts.kv_compact(**{**good, "path": torch.zeros(2, 65, dtype=torch.int32, device="cuda")})
    good = dict(k_cache=z["c"][0], v_cache=z["c"][1], page_tables=z["tables"], kv_lens=z["kv"],
                parents=cuda([0, 1]), new_pages=cuda([-1, -1]), k_scale=z["s"][0], v_scale=z["s"][1])
    tts.kv_fork(**good)
    for bad in (dict(new_pages=cuda([1])), dict(parents=cuda([0, 1]).long()),
                dict(tables_out=z["tables"][:1]), dict(lens_out=cuda([0]))):
        with pytest.raises(ValueError):
            tts.kv_fork(**{**good, **bad})
    with pytest.raises(tts.TTSError):
        tts.kv_fork(**{**good, "tables_out": z["tables"]})


def test_another_stream(tts):
    """A call inside another stream's context is ordered behind that stream's work."""
    z = setup(13, [12, 8], [400, 90], 8, 2, 64, 32, False)
    want = attend(tts, z)
    st = torch.cuda.Stream()
    q = torch.zeros_like(z["q"])
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
        q.copy_(z["q"])
        got = attend(tts, z, q)
    st.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("d,ps", [(128, 64), (64, 16)])
def test_a_step_at_positions_outside_the_table(tts, f8, d, ps):
    """Tokens outside the rotation table are cached with zero keys and get zero queries: on fresh pages their
    attention is the mean of the values that they see. A padded batch of zeros is the same."""
    new, hq, hkv = [12, 1, 30], 8, 2
    rng = np.random.default_rng(d)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    masks = [m for n in new for m in tree_ref.masks_of(tree_ref.random_tree(rng, n))]
    tables = np.arange(9).reshape(3, 3).astype(np.int32)
    for max_pos, gain in ((4, 1.0), (400, 0.0)):
        c = cache(10, hkv, ps, d, f8)
        x = torch.tensor(rng.standard_normal((43, hq + 2 * hkv, d)))
        x[:, :hq + hkv] *= gain
        x = x.to(torch.bfloat16).cuda()
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        q, _ = tts.rope_kv_append_axes(
            x[:, hq:hq + hkv], x[:, hq + hkv:], *c[:2], cuda(tables), cuda([0, 0, 0]), cuda(cu), 30,
            cuda(np.arange(100, 143)[None]), tts.rope_axes([d // 2]), tts.rope_cache(max_pos, d),
            k_scale=c[2], v_scale=c[3], q=x[:, :hq], status=st)
        assert int(st.item()) == (tts.TTS_DEV_INDEX_RANGE if gain else 0)
        assert bool((q == 0).all())
        st.zero_()
        out, lse = tts.attn_decode_tree(q, *c[:2], cuda(tables), cuda(new), masks_tensor(masks), d ** -0.5,
                                        cuda(cu), 30, k_scale=c[2], v_scale=c[3], status=st)
        tts.check_status(st)
        s = [None if t is None else t.cpu().numpy() for t in c[2:]]
        o, l, tol, tol_l = tree_ref.attend_tree(
            q.float().cpu().numpy(), ref.codes_of(c[0]), ref.codes_of(c[1]), *s, tables, new, cu, masks,
            d ** -0.5, 0, 0)
        assert bool((np.abs(out.cpu().double().numpy() - o) <= tol).all())
        assert bool((np.abs(lse.cpu().double().numpy() - l) <= tol_l).all())
