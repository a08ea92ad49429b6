"""GPU parity of rotations with positions on several axes: the append (tts_rope_kv_append_axes) and
the vision projection (tts_qkv_rope_axes) with their definitions."""
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


def append(tts, seed, new, past, hq, hkv, d, ps, f8, axis, axes, max_pos=500, positions=None,
           with_q=True, cos_sin=None, pad=0):
    rng = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1]) + pad
    need = [-(-(a + b) // ps) for a, b in zip(past, new)]
    perm = rng.permutation(sum(need) + 2)
    tables = np.full((len(new), max(need) + 1), -1, np.int32)
    at = 0
    for r, n in enumerate(need):
        tables[r, :n] = perm[at:at + n]
        at += n
    pages = sum(need) + 2
    x = torch.tensor(rng.standard_normal((T, hq + 2 * hkv, d))).to(torch.bfloat16)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if positions is None:
        positions = rng.integers(0, max_pos, (axes, T)).astype(np.int32)
    cs = ref.rope_table(max_pos, d) if cos_sin is None else cos_sin
    if f8:
        c = [torch.tensor(rng.standard_normal((pages, hkv, ps, d)) * 60, dtype=torch.float32).to(
            torch.float8_e4m3fn).view(torch.uint8) for _ in range(2)]
        s = [torch.tensor(2.0 ** rng.integers(-9, -4, (pages, hkv)), dtype=torch.float32)
             for _ in range(2)]
    else:
        c = [torch.tensor(rng.standard_normal((pages, hkv, ps, d))).to(torch.bfloat16)
             for _ in range(2)]
        s = [None, None]
    D = [None if t is None else t.cuda() for t in (*c, *s)]
    X = x.cuda()
    q_out = torch.full((T, hq, d), 7.0, dtype=torch.bfloat16, device="cuda") if with_q else None
    k_out = torch.full((T, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tts.rope_kv_append_axes(X[:, hq:hq + hkv], X[:, hq + hkv:], D[0], D[1], cuda(tables), cuda(past),
                            cuda(cu), max(new), cuda(positions), axis, cuda(cs, torch.float32),
                            k_scale=D[2], v_scale=D[3], q=X[:, :hq] if with_q else None, q_out=q_out,
                            k_out=k_out, status=st)
    n = int(cu[-1])
    t = tree_ref.turns(cs, np.clip(positions, 0, cs.shape[0] - 1), axis)[:n]
    fine = ((positions >= 0) & (positions < cs.shape[0])).all(0)[:n]
    qr = ref.rotate32(q[:n].float().numpy(), t) * fine[:, None, None]
    kr = ref.rotate32(k[:n].float().numpy(), t) * fine[:, None, None]
    want = ref.append(None, kr, v[:n].float().numpy(), ref.codes_of(c[0]), ref.codes_of(c[1]),
                      *(None if z is None else z.numpy() for z in s), tables, past, cu, None, ps)
    if with_q:
        assert torch.equal(q_out[:n].cpu(), torch.tensor(qr).to(torch.bfloat16))
        assert bool((q_out[n:] == 7).all())
    assert torch.equal(k_out[:n].cpu(), torch.tensor(kr).to(torch.bfloat16))
    assert bool((k_out[n:] == 7).all())
    if f8:
        np.testing.assert_array_equal(D[2].cpu().numpy(), want[4].astype(np.float32))
        np.testing.assert_array_equal(D[3].cpu().numpy(), want[5].astype(np.float32))
        np.testing.assert_array_equal(ref.codes_of(D[0]), want[2])
        np.testing.assert_array_equal(ref.codes_of(D[1]), want[3])
    else:
        assert torch.equal(D[0].cpu(), torch.tensor(want[2]).float().to(torch.bfloat16))
        assert torch.equal(D[1].cpu(), torch.tensor(want[3]).float().to(torch.bfloat16))
    return int(st.item()), D, q_out, k_out


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("axes,kind", [(1, "one"), (2, "runs"), (3, "runs"), (3, "turns"), (4, "any")])
@pytest.mark.parametrize("new,past,hq,hkv,d,ps", [
    ([1, 1, 2], [0, 63, 100], 8, 2, 128, 64),      # steps
    ([30, 0, 64, 5], [15, 14, 5, 16], 5, 1, 128, 16),
    ([200, 33], [57, 0], 4, 2, 64, 128),
])
def test_append(tts, f8, axes, kind, new, past, hq, hkv, d, ps):
    rng = np.random.default_rng(axes)
    pairs = d // 2
    if kind == "any":
        axis = bytes(rng.integers(0, axes, pairs).tolist())
    elif kind == "turns":
        axis = tts.rope_axes([pairs - 2 * (pairs // 3 - 1)] + [pairs // 3 - 1] * 2, True)
    else:
        axis = tts.rope_axes([pairs - 12 * (axes - 1)] + [12] * (axes - 1))
    st, *_ = append(tts, sum(new) + axes, new, past, hq, hkv, d, ps, f8, axis, axes, pad=2)
    assert st == 0
    append(tts, sum(new) + axes, new, past, hq, hkv, d, ps, f8, axis, axes, with_q=False)


def test_one_axis_is_the_plain_append(tts):
    """Positions past + i on one axis: the bits of rope_kv_append."""
    new, past = [40, 3], [10, 64]
    pos = np.concatenate([np.arange(p, p + n) for p, n in zip(past, new)])[None].astype(np.int32)
    _, D, q, k = append(tts, 7, new, past, 4, 2, 128, 64, True, bytes(64), 1, positions=pos)
    rng = np.random.default_rng(7)
    perm = rng.permutation(3 + 2)  # the same inputs again
    tables = np.full((2, 3), -1, np.int32)
    tables[0, :1], tables[1, :2] = perm[:1], perm[1:3]
    x = torch.tensor(rng.standard_normal((43, 8, 128))).to(torch.bfloat16).cuda()
    c = [torch.tensor(rng.standard_normal((5, 2, 64, 128)) * 60, dtype=torch.float32).to(
        torch.float8_e4m3fn).view(torch.uint8).cuda() for _ in range(2)]
    s = [torch.tensor(2.0 ** rng.integers(-9, -4, (5, 2)), dtype=torch.float32).cuda() for _ in range(2)]
    q2, k2 = tts.rope_kv_append(x[:, 4:6], x[:, 6:], c[0], c[1], cuda(tables), cuda(past),
                                cuda([0, 40, 43]), 40, k_scale=s[0], v_scale=s[1],
                                cos_sin=cuda(ref.rope_table(500, 128), torch.float32), q=x[:, :4],
                                want_k=True)
    assert torch.equal(q, q2) and torch.equal(k, k2)
    for a, b in zip(D, (*c, *s)):
        assert torch.equal(a, b)


def test_positions_outside_the_table(tts):
    """Their tokens' q and k are zeros and it is said; rows behind max_pos as such are fine."""
    for new in ([3], [90]):
        pos = np.full((3, new[0]), 5, np.int32)
        pos[1, 1], pos[2, 2] = -1, 16
        st, *_ = append(tts, 3, new, [40], 4, 2, 64, 32, True, tts.rope_axes([8, 12, 12]), 3, max_pos=16,
                        positions=pos)
        assert st == tts.TTS_DEV_INDEX_RANGE
    pos = np.full((1, 3), 15, np.int32)
    st, *_ = append(tts, 3, [3], [40], 4, 2, 64, 32, False, bytes(32), 1, max_pos=16, positions=pos)
    assert st == 0


# -------------------------------------------------------------------------------- vision
def axes_table(max_pos, sizes):
    """Every axis has its own run of frequencies."""
    return np.concatenate([ref.rope_table(max_pos, 2 * n) for n in sizes], 1)


@pytest.mark.parametrize("n,hidden,heads,d,sizes,mixed", [
    (1, 64, 4, 64, [16, 16], False),
    (300, 520, 4, 64, [10, 11, 11], False),
    (129, 256, 5, 80, [20, 20], False),
    (700, 1280, 16, 80, [8, 16, 16], True),
    (257, 136, 2, 128, [64], False),
    (513, 512, 6, 128, [16, 24, 24], True),
    (40, 64, 4, 64, [8, 8, 8, 8], True),
])
def test_vision_projection(tts, n, hidden, heads, d, sizes, mixed):
    rng = np.random.default_rng(n)
    axis = tts.rope_axes(sizes, mixed)
    x = torch.tensor(rng.standard_normal((n, hidden))).to(torch.bfloat16)
    w = torch.tensor(rng.standard_normal((3 * heads * d, hidden)) / hidden ** 0.5).to(torch.bfloat16)
    b = rng.standard_normal(3 * heads * d).astype(np.float32)
    pos = rng.integers(0, 100, (len(sizes), n)).astype(np.int32)
    cs = axes_table(100, sizes)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bias in (b, None):
        got = tts.qkv_rope_axes(x.cuda(), w.cuda(), None if bias is None else cuda(bias, torch.float32),
                                cuda(pos), axis, cuda(cs, torch.float32), heads, status=st)
        tts.check_status(st)
        X, W = x.float().double().numpy(), w.float().double().numpy()
        y = X @ W.T + (0 if bias is None else bias.astype(np.float64))
        size = np.abs(X) @ np.abs(W).T + (0 if bias is None else np.abs(bias))
        y, size = y.reshape(n, 3, heads, d), size.reshape(n, 3, heads, d)
        t = tree_ref.turns(cs.astype(np.float64), pos, axis)[:, None]
        for i in range(3):
            lo, hi = y[:, i, :, :d // 2], y[:, i, :, d // 2:]
            e = (size[:, i, :, :d // 2] + size[:, i, :, d // 2:]) * (hidden + 8) * 2.0 ** -24
            e = np.concatenate([e, e], -1)
            want = y[:, i] if i == 2 else np.concatenate(
                [lo * t[..., 0] - hi * t[..., 1], lo * t[..., 1] + hi * t[..., 0]], -1)
            tol = e + 2.0 ** -8 * (np.abs(want) + e)  # sums of hidden products in fp32, one rounding
            off = np.abs(got[i].float().cpu().double().numpy() - want) - tol
            assert off.max() <= 0, off.max()


def test_vision_one_axis_is_the_plain_projection(tts):
    rng = np.random.default_rng(0)
    x = torch.tensor(rng.standard_normal((333, 256))).to(torch.bfloat16).cuda()
    w = torch.tensor(rng.standard_normal((3 * 5 * 80, 256)) / 16).to(torch.bfloat16).cuda()
    pos = cuda(rng.integers(0, 64, (1, 333)))
    cs = tts.rope_cache(64, 80)
    a = tts.qkv_rope(x, w, None, pos[0].contiguous(), cs, 5)
    b = tts.qkv_rope_axes(x, w, None, pos, bytes(40), cs, 5)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_vision_positions_outside_the_table(tts):
    rng = np.random.default_rng(0)
    x = torch.tensor(rng.standard_normal((20, 64))).to(torch.bfloat16).cuda()
    w = torch.tensor(rng.standard_normal((3 * 4 * 64, 64)) / 8).to(torch.bfloat16).cuda()
    pos = np.full((2, 20), 3, np.int32)
    pos[1, 7], pos[0, 11] = 64, -1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    cs = cuda(axes_table(64, [16, 16]), torch.float32)
    q, k, v = tts.qkv_rope_axes(x, w, None, cuda(pos), tts.rope_axes([16, 16]), cs, 4, status=st)
    assert int(st.item()) == tts.TTS_DEV_INDEX_RANGE
    assert bool((q[[7, 11]] == 0).all()) and bool((k[[7, 11]] == 0).all())
    assert bool((v[[7, 11]] != 0).any()) and bool((q[8] != 0).any())


@pytest.mark.parametrize("d,heads", [(64, 8), (128, 4), (80, 6)])
def test_vision_rows_do_not_depend_on_the_others(tts, d, heads):
    """A token's row is the same to the bit in a call of few tokens, whose tiles are one head's, and in
    one of many: every element is the same products in the same order."""
    g = torch.Generator("cpu").manual_seed(d)
    n, hidden = 2400, 192
    x = torch.randn(n, hidden, generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn(3 * heads * d, hidden, generator=g) * 0.1).to(torch.bfloat16).cuda()
    bias = torch.randn(3 * heads * d, generator=g).cuda()
    pos = torch.randint(0, 64, (2, n), generator=g, dtype=torch.int32).cuda()
    cs, axis = tts.rope_cache(64, d, device="cuda"), tts.rope_axes([d // 8, d // 2 - d // 8])
    full = tts.qkv_rope_axes(x, w, bias, pos, axis, cs, heads)
    plain = tts.qkv_rope(x, w, bias, pos[1].contiguous(), cs, heads)
    for m in (1, 130, 256, 500):
        few = tts.qkv_rope_axes(x[:m], w, bias, pos[:, :m].contiguous(), axis, cs, heads)
        assert all(torch.equal(a, b[:m]) for a, b in zip(few, full)), m
        few = tts.qkv_rope(x[:m], w, bias, pos[1, :m].contiguous(), cs, heads)
        assert all(torch.equal(a, b[:m]) for a, b in zip(few, plain)), m


@pytest.mark.parametrize("captured", [False, True])
def test_vision_behind_what_writes_its_inputs(tts, captured):
    """The projection may be set up while the launch before it runs: it reads what that one wrote."""
    g = torch.Generator("cpu").manual_seed(5)
    n, hidden, heads, d = 700, 256, 4, 64
    w = (torch.randn(3 * heads * d, hidden, generator=g) * 0.1).to(torch.bfloat16).cuda()
    pos = torch.randint(0, 64, (2, n), generator=g, dtype=torch.int32).cuda()
    cs, axis = tts.rope_cache(64, d, device="cuda"), tts.rope_axes([d // 4, d // 4])
    xs = [torch.randn(n, hidden, generator=g).to(torch.bfloat16).cuda() for _ in range(8)]
    want = [[t.clone() for t in tts.qkv_rope_axes(x, w, None, pos, axis, cs, heads)] for x in xs]
    x = torch.empty_like(xs[0])
    out = [torch.empty(n, heads, d, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    got = [[torch.empty_like(t) for t in out] for _ in xs]

    def steps():
        for src, dst in zip(xs, got):
            x.copy_(src)
            tts.qkv_rope_axes(x, w, None, pos, axis, cs, heads, *out)
            for a, b in zip(dst, out):
                a.copy_(b)

    steps()
    if captured:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            steps()
        for dst in got:
            for t in dst:
                t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_vision_without_the_binding(tts, monkeypatch):
    """A machine without Python's C headers has no binding: the projection with axes is made all the same,
    with its checks, as the one without axes is."""
    g = torch.Generator("cpu").manual_seed(6)
    n, hidden, heads, d = 130, 128, 4, 64
    a = dict(x=torch.randn(n, hidden, generator=g).to(torch.bfloat16).cuda(),
             w=(torch.randn(3 * heads * d, hidden, generator=g) * 0.1).to(torch.bfloat16).cuda(),
             bias=torch.randn(3 * heads * d, generator=g).cuda(),
             positions=torch.randint(0, 64, (2, n), generator=g, dtype=torch.int32).cuda(),
             pair_axis=tts.rope_axes([8, 24]), cos_sin=tts.rope_cache(64, d), num_heads=heads)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = tts.qkv_rope_axes(**a, status=st)

    def missing():
        raise ImportError("the native binding is not built")

    monkeypatch.setattr(tts, "_nat", None)
    monkeypatch.setattr(tts, "_binding", missing)
    got = tts.qkv_rope_axes(**a, status=st)
    tts.check_status(st)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    assert all(torch.equal(p, q) for p, q in zip(tts.qkv_rope_axes(**{**a, "bias": None}),
                                                 tts.qkv_rope_axes(**{**a, "bias": a["bias"] * 0})))
    z = torch.empty(n, heads, d, device="cuda")
    for bad in (dict(w=a["w"][:100]), dict(bias=a["bias"][:5]), dict(positions=a["positions"][:, 1:]),
                dict(positions=a["positions"].long()), dict(positions=a["positions"].cpu()),
                dict(positions=a["positions"].t()), dict(pair_axis=bytes(33)), dict(pair_axis=[0] * 32),
                dict(cos_sin=a["cos_sin"][:0]), dict(cos_sin=a["cos_sin"][:, 1:].contiguous()),
                dict(num_heads=5), dict(num_heads=0), dict(q=z), dict(k=z[1:].bfloat16()),
                dict(status=st.cpu())):
        with pytest.raises(ValueError):
            tts.qkv_rope_axes(**{**a, **bad})
    with pytest.raises(tts.TTSError):
        tts.qkv_rope_axes(**{**a, "pair_axis": bytes([2] * 32)})
    a.update(x=a["x"][:0], positions=a["positions"][:, :0].contiguous())
    assert tts.qkv_rope_axes(**a)[0].shape == (0, heads, d)
