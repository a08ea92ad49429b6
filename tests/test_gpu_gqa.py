"""GPU parity for the grouped-query cache: tts_rope_kv_append against its 64-bit definition
(codes, scales and rotated rows), tts_attn_decode_paged against 64-bit attention over the very
values the cache holds, and the two in turn as a serving loop uses them."""
import numpy as np
import pytest
import torch

import gqa_ref as ref

pytestmark = pytest.mark.gpu

F16_HALF, BF16_HALF = 2.0 ** -11, 2.0 ** -8


@pytest.fixture(scope="module")
def tts():
    import tiled_top_sparse_gb300 as m
    m.lib()
    return m


def dev(t):
    return t.to("cuda")


def gen(seed):
    g = torch.Generator("cpu")
    g.manual_seed(seed)
    return g


def make_pool(seed, pages, hkv, ps, d, f8, spread=True):
    """Cache contents: random values, e4m3 pages with scales of different sizes."""
    g = gen(seed)
    out = []
    for _ in range(2):
        x = torch.randn(pages, hkv, ps, d, generator=g)
        if f8:
            codes = (x * 60).to(torch.float8_e4m3fn)
            e = torch.randint(-9, -3, (pages, hkv), generator=g) if spread else torch.full(
                (pages, hkv), -6)
            out += [codes.view(torch.uint8), torch.exp2(e.float())]
        else:
            out += [x.to(torch.bfloat16), None]
    return out  # k, k_scale, v, v_scale


def make_tables(seed, lens, ps, extra=2):
    need = [-(-n // ps) for n in lens]
    perm = torch.randperm(sum(need) + extra, generator=gen(seed)).to(torch.int32)
    width = max(need + [1]) + 1
    t = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        t[r, :n] = perm[at:at + n]
        at += n
    return t, sum(need) + extra


def cum(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


# ------------------------------------------------------------------------------- append
def run_append(tts, seed, new, past, hq, hkv, d, ps, f8, rope=True, with_q=True, packed=True,
               gain=1.0, pool=None, pad_rows=0, max_new=None, front=0):
    cu = cum(new) + np.int32(front)
    T = int(cu[-1]) + pad_rows
    ends = [a + b for a, b in zip(past, new)]
    tables, pages = make_tables(seed, ends, ps)
    kc, ks, vc, vs = pool if pool is not None else make_pool(seed + 1, pages, hkv, ps, d, f8)
    g = gen(seed + 2)
    qkv = (torch.randn(T, hq + 2 * hkv, d, generator=g) * gain).to(torch.bfloat16)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    cs = ref.rope_table(max(ends), d) if rope else None
    D = dev(qkv)
    dq, dk, dv = D[:, :hq], D[:, hq:hq + hkv], D[:, hq + hkv:]
    if not packed:
        dq, dk, dv = dq.contiguous(), dk.contiguous(), dv.contiguous()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = [None if t is None else dev(t).clone() for t in (kc, ks, vc, vs)]
    q_out = torch.full((T, hq, d), 7.0, dtype=torch.bfloat16, device="cuda") if with_q else None
    k_out = torch.full((T, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    tts.rope_kv_append(dk, dv, c[0], c[2], dev(tables), dev(torch.tensor(past, dtype=torch.int32)),
                       dev(torch.tensor(cu)), max_new or max(new), k_scale=c[1], v_scale=c[3],
                       cos_sin=None if cs is None else dev(torch.tensor(cs)),
                       q=dq if with_q else None, q_out=q_out, k_out=k_out, status=st)
    tts.check_status(st)
    n = int(cu[-1])
    want = ref.append(q[:n].float().numpy(), k[:n].float().numpy(), v[:n].float().numpy(),
                      ref.codes_of(kc), ref.codes_of(vc), None if ks is None else ks.numpy(),
                      None if vs is None else vs.numpy(), tables.numpy(), past, cu, cs, ps)
    return c, q_out, k_out, want, n


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("new,past,hq,hkv,d,ps", [
    ([1, 1, 1], [0, 63, 100], 8, 2, 128, 64),               # decode steps; a page begun, filled
    ([1, 4, 0, 2], [15, 14, 5, 16], 4, 4, 128, 16),         # steps across a page border
    ([8, 3], [60, 0], 4, 1, 64, 32),                        # steps of eight, heads of 64
    ([5, 9, 0, 1], [0, 127, 3, 130], 10, 2, 128, 128),      # tiles: pages of 128
    ([300, 1, 77], [10, 0, 64], 6, 3, 128, 64),             # prompts, odd head count
    ([129, 40], [0, 31], 12, 2, 64, 16),                    # small pages, heads of 64
    ([200], [57], 9, 1, 64, 128),
])
def test_append_parity(tts, f8, new, past, hq, hkv, d, ps):
    c, q_out, k_out, (qr, kr, kc, vc, ks, vs), n = run_append(
        tts, sum(new) + ps, new, past, hq, hkv, d, ps, f8, pad_rows=3)
    # rotated rows: fp32 as documented, then one rounding to bf16 -- the same bits
    assert torch.equal(q_out[:n].cpu(), torch.tensor(qr).to(torch.bfloat16))
    assert torch.equal(k_out[:n].cpu(), torch.tensor(kr).to(torch.bfloat16))
    assert bool((q_out[n:] == 7).all()) and bool((k_out[n:] == 7).all())  # rows behind the last
    if f8:
        np.testing.assert_array_equal(c[1].cpu().numpy(), ks.astype(np.float32))
        np.testing.assert_array_equal(c[3].cpu().numpy(), vs.astype(np.float32))
        np.testing.assert_array_equal(ref.codes_of(c[0]), kc)
        np.testing.assert_array_equal(ref.codes_of(c[2]), vc)
    else:
        assert torch.equal(c[0].cpu(), torch.tensor(kc).float().to(torch.bfloat16))
        assert torch.equal(c[2].cpu(), torch.tensor(vc).float().to(torch.bfloat16))


@pytest.mark.parametrize("with_q,rope,packed", [(False, True, True), (True, False, False),
                                                (False, False, True)])
def test_append_without_q_or_rotation(tts, with_q, rope, packed):
    c, q_out, k_out, (qr, kr, kc, vc, ks, vs), n = run_append(
        tts, 5, [70, 3], [3, 60], 4, 2, 128, 64, True, rope=rope, with_q=with_q, packed=packed)
    if with_q:
        assert torch.equal(q_out.cpu(), torch.tensor(qr).to(torch.bfloat16))
    assert torch.equal(k_out.cpu(), torch.tensor(kr).to(torch.bfloat16))
    np.testing.assert_array_equal(ref.codes_of(c[0]), kc)
    np.testing.assert_array_equal(c[1].cpu().numpy(), ks.astype(np.float32))


@pytest.mark.parametrize("gain", [0.0, 1e-6, 1e-20, 1e4, 1e30])
def test_append_scales_of_any_size(tts, gain):
    """Zero rows take the smallest scale, large ones a large one; codes stay exact."""
    c, _, _, (_, _, kc, vc, ks, vs), _ = run_append(tts, 11, [1, 90], [0, 0], 2, 2, 128, 64, True,
                                                    gain=gain, with_q=False)
    np.testing.assert_array_equal(c[1].cpu().numpy(), ks.astype(np.float32))
    np.testing.assert_array_equal(ref.codes_of(c[0]), kc)
    np.testing.assert_array_equal(ref.codes_of(c[2]), vc)


def test_append_token_by_token_equals_the_definition(tts):
    """A page filled by single tokens of growing size: every growth of the scale moves the
    earlier codes."""
    hkv, d, ps, n = 2, 64, 16, 40
    tables, pages = make_tables(3, [n], ps)
    kc, ks, vc, vs = make_pool(4, pages, hkv, ps, d, True)
    g = gen(5)
    x = torch.randn(n, hkv, d, generator=g) * torch.exp2(torch.arange(n) % 13 - 6.0)[:, None, None]
    y = torch.randn(n, hkv, d, generator=g) * torch.exp2(-(torch.arange(n) % 7).float())[:, None, None]
    x, y = x.to(torch.bfloat16), y.to(torch.bfloat16)
    cs = ref.rope_table(n, d)
    c = [dev(t).clone() for t in (kc, ks, vc, vs)]
    want = (ref.codes_of(kc), ref.codes_of(vc), ks.numpy(), vs.numpy())
    one = dev(torch.tensor([0, 1], dtype=torch.int32))
    for i in range(n):
        tts.rope_kv_append(dev(x[i:i + 1]), dev(y[i:i + 1]), c[0], c[2], dev(tables),
                           torch.tensor([i], dtype=torch.int32, device="cuda"), one, 1,
                           k_scale=c[1], v_scale=c[3], cos_sin=dev(torch.tensor(cs)))
        w = ref.append(None, x[i:i + 1].float().numpy(), y[i:i + 1].float().numpy(), want[0],
                       want[1], want[2], want[3], tables.numpy(), [i], cum([1]), cs, ps)
        want = w[2:]
    np.testing.assert_array_equal(c[1].cpu().numpy(), want[2].astype(np.float32))
    np.testing.assert_array_equal(ref.codes_of(c[0]), want[0])
    np.testing.assert_array_equal(ref.codes_of(c[2]), want[1])


@pytest.mark.parametrize("max_new", [1, 40])
def test_append_skips_and_reports(tts, max_new):
    """Requests that do not fit, bad pages, bad lengths and a scale no page can have."""
    hkv, d, ps = 2, 64, 16
    new = [1, 1, 1, 1, 1] if max_new == 1 else [1, 40, 1, 3, 1]
    cu = cum(new)
    T = int(cu[-1])
    past = [0, 16 * 8 - 1 if max_new == 1 else 100, 5, -1, 3]
    tables, pages = make_tables(8, [16 * 8] * 5, ps)
    tables = tables[:, :8].contiguous()
    past[1] = 16 * 8 if max_new == 1 else past[1]      # past the table's end
    tables[2, 0] = pages                               # no such page
    kc, ks, vc, vs = make_pool(9, pages, hkv, ps, d, True)
    ks[tables[4, 0], 1] = float("nan")                 # request 4 appends at slot 3 of this page
    x = torch.randn(T, hkv, d, generator=gen(10)).to(torch.bfloat16)
    cs = ref.rope_table(128, d)

    def run(which):
        c = [dev(t).clone() for t in (kc, ks, vc, vs)]
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        keep = [n if r in which else 0 for r, n in enumerate(new)]
        rows = torch.cat([x[cu[r]:cu[r] + k] for r, k in enumerate(keep)])
        q_out, k_out = tts.rope_kv_append(
            dev(rows), dev(rows), c[0], c[2], dev(tables),
            dev(torch.tensor(past, dtype=torch.int32)), dev(torch.tensor(cum(keep))), max_new,
            k_scale=c[1], v_scale=c[3], cos_sin=dev(torch.tensor(cs)), q=dev(rows),
            k_out=torch.full(rows.shape, 7.0, dtype=torch.bfloat16, device="cuda"), status=st)
        return c, q_out, k_out, int(st.item())

    c, q_out, k_out, st = run([0, 1, 2, 3])
    assert st == tts.TTS_DEV_INDEX_RANGE
    ok = ref.append(None, x[:1].float().numpy(), x[:1].float().numpy(), ref.codes_of(kc),
                    ref.codes_of(vc), ks.numpy(), vs.numpy(), tables[:1].numpy(), [0], cum([1]),
                    cs, ps)
    np.testing.assert_array_equal(ref.codes_of(c[0]), ok[2])   # request 0 alone was cached
    np.testing.assert_array_equal(ref.codes_of(c[2]), ok[3])
    for r in (1, 3):                                           # no position: zero rows
        assert not q_out[cu[r]:cu[r + 1]].any() and not k_out[cu[r]:cu[r + 1]].any()
    assert q_out[cu[2]].any() and k_out[cu[2]].any()           # a bad page still rotates
    c, _, _, st = run([4])
    assert st == tts.TTS_DEV_BAD_ARG
    want = ref.page_scale(np.abs(ref.rotate32(x[cu[4]:cu[4] + 1].float().numpy(), cs[3:4]))[0, 1].max())
    assert float(c[1][tables[4, 0], 1]) == want
    # lengths that decrease, and one above max_new, take no rows
    for bad_cu in ([0, 1, 0, 1, 1, 1], [0, 0, 0, 0, 0, max_new + 1]):
        c = [dev(t).clone() for t in (kc, ks, vc, vs)]
        s = torch.zeros(1, dtype=torch.int32, device="cuda")
        rows = torch.zeros(max_new + 1, hkv, d, dtype=torch.bfloat16, device="cuda")
        tts.rope_kv_append(rows, rows, c[0], c[2], dev(tables),
                           torch.zeros(5, dtype=torch.int32, device="cuda"),
                           torch.tensor(bad_cu, dtype=torch.int32, device="cuda"), max_new,
                           k_scale=c[1], v_scale=c[3], status=s)
        assert int(s.item()) & tts.TTS_DEV_BAD_ARG


# ------------------------------------------------------------------------------- decode
def poison(c, tables, kv_lens, new, ps, window, sinks, f8):
    """What no new token sees becomes NaN: slots behind the end, keys outside the window; the
    table entries of pages without a visible key become nonsense."""
    kc, ks, vc, vs = [None if t is None else t.clone() for t in c]
    t = tables.clone()
    bad = torch.tensor(0x7F, dtype=torch.uint8) if f8 else torch.tensor(float("nan"),
                                                                      dtype=torch.bfloat16)
    seen_pages = set()
    for r, L in enumerate(kv_lens):
        lo = max(0, L - new[r] + 1 - window) if window > 0 else 0
        for a in range(t.shape[1]):
            j = np.arange(a * ps, (a + 1) * ps)
            see = (j < L) & ((j >= lo) | (j < sinks))
            if not see.any() or new[r] == 0:
                t[r, a] = 10 ** 9 if a % 2 else -5
                continue
            pg = int(t[r, a])
            seen_pages.add(pg)
            kc[pg, :, torch.tensor(~see)] = bad
            vc[pg, :, torch.tensor(~see)] = bad
    for pg in range(kc.shape[0]):
        if pg not in seen_pages:
            kc[pg] = bad
            vc[pg] = bad
            if f8:
                ks[pg] = float("nan")
                vs[pg] = -1.0
    return (kc, ks, vc, vs), t


def run_decode(tts, seed, new, kv, hq, hkv, d, ps, f8, window=0, sinks=0, out_dtype=torch.float32,
               one=False, clean=False, q_gain=1.0, max_q=None, front=0):
    cu = cum(new) + np.int32(front)
    T = int(cu[-1])
    tables, pages = make_tables(seed, kv, ps)
    pool = make_pool(seed + 1, pages, hkv, ps, d, f8)
    if not clean:
        pool, tables = poison(pool, tables, kv, new, ps, window, sinks, f8)
    q = (torch.randn(T + 2, hq, d, generator=gen(seed + 2)) * q_gain).to(torch.bfloat16)
    if one:
        q = q[:T]
    kc, ks, vc, vs = [None if t is None else dev(t) for t in pool]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = q.shape[0]
    out = torch.full((rows, hq, d), 7.0, dtype=out_dtype, device="cuda")
    lse = torch.full((rows, hq), 7.0, device="cuda")
    scale = 1.0 / d ** 0.5

    def call():
        return tts.attn_decode_paged(
            dev(q), kc, vc, dev(tables), dev(torch.tensor(kv, dtype=torch.int32)), scale,
            cu_seqlens_q=None if one else dev(torch.tensor(cu)),
            max_seqlen_q=max_q or max(new + [1]), k_scale=ks, v_scale=vs, window=window,
            sinks=sinks, out=out, lse=lse, status=st)

    call()
    tts.check_status(st)
    ro, rl, tol, tol_l = ref.attend(
        q[:T].float().numpy(), ref.codes_of(pool[0]), ref.codes_of(pool[2]),
        None if ks is None else pool[1].numpy(), None if vs is None else pool[3].numpy(),
        tables.numpy(), kv, cu, scale, window, sinks, F16_HALF if f8 else BF16_HALF)
    if out_dtype == torch.bfloat16:
        tol = tol + (np.abs(ro) + tol) * BF16_HALF
    o, l = out.float().cpu().numpy(), lse.cpu().numpy()
    assert (o[:front] == 7).all() and (l[:front] == 7).all()  # rows in front of the first
    o[:front], l[:front] = ro[:front], rl[:front]
    assert np.array_equal(np.isneginf(l[:T]), np.isneginf(rl))
    fin = np.isfinite(rl)
    assert np.all(np.abs(l[:T][fin] - rl[fin]) <= tol_l[fin]), np.abs(l[:T][fin] - rl[fin]).max()
    err = np.abs(o[:T] - ro)
    assert np.all(err <= tol), f"{(err / np.maximum(tol, 1e-30)).max()} of the bound"
    assert bool((out[T:] == 7).all()) and bool((lse[T:] == 7).all())  # rows behind the last
    a, b = out.clone(), lse.clone()
    call()
    assert torch.equal(a, out) and torch.equal(b, lse)  # the same bits again
    return float((err / np.maximum(tol, 1e-30)).max())


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("new,kv,hq,hkv,d,ps,window,sinks", [
    ([1, 1, 1, 1], [1, 64, 65, 700], 8, 2, 128, 64, 0, 0),
    ([1, 1, 1], [0, 31, 2590], 4, 4, 128, 16, 0, 0),             # an empty cache, MHA
    ([1], [4000], 8, 1, 64, 128, 0, 0),                          # one group of eight, one request
    ([1, 1], [513, 129], 16, 1, 64, 32, 0, 0),                   # 16 heads to one KV head
    ([1, 1, 1], [40, 500, 1500], 32, 1, 128, 32, 0, 0),          # 32 heads: several row tiles
    ([3, 1, 0, 6], [3, 100, 50, 641], 4, 2, 128, 64, 0, 0),      # drafts; one without new tokens
    ([5, 2], [2, 300], 10, 2, 64, 16, 0, 0),                     # more new tokens than keys
    ([64], [400], 2, 1, 128, 64, 0, 0),                          # the most new tokens
    ([1, 1, 1, 1], [1000, 90, 17, 3000], 8, 2, 128, 64, 100, 4),
    ([1, 1, 1], [777, 2000, 64], 5, 1, 64, 16, 33, 0),           # window without sinks
    ([4, 3, 1], [900, 1200, 300], 8, 4, 128, 32, 64, 70),        # sinks over a tile border
    ([2, 1], [1500, 1300], 4, 2, 64, 128, 1, 1),                 # only itself and the first
    ([1, 1], [600, 200], 4, 2, 128, 64, 500, 300),               # sinks meet the window
    ([1], [300], 4, 2, 128, 64, 2 ** 31 - 1, 2 ** 31 - 1),
    ([6, 1, 3], [700, 80, 2000], 16, 2, 128, 64, 0, 0),          # 48, 8 and 24 rows of a unit
    ([6, 4, 0, 5], [1300, 40, 9, 500], 12, 2, 64, 32, 200, 4),   # 36 rows, a window per token
    ([9, 2], [1000, 300], 20, 2, 128, 16, 0, 0),                 # 90 rows: two units
])
def test_decode_parity(tts, f8, new, kv, hq, hkv, d, ps, window, sinks):
    run_decode(tts, sum(kv) + ps, new, kv, hq, hkv, d, ps, f8, window, sinks)


@pytest.mark.parametrize("f8", [True, False])
def test_decode_many_requests_bf16_out(tts, f8):
    r = np.random.default_rng(3)
    kv = [int(x) for x in r.integers(1, 900, 200)]
    run_decode(tts, 20, [1] * 200, kv, 4, 2, 128, 64, f8, out_dtype=torch.bfloat16, one=True)


@pytest.mark.parametrize("f8", [True, False])
def test_decode_one_long_request(tts, f8):
    """One KV head of one request over the whole GPU: hundreds of parts joined."""
    run_decode(tts, 25, [1], [40000], 2, 1, 128, 64, f8)
    run_decode(tts, 26, [6], [20000], 8, 1, 64, 16, f8)


def test_decode_queries_of_any_size(tts):
    """The q rows' power-of-two scaling: tiny, large and zero queries."""
    for gain in (0.0, 1e-12, 40.0):
        run_decode(tts, 30, [1, 2], [300, 65], 4, 2, 128, 64, True, q_gain=gain)


def test_decode_first_key_far_above_the_rest(tts):
    """A first token with a score far above the others (an attention sink) keeps the weights of
    the rest at full precision: they carry the result when the sink's value is zero."""
    d, ps, L, hkv = 128, 64, 3000, 1
    tables, pages = make_tables(40, [L], ps)
    kc, ks, vc, vs = make_pool(41, pages, hkv, ps, d, True, spread=False)
    q = torch.randn(1, 4, d, generator=gen(42)).to(torch.bfloat16)
    q[:, :, 0] = 8.0
    first = int(tables[0, 0])
    kv = kc.view(torch.float8_e4m3fn).float()
    kv[first, 0, 0] = 0
    kv[first, 0, 0, 0] = 448.0  # score 448 / 64 * 8 / sqrt(128) * 2: about 10 above
    ks[first] = 2.0 ** -5
    kc = kv.to(torch.float8_e4m3fn).view(torch.uint8)
    vv = vc.view(torch.float8_e4m3fn).float()
    vv[first, 0, 0] = 0
    vc = vv.to(torch.float8_e4m3fn).view(torch.uint8)
    out, lse = tts.attn_decode_paged(dev(q), dev(kc), dev(vc), dev(tables),
                                     torch.tensor([L], dtype=torch.int32, device="cuda"),
                                     d ** -0.5, k_scale=dev(ks), v_scale=dev(vs))
    ro, rl, tol, tol_l = ref.attend(q.float().numpy(), ref.codes_of(kc), ref.codes_of(vc),
                                    ks.numpy(), vs.numpy(), tables.numpy(), [L], cum([1]),
                                    d ** -0.5, 0, 0, F16_HALF)
    assert np.all(np.abs(out.cpu().numpy() - ro) <= tol)
    assert np.all(np.abs(lse.cpu().numpy() - rl) <= tol_l)


def test_decode_value_scales_far_apart(tts):
    """Pages whose value scales differ by 2^40: their weights share the fp16 product."""
    d, ps, L, hkv = 64, 16, 500, 2
    tables, pages = make_tables(50, [L], ps)
    kc, ks, vc, vs = make_pool(51, pages, hkv, ps, d, True)
    vs = torch.exp2(torch.randint(-20, 21, vs.shape, generator=gen(52)).float()) * 1.5
    q = torch.randn(1, 4, d, generator=gen(53)).to(torch.bfloat16)
    out, lse = tts.attn_decode_paged(dev(q), dev(kc), dev(vc), dev(tables),
                                     torch.tensor([L], dtype=torch.int32, device="cuda"),
                                     d ** -0.5, k_scale=dev(ks), v_scale=dev(vs))
    ro, rl, tol, tol_l = ref.attend(q.float().numpy(), ref.codes_of(kc), ref.codes_of(vc),
                                    ks.numpy(), vs.numpy(), tables.numpy(), [L], cum([1]),
                                    d ** -0.5, 0, 0, F16_HALF)
    assert np.all(np.abs(out.cpu().numpy() - ro) <= tol)
    assert np.all(np.abs(lse.cpu().numpy() - rl) <= tol_l)


def test_decode_skips_and_reports(tts):
    d, ps, hkv = 128, 64, 2
    kv = [200, 300, 150]
    tables, pages = make_tables(60, kv, ps)
    kc, ks, vc, vs = make_pool(61, pages, hkv, ps, d, True)
    q = torch.randn(3, 4, d, generator=gen(62)).to(torch.bfloat16)

    def run(tables=tables, kv=kv, ks=ks, cu=None, max_q=1):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = tts.attn_decode_paged(
            dev(q), dev(kc), dev(vc), dev(tables), dev(torch.tensor(kv, dtype=torch.int32)),
            d ** -0.5, cu_seqlens_q=None if cu is None else dev(torch.tensor(cu, dtype=torch.int32)),
            max_seqlen_q=max_q, k_scale=dev(ks), v_scale=dev(vs), status=st,
            out=torch.full((3, 4, d), 7.0, device="cuda"))
        return out.cpu().numpy(), lse.cpu().numpy(), int(st.item())

    def want(tables=tables, bad=lambda pg: False):
        return ref.attend(q.float().numpy(), ref.codes_of(kc), ref.codes_of(vc), ks.numpy(),
                          vs.numpy(), tables.numpy(), kv, cum([1, 1, 1]), d ** -0.5, 0, 0,
                          F16_HALF, bad)

    t = tables.clone()
    t[1, 1] = pages  # no such page: its keys are skipped
    o, l, st = run(tables=t)
    assert st == tts.TTS_DEV_INDEX_RANGE
    ro, rl, tol, tol_l = want(t, lambda pg: pg >= pages)
    assert np.all(np.abs(o - ro) <= tol) and np.all(np.abs(l - rl) <= tol_l)
    bad = ks.clone()
    pg = int(tables[2, 0])
    bad[pg] = 0.0
    o, l, st = run(ks=bad)
    assert st == tts.TTS_DEV_BAD_ARG
    ro, rl, tol, tol_l = want(bad=lambda x: x == pg)
    assert np.all(np.abs(o - ro) <= tol) and np.all(np.abs(l - rl) <= tol_l)
    for L in (-1, ps * tables.shape[1] + 1):
        o, l, st = run(kv=[200, L, 150])
        assert st == tts.TTS_DEV_INDEX_RANGE
        assert not o[1].any() and np.isneginf(l[1]).all()
        ro, rl, tol, _ = want()
        assert np.all(np.abs(o[0] - ro[0]) <= tol[0]) and np.all(np.abs(o[2] - ro[2]) <= tol[2])
    o, l, st = run(cu=[0, 1, 0, 1])  # decreasing: that request is skipped, its row untouched
    assert st == tts.TTS_DEV_BAD_ARG and (o[1:] == 7).all()
    o, l, st = run(cu=[0, 1, 3, 3], max_q=1)  # longer than max_seqlen_q
    assert st == tts.TTS_DEV_BAD_ARG and (o[1:] == 7).all()


# ------------------------------------------------------------------------------- together
@pytest.mark.parametrize("f8", [True, False])
def test_serving_loop(tts, f8):
    """Prompts appended, then steps of one and of a few tokens, each appended and attended:
    every step against 64-bit attention over the cache's own values."""
    hq, hkv, d, ps, window, sinks = 8, 2, 128, 32, 96, 4
    new0, steps = [70, 33, 129], [1, 3, 1, 1, 2]
    total = [n + sum(steps) for n in new0]
    tables, pages = make_tables(70, total, ps)
    kc, ks, vc, vs = [None if t is None else dev(t) for t in make_pool(71, pages, hkv, ps, d, f8)]
    cs = tts.rope_cache(max(total), d)
    g = gen(72)
    T = dev(tables)
    past = [0, 0, 0]
    for step, n in enumerate([None] + steps):
        new = new0 if n is None else [n] * 3
        cu = cum(new)
        qkv = dev(torch.randn(int(cu[-1]), hq + 2 * hkv, d, generator=g).to(torch.bfloat16))
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        q, _ = tts.rope_kv_append(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], kc, vc, T,
                                  dev(torch.tensor(past, dtype=torch.int32)), dev(torch.tensor(cu)),
                                  max(new), k_scale=ks, v_scale=vs, cos_sin=cs, q=qkv[:, :hq],
                                  status=st)
        past = [p + m for p, m in zip(past, new)]
        if n is None:
            continue
        out, lse = tts.attn_decode_paged(q, kc, vc, T, dev(torch.tensor(past, dtype=torch.int32)),
                                         d ** -0.5, cu_seqlens_q=dev(torch.tensor(cu)),
                                         max_seqlen_q=max(new), k_scale=ks, v_scale=vs,
                                         window=window, sinks=sinks, status=st)
        tts.check_status(st)
        ro, rl, tol, tol_l = ref.attend(
            q.float().cpu().numpy(), ref.codes_of(kc), ref.codes_of(vc),
            None if ks is None else ks.cpu().numpy(), None if vs is None else vs.cpu().numpy(),
            tables.numpy(), past, cu, d ** -0.5, window, sinks, F16_HALF if f8 else BF16_HALF)
        assert np.all(np.abs(out.cpu().numpy() - ro) <= tol), step
        assert np.all(np.abs(lse.cpu().numpy() - rl) <= tol_l), step


# ------------------------------------------------------------------------------- as used
def test_append_many_requests(tts):
    """More requests than one round of bounds finds, prompts and steps, empty ones among them."""
    r = np.random.default_rng(5)
    for hi, ps, d in ((30, 16, 64), (2, 64, 128)):
        new = [int(x) for x in r.integers(0, hi, 75)]
        past = [int(x) for x in r.integers(0, 70, 75)]
        new[-1] = hi - 1
        c, q_out, k_out, (qr, kr, kc, vc, ks, vs), n = run_append(tts, 81, new, past, 4, 2, d, ps, True)
        assert torch.equal(q_out.cpu(), torch.tensor(qr).to(torch.bfloat16))
        assert torch.equal(k_out.cpu(), torch.tensor(kr).to(torch.bfloat16))
        np.testing.assert_array_equal(c[1].cpu().numpy(), ks.astype(np.float32))
        np.testing.assert_array_equal(ref.codes_of(c[0]), kc)
        np.testing.assert_array_equal(ref.codes_of(c[2]), vc)


@pytest.mark.parametrize("f8", [True, False])
def test_cache_beyond_32_bits(tts, f8):
    """The last pages of a cache whose offsets pass 2^31 values and 2^32 bytes."""
    hkv, ps, d = 4, 128, 128
    pages = (5 << 30 if f8 else 5 << 29) // (hkv * ps * d) + 1
    kc, vc = (torch.empty(pages, hkv, ps, d, dtype=torch.uint8 if f8 else torch.bfloat16,
                          device="cuda") for _ in range(2))
    ks, vs = ((torch.ones(pages, hkv, device="cuda") for _ in range(2)) if f8 else (None, None))
    assert kc.numel() > 2 ** 31 and kc.nbytes > 2 ** 32
    n = 200
    tables = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32)
    x = torch.randn(n, 4 + 2 * hkv, d, generator=gen(90)).to(torch.bfloat16)
    D = dev(x)
    q, _ = tts.rope_kv_append(D[:, 4:4 + hkv], D[:, 4 + hkv:], kc, vc, dev(tables),
                              torch.zeros(1, dtype=torch.int32, device="cuda"),
                              torch.tensor([0, n], dtype=torch.int32, device="cuda"), n, k_scale=ks,
                              v_scale=vs, q=D[:, :4].contiguous())
    last = [t[-2:] if t is not None else None for t in (kc, vc, ks, vs)]
    want = ref.append(None, x[:, 4:4 + hkv].float().numpy(), x[:, 4 + hkv:].float().numpy(),
                      np.zeros((2, hkv, ps, d)), np.zeros((2, hkv, ps, d)),
                      np.ones((2, hkv)) if f8 else None, np.ones((2, hkv)) if f8 else None,
                      np.array([[1, 0]]), [0], cum([n]), None, ps)
    got = ref.codes_of(last[0])
    np.testing.assert_array_equal(got[1], want[2][1])
    np.testing.assert_array_equal(got[0][:, :n - ps], want[2][0][:, :n - ps])
    out, lse = tts.attn_decode_paged(q[-1:].contiguous(), kc, vc, dev(tables),
                                     torch.tensor([n], dtype=torch.int32, device="cuda"), d ** -0.5,
                                     k_scale=ks, v_scale=vs)
    ro, rl, tol, tol_l = ref.attend(
        q[-1:].float().cpu().numpy(), got, ref.codes_of(last[1]),
        None if ks is None else last[2].cpu().numpy(), None if vs is None else last[3].cpu().numpy(),
        np.array([[1, 0]]), [n], cum([1]), d ** -0.5, 0, 0, F16_HALF if f8 else BF16_HALF)
    assert np.all(np.abs(out.cpu().numpy() - ro) <= tol)
    assert np.all(np.abs(lse.cpu().numpy() - rl) <= tol_l)


def test_step_in_a_graph(tts):
    """Append and decode captured once, replayed as the lengths grow and on two graphs that share
    the workspace: the same bits as the same calls made one by one."""
    hq, hkv, d, ps, nreq = 8, 2, 128, 16, 3
    tables, pages = make_tables(95, [100] * nreq, ps)
    pool = make_pool(96, pages, hkv, ps, d, True)
    cs = tts.rope_cache(100, d)
    T = dev(tables)
    cu = torch.arange(nreq + 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(tts.attn_decode_workspace_bytes(1, hq, hkv, d), dtype=torch.uint8, device="cuda")
    steps = [dev(torch.randn(nreq, hq + 2 * hkv, d, generator=gen(97 + i)).to(torch.bfloat16))
             for i in range(6)]

    def state():
        return dict(c=[dev(t).clone() for t in pool], qkv=steps[0].clone(),
                    past=torch.tensor([5, 31, 60], dtype=torch.int32, device="cuda"),
                    lens=torch.tensor([6, 32, 61], dtype=torch.int32, device="cuda"),
                    q=torch.empty(nreq, hq, d, dtype=torch.bfloat16, device="cuda"),
                    out=torch.empty(nreq, hq, d, device="cuda"),
                    lse=torch.empty(nreq, hq, device="cuda"))

    def step(s):
        kc, ks, vc, vs = s["c"]
        x = s["qkv"]
        tts.rope_kv_append(x[:, hq:hq + hkv], x[:, hq + hkv:], kc, vc, T, s["past"], cu, 1, k_scale=ks,
                           v_scale=vs, cos_sin=cs, q=x[:, :hq], q_out=s["q"])
        tts.attn_decode_paged(s["q"], kc, vc, T, s["lens"], d ** -0.5, k_scale=ks, v_scale=vs,
                              window=40, sinks=2, out=s["out"], lse=s["lse"], workspace=ws)
        s["past"].add_(1)
        s["lens"].add_(1)

    plain, want = state(), []
    for x in steps:
        plain["qkv"].copy_(x)
        step(plain)
        want.append((plain["out"].clone(), plain["lse"].clone()))
    step(state())  # what a first call sets up is not captured
    torch.cuda.synchronize()
    held = [state(), state()]
    graphs = []
    for s in held:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(s)
        graphs.append(g)
    for i, x in enumerate(steps):
        for s, g in zip(held, graphs):
            s["qkv"].copy_(x)
            g.replay()
        for s in held:
            assert torch.equal(s["out"], want[i][0]) and torch.equal(s["lse"], want[i][1]), i
    for s in held:
        assert all(torch.equal(a, b) for a, b in zip(s["c"], plain["c"]))


@pytest.mark.parametrize("f8", [True, False])
def test_bounds_above_the_lengths(tts, f8):
    """max_seqlen_q and max_new are bounds: single tokens through the kernels for many rows."""
    for max_q in (3, 9, 64):
        run_decode(tts, 140, [1, 2, 0, 1], [300, 65, 40, 1], 8, 2, 128, 64, f8, max_q=max_q)
        run_decode(tts, 141, [1, 1], [700, 33], 8, 2, 64, 16, f8, window=50, sinks=3, max_q=max_q)
    for max_new in (2, 5, 100):
        c, q_out, k_out, (qr, kr, kc, vc, ks, vs), n = run_append(
            tts, 142, [1, 0, 1, 1], [5, 9, 63, 64], 4, 2, 128, 64, f8, max_new=max_new)
        assert torch.equal(q_out.cpu(), torch.tensor(qr).to(torch.bfloat16))
        if f8:
            np.testing.assert_array_equal(ref.codes_of(c[0]), kc)
            np.testing.assert_array_equal(c[3].cpu().numpy(), vs.astype(np.float32))
        else:
            assert torch.equal(c[2].cpu(), torch.tensor(vc).float().to(torch.bfloat16))


@pytest.mark.parametrize("front", [1, 37, 300])
def test_rows_in_front_of_the_first_request(tts, front):
    """cu_new / cu_seqlens_q begin above 0: the rows in front belong to nobody."""
    for new, past in (([1, 2, 1], [0, 63, 100]), ([70, 0, 130], [0, 5, 61])):
        c, q_out, k_out, (qr, kr, kc, vc, ks, vs), n = run_append(
            tts, 150, new, past, 4, 2, 128, 64, True, pad_rows=2, front=front)
        for got, want in ((q_out, qr), (k_out, kr)):
            assert bool((got[:front] == 7).all()) and bool((got[n:] == 7).all())
            assert torch.equal(got[front:n].cpu(), torch.tensor(want[front:]).to(torch.bfloat16))
        np.testing.assert_array_equal(ref.codes_of(c[0]), kc)
        np.testing.assert_array_equal(ref.codes_of(c[2]), vc)
    run_decode(tts, 151, [1, 2, 0, 3], [300, 65, 40, 3], 8, 2, 128, 64, True, front=front)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("f8", [True, False])
def test_units_of_mixed_rows(tts, d, f8):
    """Requests of 1 to 64 new tokens side by side: a CTA goes from units of one number of row
    groups to another's, over and over; every call gives the same bits."""
    g = gen(160)
    new = torch.randint(0, 65, (60,), generator=g).tolist()
    new[::3] = [min(n, 5) for n in new[::3]]
    kv = [max(n, int(x)) for n, x in zip(new, torch.randint(1, 200, (60,), generator=g))]
    run_decode(tts, 161, new, kv, 10, 2, d, 64, f8, max_q=64)
    tables, pages = make_tables(162, kv, 64)
    kc, ks, vc, vs = [None if t is None else dev(t) for t in make_pool(163, pages, 2, 64, d, f8)]
    q = dev(torch.randn(sum(new), 10, d, generator=g).to(torch.bfloat16))
    cu, lens = dev(torch.tensor(cum(new))), dev(torch.tensor(kv, dtype=torch.int32))
    tables = dev(tables)
    first = None
    for _ in range(300):
        got = tts.attn_decode_paged(q, kc, vc, tables, lens, 0.1, cu_seqlens_q=cu,
                                    max_seqlen_q=64, k_scale=ks, v_scale=vs)
        if first is None:
            first = got
        assert torch.equal(first[0], got[0]) and torch.equal(first[1], got[1])


def test_calls_on_two_streams(tts):
    """Two decode calls in flight at once, each with a workspace of its own."""
    d, ps, hkv, kv = 128, 64, 2, [9000, 500]
    tables, pages = make_tables(110, kv, ps)
    kc, ks, vc, vs = [dev(t) for t in make_pool(111, pages, hkv, ps, d, True)]
    T, L = dev(tables), dev(torch.tensor(kv, dtype=torch.int32))
    qs = [dev(torch.randn(2, 8, d, generator=gen(112 + i)).to(torch.bfloat16)) for i in range(2)]
    need = tts.attn_decode_workspace_bytes(1, 8, hkv, d)
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    call = lambda i: tts.attn_decode_paged(qs[i], kc, vc, T, L, d ** -0.5, k_scale=ks, v_scale=vs,  # noqa: E731
                                           workspace=ws[i])
    want = [tuple(t.clone() for t in call(i)) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(call(i))
    torch.cuda.synchronize()
    for i in range(2):
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


def test_workspace_is_found_or_made(tts):
    """Without a workspace, and with one that is too small, the binding makes one."""
    tables, pages = make_tables(120, [300], 64)
    kc, ks, vc, vs = [dev(t) for t in make_pool(121, pages, 2, 64, 128, True)]
    q = dev(torch.randn(1, 4, 128, generator=gen(122)).to(torch.bfloat16))
    L = torch.tensor([300], dtype=torch.int32, device="cuda")
    a = tts.attn_decode_paged(q, kc, vc, dev(tables), L, 0.1, k_scale=ks, v_scale=vs)
    b = tts.attn_decode_paged(q, kc, vc, dev(tables), L, 0.1, k_scale=ks, v_scale=vs,
                              workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_binding_refuses_tensors_that_do_not_fit(tts):
    tables, pages = make_tables(130, [100], 64)
    kc, ks, vc, vs = [dev(t) for t in make_pool(131, pages, 2, 64, 128, True)]
    T, L = dev(tables), torch.tensor([100], dtype=torch.int32, device="cuda")
    q = dev(torch.randn(1, 4, 128, generator=gen(132)).to(torch.bfloat16))
    good = dict(q=q, k_cache=kc, v_cache=vc, page_tables=T, kv_lens=L, scale=0.1, k_scale=ks,
                v_scale=vs)
    tts.attn_decode_paged(**good)
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:, :, :64]), dict(k_cache=kc[:-1]),
                dict(k_cache=kc.view(torch.int8)), dict(k_scale=None), dict(v_scale=vs[:, :1]),
                dict(page_tables=T.long()), dict(page_tables=T[0]), dict(kv_lens=L.cpu()),
                dict(kv_lens=torch.cat([L, L])), dict(cu_seqlens_q=L), dict(out=q.half()),
                dict(out=torch.empty(2, 4, 128, device="cuda")), dict(lse=torch.empty(4, device="cuda")),
                dict(v_cache=vc.transpose(1, 2)), dict(status=torch.zeros(1, device="cuda"))):
        with pytest.raises(ValueError):
            tts.attn_decode_paged(**{**good, **bad})
    for bad in (dict(scale=0.0), dict(window=-1), dict(max_seqlen_q=65)):
        with pytest.raises(tts.TTSError):
            tts.attn_decode_paged(**{**good, **bad})
    k = dev(torch.randn(3, 2, 128, generator=gen(133)).to(torch.bfloat16))
    cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    good = dict(k=k, v=k, k_cache=kc, v_cache=vc, page_tables=T, past_lens=L, cu_new=cu, max_new=3,
                k_scale=ks, v_scale=vs)
    tts.rope_kv_append(**good)
    for bad in (dict(k=k.float()), dict(v=k[:2]), dict(k=k[:, :1]), dict(k=k.transpose(0, 1)),
                dict(q=k[:2]), dict(q_out=k), dict(k_out=k[:2]), dict(cu_new=cu.long()),
                dict(cu_new=cu[:1]), dict(cos_sin=torch.zeros(9, 32, 2, device="cuda")),
                dict(past_lens=L.cpu()), dict(v_scale=None)):
        with pytest.raises(ValueError):
            tts.rope_kv_append(**{**good, **bad})
    with pytest.raises(tts.TTSError):
        tts.rope_kv_append(**{**good, "max_new": -1})
