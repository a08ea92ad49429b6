"""GPU parity for tts_attn_fwd_varlen_window: sliding-window prefill with first tokens that stay
visible against 64-bit attention, row by row, and against the plain causal entry point where
the window holds every key."""
import numpy as np
import pytest
import torch

import gqa_ref as ref

pytestmark = pytest.mark.gpu

BF16_HALF = 2.0 ** -8


@pytest.fixture(scope="module")
def tts():
    import tiled_top_sparse_gb300 as m
    m.lib()
    return m


def cum(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def inputs(seed, lq, lk, hq, hkv, d, dtype, tail=0):
    """q, k, v on the device; `tail` rows behind the last sequence hold NaN."""
    g = torch.Generator("cpu")
    g.manual_seed(seed)
    t = [torch.randn(int(sum(n)) + tail, h, d, generator=g) for n, h in ((lq, hq), (lk, hkv),
                                                                         (lk, hkv))]
    for x in t:
        if tail:
            x[-tail:] = float("nan")
    return [x.to(dtype).cuda() for x in t]


def check(tts, seed, lq, lk, hq, hkv, d, window, sinks, dtype=torch.bfloat16,
          out_dtype=torch.float32, tail=5, out_at=0):
    lk = lq if lk is None else lk
    q, k, v = inputs(seed, lq, lk, hq, hkv, d, dtype, tail)
    cq, ck = cum(lq), cum(lk)
    T = int(cq[-1])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    flat = torch.full((out_at + q.numel() + 64,), 7.0, dtype=out_dtype, device="cuda")
    out = flat[out_at:out_at + q.numel()].view(q.shape)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")

    def call():
        return tts.attn_fwd_varlen_window(q, k, v, torch.tensor(cq).cuda(), torch.tensor(ck).cuda(),
                                          max(lq), max(lk), window, sinks, d ** -0.5, out=out,
                                          lse=lse, status=st)

    call()
    tts.check_status(st)
    h = [x.to(torch.bfloat16).float().cpu().numpy() for x in (q, k, v)]
    ro, rl, tol, tol_l = ref.attend_packed(h[0][:T], h[1], h[2], cq, ck, d ** -0.5, window, sinks,
                                           BF16_HALF)
    if out_dtype == torch.bfloat16:
        tol = tol + (np.abs(ro) + tol) * BF16_HALF
    o, l = out.float().cpu().numpy(), lse.cpu().numpy()
    assert np.array_equal(np.isneginf(l[:T]), np.isneginf(rl))
    fin = np.isfinite(rl)
    assert np.all(np.abs(l[:T][fin] - rl[fin]) <= tol_l[fin])
    err = np.abs(o[:T] - ro)
    assert np.all(err <= tol), (err - tol).max()
    assert (o[T:] == 7).all() and (l[T:] == 7).all()
    assert bool((flat[:out_at] == 7).all()) and bool((flat[out_at + q.numel():] == 7).all())
    a, b = out.clone(), lse.clone()
    call()
    assert torch.equal(a, out) and torch.equal(b, lse)


@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("lq,lk,hq,hkv,window,sinks", [
    ([700], None, 4, 2, 256, 4),
    ([1, 129, 385, 256], None, 2, 1, 100, 0),          # ragged; a window inside a tile
    ([1000], None, 2, 2, 1, 1),                        # only itself and the first
    ([900, 300], None, 3, 1, 300, 130),                # sinks over a tile border
    ([640], None, 2, 1, 128, 300),                     # sinks meet the window
    ([257], None, 2, 1, 10 ** 9, 0),                   # no key ever leaves
    ([100, 260], [700, 900], 4, 1, 200, 5),            # new tokens behind cached keys
    ([300, 200], [120, 1], 2, 1, 64, 2),               # more rows than keys: rows that see none
    ([0, 200, 0], [5, 200, 0], 2, 2, 50, 3),           # empty sequences
])
def test_window_parity(tts, d, lq, lk, hq, hkv, window, sinks):
    check(tts, sum(lq) + d, lq, lk, hq, hkv, d, window, sinks)


@pytest.mark.parametrize("d", [64, 80, 128])
def test_bf16_out_and_fp32_in(tts, d):
    check(tts, 5, [333, 70], None, 4, 2, d, 96, 4, out_dtype=torch.bfloat16)
    check(tts, 6, [333, 70], None, 4, 2, d, 96, 4, dtype=torch.float32)


@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_rows_that_end_inside_a_store(tts, d, out_dtype):
    """Rows leave 32 at a time: lengths around multiples of 32 and 128, an output that begins at 16
    bytes of a line, with few and with many items per CTA."""
    at = 4 if out_dtype == torch.float32 else 8
    check(tts, 20, [1, 31, 32, 33, 127, 128, 129, 159, 160], None, 4, 2, d, 70, 2,
          out_dtype=out_dtype, out_at=at)
    check(tts, 21, [481, 672, 95, 800, 1], None, 24, 6, d, 150, 9, out_dtype=out_dtype, out_at=at)
    check(tts, 22, [481, 95, 64], [490, 30, 700], 15, 5, d, 150, 9, out_dtype=out_dtype, tail=0)


def test_captured(tts):
    """Two graphs of windowed calls with workspaces of their own, replayed in turn and over new
    inputs, give what the calls give."""
    cases = []
    for lens, hq, d in (([700], 4, 64), ([900, 300, 411], 32, 128)):
        q, k, v = inputs(23, lens, lens, hq, 2, d, torch.bfloat16)
        cu = torch.tensor(cum(lens)).cuda()
        out, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:2], device="cuda")
        ws = torch.empty(256, dtype=torch.uint8, device="cuda")

        def call(q=q, k=k, v=v, cu=cu, lens=lens, d=d, out=out, lse=lse, ws=ws):
            tts.attn_fwd_varlen_window(q, k, v, cu, cu, max(lens), max(lens), 200, 4, d ** -0.5,
                                       out=out, lse=lse, workspace=ws)

        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        cases.append((g, call, q, out, lse))
    for turn in range(3):
        for g, call, q, out, lse in cases:
            q.copy_(torch.roll(q, turn + 1, 0))
            out.fill_(7)
            g.replay()
        for g, call, q, out, lse in cases:
            a, b = out.clone(), lse.clone()
            call()
            assert torch.equal(a, out) and torch.equal(b, lse)


def test_many_items_per_cta(tts):
    """More items than CTAs: the ring, the Q tiles and the accumulators are reused."""
    check(tts, 7, [1500, 700, 1100], None, 16, 4, 128, 300, 4)
    check(tts, 8, [1200, 900], None, 32, 8, 64, 200, 130)
    check(tts, 11, [1500, 700], None, 15, 5, 128, 260, 4)   # an odd group: pairs of row tiles
    check(tts, 12, [1300, 500, 129], None, 12, 12, 80, 100, 1)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_items_that_start_late(tts, out_dtype):
    """Few items, most of which start after their neighbours have ended, because another stream
    holds the SMs: every item writes its own rows and no other's."""
    q, k, v = inputs(13, [1920], [1920], 8, 2, 64, torch.bfloat16)
    cu = torch.tensor([0, 1920], dtype=torch.int32).cuda()
    out = torch.empty(q.shape, dtype=out_dtype, device="cuda")
    lse = torch.empty(q.shape[:2], device="cuda")

    def call():
        tts.attn_fwd_varlen_window(q, k, v, cu, cu, 1920, 1920, 500, 4, 0.125, out=out, lse=lse)

    call()
    want, want_l = out.clone(), lse.clone()
    bq, bk, bv = inputs(14, [256], [40000], 120, 1, 128, torch.bfloat16)  # 120 long items
    cq, ck = (torch.tensor([0, n], dtype=torch.int32).cuda() for n in (256, 40000))
    busy = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(busy):
            tts.attn_fwd_varlen(bq, bk, bv, cq, ck, 256, 40000, False, 0.1)
        call()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_l)


@pytest.mark.parametrize("d", [64, 80, 128])
def test_wide_window_equals_causal(tts, d):
    """A window that holds every key takes the same tiles in the same order as the plain causal
    call: the same bits."""
    lens = [500, 129, 1, 300]
    q, k, v = inputs(9, lens, lens, 4, 2, d, torch.bfloat16)
    cu = torch.tensor(cum(lens)).cuda()
    a = tts.attn_fwd_varlen_window(q, k, v, cu, cu, 500, 500, 500, 3, d ** -0.5)
    b = tts.attn_fwd_varlen(q, k, v, cu, cu, 500, 500, True, d ** -0.5)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for hq, hkv in ((24, 6), (21, 7)):  # more tiles than SMs: pairs of heads, pairs of row tiles
        q, k, v = inputs(13, lens, lens, hq, hkv, d, torch.bfloat16)
        a = tts.attn_fwd_varlen_window(q, k, v, cu, cu, 500, 500, 500, 3, d ** -0.5)
        b = tts.attn_fwd_varlen(q, k, v, cu, cu, 500, 500, True, d ** -0.5)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_bounds_far_above_the_lengths(tts):
    """max_seqlen_q and max_seqlen_k are bounds: the largest int gives what the lengths give."""
    top = 2 ** 31 - 1
    for lens, hq, hkv, d in (([300, 129], 4, 2, 64), ([900, 411], 32, 8, 128), ([700, 500], 15, 5, 80)):
        q, k, v = inputs(24, lens, lens, hq, hkv, d, torch.bfloat16)
        cu = torch.tensor(cum(lens)).cuda()
        a = tts.attn_fwd_varlen_window(q, k, v, cu, cu, max(lens), max(lens), 200, 3, d ** -0.5)
        b = tts.attn_fwd_varlen_window(q, k, v, cu, cu, top, top, 200, 3, d ** -0.5)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_bad_sequences_are_reported(tts):
    q, k, v = inputs(10, [100, 100], [100, 100], 2, 1, 64, torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 100, 201], dtype=torch.int32, device="cuda")  # past the end
    out = torch.full(q.shape, 7.0, device="cuda")
    tts.attn_fwd_varlen_window(q, k, v, cu, cu, 101, 101, 30, 2, 0.125, out=out, status=st)
    assert int(st.item()) == tts.TTS_DEV_BAD_ARG
    assert bool((out[100:] == 7).all()) and not bool((out[:100] == 7).all())


@pytest.mark.parametrize("f8", [True, False])
def test_prefill_then_decode(tts, f8):
    """A prompt through append and windowed prefill, then decode steps over the cache: the
    prefill's rows equal 64-bit attention over its rotated keys, the steps' rows over the cache."""
    hq, hkv, d, ps, window, sinks = 8, 2, 128, 64, 200, 4
    lens, steps = [500, 77, 260], 3
    pages = sum(-(-(n + steps) // ps) for n in lens)
    tables = torch.full((3, 10), -1, dtype=torch.int32)
    perm = torch.randperm(pages, generator=torch.Generator("cpu").manual_seed(1)).int()
    at = 0
    for r, n in enumerate(lens):
        m = -(-(n + steps) // ps)
        tables[r, :m] = perm[at:at + m]
        at += m
    dt = torch.uint8 if f8 else torch.bfloat16
    kc, vc = (torch.zeros(pages, hkv, ps, d, dtype=dt, device="cuda") for _ in range(2))
    ks, vs = ((torch.zeros(pages, hkv, device="cuda") for _ in range(2)) if f8 else (None, None))
    cs = tts.rope_cache(600, d)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.Generator("cpu")
    g.manual_seed(2)
    past = [0, 0, 0]
    for step in range(steps + 1):
        new = lens if step == 0 else [1, 1, 1]
        cu = cum(new)
        qkv = torch.randn(int(cu[-1]), hq + 2 * hkv, d, generator=g).to(torch.bfloat16).cuda()
        v = qkv[:, hq + hkv:]
        q, k = tts.rope_kv_append(qkv[:, hq:hq + hkv], v, kc, vc, tables.cuda(),
                                  torch.tensor(past, dtype=torch.int32).cuda(),
                                  torch.tensor(cu).cuda(), max(new), k_scale=ks, v_scale=vs,
                                  cos_sin=cs, q=qkv[:, :hq], want_k=step == 0, status=st)
        past = [a + b for a, b in zip(past, new)]
        if step == 0:
            c = torch.tensor(cu).cuda()
            out, lse = tts.attn_fwd_varlen_window(q, k, v.contiguous(), c, c, max(new), max(new),
                                                  window, sinks, d ** -0.5, status=st)
            want = ref.attend_packed(q.float().cpu().numpy(), k.float().cpu().numpy(),
                                     v.float().cpu().numpy(), cu, cu, d ** -0.5, window, sinks,
                                     BF16_HALF)
        else:
            out, lse = tts.attn_decode_paged(q, kc, vc, tables.cuda(),
                                             torch.tensor(past, dtype=torch.int32).cuda(),
                                             d ** -0.5, k_scale=ks, v_scale=vs, window=window,
                                             sinks=sinks, status=st)
            want = ref.attend(q.float().cpu().numpy(), ref.codes_of(kc), ref.codes_of(vc),
                              None if ks is None else ks.cpu().numpy(),
                              None if vs is None else vs.cpu().numpy(), tables.numpy(), past, cu,
                              d ** -0.5, window, sinks, 2.0 ** -11 if f8 else BF16_HALF)
        tts.check_status(st)
        assert np.all(np.abs(out.cpu().numpy() - want[0]) <= want[2]), step
        assert np.all(np.abs(lse.cpu().numpy() - want[1]) <= want[3]), step
