"""GPU tests of the grouped-query calls at the edges of what their documentation allows."""
import math

import numpy as np
import pytest
import torch

import gqa_ref as ref
from test_gpu_gqa import F16_HALF, cum, dev, gen, make_pool, make_tables, run_append

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tts():
    import tiled_top_sparse_gb300 as m
    m.lib()
    return m


# ------------------------------------------------------------------------------- append
@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("hkv,batch,d", [(1, 1, 128), (1, 3, 64), (3, 1, 64), (3, 5, 128),
                                         (1, 33, 128)])
def test_append_step_without_q_odd_heads(tts, f8, hkv, batch, d):
    """One token per request, no q, an odd number of (request, KV head) pairs: the launch's last
    block has warps without a row."""
    past = [(17 * r) % 70 for r in range(batch)]
    c, _, k_out, (qr, kr, kc, vc, ks, vs), n = run_append(
        tts, 200 + batch, [1] * batch, past, 2, hkv, d, 16, f8, with_q=False, front=1, pad_rows=2)
    assert torch.equal(k_out[1:n].cpu(), torch.tensor(kr[1:]).to(torch.bfloat16))
    assert bool((k_out[:1] == 7).all()) and bool((k_out[n:] == 7).all())
    if f8:
        np.testing.assert_array_equal(ref.codes_of(c[0]), kc)
        np.testing.assert_array_equal(c[3].cpu().numpy(), vs.astype(np.float32))
    else:
        assert torch.equal(c[2].cpu(), torch.tensor(vc).float().to(torch.bfloat16))


def test_append_step_without_q_reads_no_bounds_in_front(tts):
    """cu_new and past_lens are the middle of larger tensors whose neighbours would make a request:
    it is nobody's, and the status stays clear."""
    hkv, d, ps = 1, 64, 16
    tables, pages = make_tables(210, [40], ps)
    pool = make_pool(211, pages, hkv, ps, d, True)
    x = torch.randn(2, hkv, d, generator=gen(212)).to(torch.bfloat16)
    c = [dev(t).clone() for t in pool]
    bounds = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    past = torch.tensor([7, 33], dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tts.rope_kv_append(dev(x), dev(x), c[0], c[2], dev(tables), past[1:], bounds[1:], 1,
                       k_scale=c[1], v_scale=c[3], status=st)
    assert int(st.item()) == 0
    want = ref.append(None, x.float().numpy(), x.float().numpy(), ref.codes_of(pool[0]),
                      ref.codes_of(pool[2]), pool[1].numpy(), pool[3].numpy(), tables.numpy(), [33],
                      cum([1]) + 1, None, ps)
    np.testing.assert_array_equal(ref.codes_of(c[0]), want[2])
    np.testing.assert_array_equal(ref.codes_of(c[2]), want[3])
    np.testing.assert_array_equal(c[1].cpu().numpy(), want[4].astype(np.float32))


def test_append_refuses_an_empty_rotation_table(tts):
    """A table without positions is not `no rotation`."""
    tables, pages = make_tables(250, [10], 16)
    kc, ks, vc, vs = [dev(t) for t in make_pool(251, pages, 1, 16, 64, True)]
    x = dev(torch.randn(1, 1, 64, generator=gen(252)).to(torch.bfloat16))
    with pytest.raises(ValueError):
        tts.rope_kv_append(x, x, kc, vc, dev(tables), torch.zeros(1, dtype=torch.int32, device="cuda"),
                           torch.tensor([0, 1], dtype=torch.int32, device="cuda"), 1, k_scale=ks,
                           v_scale=vs, cos_sin=torch.empty(0, 32, 2, device="cuda"))


# ------------------------------------------------------------------------------- decode
@pytest.mark.parametrize("tiny", [1e-40, 2.0 ** -149, 2.0 ** -128])
@pytest.mark.parametrize("new,kv,hq,hkv,d,ps,window,sinks", [
    ([1, 1], [20, 70], 8, 2, 128, 16, 0, 0),            # pages behind the end, inside its tile
    ([1, 1], [1, 33], 4, 2, 128, 32, 0, 0),
    ([1], [60], 4, 1, 64, 64, 0, 0),                    # two pages of 64 to a tile
    ([1, 1], [500, 300], 8, 2, 128, 16, 30, 4),         # between the first tokens and the window
    ([3, 2], [90, 700], 8, 2, 64, 16, 70, 1),
    ([6, 1], [300, 40], 16, 2, 128, 16, 50, 0),         # row groups
])
def test_decode_scales_of_unseen_pages(tts, tiny, new, kv, hq, hkv, d, ps, window, sinks):
    """Table entries without a visible key name a page of the pool that was never written: its
    scales are subnormal (small integers read as fp32), its codes NaN."""
    tables, pages = make_tables(sum(kv), kv, ps)
    kc, ks, vc, vs = make_pool(220, pages + 1, hkv, ps, d, True)
    ks[pages], vs[pages] = tiny, tiny
    kc[pages], vc[pages] = 0x7F, 0x7F
    tables = torch.cat([tables, torch.full((len(kv), 8), -1, dtype=torch.int32)], 1)
    for r, L in enumerate(kv):
        lo = max(0, L - new[r] + 1 - window) if window > 0 else 0
        for a in range(tables.shape[1]):
            j = np.arange(a * ps, (a + 1) * ps)
            if not ((j < L) & ((j >= lo) | (j < sinks))).any():
                tables[r, a] = pages
    cu = cum(new)
    q = torch.randn(int(cu[-1]), hq, d, generator=gen(221)).to(torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = tts.attn_decode_paged(
        dev(q), dev(kc), dev(vc), dev(tables), dev(torch.tensor(kv, dtype=torch.int32)), d ** -0.5,
        cu_seqlens_q=dev(torch.tensor(cu)), max_seqlen_q=max(new), k_scale=dev(ks), v_scale=dev(vs),
        window=window, sinks=sinks, status=st)
    assert int(st.item()) == 0
    ro, rl, tol, tol_l = ref.attend(q.float().numpy(), ref.codes_of(kc), ref.codes_of(vc),
                                    ks.numpy(), vs.numpy(), tables.numpy(), kv, cu, d ** -0.5,
                                    window, sinks, F16_HALF)
    assert np.all(np.abs(out.cpu().numpy() - ro) <= tol)
    assert np.all(np.abs(lse.cpu().numpy() - rl) <= tol_l)


@pytest.mark.parametrize("low,high,L", [(-80, -80, 40000), (-80, -60, 500), (-80, 20, 500),
                                        (0, 100, 500), (100, 100, 3000)])
def test_decode_value_scales_at_the_bounds(tts, low, high, L):
    """Value scales down to 2^-80 and pages 2^100 apart. The scale's log2 rides in the score, up to
    2^7 in size, so what is rounded there is rounded to half a step of 2^-17: the score with it, and
    log2 itself to one step. Both move a weight by a factor of 2^(3 x 2^-18) at most, once in the
    result's numerator and once in its denominator. lse adds the reference less its bias (half a
    step) and log2 of the sum (one step)."""
    d, ps, hkv = 64, 16, 1
    tables, pages = make_tables(230, [L], ps)
    kc, ks, vc, vs = make_pool(231, pages, hkv, ps, d, True)
    e = torch.randint(low, high + 1, vs.shape, generator=gen(232))
    e[0], e[1] = low, high
    # 1.5 times a power of two, the smallest exactly at the bound
    vs = torch.exp2(e.double()).float() * torch.where(e == low, 1.0, 1.5)
    q = torch.randn(1, 4, d, generator=gen(233)).to(torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = tts.attn_decode_paged(dev(q), dev(kc), dev(vc), dev(tables),
                                     torch.tensor([L], dtype=torch.int32, device="cuda"),
                                     d ** -0.5, k_scale=dev(ks), v_scale=dev(vs), status=st)
    assert int(st.item()) == 0
    ro, rl, tol, tol_l = ref.attend(q.float().numpy(), ref.codes_of(kc), ref.codes_of(vc),
                                    ks.numpy(), vs.numpy(), tables.numpy(), [L], cum([1]),
                                    d ** -0.5, 0, 0, F16_HALF)
    move = math.log(2) * 3 * 2.0 ** -18
    # tol's first part is at least F16_HALF of sum p|v| / l: its size, to add the factor to
    tol = tol * (1 + 2 * move / F16_HALF)
    assert np.all(np.abs(out.cpu().numpy() - ro) <= tol)
    assert np.all(np.abs(lse.cpu().numpy() - rl) <= tol_l + 2 * move)


@pytest.mark.parametrize("bad", [2.0 ** -81, 2.0 ** -118, 2.0 ** -130, 2.0 ** -149])
def test_decode_value_scale_below_the_bound(tts, bad):
    """A value scale too small for the denominator's range is reported and its page's keys are
    skipped, like a scale that is not positive; a request of such pages alone sees no key."""
    d, ps, hkv, kv = 128, 32, 2, [300, 200, 1]
    tables, pages = make_tables(240, kv, ps)
    kc, ks, vc, vs = make_pool(241, pages, hkv, ps, d, True)
    gone = [int(tables[0, 3]), int(tables[2, 0])]
    for pg in gone:
        vs[pg] = bad
    q = torch.randn(3, 4, d, generator=gen(242)).to(torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = tts.attn_decode_paged(dev(q), dev(kc), dev(vc), dev(tables),
                                     dev(torch.tensor(kv, dtype=torch.int32)), d ** -0.5,
                                     k_scale=dev(ks), v_scale=dev(vs), status=st)
    assert int(st.item()) == tts.TTS_DEV_BAD_ARG
    ro, rl, tol, tol_l = ref.attend(q.float().numpy(), ref.codes_of(kc), ref.codes_of(vc),
                                    ks.numpy(), vs.numpy(), tables.numpy(), kv, cum([1, 1, 1]),
                                    d ** -0.5, 0, 0, F16_HALF, lambda pg: pg in gone)
    assert np.all(np.abs(out.cpu().numpy() - ro) <= tol)
    l = lse.cpu().numpy()
    assert np.array_equal(np.isneginf(l), np.isneginf(rl)) and np.isneginf(l[2]).all()
    assert np.all(np.abs(l[:2] - rl[:2]) <= tol_l[:2])
