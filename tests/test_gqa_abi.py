"""CPU checks of the grouped-query entry points: bad host-side arguments are refused before any
CUDA call, and the 64-bit definitions agree with brute force."""
import ctypes

import numpy as np
import pytest
import torch

import gqa_ref as ref

A = ctypes.c_void_p(0x10000)   # 16-byte aligned, never dereferenced
B = ctypes.c_void_p(0x10008)   # misaligned
NUL = None


@pytest.fixture(scope="module")
def L():
    from tiled_top_sparse_gb300 import _build
    _build.build()
    import tiled_top_sparse_gb300 as tts
    return tts.lib()


def append(L, **kw):
    a = dict(q=A, qs=1024, hq=8, k=A, ks=256, v=A, vs=256, total=10, cu=A, past=A, batch=2,
             max_new=5, hkv=2, d=128, cs=A, max_pos=100, pt=A, max_pages=4, kc=A, vc=A, ksc=A,
             vsc=A, dt=2, pages=16, ps=64, qo=A, ko=A, st=NUL, stream=NUL)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.tts_rope_kv_append(*a.values())


def test_append_refusals(L):
    import tiled_top_sparse_gb300 as tts
    for n in ("k", "v", "cu", "past", "pt", "kc", "vc", "ksc", "vsc", "qo"):
        assert append(L, **{n: NUL}) == tts.TTS_ERR_INVALID_ARG, n
    for n in ("q", "k", "v", "kc", "vc", "qo", "ko", "cs"):
        assert append(L, **{n: B}) == tts.TTS_ERR_INVALID_ARG, n
    for kw in (dict(total=-1), dict(batch=0), dict(max_new=-1), dict(hkv=0), dict(d=0),
               dict(max_pages=0), dict(pages=0), dict(ps=0), dict(dt=1), dict(dt=3), dict(ks=255),
               dict(ks=260), dict(vs=128), dict(qs=1000), dict(qs=1028), dict(hq=0),
               dict(max_pos=0)):
        assert append(L, **kw) == tts.TTS_ERR_INVALID_ARG, kw
    for kw in (dict(d=80), dict(ps=48), dict(ps=8), dict(ps=256), dict(max_pages=1 << 25),
               dict(pages=2 ** 31 - 1)):
        assert append(L, **kw) == tts.TTS_ERR_UNSUPPORTED, kw
    assert append(L, total=0) == tts.TTS_OK          # nothing to append
    assert append(L, max_new=0, k=NUL) == tts.TTS_OK


def decode(L, **kw):
    a = dict(q=A, total=10, cu=A, batch=2, max_q=5, hq=8, hkv=2, d=128, kc=A, vc=A, ksc=A, vsc=A,
             dt=2, pages=16, ps=64, pt=A, max_pages=4, lens=A, window=0, sinks=0, scale=0.1,
             out=A, odt=1, lse=NUL, ws=A, wsb=1 << 30, st=NUL, stream=NUL)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.tts_attn_decode_paged(*a.values())


def test_decode_refusals(L):
    import tiled_top_sparse_gb300 as tts
    for n in ("q", "kc", "vc", "ksc", "vsc", "pt", "lens", "out"):
        assert decode(L, **{n: NUL}) == tts.TTS_ERR_INVALID_ARG, n
    for n in ("q", "kc", "vc", "out"):
        assert decode(L, **{n: B}) == tts.TTS_ERR_INVALID_ARG, n
    for kw in (dict(total=-1), dict(batch=0), dict(max_q=0), dict(hq=0), dict(hkv=3), dict(d=0),
               dict(pages=0), dict(ps=0), dict(max_pages=0), dict(window=-1), dict(sinks=-1),
               dict(scale=0.0), dict(scale=float("inf")), dict(dt=1), dict(odt=2),
               dict(cu=NUL, total=1)):
        assert decode(L, **kw) == tts.TTS_ERR_INVALID_ARG, kw
    for kw in (dict(d=80), dict(ps=24), dict(max_q=65), dict(max_pages=1 << 25),
               dict(batch=1 << 12, max_pages=1 << 23)):  # more tiles than 32 bits count
        assert decode(L, **kw) == tts.TTS_ERR_UNSUPPORTED, kw
    assert decode(L, ws=NUL) == tts.TTS_ERR_WORKSPACE
    assert decode(L, ws=B) == tts.TTS_ERR_WORKSPACE
    assert decode(L, total=0) == tts.TTS_OK
    f = L.tts_attn_decode_workspace_bytes
    assert f(0, 8, 2, 128) == 0 and f(65, 8, 2, 128) == 0 and f(1, 8, 3, 128) == 0
    assert f(1, 8, 2, 80) == 0


def test_binding_refusals():
    import tiled_top_sparse_gb300 as tts
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        tts.rope_kv_append(x, x, x, x, x, x, x, 1)
    with pytest.raises(ValueError):
        tts.attn_decode_paged(x, x, x, x, x, 0.1)


def test_e4m3_rounding_matches_torch():
    y = np.concatenate([np.linspace(-500, 500, 20001), 2.0 ** -np.arange(4, 16),
                        np.random.default_rng(0).standard_normal(20000) * 0.02])
    want = torch.tensor(y).clamp(-448, 448).float()
    same = want.double() == torch.tensor(y).clamp(-448, 448)
    got = torch.tensor(ref.round_e4m3(y)).float()[same]
    assert torch.equal(got, want[same].to(torch.float8_e4m3fn).float())


def test_page_scale_is_the_smallest_power_of_two():
    for a in [0.0, 1e-30, 2.0 ** -60 * 448, 1e-3, 1.0, 447.9, 448.0, 448.1, 895.9, 896.0, 1e30]:
        s = ref.page_scale(a)
        assert a <= 448 * s and (s == 2.0 ** -60 or a > 448 * s / 2)
        assert np.log2(s) == np.rint(np.log2(s))


def test_visible_keys_brute_force():
    for pos in (0, 5, 9):
        for w in (0, 1, 3, 100):
            for s in (0, 2):
                got = ref.visible(pos, 10, w, s)
                for j in range(10):
                    want = j <= pos and (w == 0 or j > pos - w or j < s)
                    assert got[j] == want


def test_window_refusals(L):
    import tiled_top_sparse_gb300 as tts

    def window(**kw):
        a = dict(q=A, k=A, v=A, dt=0, tq=256, tk=256, cq=A, ck=A, b=1, mq=256, mk=256, hq=2,
                 hkv=1, d=64, window=100, sinks=4, scale=0.125, out=A, odt=0, lse=NUL, ws=A,
                 wsb=1 << 30, st=NUL, stream=NUL)
        assert set(kw) <= set(a)
        a.update(kw)
        return L.tts_attn_fwd_varlen_window(*a.values())

    for n in ("q", "k", "v", "cq", "ck", "out"):
        assert window(**{n: NUL}) == tts.TTS_ERR_INVALID_ARG, n
    for n in ("q", "k", "v", "out"):
        assert window(**{n: B}) == tts.TTS_ERR_INVALID_ARG, n
    for kw in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(dt=2), dict(odt=2),
               dict(hq=3, hkv=2), dict(scale=-1.0), dict(b=0)):
        assert window(**kw) == tts.TTS_ERR_INVALID_ARG, kw
    assert window(d=96) == tts.TTS_ERR_UNSUPPORTED
    assert window(ws=NUL) == tts.TTS_ERR_WORKSPACE
    assert window(tq=0) == tts.TTS_OK
