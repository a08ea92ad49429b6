"""CPU checks of the entry points for drafted trees, position axes and moved cache rows: bad
host-side arguments are refused before any CUDA call, the binding's checks with stand-ins for
tensors, and the 64-bit definitions against brute force."""
import ctypes
import importlib.machinery
import importlib.util
import shutil

import numpy as np
import pytest
import torch

import tree_ref
from test_native_binding import BF16, E4M3, F32, I32, U8, Fake, counting

A = ctypes.c_void_p(0x10000)   # 16-byte aligned, never dereferenced
B = ctypes.c_void_p(0x10008)   # misaligned
NUL = None
I64 = "i64"


@pytest.fixture(scope="module")
def L():
    from tiled_top_sparse_gb300 import _build
    _build.build()
    import tiled_top_sparse_gb300 as tts
    return tts.lib()


def call(f, defaults, **kw):
    assert set(kw) <= set(defaults)
    return f(*{**defaults, **kw}.values())


def append(L, **kw):
    a = dict(q=A, qs=1024, hq=8, k=A, ks=256, v=A, vs=256, total=10, cu=A, past=A, batch=2, max_new=5,
             hkv=2, d=128, cs=A, max_pos=100, pos=A, axes=3, axis=bytes(16) + bytes([1, 2] * 24), pt=A,
             max_pages=4, kc=A, vc=A, ksc=A, vsc=A, dt=2, pages=16, ps=64, qo=A, ko=A, st=NUL,
             stream=NUL)
    return call(L.tts_rope_kv_append_axes, a, **kw)


def test_append_axes_refusals(L):
    import tiled_top_sparse_gb300 as tts
    for n in ("k", "v", "cu", "past", "pt", "kc", "vc", "ksc", "vsc", "qo", "pos", "cs", "axis"):
        assert append(L, **{n: NUL}) == tts.TTS_ERR_INVALID_ARG, n
    for n in ("q", "k", "v", "kc", "vc", "qo", "ko", "cs"):
        assert append(L, **{n: B}) == tts.TTS_ERR_INVALID_ARG, n
    for kw in (dict(axes=0), dict(axes=5), dict(axes=-1), dict(axes=2), dict(axis=bytes(63) + b"\x03"),
               dict(max_pos=0), dict(total=-1), dict(batch=0), dict(d=0), dict(ks=260), dict(dt=1)):
        assert append(L, **kw) == tts.TTS_ERR_INVALID_ARG, kw
    for kw in (dict(d=80), dict(ps=48), dict(max_pages=1 << 25)):
        assert append(L, **kw) == tts.TTS_ERR_UNSUPPORTED, kw
    assert append(L, total=0, pos=NUL, cs=NUL) == tts.TTS_OK  # nothing to append


def tree(L, **kw):
    a = dict(q=A, total=10, cu=A, mask=A, batch=2, max_q=5, hq=8, hkv=2, d=128, kc=A, vc=A, ksc=A,
             vsc=A, dt=2, pages=16, ps=64, pt=A, max_pages=4, lens=A, window=0, sinks=0, scale=0.1,
             out=A, odt=1, lse=NUL, ws=A, wsb=1 << 40, st=NUL, stream=NUL)
    return call(L.tts_attn_decode_tree, a, **kw)


def test_tree_refusals(L):
    import tiled_top_sparse_gb300 as tts
    for n in ("q", "mask", "kc", "vc", "ksc", "vsc", "pt", "lens", "out"):
        assert tree(L, **{n: NUL}) == tts.TTS_ERR_INVALID_ARG, n
    for n in ("q", "kc", "vc", "out"):
        assert tree(L, **{n: B}) == tts.TTS_ERR_INVALID_ARG, n
    assert tree(L, mask=ctypes.c_void_p(0x10004)) == tts.TTS_ERR_INVALID_ARG
    for kw in (dict(total=-1), dict(batch=0), dict(max_q=0), dict(hkv=3), dict(window=-1),
               dict(sinks=-1), dict(scale=0.0), dict(scale=float("nan")), dict(dt=1), dict(odt=2),
               dict(cu=NUL, total=1)):
        assert tree(L, **kw) == tts.TTS_ERR_INVALID_ARG, kw
    for kw in (dict(d=80), dict(ps=24), dict(max_q=65), dict(max_pages=1 << 25),
               dict(batch=1 << 12, max_pages=1 << 23)):
        assert tree(L, **kw) == tts.TTS_ERR_UNSUPPORTED, kw
    assert tree(L, ws=NUL) == tts.TTS_ERR_WORKSPACE
    assert tree(L, ws=B) == tts.TTS_ERR_WORKSPACE
    assert tree(L, total=0) == tts.TTS_OK
    f = L.tts_attn_decode_tree_workspace_bytes
    assert f(0, 8, 2, 128) == 0 and f(65, 8, 2, 128) == 0 and f(1, 8, 3, 128) == 0
    assert f(1, 8, 2, 80) == 0


def compact(L, **kw):
    a = dict(kc=A, vc=A, ksc=A, vsc=A, dt=2, pages=16, hkv=2, ps=64, d=128, pt=A, max_pages=4,
             past=A, batch=2, path=A, max_path=8, plens=A, lens=ctypes.c_void_p(0x20000), st=NUL,
             stream=NUL)
    return call(L.tts_kv_compact, a, **kw)


def fork(L, **kw):
    a = dict(kc=A, vc=A, ksc=A, vsc=A, dt=2, pages=16, hkv=2, ps=64, d=128, pt=A, max_pages=4,
             lens=A, batch=2, parents=A, new=A, children=3, to=ctypes.c_void_p(0x20000),
             tl=ctypes.c_void_p(0x20000), st=NUL, stream=NUL)
    return call(L.tts_kv_fork, a, **kw)


@pytest.mark.parametrize("f,ptrs", [
    (compact, ("kc", "vc", "ksc", "vsc", "pt", "past", "path", "plens", "lens")),
    (fork, ("kc", "vc", "ksc", "vsc", "pt", "lens", "parents", "new", "to", "tl"))])
def test_move_refusals(L, f, ptrs):
    import tiled_top_sparse_gb300 as tts
    for n in ptrs:
        assert f(L, **{n: NUL}) == tts.TTS_ERR_INVALID_ARG, n
    for kw in (dict(kc=B), dict(vc=B), dict(dt=1), dict(dt=3), dict(pages=0), dict(hkv=0), dict(ps=0),
               dict(d=0), dict(max_pages=0), dict(batch=0)):
        assert f(L, **kw) == tts.TTS_ERR_INVALID_ARG, kw
    for kw in (dict(d=80), dict(ps=8), dict(max_pages=1 << 25), dict(pages=2 ** 31 - 1)):
        assert f(L, **kw) == tts.TTS_ERR_UNSUPPORTED, kw


def test_move_sizes(L):
    import tiled_top_sparse_gb300 as tts
    assert compact(L, max_path=-1) == tts.TTS_ERR_INVALID_ARG
    assert compact(L, max_path=65) == tts.TTS_ERR_UNSUPPORTED
    assert compact(L, lens=A) == tts.TTS_ERR_INVALID_ARG  # in place of past_lens
    assert fork(L, children=-1) == tts.TTS_ERR_INVALID_ARG
    assert compact(L, lens=A, past=ctypes.c_void_p(0x30000)) == tts.TTS_ERR_INVALID_ARG  # of path_lens
    assert fork(L, to=A) == tts.TTS_ERR_INVALID_ARG and fork(L, tl=A) == tts.TTS_ERR_INVALID_ARG
    assert fork(L, children=0, parents=NUL, new=NUL) == tts.TTS_OK


def test_vision_axes_refusals(L):
    import tiled_top_sparse_gb300 as tts

    def vision(**kw):
        a = dict(x=A, n=10, hidden=64, w=A, bias=NUL, pos=A, axes=2, axis=bytes([0, 1] * 16), cs=A,
                 max_pos=9, heads=4, d=64, q=A, k=A, v=A, st=NUL, stream=NUL)
        return call(L.tts_qkv_rope_axes, a, **kw)

    for n in ("x", "w", "pos", "axis", "cs", "q", "k", "v"):
        assert vision(**{n: NUL}) == tts.TTS_ERR_INVALID_ARG, n
    for n in ("x", "w", "cs", "q", "k", "v"):
        assert vision(**{n: B}) == tts.TTS_ERR_INVALID_ARG, n
    for kw in (dict(axes=0), dict(axes=5), dict(axes=1), dict(n=-1), dict(hidden=12), dict(d=1),
               dict(max_pos=0), dict(heads=0)):
        assert vision(**kw) == tts.TTS_ERR_INVALID_ARG, kw
    assert vision(d=96) == tts.TTS_ERR_UNSUPPORTED and vision(heads=3) == tts.TTS_ERR_UNSUPPORTED
    assert vision(n=0, x=NUL) == tts.TTS_OK


# ------------------------------------------------------------------------------- binding
@pytest.fixture()
def bound(tmp_path):
    """A copy of the built module bound to an entry point that counts its calls."""
    from tiled_top_sparse_gb300 import _build
    path = str(tmp_path / "_native.so")
    shutil.copy(_build.build_native(), path)

    def make(get=lambda: 0, put=lambda dev: None, more=True):
        calls, keep, addr = counting()
        loader = importlib.machinery.ExtensionFileLoader("_native", path)
        m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_native", loader))
        loader.exec_module(m)
        m.bind((addr,) * 3, (BF16, F32, U8, E4M3, I32), (lambda dev: 0, get, put))
        if more:
            m.bind_more((addr,) * 5, I64)
        return m, calls, keep

    return make


def t(shape, dtype, device=0):
    return Fake(shape, dtype, device=device)


def args_of(name, device=0):
    x = lambda shape, dtype: t(shape, dtype, device)  # noqa: E731
    cache = [x((4, 2, 16, 64), U8), x((4, 2, 16, 64), U8)]
    scales = [x((4, 2), F32), x((4, 2), F32)]
    if name == "rope_kv_append_axes":
        return [x((3, 2, 64), BF16), x((3, 2, 64), BF16), *cache, x((1, 2), I32), x((1,), I32),
                x((2,), I32), 3, *scales, x((9, 32, 2), F32), None, None, None, None, x((2, 3), I32),
                bytes(32)]
    if name == "attn_decode_tree":
        return [x((3, 4, 64), BF16), *cache, *scales, x((1, 2), I32), x((1,), I32), x((2,), I32), 3,
                0, 0, 0.1, x((3, 4, 64), F32), None, x((1,), U8), None, x((3,), I64)]
    if name == "kv_compact":
        return [*cache, x((1, 2), I32), x((1,), I32), x((1, 5), I32), x((1,), I32), *scales,
                x((1,), I32), None]
    if name == "kv_fork":
        return [*cache, x((1, 2), I32), x((1,), I32), x((3,), I32), x((3,), I32), *scales,
                x((3, 2), I32), x((3,), I32), None]
    return [x((3, 16), BF16), x((3 * 4 * 64, 16), BF16), None, x((2, 3), I32), bytes(32),
            x((9, 32, 2), F32), 4, *[x((3, 4, 64), BF16)] * 3, None]


NAMES = ["rope_kv_append_axes", "attn_decode_tree", "kv_compact", "kv_fork", "qkv_rope_axes"]


@pytest.mark.parametrize("name", NAMES)
def test_binding_makes_the_call_on_the_tensors_device(bound, name):
    now = [0]
    m, calls, _ = bound(get=lambda: now[0], put=lambda dev: now.__setitem__(0, dev))
    assert getattr(m, name)(*args_of(name, device=1)) == 0 and now[0] == 0 and len(calls) == 1
    with pytest.raises(TypeError):
        getattr(m, name)(1)


@pytest.mark.parametrize("name", NAMES)
def test_binding_without_the_entry_points(bound, name):
    m, calls, _ = bound(more=False)  # a copy of its own, so that nothing is bound yet
    with pytest.raises(RuntimeError, match="bind_more"):
        getattr(m, name)(*args_of(name))
    assert calls == []


@pytest.mark.parametrize("name,at,wrong,match", [
    ("rope_kv_append_axes", 15, t((2, 4), I32), "positions"),
    ("rope_kv_append_axes", 15, t((3,), I32), "positions"),
    ("rope_kv_append_axes", 15, t((2, 3), F32), "positions"),
    ("rope_kv_append_axes", 15, t((2, 3), I32, 1), "positions"),
    ("rope_kv_append_axes", 16, bytes(31), "pair_axis"),
    ("rope_kv_append_axes", 16, [0] * 32, "pair_axis"),
    ("rope_kv_append_axes", 10, None, "cos_sin"),
    ("attn_decode_tree", 16, t((2,), I64), "tree_mask"),
    ("attn_decode_tree", 16, t((3,), I32), "tree_mask"),
    ("attn_decode_tree", 16, t((3, 1), I64), "tree_mask"),
    ("attn_decode_tree", 16, None, "tree_mask"),
    ("kv_compact", 4, t((2, 5), I32), "path"),
    ("kv_compact", 4, t((5,), I32), "path"),
    ("kv_compact", 5, t((2,), I32), "path"),
    ("kv_compact", 8, t((2,), I32), "kv_lens"),
    ("kv_compact", 6, None, "scale"),
    ("kv_fork", 5, t((2,), I32), "new_pages"),
    ("kv_fork", 8, t((3, 3), I32), "tables_out"),
    ("kv_fork", 9, t((2,), I32), "lens_out"),
    ("kv_fork", 3, t((2,), I32), "page_tables"),
    ("kv_fork", 1, t((4, 2, 16, 64), BF16), "v_cache"),
    ("qkv_rope_axes", 1, t((100, 16), BF16), "x and w"),
    ("qkv_rope_axes", 2, t((5,), F32), "bias"),
    ("qkv_rope_axes", 3, t((2, 4), I32), "positions"),
    ("qkv_rope_axes", 4, bytes(33), "pair_axis"),
    ("qkv_rope_axes", 5, t((0, 32, 2), F32), "cos_sin"),
    ("qkv_rope_axes", 6, 5, "x and w"),
    ("qkv_rope_axes", 8, t((3, 4, 32), BF16), "k must be"),
])
def test_binding_refusals(bound, name, at, wrong, match):
    m, calls, _ = bound()
    a = args_of(name)
    a[at] = wrong
    with pytest.raises(ValueError, match=match):
        getattr(m, name)(*a)
    assert calls == []


def test_cpu_tensors_are_refused():
    import tiled_top_sparse_gb300 as tts
    x, i = torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=torch.int32)
    for f in (lambda: tts.rope_kv_append_axes(x, x, x, x, i, i, i, 1, i, bytes(32), x),
              lambda: tts.attn_decode_tree(x, x, x, i, i, i, 0.1),
              lambda: tts.kv_compact(x, x, i, i, i, i), lambda: tts.kv_fork(x, x, i, i, i, i),
              lambda: tts.qkv_rope_axes(x[0], x[0], None, i, bytes(32), x, 1)):
        with pytest.raises(ValueError):
            f()


def test_rope_axes():
    import tiled_top_sparse_gb300 as tts
    assert tts.rope_axes([2, 3]) == bytes([0, 0, 1, 1, 1])
    assert tts.rope_axes([4, 2, 2], True) == bytes([0, 1, 2, 0, 1, 2, 0, 0])
    assert tts.rope_axes([0, 2]) == bytes([1, 1])
    for bad in ([], [1] * 5, [3, -1]):
        with pytest.raises(ValueError):
            tts.rope_axes(bad)


# --------------------------------------------------------------------------- definitions
def test_seen_keys_brute_force():
    rng = np.random.default_rng(0)
    for _ in range(300):
        n, past = int(rng.integers(1, 9)), int(rng.integers(-3, 12))
        mask, w, s = int(rng.integers(0, 1 << n)), int(rng.integers(0, 8)), int(rng.integers(0, 4))
        L = past + n
        got = tree_ref.sees(mask, n, L, w, s)
        pos = past + max(bin(mask).count("1") - 1, 0)
        for j in range(max(L, 0)):
            if j < past:
                want = w == 0 or j > pos - w or j < s
            else:
                want = bool(mask >> (j - past) & 1)
            assert got[j] == want


def test_chain_masks_are_causal():
    import gqa_ref as ref
    for i in range(5):
        want = ref.visible(7 + i, 12, 4, 2)
        got = tree_ref.sees((1 << (i + 1)) - 1, 5, 12, 4, 2)
        base = 7
        assert (got[:base] == want[:base]).all()
        assert (got[base:] == (np.arange(base, 12) <= base + i)).all()


def test_chain_masks_are_plain_decoding_where_the_window_holds_the_chain():
    """In a shorter window plain decoding hides new tokens too, which a mask's bits do not."""
    import gqa_ref as ref
    other = 0
    for n in range(1, 7):
        for past in range(9):
            for w in range(1, 10):
                for s in range(3):
                    for i in range(n):
                        same = (ref.visible(past + i, past + n, w, s)
                                == tree_ref.sees((1 << (i + 1)) - 1, n, past + n, w, s)).all()
                        assert same or w < n
                        other += not same
    assert other > 0


def test_masks_of_a_tree():
    assert tree_ref.masks_of([-1, 0, 0, 1]) == [1, 3, 5, 11]
    assert tree_ref.signed(1 << 63) == -(1 << 63) and tree_ref.signed(5) == 5
