"""CPU checks of the native module behind the grouped-query calls: a copy of it is bound to stand-ins
for the library's functions, torch's streams and devices, and tensors."""
import ctypes
import importlib.machinery
import importlib.util
import shutil
import threading
import time

import pytest


class Fake:
    """What the module looks at in a tensor."""

    def __init__(self, shape, dtype, ptr=0x10000, device=0):
        self.shape, self.dtype, self.ptr, self.device = tuple(shape), dtype, ptr, device

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.ptr

    def stride(self):
        out, n = [], 1
        for s in reversed(self.shape):
            out.append(n)
            n *= s
        return tuple(reversed(out))

    @property
    def nbytes(self):
        return 1 << 30


BF16, F32, U8, E4M3, I32 = "bf16", "f32", "u8", "e4m3", "i32"


@pytest.fixture()
def load(tmp_path):
    """A copy of the built module, with state of its own, bound to the given functions."""
    from tiled_top_sparse_gb300 import _build
    path = str(tmp_path / "_native.so")
    shutil.copy(_build.build_native(), path)

    def make(fns=(0, 0, 0), stream=lambda dev: 0, get=lambda: 0, put=lambda dev: None):
        loader = importlib.machinery.ExtensionFileLoader("_native", path)
        m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_native", loader))
        loader.exec_module(m)
        m.bind(tuple(fns), (BF16, F32, U8, E4M3, I32), (stream, get, put))
        return m

    return make


def counting():
    """An entry point that counts its calls and returns TTS_OK."""
    calls = []
    fn = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: calls.append(1) or 0)
    return calls, fn, ctypes.cast(fn, ctypes.c_void_p).value


def append_args(device=0, ptr=0x10000, **kw):
    t = lambda shape, dtype: Fake(shape, dtype, ptr, device)  # noqa: E731
    a = dict(k=t((3, 2, 64), BF16), v=t((3, 2, 64), BF16), k_cache=t((4, 2, 16, 64), U8),
             v_cache=t((4, 2, 16, 64), U8), page_tables=t((1, 2), I32), past_lens=t((1,), I32),
             cu_new=t((2,), I32), max_new=3, k_scale=t((4, 2), F32), v_scale=t((4, 2), F32),
             cos_sin=t((9, 32, 2), F32), q=None, q_out=None, k_out=None, status=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return list(a.values())


def test_empty_rotation_table_is_refused(load):
    """A table without positions has a null address, which the library takes as no rotation."""
    calls, keep, addr = counting()
    m = load((addr, addr, addr))
    assert m.rope_kv_append(*append_args()) == 0 and len(calls) == 1
    assert m.rope_kv_append(*append_args(cos_sin=None)) == 0 and len(calls) == 2
    with pytest.raises(ValueError, match="cos_sin"):
        m.rope_kv_append(*append_args(cos_sin=Fake((0, 32, 2), F32, 0)))
    assert len(calls) == 2


def decode_args(device=0, ptr=0x10000):
    t = lambda shape, dtype: Fake(shape, dtype, ptr, device)  # noqa: E731
    return [t((1, 4, 64), BF16), t((4, 2, 16, 64), BF16), t((4, 2, 16, 64), BF16), None, None,
            t((1, 2), I32), t((1,), I32), None, 1, 0, 0, 0.1, t((1, 4, 64), F32), None,
            t((1,), U8), None]


def window_args(device=0, ptr=0x10000):
    t = lambda shape, dtype: Fake(shape, dtype, ptr, device)  # noqa: E731
    return [t((5, 4, 64), BF16), t((5, 2, 64), BF16), t((5, 2, 64), BF16), t((2,), I32),
            t((2,), I32), 5, 5, 3, 1, 0.1, t((5, 4, 64), F32), None, t((1,), U8), None]


CALLS = [("rope_kv_append", append_args), ("attn_decode_paged", decode_args),
         ("attn_fwd_varlen_window", window_args)]


@pytest.mark.parametrize("name,args", CALLS)
def test_device_is_restored(load, name, args):
    """The caller's device is current again after a call, also where the stream of the tensors'
    device cannot be had; that error is the one that is raised."""
    now = [0]
    calls, keep, addr = counting()

    def put(dev):
        now[0] = dev

    def no_stream(dev):
        assert now[0] == 1
        raise RuntimeError("no stream")

    m = load((addr, addr, addr), get=lambda: now[0], put=put)
    assert getattr(m, name)(*args(device=1)) == 0 and now[0] == 0 and len(calls) == 1
    m = load((addr, addr, addr), stream=no_stream, get=lambda: now[0], put=put)
    with pytest.raises(RuntimeError, match="no stream"):
        getattr(m, name)(*args(device=1))
    assert now[0] == 0 and len(calls) == 1


@pytest.mark.parametrize("name,args", CALLS)
def test_other_threads_run_during_a_call(load, name, args):
    """A call that blocks (a full queue, a kernel's first load) leaves the interpreter to the other
    threads. The stand-in is the C library's usleep, whose microseconds are the first tensor's
    address (the append's is its q)."""
    pause = 400000
    addr = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p).value
    m = load((addr, addr, addr))
    a = args(ptr=pause)
    if name == "rope_kv_append":
        a[11] = a[12] = Fake((3, 4, 64), BF16, pause)
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.monotonic())
            time.sleep(0.001)

    other = threading.Thread(target=tick)
    other.start()
    try:
        begin = time.monotonic()
        assert getattr(m, name)(*a) == 0
        end = time.monotonic()
    finally:
        stop.set()
        other.join()
    assert end - begin >= 0.9e-6 * pause
    assert any(begin + 0.1 < t < end - 0.1 for t in ticks)
