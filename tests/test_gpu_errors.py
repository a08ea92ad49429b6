"""GPU tests of what a failed call leaves behind: nothing."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


def cudart():
    """The CUDA runtime that torch loaded."""
    import glob
    import os
    for line in open("/proc/self/maps"):
        path = line.split()[-1]
        if "libcudart.so" in os.path.basename(path):
            return ctypes.CDLL(path)
    found = glob.glob("/usr/local/cuda/lib64/libcudart.so*")
    return ctypes.CDLL(found[0])


def test_a_failed_call_does_not_reach_the_next():
    """A call on the default stream while a blocking stream is captured is refused by the CUDA
    runtime. The calls after the capture's end are good ones and say so."""
    import tiled_top_sparse_gb300 as tts
    x = torch.randn(1, 1, 64, device="cuda").to(torch.bfloat16)
    kc, vc = (torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tables = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    past, cu = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([0], [0, 1]))
    logits = torch.randn(1, 100, device="cuda")
    starts, lens = (torch.tensor([t], dtype=torch.int32, device="cuda") for t in (0, 100))
    append = lambda: tts.rope_kv_append(x, x, kc, vc, tables, past, cu, 1)  # noqa: E731
    topk = lambda: tts.topk_select(logits, starts, lens, 8)  # noqa: E731
    append()
    want = topk()
    torch.cuda.synchronize()
    rt, stream, graph = cudart(), ctypes.c_void_p(), ctypes.c_void_p()
    assert rt.cudaStreamCreate(ctypes.byref(stream)) == 0
    assert rt.cudaStreamBeginCapture(stream, 2) == 0  # relaxed: other streams may be used
    with pytest.raises(tts.TTSError) as e:
        append()
    assert e.value.code == tts.TTS_ERR_CUDA
    rt.cudaStreamEndCapture(stream, ctypes.byref(graph))
    rt.cudaGetLastError()  # of the test's own runtime
    if graph.value:
        rt.cudaGraphDestroy(graph)
    assert rt.cudaStreamDestroy(stream) == 0
    assert torch.equal(topk(), want)
    append()
    torch.cuda.synchronize()
    assert torch.equal(kc[0, 0, 0], x[0, 0])
