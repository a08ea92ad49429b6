"""GPU tests of windowed prefill behind cached keys: what no row of a sequence sees may hold
anything."""
import numpy as np
import pytest
import torch

import gqa_ref as ref
from test_gpu_window import BF16_HALF, cum, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tts():
    import tiled_top_sparse_gb300 as m
    m.lib()
    return m


@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("lq,lk,hq,hkv,window,sinks", [
    ([100, 260, 1], [700, 900, 513], 4, 1, 200, 5),      # one query tile per item
    ([33], [5000], 2, 2, 990, 0),                       # a long prefix, no first tokens
    ([200, 129], [1500, 640], 4, 2, 64, 300),            # hidden keys behind 300 first tokens
    ([1], [200], 2, 1, 1, 1),
    ([700, 500, 64], [1900, 777, 3000], 32, 8, 150, 4),  # pairs of heads, many items per CTA
    ([900, 411], [1300, 2000], 15, 5, 260, 130),         # an odd group: pairs of row tiles
    ([300, 77], [290, 300], 2, 1, 100, 3),               # more rows than keys beside hidden keys
])
def test_keys_hidden_from_every_row(tts, d, lq, lk, hq, hkv, window, sinks):
    """Keys of a sequence that none of its rows sees (behind the first row's window and the first
    tokens) hold NaN and infinities."""
    q, k, v = inputs(sum(lk) + d, lq, lk, hq, hkv, d, torch.bfloat16)
    cq, ck = cum(lq), cum(lk)
    hk, hv = k.clone(), v.clone()
    for r in range(len(lq)):
        a, b = int(ck[r]) + sinks, int(ck[r]) + lk[r] - lq[r] + 1 - window
        if b > a:
            k[a:b], v[a:b] = 0, 0
            hk[a:b], hv[a:b] = float("nan"), float("nan")
            hk[a:b:3], hv[a:b:3] = float("inf"), float("-inf")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = tts.attn_fwd_varlen_window(q, hk, hv, torch.tensor(cq).cuda(), torch.tensor(ck).cuda(),
                                          max(lq), max(lk), window, sinks, d ** -0.5, status=st)
    tts.check_status(st)
    ro, rl, tol, tol_l = ref.attend_packed(*(x.float().cpu().numpy() for x in (q, k, v)), cq, ck,
                                           d ** -0.5, window, sinks, BF16_HALF)
    assert np.all(np.abs(out.cpu().numpy() - ro) <= tol)
    l = lse.cpu().numpy()
    assert np.array_equal(np.isneginf(l), np.isneginf(rl))
    fin = np.isfinite(rl)
    assert np.all(np.abs(l[fin] - rl[fin]) <= tol_l[fin])
    a = tts.attn_fwd_varlen_window(q, k, v, torch.tensor(cq).cuda(), torch.tensor(ck).cuda(),
                                   max(lq), max(lk), window, sinks, d ** -0.5)
    assert torch.equal(a[0], out) and torch.equal(a[1], lse)  # what is hidden moves no bit
