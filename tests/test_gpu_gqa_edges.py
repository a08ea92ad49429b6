"""GPU tests of the grouped-query calls at the edges of what their documentation allows."""
import numpy as np
import pytest
import torch

import gqa_ref as ref
from test_gpu_gqa import cum, dev, gen, make_pool, make_tables, run_append

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
