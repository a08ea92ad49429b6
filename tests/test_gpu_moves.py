"""GPU parity of rows moved inside the paged cache: accepted paths brought together
(tts_kv_compact) and forked requests (tts_kv_fork), with their definitions."""
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


def pool(rng, pages, hkv, ps, d, f8, lo=-6, hi=-2):
    """Caches whose pages have scales of different sizes: moves between them grow scales."""
    c, s = [], []
    for _ in range(2):
        x = torch.tensor(rng.standard_normal((pages, hkv, ps, d)), dtype=torch.float32)
        if f8:
            c.append((x * 100).to(torch.float8_e4m3fn).view(torch.uint8))
            s.append(torch.tensor(2.0 ** rng.integers(lo, hi + 1, (pages, hkv)), dtype=torch.float32))
        else:
            c.append(x.to(torch.bfloat16))
            s.append(None)
    return c, s


def tables_for(rng, lens, ps, extra=3):
    need = [-(-n // ps) for n in lens]
    perm = rng.permutation(sum(need) + extra)
    t = np.full((len(lens), max(need + [1]) + 1), -1, np.int32)
    at = 0
    for r, n in enumerate(need):
        t[r, :n] = perm[at:at + n]
        at += n
    return t, sum(need) + extra, perm[at:]


def cuda(x, dtype=torch.int32):
    return None if x is None else (x.cuda() if isinstance(x, torch.Tensor)
                                   else torch.tensor(np.asarray(x)).to(dtype).cuda())


def values(t):
    return ref.codes_of(t)


def padded(path, width=None):
    width = max([len(p) for p in path] + [1]) if width is None else width
    return np.array([p + [-7] * (width - len(p)) for p in path], np.int32)


def compact(tts, c, s, tables, past, path, lens=None, **kw):
    d = [cuda(t) for t in (*c, *s)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = tts.kv_compact(d[0], d[1], cuda(tables), cuda(past), cuda(padded(path)),
                         cuda([len(p) for p in path] if lens is None else lens), k_scale=d[2],
                         v_scale=d[3], status=st, **kw)
    return d, out, int(st.item())


def same(d, want):
    for t, w in zip(d, want):
        if t is not None:
            np.testing.assert_array_equal(
                values(t) if t.dtype in (torch.uint8, torch.bfloat16) else t.cpu().double().numpy(), w)


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("hkv,d,ps", [(1, 128, 64), (3, 64, 16), (2, 128, 16), (2, 64, 128), (8, 128, 32)])
def test_compact(tts, f8, hkv, d, ps):
    rng = np.random.default_rng(ps + d + hkv)
    n = [1, 5, 64, 64, 20, 33, 16, 2, 64]
    past = [0, 63, 100, 0, 15, 31, 77, 200, 1]
    path = [[0], [0, 3, 4], sorted(rng.choice(64, 40, replace=False).tolist()), list(range(64)), [],
            [5, 32], [0, 1, 2, 9, 15], [1], list(range(1, 64))]
    tables, pages, _ = tables_for(rng, [a + b for a, b in zip(past, n)], ps)
    c, s = pool(rng, pages, hkv, ps, d, f8)
    k, v, ks, vs, lens = tree_ref.compact(values(c[0]), values(c[1]),
                                          *(None if t is None else t.numpy() for t in s), tables,
                                          past, path, [len(p) for p in path])
    got, out, st = compact(tts, c, s, tables, past, path)
    assert st == 0
    np.testing.assert_array_equal(out.cpu().numpy(), lens)
    same(got, [k, v, ks, vs])


@pytest.mark.parametrize("lo,hi", [(-59, -40), (-30, 30), (0, 0)])
def test_compact_scales_of_any_size(tts, lo, hi):
    rng = np.random.default_rng(hi - lo)
    past, path = [10, 3], [[2, 7, 30, 31, 45, 50], [0, 9, 40, 63]]
    tables, pages, _ = tables_for(rng, [74, 67], 16)
    c, s = pool(rng, pages, 2, 16, 128, True, lo, hi)
    want = tree_ref.compact(values(c[0]), values(c[1]), s[0].numpy(), s[1].numpy(), tables, past, path,
                            [6, 4])
    got, _, st = compact(tts, c, s, tables, past, path)
    assert st == 0
    same(got, want[:4])


def test_compact_keeps_bits_and_rows_that_are_not_moved(tts):
    """NaN codes and bytes of bf16 keep their bits where no scale changes; a whole path that stays moves
    nothing, whatever the scales hold."""
    rng = np.random.default_rng(5)
    tables, pages, _ = tables_for(rng, [40], 64)
    for f8 in (True, False):
        c, s = pool(rng, pages, 2, 64, 64, f8, -3, -3)
        raw = torch.tensor(rng.integers(0, 256, c[0].view(torch.uint8).shape), dtype=torch.uint8)
        c[0] = raw if f8 else raw.view(torch.bfloat16)
        got, _, st = compact(tts, c, s, tables, [20], [[0, 4, 9, 19]])
        want = c[0].clone().view(torch.uint8)
        for i, x in enumerate([0, 4, 9, 19]):
            want[tables[0, 0], :, 20 + i] = c[0].view(torch.uint8)[tables[0, 0], :, 20 + x]
        assert st == 0 and torch.equal(got[0].cpu().view(torch.uint8), want)
    s[0:2] = [None, None]
    c8, s8 = pool(rng, pages, 2, 64, 64, True)
    s8[0][:] = float("nan")
    got, out, st = compact(tts, c8, s8, tables, [20], [[0, 1, 2, 3]])
    assert st == 0 and torch.equal(got[0].cpu(), c8[0]) and int(out[0]) == 24


def test_compact_twice_is_the_same(tts):
    """A path whose rows lie behind the places they go to can be moved again."""
    rng = np.random.default_rng(6)
    tables, pages, _ = tables_for(rng, [100], 16)
    c, s = pool(rng, pages, 2, 16, 128, True)
    a, _, _ = compact(tts, c, s, tables, [36], [[0, 7, 20, 41, 63]])
    b, _, _ = compact(tts, [t.cpu() for t in a[:2]], [t.cpu() for t in a[2:]], tables, [36],
                      [[0, 7, 20, 41, 63]])
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_compact_device_errors(tts):
    rng = np.random.default_rng(7)
    past = [10, 20, 30, -4, 5, 8]
    path = [[0, 2, 1], [0, 3], [3, 30], [1], [0, 6], [1, 5]]
    tables, pages, _ = tables_for(rng, [40, 40, 64, 10, 40, 40], 16)
    c, s = pool(rng, pages, 2, 16, 128, False)
    same_as = [t.clone() for t in c]
    got, out, st = compact(tts, c, s, tables, past, path, lens=[3, 9, 2, 1, -1, 2])
    # not increasing; longer than the path; behind the table; before it; negative; fine
    assert st == tts.TTS_DEV_BAD_ARG | tts.TTS_DEV_INDEX_RANGE
    width = tables.shape[1] * 16
    behind = 30 + 30 >= width
    np.testing.assert_array_equal(out.cpu().numpy(), [10, 20, 30 if behind else 32, 0, 5, 10])
    want = [t.clone() for t in same_as]
    for t, o in zip(want, same_as):
        for i, x in ((0, 1), (1, 5)):
            t[tables[5, (8 + i) // 16], :, (8 + i) % 16] = o[tables[5, (8 + x) // 16], :, (8 + x) % 16]
        if not behind:
            for i, x in ((0, 3), (1, 30)):
                t[tables[2, (30 + i) // 16], :, (30 + i) % 16] = \
                    o[tables[2, (30 + x) // 16], :, (30 + x) % 16]
    assert all(torch.equal(a.cpu(), b) for a, b in zip(got[:2], want))


def test_compact_missing_pages_and_scales(tts):
    rng = np.random.default_rng(8)
    tables, pages, _ = tables_for(rng, [64, 64], 16)
    c, s = pool(rng, pages, 1, 16, 64, True, -3, -3)
    t2 = tables.copy()
    t2[0, 3] = 1 << 29          # request 0: the source of its last row is gone
    s[0][int(tables[1, 2]), 0] = float("nan")  # request 1: so is its second row's scale
    got, out, st = compact(tts, c, s, t2, [10, 10], [[0, 9, 50], [1, 30, 45]])
    assert st == tts.TTS_DEV_BAD_ARG | tts.TTS_DEV_INDEX_RANGE
    np.testing.assert_array_equal(out.cpu().numpy(), [13, 13])
    before = values(c[0])
    at = lambda r, x: (tables[r, x // 16], 0, x % 16)  # noqa: E731
    after = values(got[0])
    np.testing.assert_array_equal(after[at(0, 11)], before[at(0, 19)])
    np.testing.assert_array_equal(after[at(0, 12)], before[at(0, 12)])  # not moved
    np.testing.assert_array_equal(after[at(1, 10)], before[at(1, 11)])
    np.testing.assert_array_equal(after[at(1, 11)], before[at(1, 11)])  # not moved
    np.testing.assert_array_equal(after[at(1, 12)], before[at(1, 55)])


def test_compact_into_a_page_without_a_scale(tts):
    """Rows moved into a page whose scale is no number: it takes the one that they need."""
    rng = np.random.default_rng(9)
    tables, pages, _ = tables_for(rng, [64], 16)
    c, s = pool(rng, pages, 1, 16, 64, True, -3, -3)
    s[1][int(tables[0, 1]), 0] = 0.0
    got, _, st = compact(tts, c, s, tables, [16], [[20, 21, 40]])
    assert st == tts.TTS_DEV_BAD_ARG
    x = values(c[1])[tables[0, 2:4], 0] * 2.0 ** -3  # positions 32 .. 63
    rows = np.concatenate(x)[[4, 5, 24]]
    t = ref.page_scale(np.abs(rows).max())
    assert float(got[3][int(tables[0, 1]), 0]) == t
    np.testing.assert_array_equal(values(got[1])[tables[0, 1], 0, :3], ref.round_e4m3(rows / t))


def test_compact_after_an_append_of_a_tree(tts):
    """The path's keys and values are what an append of the path alone would have cached (bf16)."""
    rng = np.random.default_rng(10)
    hkv, d, ps, past, n, path = 2, 64, 16, [21], 30, [0, 4, 11, 29]
    tables, pages, _ = tables_for(rng, [60], ps)
    x = [torch.tensor(rng.standard_normal((n, hkv, d))).to(torch.bfloat16).cuda() for _ in range(2)]
    depth = torch.tensor([[21 + int(rng.integers(0, 5)) for _ in range(n)]], dtype=torch.int32).cuda()
    cs = tts.rope_cache(64, d)
    one = tts.rope_axes([d // 2])
    caches = []
    for keep in (None, path):
        c = [torch.zeros(pages, hkv, ps, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        sel = list(range(n)) if keep is None else keep
        tts.rope_kv_append_axes(x[0][sel].contiguous(), x[1][sel].contiguous(), *c, cuda(tables),
                                cuda(past), cuda([0, len(sel)]), len(sel),
                                depth[:, sel].contiguous(), one, cs)
        if keep is None:
            tts.kv_compact(*c, cuda(tables), cuda(past), cuda([path]), cuda([4]))
        caches.append(c)
    for a, b in zip(*caches):
        for i in range(21, 25):
            assert torch.equal(a[tables[0, i // ps], :, i % ps], b[tables[0, i // ps], :, i % ps])


def test_compact_entries_at_the_end_of_32_bits(tts):
    """A last entry up to the largest int lies behind the table, whatever the sum would be in 32 bits:
    said, and nothing of that request is moved."""
    rng = np.random.default_rng(11)
    top = 2 ** 31 - 1
    past = [5, 0, 40, 10, 1]
    path = [[0, top], [top], list(range(39)) + [top], [2, top - 9], [0, 3]]
    tables, pages, _ = tables_for(rng, [60] * 5, 16)
    for f8 in (True, False):
        c, s = pool(rng, pages, 2, 16, 64, f8, -3, -3)
        got, out, st = compact(tts, c, s, tables, past, path)
        assert st == tts.TTS_DEV_INDEX_RANGE
        np.testing.assert_array_equal(out.cpu().numpy(), [5, 0, 40, 10, 3])
        want = [t.clone() for t in c]
        for t, o in zip(want, c):
            t[tables[4, 0], :, 2] = o[tables[4, 0], :, 4]
        assert all(torch.equal(a.cpu(), b) for a, b in zip(got[:2], want))


def test_compact_rows_of_zeros_between_far_scales(tts):
    """Zero rows of a page with a huge scale stay zeros in a page whose scale is 2^160 times smaller; NaN
    codes beside them stay NaN, and rows with values make the page's scale grow."""
    rng = np.random.default_rng(12)
    tables, pages, _ = tables_for(rng, [70, 70], 16)
    c, s = pool(rng, pages, 2, 16, 128, True, -3, -3)
    for x, sc in zip(c, s):
        for r in range(2):
            sc[int(tables[r, 0])] = 2.0 ** -60  # a page that was begun with zeros
            x[int(tables[r, 0])] = 0
            sc[int(tables[r, 2])] = 2.0 ** 100  # beside a huge row
            x[int(tables[r, 2]), :, :6] = 0
            x[int(tables[r, 2]), :, 3, 5] = 0x7F
            x[int(tables[r, 2]), :, 4, 9] = 0xFF
    past, path = [8, 8], [[0, 24, 25, 26, 27, 28, 29], [0, 24, 27, 31]]  # the last: row 39, with values
    want = tree_ref.compact(values(c[0]), values(c[1]), s[0].numpy(), s[1].numpy(), tables, past, path,
                            [7, 4])
    got, out, st = compact(tts, c, s, tables, past, path)
    assert st == 0
    np.testing.assert_array_equal(out.cpu().numpy(), want[4])
    same(got, want[:4])
    assert float(got[2][int(tables[0, 0]), 0]) == 2.0 ** -60
    assert float(got[2][int(tables[1, 0]), 0]) > 2.0 ** 90


# --------------------------------------------------------------------------------- fork
def run_fork(tts, c, s, tables, kv, parents, new_pages, **kw):
    d = [cuda(t) for t in (*c, *s)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, lens = tts.kv_fork(d[0], d[1], cuda(tables), cuda(kv), cuda(parents), cuda(new_pages),
                          k_scale=d[2], v_scale=d[3], status=st, **kw)
    return d, t, lens, int(st.item())


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("hkv,d,ps", [(1, 128, 64), (3, 64, 16), (8, 128, 128), (2, 64, 32)])
def test_fork(tts, f8, hkv, d, ps):
    rng = np.random.default_rng(ps + hkv)
    kv = [1, ps, 3 * ps, 5 * ps - 1, 0, 2 * ps + 7]
    parents = [0, 0, 3, 1, 2, 4, 5, 5, 3, 5]
    tables, pages, free = tables_for(rng, kv, ps, extra=12)
    c, s = pool(rng, pages, hkv, ps, d, f8)
    new = free[:10].copy()
    new[7] = -1  # one child goes on in its parent's place
    want = tree_ref.fork(values(c[0]), values(c[1]), *(None if t is None else t.numpy() for t in s),
                         tables, kv, parents, new)
    got, t, lens, st = run_fork(tts, c, s, tables, kv, parents, new)
    assert st == 0
    same(got, want[:4])
    np.testing.assert_array_equal(t.cpu().numpy(), want[4])
    np.testing.assert_array_equal(lens.cpu().numpy(), want[5])


def test_fork_full_tables(tts):
    """A parent whose last page is the table's last, full one: there is no entry for a next page."""
    rng = np.random.default_rng(1)
    c, s = pool(rng, 6, 2, 16, 64, False)
    tables = np.array([[4, 2]], np.int32)
    got, t, lens, st = run_fork(tts, c, s, tables, [32], [0, 0], [0, 1])
    assert st == 0 and t.cpu().tolist() == [[4, 2], [4, 2]] and lens.cpu().tolist() == [32, 32]
    assert torch.equal(got[0].cpu(), c[0])


def test_fork_device_errors(tts):
    rng = np.random.default_rng(2)
    c, s = pool(rng, 8, 2, 16, 64, True)
    tables = np.array([[4, 2, -1], [3, 77, 5]], np.int32)
    got, t, lens, st = run_fork(tts, c, s, tables, [20, 20], [5, -1, 0, 1, 0], [0, 1, 99, 6, 7])
    assert st == tts.TTS_DEV_INDEX_RANGE
    assert t.cpu().tolist() == [[-1] * 3, [-1] * 3, [4, -1, -1], [3, 6, -1], [4, 7, -1]]
    assert lens.cpu().tolist() == [0, 0, 20, 20, 20]
    want = c[0].clone()
    want[7, :, :4] = c[0][2, :, :4]
    assert torch.equal(got[0].cpu(), want)
    _, t, lens, st = run_fork(tts, c, s, tables, [49, -2], [0, 1], [0, 1])
    assert st == tts.TTS_DEV_INDEX_RANGE and lens.cpu().tolist() == [0, 0]
    assert t.cpu().tolist() == [[-1] * 3] * 2


def test_fork_no_children(tts):
    c, s = pool(np.random.default_rng(3), 4, 1, 16, 64, False)
    _, t, lens, st = run_fork(tts, c, s, np.array([[1, 2]], np.int32), [20], [], [])
    assert st == 0 and t.shape == (0, 2) and lens.numel() == 0


def test_moves_in_a_captured_graph(tts):
    """Compaction and a fork captured once and replayed with other lengths, paths and parents."""
    rng = np.random.default_rng(4)
    ps, hkv, d = 16, 2, 64
    tables, pages, free = tables_for(rng, [90, 90], ps, extra=8)
    c, s = pool(rng, pages, hkv, ps, d, True)
    D = [cuda(t) for t in (*c, *s)]
    first = [t.clone() for t in D]
    tab, past = cuda(tables), cuda([20, 26])
    path, m, lens = cuda([[0, 5, 9], [2, 3, 60]]), cuda([3, 2]), cuda([0, 0])
    par, new = cuda([1, 0, 1]), cuda(free[:3])
    to, tl = cuda(np.zeros((3, tables.shape[1]))), cuda([0, 0, 0])

    def step():
        tts.kv_compact(D[0], D[1], tab, past, path, m, k_scale=D[2], v_scale=D[3], kv_lens=lens)
        tts.kv_fork(D[0], D[1], tab, lens, par, new, k_scale=D[2], v_scale=D[3], tables_out=to,
                    lens_out=tl)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for p, q, k in (([20, 26], [[0, 5, 9], [2, 3, 60]], [3, 2]), ([3, 40], [[1, 2, 3], [0, 1, 2]], [3, 1])):
        for t, f in zip(D, first):
            t.copy_(f)
        past.copy_(cuda(p)), path.copy_(cuda(q)), m.copy_(cuda(k))
        g.replay()
        torch.cuda.synchronize()
        kk, vv, ks, vs, ln = tree_ref.compact(values(c[0]), values(c[1]), s[0].numpy(), s[1].numpy(),
                                              tables, p, q, k)
        want = tree_ref.fork(kk, vv, ks, vs, tables, ln, [1, 0, 1], free[:3])
        same(D, want[:4])
        np.testing.assert_array_equal(to.cpu().numpy(), want[4])
        np.testing.assert_array_equal(tl.cpu().numpy(), want[5])
