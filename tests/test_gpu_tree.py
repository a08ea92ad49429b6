"""GPU parity of attention under drafted trees' masks (tts_attn_decode_tree) with its 64-bit
definition over the very values that the cache holds."""
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


def cum(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


class Case:
    """A cache, its tables, queries and trees; `junk`: whatever no token sees holds NaN."""

    def __init__(self, seed, new, kv, hq, hkv, d, ps, f8, window=0, sinks=0, masks=None, junk=True,
                 front=0, back=0, spread=True, gain=1.0):
        rng = np.random.default_rng(seed)
        self.new, self.kv, self.ps, self.f8 = new, kv, ps, f8
        self.window, self.sinks, self.scale = window, sinks, d ** -0.5
        self.cu = cum(new) + np.int32(front)
        T = int(self.cu[-1]) + back
        self.q = torch.tensor(rng.standard_normal((T, hq, d)) * gain).to(torch.bfloat16)
        if masks is None:
            masks = [m for n in new for m in tree_ref.masks_of(tree_ref.random_tree(rng, n))[:n]]
        self.masks = [0] * front + list(masks) + [0] * back
        need = [-(-max(L, 0) // ps) for L in kv]
        pages = sum(need) + 2
        perm = rng.permutation(pages)
        self.tables = np.full((len(kv), max(need + [1]) + 1), -1, np.int32)
        at = 0
        for r, n in enumerate(need):
            self.tables[r, :n] = perm[at:at + n]
            at += n
        x = [torch.tensor(rng.standard_normal((pages, hkv, ps, d)), dtype=torch.float32)
             for _ in range(2)]
        if f8:
            self.c = [(t * 60).to(torch.float8_e4m3fn).view(torch.uint8) for t in x]
            lo, hi = (-9, -3) if spread else (-6, -5)
            self.s = [torch.tensor(2.0 ** rng.integers(lo, hi, (pages, hkv)), dtype=torch.float32)
                      for _ in range(2)]
        else:
            self.c = [t.to(torch.bfloat16) for t in x]
            self.s = [None, None]
        if junk:
            used = np.zeros((pages, ps), bool)
            for r, L in enumerate(kv):
                n = new[r]
                if L <= 0 or n == 0:
                    continue
                see = np.zeros(L, bool)
                for i in range(n):
                    see |= tree_ref.sees(self.masks[self.cu[r] + i], n, L, window, sinks)
                j = np.arange(L)[see]
                used[self.tables[r, j // ps], j % ps] = True
                # pages that no token of the request can see any more have been given back
                if window > 0:
                    lo = max(0, L - n + 1 - window)
                    for a in range(need[r]):
                        if (a + 1) * ps <= lo and a * ps >= sinks:
                            self.tables[r, a] = [-1, 1 << 30][a % 2]
            free = torch.tensor(~used)[:, None, :, None].expand_as(self.c[0])
            for t in self.c:
                if f8:
                    t[free] = 0x7F
                else:
                    t[free] = float("nan")

    def run(self, tts, out_dtype=torch.float32, status=None, **kw):
        dev = [None if t is None else t.cuda() for t in (*self.c, *self.s)]
        T, hq, d = self.q.shape
        out = torch.full((T, hq, d), 7.0, dtype=out_dtype, device="cuda")
        lse = torch.full((T, hq), 7.0, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda") if status is None else status
        a = dict(window=self.window, sinks=self.sinks, k_scale=dev[2], v_scale=dev[3])
        a.update(kw)
        tts.attn_decode_tree(self.q.cuda(), dev[0], dev[1], torch.tensor(self.tables).cuda(),
                             torch.tensor(self.kv, dtype=torch.int32).cuda(),
                             torch.tensor([tree_ref.signed(m) for m in self.masks]).cuda(),
                             self.scale, torch.tensor(self.cu).cuda(), max(max(self.new), 1),
                             out=out, lse=lse, status=st, **a)
        if status is None:
            tts.check_status(st)
        return out, lse

    def want(self, **kw):
        k, v = (np.nan_to_num(ref.codes_of(t)) for t in self.c)
        s = [None if t is None else t.numpy() for t in self.s]
        return tree_ref.attend_tree(self.q.float().numpy(), k, v, s[0], s[1],
                                    np.where(self.tables < k.shape[0], self.tables, 0), self.kv,
                                    self.cu, self.masks, self.scale, self.window, self.sinks, **kw)

    def check(self, tts, out_dtype=torch.float32, **kw):
        out, lse = self.run(tts, out_dtype, **kw)
        self.compare(out, lse, *self.want())

    def compare(self, out, lse, o, l, tol, tol_l):
        a, b = int(self.cu[0]), int(self.cu[-1])
        assert bool((out[:a] == 7).all()) and bool((out[b:] == 7).all())  # rows of no request
        assert bool((lse[:a] == 7).all()) and bool((lse[b:] == 7).all())
        got, gl = out.float().cpu().double().numpy()[a:b], lse.cpu().double().numpy()[a:b]
        o, l, tol, tol_l = o[a:b], l[a:b], tol[a:b], tol_l[a:b]
        if out.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * np.abs(o) + 1e-38
        assert np.isfinite(got).all()
        bad = np.abs(got - o) - tol
        assert bad.max(initial=-1) <= 0, f"out off by {np.abs(got - o).max()}, over by {bad.max()}"
        none = np.isinf(l)
        np.testing.assert_array_equal(none, np.isinf(gl))
        off = np.abs(np.where(none, 0, gl) - np.where(none, 0, l)) - tol_l
        assert off.max(initial=-1) <= 0, f"lse over by {off.max()}"


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("new,kv,hq,hkv,d,ps", [
    ([1], [1], 1, 1, 128, 64),                                # the smallest call
    ([5, 1, 16], [70, 1, 333], 4, 2, 128, 64),                # a few rows, ragged
    ([16], [2590], 8, 2, 128, 64),                            # one request over many CTAs
    ([9, 0, 3, 7], [100, 50, 3, 127], 6, 3, 64, 16),          # small pages, heads of 64
    ([64, 33], [700, 64], 8, 4, 128, 32),                     # 128 rows
    ([64, 10, 61], [1000, 129, 400], 12, 3, 128, 64),         # up to 256 rows
    ([64, 2], [515, 300], 16, 2, 64, 128),                    # 512 rows: several row blocks
    ([64, 47], [300, 900], 5, 1, 128, 128),                   # group of five, 320 rows
    ([64], [8000], 8, 2, 64, 16),
])
def test_parity(tts, f8, new, kv, hq, hkv, d, ps):
    Case(sum(new) + ps + hq, new, kv, hq, hkv, d, ps, f8, front=2, back=3).check(tts)


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 2), (64, 0), (100, 130), (300, 4), (5000, 4)])
def test_windows(tts, f8, window, sinks):
    Case(window, [12, 3, 20], [900, 40, 260], 8, 2, 128, 32, f8, window, sinks).check(tts)
    Case(window + 1, [40], [700], 8, 2, 64, 64, f8, window, sinks).check(tts)


@pytest.mark.parametrize("f8", [True, False])
def test_masks_of_any_kind(tts, f8):
    """Empty masks, masks without the token itself, bits behind the request's tokens, forward bits."""
    rng = np.random.default_rng(3)
    n = [7, 64, 3]
    masks = [int.from_bytes(rng.bytes(8), "little") for _ in range(sum(n))]
    masks[0] = 0
    masks[3] = 1 << 63
    masks[-2] = 0
    masks[20] = (1 << 64) - 1
    c = Case(5, n, [150, 64, 3], 8, 2, 128, 16, f8, masks=masks)
    c.check(tts)
    # request 2 has new tokens only: its token without a mask sees nothing
    out, lse = c.run(tts)
    assert bool((out[-2] == 0).all()) and bool((lse[-2] == float("-inf")).all())


@pytest.mark.parametrize("f8", [True, False])
def test_lengths_of_nothing(tts, f8):
    """A length of 0, one under the number of new tokens, a request without new tokens."""
    c = Case(9, [4, 6, 0, 2], [0, 3, 200, 65], 8, 2, 128, 64, f8)
    c.check(tts)


@pytest.mark.parametrize("f8", [True, False])
def test_output_types_and_no_lse(tts, f8):
    c = Case(11, [30, 5], [600, 77], 16, 4, 128, 64, f8, back=1)
    c.check(tts, torch.bfloat16)
    a, _ = c.run(tts)
    dev = [None if t is None else t.cuda() for t in (*c.c, *c.s)]
    out, none = tts.attn_decode_tree(
        c.q.cuda(), dev[0], dev[1], torch.tensor(c.tables).cuda(),
        torch.tensor(c.kv, dtype=torch.int32).cuda(),
        torch.tensor([tree_ref.signed(m) for m in c.masks]).cuda(), c.scale,
        torch.tensor(c.cu).cuda(), 30, k_scale=dev[2], v_scale=dev[3], want_lse=False)
    assert none is None and torch.equal(out[:35], a[:35])


@pytest.mark.parametrize("gain", [1e-30, 1e-3, 30.0, 1e20])
def test_queries_of_any_size(tts, gain):
    """Rows of any magnitude are scaled exactly; large scores make one key's weight the only one."""
    for f8 in (True, False):
        c = Case(13, [9, 3], [90, 20], 4, 2, 128, 64, f8, gain=gain)
        if gain > 1e10:
            c.scale = 1e-18
        c.check(tts)


def test_a_dominant_key_and_a_flat_tail(tts):
    """One key with a weight 2^14 times the others' each: together these still weigh as much."""
    for f8 in (True, False):
        c = Case(17, [4], [20000], 4, 1, 128, 64, f8, junk=False, spread=False)
        c.q[:] = 0
        c.q[..., 0] = 1.0
        c.scale = 1.0
        pg = c.tables[0]
        k = torch.zeros(c.c[0].shape, dtype=torch.float32)
        k[int(pg[0]), :, 5, 0] = 9.5
        c.c[0] = (k * 32).to(torch.float8_e4m3fn).view(torch.uint8) if f8 else k.to(torch.bfloat16)
        if f8:
            c.s[0][:] = 1 / 32
        c.check(tts)


def test_values_of_pages_with_far_scales(tts):
    c = Case(19, [6, 2], [300, 40], 4, 2, 64, 32, True)
    c.s[1] = torch.exp2(torch.tensor(np.random.default_rng(1).integers(-40, 40, c.s[1].shape))).float()
    c.check(tts)


def test_device_errors_are_reported(tts):
    """Pages outside the pool and scales that no page has: their keys are skipped, and it is said."""
    c = Case(23, [3, 2], [200, 100], 4, 2, 128, 32, True, junk=False)
    bad = int(c.tables[0, 2])
    c.s[0][bad, 1] = float("nan")
    c.s[1][int(c.tables[1, 0]), 0] = 0.0
    zero = int(c.tables[1, 0])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c.run(tts, status=st)
    assert int(st.item()) == tts.TTS_DEV_BAD_ARG
    s1 = c.s[1].clone()
    gone = lambda p, h: (p == bad and h == 1) or (p == zero and h == 0)  # noqa: E731
    c.s[0][bad, 1] = 1.0
    c.compare(out, lse, *c.want(gone=gone))
    c.s[1] = s1
    c = Case(24, [3, 2], [200, 100], 4, 2, 128, 32, False, junk=False)
    c.tables[0, 3] = 1 << 29
    c.tables[1, 1] = -1
    st.zero_()
    out, lse = c.run(tts, status=st)
    assert int(st.item()) == tts.TTS_DEV_INDEX_RANGE
    full = c.tables.copy()
    c.tables = np.where((full < 0) | (full > 1 << 20), -5, full)
    c.compare(out, lse, *c.want(gone=lambda p, h: p == -5))


def test_bad_bounds_are_reported(tts):
    c = Case(29, [3, 4, 2], [50, 60, 70], 4, 2, 64, 16, False)
    want = c.want()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.kv[1] = -3  # reads as 0: that request's rows see nothing
    out, lse = c.run(tts, status=st)
    assert int(st.item()) == tts.TTS_DEV_INDEX_RANGE
    assert bool((out[3:7] == 0).all()) and bool((lse[3:7] == float("-inf")).all())
    c.kv[1] = 60
    for x in (0, 1, 2):  # the others as before
        rows = slice(int(c.cu[x]), int(c.cu[x + 1]))
        if x != 1:
            assert np.abs(out[rows].cpu().double().numpy() - want[0][rows]).max() <= want[2][rows].max()
    c.cu = np.array([0, 3, 3 + 64, 9], np.int32)  # longer than the bound, and decreasing
    st.zero_()
    out, _ = c.run(tts, status=st)
    assert int(st.item()) == tts.TTS_DEV_BAD_ARG
    rows = slice(0, 3)
    assert np.abs(out[rows].cpu().double().numpy() - want[0][rows]).max() <= want[2][rows].max()


def test_a_chain_is_plain_decoding(tts):
    """Masks of a chain: the tokens of attn_decode_paged."""
    for f8 in (True, False):
        n = [5, 8]
        masks = [(1 << (i + 1)) - 1 for m in n for i in range(m)]
        c = Case(31, n, [300, 77], 8, 2, 128, 64, f8, 50, 3, masks=masks, junk=False)
        out, lse = c.run(tts)
        dev = [None if t is None else t.cuda() for t in (*c.c, *c.s)]
        o2, l2 = tts.attn_decode_paged(
            c.q.cuda(), dev[0], dev[1], torch.tensor(c.tables).cuda(),
            torch.tensor(c.kv, dtype=torch.int32).cuda(), c.scale, torch.tensor(c.cu).cuda(), 8,
            k_scale=dev[2], v_scale=dev[3], window=50, sinks=3)
        _, _, tol, tol_l = c.want()
        assert bool((np.abs((out - o2).cpu().double().numpy()) <= 2 * tol).all())
        assert bool((np.abs((lse - l2).cpu().double().numpy()) <= 2 * tol_l).all())


def test_same_bits_every_time(tts):
    c = Case(37, [64, 9, 30], [3000, 100, 900], 16, 4, 128, 64, True)
    a = c.run(tts)
    for _ in range(3):
        b = c.run(tts)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_many_requests(tts):
    rng = np.random.default_rng(41)
    new = [int(x) for x in rng.integers(0, 9, 200)]
    kv = [int(x) + n for x, n in zip(rng.integers(0, 300, 200), new)]
    Case(41, new, kv, 8, 4, 64, 32, True).check(tts)
    Case(42, new, kv, 4, 1, 128, 16, False, 60, 2).check(tts)


@pytest.mark.parametrize("f8", [True, False])
def test_more_requests_than_threads(tts, f8):
    """The list of tiles is added up in rounds of the block's threads."""
    rng = np.random.default_rng(47)
    new = [int(x) for x in rng.integers(0, 4, 900)]
    kv = [int(x) + n for x, n in zip(rng.integers(0, 150, 900), new)]
    new[-1], kv[-1], new[400], kv[400] = 3, 900, 40, 300
    Case(47, new, kv, 2, 1, 64, 16, f8).check(tts)


def test_scales_that_are_no_powers_of_two(tts):
    c = Case(53, [20, 3], [700, 90], 8, 2, 128, 16, True)
    rng = np.random.default_rng(1)
    c.s = [torch.tensor(np.exp(rng.uniform(-9, 1, t.shape)), dtype=torch.float32) for t in c.s]
    c.check(tts)


def test_a_large_group(tts):
    """16 q heads per KV head and 64 tokens: four row blocks of each KV head."""
    Case(59, [64, 1, 33], [500, 200, 33], 16, 1, 64, 32, True).check(tts)
    Case(61, [64], [900], 32, 1, 128, 64, False, 300, 5).check(tts)


def test_random_calls(tts):
    rng = np.random.default_rng(43)
    for i in range(40):
        hkv = int(rng.choice([1, 2, 3]))
        hq = hkv * int(rng.choice([1, 2, 4, 5, 8]))
        b = int(rng.integers(1, 6))
        most = int(rng.choice([1, 4, 16, 64]))
        new = [int(x) for x in rng.integers(0, most + 1, b)]
        kv = [int(x) for x in rng.integers(0, int(rng.choice([40, 300, 2000])), b)]
        w, s = [(0, 0), (0, 0), (int(rng.integers(1, 400)), int(rng.integers(0, 70)))][rng.integers(3)]
        Case(100 + i, new if max(new) else [1] * b, kv, hq, hkv, int(rng.choice([64, 128])),
             int(rng.choice([16, 32, 64, 128])), bool(rng.integers(2)), w, s).check(
                 tts, [torch.float32, torch.bfloat16][rng.integers(2)])


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("new,kv,hq,hkv,d,window", [
    ([3], [9000], 4, 1, 128, 0),             # one unit in as many parts as it has tiles
    ([64], [5000], 8, 1, 64, 0),             # two blocks of 256 rows, a tile counting twice
    ([40], [3003], 8, 1, 128, 700),          # one of 256 and one of 64 rows
    ([5, 0, 16], [7000, 300, 2100], 16, 2, 128, 0),  # a request without tokens between two
    ([4, 9], [0, 6001], 4, 2, 64, 0),        # nothing cached
    ([64, 1], [65, 8191], 20, 2, 128, 0),    # whole units beside cut ones, odd groups
])
def test_few_units_in_many_parts(tts, f8, new, kv, hq, hkv, d, window):
    """The workspace holds NaN before the call: what is read from it was written by the call."""
    c = Case(7, new, kv, hq, hkv, d, 64, f8, window=window, sinks=3 if window else 0)
    need = tts.attn_decode_tree_workspace_bytes(max(new), hq, hkv, d)
    for out_dtype in (torch.float32, torch.bfloat16):
        c.check(tts, out_dtype, workspace=torch.full((need,), 255, dtype=torch.uint8, device="cuda"))


def test_parts_of_rows_that_follow_in_one_run(tts):
    """Runs of many short units of 1 to 256 rows, e4m3 and bf16: the q rows of the next are written, and
    its first scores computed, while the sums of one leave."""
    rng = np.random.default_rng(11)
    for f8, d in ((True, 128), (True, 64), (False, 128), (False, 64)):
        new = [int(x) for x in rng.choice([1, 2, 15, 16, 17, 33, 64], 90)]
        kv = [n + int(x) for n, x in zip(new, rng.choice([0, 1, 63, 128, 300], 90))]
        c = Case(12, new, kv, 16, 4, d, 32, f8)
        need = tts.attn_decode_tree_workspace_bytes(64, 16, 4, d)
        c.check(tts, workspace=torch.full((need,), 255, dtype=torch.uint8, device="cuda"))


def zero_keys(c, pages=None):
    """The keys that some token sees become zeros on these pages (None: on all), with the scale that a
    page of zeros is given; the others keep what they hold."""
    at = range(c.c[0].shape[0]) if pages is None else pages
    for p in at:
        if c.f8:
            c.c[0][p] = torch.where(c.c[0][p] == 0x7F, c.c[0][p], torch.zeros_like(c.c[0][p]))
            c.s[0][p] = 2.0 ** -60
        else:
            c.c[0][p] = torch.where(c.c[0][p].isnan(), c.c[0][p], torch.zeros_like(c.c[0][p]))


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("new,kv,hq,hkv,d,ps,window,sinks", [
    ([1], [1], 1, 1, 128, 64, 0, 0),                  # one visible key
    ([9, 3], [90, 20], 4, 2, 128, 16, 0, 0),          # one tile
    ([9, 3], [90, 20], 4, 2, 64, 64, 0, 0),
    ([5], [2590], 8, 2, 64, 64, 0, 0),                # one request in many parts
    ([16, 1, 7], [900, 130, 7], 8, 2, 128, 32, 0, 0),
    ([64, 40], [700, 64], 8, 2, 128, 64, 0, 0),       # up to 256 rows: both warpgroups a q tile each
    ([12, 20] * 20, [300, 77] * 20, 4, 2, 128, 64, 100, 3),  # a window, more units than parts
    ([30, 64], [500, 300], 8, 2, 64, 16, 70, 2),
])
def test_rows_of_zeros_over_keys_of_zeros(tts, f8, new, kv, hq, hkv, d, ps, window, sinks):
    """Rows of zero q over pages of zero keys, as padding leaves them: the mean of the visible values, and
    whatever hidden keys and values hold. Zeros on one side alone, too."""
    for all_q, pages in ((True, None), (False, None), (True, "last"), (False, "last")):
        c = Case(sum(kv) + ps, new, kv, hq, hkv, d, ps, f8, window, sinks)
        zero_keys(c, None if pages is None else
                  [int(c.tables[r, (L - 1) // ps]) for r, L in enumerate(kv)])
        c.q[slice(None) if all_q else slice(0, None, 2)] = 0
        c.check(tts)


def test_zero_values_beside_others(tts):
    """Pages whose values are zeros, with the scale that they are given, among pages with others."""
    c = Case(67, [9, 20], [300, 90], 4, 2, 128, 32, True)
    for p in (int(c.tables[0, 1]), int(c.tables[1, 2])):
        c.c[1][p] = torch.where(c.c[1][p] == 0x7F, c.c[1][p], torch.zeros_like(c.c[1][p]))
        c.s[1][p] = 2.0 ** -60
    c.q[3] = 0
    zero_keys(c, [int(c.tables[0, 1])])
    c.check(tts)


@pytest.mark.parametrize("scale", [1e-38, 1e-45])
def test_the_smallest_scales(tts, scale):
    """A scale whose product with a page's underflows: every visible key has the same weight."""
    for f8 in (True, False):
        c = Case(71, [9, 3], [400, 20], 4, 2, 128, 64, f8)
        c.scale = scale
        if f8:
            c.s[0][:] = 2.0 ** -40
        c.check(tts)


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("new,kv,hq,hkv,d,ps", [
    ([9, 3], [300, 20], 4, 2, 128, 64),
    ([5], [2590], 8, 2, 64, 16),
    ([64], [700], 8, 2, 128, 32),
])
@pytest.mark.parametrize("exp", [10, 20, 22])
def test_scores_up_to_their_limit(tts, f8, new, kv, hq, hkv, d, ps, exp):
    """Scores up to 2^exp in units of log2: finite, and the value of the key with the largest score where that
    one leads by more than scores are off. Masks of a chain, so that plain decoding is the same."""
    masks = [(1 << (i + 1)) - 1 for n in new for i in range(n)]
    c = Case(73 + exp, new, kv, hq, hkv, d, ps, f8, masks=masks, gain=16.0)
    if f8:
        c.s[0][:] = 2.0 ** -3
    k, v = (np.nan_to_num(ref.codes_of(t)) for t in c.c)
    s = [1.0 if t is None else t.numpy()[:, :, None, None] for t in c.s]
    k, v = k * s[0], v * s[1]
    rows, most = [], 0
    for r, (n, L) in enumerate(zip(new, kv)):
        j = np.arange(L)
        at = (c.tables[r, j // ps], slice(None), j % ps)
        for i in range(n):
            q = c.q[c.cu[r] + i].double().numpy().reshape(hkv, hq // hkv, d)
            see = tree_ref.sees(masks[c.cu[r] + i], n, L, 0, 0)
            K, V = k[at][see].transpose(1, 0, 2), v[at][see].transpose(1, 0, 2)
            x = q @ K.transpose(0, 2, 1) * np.log2(np.e)
            most = max(most, np.abs(x).max())
            # products summed in fp32, q over e4m3 keys to 2^-17 of its row's largest value
            off = 3 * d * 2.0 ** -24 * (np.abs(q) @ np.abs(K).transpose(0, 2, 1)).max(-1) + \
                2.0 ** -16 * np.abs(q).max(-1) * np.abs(K).sum(-1).max()
            rows.append((x, off * np.log2(np.e), V))
    c.scale = float(np.float32(2.0 ** exp / most))
    dev = [None if t is None else t.cuda() for t in (*c.c, *c.s)]
    plain = tts.attn_decode_paged(
        c.q.cuda(), dev[0], dev[1], torch.tensor(c.tables).cuda(),
        torch.tensor(c.kv, dtype=torch.int32).cuda(), c.scale, torch.tensor(c.cu).cuda(), max(new),
        k_scale=dev[2], v_scale=dev[3])
    for out, lse in (c.run(tts), plain):
        got = out.cpu().double().numpy().reshape(len(rows), hkv, hq // hkv, d)
        l = lse.cpu().double().numpy().reshape(len(rows), hkv, hq // hkv)
        assert np.isfinite(got).all() and np.isfinite(l).all()
        led = 0
        for (x, off, V), o, lo in zip(rows, got, l):
            x, off = x * c.scale, off * c.scale + 8
            top = np.sort(x, -1)
            lead = top[..., -1] - top[..., -2] if x.shape[-1] > 1 else np.full(x.shape[:2], np.inf)
            for g, h in zip(*np.nonzero(lead > 2 * off + 40)):
                led += 1
                want = V[g, x[g, h].argmax()]
                # the weight is rounded to fp16 or bf16; the others are under 2^-25 of it
                assert (np.abs(o[g, h] - want) <= 2.0 ** (-9 if f8 else -7) * np.abs(want)
                        + 2.0 ** -25 * np.abs(V[g]).sum(0)).all()
                assert abs(lo[g, h] * np.log2(np.e) - top[g, h, -1]) <= off[g, h] + 20
        assert led > 0 or exp < 20
