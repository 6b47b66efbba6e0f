"""ssd_kv_attend_tree against a plain form in 64 bits, at the trees, sizes and masks where it can go wrong.
The tolerance is derived in _tree_ref.attend_bound."""
import numpy as np
import pytest

import _loop_ref as loop
import _tree_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
VALUES = loop.e4m3_values()
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_ssd_gb300 as m
    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    """Inputs on the host, with spare pages full of NaN that no table names."""

    def __init__(self, seed, pairs, Hq, Hkv, D, P, dtype, kind="random", spread=1.0, spare=2):
        rng = self.rng = np.random.default_rng(seed)
        self.P, self.D, self.dtype = P, D, dtype
        blocks = [-(-max(kv, 0) // P) for kv, _ in pairs]
        N = sum(blocks) + spare
        pages = rng.permutation(N)
        self.table = np.full((len(pairs), max(1, max(blocks))), -1, np.int32)
        at = 0
        for b, m in enumerate(blocks):
            self.table[b, :m] = pages[at:at + m]
            at += m

        def cache():
            codes = rng.integers(0, 256, (N, Hkv, P, D)).astype(np.uint8)
            # mostly small values, as quantised activations are
            codes = np.where(rng.random(codes.shape) < 0.9, (codes & 0x80) | (0x20 + (codes & 0x1F)), codes).astype(np.uint8)
            codes[(codes & 127) == 127] = 0x30
            # rows behind a sequence's end and pages that nobody holds are full of NaN
            codes[pages[at:]] = 0x7F
            for b, (kv, _) in enumerate(pairs):
                if kv % P and kv > 0:
                    codes[self.table[b, kv // P], :, kv % P:] = 0xFF if b % 2 else 0x7F
            scale = (0.02 * np.exp(0.5 * rng.standard_normal((N, Hkv)))).astype(np.float32)
            return codes, scale

        (self.k, self.ks), (self.v, self.vs) = cache(), cache()
        self.kv = np.array([kv for kv, _ in pairs], np.int32)
        self.cu = np.concatenate([[0], np.cumsum([n for _, n in pairs])]).astype(np.int32)
        T = int(self.cu[-1])
        self.max_new = max(1, max(n for _, n in pairs))
        parent = sum([ref.parents(kind, n, rng) for _, n in pairs], [])
        self.sees = ref.tree_plan(parent, self.cu.tolist(), [0] * len(pairs), T, self.max_new)[1]
        self.q = torch.from_numpy(rng.standard_normal((T, Hq, D)) * spread).to(dtype)
        self.scale = 1 / np.sqrt(D)

    def run(self, ssd, window=0, pad=0, mask=None, **kw):
        T, Hq, D = self.q.shape
        q = torch.zeros((T, Hq * D + pad), dtype=self.dtype, device="cuda")
        q[:, :Hq * D] = self.q.reshape(T, -1).cuda()
        max_new = kw.pop("max_new", self.max_new)
        if mask is None:
            W = -(-max_new // 32)
            mask = ref.words([{j for j in s if j < 32 * W} for s in self.sees], W)
        out = ssd.ssd_kv_attend_tree(q[:, :Hq * D].unflatten(1, (Hq, D)), dev(self.k), dev(self.v), dev(self.ks), dev(self.vs),
                                     dev(self.table), dev(self.cu), dev(self.kv), dev(mask), max_new, self.scale, window=window, **kw)
        torch.cuda.synchronize()
        return out

    def want(self, window=0, max_new=1 << 30):
        with np.errstate(invalid="ignore"):
            return ref.attend_tree(self.q.double().numpy(), VALUES[self.k], VALUES[self.v], self.ks.astype(np.float64),
                                   self.vs.astype(np.float64), self.table, self.cu, self.kv, self.sees, self.P, self.scale, window, max_new)

    def check(self, ssd, window=0, pad=0, **kw):
        got = self.run(ssd, window, pad, **kw).double().cpu().numpy()
        want = self.want(window, kw.get("max_new", 1 << 30))
        bound = ref.attend_bound(self.dtype, self.D, *want)
        assert not np.isnan(got).any()
        over = np.abs(got - want[0]) - bound
        assert over.max() <= 0, (over.max(), np.unravel_index(over.argmax(), over.shape))
        return got


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("pairs,Hq,Hkv,D,P", [
    ([(1, 1)], 1, 1, 64, 16),
    ([(1, 1)], 8, 1, 128, 128),
    ([(7, 7)], 4, 1, 128, 16),
    ([(15, 1), (16, 2), (17, 3)], 4, 2, 64, 16),
    ([(127, 1), (128, 5), (129, 6), (255, 2), (256, 3), (257, 4)], 8, 2, 128, 64),
    ([(640, 5), (5, 5), (6, 5), (133, 5), (3, 5)], 32, 8, 128, 64),           # the last one: kv < new
    ([(0, 1), (0, 3), (200, 4), (0, 0), (129, 0)], 4, 4, 64, 32),             # nothing cached, nothing new
    ([(2500, 9)], 8, 8, 128, 128),
    ([(3000, 1)], 16, 1, 64, 32),
    ([(300, 37), (44, 21)], 12, 4, 128, 32),                                  # groups of three
    ([(700, 37)], 7, 1, 64, 64),                                              # groups of seven, 259 rows
    ([(700, 32), (500, 33)], 8, 2, 128, 64),                                  # 128 and 132 rows
    ([(900, 64), (90, 64), (64, 64), (1200, 65)], 8, 2, 128, 128),            # 256 and 260 rows
    ([(260, 130)], 6, 2, 128, 16),                                            # the tree over tile edges
    ([(600, 509), (700, 33)], 4, 2, 64, 64),
    ([(1500, 1024)], 2, 1, 64, 16),
])
def test_attend_matches_plain_form(ssd, pairs, Hq, Hkv, D, P, dtype):
    Case(len(pairs) * 100 + Hq + D, pairs, Hq, Hkv, D, P, dtype).check(ssd)


@pytest.mark.parametrize("kind", ["chain", "star", "flat"])
def test_kinds_of_trees(ssd, kind):
    Case(1, [(300, 20), (9, 9), (130, 40)], 8, 2, 128, 16, BF, kind).check(ssd)
    Case(2, [(300, 20), (9, 9), (130, 40)], 4, 4, 64, 64, FP, kind).check(ssd)


@pytest.mark.parametrize("window", [1, 2, 3, 7, 31, 128, 129, 200, 100000])
def test_window(ssd, window):
    Case(window, [(513, 25), (128, 1), (140, 70), (12, 5), (900, 3)], 8, 2, 128, 16, BF).check(ssd, window=window)
    Case(window, [(385, 129), (1, 1)], 2, 2, 64, 64, FP).check(ssd, window=window)


def test_any_mask(ssd):
    """Masks that are no tree's: bits of later nodes do not count, a token need not see itself, and some see nothing."""
    for window in (0, 3):
        c = Case(3, [(300, 40), (40, 40), (9, 9)], 8, 2, 64, 16, BF)
        c.sees = [set(c.rng.choice(40, int(c.rng.integers(0, 30)), replace=False).tolist()) for _ in c.sees]
        c.sees[45] = set()
        c.sees[50] = {39}
        got = c.check(ssd, window=window)
        assert not got[45].any() and not got[50].any() and got[0].any()


@pytest.mark.parametrize("window", [0, 50])
def test_a_chain_is_causal_attention(ssd, window):
    """Against ssd_kv_attend: both within their bounds of the same values."""
    c = Case(4, [(513, 25), (128, 1), (7, 7), (900, 60)], 8, 2, 128, 32, BF, "chain")
    got = c.check(ssd, window=window)
    other = ssd.ssd_kv_attend(c.q.cuda(), dev(c.k), dev(c.v), dev(c.ks), dev(c.vs), dev(c.table), dev(c.cu), dev(c.kv), c.max_new, c.scale,
                              window=window).double().cpu().numpy()
    want = loop.attend(c.q.double().numpy(), VALUES[c.k], VALUES[c.v], c.ks.astype(np.float64), c.vs.astype(np.float64), c.table, c.cu, c.kv,
                       c.P, c.scale, window)
    far = ref.attend_bound(BF, c.D, *c.want(window)) + loop.attend_bound(BF, c.D, *want)
    assert (np.abs(got - other) <= far).all()


@pytest.mark.parametrize("B,hi", [(40, 1500), (300, 90), (700, 40)])
def test_many_ragged_sequences(ssd, B, hi):
    rng = np.random.default_rng(B)
    pairs = [(int(rng.integers(0, hi)), int(rng.integers(0, 9))) for _ in range(B)]
    Case(B, pairs, 4, 2, 64, 16, BF).check(ssd)


def test_many_sequences_of_several_row_blocks(ssd):
    """More (sequence, row block) pairs than every CTA puts in order for itself."""
    rng = np.random.default_rng(8)
    pairs = [(int(rng.integers(60, 200)), int(rng.choice([0, 1, 33, 70]))) for _ in range(150)]
    Case(8, pairs, 8, 1, 64, 32, BF).check(ssd)


def test_strided_queries(ssd):
    Case(1, [(300, 15), (77, 3)], 8, 2, 128, 32, BF).check(ssd, pad=1024)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_sharp_softmax(ssd, dtype):
    """Scores of some hundreds: one key takes all."""
    Case(2, [(500, 13), (90, 2)], 4, 2, 64, 32, dtype, spread=60.0).check(ssd)


def test_maxima_that_rise_and_fall(ssd):
    """Keys whose size grows along the sequence, or falls: the running maximum is passed again and again."""
    for up in (1, -1):
        c = Case(5, [(3000, 20), (2999, 70)], 8, 2, 128, 32, BF, spread=4.0)
        for b in range(2):
            held = c.table[b][c.table[b] >= 0]
            c.ks[held] *= (2.0 ** (np.arange(len(held))[::up] * 0.08))[:, None].astype(np.float32)
        c.check(ssd)


def test_flat_tail_next_to_a_large_weight(ssd):
    """One key of weight 1/2 and 60000 that share the other half: the small ones must not vanish."""
    n, D = 60001, 64
    for place in (0, 30000, 59990):
        k = torch.zeros((469, 1, 128, D), dtype=torch.float32)
        k.view(-1, D)[place, 0] = 256.0
        v = torch.ones((469, 1, 128, D))
        v.view(-1, D)[place] = 0.0
        q = torch.zeros((1, 1, D), dtype=BF)
        q[0, 0, 0] = 1.0
        g = lambda a: a.to(torch.float8_e4m3fn).cuda()  # noqa: E731
        one = torch.ones((469, 1), device="cuda")
        i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
        scale = float(np.log(60000.0) / 256.0)
        out = ssd.ssd_kv_attend_tree(q.cuda(), g(k), g(v), one, one, torch.arange(469, dtype=torch.int32, device="cuda")[None], i([0, 1]),
                                     i([n]), i([[1]]), 1, scale)
        assert float((out.float() - 0.5).abs().max()) <= 0.5 * (2.0 ** -8 + 2.0 ** -9)


def test_scales_of_very_different_size(ssd):
    for dtype in (BF, FP):
        c = Case(3, [(700, 25)], 4, 2, 64, 16, dtype)
        c.vs *= (10.0 ** np.random.default_rng(3).uniform(-6, 2, c.vs.shape)).astype(np.float32)
        c.vs[c.table[0, 3]] = 0.0
        c.vs[c.table[0, 5]] *= -1
        c.ks[c.table[0, 6]] *= -1
        c.ks[c.table[0, 7]] = 0.0
        c.check(ssd)


def test_nan_in_some_nodes_stays_with_those_that_see_them(ssd):
    for n, Hq in ((12, 4), (90, 8)):
        c = Case(4, [(300, n), (200, 3)], Hq, 2, 64, 32, BF)
        want = c.run(ssd).double().cpu().numpy()
        node = n // 3
        j = 300 - n + node
        c.v[c.table[0, j // 32], 1, j % 32, 7] = 0x7F      # head 1, channel 7
        j = 300 - n + node + 1
        c.k[c.table[0, j // 32], 0, j % 32, 9] = 0xFF      # head 0: every channel of those that see it
        got = c.run(ssd).double().cpu().numpy()
        nan = np.zeros(got.shape, bool)
        G = Hq // 2
        for t in range(n):
            if node in c.sees[t]:
                nan[t, G:, 7] = True
            if node + 1 in c.sees[t]:
                nan[t, :G] = True
        assert nan[:, :G].any() and nan[:, G:].any()
        np.testing.assert_array_equal(np.isnan(got), nan)
        np.testing.assert_allclose(got[~nan], want[~nan], rtol=2.0 ** -7, atol=1e-6)


def test_nan_in_masked_nodes_has_no_effect(ssd):
    """Values and keys of nodes that a window hides from all, and queries that are not finite."""
    c = Case(6, [(300, 20)], 4, 2, 64, 32, BF, "chain")
    want = c.check(ssd, window=5)
    for j in range(290 - 30):
        c.v[c.table[0, j // 32], :, j % 32] = 0x7F
        c.k[c.table[0, j // 32], :, j % 32] = 0xFF
    np.testing.assert_array_equal(c.run(ssd, window=5).double().cpu().numpy(), want)
    c.q[3, 1, 5], c.q[7, 2, 0] = float("nan"), float("inf")
    got = c.run(ssd, window=5).double().cpu().numpy()
    bad = np.zeros(got.shape[:2], bool)
    bad[3, 1] = bad[7, 2] = True
    np.testing.assert_array_equal(np.isnan(got).all(axis=2), bad)
    np.testing.assert_array_equal(got[~bad], want[~bad])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("window,page", [(0, 18), (10, 17)])
def test_a_value_scale_that_is_not_finite_stays_with_those_that_see_it(ssd, dtype, bad, window, page):
    """Of tokens at 285 to 290 the last three see the page of positions 288 on; of those at 294 to 299, with a window of 10,
    the first three that of 272 to 287."""
    c = Case(12, [(291, 6)] if window == 0 else [(300, 6)], 4, 2, 64, 16, dtype, "chain")
    c.vs[c.table[0, page], 1] = bad
    got = c.run(ssd, window=window).double().cpu().numpy()
    want = c.want(window)
    sees = ~np.isfinite(want[0])
    assert sees[:, 2:].any() and not sees[:, 2:].all() and not sees[:, :2].any()
    np.testing.assert_array_equal(~np.isfinite(got), sees)
    c.vs[c.table[0, page], 1] = 0.02       # what the bound is relative to, without it
    bound = ref.attend_bound(dtype, c.D, *c.want(window))
    assert (np.abs(got - want[0])[~sees] <= bound[~sees]).all()


@pytest.mark.parametrize("dtype,scale,spread", [(BF, 0.0, 1.0), (FP, 0.0, 1.0), (BF, -0.0, 1.0), (BF, 1e-30, 1e-30), (BF, -1e-44, 1.0),
                                                (FP, 1e-38, 1.0), (FP, 3e-41, 1e-3), (BF, -0.1, 1.0)])
def test_scale_of_zero_and_scales_that_vanish(ssd, dtype, scale, spread):
    c = Case(13, [(300, 6), (17, 17), (700, 1), (3, 5)], 4, 2, 64, 16, dtype, spread=spread)
    c.scale = scale
    c.check(ssd)
    c.check(ssd, window=37)


def test_pages_outside_the_cache_count_as_not_there(ssd):
    c = Case(5, [(200, 13), (90, 2)], 4, 2, 64, 16, BF)
    c.table[0, 2], c.table[0, 12], c.table[1, 0] = -1, 10 ** 6, len(c.k)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(ssd, dev_status=status)
    assert int(status) == ssd.SSD_DEV_BAD_PAGE


def _status(ssd, c, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(ssd, dev_status=status, **kw)
    return int(status)


@pytest.mark.parametrize("kv", [65, 70, 10 ** 9, -1, -5])
def test_a_length_that_the_table_cannot_hold_is_reported(ssd, kv):
    c = Case(6, [(64, 4), (50, 3)], 2, 2, 64, 16, BF)
    assert _status(ssd, c) == 0
    c.kv[0] = kv
    assert _status(ssd, c) == ssd.SSD_DEV_BAD_LENGTH


def test_tokens_beyond_the_bound_get_zeros(ssd):
    c = Case(6, [(64, 4), (50, 9)], 2, 2, 64, 16, BF)
    assert _status(ssd, c, max_new=5) == ssd.SSD_DEV_BAD_LENGTH
    got = c.check(ssd, max_new=5)
    assert not got[9:].any()
    c = Case(7, [(64, 4)], 2, 2, 64, 16, BF)
    c.q = torch.cat([c.q, c.q])
    c.sees = c.sees * 2
    got = c.run(ssd).cpu()
    assert got[:4].abs().sum() > 0 and not got[4:].any()


def test_token_counts_that_pass_the_queries_or_fall_are_reported(ssd):
    c = Case(6, [(64, 4), (50, 3)], 2, 2, 64, 16, BF)
    want = c.run(ssd)
    ws = ssd.kv_tree_workspace()
    for cu in ([0, 4, 9], [0, 9, 4], [-2, 4, 7]):
        bad = Case(6, [(64, 4), (50, 3)], 2, 2, 64, 16, BF)
        bad.cu = np.array(cu, np.int32)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        bad.run(ssd, max_new=5, dev_status=status, workspace=ws)
        assert int(status) & ssd.SSD_DEV_BAD_LENGTH
        assert torch.equal(c.run(ssd, workspace=ws), want)


def test_token_counts_that_go_back_and_forth_are_bounded(ssd):
    """cu_new going back and forth would make many row blocks of few tokens."""
    ws = ssd.kv_tree_workspace()
    good = Case(14, [(300, 200), (90, 70)], 8, 2, 64, 16, BF)
    want = good.run(ssd, workspace=ws)
    c = Case(14, [(300, 200)] + [(20, 0)] * 39, 8, 2, 64, 16, BF)
    c.cu = np.array([0, 200] * 20 + [0], np.int32)
    c.kv[:] = 300
    c.table[:] = c.table[0]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.run(ssd, workspace=ws, dev_status=status)
    assert int(status) == ssd.SSD_DEV_BAD_LENGTH
    assert torch.equal(good.run(ssd, workspace=ws), want)


def test_cache_beyond_32_bits_of_bytes(ssd):
    N, H, P, D = 70000, 8, 128, 64          # 4.6 GB each
    small = Case(8, [(300, 12)], 8, 8, 64, 128, BF)
    k = torch.full((N, H, P, D), 0x7F, dtype=torch.uint8, device="cuda")
    v = k.clone()
    s = [torch.full((N, H), float("nan"), device="cuda") for _ in range(2)]
    at = [N - 1, 3, N // 2 + 1]
    for dst, src in zip(at, small.table[0]):
        k[dst], v[dst] = dev(small.k[src]), dev(small.v[src])
        s[0][dst], s[1][dst] = dev(small.ks[src]), dev(small.vs[src])
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    got = ssd.ssd_kv_attend_tree(small.q.cuda(), k, v, s[0], s[1], i([at]), i([0, 12]), i([300]), dev(ref.words(small.sees, 1)), 12,
                                 small.scale)
    assert torch.equal(got, small.run(ssd))


def test_same_bits_every_time_with_one_workspace(ssd):
    c = Case(9, [(5000, 37), (17, 2), (3001, 50)], 8, 2, 128, 64, BF)
    ws = ssd.kv_tree_workspace()
    first = c.run(ssd, workspace=ws)
    for _ in range(5):
        assert torch.equal(c.run(ssd, workspace=ws), first)
    small = Case(10, [(9, 1)], 8, 2, 128, 64, BF)
    assert torch.equal(small.run(ssd, workspace=ws), small.run(ssd))


def test_in_a_graph_and_on_another_stream(ssd):
    c = Case(11, [(1500, 15), (800, 15)], 8, 2, 128, 64, BF)
    want = c.run(ssd)
    q, k, v, ks, vs, table, cu, kv = c.q.cuda(), dev(c.k), dev(c.v), dev(c.ks), dev(c.vs), dev(c.table), dev(c.cu), dev(c.kv)
    mask = dev(ref.words(c.sees, 1))
    ws, out = ssd.kv_tree_workspace(), torch.zeros_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = ssd.ssd_kv_attend_tree(q, k, v, ks, vs, table, cu, kv, mask, 15, c.scale, stream=s)
    s.synchronize()
    assert torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssd.ssd_kv_attend_tree(q, k, v, ks, vs, table, cu, kv, mask, 15, c.scale, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    kv[0] = 700  # lengths and masks are read on the device: a replay follows them
    mask[3] = 1
    graph.replay()
    c.kv[0], c.sees[3] = 700, {0}
    torch.cuda.synchronize()
    assert torch.equal(out, c.run(ssd))


def test_two_graphs_with_one_workspace(ssd):
    """Captured one after the other and replayed in turn: one makes its schedule in every CTA, one in the workspace."""
    ws = ssd.kv_tree_workspace()
    made = []
    for c in (Case(21, [(1500, 15), (800, 15)], 8, 2, 128, 64, BF), Case(22, [(900, 150), (3000, 90), (70, 70)] + [(40, 2)] * 300, 8, 2, 128, 64, BF)):
        want = c.run(ssd)
        out = torch.zeros_like(want)
        mask = dev(ref.words(c.sees, -(-c.max_new // 32)))
        a = (c.q.cuda(), dev(c.k), dev(c.v), dev(c.ks), dev(c.vs), dev(c.table), dev(c.cu), dev(c.kv), mask, c.max_new, c.scale)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ssd.ssd_kv_attend_tree(*a, out=out, workspace=ws)
        made.append((graph, out, want, a))
    for turn in ((0, 1, 0), (1, 1, 0, 1)):
        for i in turn:
            made[i][1].zero_()
            made[i][0].replay()
        torch.cuda.synchronize()
        for _, out, want, _ in made:
            assert torch.equal(out, want)


def test_no_tokens(ssd):
    c = Case(23, [(50, 2), (9, 1)], 4, 2, 64, 16, BF)
    none = torch.zeros((0, 1), dtype=torch.int32, device="cuda")
    out = ssd.ssd_kv_attend_tree(c.q[:0].cuda(), dev(c.k), dev(c.v), dev(c.ks), dev(c.vs), dev(c.table), dev(c.cu * 0), dev(c.kv), none, 2,
                                 c.scale)
    assert out.shape == (0, 4, 64)
    c.cu[:] = 0                            # tokens, but none of any sequence's
    assert not c.run(ssd).any()


def test_bounds_far_above_what_comes(ssd):
    """max_new at its limit over one-token sequences, a window of the largest integer, and mask bits of nodes that are not there."""
    c = Case(24, [(300, 1), (7, 7), (0, 0), (33, 2)], 8, 2, 64, 16, BF)
    c.max_new = ssd.SSD_TREE_MAX
    mask = np.array(ref.words(c.sees, 32))
    c.check(ssd, window=2 ** 31 - 1)
    for t, i in zip(range(10), [0, 0, 1, 2, 3, 4, 5, 6, 0, 1]):
        mask[t, 1:] = -1
        mask[t, 0] |= np.int32(-2) << i    # later nodes
    assert torch.equal(c.run(ssd, mask=mask), c.run(ssd))


@pytest.mark.parametrize("times", [30.0, 1000.0])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_queries_with_one_large_channel(ssd, dtype, times):
    """A query's digits end at 2^-17 of its row's largest channel: what that can move a score by, 2^-17 |scale| max |q| sum |k|,
    moves a weight by as much and their total once more, next to the bound of the other roundings."""
    c = Case(17, [(700, 25), (40, 40)], 8, 2, 128, 32, dtype)
    c.q[:, :, 5] *= times
    c.k[..., 5] = 1                        # 2^-9: the scores are those of the small channels
    got = c.run(ssd).double().cpu().numpy()
    want = c.want()
    held = np.unique(c.table[c.table >= 0])
    k = np.nansum(np.abs(VALUES[c.k[held]]) * c.ks[held][:, :, None, None], axis=3).max()
    moved = 2.0 ** -17 * c.scale * np.abs(c.q.double().numpy()).max(axis=2, keepdims=True) * k
    bound = ref.attend_bound(dtype, c.D, *want) + 2 * moved * want[1]
    assert (np.abs(got - want[0]) <= bound).all()


def check_seen(c, got, window=0, rows=slice(None)):
    """Against the bound that is relative to what each token attends to, and to nothing else."""
    args = (c.table, c.cu, c.kv, c.sees, c.P, c.scale, window)
    ks, vs = c.ks.astype(np.float64), c.vs.astype(np.float64)
    out, weight, score, _, count = c.want(window)
    floor = ref.seen_floor(c.q.double().numpy(), VALUES[c.k], ks, vs, *args)
    bound = ref.seen_bound(c.dtype, c.D, out, weight, score, floor, count)
    over = (np.abs(got.double().cpu().numpy() - out) - bound)[rows]
    assert over.max() <= 0, (over.max(), np.unravel_index(over.argmax(), over.shape))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("times", [30, 60, 100])
@pytest.mark.parametrize("n,window", [(40, 0), (40, 40), (150, 0)])
def test_a_large_value_scale_concerns_those_alone_that_see_it(ssd, dtype, times, n, window):
    """Nodes 12 to 27 lie in a page of far larger scale, and every other token attends to none of them."""
    c = Case(31, [(260 + n, n), (300, 3)], 4, 2, 64, 16, dtype, "chain")
    hidden = set(range(12, 28))
    for t in range(0, n, 2):
        c.sees[t] -= hidden
    want = c.run(ssd, window=window)
    check_seen(c, want, window)
    c.vs[c.table[0, 17]] *= np.float32(2.0 ** times)
    got = c.run(ssd, window=window)
    check_seen(c, got, window, slice(None) if dtype == BF else slice(0, n, 2))      # (what fp16 does not hold is left out)
    if times == 30:
        assert torch.equal(got[0:n:2], want[0:n:2])


@pytest.mark.parametrize("times", [30, 60])
@pytest.mark.parametrize("page", [0, 5, 17])
def test_the_largest_score_next_to_the_largest_value_scale(ssd, times, page):
    """A page of far larger value scale, whose keys all score 2^-(times + 20) of the others: what it adds is little, and
    the others' weights keep their bits."""
    for dtype in (BF, FP):
        c = Case(32, [(300, 20), (77, 7)], 4, 2, 64, 16, dtype)
        p = c.table[0, page]
        c.q[:, :, 5] = 4.0
        c.k[..., 5] = 0
        c.k[p, ..., 5] = 0xFE                                    # -448
        c.ks[p] = 0.02
        c.scale = (times + 20) * float(np.log(2.0)) / (4 * 448 * 0.02)
        c.vs[p] = 0.02 * 2.0 ** times
        check_seen(c, c.run(ssd))


def test_value_scales_of_all_sizes(ssd):
    """From 2^-120 to 2^100, none and negative ones among them, with a mask that shows each token some pages."""
    for seed, dtype in ((33, BF), (34, BF)):
        c = Case(seed, [(400, 60), (200, 9)], 4, 2, 64, 16, dtype, spread=8.0)
        c.vs *= (2.0 ** c.rng.uniform(-115, 105, c.vs.shape)).astype(np.float32)
        c.vs[c.table[0, 3]] = 0.0
        c.vs[c.table[0, 5]] *= -1
        c.sees = [{j for j in s if c.rng.random() < 0.7} for s in c.sees]
        for window in (0, 23):
            check_seen(c, c.run(ssd, window=window), window)


@pytest.mark.parametrize("size", [40.0, 64.0, 2.0 ** 13, 2.0 ** 20, 2.0 ** 27, 1e15, 1e28, 1e31])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_scores_of_any_size(ssd, dtype, size, sign):
    """Scores are whole multiples of `size`, so that the keys of the largest share all: a weight's half, the sums of equal
    numbers and half a step of the output are what is rounded, and exponents up to 8192 twice (half a step of fp32, 2^-24 of
    the score), for a weight and for their total; larger scores enter as their differences."""
    for seed, (kv, n) in enumerate(((500, 30), (40, 30), (1300, 90))):
        c = Case(seed, [(kv, n)], 4, 2, 64, 64, dtype, "chain")
        level = c.rng.integers(2, 9, c.k.shape[:3])
        at = [(c.table[0, j // 64], j % 64) for j in (3, kv - n // 2)]
        for page, row in at:
            level[page, :, row] = 1 if sign < 0 else 9
        if kv > 500:                                             # one that only some see is by itself
            level[at[0][0], :, at[0][1]] = 5
        c.k[:] = 0
        c.k[..., 0] = np.array([loop.e4m3_values().tolist().index(float(v)) for v in range(10)])[level]
        c.ks[:], c.q[:], c.scale = 1.0, 0, size
        c.q[..., 0] = float(sign)
        got = c.run(ssd).double().cpu().numpy()
        out, weight, score, _, count = c.want()
        half = torch.finfo(dtype).eps / 2
        d = 2.0 ** -11 + 2.0 ** -20 + 2 * count * 2.0 ** -23 + 4 * 2.0 ** -24 * np.minimum(score, 8192 * np.log(2))
        bound = half * np.abs(out) + (1 + half) * d * weight + 2.0 ** -24
        over = np.abs(got - out) - bound
        assert over.max() <= 0, (over.max(), np.unravel_index(over.argmax(), over.shape))


@pytest.mark.parametrize("rest", [[40], [40, 60], [40, 60, 0, 90, 300], [0] * 300, [40, 90] * 200])
@pytest.mark.parametrize("n", [50, 150])
def test_a_batch_ends_where_its_token_counts_fall(ssd, n, rest):
    """Sequences before the fall are what they are without the rest, and no other token has an owner."""
    c = Case(41, [(400 + n, n)] + [(90, 0)] * len(rest), 8, 2, 64, 16, BF)
    c.q = torch.cat([c.q, c.q])
    c.sees = c.sees * 2
    c.kv[:] = 400 + n
    c.table[:] = c.table[0]
    want = c.run(ssd)
    assert want[:n].abs().sum() > 0 and not want[n:].any()
    c.cu[2:] = rest
    c.cu[2] = min(c.cu[2], n - 1)
    for _ in range(10):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        assert torch.equal(c.run(ssd, dev_status=status), want)
        assert int(status) == ssd.SSD_DEV_BAD_LENGTH


@pytest.mark.parametrize("withheld", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("n", [20, 50])
def test_waits_that_run_out_end_the_launch(ssd, n, withheld):
    """One signal left out in every CTA: each role leaves by itself, the status says so, and the next call is as ever."""
    import ctypes
    c = Case(42, [(40000, n), (300, 3), (129, 4)], 4, 1, 64, 64, BF)
    want = c.run(ssd)
    q, out, status = c.q.cuda(), torch.empty_like(want), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = ssd.kv_tree_workspace()
    held = [dev(a) for a in (c.k, c.v, c.ks, c.vs, c.table, c.cu, c.kv, ref.words(c.sees, -(-c.max_new // 32)))]
    k, v, ks, vs, table, cu, kv, mask = (t.data_ptr() for t in held)
    T, Hq, D = q.shape
    call = (q.data_ptr(), ssd.SSD_BF16, Hq * D, k, v, ks, vs, len(c.k), c.P, Hq, 1, D, table, c.table.shape[1], cu, kv, mask, 3, T, c.max_new,
            ctypes.c_float(c.scale), 0, out.data_ptr(), ws.data_ptr(), ws.numel(), status.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert ssd.lib().ssd_check_tree_timeout(withheld, *call) == ssd.SSD_OK
    torch.cuda.synchronize()
    assert int(status) == ssd.SSD_DEV_TIMEOUT
    ws.zero_()
    status.zero_()
    out.zero_()
    assert ssd.lib().ssd_kv_attend_tree(*call) == ssd.SSD_OK
    assert torch.equal(out, want) and int(status) == 0


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("times", [0.12, 0.49, 0.51, 2.0, 100.0])
def test_scores_as_large_as_their_digits_can_make_them(ssd, dtype, D, times):
    """Every channel of queries and keys at the end of its range, alike or opposite: no weight leaves fp16's."""
    c = Case(43, [(700, 30), (90, 5)], 4, 2, D, 64, dtype)
    c.q = torch.where(c.q > 0, 255.0, -255.0).to(dtype)
    sign = np.where(np.asarray(c.q[0, ::2].double()) > 0, 0, 0x80).astype(np.uint8)             # of each cache head's first query
    level = c.rng.choice([0x7E, 0x7D, 0x70], c.k.shape[:3] + (1,)) | (c.rng.random(c.k.shape[:3] + (1,)) < 0.5) * 0x80
    c.k[:] = (level.astype(np.uint8) ^ sign[None, :, None, :])
    c.q[:, ::2] = c.q[0, ::2]
    c.ks[:] = 1.0
    c.scale = times / float(np.log2(np.e))
    c.check(ssd)
