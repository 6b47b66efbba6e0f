"""ssd_kv_attend against a plain form in 64 bits, at the sizes and masks where it can go wrong.
The tolerance is derived in _loop_ref.attend_bound."""
import numpy as np
import pytest

import _loop_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
VALUES = ref.e4m3_values()
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_ssd_gb300 as m
    return m


class Case:
    """Inputs on the host, with spare pages full of NaN that no table names."""

    def __init__(self, seed, pairs, Hq, Hkv, D, P, dtype, spread=1.0, spare=2):
        rng = np.random.default_rng(seed)
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
        self.q = torch.from_numpy(rng.standard_normal((T, Hq, D)) * spread).to(dtype)
        self.max_new = max(1, max(n for _, n in pairs))
        self.scale = 1 / np.sqrt(D)

    def run(self, ssd, window=0, pad=0, **kw):
        T, Hq, D = self.q.shape
        q = torch.zeros((T, Hq * D + pad), dtype=self.dtype, device="cuda")
        q[:, :Hq * D] = self.q.reshape(T, -1).cuda()
        g = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        out = ssd.ssd_kv_attend(q[:, :Hq * D].unflatten(1, (Hq, D)), g(self.k), g(self.v), g(self.ks), g(self.vs),
                                g(self.table), g(self.cu), g(self.kv), kw.pop("max_new", self.max_new), self.scale,
                                window=window, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, ssd, window=0, pad=0, **kw):
        got = self.run(ssd, window, pad, **kw).double().cpu().numpy()
        want = ref.attend(self.q.double().numpy(), VALUES[self.k], VALUES[self.v], self.ks.astype(np.float64),
                          self.vs.astype(np.float64), self.table, self.cu, self.kv, self.P, self.scale, window,
                          kw.get("max_new", 1 << 30))
        bound = ref.attend_bound(self.dtype, self.D, *want)
        assert not np.isnan(got).any()
        over = np.abs(got - want[0]) - bound
        assert over.max() <= 0, (over.max(), np.unravel_index(over.argmax(), over.shape))
        return got


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("pairs,Hq,Hkv,D,P", [
    ([(1, 1)], 1, 1, 64, 16),
    ([(1, 1)], 8, 1, 128, 128),
    ([(15, 1), (16, 1), (17, 1)], 4, 2, 64, 16),
    ([(127, 1), (128, 1), (129, 1), (255, 2), (256, 3), (257, 4)], 8, 2, 128, 64),
    ([(640, 5), (5, 5), (6, 5), (133, 5), (3, 5)], 32, 8, 128, 64),           # the fourth row group: kv < new
    ([(0, 1), (0, 3), (200, 4), (0, 0), (129, 0)], 4, 4, 64, 32),             # nothing cached, nothing new
    ([(2500, 9)], 8, 8, 128, 128),
    ([(3000, 1)], 16, 1, 64, 32),
    ([(300, 17), (44, 2)], 12, 4, 128, 32),                                   # groups of three
    ([(700, 7)], 7, 1, 64, 64),                                               # groups of seven
    ([(260, 130)], 6, 2, 128, 16),                                            # a prompt piece over tile edges
    ([(129, 129), (64, 64), (1, 1), (200, 33)], 8, 4, 64, 64),
    ([(400, 400)], 4, 1, 128, 128),
])
def test_attend_matches_plain_form(ssd, pairs, Hq, Hkv, D, P, dtype):
    Case(len(pairs) * 100 + Hq + D, pairs, Hq, Hkv, D, P, dtype).check(ssd)


@pytest.mark.parametrize("window", [1, 2, 31, 128, 129, 200, 100000])
def test_window(ssd, window):
    Case(window, [(513, 5), (128, 1), (140, 70), (2, 5), (900, 3)], 8, 2, 128, 16, BF).check(ssd, window=window)
    Case(window, [(385, 129), (1, 1)], 2, 2, 64, 64, FP).check(ssd, window=window)


@pytest.mark.parametrize("B,hi", [(40, 1500), (300, 90), (700, 40)])
def test_many_ragged_sequences(ssd, B, hi):
    rng = np.random.default_rng(B)
    pairs = [(int(rng.integers(0, hi)), int(rng.integers(0, 4))) for _ in range(B)]
    Case(B, pairs, 4, 2, 64, 16, BF).check(ssd)


def test_strided_queries(ssd):
    Case(1, [(300, 5), (77, 3)], 8, 2, 128, 32, BF).check(ssd, pad=1024)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_sharp_softmax(ssd, dtype):
    """Scores of some hundreds: one key takes all."""
    Case(2, [(500, 3), (90, 2)], 4, 2, 64, 32, dtype, spread=60.0).check(ssd)


def test_flat_tail_next_to_a_large_weight(ssd):
    """One key of weight 1/2 and 60000 that share the other half: the small ones must not vanish."""
    n, D = 60001, 64
    k = torch.zeros((469, 1, 128, D), dtype=torch.float32)
    k[0, 0, 0, 0] = 256.0
    v = torch.ones((469, 1, 128, D))
    v[0, 0, 0] = 0.0
    q = torch.zeros((1, 1, D), dtype=BF)
    q[0, 0, 0] = 1.0
    g = lambda a: a.to(torch.float8_e4m3fn).cuda()  # noqa: E731
    one = torch.ones((469, 1), device="cuda")
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    scale = float(np.log(60000.0) / 256.0)
    out = ssd.ssd_kv_attend(q.cuda(), g(k), g(v), one, one, torch.arange(469, dtype=torch.int32, device="cuda")[None], i([0, 1]),
                            i([n]), 1, scale)
    assert float((out.float() - 0.5).abs().max()) <= 0.5 * (2.0 ** -8 + 2.0 ** -9)


def test_scales_of_very_different_size(ssd):
    c = Case(3, [(700, 5)], 4, 2, 64, 16, BF)
    c.vs *= (10.0 ** np.random.default_rng(3).uniform(-6, 3, c.vs.shape)).astype(np.float32)
    c.vs[c.table[0, 3]] = 0.0
    c.check(ssd)


def test_nan_in_later_tokens_stays_with_those_that_see_it(ssd):
    """A NaN among the new tokens reaches the tokens from it on, none before."""
    c = Case(4, [(300, 6)], 4, 2, 64, 32, BF)
    want = c.run(ssd).double().cpu().numpy()
    j = 300 - 6 + 3
    c.v[c.table[0, j // 32], 1, j % 32, 7] = 0x7F      # head 1, channel 7
    c.k[c.table[0, (j + 1) // 32], 0, (j + 1) % 32, 9] = 0xFF  # head 0: every channel of tokens 4 and 5
    got = c.run(ssd).double().cpu().numpy()
    nan = np.zeros(got.shape, bool)
    nan[3:, 2:, 7] = True
    nan[4:, :2] = True
    np.testing.assert_array_equal(np.isnan(got), nan)
    np.testing.assert_allclose(got[~nan], want[~nan], rtol=2.0 ** -7, atol=1e-6)


def test_pages_outside_the_cache_count_as_not_there(ssd):
    c = Case(5, [(200, 3), (90, 2)], 4, 2, 64, 16, BF)
    c.table[0, 2], c.table[0, 12], c.table[1, 0] = -1, 10 ** 6, len(c.k)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(ssd, dev_status=status)
    assert int(status) == ssd.SSD_DEV_BAD_PAGE


def test_lengths_beyond_the_table_and_the_bound(ssd):
    """kv_len beyond max_blocks pages is cut there; tokens beyond max_new and behind cu_new[B] get zeros."""
    c = Case(6, [(64, 4), (50, 9)], 2, 2, 64, 16, BF)
    c.kv[0] = 70
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = c.check(ssd, max_new=5, dev_status=status)
    assert int(status) & ssd.SSD_DEV_BAD_LENGTH and not got[9:].any()
    c = Case(7, [(64, 4)], 2, 2, 64, 16, BF)
    c.q = torch.cat([c.q, c.q])
    got = c.run(ssd).cpu()
    assert got[:4].abs().sum() > 0 and not got[4:].any()


def test_cache_beyond_32_bits_of_bytes(ssd):
    N, H, P, D = 70000, 8, 128, 64          # 4.6 GB each
    gen = torch.Generator(device="cuda").manual_seed(1)
    small = Case(8, [(300, 2)], 8, 8, 64, 128, BF)
    k = torch.full((N, H, P, D), 0x7F, dtype=torch.uint8, device="cuda")
    v = k.clone()
    s = [torch.full((N, H), float("nan"), device="cuda") for _ in range(2)]
    at = [N - 1, 3, N // 2 + 1]
    for dst, src in zip(at, small.table[0]):
        k[dst], v[dst] = torch.from_numpy(small.k[src]).cuda(), torch.from_numpy(small.v[src]).cuda()
        s[0][dst], s[1][dst] = torch.from_numpy(small.ks[src]).cuda(), torch.from_numpy(small.vs[src]).cuda()
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    got = ssd.ssd_kv_attend(small.q.cuda(), k, v, s[0], s[1], i([at]), i([0, 2]), i([300]), 2, small.scale)
    assert torch.equal(got, small.run(ssd))
    del gen


def test_same_bits_every_time_with_one_workspace(ssd):
    c = Case(9, [(5000, 5), (17, 2), (3001, 5)], 8, 2, 128, 64, BF)
    ws = ssd.kv_workspace()
    first = c.run(ssd, workspace=ws)
    for _ in range(5):
        assert torch.equal(c.run(ssd, workspace=ws), first)
    small = Case(10, [(9, 1)], 8, 2, 128, 64, BF)
    assert torch.equal(small.run(ssd, workspace=ws), small.run(ssd))


def test_in_a_graph_and_on_another_stream(ssd):
    c = Case(11, [(1500, 5), (800, 5)], 8, 2, 128, 64, BF)
    want = c.run(ssd)
    g = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    q, k, v, ks, vs, table, cu, kv = c.q.cuda(), g(c.k), g(c.v), g(c.ks), g(c.vs), g(c.table), g(c.cu), g(c.kv)
    ws, out = ssd.kv_workspace(), torch.zeros_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = ssd.ssd_kv_attend(q, k, v, ks, vs, table, cu, kv, 5, c.scale, stream=s)
    s.synchronize()
    assert torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssd.ssd_kv_attend(q, k, v, ks, vs, table, cu, kv, 5, c.scale, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    kv[0] = 700  # the lengths are read on the device: a replay follows them
    graph.replay()
    c.kv[0] = 700
    torch.cuda.synchronize()
    assert torch.equal(out, c.run(ssd))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("window,page", [(0, 18), (10, 17)])
def test_a_value_scale_that_is_not_finite_stays_with_those_that_see_it(ssd, dtype, bad, window, page):
    """Of tokens at 285 to 290 the last three see the page of positions 288 on; of those at 294 to 299, with a window of 10,
    the first three that of 272 to 287."""
    pairs = [(291, 6)] if window == 0 else [(300, 6)]
    c = Case(12, pairs, 4, 2, 64, 16, dtype)
    c.vs[c.table[0, page], 1] = bad
    got = c.run(ssd, window=window).double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        want = ref.attend(c.q.double().numpy(), VALUES[c.k], VALUES[c.v], c.ks.astype(np.float64), c.vs.astype(np.float64),
                          c.table, c.cu, c.kv, c.P, c.scale, window)
        bound = ref.attend_bound(dtype, c.D, *want)
    sees = ~np.isfinite(want[0])
    assert sees[:, 2:].any() and not sees[:, 2:].all() and not sees[:, :2].any()
    np.testing.assert_array_equal(~np.isfinite(got), sees)
    assert (np.abs(got - want[0])[~sees] <= bound[~sees]).all()


@pytest.mark.parametrize("dtype,scale,spread", [(BF, 0.0, 1.0), (FP, 0.0, 1.0), (BF, -0.0, 1.0), (BF, 1e-30, 1e-30), (BF, -1e-44, 1.0),
                                                (FP, 1e-38, 1.0), (FP, 3e-41, 1e-3)])
def test_scale_of_zero_and_scales_that_vanish(ssd, dtype, scale, spread):
    """Scores of 0, or too small to matter: the mean of the values that a token attends to."""
    c = Case(13, [(300, 6), (17, 17), (700, 1), (3, 5)], 4, 2, 64, 16, dtype, spread=spread)
    c.scale = scale
    c.check(ssd)
    c.check(ssd, window=37)


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


def test_the_length_of_a_sequence_without_tokens_does_not_matter(ssd):
    c = Case(6, [(64, 4), (50, 0)], 2, 2, 64, 16, BF)
    c.kv[1] = -7
    assert _status(ssd, c) == 0


def test_more_tokens_than_the_bound_are_reported(ssd):
    assert _status(ssd, Case(6, [(64, 4), (50, 9)], 2, 2, 64, 16, BF), max_new=5) == ssd.SSD_DEV_BAD_LENGTH


def test_token_counts_that_pass_the_queries_are_reported(ssd):
    """cu_new beyond the T tokens of q is cut there."""
    c = Case(6, [(64, 4), (50, 3)], 2, 2, 64, 16, BF)
    want = c.run(ssd)
    c.cu[2] = 9
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.kv[1] = 52          # of five tokens; three are there, and attend from the end all the same
    got = c.run(ssd, max_new=5, dev_status=status)
    assert int(status) == ssd.SSD_DEV_BAD_LENGTH
    assert torch.equal(got[:4], want[:4])


@pytest.mark.parametrize("entry", [-1, -2, -3, -2 ** 31, 2 ** 31 - 1])
def test_every_entry_outside_the_cache_is_reported(ssd, entry):
    c = Case(5, [(200, 3)], 4, 2, 64, 16, BF)
    c.table[0, 2] = entry
    assert _status(ssd, c) == ssd.SSD_DEV_BAD_PAGE
    # behind the end of the sequence it is nobody's
    c = Case(5, [(200, 3), (300, 3)], 4, 2, 64, 16, BF)
    c.table[0, 13:] = entry
    assert _status(ssd, c) == 0


def test_token_counts_that_fall_are_reported_and_bounded(ssd):
    """cu_new going back and forth would make 13 row blocks for each of 20 sequences, of tokens that make 13 in all."""
    ws = ssd.kv_workspace()
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


@pytest.mark.parametrize("dtype", [BF, FP])
def test_nan_in_some_of_many_items(ssd, dtype):
    """Several items to a CTA, some with NaN that only the later tokens see: it stays in its own item."""
    rng = np.random.default_rng(16)
    c = Case(16, [(int(rng.integers(5, 600)), 4) for _ in range(330)], 4, 2, 64, 16, dtype)
    for b in rng.choice(330, 40, replace=False):
        j = int(c.kv[b]) - int(rng.integers(1, 4))
        c.v[c.table[b, j // 16], rng.integers(2), j % 16, rng.integers(64)] = 0xFF
    got = c.run(ssd).double().cpu().numpy()
    want = ref.attend(c.q.double().numpy(), VALUES[c.k], VALUES[c.v], c.ks.astype(np.float64), c.vs.astype(np.float64), c.table,
                      c.cu, c.kv, c.P, c.scale, 0)
    nan = np.isnan(want[0])
    assert 40 < nan.sum() < 40 * 2 * 3 + 1
    np.testing.assert_array_equal(np.isnan(got), nan)
    want[3][:] = np.nanmax(np.abs(VALUES[c.v]) * c.vs[:, :, None, None])   # the largest |v| of a row is NaN with it
    bound = ref.attend_bound(dtype, c.D, *want)
    assert (np.abs(got - want[0])[~nan] <= bound[~nan]).all()


@pytest.mark.parametrize("times", [30.0, 1000.0])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_queries_with_one_large_channel(ssd, dtype, times):
    """Digits end at 2^-17 of a row's largest channel: what that can move a score by, 2^-17 |scale| max |q| sum |k|, moves a
    weight by as much and their total once more, next to the bound of the other roundings."""
    c = Case(17, [(700, 5), (40, 40)], 8, 2, 128, 32, dtype)
    c.q[:, :, 5] *= times
    c.k[..., 5] = 1                        # 2^-9: the scores are those of the small channels
    got = c.run(ssd).double().cpu().numpy()
    want = ref.attend(c.q.double().numpy(), VALUES[c.k], VALUES[c.v], c.ks.astype(np.float64), c.vs.astype(np.float64), c.table,
                      c.cu, c.kv, c.P, c.scale, 0)
    held = np.unique(c.table[c.table >= 0])
    k = np.nansum(np.abs(VALUES[c.k[held]]) * c.ks[held][:, :, None, None], axis=3).max()
    moved = 2.0 ** -17 * c.scale * np.abs(c.q.double().numpy()).max(axis=2, keepdims=True) * k
    bound = ref.attend_bound(dtype, c.D, *want) + 2 * moved * want[1]
    assert (np.abs(got - want[0]) <= bound).all()


@pytest.mark.parametrize("rest", [[40], [40, 60], [40, 60, 0, 90, 300], [0] * 300, [40, 90] * 200])
@pytest.mark.parametrize("n", [13, 150])
def test_a_batch_ends_where_its_token_counts_fall(ssd, n, rest):
    """Sequences before the fall are what they are without the rest, and no other token has an owner."""
    c = Case(41, [(400 + n, n)] + [(90, 0)] * len(rest), 8, 2, 64, 16, BF)
    c.q = torch.cat([c.q, c.q])
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


def seen_parts(c, window=0):
    """ref.attend's arrays, and the largest value that a token attends to times its weight: 448 times the largest of those products
    with the scale alone."""
    ks, vs = c.ks.astype(np.float64), c.vs.astype(np.float64)
    want = ref.attend(c.q.double().numpy(), VALUES[c.k], VALUES[c.v], ks, vs, c.table, c.cu, c.kv, c.P, c.scale, window)
    T, Hq, _ = c.q.shape
    G, most = Hq // c.k.shape[1], np.zeros((T, Hq, 1))
    for b in range(len(c.kv)):
        n = c.cu[b + 1] - c.cu[b]
        for i in range(n):
            last = c.kv[b] - n + i
            js = np.arange(max(0, last + 1 - window) if window else 0, last + 1)
            pages, rows = c.table[b][js // c.P], js % c.P
            for h in range(Hq):
                s = c.scale * ((VALUES[c.k[pages, h // G, rows]] * ks[pages, h // G][:, None]) @ c.q[c.cu[b] + i, h].double().numpy())
                p = np.exp(s - s.max())
                most[c.cu[b] + i, h] = 448 * np.max(p / p.sum() * np.abs(vs[pages, h // G]))
    return want, most


def check_seen(c, got, window=0, rows=slice(None)):
    """As ref.attend_bound, with what the digits' end is relative to taken from the token's own keys: digits end at 2^-18 or 2^-23 of the
    largest weight times value scale of a step, whose scales are within 2^4 of each other, or at 2^-14 and 2^-19 of the largest
    that the token gives in that step, once for each of its keys."""
    (out, weight, score, largest), most = seen_parts(c, window)
    half = torch.finfo(c.dtype).eps / 2
    end = 2.0 ** -14 if c.dtype is BF else 2.0 ** -19
    keys = 256 * -(-c.kv.max() // 256)
    bound = ref.attend_bound(c.dtype, c.D, out, weight, score, 0 * largest) + (1 + half) * end * keys * most
    held = np.abs(out) + bound <= torch.finfo(c.dtype).max          # (beyond that the type has an infinity)
    with np.errstate(invalid="ignore"):
        over = np.where(held, np.abs(got.double().cpu().numpy() - out) - bound, -1.0)[rows]
    assert over.max() <= 0, (over.max(), np.unravel_index(over.argmax(), over.shape))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("times", [12, 30, 60, 100])
@pytest.mark.parametrize("n,window", [(40, 0), (40, 9), (5, 0)])
def test_a_large_value_scale_concerns_those_alone_that_see_it(ssd, dtype, times, n, window):
    """The last tokens' page is of far larger scale, and the others do not attend to it: what those get does not depend on it."""
    c = Case(51, [(290, n), (300, 3)], 4, 2, 64, 16, dtype)         # (288 on is page 18)
    want = c.run(ssd, window=window)
    c.vs[c.table[0, 18]] *= np.float32(2.0 ** times)
    got = c.run(ssd, window=window)
    others = slice(0, n - 2)
    check_seen(c, got, window, others if dtype == FP else slice(None))
    off = (got[others].double() - want[others].double()).abs()
    # both are within the weights' digits of the same values, and half a step of the type
    assert bool((off <= 2 * 2.0 ** -8 * want[others].double().abs().amax(dim=2, keepdim=True)).all())
    assert torch.equal(got[n:], want[n:])


@pytest.mark.parametrize("times", [12, 30, 60])
@pytest.mark.parametrize("page", [0, 5, 17])
def test_the_largest_score_next_to_the_largest_value_scale(ssd, times, page):
    """A page of far larger value scale, whose keys all score 2^-(times + 20) of the others: the others' weights keep their bits."""
    for dtype in (BF, FP):
        c = Case(52, [(300, 20), (77, 7)], 4, 2, 64, 16, dtype)
        p = c.table[0, page]
        c.q[:, :, 5] = 4.0
        c.k[..., 5] = 0
        c.k[p, ..., 5] = 0xFE                                    # -448
        c.ks[p] = 0.02
        c.scale = (times + 20) * float(np.log(2.0)) / (4 * 448 * 0.02)
        c.vs[p] = 0.02 * 2.0 ** times
        check_seen(c, c.run(ssd))


@pytest.mark.parametrize("P", [16, 64, 128])
def test_value_scales_of_all_sizes(ssd, P):
    """From 2^-100 to 2^100 in one step, none and negative ones among them, in items of several row blocks and of one token."""
    for n in (1, 40):
        c = Case(53, [(1000, n), (200, 9)], 8, 2, 64, P, BF, spread=4.0)
        c.vs *= (2.0 ** np.random.default_rng(P).uniform(-100, 100, c.vs.shape)).astype(np.float32)
        c.vs[c.table[0, 1]] = 0.0
        c.vs[c.table[0, 2]] *= -1
        for window in (0, 130):
            check_seen(c, c.run(ssd, window=window), window)
