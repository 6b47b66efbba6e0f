"""ssd_tree_plan, ssd_tree_accept and ssd_kv_compact against plain forms."""
import numpy as np
import pytest

import _loop_ref as loop
import _tree_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
VALUES = loop.e4m3_values()
CODE = {v: c for c, v in reversed(list(enumerate(VALUES))) if v == v}


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_ssd_gb300 as m
    return m


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).cuda()


def trees(seed, counts, kinds=("random", "chain", "star", "flat")):
    rng = np.random.default_rng(seed)
    parent = sum([ref.parents(kinds[b % len(kinds)], n, rng) for b, n in enumerate(counts)], [])
    return [0] + np.cumsum(counts).tolist(), parent, rng


# ---- plan ---------------------------------------------------------------------------------

def check_plan(ssd, cu, parent, seq_len, max_new, extra=0):
    T = len(parent) + extra
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    W = -(-max_new // 32)
    out = {"positions": torch.full((T,), 77, dtype=torch.int32, device="cuda"), "mask": torch.full((T, W), 77, dtype=torch.int32, device="cuda")}
    got = ssd.ssd_tree_plan(dev(parent + [9] * extra), dev(cu), dev(seq_len), max_new, out=out, dev_status=status)
    positions, sees, want = ref.tree_plan(parent, cu, seq_len, T, max_new)
    assert got["positions"].tolist() == positions
    np.testing.assert_array_equal(got["mask"].cpu().numpy(), ref.words(sees, W))
    assert int(status) == want
    return want


@pytest.mark.parametrize("counts", [[1], [0, 1, 0], [37] * 9, [31, 32, 33, 63, 64, 65, 1, 127], [509, 3, 400, 129], [1024, 1000, 1023, 1024]])
def test_plan(ssd, counts):
    cu, parent, rng = trees(len(counts), counts)
    assert check_plan(ssd, cu, parent, rng.integers(0, 9000, len(counts)).tolist(), max(counts), extra=3) == 0


def test_plan_of_many_sequences(ssd):
    rng = np.random.default_rng(5)
    counts = rng.integers(0, 9, 4096).tolist()
    cu, parent, _ = trees(6, counts)
    check_plan(ssd, cu, parent, rng.integers(0, 2 ** 20, 4096).tolist(), 8)


@pytest.mark.parametrize("bad", [-2, 5, 6, 100, 2 ** 31 - 1, -2 ** 31])
def test_plan_counts_a_parent_that_is_not_before_its_node_as_none(ssd, bad):
    cu, parent, _ = trees(7, [10, 10])
    parent[5] = bad
    assert check_plan(ssd, cu, parent, [3, 4], 10) == ssd.SSD_DEV_BAD_TREE


def test_plan_reports_lengths(ssd):
    cu, parent, _ = trees(8, [10, 7])
    assert check_plan(ssd, cu, parent, [3, 4], 8) == ssd.SSD_DEV_BAD_LENGTH
    for cu, seq in (([0, 12, 40], [3, 4]), ([-3, 5, 17], [3, 4]), ([0, 9, 5], [3, 4]), ([0, 10, 17], [-1, 4]), ([0, 10, 17], [2 ** 31 - 5, 4])):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ssd.ssd_tree_plan(dev(parent), dev(cu), dev(seq), 64, dev_status=status)
        assert int(status) & ssd.SSD_DEV_BAD_LENGTH, cu


@pytest.mark.parametrize("rest", [[4], [4, 12], [4, 12, 0, 20, 90], [0] * 300, [7, 60] * 200])
@pytest.mark.parametrize("n", [9, 140])
def test_plan_of_a_batch_ends_where_its_token_counts_fall(ssd, n, rest):
    """Sequences before the fall are what they are without the rest, and no other token has an owner."""
    cu, parent, _ = trees(13, [n, 60])
    seq = [5] + [1000] * len(rest)
    want = ref.tree_plan(parent[:n], [0, n], [5], n + 60, n)
    for _ in range(10):
        out = {"positions": torch.full((n + 60,), 77, dtype=torch.int32, device="cuda"),
               "mask": torch.full((n + 60, -(-n // 32)), 77, dtype=torch.int32, device="cuda")}
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ssd.ssd_tree_plan(dev(parent), dev([0, n] + rest), dev(seq), n, out=out, dev_status=status)
        assert out["positions"].tolist() == want[0]
        np.testing.assert_array_equal(out["mask"].cpu().numpy(), ref.words(want[1], -(-n // 32)))
        assert int(status) & ssd.SSD_DEV_BAD_LENGTH


# ---- accept -------------------------------------------------------------------------------

def check_accept(ssd, cu, parent, tokens, sampled, max_new, max_path):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ssd.ssd_tree_accept(dev(parent), dev(tokens), dev(sampled), dev(cu), max_new, max_path, dev_status=status)
    accept, bonus, path, want = ref.tree_accept(parent, tokens, sampled, cu, max_new, max_path)
    assert got["accept_len"].tolist() == accept and got["bonus"].tolist() == bonus and got["path"].tolist() == path
    assert int(status) == want
    return accept, want


@pytest.mark.parametrize("max_path", [1, 2, 5, 33])
@pytest.mark.parametrize("counts", [[1], [0, 1, 0, 2], [37] * 12, [509, 3, 400, 129, 1024]])
def test_accept(ssd, counts, max_path):
    """Few different tokens: siblings that share one, and long paths."""
    cu, parent, rng = trees(9, counts, ("random", "chain", "random", "star"))
    T = len(parent)
    accept, status = check_accept(ssd, cu, parent, rng.integers(0, 2, T).tolist(), rng.integers(0, 2, T).tolist(), max(counts), max_path)
    assert status == 0 and (max_path == 1 or max(counts) < 30 or max(accept) > 0)


def test_accept_with_draws_that_are_not_tokens(ssd):
    """A draw of -1 (a row that the sampler refused) makes its sequence invalid where the path meets it, not elsewhere."""
    cu, parent, rng = trees(10, [20] * 40, ("random",))
    T = len(parent)
    tokens, sampled = rng.integers(0, 2, T).tolist(), rng.integers(0, 2, T).tolist()
    for t in rng.choice(T, 100, replace=False):
        sampled[t] = -1
    accept, status = check_accept(ssd, cu, parent, tokens, sampled, 20, 9)
    assert status == ssd.SSD_DEV_BAD_TOKEN and 0 < accept.count(-1) < 40


def test_accept_with_bad_parents_and_too_many_nodes(ssd):
    cu, parent, rng = trees(11, [20] * 6, ("random",))
    T = len(parent)
    for i, bad in ((3, 3), (25, 17), (45, -2), (60, 0), (85, 2 ** 31 - 1)):
        parent[i] = bad
    tokens, sampled = [1] * T, [1] * T
    assert check_accept(ssd, cu, parent, tokens, sampled, 20, 9)[1] == ssd.SSD_DEV_BAD_TREE
    assert check_accept(ssd, cu, parent, tokens, sampled, 15, 9)[1] == ssd.SSD_DEV_BAD_TREE | ssd.SSD_DEV_BAD_LENGTH


def test_accept_of_no_tokens(ssd):
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    got = ssd.ssd_tree_accept(e, e, e, dev([0, 0, 0]), 4, 3)
    assert got["accept_len"].tolist() == [-1, -1] and got["bonus"].tolist() == [-1, -1] and got["path"].tolist() == [[-1] * 3] * 2


# ---- compact ------------------------------------------------------------------------------

class Cache:
    """Pages for B sequences of up to `rows` positions, with scales that differ by powers of two."""

    def __init__(self, seed, B, rows, H, D, P, spread=3, odd=False):
        rng = self.rng = np.random.default_rng(seed)
        self.P, blocks = P, -(-rows // P)
        N = B * blocks + 2
        self.table = rng.permutation(N)[:B * blocks].reshape(B, blocks).astype(np.int32)
        self.codes, self.scales = [], []
        for _ in range(2):
            codes = rng.integers(0, 256, (N, H, P, D)).astype(np.uint8)
            codes[(codes & 127) == 127] = 0x30
            self.codes.append(codes)
            s = 2.0 ** rng.integers(-spread, spread + 1, (N, H))
            self.scales.append((s * (rng.uniform(1, 2, (N, H)) if odd else 1)).astype(np.float32))

    def run(self, ssd, path, accept, keep, check=True):
        g = [torch.from_numpy(c).cuda() for c in self.codes] + [torch.from_numpy(s).cuda() for s in self.scales]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ssd.ssd_kv_compact(dev(path), dev(accept), dev(keep), dev(self.table), *g, dev_status=status)
        got = [x.cpu().numpy() for x in g]
        if check:
            for i in range(2):
                values, scale = VALUES[self.codes[i]], self.scales[i].copy()
                ref.compact(path, accept, keep, self.table, values, scale, self.P)
                np.testing.assert_array_equal(got[2 + i], scale)
                np.testing.assert_array_equal(VALUES[got[i]], values)
        return got, int(status)


def paths(rng, accept, n, J):
    """Ascending paths from 0: any nodes, places and sources mixed."""
    out = np.full((len(accept), J), -1)
    for b, a in enumerate(accept):
        if a >= 0:
            out[b, 0] = 0
            out[b, 1:a + 1] = np.sort(rng.permutation(np.arange(1, n))[:a])
    return out


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("H,D,P", [(1, 64, 16), (2, 128, 16), (3, 64, 32), (2, 128, 64), (1, 64, 128), (4, 128, 128)])
@pytest.mark.parametrize("J,n", [(2, 2), (5, 6), (9, 40), (33, 33), (33, 34), (33, 200)])
def test_compact(ssd, H, D, P, J, n, odd):
    B = 14
    c = Cache(J * n + P, B, max(75, P) + n, H, D, P, odd=odd)
    keep = c.rng.integers(0, 75, B)
    keep[:3] = 0, P - 1, 16
    accept = c.rng.integers(-1, J, B)
    accept[:4] = J - 1, J - 1, 0, -1
    assert c.run(ssd, paths(c.rng, accept, n, J), accept, keep)[1] == 0


def test_compact_keeps_what_stays(ssd):
    """A chain accepted in place moves nothing; with equal scales bytes are moved as they are."""
    c = Cache(1, 4, 100, 2, 64, 32)
    accept = np.array([8, 3, 0, -1])
    got, _ = c.run(ssd, np.where(np.arange(9)[None] <= accept[:, None], np.arange(9)[None], -1), accept, np.array([3, 31, 60, 9]))
    for i in range(2):
        np.testing.assert_array_equal(got[i], c.codes[i])
        np.testing.assert_array_equal(got[2 + i], c.scales[i])


def test_compact_with_odd_values(ssd):
    """NaN among the tokens, scales that are no positive finite number, and pages of zeros."""
    c = Cache(2, 12, 100, 2, 64, 16)
    c.codes[0][c.rng.random(c.codes[0].shape) < 0.02] = 0x7F
    c.codes[1][c.table[3, 1:]] = 0
    for p, s in ((c.table[1, 1], 0.0), (c.table[2, 2], np.inf), (c.table[4, 1], np.nan), (c.table[5, 1], -2.0), (c.table[6, 0], 0.0),
                 (c.table[7, 1], np.nan), (c.table[8, 0], 1e-38), (c.table[8, 1], 3e38)):
        c.scales[0][p, 0] = s
        c.scales[1][p, 1] = s
    accept = np.full(12, 6)
    with np.errstate(invalid="ignore", over="ignore"):
        c.run(ssd, paths(c.rng, accept, 60, 9), accept, c.rng.integers(0, 30, 12))


@pytest.mark.parametrize("k", [100, 119, 120, 121, 123])
def test_compact_of_values_next_to_the_largest(ssd, k):
    """A byte times its page's scale may pass fp32: 3.3e38 in bf16 is stored as 256 * 2^120.  The scale
    grows to hold the largest all the same, and powers of two leave the values exact."""
    c = Cache(6, 3, 100, 2, 64, 16)
    c.codes[0][:] = CODE[1.0]
    c.scales[0][:], c.scales[1][:] = 1.0, 1.0
    path, accept, keep = np.array([[0, 20, 37, 40]] * 3), np.full(3, 3), np.array([2, 3, 9])
    byte = {100: 448.0, 119: 448.0, 120: 256.0, 121: 240.0, 123: 416.0}[k]
    for b in range(3):
        pages = c.table[b][[(int(keep[b]) + n) // 16 for n in (20, 37, 40)]]
        c.scales[0][pages] = 2.0 ** k
        for n, page in zip((20, 37, 40), pages):
            c.codes[0][page, :, (keep[b] + n) % 16, 5] = CODE[byte]
    got, status = c.run(ssd, path, accept, keep, check=False)
    assert status == 0
    need = 2.0 ** int(np.ceil(np.log2(byte / 448) + k))
    for b in range(3):
        page, at = c.table[b][int(keep[b]) // 16], (int(keep[b]) + np.arange(4)) % 16
        assert (got[2][page] == need).all()
        want = np.full((2, 3, 64), 2.0 ** k)
        want[:, :, 5] = byte * 2.0 ** k
        np.testing.assert_array_equal(VALUES[got[0][page][:, at[1:]]] * need, np.where(want / need < 2.0 ** -9, 0, want))
        # rows that were there, of ones, are nothing under the new scale
        assert not VALUES[got[0][page][:, :at[0] + 1]].any()


def test_compact_leaves_a_sequence_that_it_cannot_move(ssd):
    path = np.array([[0, 2, 3, 7], [0, 1, 5, 6]])

    def left(status, *, first=None, accept=3, keep=5, table=None, p=None):
        c = Cache(3, 2, 60, 2, 64, 16)
        q = path.copy()
        if p is not None:
            q[0] = p
        if table is not None:
            c.table[0, table[0]] = table[1]
        got, said = c.run(ssd, q, np.array([accept, 3]), np.array([keep, 7]), check=False)
        assert said == status, (said, status)
        good = Cache(3, 2, 60, 2, 64, 16)
        want, _ = good.run(ssd, q, np.array([-1, 3]), np.array([0, 7]))
        for a, b in zip(got, want):
            np.testing.assert_array_equal(a, b)

    tree, length, page = ssd.SSD_DEV_BAD_TREE, ssd.SSD_DEV_BAD_LENGTH, ssd.SSD_DEV_BAD_PAGE
    left(tree, p=[1, 2, 3, 7])
    left(tree, p=[0, 2, 2, 7])
    left(tree, p=[0, 2, -1, -1])
    left(tree, p=[0, 3, 2, 7])
    left(tree, p=[-1, -1, -1, -1])
    left(length, accept=4)
    left(length, accept=2 ** 31 - 1)
    left(length, keep=-1)
    left(length, keep=57)
    left(length, keep=2 ** 31 - 1)
    left(length, p=[0, 2, 3, 2 ** 31 - 1])
    left(page, table=(0, -1))
    left(page, table=(0, 10 ** 6))


def test_compact_beyond_32_bits_of_bytes(ssd):
    N, H, P, D = 70000, 8, 128, 64          # 4.6 GB each
    small = Cache(4, 1, 250, 8, 64, 128)
    k = torch.zeros((N, H, P, D), dtype=torch.uint8, device="cuda")
    v, s = k.clone(), [torch.ones((N, H), device="cuda") for _ in range(2)]
    at = [N - 1, N // 2 + 1]
    for dst, src in zip(at, small.table[0]):
        k[dst], v[dst] = torch.from_numpy(small.codes[0][src]).cuda(), torch.from_numpy(small.codes[1][src]).cuda()
        s[0][dst], s[1][dst] = torch.from_numpy(small.scales[0][src]).cuda(), torch.from_numpy(small.scales[1][src]).cuda()
    path, accept, keep = np.array([[0, 3, 50, 90]]), np.array([3]), np.array([125])
    ssd.ssd_kv_compact(dev(path), dev(accept), dev(keep), dev([at]), k, v, *s)
    want, _ = small.run(ssd, path, accept, keep)
    for dst, src in zip(at, small.table[0]):
        np.testing.assert_array_equal(k[dst].cpu().numpy(), want[0][src])
        np.testing.assert_array_equal(v[dst].cpu().numpy(), want[1][src])
        np.testing.assert_array_equal(s[1][dst].cpu().numpy(), want[3][src])


# ---- streams and graphs -------------------------------------------------------------------

def test_in_graphs_and_on_another_stream(ssd):
    cu, parent, rng = trees(12, [20, 5, 33], ("random",))
    T = len(parent)
    a = [dev(x) for x in (parent, rng.integers(0, 2, T), rng.integers(0, 2, T))]
    seq = dev([3, 40, 17])
    plan, accept = ssd.ssd_tree_plan(a[0], dev(cu), seq, 33), ssd.ssd_tree_accept(*a, dev(cu), 33, 9)
    c = Cache(5, 3, 100, 2, 64, 16)
    cache = [torch.from_numpy(x).cuda() for x in c.codes + c.scales]
    args = (accept["path"], accept["accept_len"], seq, dev(c.table))
    want = [x.clone() for x in cache]
    ssd.ssd_kv_compact(*args, *want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cu_dev, other = dev(cu), [x.clone() for x in cache]
    s.wait_stream(torch.cuda.current_stream())
    p2, a2 = ssd.ssd_tree_plan(a[0], cu_dev, seq, 33, stream=s), ssd.ssd_tree_accept(*a, cu_dev, 33, 9, stream=s)
    ssd.ssd_kv_compact(*args, *other, stream=s)
    s.synchronize()
    room = [x.clone() for x in cache]
    p3 = {k: torch.zeros_like(v) for k, v in plan.items()}
    a3 = {k: torch.zeros_like(v) for k, v in accept.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssd.ssd_tree_plan(a[0], cu_dev, seq, 33, out=p3)
        ssd.ssd_tree_accept(*a, cu_dev, 33, 9, out=a3)
        ssd.ssd_kv_compact(a3["path"], a3["accept_len"], seq, args[3], *room)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in ((plan, p2), (plan, p3), (accept, a2), (accept, a3)):
        assert all(torch.equal(x[k], y[k]) for k in x)
    assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(want, other, room))
