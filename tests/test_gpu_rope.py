"""ssd_qk_rope against the formula in 64 bits."""
import numpy as np
import pytest

import _tree_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_ssd_gb300 as m
    return m


class Case:
    def __init__(self, seed, T, Hq, Hkv, D, rot, dtype, norm=True, interleaved=False, far=10000, pad=0):
        rng = np.random.default_rng(seed)
        x = rng.standard_normal((T, Hq + 2 * Hkv, D)) * np.exp(rng.standard_normal((1, Hq + 2 * Hkv, 1)))
        full = torch.zeros((T, (Hq + 2 * Hkv) * D + pad), dtype=dtype)
        full[:, :(Hq + 2 * Hkv) * D] = torch.from_numpy(x.reshape(T, -1)).to(dtype)
        x = full.cuda()[:, :(Hq + 2 * Hkv) * D].unflatten(1, (Hq + 2 * Hkv, D))
        self.q, self.k = x[:, :Hq], x[:, Hq:Hq + Hkv]
        self.w = [torch.from_numpy(1 + 0.3 * rng.standard_normal(D)).float().cuda() for _ in range(2)] if norm else [None, None]
        self.positions = torch.from_numpy(rng.integers(0, far, T).astype(np.int32)).cuda()
        self.inv_freq = 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
        self.interleaved, self.eps, self.far, self.dtype = interleaved, 1e-5, far, dtype

    def args(self, ssd, **kw):
        return dict(q_weight=self.w[0], k_weight=self.w[1], eps=self.eps, interleaved=self.interleaved, **kw)

    def want(self):
        out = []
        for x, w in zip((self.q, self.k), self.w):
            out.append(ref.rope(x.double().cpu().numpy(), None if w is None else w.double().cpu().numpy(), self.eps,
                                self.positions.cpu().numpy(), self.inv_freq, self.interleaved))
        return out

    def near(self, got, want):
        for g, (y, size) in zip(got, want):
            over = np.abs(g.double().cpu().numpy() - y) - ref.rope_bound(self.dtype, y, size, self.far)
            assert over.max() <= 0, (over.max(), np.unravel_index(over.argmax(), over.shape))

    def check(self, ssd):
        want = self.want()
        got = ssd.ssd_qk_rope(self.q, self.k, self.positions, ssd.rope_turns(self.inv_freq.tolist()), **self.args(ssd))
        assert got[0].shape == self.q.shape and got[1].shape == self.k.shape and got[0].is_contiguous() and got[0].dtype == self.dtype
        self.near(got, want)
        return got


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot", [
    (1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (3, 7, 1, 128, 128), (33, 5, 5, 64, 32), (130, 16, 4, 64, 16), (17, 3, 2, 128, 48),
    (5, 4, 4, 128, 0), (1000, 8, 2, 64, 64)])
def test_matches_the_formula(ssd, dtype, T, Hq, Hkv, D, rot):
    for norm in (True, False):
        for interleaved in (False, True):
            Case(T + rot, T, Hq, Hkv, D, rot, dtype, norm, interleaved).check(ssd)


@pytest.mark.parametrize("far", [1 << 20, 1 << 30])
def test_far_positions(ssd, far):
    """Whole turns drop out exactly: fp32 results hold at positions where an fp32 angle has none of its digits left."""
    Case(1, 300, 4, 2, 128, 128, F32, far=far).check(ssd)


def test_negative_positions_turn_back(ssd):
    c = Case(2, 50, 4, 2, 64, 64, F32, norm=False)
    c.positions.neg_()
    c.check(ssd)


@pytest.mark.parametrize("dtype,pad", [(BF, 8), (BF, 3), (FP, 1), (F32, 4), (F32, 1)])
def test_strides(ssd, dtype, pad):
    """Tokens further apart than their heads, on and off the 16-byte grid."""
    Case(3, 40, 6, 2, 128, 128, dtype, pad=pad).check(ssd)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place_and_into_views(ssd, dtype):
    c = Case(4, 70, 8, 2, 128, 64, dtype)
    want = c.check(ssd)
    turns = ssd.rope_turns(c.inv_freq.tolist())
    room = torch.full((70, 11, 128), 7.0, dtype=dtype, device="cuda")
    ssd.ssd_qk_rope(c.q, c.k, c.positions, turns, q_out=room[:, 1:9], k_out=room[:, 9:], **c.args(ssd))
    assert torch.equal(room[:, 1:9], want[0]) and torch.equal(room[:, 9:], want[1]) and bool((room[:, 0] == 7).all())
    ssd.ssd_qk_rope(c.q, c.k, c.positions, turns, q_out=c.q, k_out=c.k, **c.args(ssd))
    assert torch.equal(c.q, want[0]) and torch.equal(c.k, want[1])


def test_large_and_odd_values(ssd):
    """A NaN or an infinity stays in its own head; zeros give zeros; large fp32 values do not overflow the norm."""
    c = Case(5, 6, 4, 2, 64, 64, BF)
    c.q[1, 2, 5], c.q[2, 0, 3], c.q[3, 1] = float("nan"), float("inf"), 0.0
    q, k = ssd.ssd_qk_rope(c.q, c.k, c.positions, ssd.rope_turns(c.inv_freq.tolist()), **c.args(ssd))
    bad = torch.zeros(q.shape, dtype=torch.bool, device="cuda")
    bad[1, 2], bad[2, 0] = True, True
    assert torch.equal(torch.isnan(q).any(dim=2), bad.any(dim=2)) and not torch.isnan(k).any()
    assert not q[3, 1].any()


def test_channels_that_are_not_turned_keep_their_bits(ssd):
    c = Case(6, 20, 4, 2, 128, 32, BF, norm=False)
    c.q[3, 1, 40] = float("inf")
    q, _ = ssd.ssd_qk_rope(c.q, c.k, c.positions, ssd.rope_turns(c.inv_freq.tolist()))
    assert torch.equal(q[..., 32:], c.q[..., 32:])


def test_no_tokens(ssd):
    q, k = torch.zeros((0, 4, 64), dtype=BF, device="cuda"), torch.zeros((0, 2, 64), dtype=BF, device="cuda")
    out = ssd.ssd_qk_rope(q, k, torch.zeros(0, dtype=torch.int32, device="cuda"), ssd.rope_turns([1.0] * 32))
    assert out[0].shape == (0, 4, 64)


def test_rows_beyond_32_bits_of_elements(ssd):
    """Tokens 2^28 elements apart: the last one's offset passes 2^32 bytes, and 2^31 elements."""
    room = torch.zeros(9 * 2 ** 28 + 1024, dtype=BF, device="cuda")
    q = room.as_strided((10, 4, 64), (2 ** 28, 64, 1))
    c = Case(7, 10, 4, 2, 64, 64, BF)
    q.copy_(c.q)
    turns = ssd.rope_turns(c.inv_freq.tolist())
    got = ssd.ssd_qk_rope(q, c.k, c.positions, turns, q_out=q, **c.args(ssd))
    assert torch.equal(got[0], ssd.ssd_qk_rope(c.q, c.k, c.positions, turns, **c.args(ssd))[0])


def test_in_a_graph_and_on_another_stream(ssd):
    c = Case(8, 100, 8, 2, 128, 128, BF)
    turns = ssd.rope_turns(c.inv_freq.tolist())
    want = ssd.ssd_qk_rope(c.q, c.k, c.positions, turns, **c.args(ssd))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = ssd.ssd_qk_rope(c.q, c.k, c.positions, turns, stream=s, **c.args(ssd))
    s.synchronize()
    assert torch.equal(other[0], want[0]) and torch.equal(other[1], want[1])
    out = [torch.zeros_like(x) for x in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssd.ssd_qk_rope(c.q, c.k, c.positions, turns, q_out=out[0], k_out=out[1], **c.args(ssd))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    c.positions.add_(5)
    graph.replay()
    torch.cuda.synchronize()
    c.near(out, c.want())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,Hkv", [(64, 2), (128, 3)])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-30])
def test_norms_of_heads_of_any_size(ssd, dtype, D, Hkv, eps):
    """Squares that fp32 does not hold, large or small, in a head by itself or next to ordinary ones; one channel far above the
    rest; and eps above, among or below the squares."""
    c = Case(9, 9, 9, Hkv, D, D, dtype)
    c.eps = eps
    for h, size in enumerate((1e25, 1e-25, 1e-12, 1e19, 3e37, 1.0, 1e-38, 1e-21)):
        c.q[:, h] *= size
    c.q[:, 3, 5] = 1e30
    c.k[1::2, 0] *= 1e22
    c.k[2, 1:] *= 1e-30
    assert not torch.isinf(c.q).any() and not torch.isinf(c.k).any()
    got = ssd.ssd_qk_rope(c.q, c.k, c.positions, ssd.rope_turns(c.inv_freq.tolist()), **c.args(ssd))
    # below the normal range, which the bound leaves out: half a step of the output's smallest, and the smallest step of fp32
    # for each of a rotation's three roundings
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2 + 3 * 2.0 ** -149
    for g, (y, size) in zip(got, c.want()):
        over = np.abs(g.double().cpu().numpy() - y) - ref.rope_bound(dtype, y, size, c.far) - tiny
        assert over.max() <= 0, (over.max(), np.unravel_index(over.argmax(), over.shape))


def test_many_heads(ssd):
    """More heads than a warp has marks for those of odd size, with enough tokens that each has a warp: any token's results are those
    that it has by itself, odd heads, in place and not."""
    c = Case(10, 50, 300, 8, 64, 64, BF)
    for h, size in ((0, 1e25), (7, 1e-30), (8, 1e22), (150, 1e25), (299, 1e30)):
        c.q[:, h] *= size
    c.k[:, 7] *= 1e25
    c.eps = 0.0
    turns = ssd.rope_turns(c.inv_freq.tolist())
    want = ssd.ssd_qk_rope(c.q, c.k, c.positions, turns, **c.args(ssd))
    c.near([x[:3] for x in want], [(y[:3], z[:3]) for y, z in c.want()])
    q, k, positions = c.q.repeat(110, 1, 1), c.k.repeat(110, 1, 1), c.positions.repeat(110)
    got = ssd.ssd_qk_rope(q, k, positions, turns, **c.args(ssd))
    for g, w in zip(got, want):
        assert torch.equal(g.view(110, *w.shape), w[None].expand(110, -1, -1, -1))
    ssd.ssd_qk_rope(q, k, positions, turns, q_out=q, k_out=k, **c.args(ssd))
    assert torch.equal(q, got[0]) and torch.equal(k, got[1])
