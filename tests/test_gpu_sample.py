"""ssd_sample against a plain form in 64 bits.  The token has to be the same wherever the draw and the
truncations' borders are further than 2^-24 of the total from the next value that would decide otherwise
(weights are exact to 2^-28 of themselves, so sums are to 2^-28 of the total at most; 16 times that)."""
import numpy as np
import pytest

import _loop_ref as ref
import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
MARGIN = 2.0 ** -24


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_ssd_gb300 as m
    return m


def _t(x, dtype=torch.float32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def _check(ssd, z, tau, k, p, mp, u, pad=0, want_filtered=True):
    """z: a host tensor [R, V], fp32 or bf16."""
    R, V = z.shape
    buf = torch.full((R, V + pad), float("nan"), dtype=z.dtype, device="cuda")
    buf[:, :V] = z.cuda()
    u = np.asarray(u, np.float32)
    tau, p, mp = (np.asarray(a, np.float32) for a in (tau, p, mp))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ssd.ssd_sample(buf[:, :V], _t(tau), _t(u), top_k=_t(k, torch.int32), top_p=_t(p), min_p=_t(mp),
                         filtered=want_filtered, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    tokens, prob = out["tokens"].cpu().numpy(), out["prob"].cpu().numpy().astype(np.float64)
    zs = z.double().numpy()
    near = 0
    for r in range(R):
        token, pr, kept, margin = ref.sample(zs[r], float(tau[r]), int(k[r]), float(p[r]), float(mp[r]), float(u[r]))
        if margin < MARGIN:
            near += 1
            continue
        assert tokens[r] == token, (r, tokens[r], token, margin)
        # weight and total are exact to 2^-28, the quotient is rounded to fp32
        assert abs(prob[r] - pr) <= pr * (2.0 ** -24 + 2.0 ** -26), r
        if want_filtered:
            row = np.full(V, float(torch.tensor(ssd.SSD_DROPPED_LOGIT).to(z.dtype)))
            row[kept] = zs[r][kept]
            np.testing.assert_array_equal(out["filtered"][r].double().cpu().numpy(), row)
    assert near <= max(1, R // 50)
    return tokens


def _rows(seed, R, V, dtype, sigma=3.0):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((R, V), dtype=np.float32) * np.float32(sigma) + synth.zipf_log_bias(V, 1.1)
    return torch.from_numpy(z).to(dtype), rng


DT = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("V", [2, 3, 31, 33, 100, 1000, 4099, 32000, 128256, 152064])
def test_every_truncation(ssd, V, dtype):
    R = 40 if V < 10000 else 24
    z, rng = _rows(V, R, V, dtype)
    i = np.arange(R)
    tau = np.array([1.0, 0.7, 0.0, 1.3, 0.25, 5.0])[i % 6]
    k = np.array([0, 1, 50, V, 7, V - 1, 3 * V, -1, 2, 1500])[i % 10]
    p = np.array([1.0, 0.9, 0.99, 0.5, 0.0, 2.0, 0.95])[i % 7]
    mp = np.array([0.0, 0.05, 0.0, 0.001, 1.0, 0.0, 0.0, 1e-9])[(i // 2) % 8]
    _check(ssd, z, tau, k, p, mp, rng.random(R), pad=(0, 1, 8)[V % 3])


@pytest.mark.parametrize("dtype", DT)
def test_plain_temperature_over_a_flat_row(ssd, dtype):
    z, rng = _rows(1, 64, 50021, dtype, sigma=0.3)
    z = (z * 0.01).to(dtype)
    _check(ssd, z, np.full(64, 0.8), np.zeros(64, int), np.ones(64), np.zeros(64), rng.random(64), want_filtered=False)


@pytest.mark.parametrize("dtype", DT)
def test_nucleus_of_tens_of_thousands(ssd, dtype):
    z, rng = _rows(2, 16, 120000, dtype, sigma=0.5)
    z = (z * 0.1).to(dtype)
    _check(ssd, z, np.full(16, 1.0), np.array([0, 30000] * 8), np.array([0.95, 0.6, 0.999, 0.3] * 4), np.zeros(16), rng.random(16))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("V", [5, 64, 3001, 70000])
def test_ties_go_to_the_lowest_id(ssd, V, dtype):
    """All logits equal, and all but a few of two values, with every kind of border inside the ties."""
    rng = np.random.default_rng(V)
    rows = [np.full(V, 1.5), np.where(np.arange(V) % 3 == 0, 2.0, -1.0), np.where(np.arange(V) == V - 1, 4.0, 0.0),
            np.where(np.arange(V) % 2 == 0, 0.0, -0.0)]
    z = torch.tensor(np.array(rows * 6), dtype=torch.float32).to(dtype)
    R = z.shape[0]
    k = np.array([0, 2, V // 2 + 1, V - 1, 0, 3])[np.arange(R) // 4]
    p = np.array([0.371, 1.0, 1.0, 0.613, 1.0, 0.55])[np.arange(R) // 4]
    _check(ssd, z, np.full(R, 0.9), k, p, np.array([0.0] * 20 + [0.5] * 4), rng.random(R))


@pytest.mark.parametrize("dtype", DT)
def test_masked_logits(ssd, dtype):
    """-inf and the type's lowest value have no weight and are never drawn."""
    z, rng = _rows(3, 12, 5000, dtype)
    z[:, ::3] = float("-inf")
    z[:, 1::3] = torch.finfo(dtype).min
    z[5] = float("-inf")
    z[5, 77] = -3.0
    k = np.array([0, 40, 4000, 0, 0, 0] * 2)
    t = _check(ssd, z, np.full(12, 1.0), k, np.array([1.0, 1.0, 0.9] * 4), np.zeros(12), rng.random(12), want_filtered=False)
    assert t[5] == 77 and all(i % 3 == 2 for r, i in enumerate(t) if r != 5)


def test_draws_at_the_ends(ssd):
    z = torch.tensor([[0.0, 0.0, -1e4, 0.0]] * 3)
    got = ssd.ssd_sample(z.cuda(), _t([1.0] * 3), _t([0.0, 0.34, 1 - 2.0 ** -24]))
    assert got["tokens"].tolist() == [0, 1, 3]


def test_parameters_may_be_left_out(ssd):
    z, rng = _rows(4, 8, 999, torch.float32)
    u = rng.random(8).astype(np.float32)
    a = ssd.ssd_sample(z.cuda(), _t(np.ones(8)), _t(u))
    b = ssd.ssd_sample(z.cuda(), _t(np.ones(8)), _t(u), top_k=_t(np.zeros(8), torch.int32), top_p=_t(np.ones(8)),
                       min_p=_t(np.zeros(8)))
    assert torch.equal(a["tokens"], b["tokens"]) and torch.equal(a["prob"], b["prob"]) and "filtered" not in a


def test_bad_rows_are_reported_and_the_others_served(ssd):
    z, rng = _rows(5, 10, 300, torch.float32)
    good = z.clone()
    z[1, 7], z[2, 9] = float("nan"), float("inf")
    z[3] = float("-inf")
    tau = np.array([1, 1, 1, 1, -1.0, np.nan, 1, 1, 1, 1], np.float32)
    p = np.array([1, 1, 1, 1, 1, 1, np.nan, 1, 1, 1], np.float32)
    mp = np.array([0, 0, 0, 0, 0, 0, 0, np.nan, 0, 0], np.float32)
    u = np.array([0.3] * 8 + [1.0, 0.6], np.float32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ssd.ssd_sample(z.cuda(), _t(tau), _t(u), top_p=_t(p), min_p=_t(mp), filtered=True, dev_status=status)
    assert out["tokens"][1:9].tolist() == [-1] * 8 and bool(torch.isnan(out["prob"][1:9]).all())
    assert int(status) == ssd.SSD_DEV_NONFINITE | ssd.SSD_DEV_BAD_TEMPERATURE | ssd.SSD_DEV_BAD_PARAM
    for r in (0, 9):
        assert int(out["tokens"][r]) == ref.sample(good[r].numpy(), 1.0, 0, 1.0, 0.0, float(u[r]))[0]
    np.testing.assert_array_equal(out["filtered"][1:9].cpu().numpy(), z[1:9].numpy())


def test_tiny_and_huge_temperatures(ssd):
    z, rng = _rows(6, 6, 2000, torch.float32)
    _check(ssd, z, np.array([1e-30, 1e-6, 1e-3, 1e3, 1e30, 3e38]), np.zeros(6, int), np.array([1.0, 0.9] * 3), np.zeros(6),
           rng.random(6))


@pytest.mark.parametrize("B,V", [(4, 5000), (48, 32000)])
def test_filtered_rows_verify_as_the_truncated_distributions(ssd, B, V):
    """A round over filtered draft and target rows accepts with p and q of the truncated distributions."""
    import oracle
    K = 3
    rng = np.random.default_rng(7)
    d = rng.standard_normal((B, K, V), dtype=np.float32) * 3
    t = np.concatenate([d, rng.standard_normal((B, 1, V), dtype=np.float32) * 3], axis=1)
    t = t + 0.5 * rng.standard_normal(t.shape, dtype=np.float32)
    ones = lambda n, x, ty=torch.float32: torch.full((n,), x, dtype=ty, device="cuda")  # noqa: E731
    drawn = ssd.ssd_sample(torch.from_numpy(d).cuda().view(B * K, V), ones(B * K, 0.8), torch.rand(B * K, device="cuda"),
                           top_k=ones(B * K, 40, torch.int32), filtered=True)
    tgt = ssd.ssd_sample(torch.from_numpy(t).cuda().view(B * (K + 1), V), ones(B * (K + 1), 0.8), ones(B * (K + 1), 0.5),
                         top_p=ones(B * (K + 1), 0.9), filtered=True)["filtered"].view(B, K + 1, V)
    drf, tok = drawn["filtered"].view(B, K, V), drawn["tokens"].view(B, K)
    u = torch.rand((B, K + 1), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ssd.ssd_verify(tgt, drf, tok, u, ones(B, 0.8), dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    q = drawn["prob"].view(B, K).cpu().numpy()
    want = oracle.verify(tgt.cpu().numpy(), drf.cpu().numpy(), tok.cpu().numpy(), u.cpu().numpy(),
                         np.full(B, 0.8, np.float32), "f32")
    np.testing.assert_array_equal(out["accept_len"].cpu().numpy(), want["accept_len"])
    np.testing.assert_array_equal(out["bonus"].cpu().numpy(), want["bonus"])
    for b in range(B):
        a = int(want["accept_len"][b])
        n = min(a + 1, K)
        np.testing.assert_allclose(out["q_tok"].cpu().numpy()[b, :n], q[b, :n], rtol=1e-5)
        assert float(tgt[b, a, int(want["bonus"][b])]) != ssd.SSD_DROPPED_LOGIT


@pytest.mark.parametrize("dtype", DT)
def test_rows_too_low_for_filtered_logits_are_reported(ssd, dtype):
    """A dropped logit has weight 0 next to one that is 104 tau above it.  Rows that lie lower keep their logits, and the status
    says so; their tokens are drawn as ever."""
    V = 500
    z, rng = _rows(8, 8, V, dtype)
    drop = float(torch.tensor(ssd.SSD_DROPPED_LOGIT).to(dtype))
    low = (z.float() - z.float().max(dim=1, keepdim=True).values).clamp_min(-20.0) * 512 + drop    # the largest is `drop`
    low = low.to(dtype)

    def run(x, tau, k):
        n = x.shape[0]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        u = rng.random(n).astype(np.float32)
        out = ssd.ssd_sample(x.cuda(), _t([tau] * n), _t(u), top_k=_t([k] * n, torch.int32), filtered=True, dev_status=status)
        want = [ref.sample(r.double().numpy(), float(np.float32(tau)), k, 1.0, 0.0, float(v)) for r, v in zip(x, u)]
        for t, w in zip(out["tokens"].tolist(), want):
            assert w[3] < MARGIN or t == w[0]
        return out["filtered"].cpu(), int(status)

    for shift, tau, k in ((0.0, 300.0, 7), (-2e5, 300.0, 7), (0.0, 0.0, 0), (-1024.0, 0.0, 0), (1024.0, 20.0, 7)):
        x = (low.float() + shift).to(dtype)
        got, status = run(x, tau, k)
        assert status == ssd.SSD_DEV_LOW_LOGITS, (shift, tau)
        assert torch.equal(got, x)
    # nothing dropped, or the largest far enough above
    x = (low.float() - 2e5).to(dtype)
    got, status = run(x, 300.0, 0)
    assert status == 0 and torch.equal(got, x)
    for shift, tau, k in ((1024.0, 0.0, 0), (1024.0, 2.0, 7), (1e5, 900.0, 7)):
        x = (low.float() + shift).to(dtype)
        got, status = run(x, tau, k)
        assert status == 0, (shift, tau)
        assert ((got == drop).sum(dim=1) >= V - max(k, 1) - 1).all()
