"""ssd_kv_append against a plain form in 64 bits.  Scales are powers of two, so every stored value is the
correctly rounded one: equality of every byte's value and every scale."""
import numpy as np
import pytest

import _loop_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
VALUES = ref.e4m3_values()


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_ssd_gb300 as m
    return m


def _cache(rng, N, H, P, D):
    codes = rng.integers(0, 256, (N, H, P, D)).astype(np.uint8)
    codes[(codes & 127) == 127] = 0
    scale = 2.0 ** rng.integers(-12, 3, (N, H))
    return codes, scale


def _x(rng, T, H, D, dtype):
    x = rng.standard_normal((T, H, D)) * 2.0 ** rng.integers(-8, 9, (T, H, 1))
    return torch.from_numpy(x).to(dtype)


def _run(ssd, x2, slots, caches, scales, P, stride_pad=0, status=None):
    """The call on views with a longer token stride; returns the caches and scales after it."""
    T, H, D = x2[0].shape
    dev = []
    for x in x2:
        t = torch.zeros((T, H * D + stride_pad), dtype=x.dtype, device="cuda")
        t[:, :H * D] = x.reshape(T, H * D).cuda()
        dev.append(t[:, :H * D].unflatten(1, (H, D)))
    c = [torch.from_numpy(a).cuda() for a in caches]
    s = [torch.from_numpy(a.astype(np.float32)).cuda() for a in scales]
    ssd.ssd_kv_append(dev[0], dev[1], torch.tensor(slots, dtype=torch.int32, device="cuda"), c[0], c[1], s[0], s[1],
                      dev_status=status)
    torch.cuda.synchronize()
    return [a.cpu().numpy() for a in c], [a.cpu().numpy().astype(np.float64) for a in s]


def _compare(ssd, rng, N, H, P, D, slots, dtype, pad=0, x2=None, caches=None):
    both = caches or [_cache(rng, N, H, P, D) for _ in range(2)]
    x2 = x2 or [_x(rng, len(slots), H, D, dtype) for _ in range(2)]
    codes, scales = _run(ssd, x2, slots, [b[0] for b in both], [b[1] for b in both], P, pad)
    for i in range(2):
        values, scale = VALUES[both[i][0]], both[i][1].copy()
        ref.append(x2[i].to(torch.float64).numpy(), slots, values, scale, P)
        np.testing.assert_array_equal(scales[i], scale)
        np.testing.assert_array_equal(VALUES[codes[i]], values)


def _runs(rng, N, P, runs):
    """Slots of `runs` (row0, tokens) runs, each going over into further pages of its own."""
    pages, slots = list(rng.permutation(N)), []
    for row0, n in runs:
        pos = row0
        page = pages.pop()
        for _ in range(n):
            if pos == P:
                page, pos = pages.pop(), 0
            slots.append(int(page) * P + pos)
            pos += 1
    return slots


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("H,P,D,runs", [
    (1, 16, 64, [(0, 1)]), (2, 16, 64, [(15, 1), (3, 13), (0, 16), (0, 17)]),
    (3, 32, 128, [(31, 2), (1, 1), (5, 100), (0, 0), (9, 23)]), (8, 64, 128, [(63, 5), (61, 5), (7, 5)] * 9),
    (4, 128, 64, [(100, 300), (0, 128), (127, 1)]), (2, 128, 128, [(1, 127), (64, 200)]),
    (8, 64, 64, [(i % 64, 1 + i % 7) for i in range(300)])])
def test_append_matches_plain_form(ssd, H, P, D, runs, dtype):
    rng = np.random.default_rng(H * 1000 + P + D)
    N = sum(2 + (a + n) // P for a, n in runs) + 2
    _compare(ssd, rng, N, H, P, D, _runs(rng, N, P, runs), dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [31, 32, 33, 50, 64, 65, 100])
def test_runs_that_end_before_their_page(ssd, n, D, dtype):
    """Runs longer than the slots looked at at once, other sequences' tokens right behind them."""
    rng = np.random.default_rng(900 + n)
    slots = _runs(rng, 12, 128, [(0, n), (3, n), (128 - n, n), (0, 128), (17, n), (0, 1)])
    _compare(ssd, rng, 12, 2, 128, D, slots, dtype)


@pytest.mark.parametrize("pad", [8, 3])  # 3: rows that no 16-byte load can take
def test_strided_tokens(ssd, pad):
    rng = np.random.default_rng(pad)
    _compare(ssd, rng, 12, 3, 32, 64, _runs(rng, 12, 32, [(5, 60), (31, 3)]), torch.bfloat16, pad)


def test_padding_and_slots_beyond_the_cache_are_skipped(ssd):
    rng = np.random.default_rng(3)
    slots = [-1, 5, 6, -1, 7 * 16, 99999, 2147483647, 3 * 16 + 15, -5]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    both = [_cache(rng, 8, 2, 16, 64) for _ in range(2)]
    x2 = [_x(rng, len(slots), 2, 64, torch.bfloat16) for _ in range(2)]
    codes, scales = _run(ssd, x2, slots, [b[0] for b in both], [b[1] for b in both], 16, status=status)
    assert int(status) == ssd.SSD_DEV_BAD_PAGE
    for i in range(2):
        values, scale = VALUES[both[i][0]], both[i][1].copy()
        ref.append(x2[i].to(torch.float64).numpy(), slots, values, scale, 16)
        np.testing.assert_array_equal(scales[i], scale)
        np.testing.assert_array_equal(VALUES[codes[i]], values)


def test_a_page_whose_scale_grows_is_stored_again(ssd):
    rng = np.random.default_rng(4)
    both = [_cache(rng, 3, 2, 16, 128) for _ in range(2)]
    for codes, scale in both:
        scale[:] = 2.0 ** -9
    x2 = [_x(rng, 4, 2, 128, torch.float32) * 2.0 ** 20 for _ in range(2)]
    _compare(ssd, rng, 3, 2, 16, 128, [16 + 11, 16 + 12, 16 + 13, 16 + 14], torch.float32, x2=x2, caches=both)


@pytest.mark.parametrize("value", [0.0, 448.0, 448.0000305, 449.0, 1e-38, 3e38, 896.0, 2.0 ** -92, 1.75 * 2.0 ** -92])
def test_scale_at_the_edges(ssd, value):
    rng = np.random.default_rng(7)
    x = torch.full((1, 1, 64), value, dtype=torch.float32)
    _compare(ssd, rng, 2, 1, 16, 64, [16], torch.float32, x2=[x, -x])


def test_infinities_and_nan(ssd):
    """They do not count for the scale; infinities become the largest value, NaN stays."""
    rng = np.random.default_rng(8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    both = [_cache(rng, 2, 1, 16, 64) for _ in range(2)]
    x2 = [_x(rng, 2, 1, 64, torch.bfloat16) for _ in range(2)]
    x2[0][0, 0, 3], x2[0][1, 0, 5], x2[1][0, 0, 0] = float("inf"), float("nan"), float("-inf")
    codes, scales = _run(ssd, x2, [0, 1], [b[0] for b in both], [b[1] for b in both], 16, status=status)
    assert int(status) == ssd.SSD_DEV_NONFINITE
    for i in range(2):
        values, scale = VALUES[both[i][0]], both[i][1].copy()
        ref.append(x2[i].to(torch.float64).numpy(), [0, 1], values, scale, 16)
        np.testing.assert_array_equal(scales[i], scale)
        np.testing.assert_array_equal(VALUES[codes[i]], values)
    assert VALUES[codes[0]][0, 0, 0, 3] == 448.0 and np.isnan(VALUES[codes[0]][0, 0, 1, 5])


def test_no_tokens(ssd):
    rng = np.random.default_rng(9)
    codes, scale = _cache(rng, 2, 1, 16, 64)
    e = torch.zeros((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    c, s = torch.from_numpy(codes).cuda(), torch.from_numpy(scale.astype(np.float32)).cuda()
    ssd.ssd_kv_append(e, e, torch.zeros(0, dtype=torch.int32, device="cuda"), c, c.clone(), s, s.clone())
    assert np.array_equal(c.cpu().numpy(), codes)


def test_cache_beyond_32_bits_of_bytes(ssd):
    N, H, P, D = 70000, 8, 128, 64          # 4.6 GB
    c = [torch.zeros((N, H, P, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    s = [torch.ones((N, H), device="cuda") for _ in range(2)]
    rng = np.random.default_rng(10)
    x = _x(rng, 3, H, D, torch.bfloat16)
    slots = [(N - 1) * P + 5, (N - 1) * P + 6, 33000 * P]
    ssd.ssd_kv_append(x.cuda(), x.cuda(), torch.tensor(slots, dtype=torch.int32, device="cuda"), c[0], c[1], s[0], s[1])
    for page, row0, rows, a in ((N - 1, 5, [5, 6], 0), (33000, 0, [0], 2)):
        values, scale = np.zeros((1, H, P, D)), np.ones((1, H))
        ref.append(x[a:a + len(rows)].to(torch.float64).numpy(), rows, values, scale, P)
        np.testing.assert_array_equal(VALUES[c[1][page].cpu().numpy()], values[0])
        np.testing.assert_array_equal(s[1][page].cpu().numpy().astype(np.float64), scale[0])
    assert int(c[0].count_nonzero(dim=(1, 2, 3)).count_nonzero()) == 2
