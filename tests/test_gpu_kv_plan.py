"""ssd_kv_plan against a plain form, request by request: whole numbers, so exact equality."""
import os
import random
import subprocess
import sys

import pytest

import _loop_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_ssd_gb300 as m
    return m


def _i(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _random_state(rng, B, P, most, spare, accept):
    lens = [rng.choice([0, rng.randint(0, most)]) for _ in range(B)]
    held = [min(-(-most // P) + 2, -(-n // P) + rng.choice([0, 0, 1, 2])) for n in lens]
    m = -(-most // P) + 4
    n = sum(held) + spare
    pages = list(range(n))
    rng.shuffle(pages)
    table, at = [], 0
    for h in held:
        table.append(pages[at:at + h] + [-1] * (m - h))
        at += h
    head = rng.randrange(n)
    ring = [-7] * n
    for i, p in enumerate(pages[at:]):
        ring[(head + i) % n] = p
    acc = [rng.randint(-1, 4) for _ in range(B)] if accept else None
    return lens, acc, held, table, ring, head, n - at


def _check(ssd, lens, acc, new, held, table, ring, head, count, P, cap):
    want, status = ref.plan(lens, acc, new, held, table, ring, head, count, P, cap)
    st = dict(seq_len=_i(lens), held=_i(held), block_table=_i(table), ring=_i(ring), ring_state=_i([head, count]))
    dev = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ssd.ssd_kv_plan(st["seq_len"], _i(new), st["held"], st["block_table"], st["ring"], st["ring_state"], P, cap,
                          accept_len=None if acc is None else _i(acc), dev_status=dev)
    torch.cuda.synchronize()
    got = {k: v.cpu().tolist() for k, v in {**out, **st}.items()}
    for k in want:
        assert got[k] == want[k], k
    assert int(dev) == status
    return got


@pytest.mark.parametrize("accept", [False, True])
@pytest.mark.parametrize("B,P,most,new_max,spare", [
    (1, 16, 0, 1, 1), (1, 128, 500, 3, 2), (7, 16, 100, 40, 60), (33, 64, 700, 5, 40), (256, 64, 4000, 5, 256),
    (513, 32, 90, 9, 200), (1500, 16, 60, 3, 900), (40, 16, 300, 900, 2600), (5, 128, 9000, 4000, 200),
    (4096, 128, 200, 2, 4096)])
def test_plan_matches_plain_form(ssd, B, P, most, new_max, spare, accept):
    rng = random.Random(B * 1000 + P + accept)
    lens, acc, held, table, ring, head, count = _random_state(rng, B, P, most + new_max, spare, accept)
    new = [rng.choice([0, rng.randint(0, new_max)]) for _ in range(B)]
    _check(ssd, lens, acc, new, held, table, ring, head, count, P, sum(new) + rng.randint(0, 5))


def test_pages_run_out(ssd):
    rng = random.Random(5)
    lens, acc, held, table, ring, head, count = _random_state(rng, 60, 16, 400, 25, True)
    new = [rng.randint(0, 90) for _ in range(60)]
    _check(ssd, lens, acc, new, held, table, ring, head, count, 16, sum(new))


def test_lengths_that_cannot_be(ssd):
    rng = random.Random(6)
    lens, acc, held, table, ring, head, count = _random_state(rng, 9, 16, 100, 60, False)
    new = [1, -3, 4, 5, 100000, 0, 2, 7, 1]
    lens[3], held[6] = -5, -1
    _check(ssd, lens, acc, new, held, table, ring, head, count, 16, 100030)
    # the tokens of the last requests end beyond the cap
    lens, acc, held, table, ring, head, count = _random_state(rng, 9, 16, 100, 60, False)
    _check(ssd, lens, acc, [3] * 9, held, table, ring, head, count, 16, 17)


def test_nothing_asked(ssd):
    rng = random.Random(8)
    lens, acc, held, table, ring, head, count = _random_state(rng, 4, 32, 100, 3, False)
    _check(ssd, lens, acc, [0] * 4, held, table, ring, head, count, 32, 0)


def test_a_loop_conserves_the_pages(ssd):
    """Sixty rounds of growing, accepting and finishing: every page is either held once or free."""
    rng = random.Random(9)
    B, P, N = 12, 16, 200
    st = ssd.kv_state(B, 40, N)
    acc = None
    for step in range(60):
        new = [rng.choice([5, 5, 5, 37, 0]) for _ in range(B)]
        if step % 7 == 6:
            st["seq_len"][rng.randrange(B)] = 0
        if step % 5 == 0:
            acc = None
        a = None if acc is None else _i(acc)
        out = ssd.ssd_kv_plan(st["seq_len"], _i(new), st["held"], st["block_table"], st["ring"], st["ring_state"], P,
                              sum(new), accept_len=a)
        torch.cuda.synchronize()
        # greedy lengths stay within the table: reset the long ones
        long = (st["seq_len"] > 500).nonzero().flatten().tolist()
        for b in long:
            st["seq_len"][b] = 0
        held, table = st["held"].tolist(), st["block_table"].tolist()
        head, count = st["ring_state"].tolist()
        ring = st["ring"].tolist()
        owned = [p for b in range(B) for p in table[b][:held[b]]]
        assert all(p == -1 for b in range(B) for p in table[b][held[b]:])
        assert sorted(owned + [ring[(head + i) % N] for i in range(count)]) == list(range(N))
        assert out["cu_new"][-1] == sum(new)
        acc = [rng.randint(0, max(0, n - 1)) if n else -1 for n in new]


def test_a_broken_ring_serves_nobody(ssd):
    dev = torch.zeros(1, dtype=torch.int32, device="cuda")
    st = ssd.kv_state(2, 4, 8)
    st["ring_state"][1] = 9
    out = ssd.ssd_kv_plan(st["seq_len"], _i([3, 0]), st["held"], st["block_table"], st["ring"], st["ring_state"], 16, 3,
                          dev_status=dev)
    assert out["slots"].tolist() == [-1, -1, -1] and st["held"].tolist() == [0, 0]
    assert int(dev) & ssd.SSD_DEV_BAD_PAGE


def _batch(ssd, B):
    rng = random.Random(B)
    lens, acc, held, table, ring, head, count = _random_state(rng, B, 64, 300, B, True)
    new = [rng.randint(0, 5) for _ in range(B)]
    _check(ssd, lens, acc, new, held, table, ring, head, count, 64, sum(new))


def test_batches_around_48_kb_of_sums_in_a_fresh_process(ssd):
    """The sums of 2043 requests and the kernel's fixed shared memory pass 48 KB together: no larger batch has raised
    the limit before."""
    here = os.path.dirname(os.path.abspath(__file__))
    code = ("import test_gpu_kv_plan as t, speculative_decoding_verification_ssd_gb300 as ssd\n"
            "for B in (2042, 2043, 2048, 2049): t._batch(ssd, B)")
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([os.path.dirname(here), here]))
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
