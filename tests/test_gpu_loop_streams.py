"""The serving loop's operators on another stream than the current one, and captured into graphs: the same
results as a plain call, and memory that a call allocates stays its own until that stream has used it."""
import random

import numpy as np
import pytest

import test_gpu_kv_plan as plans
from test_gpu_kv_attend import Case

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
BUSY = 40_000_000      # clocks, some 20 ms


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_ssd_gb300 as m
    return m


def _i(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Plan:
    def __init__(self, ssd):
        rng = random.Random(3)
        lens, acc, held, table, ring, head, count = plans._random_state(rng, 50, 16, 300, 400, True)
        self.new = [rng.randint(0, 60) for _ in range(50)]
        self.start = [_i(x) for x in (lens, held, table, ring, [head, count])]
        self.state = [t.clone() for t in self.start]
        self.args = _i(self.new), _i(acc)
        self.ssd = ssd

    def reset(self):
        for t, s in zip(self.state, self.start):
            t.copy_(s)

    def __call__(self, **kw):
        seq, held, table, ring, at = self.state
        out = self.ssd.ssd_kv_plan(seq, self.args[0], held, table, ring, at, 16, sum(self.new), accept_len=self.args[1], **kw)
        return list(out.values()) + self.state


class Append:
    def __init__(self, ssd):
        rng = np.random.default_rng(4)
        self.x = [torch.from_numpy(rng.standard_normal((90, 2, 64))).to(torch.bfloat16).cuda() for _ in range(2)]
        pages = rng.permutation(12)
        self.slots = _i(np.concatenate([p * 16 + np.arange(o, o + 7) for p, o in zip(pages, rng.integers(0, 9, 12))] +
                                       [[-1] * 6]).tolist())
        shape = (12, 2, 16, 64)
        self.start = [torch.from_numpy(rng.integers(0, 120, shape).astype(np.uint8)).cuda() for _ in range(2)] + \
            [torch.from_numpy(2.0 ** rng.integers(-12, -8, (12, 2))).float().cuda() for _ in range(2)]
        self.state = [t.clone() for t in self.start]
        self.ssd = ssd
    reset = Plan.reset

    def __call__(self, **kw):
        self.ssd.ssd_kv_append(*self.x, self.slots, *self.state, **kw)
        return self.state


class Attend:
    def __init__(self, ssd):
        c = Case(21, [(900, 5), (40, 3), (2000, 1)], 8, 2, 64, 32, torch.bfloat16)
        g = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.args = (c.q.cuda(), *(g(a) for a in (c.k, c.v, c.ks, c.vs, c.table, c.cu, c.kv)), 5, c.scale)
        self.ssd = ssd

    def reset(self):
        pass

    def __call__(self, **kw):
        return [self.ssd.ssd_kv_attend(*self.args, **kw)]


class Sample:
    def __init__(self, ssd):
        rng = np.random.default_rng(5)
        f = lambda a: torch.from_numpy(np.asarray(a, np.float32)).cuda()  # noqa: E731
        self.args = f(rng.standard_normal((20, 40000)) * 3), f(np.full(20, 0.8)), f(rng.random(20))
        self.kw = dict(top_k=_i([0, 40] * 10), top_p=f([0.9, 1.0] * 10), filtered=True)
        self.ssd = ssd
    reset = Attend.reset

    def __call__(self, **kw):
        return list(self.ssd.ssd_sample(*self.args, **self.kw, **kw).values())


@pytest.fixture(params=[Plan, Append, Attend, Sample])
def op(request, ssd):
    return request.param(ssd)


def _results(op, **kw):
    op.reset()
    return [t.clone() for t in op(**kw)]


@pytest.mark.parametrize("as_number", [False, True])
def test_on_another_stream(op, as_number):
    want = _results(op)
    op.reset()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = op(stream=s.cuda_stream if as_number else s)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_what_a_call_allocates_is_not_handed_on_before_its_stream_has_used_it(op):
    op.reset()
    sizes = {t.numel() * t.element_size() for t in op()} | {1 << 20}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
    out = op(stream=s)
    del out
    mine = [torch.full((n,), 77, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    for t in mine:
        assert bool((t == 77).all())


def test_in_a_graph(op):
    want = _results(op)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    op.reset()
    with torch.cuda.stream(s):
        op()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = op()
    for _ in range(3):
        op.reset()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
