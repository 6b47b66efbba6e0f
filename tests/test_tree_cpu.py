"""CPU checks of the operators for trees: what the library and the binding refuse before anything reaches a GPU,
the frequencies' form, and the plain forms that the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest

import _loop_ref as loop
import _tree_ref as ref
from test_kv_cpu import ODD, P, Somewhere

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ssd():
    from speculative_decoding_verification_ssd_gb300 import _build
    _build.build()
    import speculative_decoding_verification_ssd_gb300 as m
    return m


def test_rope_refuses(ssd):
    def call(q=P, k=P, dtype=ssd.SSD_BF16, qs=4096, ks=1024, T=3, Hq=32, Hkv=8, D=128, qw=P, kw=P, eps=1e-6, pos=P, turns=P, rot=128,
             qo=P, ko=P, qos=4096, kos=1024):
        return ssd.lib().ssd_qk_rope(q, k, dtype, qs, ks, T, Hq, Hkv, D, qw, kw, ctypes.c_float(eps), pos, turns, rot, 0, qo, ko, qos, kos, None)
    for kw in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(pos=None), dict(turns=None), dict(T=-1), dict(Hq=0), dict(Hkv=0),
               dict(D=96), dict(rot=8), dict(rot=144), dict(rot=-16), dict(qw=None), dict(kw=None), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(qs=4095), dict(ks=8), dict(qos=0), dict(kos=1023)):
        assert call(**kw) == ssd.SSD_ERR_INVALID_ARG, kw
    assert call(dtype=3) == ssd.SSD_ERR_DTYPE
    assert call(T=1, Hq=2 ** 27, qs=2 ** 34, qos=2 ** 34) == ssd.SSD_ERR_UNSUPPORTED
    assert call(T=0, q=None, k=None, qo=None, ko=None, pos=None) == ssd.SSD_OK


def test_tree_plan_refuses(ssd):
    def call(parent=P, cu=P, seq=P, B=2, T=5, max_new=4, pos=P, mask=P):
        return ssd.lib().ssd_tree_plan(parent, cu, seq, B, T, max_new, pos, mask, None, None)
    for kw in (dict(parent=None), dict(cu=None), dict(seq=None), dict(pos=None), dict(mask=None), dict(B=0), dict(T=-1), dict(max_new=0)):
        assert call(**kw) == ssd.SSD_ERR_INVALID_ARG, kw
    for kw in (dict(B=ssd.SSD_KV_MAX_B + 1), dict(max_new=ssd.SSD_TREE_MAX + 1)):
        assert call(**kw) == ssd.SSD_ERR_UNSUPPORTED, kw
    assert call(T=0, parent=None, pos=None, mask=None) == ssd.SSD_OK


def test_tree_accept_refuses(ssd):
    def call(parent=P, tokens=P, sampled=P, cu=P, B=2, T=5, max_new=4, max_path=3, accept=P, bonus=P, path=P):
        return ssd.lib().ssd_tree_accept(parent, tokens, sampled, cu, B, T, max_new, max_path, accept, bonus, path, None, None)
    for kw in (dict(parent=None), dict(tokens=None), dict(sampled=None), dict(cu=None), dict(accept=None), dict(bonus=None), dict(path=None),
               dict(B=0), dict(T=-1), dict(max_new=0), dict(max_path=0), dict(max_path=ssd.SSD_MAX_K + 2)):
        assert call(**kw) == ssd.SSD_ERR_INVALID_ARG, kw
    for kw in (dict(B=ssd.SSD_KV_MAX_B + 1), dict(max_new=ssd.SSD_TREE_MAX + 1)):
        assert call(**kw) == ssd.SSD_ERR_UNSUPPORTED, kw


def test_compact_refuses(ssd):
    def call(path=P, accept=P, seq=P, B=2, J=5, table=P, blocks=4, H=8, D=128, kc=P, vc=P, ks=P, vs=P, pages=10, page=16):
        return ssd.lib().ssd_kv_compact(path, accept, seq, B, J, table, blocks, H, D, kc, vc, ks, vs, pages, page, None, None)
    for kw in (dict(path=None), dict(accept=None), dict(seq=None), dict(table=None), dict(kc=None), dict(vc=None), dict(ks=None), dict(vs=None),
               dict(B=0), dict(J=0), dict(J=ssd.SSD_MAX_K + 2), dict(blocks=0), dict(H=0), dict(D=32), dict(pages=0), dict(page=24), dict(kc=ODD),
               dict(vc=ODD)):
        assert call(**kw) == ssd.SSD_ERR_INVALID_ARG, kw
    for kw in (dict(B=5000), dict(pages=2 ** 27), dict(pages=2 ** 25, H=8), dict(B=2048, blocks=2 ** 20), dict(blocks=2 ** 27)):
        assert call(**kw) == ssd.SSD_ERR_UNSUPPORTED, kw


def test_attend_tree_refuses(ssd):
    n = ssd.lib().ssd_kv_tree_workspace_size()
    assert n % 256 == 0

    def call(q=P, dtype=ssd.SSD_BF16, stride=4096, kc=P, vc=P, ks=P, vs=P, pages=10, page=16, Hq=32, Hkv=8, D=128, table=P, blocks=4,
             cu=P, kv=P, mask=P, B=2, T=3, max_new=2, scale=0.1, window=0, out=P, ws=P, nbytes=n):
        return ssd.lib().ssd_kv_attend_tree(q, dtype, stride, kc, vc, ks, vs, pages, page, Hq, Hkv, D, table, blocks, cu, kv, mask, B, T, max_new,
                                            ctypes.c_float(scale), window, out, ws, nbytes, None, None)
    for kw in (dict(q=None), dict(kc=None), dict(vc=None), dict(ks=None), dict(vs=None), dict(table=None), dict(cu=None), dict(mask=None),
               dict(kv=None), dict(out=None), dict(q=ODD), dict(kc=ODD), dict(vc=ODD), dict(out=ODD), dict(stride=4095),
               dict(stride=4100), dict(B=0), dict(T=-1), dict(max_new=0), dict(pages=0), dict(blocks=0), dict(Hkv=0), dict(Hq=0),
               dict(Hq=12), dict(window=-1), dict(page=20), dict(D=32), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=2.5e38)):
        assert call(**kw) == ssd.SSD_ERR_INVALID_ARG, kw
    for dtype in (ssd.SSD_F32, 7):
        assert call(dtype=dtype) == ssd.SSD_ERR_DTYPE
    for kw in (dict(ws=None), dict(ws=ODD), dict(nbytes=n - 1)):
        assert call(**kw) == ssd.SSD_ERR_WORKSPACE, kw
    for kw in (dict(pages=2 ** 27), dict(pages=2 ** 25), dict(B=2048, blocks=2 ** 20), dict(blocks=2 ** 27), dict(B=5000),
               dict(max_new=ssd.SSD_TREE_MAX + 1)):
        assert call(**kw) == ssd.SSD_ERR_UNSUPPORTED, kw
    assert call(T=0, q=None, out=None, mask=None) == ssd.SSD_OK


def test_timeout_check_refuses(ssd):
    n = ssd.lib().ssd_kv_tree_workspace_size()

    def call(withheld, dtype=ssd.SSD_BF16, D=128, q=P):
        return ssd.lib().ssd_check_tree_timeout(withheld, q, dtype, 4096, P, P, P, P, 10, 16, 32, 8, D, P, 4, P, P, P, 2, 3, 2,
                                                ctypes.c_float(0.1), 0, P, P, n, None, None)
    for withheld in (-1, 0, 6):
        assert call(withheld) == ssd.SSD_ERR_INVALID_ARG
    assert call(1, q=None) == ssd.SSD_ERR_INVALID_ARG
    assert call(1, dtype=ssd.SSD_F32) == ssd.SSD_ERR_DTYPE


def test_turns_hold_the_frequencies(ssd):
    f = [0.0, 1.0, 1e-4, 2 * math.pi * 0.75, -1.0, 10.0, 2 * math.pi * 5e-20]
    got = ssd.rope_turns(f, device="cpu")
    assert got.dtype == torch.int64
    for v, x in zip(got.tolist(), f):
        want = x / (2 * math.pi)
        assert abs((v / 2.0 ** 64 - want + 0.5) % 1.0 - 0.5) <= 2.0 ** -53
    assert torch.equal(ssd.rope_turns(torch.tensor(f, dtype=torch.float64)), got)
    for bad in (float("nan"), float("inf")):
        with pytest.raises(ValueError):
            ssd.rope_turns([bad], device="cpu")


def _calls(ssd, where):
    """(call, names of its tensors) for the operators; where: the device of each tensor by name."""
    def t(name, shape, dtype=torch.int32):
        x = torch.zeros(shape, dtype=dtype).as_subclass(Somewhere)
        x.where = where.get(name, where.get("*", 0))
        return x
    f32, bf16, u8 = torch.float32, torch.bfloat16, torch.uint8
    c = ["k_cache", "v_cache", "k_scale", "v_scale"]

    def cache():
        return (t("k_cache", (3, 2, 16, 64), u8), t("v_cache", (3, 2, 16, 64), u8), t("k_scale", (3, 2), f32), t("v_scale", (3, 2), f32))

    def rope():
        ssd.ssd_qk_rope(t("q", (5, 4, 64), bf16), t("k", (5, 2, 64), bf16), t("positions", 5), t("turns", 16, torch.int64),
                        q_weight=t("q_weight", 64, f32), k_weight=t("k_weight", 64, f32), q_out=t("q_out", (5, 4, 64), bf16),
                        k_out=t("k_out", (5, 2, 64), bf16))

    def plan():
        ssd.ssd_tree_plan(t("parent", 5), t("cu_new", 3), t("seq_len", 2), 40, out={"positions": t("positions", 5), "mask": t("mask", (5, 2))},
                          dev_status=t("dev_status", 1))

    def attend():
        ssd.ssd_kv_attend_tree(t("q", (5, 4, 64), bf16), *cache(), t("block_table", (2, 4)), t("cu_new", 3), t("kv_len", 2), t("mask", (5, 2)), 40,
                               1.0, out=t("out", (5, 4, 64), bf16), workspace=t("workspace", 256, u8), dev_status=t("dev_status", 1))

    def accept():
        out = {"accept_len": t("accept_len", 2), "bonus": t("bonus", 2), "path": t("path", (2, 3))}
        ssd.ssd_tree_accept(t("parent", 5), t("tokens", 5), t("sampled", 5), t("cu_new", 3), 4, 3, out=out, dev_status=t("dev_status", 1))

    def compact():
        ssd.ssd_kv_compact(t("path", (2, 3)), t("accept_len", 2), t("seq_len", 2), t("block_table", (2, 4)), *cache(), dev_status=t("dev_status", 1))

    return [(rope, ["q", "k", "positions", "turns", "q_weight", "k_weight", "q_out", "k_out"]),
            (plan, ["parent", "cu_new", "seq_len", "positions", "mask", "dev_status"]),
            (attend, ["q", "block_table", "cu_new", "kv_len", "mask", "out", "workspace", "dev_status"] + c),
            (accept, ["parent", "tokens", "sampled", "cu_new", "accept_len", "bonus", "path", "dev_status"]),
            (compact, ["path", "accept_len", "seq_len", "block_table", "dev_status"] + c)]


def test_binding_refuses_tensors_of_another_device(ssd, monkeypatch):
    launched = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: launched.append(name) or 0

    monkeypatch.setattr(ssd, "lib", Lib)
    monkeypatch.setattr(ssd, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(ssd, "_current_stream", lambda device: 0)
    for i in range(5):
        call, names = _calls(ssd, {})[i]
        call()
        assert len(launched) == 1
        launched.clear()
        for name in names + ["*"]:
            with pytest.raises(ValueError, match="current device"):
                _calls(ssd, {name: 1})[i][0]()
            assert not launched, name


def test_binding_refuses_host_tensors_and_shapes(ssd, monkeypatch):
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros((2, 1, 64), dtype=torch.bfloat16)
    c, s = torch.zeros((2, 1, 16, 64), dtype=torch.uint8), torch.zeros((2, 1))
    for call in (lambda: ssd.ssd_qk_rope(x, x, i, i.long()), lambda: ssd.ssd_tree_plan(i, i, i, 4),
                 lambda: ssd.ssd_kv_attend_tree(x, c, c, s, s, i.view(1, 2), i, i[:1], i.view(2, 1), 1, 1.0),
                 lambda: ssd.ssd_tree_accept(i, i, i, i, 4, 3), lambda: ssd.ssd_kv_compact(i.view(1, 2), i, i, i.view(1, 2), c, c, s, s)):
        with pytest.raises(TypeError):
            call()
    monkeypatch.setattr(ssd, "_current_device", lambda: 0, raising=False)

    def t(shape, dtype=torch.int32):
        return torch.zeros(shape, dtype=dtype).as_subclass(Somewhere)
    b16 = torch.bfloat16
    for call in (lambda: ssd.ssd_qk_rope(t((5, 4, 64), b16), t((4, 2, 64), b16), t(5), t(16, torch.int64)),
                 lambda: ssd.ssd_qk_rope(t((5, 4, 64), b16), t((5, 2, 64), b16), t(6), t(16, torch.int64)),
                 lambda: ssd.ssd_qk_rope(t((5, 256), b16), t((5, 2, 64), b16), t(5), t(16, torch.int64)),
                 lambda: ssd.ssd_tree_plan(t(5), t(4), t(2), 4), lambda: ssd.ssd_tree_plan(t(5), t(3), t(2), 0),
                 lambda: ssd.ssd_tree_accept(t(5), t(4), t(5), t(3), 4, 3),
                 lambda: ssd.ssd_kv_compact(t((2, 3)), t(2), t(3), t((2, 4)), t((3, 2, 16, 64), torch.uint8), t((3, 2, 16, 64), torch.uint8),
                                            t((3, 2), torch.float32), t((3, 2), torch.float32))):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("size", [1 << 31, 1 << 32, (1 << 32) + 5, 1 << 40, -(1 << 32) + 5])
def test_binding_refuses_sizes_beyond_32_bits(ssd, monkeypatch, size):
    """Not their lower bits in their place, and not a tensor of that size on the way."""
    class Lib:
        def __getattr__(self, name):
            def launch(*a):
                raise AssertionError(f"{name} was called")
            return launch

    monkeypatch.setattr(ssd, "lib", Lib)
    monkeypatch.setattr(ssd, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(ssd, "_current_stream", lambda device: 0)
    monkeypatch.setattr(ssd, "strerror", str)

    def t(shape, dtype=torch.int32):
        return torch.zeros(shape, dtype=dtype).as_subclass(Somewhere)
    f32, b16, u8 = torch.float32, torch.bfloat16, torch.uint8
    cache = (t((3, 2, 16, 64), u8), t((3, 2, 16, 64), u8), t((3, 2), f32), t((3, 2), f32))
    q, lens = t((5, 4, 64), b16), (t((2, 4)), t(3), t(2))
    kw = dict(out=t((5, 4, 64), b16), workspace=t(256, u8))
    for call in (lambda: ssd.ssd_kv_attend(q, *cache, *lens, 4, 1.0, window=size, **kw), lambda: ssd.ssd_kv_attend(q, *cache, *lens, size, 1.0, **kw),
                 lambda: ssd.ssd_kv_attend_tree(q, *cache, *lens, t((5, 1)), 4, 1.0, window=size, **kw),
                 lambda: ssd.ssd_kv_attend_tree(q, *cache, *lens, t((5, 1)), size, 1.0, **kw),
                 lambda: ssd.ssd_tree_plan(t(5), t(3), t(2), size), lambda: ssd.ssd_tree_accept(t(5), t(5), t(5), t(3), size, 3),
                 lambda: ssd.ssd_tree_accept(t(5), t(5), t(5), t(3), 4, size)):
        with pytest.raises((ValueError, ssd.SSDError)):
            call()


def test_plain_forms_of_a_small_tree():
    """     0 -> 1 -> 3 -> 5,  0 -> 2 -> 4"""
    parent = [-1, 0, 0, 1, 2, 3]
    pos, sees, status = ref.tree_plan(parent, [0, 6], [10], 6, 6)
    assert pos == [10, 11, 11, 12, 12, 13] and sees[5] == {0, 1, 3, 5} and sees[4] == {0, 2, 4} and status == 0
    assert ref.words(sees, 1)[5, 0] == 0b101011
    tokens = [9, 4, 5, 6, 7, 8]
    assert ref.tree_accept(parent, tokens, [5, 0, 7, 0, 3, 0], [0, 6], 6, 4) == ([2], [3], [[0, 2, 4, -1]], 0)
    assert ref.tree_accept(parent, tokens, [5, 0, 7, 0, 3, 0], [0, 6], 6, 2) == ([1], [7], [[0, 2]], 0)
    assert ref.seen(16, 6, 5, sees[5], 0, 99) == list(range(10)) + [10, 11, 13, 15]
    assert ref.seen(16, 6, 5, sees[5], 5, 99) == [9, 10, 11, 13, 15]


def test_plain_compact_moves_values():
    values, scale = np.zeros((3, 1, 16, 4)), np.array([[1.0], [2.0], [1.0]], np.float32)
    values[1, 0, :, 0] = np.arange(16)
    values[0, 0, :, 1] = 448
    table = np.array([[0, 1]])
    ref.compact([[0, 3, 9]], [2], [13], table, values, scale, 16)
    # position 13 stays; 16 (page 1) comes to row 14, where 2 * 0 fits the scale; 22 comes to row 15: 2 * 6
    assert scale[0, 0] == 1.0 and values[0, 0, 15, 0] == 12 and values[0, 0, 14, 0] == 0 and values[0, 0, 14, 1] == 0
    values[1, 0, 7, 0] = 448
    ref.compact([[0, 10]], [1], [13], table, values, scale, 16)
    assert scale[0, 0] == 2.0 and values[0, 0, 14, 0] == 448 and values[0, 0, 13, 1] == 224 and values[0, 0, 15, 0] == 12


def test_plain_rope_turns_pairs():
    x = np.zeros((1, 1, 64))
    x[0, 0, 0], x[0, 0, 40] = 1.0, 3.0
    y, _ = ref.rope(x, None, 0, [1], [math.pi / 2] * 8, False)
    assert abs(y[0, 0, 8] - 1) < 1e-15 and abs(y[0, 0, 0]) < 1e-15 and y[0, 0, 40] == 3
    y, _ = ref.rope(x, None, 0, [1], [math.pi / 2] * 8, True)
    assert abs(y[0, 0, 1] - 1) < 1e-15


def test_halves_hold_a_weight_as_derived():
    """fp16 rounds a normal value by 2^-11 of itself at most, a smaller one by 2^-25."""
    x = np.concatenate([2.0 ** np.linspace(-30, 15, 20001)])
    off = np.abs(torch.from_numpy(x).to(torch.float16).double().numpy() - x)
    assert (off <= np.maximum(2.0 ** -11 * x, 2.0 ** -25)).all()
    assert loop.to_e4m3(3.1) == 3.0
