"""CPU checks of the serving loop's operators: what the library and the binding refuse before anything
reaches a GPU, and the plain forms that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import _loop_ref as ref

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ssd():
    from speculative_decoding_verification_ssd_gb300 import _build
    _build.build()
    import speculative_decoding_verification_ssd_gb300 as m
    return m


P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)


def test_plan_refuses(ssd):
    def call(seq=P, new=P, held=P, B=4, table=P, blocks=8, ring=P, state=P, pages=100, page=16, cap=20, slots=P, pos=P, cu=P):
        return ssd.lib().ssd_kv_plan(seq, None, new, held, B, table, blocks, ring, state, pages, page, cap, cu, P, slots, pos, None,
                                     None)
    bad = ssd.SSD_ERR_INVALID_ARG
    for kw in (dict(seq=None), dict(new=None), dict(held=None), dict(table=None), dict(ring=None), dict(state=None), dict(cu=None),
               dict(slots=None), dict(pos=None), dict(B=0), dict(blocks=0), dict(pages=0), dict(cap=-1), dict(page=24),
               dict(page=256), dict(page=0)):
        assert call(**kw) == bad, kw
    for kw in (dict(B=ssd.SSD_KV_MAX_B + 1), dict(pages=2 ** 28, page=16), dict(B=4096, blocks=2 ** 20),
               dict(B=1, blocks=2 ** 28, page=16)):
        assert call(**kw) == ssd.SSD_ERR_UNSUPPORTED, kw


def test_append_refuses(ssd):
    def call(k=P, v=P, dtype=ssd.SSD_BF16, ks=1024, vs=1024, slots=P, T=3, H=8, D=128, kc=P, vc=P, sc=P, pages=10, page=16):
        return ssd.lib().ssd_kv_append(k, v, dtype, ks, vs, slots, T, H, D, kc, vc, sc, P, pages, page, None, None)
    for kw in (dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vc=None), dict(sc=None), dict(T=-1), dict(H=0),
               dict(D=96), dict(pages=0), dict(page=48), dict(ks=1023), dict(vs=8), dict(kc=ODD), dict(vc=ODD)):
        assert call(**kw) == ssd.SSD_ERR_INVALID_ARG, kw
    assert call(dtype=3) == ssd.SSD_ERR_DTYPE
    assert call(pages=2 ** 27) == ssd.SSD_ERR_UNSUPPORTED
    assert call(pages=2 ** 24, page=128) == ssd.SSD_ERR_UNSUPPORTED
    assert call(T=0, k=None, v=None, slots=None) == ssd.SSD_OK


def test_attend_refuses(ssd):
    n = ssd.lib().ssd_kv_workspace_size()
    assert n % 256 == 0

    def call(q=P, dtype=ssd.SSD_BF16, stride=4096, kc=P, vc=P, ks=P, vs=P, pages=10, page=16, Hq=32, Hkv=8, D=128, table=P, blocks=4,
             cu=P, kv=P, B=2, T=3, max_new=2, scale=0.1, window=0, out=P, ws=P, nbytes=n):
        return ssd.lib().ssd_kv_attend(q, dtype, stride, kc, vc, ks, vs, pages, page, Hq, Hkv, D, table, blocks, cu, kv, B, T, max_new,
                                       ctypes.c_float(scale), window, out, ws, nbytes, None, None)
    for kw in (dict(q=None), dict(kc=None), dict(vc=None), dict(ks=None), dict(vs=None), dict(table=None), dict(cu=None),
               dict(kv=None), dict(out=None), dict(q=ODD), dict(kc=ODD), dict(vc=ODD), dict(out=ODD), dict(stride=4095),
               dict(stride=4100), dict(B=0), dict(T=-1), dict(max_new=0), dict(pages=0), dict(blocks=0), dict(Hkv=0), dict(Hq=0),
               dict(Hq=12), dict(window=-1), dict(page=20), dict(D=32), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(**kw) == ssd.SSD_ERR_INVALID_ARG, kw
    for dtype in (ssd.SSD_F32, 7):
        assert call(dtype=dtype) == ssd.SSD_ERR_DTYPE
    for kw in (dict(ws=None), dict(ws=ODD), dict(nbytes=n - 1)):
        assert call(**kw) == ssd.SSD_ERR_WORKSPACE, kw
    for kw in (dict(pages=2 ** 27), dict(pages=2 ** 25), dict(B=2048, blocks=2 ** 20), dict(blocks=2 ** 27), dict(B=5000)):
        assert call(**kw) == ssd.SSD_ERR_UNSUPPORTED, kw
    assert call(T=0, q=None, out=None) == ssd.SSD_OK


def test_sample_refuses(ssd):
    def call(z=P, dtype=ssd.SSD_F32, rows=2, V=100, ld=100, tau=P, u=P, tokens=P):
        return ssd.lib().ssd_sample(z, dtype, rows, V, ld, tau, None, None, None, u, tokens, None, None, None, None)
    for kw in (dict(z=None), dict(tau=None), dict(u=None), dict(tokens=None), dict(rows=0), dict(V=1), dict(ld=99)):
        assert call(**kw) == ssd.SSD_ERR_INVALID_ARG, kw
    assert call(dtype=ssd.SSD_F16) == ssd.SSD_ERR_DTYPE
    assert call(V=400001, ld=400001) == ssd.SSD_ERR_UNSUPPORTED
    assert call(dtype=ssd.SSD_BF16, V=800001, ld=800001) == ssd.SSD_ERR_UNSUPPORTED


def test_binding_refuses_host_tensors(ssd):
    i, f = torch.zeros(2, dtype=torch.int32), torch.zeros(2)
    with pytest.raises(TypeError):
        ssd.ssd_kv_plan(i, i, i, i.view(2, 1), i, i, 16, 2)
    c, s = torch.zeros((2, 1, 16, 64), dtype=torch.uint8), torch.zeros((2, 1))
    x = torch.zeros((2, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        ssd.ssd_kv_append(x, x, i, c, c, s, s)
    with pytest.raises(TypeError):
        ssd.ssd_kv_attend(x, c, c, s, s, i.view(1, 2), i, i[:1], 1, 1.0)
    with pytest.raises(TypeError):
        ssd.ssd_sample(torch.zeros((2, 9)), f, f)


def test_e4m3_rounding_of_the_plain_form():
    """Against torch's conversion, over every halfway point and its neighbours."""
    pos = ref.e4m3_values()[:127]
    mid = (pos[1:] + pos[:-1]) / 2
    x = np.concatenate([pos, mid, np.nextafter(mid.astype(np.float32), np.float32(1e9)),
                        np.nextafter(mid.astype(np.float32), np.float32(0)), [1e-9, 448.0]]).astype(np.float32)
    x = np.concatenate([x, -x])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    np.testing.assert_array_equal(ref.to_e4m3(x), want)
    np.testing.assert_array_equal(ref.e4m3_values(), torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy())


def test_digits_of_a_query_are_exact():
    """With a row's largest channel in [128, 256), a bf16 value is the sum of two e4m3 digits from 2^-2 on and an
    fp16 value of three from 2 on; below, the digits are off by 2^-10 at most."""
    for bits, digits, exact_from in ((8, 2, -2), (11, 3, 1)):
        m = np.arange(2 ** (bits - 1), 2 ** bits, dtype=np.float64) / 2 ** (bits - 1)
        for e in range(-12, 8):
            x = rest = m * 2.0 ** e
            got = np.zeros_like(x)
            for _ in range(digits):
                t = ref.to_e4m3(rest)
                got, rest = got + t, rest - t
            if e >= exact_from:
                np.testing.assert_array_equal(got, x)
            else:
                assert np.abs(got - x).max() <= 2.0 ** -10


def test_plain_sample_keeps_prefixes():
    z = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    assert ref.sample(z, 1.0, 2, 1.0, 0.0, 0.5)[2].tolist() == [1, 3]
    assert ref.sample(z, 1.0, 0, 0.75, 0.0, 0.5)[2].tolist() == [1, 2, 3]
    assert ref.sample(z, 1.0, 0, 1.0, 0.6, 0.5)[2].tolist() == [1, 3]
    assert ref.sample(z, 1.0, 0, 1.0, 0.0, 0.55)[0] == 2
    assert ref.sample(z, 0.0, 0, 1.0, 0.0, 0.9)[0] == 1
    token, prob, _, _ = ref.sample(z, 1.0, 2, 1.0, 0.0, 0.99)
    assert token == 3 and abs(prob - 3 / 7) < 1e-12


@pytest.mark.parametrize("scale", [2.5e38, -3e38, float("nan"), -float("inf")])
def test_attend_refuses_a_scale_that_is_not_finite_in_base_2(ssd, scale):
    n = ssd.lib().ssd_kv_workspace_size()
    assert ssd.lib().ssd_kv_attend(P, ssd.SSD_BF16, 4096, P, P, P, P, 10, 16, 32, 8, 128, P, 4, P, P, 2, 3, 2, ctypes.c_float(scale), 0, P,
                                   P, n, None, None) == ssd.SSD_ERR_INVALID_ARG


def test_plan_refuses_a_cap_whose_indexes_pass_32_bits(ssd):
    """Of a turn of 2^14 tokens a thread's index starts among the first 2^12, and goes on while it is below the cap."""
    turn = 8 * 512 * 4

    def index_at_the_end(cap):
        last = cap - 1
        return last - max(0, last % turn - (turn // 4 - 1)) + turn

    assert index_at_the_end(2 ** 31 - turn - 1) < 2 ** 31
    for cap in (2 ** 31 - turn + 1, 2 ** 31 - 1):
        assert index_at_the_end(cap) >= 2 ** 31
        assert ssd.lib().ssd_kv_plan(P, None, P, P, 4, P, 8, P, P, 100, 16, cap, P, P, P, P, None, None) == ssd.SSD_ERR_UNSUPPORTED


@pytest.mark.parametrize("T,B,Hkv,blocks,page", [(8, 8, 119000000, 1, 16), (8, 8, 119000000, 1, 128), (16, 16, 70000000, 9, 16)])
def test_attend_refuses_more_steps_than_32_bits(ssd, T, B, Hkv, blocks, page):
    """One token each of B sequences: ceil(keys / 256) steps and two for the start, for every head."""
    keys, n = blocks * page, ssd.lib().ssd_kv_workspace_size()
    assert B * Hkv * (-(-keys // 256) + 2) >= 2 ** 31
    got = ssd.lib().ssd_kv_attend(P, ssd.SSD_BF16, Hkv * 64, P, P, P, P, 1, 16, Hkv, Hkv, 64, P, blocks * page // 16, P, P, B, T, 1,
                                  ctypes.c_float(1.0), 0, P, P, n, None, None)
    assert got == ssd.SSD_ERR_UNSUPPORTED


class Somewhere(torch.Tensor):
    """A host tensor that says it is on a GPU."""
    __torch_function__ = torch._C._disabled_torch_function_impl
    where = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.where


def _calls(ssd, where):
    """(call, names of its tensors) for the four operators; where: the device of each tensor by name."""
    def t(name, shape, dtype=torch.int32):
        x = torch.zeros(shape, dtype=dtype).as_subclass(Somewhere)
        x.where = where.get(name, where.get("*", 0))
        return x
    f32, bf16, u8 = torch.float32, torch.bfloat16, torch.uint8

    def cache():
        return (t("k_cache", (3, 2, 16, 64), u8), t("v_cache", (3, 2, 16, 64), u8), t("k_scale", (3, 2), f32), t("v_scale", (3, 2), f32))

    def plan():
        out = {"cu_new": t("cu_new", 3), "kv_len": t("kv_len", 2), "slots": t("slots", 5), "positions": t("positions", 5)}
        ssd.ssd_kv_plan(t("seq_len", 2), t("new_len", 2), t("held", 2), t("block_table", (2, 4)), t("ring", 3), t("ring_state", 2), 16, 5,
                        accept_len=t("accept_len", 2), out=out, dev_status=t("dev_status", 1))

    def append():
        ssd.ssd_kv_append(t("k", (5, 2, 64), bf16), t("v", (5, 2, 64), bf16), t("slots", 5), *cache(), dev_status=t("dev_status", 1))

    def attend():
        ssd.ssd_kv_attend(t("q", (5, 4, 64), bf16), *cache(), t("block_table", (2, 4)), t("cu_new", 3), t("kv_len", 2), 5, 1.0,
                          out=t("out", (5, 4, 64), bf16), workspace=t("workspace", 256, u8), dev_status=t("dev_status", 1))

    def sample():
        ssd.ssd_sample(t("logits", (2, 9), f32), t("temperature", 2, f32), t("uniforms", 2, f32), top_k=t("top_k", 2),
                       top_p=t("top_p", 2, f32), min_p=t("min_p", 2, f32), filtered=t("filtered", (2, 9), f32), tokens=t("tokens", 2),
                       prob=t("prob", 2, f32), dev_status=t("dev_status", 1))

    c = ["k_cache", "v_cache", "k_scale", "v_scale"]
    return [(plan, ["seq_len", "new_len", "held", "block_table", "ring", "ring_state", "accept_len", "cu_new", "kv_len", "slots",
                    "positions", "dev_status"]),
            (append, ["k", "v", "slots", "dev_status"] + c),
            (attend, ["q", "block_table", "cu_new", "kv_len", "out", "workspace", "dev_status"] + c),
            (sample, ["logits", "temperature", "uniforms", "top_k", "top_p", "min_p", "filtered", "tokens", "prob", "dev_status"])]


def test_binding_refuses_tensors_of_another_device(ssd, monkeypatch):
    """The kernels launch on the current device and would read another one's addresses."""
    launched = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: launched.append(name) or 0

    monkeypatch.setattr(ssd, "lib", Lib)
    monkeypatch.setattr(ssd, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(ssd, "_current_stream", lambda device: 0)
    for i in range(4):
        call, names = _calls(ssd, {})[i]
        call()
        assert len(launched) == 1
        launched.clear()
        for name in names + ["*"]:
            with pytest.raises(ValueError, match="current device"):
                _calls(ssd, {name: 1})[i][0]()
            assert not launched, name


def test_binding_refuses_a_stream_of_another_device(ssd, monkeypatch):
    class Stream:
        device_index = 1
        cuda_stream = 5
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(ssd, "_current_device", lambda: 0, raising=False)
    with pytest.raises(ValueError, match="current device"):
        ssd._stream_at(Stream(), None)
    Stream.device_index = 0
    assert ssd._stream_at(Stream(), None) == 5 and ssd._stream_at(7, None) == 7
