"""ssd_kv_attend over whole prompts, against the plain form in 64 bits: thousands of new tokens of one sequence, which
make hundreds of row blocks and go through the schedule's own launch."""
import pytest

from test_gpu_kv_attend import BF, FP, Case

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_ssd_gb300 as m
    return m


@pytest.mark.parametrize("pairs,Hq,Hkv,D,P,dtype,window", [
    ([(4000, 4000)], 2, 1, 128, 64, BF, 0),
    ([(4000, 4000)], 1, 1, 64, 16, FP, 0),
    ([(1000, 1000), (1003, 999), (1, 1)], 4, 2, 128, 32, BF, 0),
    ([(1000, 1000), (1003, 999), (1, 1)], 4, 2, 128, 128, FP, 0),
    ([(5000, 512)], 4, 2, 128, 128, BF, 0),          # a piece behind a long cache
    ([(3000, 1500), (700, 3)], 4, 1, 64, 16, BF, 1024),
    ([(3000, 1500), (700, 3)], 4, 1, 64, 64, FP, 100),
])
def test_prompts(ssd, pairs, Hq, Hkv, D, P, dtype, window):
    Case(30 + D + window, pairs, Hq, Hkv, D, P, dtype).check(ssd, window=window)
