"""The serving example, round by round: what the cache holds for every sequence is what its committed tokens say."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("B,K,D,Hkv,page", [(5, 4, 64, 2, 32), (9, 2, 128, 4, 16)])
def test_cache_follows_the_accepted_tokens(B, K, D, Hkv, page):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import serving_loop
    loop = serving_loop.Loop(B=B, K=K, V=1000, width=128, Hq=8, Hkv=Hkv, D=D, page=page, pages=B * 12, max_blocks=20, seed=B)
    rng = np.random.default_rng(B)
    history = [rng.integers(0, 1000, int(n)).tolist() for n in rng.integers(1, 70, B)]
    loop.prompt(history)
    for _ in range(12):
        accept, bonus, drafts = (t.cpu().numpy() for t in loop.round())
        assert int(loop.status) == 0
        assert ((accept >= 0) & (accept <= K)).all()
        for b in range(B):
            history[b] += drafts[b, :accept[b]].tolist() + [int(bonus[b])]
    # commit the last round
    st = loop.state
    none = torch.zeros(B, dtype=torch.int32, device="cuda")
    import speculative_decoding_verification_ssd_gb300 as ssd
    ssd.ssd_kv_plan(st["seq_len"], none, st["held"], st["block_table"], st["ring"], st["ring_state"], page, 0, accept_len=loop.accept)
    lens, held, table = st["seq_len"].tolist(), st["held"].tolist(), st["block_table"].cpu().numpy()
    assert lens == [len(h) - 1 for h in history]          # all but the token that is fed next
    assert held == [-(-n // page) for n in lens]
    pages = [p for b in range(B) for p in table[b, :held[b]]]
    head, count = st["ring_state"].tolist()
    ring = st["ring"].cpu().numpy()
    free = [ring[(head + i) % len(ring)] for i in range(count)]
    assert sorted(pages + free) == list(range(len(ring)))
    for b in range(B):
        n = lens[b]
        if n == 0:
            continue
        h = loop.target.hidden(torch.tensor(history[b][:n], device="cuda"), torch.arange(n, device="cuda"))
        _, k, v = loop.target.split(h)
        j = np.arange(n)
        at, row = torch.tensor(table[b, j // page], device="cuda").long(), torch.tensor(j % page, device="cuda")
        for want, cache, scale in ((k, loop.k, loop.ks), (v, loop.v, loop.vs)):
            s = scale[at][..., None]
            got = cache.float()[at, :, row] * s
            w = want.float()
            # e4m3 rounds by 2^-4 of a value or 2^-10 of the scale, a page stored again once more by the latter;
            # the products that made k and v may round one bf16 step apart in another batch
            bound = w.abs() * (2.0 ** -4 + 2.0 ** -7 * 1.1) + s * 2.0 ** -8 + 2.0 ** -9
            assert bool(((got - w).abs() <= bound).all())
