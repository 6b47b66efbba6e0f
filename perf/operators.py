"""The serving-side operators around a verification round: their cases, plain forms and 64-bit values.

Four operators of one loop.  ``ssd_kv_plan`` commits the accepted lengths of the last round and gives
the next tokens their cache pages and slots.  ``ssd_kv_append`` stores their keys and values as e4m3
with one scale for each (page, head).  ``ssd_kv_attend`` is the attention of those tokens over the
cache.  ``ssd_sample`` draws tokens under temperature, top-k, top-p and min-p.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
SCALE_EXP_MIN = -100       # smallest power-of-two scale that a page is given
DROPPED = -1e5             # what the filtered logits hold for a dropped token


def listed():
    return [
        # One round of a full batch: K+1 = 5 tokens each, the last round's accepted lengths committed.
        dict(name="plan_round", op="plan", B=256, new_min=5, new_max=5, kv_max=8192, page=64, accept=True),
        # Prompts join a running batch: many pages taken at once, small pages, accepted lengths on the host.
        dict(name="plan_prompts", op="plan", B=48, new_min=1, new_max=2700, kv_max=12000, page=16, accept=False),
        # One decoded token of one sequence, the smaller head and page: latency.
        dict(name="append_one", op="append", B=1, new=1, start=517, H=4, D=64, page=16, dtype="bf16"),
        # The K+1 tokens of every sequence of a full batch, landing in partly filled pages.
        dict(name="append_round", op="append", B=256, new=5, start=301, H=8, D=128, page=64, dtype="bf16"),
        # Prompts of odd length, fp16, a smaller page.
        dict(name="append_prompts", op="append", B=12, new=1365, start=0, H=8, D=128, page=32, dtype="fp16"),
        # One sequence decodes one token: few rows, a short cache, latency.
        dict(name="attend_one", op="attend", B=1, q_min=1, q_max=1, kv_min=1037, kv_max=1037, Hq=32, Hkv=8, D=128,
             page=64, window=0, dtype="bf16"),
        # Verification of K = 4 drafts for a batch of ragged lengths: the ordinary call.
        dict(name="attend_round", op="attend", B=64, q_min=5, q_max=5, kv_min=3, kv_max=8191, Hq=32, Hkv=8, D=128,
             page=64, window=0, dtype="bf16"),
        # Few sequences over a long cache, K = 8: the cache read is everything.
        dict(name="attend_long", op="attend", B=4, q_min=9, q_max=9, kv_min=90001, kv_max=131072, Hq=32, Hkv=8, D=128,
             page=128, window=0, dtype="bf16"),
        # Prompt pieces with a sliding window, fp16, the smaller head and page, ragged lengths.
        dict(name="attend_prompts", op="attend", B=6, q_min=1, q_max=1021, kv_min=700, kv_max=5003, Hq=16, Hkv=4, D=64,
             page=16, window=2048, dtype="fp16"),
        # One row of one sequence: latency.
        dict(name="sample_one", op="sample", rows=1, V=32000, dtype="f32", mode="mixed", filtered=False),
        # A full batch, every truncation in use, some rows greedy, some plain.
        dict(name="sample_round", op="sample", rows=256, V=128256, dtype="bf16", mode="mixed", filtered=False),
        # The target's rows made ready for a lossless verification of truncated sampling: filtered logits written.
        dict(name="sample_filter", op="sample", rows=96, V=152064, dtype="f32", mode="nucleus", filtered=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "sample", "sample"])
    if op == "plan":
        lo = rng.choice([0, 1, 3])
        return dict(op=op, B=_log(rng, 1, 400), new_min=lo, new_max=lo + _log(rng, 1, 150), kv_max=_log(rng, 20, 12000),
                    page=rng.choice([16, 32, 64, 128]), accept=rng.random() < 0.5)
    if op == "append":
        B = _log(rng, 1, 256)
        return dict(op=op, B=B, new=_log(rng, 1, max(2, 12000 // B)), start=rng.choice([0, _log(rng, 1, 700)]),
                    H=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
                    dtype=rng.choice(["bf16", "fp16"]))
    if op == "attend":
        hkv = rng.choice([1, 2, 4, 8])
        q = rng.choice([1, _log(rng, 2, 17), _log(rng, 2, 400)])
        B = _log(rng, 1, 64 if q < 32 else 8)
        Hq, D = hkv * rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        kv = _log(rng, 1, min(60000, 400000 // B))
        kv = max(1, min(kv, 6 * 10 ** 10 // (4 * D * Hq * q * B)))
        return dict(op=op, B=B, q_min=rng.choice([1, q]), q_max=q, kv_min=rng.choice([0, kv // 3, kv]), kv_max=kv,
                    Hq=Hq, Hkv=hkv, D=D, page=rng.choice([16, 32, 64, 128]),
                    window=rng.choice([0, 0, _log(rng, 1, 4096)]), dtype=rng.choice(["bf16", "fp16"]))
    V = _log(rng, 50, 152064)
    return dict(op="sample", rows=_log(rng, 1, min(256, 256 * 128256 // V)), V=V, dtype=rng.choice(["bf16", "f32"]),
                mode=rng.choice(["mixed", "nucleus", "topk", "minp", "plain"]), filtered=rng.random() < 0.25)


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------

def _spread(lo, hi, n):
    """n whole numbers from lo to hi at even steps."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _torch_dtype(name):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}[name]


def _perm(n, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(n, generator=g)


def _int(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


def _plan_numbers(case):
    """Lengths by rank (the seed only decides which request has which): committed length, new tokens."""
    B = case["B"]
    lens = _spread(0, case["kv_max"], B)
    new = _spread(case["new_min"], case["new_max"], B)
    return lens, [new[(i * 7 + 3) % B] for i in range(B)]


def _prepare_plan(case, seed):
    B, P = case["B"], case["page"]
    lens, new = _plan_numbers(case)
    order = _perm(B, seed).tolist()
    lens, new = [lens[i] for i in order], [new[i] for i in order]
    g = torch.Generator().manual_seed(seed + 1)
    accept = torch.randint(-1, 5, (B,), generator=g).tolist()
    # the pages held: those of the committed tokens and of the five tokens of the round before
    held = [-(-(n + 5) // P) if n else 0 for n in lens]
    max_blocks = -(-(case["kv_max"] + case["new_max"] + 16) // P)
    num_pages = sum(held) + sum(-(-m // P) + 1 for m in new) + 7
    pages = _perm(num_pages, seed + 2).tolist()
    table = torch.full((B, max_blocks), -1, dtype=torch.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = torch.tensor(pages[at:at + h], dtype=torch.int32)
        at += h
    free = num_pages - at
    head = (seed * 13 + 5) % num_pages
    ring = torch.zeros(num_pages, dtype=torch.int32)
    ring[(head + torch.arange(free)) % num_pages] = torch.tensor(pages[at:], dtype=torch.int32)
    parts = [torch.tensor(lens), torch.tensor(held), torch.tensor([head, free]), ring, table.reshape(-1)]
    saved = torch.cat([p.to(torch.int32) for p in parts]).to(DEV)
    state = dict(saved=saved, buffer=saved.clone(), new=_int(new), accept=_int(accept) if case["accept"] else None,
                 cap=sum(new) + 3, page=P, B=B, max_blocks=max_blocks, num_pages=num_pages)
    return state


def _plan_views(state):
    """The loop's state is one buffer: lengths, pages held, ring position, ring, block table."""
    B, n, m = state["B"], state["num_pages"], state["max_blocks"]
    buf = state["buffer"]
    return dict(seq_len=buf[:B], held=buf[B:2 * B], ring_state=buf[2 * B:2 * B + 2], ring=buf[2 * B + 2:2 * B + 2 + n],
                block_table=buf[2 * B + 2 + n:].view(B, m))


def _append_sizes(case):
    B, P = case["B"], case["page"]
    blocks = -(-(case["start"] + case["new"] + B) // P)
    return B * blocks + 3, blocks


def _quantise_pages(x):
    """Pages [N, H, P, D] of 32-bit values -> (e4m3 pages, scale [N, H]), the scale any 32-bit number."""
    amax = x.abs().amax(dim=(2, 3)).clamp_min(1e-20)
    scale = amax / E4M3_MAX
    return (x / scale[:, :, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _random_cache(n, H, P, D, gen, spread):
    """Pages of keys or values: some channels and some pages larger than the rest, as real ones are."""
    out = torch.empty((n, H, P, D), dtype=torch.float8_e4m3fn, device=DEV)
    scale = torch.empty((n, H), dtype=torch.float32, device=DEV)
    channel = torch.exp(spread * torch.randn((1, H, 1, D), generator=gen, device=DEV))
    for lo in range(0, n, 4096):
        m = min(4096, n - lo)
        x = torch.randn((m, H, P, D), generator=gen, device=DEV) * channel
        x *= torch.exp(0.4 * torch.randn((m, H, 1, 1), generator=gen, device=DEV))
        out[lo:lo + m], scale[lo:lo + m] = _quantise_pages(x)
    return out, scale


def _prepare_append(case, seed):
    B, P, H, D, new = (case[k] for k in ("B", "page", "H", "D", "new"))
    n, blocks = _append_sizes(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = _torch_dtype(case["dtype"])
    k_cache, k_scale = _random_cache(n, H, P, D, gen, 0.5)
    v_cache, v_scale = _random_cache(n, H, P, D, gen, 0.2)
    k_scale = torch.exp2(torch.ceil(torch.log2(k_scale)))
    v_scale = torch.exp2(torch.ceil(torch.log2(v_scale)))
    table = _perm(n, seed).to(torch.int64)[:B * blocks].view(B, blocks)
    # sequence b starts b tokens further, so that every offset in a page is met (none where the prompts start)
    start = [case["start"] + (b if case["start"] else 0) for b in range(B)]
    pos = torch.tensor(start)[:, None] + torch.arange(new)[None, :]
    slots = (torch.gather(table, 1, pos // P) * P + pos % P).reshape(-1)
    # keys and values lie in one projection's output: rows of (k, v), so their token stride is 2 H D
    kv = torch.randn((B * new, 2, H, D), generator=gen, device=DEV)
    kv *= torch.exp(0.7 * torch.randn((B * new, 2, H, 1), generator=gen, device=DEV))
    kv = kv.to(dt)
    return dict(k=kv[:, 0], v=kv[:, 1], slots=_int(slots), k_cache=k_cache, v_cache=v_cache, k_scale=k_scale,
                v_scale=v_scale)


def _attend_numbers(case):
    """By sequence rank: (cached length with the new tokens, new tokens)."""
    B = case["B"]
    kv = _spread(case["kv_min"], case["kv_max"], B)
    q = _spread(case["q_min"], case["q_max"], B)
    return [(kv[i], q[(i * 5 + 2) % B]) for i in range(B)]


def _prepare_attend(case, seed):
    B, P, Hq, Hkv, D = (case[k] for k in ("B", "page", "Hq", "Hkv", "D"))
    gen = torch.Generator(device=DEV).manual_seed(seed)
    pairs = _attend_numbers(case)
    pairs = [pairs[i] for i in _perm(B, seed).tolist()]
    kv_len, q_len = [p[0] for p in pairs], [p[1] for p in pairs]
    blocks = [-(-n // P) for n in kv_len]
    n, max_blocks = sum(blocks) + 2, max(1, max(blocks))
    k_cache, k_scale = _random_cache(n, Hkv, P, D, gen, 0.6)
    v_cache, v_scale = _random_cache(n, Hkv, P, D, gen, 0.2)
    pages = _perm(n, seed + 1).to(torch.int32)
    table = torch.full((B, max_blocks), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(blocks):
        table[b, :m] = pages[at:at + m]
        at += m
    T = sum(q_len)
    q = torch.randn((T, Hq, D), generator=gen, device=DEV) * 1.3
    return dict(q=q.to(_torch_dtype(case["dtype"])), k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale,
                block_table=table.to(DEV), kv_len=_int(kv_len),
                cu_new=torch.tensor([0] + q_len).cumsum(0).to(torch.int32).to(DEV), max_new=max(q_len),
                sm_scale=1.0 / math.sqrt(D), window=case["window"])


def _prepare_sample(case, seed):
    R, V = case["rows"], case["V"]
    gen = torch.Generator(device=DEV).manual_seed(seed)
    bias = -1.1 * torch.log1p(torch.arange(V, dtype=torch.float64)).to(torch.float32).to(DEV)
    logits = (torch.randn((R, V), generator=gen, device=DEV) * 3.0 + bias).to(_torch_dtype(case["dtype"]))
    i = torch.arange(R)
    mode = case["mode"]
    temperature = torch.tensor([1.0, 0.7, 0.6, 1.0, 0.0, 1.3, 0.9, 0.8])[i % 8] if mode == "mixed" else 0.6 + 0.1 * (i % 7)
    top_k = torch.tensor([0, 50, 0, 20, 0, 0, 1000, 1])[i % 8] if mode == "mixed" else \
        (torch.tensor([1, 8, 40, 257, 5000])[i % 5] if mode == "topk" else torch.zeros(R))
    top_p = torch.tensor([1.0, 0.9, 0.95, 1.0, 1.0, 1.0, 0.8, 1.0])[i % 8] if mode == "mixed" else \
        (torch.tensor([0.9, 0.95, 0.5, 0.99])[i % 4] if mode == "nucleus" else torch.ones(R))
    min_p = torch.tensor([0.0, 0.0, 0.0, 0.05, 0.0, 0.02, 0.0, 0.0])[i % 8] if mode == "mixed" else \
        (torch.tensor([0.1, 0.01, 0.0005])[i % 3] if mode == "minp" else torch.zeros(R))
    f32 = dict(dtype=torch.float32, device=DEV)
    return dict(logits=logits, temperature=temperature.to(**f32), top_k=_int(top_k), top_p=top_p.to(**f32),
                min_p=min_p.to(**f32), uniforms=torch.rand(R, generator=gen, device=DEV), filtered=case["filtered"])


def prepare(case, seed):
    make = dict(plan=_prepare_plan, append=_prepare_append, attend=_prepare_attend, sample=_prepare_sample)[case["op"]]
    return dict(make(case, seed), op=case["op"])


# ---------------------------------------------------------------------------
# Plain forms.
# ---------------------------------------------------------------------------

def _plain_plan(s):
    v = _plan_views(s)
    B, P, n, m, cap = s["B"], s["page"], s["num_pages"], s["max_blocks"], s["cap"]
    L = torch.int64
    keep, held, new = v["seq_len"].to(L), v["held"].to(L), s["new"].to(L)
    if s["accept"] is not None:
        a = s["accept"].to(L)
        keep = keep + torch.where(a >= 0, a + 1, 0)
    head, free = v["ring_state"][0].to(L), v["ring_state"][1].to(L)
    ring, table = v["ring"].to(L), v["block_table"].to(L)
    want = (keep + new + P - 1) // P
    take, give = (want - held).clamp_min(0), (held - want).clamp_min(0)
    demand = take.cumsum(0)
    served = (take == 0) | (demand <= free)
    granted = torch.where(served, take, 0)
    j = torch.arange(m, device=keep.device)[None, :]
    mine = served[:, None] & (j >= held[:, None]) & (j < want[:, None])
    src = (head + (demand - take)[:, None] + j - held[:, None]) % n
    back = (j >= want[:, None]) & (j < held[:, None])
    dst = (head + free + (give.cumsum(0) - give)[:, None] + j - want[:, None]) % n
    ring = torch.cat([ring, ring[:1]]).scatter(0, torch.where(back, dst, n).reshape(-1), table.reshape(-1))[:n]
    table = torch.where(mine, v["ring"].to(L)[torch.where(mine, src, 0)], table)
    table = torch.where(back, -1, table)
    held = torch.where(served, want, held)
    kv_len = torch.where(served, keep + new, keep)
    cu = torch.cat([torch.zeros(1, dtype=L, device=keep.device), new.cumsum(0)])
    t = torch.arange(cap, device=keep.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    real = (t < cu[B])
    b = b.clamp(0, B - 1)
    pos = keep[b] + t - cu[b]
    ok = real & served[b]
    page = table[b, torch.where(ok, pos // P, 0)]
    slots = torch.where(ok, page * P + pos % P, -1)
    count = free - granted.sum() + give.sum()
    head = (head + granted.sum()) % n
    i32 = torch.int32
    v["seq_len"].copy_(keep), v["held"].copy_(held), v["ring"].copy_(ring), v["block_table"].copy_(table)
    v["ring_state"].copy_(torch.stack([head, count]))
    return dict(cu_new=cu.to(i32), kv_len=kv_len.to(i32), slots=slots.to(i32), positions=torch.where(real, pos, 0).to(i32),
                **v)


def _e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _plain_append_one(x, slots, cache, scale):
    P, N = cache.shape[2], cache.shape[0]
    T = slots.shape[0]
    x = x.to(torch.float32)
    page, off = slots // P, slots % P
    lead = torch.ones(T, dtype=torch.bool, device=x.device)
    lead[1:] = page[1:] != page[:-1]
    largest = x.abs().amax(dim=2)
    amax = torch.zeros((N, x.shape[1]), device=x.device).scatter_reduce(0, page[:, None].expand_as(largest), largest, "amax")
    mant, exp = torch.frexp(amax)
    exp = torch.where(mant <= 0.875, exp - 9, exp - 8).clamp_min(SCALE_EXP_MIN)
    need = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), exp), 2.0 ** SCALE_EXP_MIN)
    # the first new token of each touched page says how many tokens the page held
    before = torch.full((N + 1,), -1, dtype=torch.int64, device=x.device)
    before[torch.where(lead, page, N)] = off
    before = before[:N, None]
    new = torch.where(before > 0, torch.maximum(scale, need), torch.where(before == 0, need, scale))
    ratio = torch.where(before > 0, scale / new, 1.0)
    row = torch.arange(P, device=x.device)[None, None, :]
    old = cache.to(torch.float32)
    again = _e4m3(old * ratio[:, :, None, None])
    change = (before[:, :, None] > row) & (ratio[:, :, None] != 1.0)
    out = torch.where(change[..., None], again.to(torch.float32), old)
    y = _e4m3(x / new[page][:, :, None]).to(torch.float32)
    out[page[:, None], torch.arange(x.shape[1], device=x.device)[None, :], off[:, None]] = y
    cache.copy_(out.to(torch.float8_e4m3fn))
    scale.copy_(new)


def _plain_append(s):
    slots = s["slots"].to(torch.int64)
    _plain_append_one(s["k"], slots, s["k_cache"], s["k_scale"])
    _plain_append_one(s["v"], slots, s["v_cache"], s["v_scale"])
    return {k: s[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _plain_attend(s):
    q, table, cu, kv_len = s["q"], s["block_table"].clamp_min(0).to(torch.int64), s["cu_new"].to(torch.int64), s["kv_len"]
    T, Hq, D = q.shape
    B, m = table.shape
    Hkv, P = s["k_cache"].shape[1:3]
    G, Q, L = Hq // Hkv, s["max_new"], m * P

    def pages(cache, scale):
        x = cache.view(torch.uint8)[table].view(cache.dtype).to(torch.float32) * scale[table][..., None, None]       # [B, m, Hkv, P, D]
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D)

    i = torch.arange(Q, device=q.device)
    n = cu[1:] - cu[:-1]
    there = i[None, :] < n[:, None]
    t = torch.where(there, cu[:-1, None] + i, T)                                   # [B, Q]; T: no token
    rows = torch.cat([q, q[:1]])[t].to(torch.float32).view(B, Q, Hkv, G, D)
    rows = rows.permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Q, D)
    score = torch.matmul(rows, pages(s["k_cache"], s["k_scale"]).transpose(2, 3)) * s["sm_scale"]
    pos = (kv_len - n)[:, None] + i                                                # the token's place in its sequence
    j = torch.arange(L, device=q.device)
    seen = (j[None, None, :] <= pos[:, :, None]) & (j[None, None, :] < kv_len[:, None, None])
    if s["window"]:
        seen &= j[None, None, :] > pos[:, :, None] - s["window"]
    seen = seen[:, None, None]
    score = score.view(B, Hkv, G, Q, L).masked_fill(~seen, -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    e = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(dim=-1, keepdim=True)
    e = (e / torch.where(total == 0, 1.0, total)).view(B, Hkv, G * Q, L)
    o = torch.matmul(e, pages(s["v_cache"], s["v_scale"])).view(B, Hkv, G, Q, D)
    o = o.permute(0, 3, 1, 2, 4).reshape(B * Q, Hq, D)
    out = torch.zeros((T + 1, Hq, D), dtype=torch.float32, device=q.device)
    out[t.reshape(-1)] = o
    return out[:T].to(q.dtype)


def _plain_sample(s):
    z = s["logits"].to(torch.float64)
    R, V = z.shape
    tau = s["temperature"].to(torch.float64)[:, None]
    greedy = tau == 0
    best, order = torch.sort(z, dim=1, descending=True, stable=True)
    e = torch.exp((best - best[:, :1]) / torch.where(greedy, 1.0, tau))
    rank = torch.arange(V, device=z.device)[None, :]
    k = s["top_k"].to(torch.int64)[:, None]
    keep = (k <= 0) | (rank < k)
    e = torch.where(keep, e, 0.0)
    cum = e.cumsum(dim=1)
    top_p = s["top_p"].to(torch.float64)[:, None]
    keep = keep & ((top_p >= 1) | (cum - e < top_p * cum[:, -1:]))
    keep = keep & (e >= s["min_p"].to(torch.float64)[:, None])      # e of the most likely token is 1
    keep = (keep & ~greedy) | (rank == 0)
    e = torch.where(keep, e, 0.0)
    w = torch.zeros_like(z).scatter(1, order, e)
    kept = torch.zeros((R, V), dtype=torch.bool, device=z.device).scatter(1, order, keep)
    cum = w.cumsum(dim=1)
    total = cum[:, -1:]
    over = (cum > s["uniforms"].to(torch.float64)[:, None] * total) & kept
    token = torch.argmax(over.to(torch.uint8), dim=1)
    prob = (w.gather(1, token[:, None]) / total)[:, 0]
    out = dict(tokens=token.to(torch.int32), prob=prob.to(torch.float32))
    if s["filtered"]:
        out["filtered"] = torch.where(kept, s["logits"], torch.tensor(DROPPED, dtype=s["logits"].dtype, device=z.device))
    return out


# ---------------------------------------------------------------------------
# The framework's operators.
# ---------------------------------------------------------------------------

def _own_plan(s):
    import speculative_decoding_verification_ssd_gb300 as ssd
    v = _plan_views(s)
    out = ssd.ssd_kv_plan(v["seq_len"], s["new"], v["held"], v["block_table"], v["ring"], v["ring_state"], s["page"], s["cap"],
                          accept_len=s["accept"])
    return dict(out, **v)


def _own_append(s):
    import speculative_decoding_verification_ssd_gb300 as ssd
    ssd.ssd_kv_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    return {k: s[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _own_attend(s):
    import speculative_decoding_verification_ssd_gb300 as ssd
    if "workspace" not in s:  # a serving loop keeps one for its stream
        s["workspace"] = ssd.kv_workspace(s["q"].device)
    return ssd.ssd_kv_attend(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"], s["cu_new"],
                             s["kv_len"], s["max_new"], s["sm_scale"], window=s["window"], workspace=s["workspace"])


def _own_sample(s):
    import speculative_decoding_verification_ssd_gb300 as ssd
    return ssd.ssd_sample(s["logits"], s["temperature"], s["uniforms"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                          filtered=s["filtered"])


def run(state):
    op = state["op"]
    if op == "plan":
        state["buffer"].copy_(state["saved"])      # the call moves the loop's state on: each pass starts from the same
        return _own_plan(state) if own else _plain_plan(state)
    if op == "append":
        return _own_append(state) if own else _plain_append(state)
    if op == "attend":
        return _own_attend(state) if own else _plain_attend(state)
    return _own_sample(state) if own else _plain_sample(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "plan":
        lens, new = _plan_numbers(case)
        P = case["page"]
        pages = sum(-(-(a + n) // P) - min(-(-(a + n) // P), -(-(a + 5) // P) if a else 0) for a, n in zip(lens, new))
        return {"bytes": 4 * (case["B"] * 7 + 2 * pages + 2 * sum(new)), "flops": case["B"] + sum(new)}
    if op == "append":
        B, new, H, D = (case[k] for k in ("B", "new", "H", "D"))
        return {"bytes": 2 * B * new * H * D * 3 + 4 * B * new, "flops": 4 * B * new * H * D}
    if op == "attend":
        Hq, Hkv, D, W = (case[k] for k in ("Hq", "Hkv", "D", "window"))
        b = f = 0
        for kv, q in _attend_numbers(case):
            lo = [max(0, kv - q + i + 1 - (W or kv)) if kv - q + i >= 0 else 0 for i in range(q)]
            seen = [max(0, min(kv, kv - q + i + 1) - lo[i]) for i in range(q)]
            used = kv - min([lo[i] for i in range(q) if seen[i]], default=kv)
            b += 2 * used * Hkv * D + 4 * q * Hq * D + 4 * (-(-used // case["page"])) * (1 + 2 * Hkv)
            f += 4 * Hq * D * sum(seen)
        return {"bytes": b, "flops": f}
    s = 4 if case["dtype"] == "f32" else 2
    n = case["rows"] * case["V"]
    return {"bytes": n * s * (2 if case["filtered"] else 1) + case["rows"] * 28, "flops": 4 * n}


# ---------------------------------------------------------------------------
# The same from the definitions in 64 bits.
# ---------------------------------------------------------------------------

def _exact_append(s):
    P = s["k_cache"].shape[2]
    slots = s["slots"].tolist()
    runs, at = [], 0
    while at < len(slots):
        end = at + 1
        while end < len(slots) and slots[end] // P == slots[at] // P:
            end += 1
        runs.append((at, end))
        at = end
    if len(runs) > 3000:
        return None

    def grid(x):
        """The nearest e4m3 value (ties to even), in 64 bits."""
        e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -30)))
        e = torch.where(torch.exp2(e) > x.abs(), e - 1, e).clamp_min(-6)
        step = torch.exp2(e - 3)
        return torch.round(x / step).mul(step).clamp(-E4M3_MAX, E4M3_MAX)

    out = {}
    for name in ("k", "v"):
        values, scale = s[name + "_cache"].to(torch.float64), s[name + "_scale"].to(torch.float64).clone()
        x = s[name].to(torch.float64)
        for a, b in runs:
            page, off = slots[a] // P, slots[a] % P
            top = x[a:b].abs().amax(dim=(0, 2)).clamp_min(E4M3_MAX * 2.0 ** SCALE_EXP_MIN)
            k = torch.ceil(torch.log2(top / E4M3_MAX))
            k = torch.where(torch.exp2(k - 1) * E4M3_MAX >= top, k - 1, k)
            fresh = torch.exp2(torch.where(torch.exp2(k) * E4M3_MAX < top, k + 1, k))
            if off:
                fresh = torch.maximum(fresh, scale[page])
                values[page, :, :off] = grid(values[page, :, :off] * (scale[page] / fresh)[:, None, None])
            scale[page] = fresh
            values[page, :, off:off + b - a] = grid(x[a:b].transpose(0, 1) / fresh[:, None, None])
        out[name + "_cache"], out[name + "_scale"] = values, scale
    return out


def _exact_attend(s):
    wide = lambda x: x.to(torch.float64)  # noqa: E731
    q = s["q"].to(torch.float64)
    T, Hq, D = q.shape
    Hkv, P = s["k_cache"].shape[1:3]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=q.device)
    cu, kv = s["cu_new"].tolist(), s["kv_len"].tolist()
    for b in range(len(kv)):
        n = cu[b + 1] - cu[b]
        ids = s["block_table"][b, :-(-kv[b] // P)].to(torch.int64)
        if n == 0 or kv[b] == 0:
            continue
        for h in range(Hkv):
            G = Hq // Hkv
            K = (wide(s["k_cache"][:, h])[ids] * s["k_scale"][ids, h].to(torch.float64)[:, None, None]).view(-1, D)[:kv[b]]
            V = (wide(s["v_cache"][:, h])[ids] * s["v_scale"][ids, h].to(torch.float64)[:, None, None]).view(-1, D)[:kv[b]]
            x = q[cu[b]:cu[b + 1], h * G:(h + 1) * G]
            score = torch.einsum("qgd,ld->qgl", x, K) * s["sm_scale"]
            at = torch.arange(kv[b] - n, kv[b], device=q.device)[:, None]
            j = torch.arange(kv[b], device=q.device)[None, :]
            hide = j > at
            if s["window"]:
                hide |= j <= at - s["window"]
            score = score.masked_fill(hide[:, None, :], -math.inf)
            p = torch.nan_to_num(torch.softmax(score, dim=-1), nan=0.0)
            out[cu[b]:cu[b + 1], h * G:(h + 1) * G] = torch.einsum("qgl,ld->qgd", p, V)
    return out


def _exact_sample(s):
    R = s["logits"].shape[0]
    tokens, probs, kept = [], [], []
    for r in range(R):
        z = s["logits"][r].to(torch.float64)
        V = z.shape[0]
        tau, p, mp, u = (float(s[k][r]) for k in ("temperature", "top_p", "min_p", "uniforms"))
        k = int(s["top_k"][r])
        rank = torch.argsort(-z, stable=True)
        if tau == 0:
            keep = rank[:1]
            w = torch.ones(1, dtype=torch.float64, device=z.device)
        else:
            keep = rank[:k] if 0 < k < V else rank
            w = torch.exp((z[keep] - z[rank[0]]) / tau)
            if p < 1:
                above = torch.cat([torch.zeros(1, dtype=torch.float64, device=z.device), w.cumsum(0)[:-1]])
                count = max(1, int((above < p * w.sum()).sum()))
                keep, w = keep[:count], w[:count]
            count = max(1, int((w >= mp).sum()))
            keep, w = keep[:count], w[:count]
        by_id = torch.argsort(keep)
        keep, w = keep[by_id], w[by_id]
        c = w.cumsum(0)
        at = min(int((c <= u * c[-1]).sum()), keep.shape[0] - 1)
        tokens.append(keep[at])
        probs.append(w[at] / c[-1])
        if s["filtered"]:
            row = torch.full((V,), float(torch.tensor(DROPPED, dtype=s["logits"].dtype)), dtype=torch.float64, device=z.device)
            row[keep] = z[keep]
            kept.append(row)
    out = dict(tokens=torch.stack(tokens).to(torch.int32), prob=torch.stack(probs))
    if kept:
        out["filtered"] = torch.stack(kept)
    return out


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    return dict(append=_exact_append, attend=_exact_attend, sample=_exact_sample)[case["op"]](s)
