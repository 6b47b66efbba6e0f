"""Plain 64-bit forms of the serving loop's operators, one item at a time, for the tests."""
import math

import numpy as np
import torch


def plan(seq_len, accept, new, held, table, ring, head, count, P, cap):
    """ssd_kv_plan on Python lists: returns the outputs and the state after the call."""
    B, n, m = len(seq_len), len(ring), len(table[0])
    seq_len, held, ring = list(seq_len), list(held), list(ring)
    table = [list(r) for r in table]
    before = [list(r) for r in table]
    src = list(ring)
    cu, kv, slots, positions, status = [0], [], [-1] * cap, [0] * cap, 0
    demand = taken = given = total = 0
    for b in range(B):
        keep = seq_len[b] + (accept[b] + 1 if accept is not None and accept[b] >= 0 else 0)
        ok = new[b] >= 0 and seq_len[b] >= 0 and 0 <= held[b] <= m
        fresh = max(0, new[b])
        want = -(-(keep + fresh) // P)
        start, total = total, total + fresh
        if want > m or (total > cap and fresh):
            ok = False
        if not ok:
            status |= 64
            want = held[b]
        take, give = max(0, want - held[b]), max(0, held[b] - want)
        demand += take
        served = ok and (take == 0 or demand <= count)
        if ok and not served:
            status |= 32
        if served:
            for i in range(take):
                table[b][held[b] + i] = src[(head + demand - take + i) % n]
            taken += take
        for i in range(give):
            ring[(head + count + given + i) % n] = before[b][want + i]
            table[b][want + i] = -1
        given += give
        for i in range(fresh):
            if start + i >= cap:
                break
            pos = keep + i
            positions[start + i] = pos
            if served:
                slots[start + i] = table[b][pos // P] * P + pos % P
        cu.append(min(total, cap))
        kv.append(keep + fresh if served else keep)
        seq_len[b] = keep
        if served:
            held[b] = want
    return dict(cu_new=cu, kv_len=kv, slots=slots, positions=positions, seq_len=seq_len, held=held, block_table=table, ring=ring,
                ring_state=[(head + taken) % n, count - taken + given]), status


def e4m3_values():
    """The 256 values of the format."""
    out = np.empty(256)
    for c in range(256):
        s, e, f = -1.0 if c & 128 else 1.0, (c >> 3) & 15, c & 7
        out[c] = math.nan if (c & 127) == 127 else s * (2.0 ** -6 * f / 8 if e == 0 else 2.0 ** (e - 7) * (1 + f / 8))
    return out


_POS = e4m3_values()[:127]


def to_e4m3(x):
    """Nearest e4m3 value of each number, ties to even, beyond 448 the nearest finite; NaN stays NaN."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    a = np.where(np.isnan(x), 0.0, a)
    hi = np.searchsorted(_POS, a)
    lo = np.maximum(hi - 1, 0)
    hi = np.minimum(hi, 126)
    dl, dh = a - _POS[lo], _POS[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isnan(x), np.nan, np.copysign(_POS[pick], x))


def append(x, slots, values, scale, P):
    """ssd_kv_append of one of keys and values on float64 arrays: values [N, H, P, D] stands for the
    bytes; both are updated in place."""
    T, H, _ = x.shape
    rows = values.shape[0] * P
    t = 0
    while t < T:
        if not 0 <= slots[t] < rows:
            t += 1
            continue
        page, end = slots[t] // P, t + 1
        while end < T and 0 <= slots[end] < rows and slots[end] // P == page:
            end += 1
        row0 = slots[t] % P
        for h in range(H):
            y = x[t:end, h]
            a = np.abs(y[np.isfinite(y)])
            k = -100
            while a.size and a.max() > 448.0 * 2.0 ** k:
                k += 1
            need = 2.0 ** k
            was = scale[page, h] if row0 else 0.0
            had = math.isfinite(was) and was > 0
            new = max(was, need) if had else need
            if row0 and new != was:
                # the kernel's quotient and product are fp32; the tests' former scales are chosen so that both are exact
                values[page, h, :row0] = to_e4m3(values[page, h, :row0] * (was / new if had else 0.0))
            scale[page, h] = new
            for i in range(t, end):
                values[page, h, slots[i] % P] = to_e4m3(x[i, h] / new)
        t = end


def attend(q, k, v, ks, vs, table, cu, kv_len, P, sm_scale, window, max_new=1 << 30):
    """Returns (out, weight, score, largest): the outputs in 64 bits, and for the error bound, per token and
    head: sum p |v| per channel, the largest sum |q k| of a score, and the largest |v|."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    out, weight = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    score, largest = np.zeros((T, Hq, 1)), np.zeros((T, Hq, 1))
    for b in range(len(kv_len)):
        n = cu[b + 1] - cu[b]
        for i in range(min(n, max_new)):
            pos = kv_len[b] - n + i
            lo = max(0, pos + 1 - window) if window else 0
            js = [j for j in range(lo, min(pos + 1, table.shape[1] * P)) if 0 <= table[b][j // P] < k.shape[0]]
            if not js:
                continue
            js = np.array(js)
            pages, rows = table[b][js // P], js % P
            for h in range(Hq):
                g = h // G
                kk = k[pages, g, rows] * ks[pages, g][:, None]
                vv = v[pages, g, rows] * vs[pages, g][:, None]
                x = q[cu[b] + i, h]
                s = sm_scale * (kk @ x)
                p = np.exp(s - np.max(s))
                p /= p.sum()
                out[cu[b] + i, h] = p @ vv
                weight[cu[b] + i, h] = p @ np.abs(vv)
                score[cu[b] + i, h] = abs(sm_scale) * np.max(np.abs(kk) @ np.abs(x))
                largest[cu[b] + i, h] = np.max(np.abs(vv))
    return out, weight, score, largest


def attend_bound(dtype, D, out, weight, score, largest):
    """How far the kernel may be from `out`.

    Half a step of the output's type, of the value itself.  Half a step of the softmax weights'
    (2^-8 for two e4m3 digits, 2^-12 for three), of sum p |v|.  fp32 sums of D products, whose error
    2^-24 (D + 8) of the largest sum |q k| moves a weight by as much, once for the weight and once for
    their total.  2^-15 (2^-19) of the largest value for the weights' digits that end; that is 128 digits
    that end at 2^-22 (2^-26) of the largest weight near them, and less than the kernel's could add up to
    (256 at 2^-18, 2^-23) if all of a step's small weights were rounded the same way.  2^-20 of sum p |v| for
    the fp32 steps of exp, the sums over keys and the last product."""
    half, weights, floor = (2.0 ** -8, 2.0 ** -8, 2.0 ** -15) if dtype == torch.bfloat16 else \
        (2.0 ** -11, 2.0 ** -12, 2.0 ** -19)
    d = weights + 2 * (D + 8) * 2.0 ** -24 * score + 2.0 ** -20
    # the smallest fp16 step, for values below its normal range
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    return half * np.abs(out) + (1 + half) * (d * weight + floor * largest) + tiny


def sample(z, tau, k, p, mp, u):
    """One row in 64 bits: (token, prob, kept ids, margin), margin the distance of the draw, of the
    nucleus' border and of min-p's from the nearest value that would decide otherwise, over the total
    (inf where nothing is near)."""
    z = np.asarray(z, np.float64)
    V = z.shape[0]
    rank = np.lexsort((np.arange(V), -z))
    if tau == 0:
        return int(rank[0]), 1.0, rank[:1], math.inf
    keep = rank[:k] if 0 < k < V else rank

    def unit(w):
        # weights that are all one number carry one error, which cancels: the border lies between whole
        # numbers of them
        return w[0] if w.min() == w.max() else w.sum()

    w = np.exp((z[keep] - z[rank[0]]) / tau)
    margin = math.inf
    if p < 1:
        c = np.cumsum(w)
        above = c - w
        n = max(1, int(np.count_nonzero(above < p * c[-1])))
        if len(w) > 1:  # the first rank is kept whatever the border is
            margin = min(margin, float(np.min(np.abs(above - p * c[-1])[1:]) / unit(w)))
        keep, w = keep[:n], w[:n]
    if mp > 0:
        n = max(1, int(np.count_nonzero(w >= mp)))
        if len(w) > 1 and mp < 1:
            margin = min(margin, float(np.min(np.abs(w - mp)[1:])))
        keep, w = keep[:n], w[:n]
    at = np.argsort(keep)
    keep, w = keep[at], w[at]
    c = np.cumsum(w)
    i = min(int(np.count_nonzero(c <= u * c[-1])), len(keep) - 1)
    inner = c[:-1] if u * c[-1] > 0 else c
    if len(inner):
        margin = min(margin, float(np.min(np.abs(inner - u * c[-1])) / unit(w)))
    return int(keep[i]), float(w[i] / c[-1]), keep[z[keep] > -math.inf], margin
