"""Plain fp64 forms of the paged grouped-query operators, one row at a time,
and the error bounds their kernels are held to.

The attention bound, element by element.  With w the exact softmax weights,
A = sum_i w_i |v_i| and n keys:
  * each numerator is rounded once to bf16: at most 2^-8 of it, 2^-8 A in sum;
  * a score is a D-term fp32 sum (2^-23 a term, products exact) times the
    scale, so off by at most ds = (D + 4) 2^-23 |scale| max_i sum_d |q_d k_id|,
    which is a relative ds of its numerator, and of the row sum again: 2 ds A;
  * at most n additions in each of the two fp32 sums, and a rescaling (one
    exponential and one product, 2^-21 together) per 16 keys: less than
    (2 n + 64) 2^-22 A together with the constant number of joining steps;
  * the output is rounded once to bf16: 2^-8 |out|.
"""
import math

import torch

EPS_BF16 = 2.0 ** -8  # half a step, relative to the value


def rotate(x, cos_sin, rot, neox):
    """x fp64 [..., D], cos_sin fp64 [rot] of the row's position -> (out, the
    sum of the magnitudes of each output's terms)."""
    out, mag = x.clone(), x.abs()
    for i in range(rot // 2):
        a, b = (i, i + rot // 2) if neox else (2 * i, 2 * i + 1)
        c, s = cos_sin[i], cos_sin[rot // 2 + i]
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
        mag[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return out, mag


def append(qkv, Hq, Hkv, D, cos_sin, rot, neox, positions, slots, cache):
    """(q rows fp64, their bound, cache fp64, its bound): what a call leaves,
    from the tensors before it.  Rows that are not rotated have bound 0."""
    T = qkv.shape[0]
    num_pages, page = cache.shape[0], cache.shape[3]
    x = qkv.double().view(T, Hq + 2 * Hkv, D)
    q, q_tol = x[:, :Hq].clone(), torch.zeros(T, Hq, D, dtype=torch.float64)
    kv, kv_tol = cache.double().clone(), torch.zeros(cache.shape, dtype=torch.float64)
    for t in range(T):
        rows, mag = x[t, :Hq + Hkv], None
        tol = torch.zeros_like(rows)
        if rot:
            p = int(positions[t])
            if not 0 <= p < cos_sin.shape[0]:
                continue
            rows, mag = rotate(rows, cos_sin[p].double(), rot, neox)
            # two fp32 roundings of the terms, one rounding to bf16
            tol = EPS_BF16 * rows.abs() + 2.0 ** -22 * mag + 2.0 ** -134
            tol[..., rot:] = 0
        q[t], q_tol[t] = rows[:Hq], tol[:Hq]
        s = int(slots[t])
        if 0 <= s < num_pages * page:
            kv[s // page, 0, :, s % page], kv_tol[s // page, 0, :, s % page] = rows[Hq:], tol[Hq:]
            kv[s // page, 1, :, s % page] = x[t, Hq + Hkv:]
    return q, q_tol, kv, kv_tol


def scores(q, bounds, pages):
    """fp64 scores of the blocks on ``pages`` for one token and kv head: q
    [G, D], bounds [num_pages, 2, D] of that head."""
    lo, hi = bounds[pages, 0].double(), bounds[pages, 1].double()
    up, down = q.double().clamp(min=0).sum(0), q.double().clamp(max=0).sum(0)
    return (hi * up + lo * down).sum(-1)  # the same order for every block: equal blocks tie


def select(q, bounds, table, lens, page, topk, first, last, requests=None):
    T, Hq, D = q.shape
    N, Hkv = bounds.shape[:2]
    G = Hq // Hkv
    out = torch.full((T, Hkv, topk), -1, dtype=torch.int32)
    for t in range(T):
        r = t if requests is None else int(requests[t])
        length = int(lens[t])
        if not 0 <= r < table.shape[0] or length < 0:
            continue
        n = -(-min(length, table.shape[1] * page) // page)
        pages = table[r, :n].long()
        ok = (pages >= 0) & (pages < N)
        j = torch.arange(n)
        for h in range(Hkv):
            s = scores(q[t, h * G:(h + 1) * G], bounds[:, h], torch.where(ok, pages, 0))
            s = torch.where(ok & ~s.isnan(), s, -math.inf)
            keep = (j < first) | (j >= n - last)
            order = sorted(range(n), key=lambda i: (not keep[i], -s[i] if not keep[i] else 0, i))
            best = sorted(order[:topk])
            out[t, h, :len(best)] = torch.tensor(best, dtype=torch.int32)
    return out


def attend(q, k, v, scale):
    """(out, bound) fp64 [G, D] of q [G, D] against k, v [n, D]."""
    q, k, v = q.double(), k.double(), v.double()
    n, D = k.shape
    if n == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    s = q @ k.T * scale
    w = torch.softmax(s, -1)
    out = w @ v
    ds = (D + 4) * 2.0 ** -23 * abs(scale) * (q.abs() @ k.abs().T).amax(-1, keepdim=True)
    A = w @ v.abs()
    return out, A * (EPS_BF16 + 2 * ds + (2 * n + 64) * 2.0 ** -22) + EPS_BF16 * out.abs()


def _keys(cache, pages, h, lo, hi):
    """Keys lo..hi-1 (and values) of the tokens on ``pages``, kv head h."""
    page = cache.shape[3]
    at = torch.arange(lo, hi)
    ids = torch.as_tensor(pages).long()[at // page]
    ok = (ids >= 0) & (ids < cache.shape[0])
    kv = cache[ids[ok], :, h, (at % page)[ok]]
    return kv[:, 0], kv[:, 1]


def sparse_attention(q, cache, table, blocks, lens, scale, requests=None):
    T, Hq, D = q.shape
    Hkv, page = cache.shape[2], cache.shape[3]
    G = Hq // Hkv
    out, tol = torch.zeros(T, Hq, D).double(), torch.zeros(T, Hq, D).double()
    for t in range(T):
        r = t if requests is None else int(requests[t])
        if not 0 <= r < table.shape[0]:
            continue
        length = max(0, min(int(lens[t]), table.shape[1] * page))
        for h in range(Hkv):
            parts = [_keys(cache, table[r], h, b * page, min(length, b * page + page))
                     for b in blocks[t, h].tolist() if b >= 0 and b * page < length]
            k = torch.cat([p[0] for p in parts]) if parts else cache.new_zeros(0, D)
            v = torch.cat([p[1] for p in parts]) if parts else cache.new_zeros(0, D)
            g = slice(h * G, (h + 1) * G)
            out[t, g], tol[t, g] = attend(q[t, g], k, v, scale)
    return out, tol


def prefix_attention(q, cache, prefix_pages, prefix_len, table, lens, scale, requests=None):
    T, Hq, D = q.shape
    Hkv, page = cache.shape[2], cache.shape[3]
    G = Hq // Hkv
    out, tol = torch.zeros(T, Hq, D).double(), torch.zeros(T, Hq, D).double()
    for h in range(Hkv):
        pk, pv = _keys(cache, prefix_pages, h, 0, prefix_len)
        for t in range(T):
            r = t if requests is None else int(requests[t])
            k, v = pk, pv
            if 0 <= r < table.shape[0]:
                length = max(0, min(int(lens[t]), table.shape[1] * page))
                sk, sv = _keys(cache, table[r], h, 0, length)
                k, v = torch.cat([pk, sk]), torch.cat([pv, sv])
            g = slice(h * G, (h + 1) * G)
            out[t, g], tol[t, g] = attend(q[t, g], k, v, scale)
    return out, tol


def check(got, want, tol, what=""):
    """Every element of bf16 ``got`` within ``tol`` of fp64 ``want``."""
    g = got.detach().cpu().double()
    bad = ~((g - want).abs() <= tol)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} values outside the bound, first at "
        f"{[int(i) for i in bad.nonzero()[0]]}: {float(g[bad][0])} for {float(want[bad][0])} "
        f"+- {float(tol[bad][0])}")
