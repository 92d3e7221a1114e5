"""Cases of the paged grouped-query operators: appending keys and values with
the rotary embedding applied, the per-page key bounds, the selection of cache
blocks by those bounds, attention over the selected blocks, and attention of a
batch that shares a long prefix.

``run`` computes each operator either in plain torch operations (``own`` is
false) or through this repository's package (``own`` is true), on the same
inputs.  The cache is bf16 [pages, 2, kv heads, page size, head dim]: keys,
then values, of each page.
"""
import math

import torch

own = False

DEV = "cuda"
THETA = 1e6


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _append(name, T, Hq, Hkv, D, rot, neox, max_pos, page):
    return dict(name=name, op="append", T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rot, neox=neox,
                max_pos=max_pos, page=page)


def _bounds(name, n, Hkv, D, page, pages):
    return dict(name=name, op="bounds", n=n, Hkv=Hkv, D=D, page=page, pages=pages)


def _select(name, B, Hq, Hkv, D, page, length, topk):
    return dict(name=name, op="select", B=B, Hq=Hq, Hkv=Hkv, D=D, page=page, length=length,
                topk=topk)


def _sparse(name, B, Hq, Hkv, D, page, length, topk):
    return dict(name=name, op="sparse", B=B, Hq=Hq, Hkv=Hkv, D=D, page=page, length=length,
                topk=topk)


def _prefix(name, B, qlen, Hq, Hkv, D, page, prefix, suffix):
    return dict(name=name, op="prefix", B=B, qlen=qlen, Hq=Hq, Hkv=Hkv, D=D, page=page,
                prefix=prefix, suffix=suffix)


def listed():
    return [
        # one decode step of a small batch: 17 new tokens, latency counts
        _append("append_T17", 17, 16, 8, 128, 128, True, 4096, 64),
        # a prompt chunk whose rotation covers a quarter of each head, in adjacent pairs
        _append("append_T4097_partial", 4097, 16, 2, 64, 16, False, 131072, 16),
        # a large prompt batch
        _append("append_T32768", 32768, 32, 8, 128, 128, True, 131072, 64),
        # a decode step refreshes the last page of each of 64 sequences
        _bounds("bounds_64", 64, 8, 128, 64, 1024),
        # every page of a prompt's cache is summarised once
        _bounds("bounds_8192", 8192, 8, 128, 64, 8192),
        # one long conversation picks its blocks
        _select("select_B1", 1, 32, 8, 128, 64, 100003, 32),
        # a decode batch of long conversations
        _select("select_B64", 64, 32, 8, 128, 64, 65536, 32),
        # one sequence attends to the blocks it picked
        _sparse("sparse_B1", 1, 32, 8, 128, 64, 32768, 32),
        # a decode batch does
        _sparse("sparse_B64", 64, 32, 8, 128, 64, 32768, 64),
        # a few answers to one system prompt
        _prefix("prefix_B4_2048", 4, 1, 32, 8, 128, 64, 2048, 300),
        # a batch of questions on one document, three draft tokens each, 64-dim heads
        _prefix("prefix_B33_q3_D64", 33, 3, 16, 2, 64, 16, 8209, 700),
        # many samples of one long prompt
        _prefix("prefix_B256_32768", 256, 1, 64, 8, 128, 64, 32768, 512),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    Hkv = rng.choice([1, 2, 3, 4, 8])
    return Hkv * rng.choice([1, 2, 4, 5, 7, 8]), Hkv


def draw(rng):
    op = rng.choice(["append", "bounds", "select", "sparse", "prefix"])
    Hq, Hkv = _heads(rng)
    D = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 64, 128])
    if op == "append":
        rot = rng.choice([D, D, D // 2, D // 4])
        T = _log(rng, 1, max(1, min(32768, 32768 * 48 * 128 // ((Hq + 2 * Hkv) * D))))
        c = _append("", T, Hq, Hkv, D, rot, rng.random() < 0.6, rng.choice([8192, 131072]), page)
    elif op == "bounds":
        n = _log(rng, 1, min(16384, 8192 * 8 * 64 * 128 // (Hkv * D * page)))
        c = _bounds("", n, Hkv, D, page, n + rng.randrange(0, 256))
    elif op == "select":
        B = _log(rng, 1, 64)
        top = min(131072, 8192 * page, 64 * 65536 * 8 * 128 * page // (64 * B * Hkv * D))
        c = _select("", B, Hq, Hkv, D, page, _log(rng, 1, top), _log(rng, 1, 64))
    elif op == "sparse":
        B = _log(rng, 1, 64)
        length = _log(rng, 1, min(65536, 64 * 32768 * 8 * 128 // (B * Hkv * D)))
        most = max(1, min(128, 64 * 64 * 64 * 8 * 128 // (B * Hkv * D * page)))
        c = _sparse("", B, Hq, Hkv, D, page, length, _log(rng, 1, most))
    else:
        qlen = rng.choice([1, 1, 1, 2, 4])
        B = _log(rng, 1, 256 // qlen)
        most = min(65536, 256 * 64 * 32768 * 128 // (B * qlen * Hq * D))
        c = _prefix("", B, qlen, Hq, Hkv, D, page, _log(rng, 1, most), _log(rng, 1, 512))
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(0.0, std, generator=g)


def _table(max_pos, rot):
    f = THETA ** (-torch.arange(rot // 2, dtype=torch.float64, device=DEV) * 2.0 / rot)
    a = torch.arange(max_pos, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _ints(g, lo, hi, *shape):
    """Whole numbers lo..hi, both included, as int32."""
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV, dtype=torch.int32)


def _pages(g, n, total):
    return torch.randperm(total, generator=g, device=DEV)[:n]


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(c)
    Hkv, D, page = c["Hkv"], c["D"], c["page"]
    if c["op"] == "append":
        T, Hq = c["T"], c["Hq"]
        pages = -(-T // page) + 8
        s["qkv"] = _normal(g, T, (Hq + 2 * Hkv) * D)
        s["positions"] = torch.randint(0, c["max_pos"], (T,), generator=g, device=DEV)
        s["cos_sin"] = _table(c["max_pos"], c["rot"])
        s["slots"] = _pages(g, T, pages * page)
        if T > 8:
            s["slots"][T // 3] = -1  # a padding token
        s["kv"] = _normal(g, pages, 2, Hkv, page, D)
        s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
        return s
    if c["op"] == "bounds":
        s["kv"] = _normal(g, c["pages"], 2, Hkv, page, D)
        s["ids"] = _pages(g, c["n"], c["pages"])
        s["lens"] = _ints(g, 1, page, c["n"])  # a decode step's last pages are partly filled
        if c["n"] > 256:
            s["lens"][: c["n"] - 16] = page  # a prompt's pages are full but for the last ones
        s["bounds"] = _normal(g, c["pages"], Hkv, 2, D)
        return s
    B, Hq, G = c["B"], c["Hq"], c["Hq"] // c["Hkv"]
    if c["op"] in ("select", "sparse"):
        length = c["length"]
        width = -(-length // page)
        lens = _ints(g, (length + 1) // 2, length, B)
        lens[0] = length
        s["lens"] = lens
        s["table"] = _pages(g, B * width, B * width).view(B, width).int()
        s["q"] = _normal(g, B, Hq, D, std=1.5)
        if c["op"] == "select":
            # bounds of a page of normal keys lie about its page's extremes
            mid = _normal(g, B * width, Hkv, 1, D, std=0.5).float()
            half = torch.rand(B * width, Hkv, 2, D, generator=g, device=DEV) + 1.5
            half[:, :, 0].neg_()
            s["bounds"] = (mid + half).bfloat16()
            return s
        s["kv"] = _normal(g, B * width, 2, Hkv, page, D)
        # the first and the last block and random ones between them, ascending
        r = torch.rand(B, Hkv, width, generator=g, device=DEV)
        j = torch.arange(width, device=DEV)
        n = ((lens + page - 1) // page)[:, None, None]
        r = torch.where((j == 0) | (j == n - 1), r + 2, r)
        r = torch.where(j < n, r, r - 8)
        k = min(c["topk"], width)
        top = r.topk(k, dim=2).values[..., -1:]
        keep = (r >= top) & (j < n)
        at = torch.where(keep, j, width + 1).sort(dim=2).values[..., :k]
        blocks = torch.full((B, Hkv, c["topk"]), -1, dtype=torch.int32, device=DEV)
        blocks[..., :k] = torch.where(at <= width, at, -1).int()
        s["blocks"] = blocks
        return s
    qlen, P = c["qlen"], -(-c["prefix"] // page)
    width = -(-c["suffix"] // page) + 1
    base = _ints(g, 0, max(0, c["suffix"] - qlen), B)  # tokens cached before this step
    s["lens"] = (base[:, None] + torch.arange(1, qlen + 1, device=DEV)).int().view(-1)
    s["requests"] = torch.arange(B, device=DEV).repeat_interleave(qlen).int()
    ids = _pages(g, P + B * width, P + B * width).int()
    s["prefix_pages"] = ids[:P].contiguous()
    s["table"] = ids[P:].view(B, width).contiguous()
    s["kv"] = _normal(g, P + B * width, 2, Hkv, page, D)
    s["q"] = _normal(g, B * qlen, Hq, D, std=1.5)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    return (_OWN if own else _PLAIN)[s["op"]](s)


def _own_append(s):
    import kv_quant_cache_gb300 as kvq
    kvq.paged_kv_rope_append(s["qkv"], s["Hq"], s["Hkv"], s["D"], s["cos_sin"], s["neox"],
                             s["positions"], s["slots"], s["kv"], q_out=s["q_out"])
    return s["q_out"], s["kv"]


def _own_bounds(s):
    import kv_quant_cache_gb300 as kvq
    return kvq.paged_kv_page_bounds(s["kv"], s["ids"], s["lens"], s["bounds"])


def _own_select(s):
    import kv_quant_cache_gb300 as kvq
    return kvq.paged_kv_block_select(s["q"], s["bounds"], s["table"], s["lens"], s["page"],
                                     s["topk"], keep_first=1, keep_last=1)


def _own_sparse(s):
    import kv_quant_cache_gb300 as kvq
    return kvq.paged_block_sparse_attention(s["q"], s["kv"], s["table"], s["blocks"], s["lens"])


def _own_prefix(s):
    import kv_quant_cache_gb300 as kvq
    return kvq.paged_shared_prefix_attention(s["q"], s["kv"], s["prefix_pages"], s["prefix"],
                                             s["table"], s["lens"], requests=s["requests"])


def _rotate(x, cos, sin, neox):
    """x fp32 [T, H, D]; cos, sin [T, rot/2]: the first rot dims rotate."""
    half = cos.shape[1]
    rot = 2 * half
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., :half], x[..., half:rot]) if neox else (x[..., 0:rot:2], x[..., 1:rot:2])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    y = torch.cat([ra, rb], -1) if neox else torch.stack([ra, rb], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_append(s):
    T, Hq, Hkv, D, page = s["T"], s["Hq"], s["Hkv"], s["D"], s["page"]
    x = s["qkv"].view(T, Hq + 2 * Hkv, D)
    cs = s["cos_sin"][s["positions"]]
    half = s["rot"] // 2
    r = _rotate(x[:, : Hq + Hkv].float(), cs[:, :half], cs[:, half:], s["neox"]).bfloat16()
    s["q_out"].copy_(r[:, :Hq])
    ok = s["slots"] >= 0
    at = s["slots"][ok]
    s["kv"][at // page, 0, :, at % page] = r[ok, Hq:]
    s["kv"][at // page, 1, :, at % page] = x[ok, Hq + Hkv:]
    return s["q_out"], s["kv"]


def _plain_bounds(s):
    k = s["kv"][s["ids"], 0].float()
    there = (torch.arange(s["page"], device=DEV) < s["lens"][:, None])[:, None, :, None]
    lo = torch.where(there, k, math.inf).amin(2)
    hi = torch.where(there, k, -math.inf).amax(2)
    s["bounds"][s["ids"]] = torch.stack([lo, hi], 2).bfloat16()
    return s["bounds"]


def _plain_select(s):
    B, Hq, Hkv, D = s["B"], s["Hq"], s["Hkv"], s["D"]
    width = s["table"].shape[1]
    b = s["bounds"][s["table"].long()].double()  # [B, width, Hkv, 2, D]
    q = s["q"].view(B, Hkv, Hq // Hkv, D).double()
    up, down = q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)
    score = torch.einsum("bhd,bwhd->bhw", up, b[:, :, :, 1])
    score += torch.einsum("bhd,bwhd->bhw", down, b[:, :, :, 0])
    n = ((s["lens"] + s["page"] - 1) // s["page"])[:, None, None]
    j = torch.arange(width, device=DEV)
    score = torch.where((j == 0) | (j == n - 1), math.inf, score)
    score = torch.where(j < n, score, -math.inf)
    k = min(s["topk"], width)
    at = score.sort(dim=2, descending=True, stable=True).indices[..., :k]
    at = torch.where(at < n, at, width).sort(dim=2).values
    out = torch.full((B, Hkv, s["topk"]), -1, dtype=torch.int32, device=DEV)
    out[..., :k] = torch.where(at < width, at, -1).int()
    return out


def _soft(score):
    """exp of scores less their row's largest, that largest, and the sum."""
    m = score.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = (score - m).exp()
    return p, m, p.sum(-1, keepdim=True)


def _plain_sparse(s):
    B, Hq, Hkv, D, page = s["B"], s["Hq"], s["Hkv"], s["D"], s["page"]
    blk = s["blocks"].long()
    ids = s["table"].long().gather(1, blk.clamp(min=0).view(B, -1)).view(blk.shape)
    h = torch.arange(Hkv, device=DEV)[None, :, None]
    k = s["kv"][ids, 0, h].float().flatten(2, 3)  # [B, Hkv, topk * page, D]
    v = s["kv"][ids, 1, h].float().flatten(2, 3)
    at = blk[..., None] * page + torch.arange(page, device=DEV)
    ok = ((blk >= 0)[..., None] & (at < s["lens"][:, None, None, None])).flatten(2)
    q = s["q"].view(B, Hkv, Hq // Hkv, D).float() / math.sqrt(D)
    score = torch.where(ok[:, :, None], q @ k.transpose(2, 3), -math.inf)
    p, _, total = _soft(score)
    o = p @ v / torch.where(total > 0, total, 1.0)
    return o.view(B, Hq, D).bfloat16()


def _plain_prefix(s):
    B, qlen, Hq, Hkv, D, page = (s[x] for x in ("B", "qlen", "Hq", "Hkv", "D", "page"))
    G, L = Hq // Hkv, s["prefix"]
    q = s["q"].view(B, qlen, Hkv, G, D).permute(2, 0, 1, 3, 4).float() / math.sqrt(D)
    pre = s["kv"][s["prefix_pages"].long()].permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :L].float()
    p1, m1, t1 = _soft(q.reshape(Hkv, -1, D) @ pre[0].transpose(1, 2))
    o1 = (p1 @ pre[1]).view(Hkv, B, qlen * G, D)
    m1, t1 = m1.view(Hkv, B, qlen * G, 1), t1.view(Hkv, B, qlen * G, 1)
    suf = s["kv"][s["table"].long()].permute(2, 3, 0, 1, 4, 5).flatten(3, 4).float()
    score = q.reshape(Hkv, B, qlen * G, D) @ suf[0].transpose(2, 3)
    ok = torch.arange(suf.shape[3], device=DEV) < s["lens"][:, None]
    ok = ok.view(B, qlen, 1, -1).expand(B, qlen, G, -1).reshape(B, qlen * G, -1)
    p2, m2, t2 = _soft(torch.where(ok, score, -math.inf))
    m = torch.maximum(m1, m2)
    a1, a2 = (m1 - m).exp(), (m2 - m).exp()
    o = (o1 * a1 + (p2 @ suf[1]) * a2) / (t1 * a1 + t2 * a2)
    return o.view(Hkv, B, qlen, G, D).permute(1, 2, 0, 3, 4).reshape(B * qlen, Hq, D).bfloat16()


_PLAIN = dict(append=_plain_append, bounds=_plain_bounds, select=_plain_select,
              sparse=_plain_sparse, prefix=_plain_prefix)
_OWN = dict(append=_own_append, bounds=_own_bounds, select=_own_select, sparse=_own_sparse,
            prefix=_own_prefix)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    Hkv, D, page = c["Hkv"], c["D"], c["page"]
    kv = Hkv * D * 2  # bytes of a token's keys (or values)
    if c["op"] == "append":
        T, Hq = c["T"], c["Hq"]
        rows = 2 * T * (Hq + 2 * Hkv) * D * 2  # each row read once and written once
        table = min(T, c["max_pos"]) * c["rot"] * 4
        return {"bytes": rows + table + 16 * T, "flops": 3 * T * (Hq + Hkv) * c["rot"]}
    if c["op"] == "bounds":
        n = c["n"]
        keys = n * page if n > 256 else n * (page + 1) // 2
        return {"bytes": keys * kv + n * (2 * kv + 12), "flops": 2 * keys * Hkv * D}
    B, Hq = c["B"], c["Hq"]
    if c["op"] == "select":
        blocks = B * -(-c["length"] // page) * 3 // 4 if B > 1 else -(-c["length"] // page)
        return {"bytes": blocks * (2 * kv + 4) + B * Hq * D * 2 + B * Hkv * c["topk"] * 4,
                "flops": blocks * Hkv * D * 4}
    if c["op"] == "sparse":
        keys = B * min(c["topk"] * page, c["length"] if B == 1 else c["length"] * 3 // 4)
        return {"bytes": keys * 2 * kv + 2 * B * Hq * D * 2 + B * Hkv * c["topk"] * 4,
                "flops": 4 * keys * Hq * D}
    tokens = B * c["qlen"]
    suffix = B * (max(0, c["suffix"] - c["qlen"]) // 2 + c["qlen"])
    return {"bytes": (c["prefix"] + suffix) * 2 * kv + 2 * tokens * Hq * D * 2,
            "flops": 4 * (tokens * c["prefix"] + c["qlen"] * suffix) * Hq * D}


# ---------------------------------------------------------------------------
# The definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[s["op"]](s)


def _exact_append(s):
    T, Hq, Hkv, D, rot, page = (s[x] for x in ("T", "Hq", "Hkv", "D", "rot", "page"))
    x = s["qkv"].double().view(T, Hq + 2 * Hkv, D)
    cs = s["cos_sin"].double()[s["positions"]]
    i = torch.arange(rot // 2, device=DEV)
    first, second = (i, i + rot // 2) if s["neox"] else (2 * i, 2 * i + 1)
    c, n = cs[:, None, : rot // 2], cs[:, None, rot // 2:]
    y = x.clone()
    y[..., first] = x[..., first] * c - x[..., second] * n
    y[..., second] = x[..., first] * n + x[..., second] * c
    flat = s["kv"].double().transpose(2, 3).reshape(-1, 2, page, Hkv, D)
    t = (s["slots"] >= 0).nonzero()[:, 0]
    slot = s["slots"][t]
    flat[slot // page, 0, slot % page] = y[t, Hq:Hq + Hkv]
    flat[slot // page, 1, slot % page] = x[t, Hq + Hkv:]
    return y[:, :Hq], flat.transpose(2, 3)


def _exact_bounds(s):
    out = s["bounds"].double()
    step = 512
    for a in range(0, s["n"], step):
        ids, lens = s["ids"][a:a + step], s["lens"][a:a + step]
        k = s["kv"][ids, 0].double()
        gone = torch.arange(s["page"], device=DEV)[None] >= lens[:, None]
        gone = gone[:, None, :, None].expand_as(k)
        out[ids, :, 0] = k.masked_fill(gone, math.inf).min(2).values
        out[ids, :, 1] = k.masked_fill(gone, -math.inf).max(2).values
    return out


def _exact_select(s):
    return None  # whole numbers


def _exact_attend(q, k, v):
    """q [n, D] against k, v [m, D]."""
    if k.shape[0] == 0:
        return torch.zeros_like(q)
    return torch.softmax(q @ k.T / math.sqrt(q.shape[1]), -1) @ v


def _exact_sparse(s):
    B, Hq, Hkv, D, page = (s[x] for x in ("B", "Hq", "Hkv", "D", "page"))
    G = Hq // Hkv
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=DEV)
    lens, blocks = s["lens"].tolist(), s["blocks"].tolist()
    for b in range(B):
        for h in range(Hkv):
            mine = [j for j in blocks[b][h] if j >= 0]
            at = (torch.tensor(mine, device=DEV)[:, None] * page
                  + torch.arange(page, device=DEV)).flatten()
            at = at[at < lens[b]]
            rows = s["kv"][s["table"][b].long()[at // page], :, h, at % page].double()
            out[b, h * G:(h + 1) * G] = _exact_attend(s["q"][b, h * G:(h + 1) * G].double(),
                                                      rows[:, 0], rows[:, 1])
    return out


def _exact_prefix(s):
    T, Hq, Hkv, D, page, L = s["q"].shape[0], s["Hq"], s["Hkv"], s["D"], s["page"], s["prefix"]
    G = Hq // Hkv
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=DEV)
    lens, req = s["lens"].tolist(), s["requests"].tolist()
    at = torch.arange(L, device=DEV)
    for h in range(Hkv):
        pre = s["kv"][s["prefix_pages"].long()[at // page], :, h, at % page].double()
        for t in range(T):
            i = torch.arange(lens[t], device=DEV)
            own_rows = s["kv"][s["table"][req[t]].long()[i // page], :, h, i % page].double()
            rows = torch.cat([pre, own_rows])
            out[t, h * G:(h + 1) * G] = _exact_attend(s["q"][t, h * G:(h + 1) * G].double(),
                                                      rows[:, 0], rows[:, 1])
    return out


_EXACT = dict(append=_exact_append, bounds=_exact_bounds, select=_exact_select,
              sparse=_exact_sparse, prefix=_exact_prefix)
