"""Cases of the operators on quantised caches: appending keys and values to a
paged cache held in 4 bits, reading them back, attention over such a cache, and
attention over the shared latent vectors of the 584-byte FP8 entries.

``run`` computes each operator either in plain torch operations (``own`` is
false) or through this repository's package (``own`` is true), on the same
inputs.

The 4-bit cache is uint8 [pages, 2, kv heads, page size, 9 D / 16]: of each page
the keys of every kv head, then the values.  A head's block of a page holds first
the codes of its tokens, D / 2 bytes each, then per token and group of 64 dims a
scale and a zero in bf16.  A code c stands for zero + scale (c - 8).  Four bytes
hold eight dims: the low nibbles dims 0 4 1 5, the high ones dims 2 6 3 7.
"""
import math

import torch

own = False

DEV = "cuda"
THETA = 1e6
GROUP = 64   # dims that share a scale and a zero
ENTRY = 584  # bytes of a latent entry: 448 codes, 64 rotary bf16, 7 exponents, a pad


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _append(name, T, Hq, Hkv, D, rot, neox, max_pos, page):
    return dict(name=name, op="append", T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rot, neox=neox,
                max_pos=max_pos, page=page)


def _gather(name, n, Hkv, D, page):
    return dict(name=name, op="gather", n=n, Hkv=Hkv, D=D, page=page)


def _attend(name, B, qlen, Hq, Hkv, D, page, length):
    return dict(name=name, op="attend", B=B, qlen=qlen, Hq=Hq, Hkv=Hkv, D=D, page=page,
                length=length)


def _latent(name, T, H, K, block):
    return dict(name=name, op="latent", T=T, H=H, K=K, block=block)


def listed():
    return [
        # one decode step of a small batch writes its tokens: latency counts
        _append("append4_T17", 17, 16, 8, 128, 128, True, 4096, 64),
        # a prompt chunk whose rotation covers a quarter of each head, in adjacent pairs
        _append("append4_T4097_partial", 4097, 16, 2, 64, 16, False, 131072, 16),
        # a large prompt batch
        _append("append4_T32768", 32768, 32, 8, 128, 128, True, 131072, 64),
        # a short conversation is read back
        _gather("gather4_1000", 1000, 8, 128, 64),
        # a long document is read back, for a prompt's attention in bf16
        _gather("gather4_65536", 65536, 8, 128, 64),
        # one long conversation decodes
        _attend("attend4_B1", 1, 1, 32, 8, 128, 64, 100003),
        # three draft tokens each of a batch, 64-dim heads
        _attend("attend4_B33_q3_D64", 33, 3, 16, 2, 64, 16, 8209),
        # a chunk of a prompt behind what is cached of it, 256-dim heads
        _attend("attend4_B2_q65_D256", 2, 65, 16, 2, 256, 64, 4100),
        # a decode batch of long conversations
        _attend("attend4_B64", 64, 1, 32, 8, 128, 64, 32768),
        # one token attends to the entries picked for it
        _latent("latent_T1_H64", 1, 64, 2051, 64),
        # a decode batch does
        _latent("latent_T64_H64", 64, 64, 2048, 64),
        # long lists, twice the heads
        _latent("latent_T16_H128", 16, 128, 16384, 64),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "gather", "attend", "attend", "latent", "latent"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 7, 8, 16])
    D = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 48, 64, 64, 128])
    if op == "append":
        rot = rng.choice([D, D, D // 2, D // 4])
        T = _log(rng, 1, max(1, min(32768, 32768 * 48 * 128 // ((Hq + 2 * Hkv) * D))))
        c = _append("", T, Hq, Hkv, D, rot, rng.random() < 0.6, rng.choice([8192, 131072]), page)
    elif op == "gather":
        c = _gather("", _log(rng, 1, min(65536, 65536 * 8 * 128 // (Hkv * D))), Hkv, D, page)
    elif op == "attend":
        qlen = rng.choice([1, 1, 1, 2, 4, 19])
        B = _log(rng, 1, 64 if qlen < 19 else 8)
        rows = max(Hq // Hkv * qlen, 16) * Hkv  # at least a tile of 16 rows a kv head
        most = min(100003, 64 * 32768 * 8 * 128 // (B * Hkv * D),
                   64 * 32768 * 8 * 16 * 128 // (B * rows * D))
        c = _attend("", B, qlen, Hq, Hkv, D, page, _log(rng, 1, most))
    else:
        H = rng.choice([1, 8, 16, 20, 32, 64, 64, 128])
        T = _log(rng, 1, 128)
        c = _latent("", T, H, _log(rng, 1, min(32768, 16 * 16384 // T)), rng.choice([1, 16, 64]))
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


def _perm(g, n, total):
    return torch.randperm(total, generator=g, device=DEV)[:n]


def _cache4(g, pages, Hkv, page, D):
    """A filled 4-bit cache of normal keys and values, some pages at a time."""
    kv = torch.empty(pages, 2, Hkv, page * D * 9 // 16, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (2 * Hkv * page * D))
    for a in range(0, pages, step):
        b = min(pages, a + step)
        codes, meta = _quantise(_normal(g, b - a, 2, Hkv, page, D).float())
        half = page * D // 2
        kv[a:b, ..., :half] = codes.flatten(3)
        kv[a:b, ..., half:] = meta.view(torch.uint8).flatten(3)
    return kv.view(pages, 2, Hkv, page, D * 9 // 16)


def _entries(g, slots):
    """Latent entries of normal vectors."""
    out = torch.empty(slots, ENTRY, dtype=torch.uint8, device=DEV)
    for a in range(0, slots, 1 << 16):
        b = min(slots, a + (1 << 16))
        x = _normal(g, b - a, 512).float()
        blocks = x[:, :448].view(b - a, 7, 64)
        e = torch.ceil(torch.log2(blocks.abs().amax(2) / 448.0))
        codes = (blocks * torch.exp2(-e)[..., None]).to(torch.float8_e4m3fn)
        out[a:b, :448] = codes.flatten(1).view(torch.uint8)
        out[a:b, 448:576] = x[:, 448:].bfloat16().view(torch.uint8)
        out[a:b, 576:583] = (e + 127).to(torch.uint8)
        out[a:b, 583] = 0
    return out


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(c)
    if c["op"] == "append":
        T, Hq, Hkv, D, page = (c[x] for x in ("T", "Hq", "Hkv", "D", "page"))
        pages = -(-T // page) + 8
        s["qkv"] = _normal(g, T, (Hq + 2 * Hkv) * D)
        s["positions"] = torch.randint(0, c["max_pos"], (T,), generator=g, device=DEV)
        s["cos_sin"] = _table(c["max_pos"], c["rot"])
        s["slots"] = _perm(g, T, pages * page)
        if T > 8:
            s["slots"][T // 3] = -1  # a padding token
        s["kv"] = torch.zeros(pages, 2, Hkv, page, D * 9 // 16, dtype=torch.uint8, device=DEV)
        s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
        return s
    if c["op"] == "gather":
        n, page = c["n"], c["page"]
        pages = -(-n // page) + 8
        s["kv"] = _cache4(g, pages, c["Hkv"], page, c["D"])
        # the pages of a request, in its own order, and their tokens one after the other
        at = torch.arange(n, device=DEV)
        s["slots"] = _perm(g, pages, pages)[at // page] * page + at % page
        return s
    if c["op"] == "attend":
        B, qlen, length, page = c["B"], c["qlen"], c["length"], c["page"]
        width = -(-length // page)
        last = _ints(g, (length + 1) // 2, length, B)
        last[0] = length
        # the last token of a request sees all its keys, the others one less each
        back = torch.arange(qlen - 1, -1, -1, device=DEV)
        s["lens"] = (last[:, None] - back).clamp(min=0).int().view(-1)
        s["table"] = _perm(g, B * width, B * width).view(B, width).int()
        s["kv"] = _cache4(g, B * width, c["Hkv"], page, c["D"])
        s["q"] = _normal(g, B * qlen, c["Hq"], c["D"], std=1.5)
        return s
    T, H, K, block = c["T"], c["H"], c["K"], c["block"]
    blocks = -(-T * K // block) + 2
    s["kv"] = _entries(g, blocks * block).view(blocks, block, ENTRY)
    s["slots"] = _perm(g, T * K, blocks * block).view(T, K).int()
    lens = _ints(g, (K + 1) // 2, K, T)
    lens[0] = K
    s["lens"] = lens
    if K > 16:
        s["slots"][:, K // 4] = -1  # a place that the selection left empty
    s["q"] = _normal(g, T, H, 512, std=1.5)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    return (_OWN if own else _PLAIN)[s["op"]](s)


def _own_append(s):
    import kv_quant_cache_gb300 as kvq
    kvq.paged_kv4_rope_append(s["qkv"], s["Hq"], s["Hkv"], s["D"], s["cos_sin"], s["neox"],
                              s["positions"], s["slots"], s["kv"], q_out=s["q_out"])
    return (s["q_out"], *kvq.paged_kv4_gather(s["kv"], s["slots"]))


def _own_gather(s):
    import kv_quant_cache_gb300 as kvq
    return kvq.paged_kv4_gather(s["kv"], s["slots"])


def _own_attend(s):
    import kv_quant_cache_gb300 as kvq
    return kvq.paged_kv4_attention(s["q"], s["kv"], s["table"], s["lens"],
                                   tokens_per_request=s["qlen"])


def _own_latent(s):
    import kv_quant_cache_gb300 as kvq
    return kvq.dsv4_latent_attention(s["q"], s["kv"], s["slots"], s["lens"])


def _rotate(x, cos, sin, neox):
    """x [T, H, D]; cos, sin [T, rot/2]: the first rot dims rotate."""
    half = cos.shape[1]
    rot = 2 * half
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., :half], x[..., half:rot]) if neox else (x[..., 0:rot:2], x[..., 1:rot:2])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    y = torch.cat([ra, rb], -1) if neox else torch.stack([ra, rb], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _quantise(x):
    """fp32 [..., D] -> codes uint8 [..., D/2] and bf16 [..., D/64, 2] of scale
    and zero."""
    v = x.unflatten(-1, (-1, GROUP))
    lo, hi = v.amin(-1), v.amax(-1)
    scale = ((hi - lo) / 15.0).bfloat16()
    zero = (lo + 8.0 * scale.float()).bfloat16()
    step = scale.float()[..., None]
    code = torch.round((v - zero.float()[..., None]) / torch.where(step > 0, step, 1.0)) + 8.0
    code = torch.where(step > 0, code.clamp(0.0, 15.0), 8.0).to(torch.uint8)
    n = code.flatten(-2).unflatten(-1, (-1, 4, 2)).transpose(-1, -2).flatten(-2)  # nibbles
    n = n.unflatten(-1, (4, 2))
    return (n[..., 0] | n[..., 1] << 4).flatten(-2), torch.stack([scale, zero], -1)


def _values(codes, meta):
    """The fp32 values of codes uint8 [..., D/2] with bf16 [..., D/64, 2]."""
    b = codes.unflatten(-1, (-1, 4))
    n = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    c = n.unflatten(-1, (2, 4)).transpose(-1, -2).flatten(-3).float()
    m = meta.float()
    return (m[..., 1:] + m[..., :1] * (c.unflatten(-1, (-1, GROUP)) - 8.0)).flatten(-2)


def _parts4(kv):
    """Views of a cache's codes [pages, 2, Hkv, page, D/2] and bf16 scales and
    zeros [pages, 2, Hkv, page, D/64, 2]."""
    page, D = kv.shape[3], kv.shape[4] * 16 // 9
    flat = kv.flatten(3)
    half = page * D // 2
    codes = flat[..., :half].unflatten(-1, (page, D // 2))
    meta = flat[..., half:].view(torch.bfloat16).unflatten(-1, (page, D // GROUP, 2))
    return codes, meta


def _plain_append(s):
    T, Hq, Hkv, D, page = s["T"], s["Hq"], s["Hkv"], s["D"], s["page"]
    x = s["qkv"].view(T, Hq + 2 * Hkv, D)
    cs = s["cos_sin"][s["positions"]].double()  # a rotated key lies next to a border of two codes
    half = s["rot"] // 2
    r = _rotate(x[:, : Hq + Hkv].double(), cs[:, :half], cs[:, half:], s["neox"]).bfloat16()
    s["q_out"].copy_(r[:, :Hq])
    codes, meta = _quantise(torch.stack([r[:, Hq:], x[:, Hq + Hkv:]], 1).float())
    ok = s["slots"] >= 0
    at = s["slots"][ok]
    to_codes, to_meta = _parts4(s["kv"])
    to_codes[at // page, :, :, at % page] = codes[ok]
    to_meta[at // page, :, :, at % page] = meta[ok]
    return (s["q_out"], *_plain_gather(s))


def _plain_gather(s):
    page = s["page"]
    codes, meta = _parts4(s["kv"])
    at = s["slots"].clamp(min=0)
    v = _values(codes[at // page, :, :, at % page], meta[at // page, :, :, at % page])
    v = torch.where((s["slots"] >= 0)[:, None, None, None], v, 0.0).bfloat16()
    return v[:, 0].contiguous(), v[:, 1].contiguous()


def _weights(score):
    """exp of scores less their row's largest, over their sum; zeros in a row
    without a key."""
    m = score.amax(-1, keepdim=True)
    p = (score - torch.where(m == -math.inf, 0.0, m)).exp()
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, 1.0)


def _plain_attend(s):
    B, qlen, Hq, Hkv, D = (s[x] for x in ("B", "qlen", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    codes, meta = _parts4(s["kv"])
    at = s["table"].long()
    # [B, width, Hkv, page, D] -> [B, Hkv, keys, D]
    k = _values(codes[at, 0], meta[at, 0]).transpose(1, 2).flatten(2, 3)
    v = _values(codes[at, 1], meta[at, 1]).transpose(1, 2).flatten(2, 3)
    q = s["q"].view(B, qlen, Hkv, G, D).transpose(1, 2).float() / math.sqrt(D)
    score = q.reshape(B, Hkv, qlen * G, D) @ k.transpose(2, 3)
    ok = torch.arange(k.shape[2], device=DEV) < s["lens"][:, None]  # [T, keys]
    ok = ok.view(B, 1, qlen, 1, -1).expand(B, 1, qlen, G, -1).reshape(B, 1, qlen * G, -1)
    o = _weights(torch.where(ok, score, -math.inf)) @ v
    return o.view(B, Hkv, qlen, G, D).transpose(1, 2).reshape(B * qlen, Hq, D).bfloat16()


def _plain_latent(s):
    T, H, K = s["T"], s["H"], s["K"]
    e = s["kv"].view(-1, ENTRY)[s["slots"].clamp(min=0).long()]  # [T, K, 584]
    codes = e[..., :448].contiguous().view(torch.float8_e4m3fn).float()
    scale = torch.exp2(e[..., 576:583].float() - 127.0)
    rope = e[..., 448:576].contiguous().view(torch.bfloat16).float()
    x = torch.cat([(codes.unflatten(-1, (7, 64)) * scale[..., None]).flatten(-2), rope], -1)
    score = s["q"].float() / math.sqrt(512.0) @ x.transpose(1, 2)
    ok = (s["slots"] >= 0) & (torch.arange(K, device=DEV) < s["lens"][:, None])
    return (_weights(torch.where(ok[:, None], score, -math.inf)) @ x).bfloat16()


_PLAIN = dict(append=_plain_append, gather=_plain_gather, attend=_plain_attend,
              latent=_plain_latent)
_OWN = dict(append=_own_append, gather=_own_gather, attend=_own_attend, latent=_own_latent)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "latent":
        T, H, K = c["T"], c["H"], c["K"]
        keys = K if T == 1 else T * K * 3 // 4
        return {"bytes": keys * (ENTRY + 4) + 2 * T * H * 512 * 2, "flops": 4 * keys * H * 512}
    Hkv, D = c["Hkv"], c["D"]
    held = 2 * Hkv * D * 9 // 16  # bytes of a token's keys and values in the cache
    if c["op"] == "append":
        # the rows in, q rows out, codes out; and the codes in again, keys and values out
        T, Hq = c["T"], c["Hq"]
        rows = T * (2 * Hq + 2 * Hkv) * D * 2
        table = min(T, c["max_pos"]) * c["rot"] * 4
        return {"bytes": rows + table + 24 * T + 2 * T * held + T * 2 * Hkv * D * 2,
                "flops": 3 * T * (Hq + Hkv) * c["rot"] + 8 * T * 2 * Hkv * D}
    if c["op"] == "gather":
        return {"bytes": c["n"] * (held + 2 * Hkv * D * 2 + 8), "flops": 2 * c["n"] * 2 * Hkv * D}
    B, qlen, Hq = c["B"], c["qlen"], c["Hq"]
    keys = c["length"] if B == 1 else B * c["length"] * 3 // 4
    return {"bytes": keys * held + 2 * B * qlen * Hq * D * 2, "flops": 4 * keys * qlen * Hq * D}


# ---------------------------------------------------------------------------
# The definitions, in 64 bits
# ---------------------------------------------------------------------------

_BYTE = (0, 2, 0, 2, 1, 3, 1, 3)   # of the four bytes of eight dims, the one of each
_SHIFT = (0, 0, 4, 4, 0, 0, 4, 4)  # and the place in it


def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[s["op"]](s)


def _exact_rows(kv, slots):
    """fp64 [n, 2, Hkv, D]: what the cache holds at ``slots``, read byte by byte."""
    pages, _, Hkv, page, held = kv.shape
    D = held * 16 // 9
    flat = kv.reshape(pages, 2, Hkv, page * held)
    d = torch.arange(D, device=DEV)
    byte = d // 8 * 4 + torch.tensor(_BYTE, device=DEV)[d % 8]
    n, off = (slots // page)[:, None], (slots % page)[:, None]
    raw = flat[n, :, :, off * (D // 2) + byte].int()  # [n, D, 2, Hkv]
    code = raw >> torch.tensor(_SHIFT, device=DEV)[d % 8][:, None, None] & 15
    at = page * (D // 2) + (off * (D // GROUP) + d // GROUP) * 4

    def number(first):  # a bf16 is the upper half of an fp32
        bits = flat[n, :, :, first].int() << 16 | flat[n, :, :, first + 1].int() << 24
        return bits.view(torch.float32).double()

    return (number(at + 2) + number(at) * (code.double() - 8.0)).permute(0, 2, 3, 1)


def _exact_gather(s):
    x = _exact_rows(s["kv"], s["slots"].clamp(min=0))
    x[s["slots"] < 0] = 0.0
    return x[:, 0].contiguous(), x[:, 1].contiguous()


def _exact_append(s):
    T, Hq, Hkv, D, rot = (s[x] for x in ("T", "Hq", "Hkv", "D", "rot"))
    x = s["qkv"].double().view(T, Hq + 2 * Hkv, D)
    cs = s["cos_sin"].double()[s["positions"]]
    i = torch.arange(rot // 2, device=DEV)
    first, second = (i, i + rot // 2) if s["neox"] else (2 * i, 2 * i + 1)
    c, n = cs[:, None, : rot // 2], cs[:, None, rot // 2:]
    y = x[:, :Hq + Hkv].clone()
    y[..., first] = x[:, :Hq + Hkv, first] * c - x[:, :Hq + Hkv, second] * n
    y[..., second] = x[:, :Hq + Hkv, first] * n + x[:, :Hq + Hkv, second] * c
    held = []
    for v in (y[:, Hq:].float().bfloat16().double(), x[:, Hq + Hkv:]):
        v = v.reshape(T, Hkv, D // GROUP, GROUP)
        lo, hi = v.min(-1, keepdim=True).values, v.max(-1, keepdim=True).values
        step = ((hi - lo) / 15).float().bfloat16().double()
        zero = (lo + 8 * step).float().bfloat16().double()
        code = ((v - zero) / step.masked_fill(step == 0, 1)).round().clamp(-8, 7)
        v = (zero + step * code).view(T, Hkv, D)
        v[s["slots"] < 0] = 0.0
        held.append(v)
    return (y[:, :Hq].contiguous(), *held)


def _exact_attend(s):
    B, qlen, Hq, Hkv, D, page = (s[x] for x in ("B", "qlen", "Hq", "Hkv", "D", "page"))
    G = Hq // Hkv
    out = torch.zeros(B * qlen, Hq, D, dtype=torch.float64, device=DEV)
    lens = s["lens"].tolist()
    for b in range(B):
        of = range(b * qlen, (b + 1) * qlen)
        n = max(lens[t] for t in of)
        if n == 0:
            continue
        at = torch.arange(n, device=DEV)
        x = _exact_rows(s["kv"], s["table"][b].long()[at // page] * page + at % page)
        q = s["q"][b * qlen:(b + 1) * qlen].double().view(qlen, Hkv, G, D)
        score = torch.einsum("qhgd,nhd->qhgn", q, x[:, 0]) / math.sqrt(D)
        unseen = at >= s["lens"][b * qlen:(b + 1) * qlen, None]
        score = score.masked_fill(unseen[:, None, None], -math.inf)
        o = torch.einsum("qhgn,nhd->qhgd", torch.softmax(score, -1), x[:, 1])
        o[s["lens"][b * qlen:(b + 1) * qlen] == 0] = 0.0
        out[b * qlen:(b + 1) * qlen] = o.reshape(qlen, Hq, D)
    return out


def _exact_latent(s):
    T, H, K = s["T"], s["H"], s["K"]
    out = torch.zeros(T, H, 512, dtype=torch.float64, device=DEV)
    byte = torch.arange(256, device=DEV)
    # e4m3: sign, four bits of exponent (bias 7), three of fraction
    e, f = byte >> 3 & 15, (byte & 7).double()
    number = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * torch.exp2(e.double() - 7))
    number = torch.where(byte < 128, number, -number)
    flat, lens = s["kv"].view(-1, ENTRY), s["lens"].tolist()
    for t in range(T):
        at = s["slots"][t, :lens[t]]
        at = at[at >= 0].long()
        if not len(at):
            continue
        entry = flat[at].long()
        scale = torch.exp2(entry[:, 576:583].double() - 127).repeat_interleave(64, 1)
        rope = flat[at, 448:576].contiguous().view(torch.bfloat16).double()
        x = torch.cat([number[entry[:, :448]] * scale, rope], 1)
        out[t] = torch.softmax(s["q"][t].double() @ x.T / math.sqrt(512), -1) @ x
    return out


_EXACT = dict(append=_exact_append, gather=_exact_gather, attend=_exact_attend,
              latent=_exact_latent)
