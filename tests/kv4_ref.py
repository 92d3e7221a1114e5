"""Plain forms of the operators on quantised caches, and the error bounds their
kernels are held to.

The 4-bit cache is a decision per value, so its bytes have to be equal.

The bound of the attention over it, element by element.  A value is v = z + s n
with n = c - 8.  With w the exact softmax weights and n_keys keys:
  * a numerator times its key's s is rounded once to bf16: 2^-8 sum_i w_i |s n|_i;
  * a score is the sum over groups of s (q . n) + z sum(q), 64-term fp32 sums of exact
    products and a few fp32 operations a group: off by at most ds = (D + 16) 2^-23 |scale|
    max_i sum_j (31 s + |z - 24 s|) sum_d |q_d|, which is a relative ds of its
    numerator, and of the row sum again.  (Terms are at most (8 s + |z|) |q|, 8/7 of the
    magnitudes above; products are added sixteen at a time, so roundings are far fewer
    than D.);
  * additions and rescalings as in the bf16 attention: (2 n_keys + 64) 2^-22;
  * the output is rounded once to bf16: 2^-8 |out|.
"""
import numpy as np
import torch

import paged_ref as ref

GROUP = 64
EPS_BF16 = ref.EPS_BF16


def held_bytes(D):
    return D * 9 // 16


def quantise(x):
    """bf16 [..., D] -> codes uint8 [..., D] (0 .. 15), scale and zero bf16
    [..., D/64]."""
    v = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = v.amin(-1), v.amax(-1)
    width = hi - lo
    bad = ~(width < float("inf"))
    scale = torch.where(bad, float("nan"), width / 15).bfloat16()
    zero = torch.where(bad, float("nan"), lo + 8 * scale.float()).bfloat16()
    t = (v - zero.float()[..., None]).double()  # the fp32 difference
    step = scale.double()[..., None]
    n = torch.round(t / torch.where(step > 0, step, 1.0)).clamp(-8, 7)
    code = torch.where(step > 0, n + 8, 8.0).nan_to_num(8.0).to(torch.uint8)
    return code.flatten(-2), scale, zero


def rotated_keys(k, cos_sin, pos, rot, neox):
    """bf16 [T, H, D]: the exact rotation rounded to fp32 and then to bf16."""
    x = k.double()
    for t in range(k.shape[0]):
        if rot:
            x[t] = ref.rotate(k[t].double(), cos_sin[int(pos[t])].double(), rot, neox)[0]
    return x.float().bfloat16()


class Cache:
    """A 4-bit cache taken apart: codes [pages, 2, Hkv, page, D], scale and zero
    [pages, 2, Hkv, page, D/64]."""

    def __init__(self, raw):
        raw = raw.cpu()
        pages, _, Hkv, page, held = raw.shape
        D = held * 16 // 9
        flat = raw.reshape(pages, 2, Hkv, page * held).numpy()
        words = flat[..., :page * D // 2].reshape(pages, 2, Hkv, page, D // 8, 4)
        words = np.ascontiguousarray(words).view("<u4")[..., 0]
        d = np.arange(D)
        at = 4 * (d % 8 // 2) + 16 * (d % 2)
        self.codes = torch.from_numpy((words[..., d // 8] >> at.astype("u4") & 15).astype("u1"))
        meta = np.ascontiguousarray(flat[..., page * D // 2:]).view("<u2").astype("<u4") << 16
        meta = torch.from_numpy(meta.view("<f4").reshape(pages, 2, Hkv, page, D // GROUP, 2))
        self.scale, self.zero = meta[..., 0], meta[..., 1]

    def terms(self, pages, off, h):
        """fp64 s n and z, [n, 2, D], of the tokens at offsets ``off`` of ``pages``."""
        n = self.codes[pages, :, h, off].double() - 8
        s = self.scale[pages, :, h, off].double().repeat_interleave(GROUP, -1)
        return s * n, self.zero[pages, :, h, off].double().repeat_interleave(GROUP, -1), s


def raw_of(codes, scale, zero):
    """The cache's bytes of codes [pages, 2, Hkv, page, D] and bf16 scale, zero."""
    pages, _, Hkv, page, D = codes.shape
    c = codes.numpy().astype("u4").reshape(pages, 2, Hkv, page, D // 8, 8)
    d = np.arange(8)
    words = (c << (4 * (d // 2) + 16 * (d % 2)).astype("u4")).sum(-1).astype("<u4")
    meta = torch.stack([scale, zero], -1).contiguous().view(torch.int16).numpy().view("u1")
    flat = np.concatenate([words.view("u1").reshape(pages, 2, Hkv, -1),
                           meta.reshape(pages, 2, Hkv, -1)], -1)
    return torch.from_numpy(flat.reshape(pages, 2, Hkv, page, held_bytes(D)).copy())


def random_cache(g, pages, Hkv, page, D):
    return raw_of(*quantise(torch.randn(pages, 2, Hkv, page, D, generator=g).bfloat16()))


def gather(raw, slots):
    """bf16 (k, v) [n, Hkv, D]: fp32 zero + scale n, then bf16."""
    c = Cache(raw)
    pages, _, Hkv, page, D = c.codes.shape
    out = torch.zeros(len(slots), 2, Hkv, D)
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            n = c.codes[s // page, :, :, s % page].float() - 8
            sc = c.scale[s // page, :, :, s % page].repeat_interleave(GROUP, -1)
            out[i] = c.zero[s // page, :, :, s % page].repeat_interleave(GROUP, -1) + sc * n
    return out[:, 0].bfloat16(), out[:, 1].bfloat16()


def attend(q, sn, z, s, scale):
    """(out, bound) fp64 [G, D] of q [G, D] against keys and values [n, 2, D] given
    as s n, z and s."""
    q = q.double()
    n, _, D = sn.shape
    if n == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    k, v = sn[:, 0] + z[:, 0], sn[:, 1] + z[:, 1]
    w = torch.softmax(q @ k.T * scale, -1)
    out = w @ v
    mag = 31 * s[:, 0] + (z[:, 0] - 24 * s[:, 0]).abs()
    ds = (D + 16) * 2.0 ** -23 * abs(scale) * (q.abs() @ mag.T).amax(-1, keepdim=True)
    codes, whole = w @ sn[:, 1].abs(), w @ (sn[:, 1].abs() + z[:, 1].abs())
    tol = EPS_BF16 * codes + whole * (2 * ds + (2 * n + 64) * 2.0 ** -22)
    return out, tol + EPS_BF16 * out.abs()


def attention(q, raw, table, lens, scale, per_request=1):
    T, Hq, D = q.shape
    c = Cache(raw)
    N, _, Hkv, page, _ = c.codes.shape
    G = Hq // Hkv
    out, tol = torch.zeros(T, Hq, D).double(), torch.zeros(T, Hq, D).double()
    for t in range(T):
        n = max(0, min(int(lens[t]), table.shape[1] * page))
        at = torch.arange(n)
        ids = table[t // per_request].long()[at // page]
        ok = (ids >= 0) & (ids < N)
        for h in range(Hkv):
            g = slice(h * G, (h + 1) * G)
            out[t, g], tol[t, g] = attend(q[t, g], *c.terms(ids[ok], (at % page)[ok], h), scale)
    return out, tol


# ---- latent entries ---------------------------------------------------------------

def entries(x):
    """Latent entries uint8 [n, 584] of bf16 vectors [n, 512]: each block's scale
    the smallest power of two that holds it."""
    x = x.float()
    out = torch.zeros(len(x), 584, dtype=torch.uint8)
    b = x[:, :448].view(-1, 7, 64)
    amax = b.abs().amax(2).double()
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax / 448, 2.0 ** -127))).clamp(-127, 127)
    codes = (b.double() * torch.exp2(-e)[..., None]).float().to(torch.float8_e4m3fn)
    out[:, :448] = codes.flatten(1).view(torch.uint8)
    out[:, 448:576] = x[:, 448:].bfloat16().view(torch.uint8)
    out[:, 576:583] = (e + 127).to(torch.uint8)
    return out


def entry_rows(raw):
    """fp64 [n, 512]: the values of entries uint8 [n, 584], as the gather reads
    them (rounded to bf16, which they fit but for the smallest)."""
    codes = raw[:, :448].contiguous().view(torch.float8_e4m3fn).double()
    scale = torch.exp2(raw[:, 576:583].double() - 127).repeat_interleave(64, 1)
    rope = raw[:, 448:576].contiguous().view(torch.bfloat16).double()
    return torch.cat([(codes * scale).float().bfloat16().double(), rope], 1)


def latent_attention(q, cache, slots, lens, scale):
    T, H, D = q.shape
    flat = cache.reshape(-1, 584)
    out, tol = torch.zeros(T, H, D).double(), torch.zeros(T, H, D).double()
    for t in range(T):
        at = slots[t, :max(0, min(int(lens[t]), slots.shape[1]))]
        at = at[(at >= 0) & (at < len(flat))].long()
        x = entry_rows(flat[at])
        out[t], tol[t] = ref.attend(q[t], x, x, scale)
    return out, tol
