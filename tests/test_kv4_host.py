"""The operators on quantised caches on the host: validation by the C ABI and by
the Python binding, workspace sizes, and the plain forms the GPU tests compare
with.  No call here reaches a kernel launch."""
import math

import pytest
import torch

import kv4_ref as ref4
import kv_quant_cache_gb300 as kvq
from kv_quant_cache_gb300 import _build

A = 0x10000    # fake, never-dereferenced device addresses
MIS = 0x10002


@pytest.fixture(scope="module")
def L():
    _build.build()
    return kvq.lib()


def rejected(status):
    """The call came back from validation (and launched nothing)."""
    assert status not in (kvq.KVQ_OK, kvq.KVQ_ERR_CUDA)
    return status


def append(L, qkv=A, q_out=None, T=4, Hq=4, Hkv=2, D=128, cs=A, max_pos=16, rot=128, neox=1,
           pos=A, slots=A, cache=A, pages=8, page=16, err=None):
    return L.paged_kv4_rope_append(qkv, q_out, T, Hq, Hkv, D, cs, max_pos, rot, neox, pos, slots,
                                   cache, pages, page, err, None)


def gather(L, cache=A, pages=8, Hkv=2, page=16, D=128, slots=A, n=3, k=0x400000, v=0x500000,
           err=None):
    return L.paged_kv4_gather(cache, pages, Hkv, page, D, slots, n, k, v, err, None)


def attend(L, q=A, stride=512, T=4, per=2, Hq=4, Hkv=2, D=128, cache=A, pages=8, page=16, table=A,
           width=5, lens=A, scale=0.1, out=0x900000, ws=0x800000, ws_bytes=1 << 40, err=None):
    return L.paged_kv4_attention(q, stride, T, per, Hq, Hkv, D, cache, pages, page, table, width,
                                 lens, scale, out, ws, ws_bytes, err, None)


def latent(L, q=A, stride=2048, T=4, H=4, cache=A, blocks=8, block=64, slots=A, width=300, lens=A,
           scale=0.1, out=0x900000, ws=0x800000, ws_bytes=1 << 40, err=None):
    return L.dsv4_latent_attention(q, stride, T, H, cache, blocks, block, slots, width, lens, scale,
                                   out, ws, ws_bytes, err, None)


def test_append_validation(L):
    bad = lambda **k: rejected(append(L, **k))  # noqa: E731
    for name in ("qkv", "cs", "pos", "slots", "cache"):
        assert bad(**{name: None}) == kvq.KVQ_ERR_NULL
        assert bad(**{name: MIS}) == kvq.KVQ_ERR_ALIGN
    assert bad(q_out=MIS) == kvq.KVQ_ERR_ALIGN and bad(err=MIS + 1) == kvq.KVQ_ERR_ALIGN
    for k in (dict(T=-1), dict(Hq=-1), dict(Hkv=0), dict(page=0), dict(page=65552),
              dict(pages=-1), dict(pages=2 ** 31), dict(max_pos=-1), dict(T=2 ** 31),
              dict(T=2 ** 30), dict(T=2 ** 62), dict(Hq=2 ** 31 - 1), dict(Hkv=2 ** 31 - 1)):
        assert bad(**k) == kvq.KVQ_ERR_SHAPE, k
    for k in (dict(D=32), dict(D=96), dict(D=512), dict(page=8), dict(page=24), dict(neox=2),
              dict(rot=8), dict(rot=24), dict(rot=144), dict(rot=-16)):
        assert bad(**k) == kvq.KVQ_ERR_UNSUPPORTED, k
    nbytes = 4 * 8 * 128 * 2
    for at in (A, A + 16, A + nbytes - 16, A - 16):
        assert bad(q_out=at) == kvq.KVQ_ERR_VALUE
    assert append(L, T=0, qkv=None, cs=None, pos=None, slots=None, cache=None) == kvq.KVQ_OK
    assert bad(rot=0, cs=None, pos=None, cache=None) == kvq.KVQ_ERR_NULL


def test_gather_validation(L):
    bad = lambda **k: rejected(gather(L, **k))  # noqa: E731
    for name in ("cache", "slots", "k", "v"):
        assert bad(**{name: None}) == kvq.KVQ_ERR_NULL
        assert bad(**{name: MIS}) == kvq.KVQ_ERR_ALIGN
    assert bad(err=MIS) == kvq.KVQ_ERR_ALIGN
    for k in (dict(n=-1), dict(n=2 ** 31), dict(n=2 ** 30), dict(n=2 ** 62), dict(Hkv=0),
              dict(page=0), dict(page=65552), dict(pages=-1), dict(pages=2 ** 31)):
        assert bad(**k) == kvq.KVQ_ERR_SHAPE, k
    for k in (dict(D=32), dict(D=192), dict(page=40)):
        assert bad(**k) == kvq.KVQ_ERR_UNSUPPORTED, k
    nbytes = 3 * 2 * 128 * 2
    for at in (0x400000, 0x400000 + nbytes - 16, 0x400000 - nbytes + 16):
        assert bad(v=at) == kvq.KVQ_ERR_VALUE
    assert gather(L, n=0, cache=None, slots=None, k=None, v=None) == kvq.KVQ_OK


def test_attention_validation(L):
    bad = lambda **k: rejected(attend(L, **k))  # noqa: E731
    for name in ("q", "cache", "table", "lens", "out"):
        assert bad(**{name: None}) == kvq.KVQ_ERR_NULL
        assert bad(**{name: MIS}) == kvq.KVQ_ERR_ALIGN
    assert bad(err=MIS) == bad(stride=516) == kvq.KVQ_ERR_ALIGN
    for k in (dict(T=-1), dict(T=2 ** 31), dict(T=2 ** 62), dict(T=2 ** 29), dict(Hq=3), dict(Hq=0),
              dict(Hkv=0), dict(page=0), dict(pages=-1), dict(width=-1), dict(width=2 ** 22 + 1),
              dict(per=0), dict(per=-2), dict(per=3), dict(per=2 ** 62), dict(stride=511),
              dict(stride=2 ** 40), dict(T=2 ** 28, per=1)):
        assert bad(**k) == kvq.KVQ_ERR_SHAPE, k
    for k in (dict(D=96), dict(page=8), dict(page=20)):
        assert bad(**k) == kvq.KVQ_ERR_UNSUPPORTED, k
    for scale in (math.nan, math.inf, -math.inf, 2.5e38, -3.4e38):
        assert bad(scale=scale) == kvq.KVQ_ERR_VALUE
    for at in (A, A + 1024, A - 1024):  # out over q
        assert bad(out=at) == kvq.KVQ_ERR_VALUE
    assert attend(L, T=0, q=None, cache=None, table=None, lens=None, out=None) == kvq.KVQ_OK
    # without pages no table is asked for
    assert bad(width=0, table=None, lens=None) == kvq.KVQ_ERR_NULL
    # sizes whose call needs a workspace: a long range that few rows see
    long = dict(T=1, per=1, Hq=4, Hkv=1, page=64, width=8192)
    need = L.paged_kv4_attention_workspace(1, 1, 4, 1, 128, 64, 8192)
    assert need > 0 and need % 16 == 0
    assert bad(ws=None, **long) == kvq.KVQ_ERR_NULL
    assert bad(ws=MIS, **long) == kvq.KVQ_ERR_ALIGN
    assert bad(ws_bytes=need - 1, **long) == bad(ws_bytes=-1, **long) == kvq.KVQ_ERR_SHAPE


def test_latent_validation(L):
    bad = lambda **k: rejected(latent(L, **k))  # noqa: E731
    for name in ("q", "cache", "slots", "lens", "out", "ws"):
        assert bad(**{name: None}) == kvq.KVQ_ERR_NULL, name
        assert bad(**{name: MIS}) == kvq.KVQ_ERR_ALIGN, name
    assert bad(err=MIS) == bad(stride=2052) == bad(cache=A + 4) == kvq.KVQ_ERR_ALIGN
    for k in (dict(T=-1), dict(T=2 ** 31), dict(T=2 ** 62), dict(T=2 ** 29), dict(H=0), dict(H=-1),
              dict(H=65537), dict(blocks=-1), dict(blocks=2 ** 31), dict(block=0), dict(block=-1),
              dict(width=-1), dict(width=2 ** 30 + 1), dict(width=2 ** 62), dict(stride=2040),
              dict(stride=2 ** 40)):
        assert bad(**k) == kvq.KVQ_ERR_SHAPE, k
    for scale in (math.nan, math.inf, -math.inf, 2.5e38, -3.4e38):
        assert bad(scale=scale) == kvq.KVQ_ERR_VALUE
    for at in (A, A + 4096, A - 4096):
        assert bad(out=at) == kvq.KVQ_ERR_VALUE
    need = L.dsv4_latent_attention_workspace(4, 4, 300)
    assert need > 0 and need % 16 == 0
    assert bad(ws_bytes=need - 1) == bad(ws_bytes=-1) == kvq.KVQ_ERR_SHAPE
    assert latent(L, T=0, q=None, cache=None, slots=None, lens=None, out=None) == kvq.KVQ_OK
    assert bad(width=0, slots=None, lens=None) == kvq.KVQ_ERR_NULL


def test_workspace_sizes(L):
    f, g = L.paged_kv4_attention_workspace, L.dsv4_latent_attention_workspace
    for args in ((0, 1, 4, 2, 128, 16, 3), (4, 0, 4, 2, 128, 16, 3), (4, 3, 4, 2, 128, 16, 3),
                 (4, 2, 3, 2, 128, 16, 3), (4, 2, 4, 0, 128, 16, 3), (4, 2, 4, 2, 96, 16, 3),
                 (4, 2, 4, 2, 128, 8, 3), (4, 2, 4, 2, 128, 16, -1), (2 ** 31, 1, 1, 1, 64, 16, 1),
                 (4, 2 ** 40, 4, 2, 128, 16, 3), (4, 2, 4, 2, 128, 16, 2 ** 22 + 1)):
        assert f(*args) == 0, args
    for args in ((0, 4, 10), (-1, 4, 10), (4, 0, 10), (4, 4, -1), (4, 4, 2 ** 30 + 1),
                 (2 ** 31, 1, 10), (2 ** 30, 8, 10)):
        assert g(*args) == 0, args
    # one range, many rows, short lists: none is needed
    assert f(4, 2, 4, 2, 128, 16, 0) == f(256, 1, 32, 8, 128, 64, 8) == 0
    assert g(4, 4, 0) == g(1, 64, 128) == g(5000, 128, 2048) == 0
    # two partial rows of 512 sums, a reference and a sum of weights per head and CTA
    assert g(1, 64, 4096) == 128 * 2 * 16 * 514 * 4  # of four times 16 heads
    assert g(2, 64, 4096) == 128 * 2 * 32 * 514 * 4
    assert g(8, 64, 4096) == 152 * 2 * 64 * 514 * 4
    assert g(64, 64, 2048) == 152 * 2 * 64 * 514 * 4
    assert g(64, 20, 2048) == 152 * 2 * 32 * 514 * 4


def test_binding_checks():
    cache = torch.zeros(4, 2, 2, 16, 36, dtype=torch.uint8)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    ids = torch.zeros(3, dtype=torch.int64)
    qkv = torch.zeros(3, 8 * 64, dtype=torch.bfloat16)
    cs = torch.zeros(9, 64)
    lq = torch.zeros(3, 4, 512, dtype=torch.bfloat16)
    entries = torch.zeros(2, 64, 584, dtype=torch.uint8)
    slots = torch.zeros(3, 5, dtype=torch.int32)
    calls = [
        lambda: kvq.paged_kv4_rope_append(qkv[:, 64:], 4, 2, 64, cs, True, ids, ids, cache),
        lambda: kvq.paged_kv4_rope_append(qkv, 4, 2, 64, cs, True, ids, ids, cache[:, :1]),
        lambda: kvq.paged_kv4_rope_append(qkv, 4, 2, 64, cs, True, ids, ids, cache[..., :32]),
        lambda: kvq.paged_kv4_rope_append(qkv, 4, 2, 64, cs, True, ids, ids, cache[0]),
        lambda: kvq.paged_kv4_rope_append(qkv, 4, 2, 64, cs, True, ids[:2], ids, cache),
        lambda: kvq.paged_kv4_rope_append(qkv, 4, 2, 64, cs, True, ids, ids[:2], cache),
        lambda: kvq.paged_kv4_rope_append(qkv, 4, 2, 64, cs, True, ids, ids, cache, q_out=q[:2]),
        lambda: kvq.paged_kv4_rope_append(qkv, 4, 2, 64, cs, True, ids, ids, cache, rotary_dim=32),
        lambda: kvq.paged_kv4_rope_append(qkv, 4, 2, 64, None, True, ids, ids, cache,
                                          rotary_dim=32),
        lambda: kvq.paged_kv4_gather(cache, ids[None]),
        lambda: kvq.paged_kv4_gather(cache, lens),
        lambda: kvq.paged_kv4_gather(cache[:, :, :, :, :35], ids),
        lambda: kvq.paged_kv4_gather(cache, ids, k=torch.zeros(3, 2, 32, dtype=torch.bfloat16)),
        lambda: kvq.paged_kv4_attention(q[..., :32], cache, table, lens),
        lambda: kvq.paged_kv4_attention(q.float(), cache, table, lens),
        lambda: kvq.paged_kv4_attention(q, cache, table[:2], lens),
        lambda: kvq.paged_kv4_attention(q, cache, table, lens, tokens_per_request=3),
        lambda: kvq.paged_kv4_attention(q, cache, table, lens, tokens_per_request=0),
        lambda: kvq.paged_kv4_attention(q, cache, table[0], lens),
        lambda: kvq.paged_kv4_attention(q, cache, table, lens[:2]),
        lambda: kvq.paged_kv4_attention(q, cache, table, lens, out=q[:2]),
        lambda: kvq.dsv4_latent_attention(lq[..., :256], entries, slots, lens),
        lambda: kvq.dsv4_latent_attention(lq.float(), entries, slots, lens),
        lambda: kvq.dsv4_latent_attention(lq, entries[..., :576], slots, lens),
        lambda: kvq.dsv4_latent_attention(lq, entries[0], slots, lens),
        lambda: kvq.dsv4_latent_attention(lq, entries, slots[:2], lens),
        lambda: kvq.dsv4_latent_attention(lq, entries, slots[0], lens),
        lambda: kvq.dsv4_latent_attention(lq, entries, slots, lens[:2]),
        lambda: kvq.dsv4_latent_attention(lq, entries, slots, lens, out=lq[:, :3]),
        # everything in order, but on the host and not pinned
        lambda: kvq.paged_kv4_rope_append(qkv, 4, 2, 64, cs, True, ids, ids, cache),
        lambda: kvq.paged_kv4_gather(cache, ids),
        lambda: kvq.paged_kv4_attention(q, cache, table, lens),
        lambda: kvq.dsv4_latent_attention(lq, entries, slots, lens),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was accepted")


def test_values_of_the_plain_cache():
    """What is read back lies within half a step and the roundings of scale, zero and
    value of what went in; the ends of a group's range have the codes 0 and 15."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(3, 2, 2, 16, 128, generator=g).bfloat16()
    codes, scale, zero = ref4.quantise(x)
    raw = ref4.raw_of(codes, scale, zero)
    assert raw.shape == (3, 2, 2, 16, 72) and raw.dtype == torch.uint8
    k, v = ref4.gather(raw, torch.arange(48))
    want = x.permute(1, 0, 3, 2, 4).reshape(2, 48, 2, 128).double()
    got = torch.stack([k, v]).double()
    grouped = want.unflatten(-1, (2, 64))
    step = (grouped.amax(-1) - grouped.amin(-1)) / 15
    size = grouped.abs().amax(-1)
    # half a step; the scale's and the zero's rounding, times up to 8 codes and once
    # (of up to size + 8 steps); the value's
    tol = 0.5 * step + 2.0 ** -8 * (8 * step + (size + 8 * step) + size) + 2.0 ** -20 * size
    tol = tol.repeat_interleave(64, -1)
    assert bool(((got - want).abs() <= tol).all())
    assert int(codes.min()) == 0 and int(codes.max()) == 15
    # equal values: a scale of zero
    same = torch.full((1, 2, 1, 16, 64), 1.5, dtype=torch.bfloat16)
    c, s, z = ref4.quantise(same)
    assert bool((c == 8).all()) and bool((s == 0).all()) and bool((z == 1.5).all())


def test_plain_attention_agrees_with_torch():
    g = torch.Generator().manual_seed(4)
    raw = ref4.random_cache(g, 6, 2, 16, 64)
    q = torch.randn(4, 4, 64, generator=g).bfloat16()
    table = torch.tensor([[4, 1, 2], [3, 0, 5]], dtype=torch.int32)
    lens = torch.tensor([40, 48, 1, 0], dtype=torch.int32)
    out, tol = ref4.attention(q, raw, table, lens, 0.125, per_request=2)
    assert bool((out[3] == 0).all()) and bool((tol[:3] > 0).all())
    c = ref4.Cache(raw)
    for t in range(3):
        n = int(lens[t])
        at = torch.arange(n)
        pages = table[t // 2].long()[at // 16]
        for h in range(4):
            sn, z, s = c.terms(pages, at % 16, h // 2)
            k, v = sn[:, 0] + z[:, 0], sn[:, 1] + z[:, 1]
            w = torch.softmax(k @ q[t, h].double() * 0.125, 0)
            assert torch.allclose(w @ v, out[t, h], rtol=0, atol=1e-12)


def test_plain_latent_attention_agrees_with_torch():
    g = torch.Generator().manual_seed(5)
    x = torch.randn(20, 512, generator=g).bfloat16()
    raw = ref4.entries(x)
    rows = ref4.entry_rows(raw)
    assert torch.equal(rows[:, 448:], x[:, 448:].double())
    # e4m3: three bits behind the point, or half a step at the bottom of a block
    size = x.double()[:, :448].abs()
    low = size.view(20, 7, 64).amax(-1).repeat_interleave(64, 1) * 2.0 ** -16
    assert bool(((rows[:, :448] - x.double()[:, :448]).abs() <= size * 2.0 ** -4 + low).all())
    q = torch.randn(2, 3, 512, generator=g).bfloat16()
    slots = torch.tensor([[3, -1, 3, 9, 0], [-1, 5, 25, 7, 1]], dtype=torch.int32)
    lens = torch.tensor([4, 3], dtype=torch.int32)
    out, _ = ref4.latent_attention(q, raw.view(2, 10, 584), slots, lens, 0.05)
    for t, at in ((0, [3, 3, 9]), (1, [5])):
        w = torch.softmax(q[t].double() @ rows[at].T * 0.05, -1)
        assert torch.allclose(w @ rows[at], out[t], rtol=0, atol=1e-12)
