"""The operators on the paged cache held in 4 bits on the GPU against plain forms
(kv4_ref.py): the append, the reading back, the attention, and a run of them."""
import math

import pytest
import torch

import kv4_ref as ref4
import kv_quant_cache_gb300 as kvq
import paged_ref as ref
import workloads as wl

pytestmark = pytest.mark.gpu

NAN = float("nan")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).bfloat16()


def ints(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g, dtype=torch.int32)


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16)


def counter():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---- append -----------------------------------------------------------------------

def append_case(T, Hq, Hkv, D, rot, page, seed):
    g = gen(seed)
    pages = -(-T // page) + 3
    cache = torch.randint(0, 256, (pages, 2, Hkv, page, ref4.held_bytes(D)), generator=g,
                          dtype=torch.uint8)
    qkv = normal(g, T, (Hq + 2 * Hkv) * D)
    slots = torch.randperm(pages * page, generator=g)[:T]
    if T > 2:
        slots[T // 2] = -1
    pos = torch.randint(0, 512, (T,), generator=g)
    table = wl.cos_sin_table(512, rot, 1e4) if rot else None
    return qkv, cache, slots, pos, table


def run_append(case, Hq, Hkv, D, neox, in_place=False, errors=None):
    qkv, cache, slots, pos, table = (None if x is None else x.cuda() for x in case)
    T = qkv.shape[0]
    q_out = None if in_place else torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    kvq.paged_kv4_rope_append(qkv, Hq, Hkv, D, table, neox, pos, slots, cache, q_out=q_out,
                              errors=errors)
    torch.cuda.synchronize()
    return qkv.cpu().view(T, Hq + 2 * Hkv, D), q_out, cache.cpu()


def want_cache(case, Hq, Hkv, D, rot, neox):
    """The cache's bytes after the append, from the tensors before it."""
    qkv, cache, slots, pos, table = case
    T, page = qkv.shape[0], cache.shape[3]
    x = qkv.view(T, Hq + 2 * Hkv, D)
    inside = (pos >= 0) & (pos < 512) if rot else torch.ones(T, dtype=torch.bool)
    k = ref4.rotated_keys(x[:, Hq:Hq + Hkv], table, torch.where(inside, pos, 0), rot, neox)
    codes, scale, zero = ref4.quantise(torch.stack([k, x[:, Hq + Hkv:]], 1))
    new = ref4.raw_of(codes[:, :, :, None].repeat(1, 1, 1, 16, 1),
                      scale[:, :, :, None].repeat(1, 1, 1, 16, 1),
                      zero[:, :, :, None].repeat(1, 1, 1, 16, 1))  # a page of 16 alike, each
    new = new.reshape(T, 2, Hkv, -1)
    out = cache.clone()
    flat = out.view(cache.shape[0], 2, Hkv, -1)
    half, words = page * D // 2, D // ref4.GROUP * 4
    for t in range(T):
        s = int(slots[t])
        if inside[t] and 0 <= s < cache.shape[0] * page:
            o = s % page
            flat[s // page, :, :, o * D // 2:(o + 1) * D // 2] = new[t, :, :, :D // 2]
            flat[s // page, :, :, half + o * words:half + (o + 1) * words] = (
                new[t, :, :, 8 * D:8 * D + words])
    return out


APPENDS = [(1, 4, 1, 128, 128, True, 64), (17, 16, 8, 128, 128, True, 64), (5, 8, 8, 64, 64, False, 16),
           (33, 6, 2, 64, 16, False, 16), (40, 5, 5, 128, 32, True, 32), (19, 7, 1, 256, 256, True, 48),
           (23, 4, 2, 256, 64, False, 128), (300, 3, 3, 64, 48, True, 16), (64, 28, 4, 128, 64, False, 64),
           (9, 4, 2, 128, 0, True, 64), (700, 32, 8, 128, 128, True, 64), (31, 0, 3, 64, 64, True, 16),
           (50, 5, 3, 256, 240, True, 16), (21, 3, 1, 128, 112, True, 80)]


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,neox,page", APPENDS)
def test_append(cuda_device, T, Hq, Hkv, D, rot, neox, page):
    case = append_case(T, Hq, Hkv, D, rot, page, seed=T + D + rot)
    want = want_cache(case, Hq, Hkv, D, rot, neox)
    err = counter()
    x, q_out, cache = run_append(case, Hq, Hkv, D, neox, errors=err)
    assert int(err.item()) == 0
    assert torch.equal(cache, want)
    assert torch.equal(bits(x), bits(case[0].view(x.shape)))
    # the query rows are those of the bf16 append
    like = torch.zeros(case[1].shape[0], 2, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    q2 = torch.empty_like(q_out)
    table = None if case[4] is None else case[4].cuda()
    kvq.paged_kv_rope_append(case[0].cuda(), Hq, Hkv, D, table, neox, case[3].cuda(),
                             case[2].cuda(), like, q_out=q2)
    assert torch.equal(bits(q2), bits(q_out))
    # in place: the same q rows, K and V as they were, the same bytes
    y, _, again = run_append(case, Hq, Hkv, D, neox, in_place=True)
    assert torch.equal(again, want) and torch.equal(bits(y[:, :Hq]), bits(q_out))
    assert torch.equal(bits(y[:, Hq:]), bits(x[:, Hq:]))


def test_append_values_on_the_border(cuda_device):
    """Values on and next to the middle of two codes, scales that round, groups of
    one value, of extremes and of the smallest numbers."""
    T, D = 64, 128
    g = gen(4)
    x = torch.zeros(T, 3, D)
    grid = torch.arange(64) / 4.0  # quotients 0, 1/4, 1/2, .. of a scale of 1
    for t in range(T):
        x[t, 1, :64] = (grid[:64] % 15.25).clamp(max=15) * 2.0 ** (t - 32) + (t % 3) * 2.0 ** (t - 32)
        x[t, 1, 64:] = float(t - 20)
        x[t, 2, :64] = torch.randint(-40, 41, (64,), generator=g) * 2.0 ** (t % 7)
        x[t, 2, 64:] = torch.randn(64, generator=g) * 2.0 ** (-2 * t)
    x[60, 1, 0], x[60, 1, 1] = 1.5e38, -1.5e38
    x[61, 1, :64] = torch.randint(0, 16, (64,), generator=g) * 2.0 ** -133
    x[62, 1, :64] = torch.randint(0, 300, (64,), generator=g) * 2.0 ** -133
    qkv = x.bfloat16().view(T, 3 * D)
    cache = torch.zeros(5, 2, 1, 16, ref4.held_bytes(D), dtype=torch.uint8)
    case = (qkv, cache, torch.randperm(80, generator=g)[:T], torch.zeros(T, dtype=torch.int64), None)
    _, _, got = run_append(case, 1, 1, D, True, in_place=True)
    assert torch.equal(got, want_cache(case, 1, 1, D, 0, True))


def test_append_nonfinite_groups(cuda_device):
    """A NaN or an infinity makes its group NaN, and no other."""
    T, Hkv, D = 6, 2, 128
    case = append_case(T, 2, Hkv, D, 0, 16, seed=6)
    x = case[0].view(T, 6, D)
    x[0, 2, 5], x[1, 5, 70], x[2, 3, 0], x[3, 4, 127] = NAN, math.inf, -math.inf, NAN
    x[4, 2, 3], x[4, 2, 4] = 3e38, -3e38
    case[2][:] = torch.arange(T)
    want = want_cache(case, 2, Hkv, D, 0, True)
    _, _, got = run_append(case, 2, Hkv, D, True, in_place=True)
    assert torch.equal(got, want)
    k, v = (t.cpu() for t in kvq.paged_kv4_gather(got.cuda(), torch.arange(T).cuda()))
    bad = torch.zeros(2, T, Hkv, D, dtype=torch.bool)
    bad[0, 0, 0, :64] = bad[1, 1, 1, 64:] = bad[0, 2, 1, :64] = True
    bad[1, 3, 0, 64:] = bad[0, 4, 0, :64] = True
    assert torch.equal(torch.stack([k, v]).isnan(), bad)


def test_append_rejects_bad_indices(cuda_device):
    T, Hq, Hkv, D, page = 50, 4, 2, 128, 16
    case = append_case(T, Hq, Hkv, D, D, page, seed=3)
    qkv, cache, slots, pos, table = case
    pos[[0, 7]] = torch.tensor([-1, 512])
    pos[20] = 2 ** 40
    slots[[9, 10]] = torch.tensor([cache.shape[0] * page, -2])
    slots[30] = 2 ** 45
    err = counter()
    _, q_out, got = run_append(case, Hq, Hkv, D, True, errors=err)
    assert int(err.item()) == 6
    assert torch.equal(got, want_cache(case, Hq, Hkv, D, D, True))
    bad = (pos < 0) | (pos >= 512)
    assert bool((q_out.cpu()[bad] == 7.0).all()) and not bool((q_out.cpu()[~bad] == 7.0).any())
    _, _, again = run_append(case, Hq, Hkv, D, True)
    assert torch.equal(again, got)


# ---- reading back --------------------------------------------------------------------

@pytest.mark.parametrize("n,Hkv,D,page", [(1, 1, 64, 16), (9, 3, 128, 64), (40, 2, 256, 48),
                                          (1300, 8, 128, 16), (700, 5, 64, 128), (333, 1, 256, 16)])
def test_gather(cuda_device, n, Hkv, D, page):
    g = gen(n + D)
    pages = -(-n // page) + 2
    raw = ref4.random_cache(g, pages, Hkv, page, D)
    slots = torch.randint(0, pages * page, (n,), generator=g)
    slots[n // 2] = -1
    want = ref4.gather(raw, slots)
    err = counter()
    got = kvq.paged_kv4_gather(raw.cuda(), slots.cuda(), errors=err)
    assert int(err.item()) == 0
    for a, b in zip(got, want):
        assert torch.equal(bits(a), bits(b))
    k, v = torch.empty_like(got[0]), torch.empty_like(got[1])
    out = kvq.paged_kv4_gather(raw.cuda(), slots.cuda(), k=k, v=v)
    assert out[0] is k and out[1] is v and torch.equal(bits(k), bits(want[0]))


def test_gather_rejects_bad_slots(cuda_device):
    raw = ref4.random_cache(gen(2), 3, 2, 16, 64)
    slots = torch.tensor([0, 48, -1, -2, 47, 2 ** 40])
    err = counter()
    k, v = kvq.paged_kv4_gather(raw.cuda(), slots.cuda(), errors=err)
    assert int(err.item()) == 3
    want = ref4.gather(raw, slots)
    assert torch.equal(bits(k), bits(want[0])) and torch.equal(bits(v), bits(want[1]))
    k2, _ = kvq.paged_kv4_gather(raw.cuda(), slots.cuda())
    assert torch.equal(bits(k2), bits(k))


# ---- attention -------------------------------------------------------------------------

def attention_case(B, qlen, Hq, Hkv, D, page, width, seed, std=1.5):
    g = gen(seed)
    N = B * width + 2
    raw = ref4.random_cache(g, N, Hkv, page, D)
    table = torch.randperm(N, generator=g)[:B * width].view(B, width).int()
    lens = ints(g, 0, width * page, B * qlen)
    lens[0] = width * page
    return normal(g, B * qlen, Hq, D, std=std), raw, table, lens


def run_attention(q, raw, table, lens, qlen=1, **kw):
    out = kvq.paged_kv4_attention(q.cuda(), raw.cuda(), table.cuda(), lens.cuda(),
                                  tokens_per_request=qlen, **kw)
    torch.cuda.synchronize()
    return out


ATTENTIONS = [(1, 1, 4, 1, 128, 64, 3), (3, 1, 8, 2, 128, 16, 9), (2, 1, 5, 5, 64, 48, 4),
              (2, 1, 32, 2, 64, 16, 40), (1, 1, 8, 1, 256, 32, 11), (4, 3, 4, 2, 128, 16, 7),
              (2, 5, 14, 2, 64, 64, 2), (1, 33, 4, 1, 256, 16, 5), (70, 1, 8, 8, 64, 16, 3),
              (1, 1, 40, 1, 128, 16, 130), (1, 1, 2, 1, 128, 1008, 9), (5, 4, 3, 1, 128, 64, 1),
              (1, 1, 8, 8, 64, 16, 600)]


@pytest.mark.parametrize("B,qlen,Hq,Hkv,D,page,width", ATTENTIONS)
def test_attention(cuda_device, B, qlen, Hq, Hkv, D, page, width):
    q, raw, table, lens = attention_case(B, qlen, Hq, Hkv, D, page, width, seed=B + D + width)
    err = counter()
    out = run_attention(q, raw, table, lens, qlen, errors=err)
    assert int(err.item()) == 0
    ref.check(out, *ref4.attention(q, raw, table, lens, D ** -0.5, qlen))


@pytest.mark.parametrize("length", [0, 1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 255, 257])
def test_attention_lengths(cuda_device, length):
    q, raw, table, _ = attention_case(2, 2, 8, 2, 128, 16, 17, seed=length)
    lens = torch.tensor([max(0, length - 1), length, length, 5], dtype=torch.int32)
    out = run_attention(q, raw, table, lens, 2)
    ref.check(out, *ref4.attention(q, raw, table, lens, 128 ** -0.5, 2))
    for t in range(4):
        if lens[t] == 0:
            assert bool((out[t] == 0).all())


def test_attention_values_of_real_spread(cuda_device):
    """Keys and values with offsets of their own per dim, large scores, a scale of
    zero and one below."""
    g = gen(21)
    B, Hq, Hkv, D, page, width = 2, 8, 2, 128, 16, 20
    x = torch.randn(B * width, 2, Hkv, page, D, generator=g)
    x[:, 0] += 6 * torch.randn(D, generator=g)
    x[:, 1] = x[:, 1] * 0.1 + 3 * torch.randn(D, generator=g)
    raw = ref4.raw_of(*ref4.quantise(x.bfloat16()))
    table = torch.randperm(B * width, generator=g).view(B, width).int()
    lens = torch.tensor([320, 201], dtype=torch.int32)
    for std, scale in ((1.0, None), (6.0, None), (1.0, 0.0), (1.0, -0.3)):
        q = normal(g, B, Hq, D, std=std)
        out = run_attention(q, raw, table, lens, scale=scale)
        want = ref4.attention(q, raw, table, lens, D ** -0.5 if scale is None else scale)
        ref.check(out, *want, f"{std} {scale}")


def test_attention_leaves_out_what_is_not_seen(cuda_device):
    """Whatever stands behind a token's length -- NaN scales in the same page, in
    the same step of 16 keys, seen by other tokens of the request -- does not
    reach it; and what it sees does."""
    g = gen(9)
    qlen, Hq, Hkv, D, page, width = 4, 4, 2, 128, 16, 6
    q, raw, table, _ = attention_case(1, qlen, Hq, Hkv, D, page, width, seed=9)
    lens = torch.tensor([40, 41, 42, 43], dtype=torch.int32)
    want, tol = ref4.attention(q, raw, table, lens, D ** -0.5, qlen)
    words = raw.view(torch.int16)[..., :].view(raw.shape[0], 2, Hkv, -1)
    meta = page * D // 2 // 2  # in 16-bit units
    for key in list(range(43, 96)):
        o = meta + (key % page) * 4
        words[int(table[0, key // page]), :, :, o:o + 4] = 0x7fc0
    ref.check(run_attention(q, raw, table, lens, qlen), want, tol)
    # key 42 is the last token's alone: its values NaN there
    o = meta + (42 % page) * 4
    words[int(table[0, 42 // page]), 1, :, o:o + 4] = 0x7fc0
    out = run_attention(q, raw, table, lens, qlen).cpu()
    assert bool(out[3].isnan().all())
    ref.check(out[:3], want[:3], tol[:3])


def test_attention_rejects_bad_indices(cuda_device):
    q, raw, table, lens = attention_case(6, 1, 8, 2, 64, 16, 5, seed=30)
    lens[:] = torch.tensor([80, -3, 81, 64, 2 ** 31 - 1, 10])
    table[3, 1], table[3, 2], table[5, 3] = raw.shape[0], -1, 2 ** 30
    err = counter()
    out = run_attention(q, raw, table, lens, errors=err)
    assert int(err.item()) > 0
    ref.check(out, *ref4.attention(q, raw, table, lens, 64 ** -0.5))
    again = run_attention(q, raw, table, lens)
    assert torch.equal(bits(again), bits(out))
    # entries past a request's length are not looked at
    q, raw, table, lens = attention_case(2, 1, 4, 2, 64, 16, 9, seed=31)
    lens[:] = torch.tensor([33, 0])
    table[0, 3:] = 2 ** 30
    table[1] = -7
    err = counter()
    out = run_attention(q, raw, table, lens, errors=err)
    assert int(err.item()) == 0
    ref.check(out, *ref4.attention(q, raw, table, lens, 64 ** -0.5))


def test_attention_empty_calls(cuda_device):
    raw = ref4.random_cache(gen(1), 2, 2, 16, 64).cuda()
    none = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    lens = torch.empty(0, dtype=torch.int32, device="cuda")
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert kvq.paged_kv4_attention(q, raw, none, lens).shape == (0, 4, 64)
    q = normal(gen(1), 3, 4, 64).cuda()
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    for width in (0, 2):
        table = torch.zeros(3, width, dtype=torch.int32, device="cuda")
        assert bool((kvq.paged_kv4_attention(q, raw, table, zero) == 0).all())


def test_attention_of_strided_queries(cuda_device):
    q, raw, table, lens = attention_case(3, 2, 6, 2, 128, 32, 4, seed=40)
    packed = torch.zeros(6, 10, 128, dtype=torch.bfloat16)
    packed[:, :6] = q
    view = packed.cuda()[:, :6]
    out = kvq.paged_kv4_attention(view, raw.cuda(), table.cuda(), lens.cuda(),
                                  tokens_per_request=2)
    assert torch.equal(bits(out), bits(run_attention(q, raw, table, lens, 2)))


def test_attention_workspace_stream_and_graph(cuda_device):
    """A long range of one request: partials in a workspace of the caller's, on a
    stream of its own, captured and replayed with other lengths."""
    B, Hq, Hkv, D, page, width = 1, 4, 1, 128, 64, 500
    q, raw, table, lens = attention_case(B, 1, Hq, Hkv, D, page, width, seed=50)
    need = kvq.lib().paged_kv4_attention_workspace(B, 1, Hq, Hkv, D, page, width)
    assert need > 0
    dq, draw, dtable, dlens = q.cuda(), raw.cuda(), table.cuda(), lens.cuda()
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN throughout
    out = torch.empty_like(dq)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        kvq.paged_kv4_attention(dq, draw, dtable, dlens, out=out, workspace=ws)
    side.synchronize()
    ref.check(out, *ref4.attention(q, raw, table, lens, D ** -0.5))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = kvq.paged_kv4_attention(dq, draw, dtable, dlens, workspace=ws)
    for n in (31999, 17, 0, 20000):
        dlens.fill_(n)
        graph.replay()
        torch.cuda.synchronize()
        ref.check(captured, *ref4.attention(q, raw, table, dlens.cpu(), D ** -0.5), str(n))


def test_pinned_tensors(cuda_device):
    q, raw, table, lens = attention_case(2, 1, 4, 2, 64, 16, 200, seed=60)
    out = kvq.paged_kv4_attention(*(x.pin_memory() for x in (q, raw, table, lens)))
    k, v = kvq.paged_kv4_gather(raw.pin_memory(), torch.arange(5).pin_memory())
    torch.cuda.synchronize()
    assert out.is_pinned() and k.is_pinned()
    ref.check(out, *ref4.attention(q, raw, table, lens, 64 ** -0.5))
    assert torch.equal(bits(v), bits(ref4.gather(raw, torch.arange(5))[1]))


# ---- as they are used ------------------------------------------------------------------

def test_prompt_and_decode_steps(cuda_device):
    """A prompt is written and attended to as one chunk, then tokens one by one,
    each appended and attending to all before it."""
    g = gen(70)
    B, Hq, Hkv, D, page, width, prompt = 3, 8, 2, 128, 16, 4, 37
    N = B * width
    cache = torch.zeros(N, 2, Hkv, page, ref4.held_bytes(D), dtype=torch.uint8, device="cuda")
    table = torch.randperm(N, generator=g).view(B, width).int()
    cs = wl.cos_sin_table(64, D, 1e4)
    want = cache.cpu()
    for pos in [list(range(prompt))] + [[p] for p in range(prompt, prompt + 4)]:
        n = len(pos)
        at = torch.tensor(pos).repeat(B)
        req = torch.arange(B).repeat_interleave(n)
        slots = table[req, at // page].long() * page + at % page
        qkv = normal(g, B * n, (Hq + 2 * Hkv) * D)
        q = torch.empty(B * n, Hq, D, dtype=torch.bfloat16, device="cuda")
        kvq.paged_kv4_rope_append(qkv.cuda(), Hq, Hkv, D, cs.cuda(), True, at.cuda(), slots.cuda(),
                                  cache, q_out=q)
        lens = (at + 1).int()
        out = kvq.paged_kv4_attention(q, cache, table.cuda(), lens.cuda(), tokens_per_request=n)
        torch.cuda.synchronize()
        x = qkv.view(B * n, -1, D)
        k = ref4.rotated_keys(x[:, Hq:Hq + Hkv], cs, at, D, True)
        got = ref4.gather(cache.cpu(), slots)
        for mine, theirs in zip(got, (k, x[:, Hq + Hkv:])):
            v = theirs.float().unflatten(-1, (-1, 64))
            step = (v.amax(-1) - v.amin(-1)) / 15
            # half a step, and the roundings of scale, zero and value to bf16
            near = (0.5 * step + 2.0 ** -7 * v.abs().amax(-1))[..., None]
            assert bool(((mine.float().unflatten(-1, (-1, 64)) - v).abs() <= near).all())
        ref.check(out, *ref4.attention(q.cpu(), cache.cpu(), table, lens, D ** -0.5, n))
    assert want.shape == cache.shape
