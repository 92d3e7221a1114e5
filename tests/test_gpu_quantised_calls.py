"""Calls of the operators on quantised caches as programs make them: caches past
4 GiB, captured calls side by side, outputs and workspaces of other streams, host
buffers, and sizes where a kernel takes another way."""
import pytest
import torch

import kv4_ref as ref4
import kv_quant_cache_gb300 as kvq
import paged_ref as ref
import workloads as wl

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).bfloat16()


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16)


def kv4_case(B, per, Hq, Hkv, D, page, width, seed):
    g = gen(seed)
    raw = ref4.random_cache(g, B * width + 1, Hkv, page, D)
    table = torch.randperm(B * width + 1, generator=g)[:B * width].view(B, width).int()
    lens = torch.randint(0, width * page + 1, (B * per,), generator=g, dtype=torch.int32)
    lens[0] = width * page
    return normal(g, B * per, Hq, D), raw, table, lens


def latent_case(T, H, K, seed, std=1.0):
    g = gen(seed)
    n = 2 * K + 7
    cache = ref4.entries(normal(g, n, 512)).view(n, 1, 584)
    slots = torch.randint(-1, n, (T, K), generator=g, dtype=torch.int32)
    lens = torch.randint(0, K + 1, (T,), generator=g, dtype=torch.int32)
    lens[-1] = K
    return normal(g, T, H, 512, std=std), cache, slots, lens


def test_a_4_bit_cache_past_4_gib(cuda_device):
    """The same tokens in a small cache and in the last and first pages of one of
    6.4 GB: the same bytes, and the same outputs bit for bit."""
    T, Hq, Hkv, D, page = 200, 8, 4, 128, 64
    g = gen(1)
    small_pages, big_pages = 5, 175000
    small = torch.zeros(small_pages, 2, Hkv, page, 72, dtype=torch.uint8, device="cuda")
    big = torch.empty(big_pages, 2, Hkv, page, 72, dtype=torch.uint8, device="cuda")
    assert big.numel() > 6 * 2 ** 30
    where = torch.tensor([big_pages - 1, 0, big_pages - 2, 116508, 3])  # of the small one's pages
    big[where.cuda()] = 0
    qkv = normal(g, T, (Hq + 2 * Hkv) * D).cuda()
    pos = torch.arange(T).cuda()
    slots = torch.randperm(small_pages * page, generator=g)[:T]
    far = where[slots // page] * page + slots % page
    cs = wl.cos_sin_table(512, 128, 1e4).cuda()
    outs = []
    for cache, s in ((small, slots), (big, far)):
        q = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        kvq.paged_kv4_rope_append(qkv.clone(), Hq, Hkv, D, cs, True, pos, s.cuda(), cache, q_out=q,
                                  errors=err)
        k, v = kvq.paged_kv4_gather(cache, s.cuda(), errors=err)
        pages = torch.arange(small_pages) if cache is small else where
        out = kvq.paged_kv4_attention(q[:4], cache, pages.int().expand(4, 5).contiguous().cuda(),
                                      torch.tensor([320, 1, 300, 77], dtype=torch.int32).cuda(),
                                      errors=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        outs.append([bits(x) for x in (q, k, v, out)])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert torch.equal(big[where.cuda()], small)


def test_latent_entries_past_4_gib(cuda_device):
    H, K, block = 64, 700, 64
    q, cache, slots, lens = latent_case(3, H, K, seed=2)
    n = cache.shape[0]
    blocks = 180000
    big = torch.empty(blocks, block, 584, dtype=torch.uint8, device="cuda")
    assert big.numel() > 6 * 2 ** 30
    far = torch.arange(n) * (blocks * block // n) + blocks * block - 1 - (n - 1) * (
        blocks * block // n)
    assert int(far[0]) >= 0 and int(far[-1]) == blocks * block - 1
    big.view(-1, 584)[far.cuda()] = cache.view(n, 584).cuda()
    moved = torch.where(slots < 0, -1, far[slots.clamp(min=0).long()].int())
    a = kvq.dsv4_latent_attention(q.cuda(), cache.cuda(), slots.cuda(), lens.cuda())
    b = kvq.dsv4_latent_attention(q.cuda(), big, moved.cuda(), lens.cuda())
    torch.cuda.synchronize()
    assert torch.equal(bits(a), bits(b))
    ref.check(a, *ref4.latent_attention(q, cache, slots, lens, 512 ** -0.5))


def test_long_lists_and_tables(cuda_device):
    """List offsets past 4 GiB: rows of 2^28 slots (of which 300 are listed) and of
    2^22 pages."""
    T, width = 6, 1 << 28
    q, cache, slots, lens = latent_case(T, 16, 300, seed=3)
    wide = torch.empty(T, width, dtype=torch.int32, device="cuda")
    wide[:, :300] = slots.cuda()
    got = kvq.dsv4_latent_attention(q.cuda(), cache.cuda(), wide, lens.cuda())
    torch.cuda.synchronize()
    ref.check(got, *ref4.latent_attention(q, cache, slots, lens, 512 ** -0.5))
    del wide
    q, raw, table, lens = kv4_case(300, 1, 2, 2, 64, 16, 3, seed=4)
    wide = torch.empty(300, 1 << 22, dtype=torch.int32, device="cuda")
    wide[:, :3] = table.cuda()
    got = kvq.paged_kv4_attention(q.cuda(), raw.cuda(), wide, lens.cuda())
    torch.cuda.synchronize()
    ref.check(got, *ref4.attention(q, raw, table, lens, 0.125))


def test_captured_calls_side_by_side(cuda_device):
    """Two graphs, of different calls with their workspaces, replayed on two streams at
    the same time."""
    a = kv4_case(2, 1, 8, 2, 128, 64, 100, seed=5)
    b = latent_case(2, 40, 3000, seed=6)
    wants = (ref4.attention(*a, 128 ** -0.5), ref4.latent_attention(*b, 512 ** -0.5))
    args = [[x.cuda() for x in c] for c in (a, b)]
    graphs, outs = [], []
    for f, x in zip((kvq.paged_kv4_attention, kvq.dsv4_latent_attention), args):
        graphs.append([])
        outs.append([])
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):  # (its workspace is of the graph's own pool)
                out = f(*x)
            graphs[-1].append(graph)
            outs[-1].append(out)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for kind in range(2):
            for s, stream in enumerate(streams):
                with torch.cuda.stream(stream):
                    graphs[kind][s].replay()
    torch.cuda.synchronize()
    for out, want in zip(outs, wants):
        ref.check(out[0], *want)
        assert torch.equal(bits(out[0]), bits(out[1]))


def test_calls_on_another_stream_than_their_tensors(cuda_device):
    """``stream`` names another stream than the current one: outputs and workspaces
    that a call allocates are not handed on before that stream is done with them."""
    a = [x.cuda() for x in kv4_case(2, 1, 8, 2, 128, 64, 100, seed=7)]
    b = [x.cuda() for x in latent_case(2, 40, 3000, seed=8)]
    slots = torch.arange(500).cuda()
    want = (bits(kvq.paged_kv4_attention(*a)), bits(kvq.dsv4_latent_attention(*b)),
            bits(kvq.paged_kv4_gather(a[1], slots)[0]))
    side = torch.cuda.Stream()
    for _ in range(5):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(3000000)
        got = (kvq.paged_kv4_attention(*a, stream=side.cuda_stream),
               kvq.dsv4_latent_attention(*b, stream=side.cuda_stream),
               kvq.paged_kv4_gather(a[1], slots, stream=side.cuda_stream)[0])
        taken = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(40)]
        torch.cuda.synchronize()
        assert all(torch.equal(bits(x), w) for x, w in zip(got, want))
        assert all(bool((x == 7).all()) for x in taken)


def test_latent_attention_on_pinned_tensors(cuda_device):
    for T, H, K in ((2, 20, 300), (1, 64, 50)):
        host = latent_case(T, H, K, seed=T + H)
        got = kvq.dsv4_latent_attention(*(x.pin_memory() for x in host))
        torch.cuda.synchronize()
        assert got.is_pinned()
        ref.check(got, *ref4.latent_attention(*host, 512 ** -0.5))


@pytest.mark.parametrize("T,H,K", [(304, 128, 300), (305, 128, 300), (608, 1, 129), (609, 1, 129),
                                   (700, 33, 128), (1500, 16, 10), (152, 64, 257), (151, 65, 1)])
def test_latent_tokens_around_what_is_shared_out(cuda_device, T, H, K):
    """Up to 608 blocks of heads are shared out over the SMs, more are a CTA each."""
    host = latent_case(T, H, K, seed=T + H + K)
    args = [x.cuda() for x in host]
    got = kvq.dsv4_latent_attention(*args)
    torch.cuda.synchronize()
    some = torch.cat([torch.arange(3), torch.randint(3, T, (20,), generator=gen(T)),
                      torch.tensor([T - 1])])
    ref.check(got[some.cuda()], *ref4.latent_attention(host[0][some], host[1], host[2][some],
                                                        host[3][some], 512 ** -0.5))
    assert torch.equal(bits(got), bits(kvq.dsv4_latent_attention(*args)))


@pytest.mark.parametrize("H", [16, 30, 64, 100])
def test_latent_lengths_of_many_tokens(cuda_device, H):
    """Enough tokens that their blocks of heads are as wide as they get: lengths around
    the tiles' ends, lists with gaps, a token without an entry, and a NaN entry that
    reaches its readers alone."""
    ends = [0, 1, 2, 63, 64, 65, 127, 128, 129, 191, 256, 257, 300]
    T = 6 * len(ends)
    q, cache, slots, lens = latent_case(T, H, 300, seed=H)
    lens[:] = torch.tensor(ends * 6, dtype=torch.int32)
    slots[5] = -1
    slots[3, :10] = -1
    slots[8, :128] = -1
    slots[slots == 77] = 78
    bad = [17, 38, 77]
    slots[bad, 0] = 77
    args = [x.cuda() for x in (q, cache, slots, lens)]
    want = ref4.latent_attention(q, cache, slots, lens, 512 ** -0.5)
    ref.check(kvq.dsv4_latent_attention(*args), *want)
    args[1][77, 0, 130] = 0x7f  # a NaN code
    got = kvq.dsv4_latent_attention(*args).cpu()
    seen = torch.zeros(T, dtype=torch.bool)
    seen[bad] = True
    assert bool(got[seen].isnan().all())
    ref.check(got[~seen], want[0][~seen], want[1][~seen])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("per,G", [(1, 1), (1, 8), (3, 3), (2, 8), (17, 1), (4, 8), (33, 1), (9, 7)])
def test_rows_of_a_tile(cuda_device, D, per, G):
    """8, 16 or 32 rows to a tile, full and partly filled, over one and several tiles."""
    host = kv4_case(3, per, 2 * G, 2, D, 32, 11, seed=D + per + G)
    got = kvq.paged_kv4_attention(*(x.cuda() for x in host), tokens_per_request=per)
    torch.cuda.synchronize()
    ref.check(got, *ref4.attention(*host, D ** -0.5, per_request=per))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_scores_far_apart(cuda_device, D):
    """Keys whose scores grow along the sequence: the softmax's reference moves again
    and again, and what came before is scaled down to nothing. Scores are multiples
    of 64 and exact, so weights are one or below 2^-90: out is the mean of the values
    with the greatest score of those seen, within the rounding of their scales (each
    value's product with its scale is rounded once to bf16) and of the output, and of
    the log2 of a part's sum, of a size below 2^14: 2^-11 in units of log2, twice."""
    page, width, Hkv = 16, 70, 2
    n = page * width
    g = gen(D)
    x = normal(g, width, 2, Hkv, page, D)
    codes, scale, zero = ref4.quantise(x)
    codes[:, 0], scale[:, 0], zero[:, 0] = 8, 0, 0  # keys: zeros, but for the first group's
    level = (torch.arange(n) // 7 * 64).view(width, page)
    zero[:, 0, :, :, 0] = level[:, None].expand(width, Hkv, page).bfloat16()
    level = zero[:, 0, 0, :, 0].double().flatten()  # as rounded to bf16: still growing
    raw = ref4.raw_of(codes, scale, zero)
    lens = torch.tensor([1, 6, 7, 8, 300, 777, n - 1, n], dtype=torch.int32)
    q = torch.zeros(8, 4, D, dtype=torch.bfloat16)
    q[:, :, 5] = 1.0
    table = torch.arange(width).int().expand(8, width).contiguous()
    got = kvq.paged_kv4_attention(q.cuda(), raw.cuda(), table.cuda(), lens.cuda(), scale=1.0)
    torch.cuda.synchronize()
    c = ref4.Cache(raw)
    at = torch.arange(n)
    want, tol = torch.zeros(8, 4, D).double(), torch.zeros(8, 4, D).double()
    for h in range(4):
        sn, z, s = c.terms(at // page, at % page, h // 2)
        for t, m in enumerate(lens.tolist()):
            top = level[:m] == level[:m].max()
            v = (sn[:m, 1] + z[:m, 1])[top]
            want[t, h] = v.mean(0)
            tol[t, h] = (ref4.EPS_BF16 * (sn[:m, 1][top].abs().mean(0) + want[t, h].abs())
                         + 2.0 ** -10 * (sn[:m, 1].abs() + z[:m, 1].abs()).amax(0))
    ref.check(got, want, tol)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0, 1e-30])
@pytest.mark.parametrize("D,per", [(64, 3), (128, 1), (256, 2)])
def test_scales_of_4_bit_scores(cuda_device, D, per, scale):
    host = kv4_case(3, per, 8, 2, D, 16, 40, seed=D + per)
    got = kvq.paged_kv4_attention(*(x.cuda() for x in host), tokens_per_request=per, scale=scale)
    torch.cuda.synchronize()
    ref.check(got, *ref4.attention(*host, scale, per_request=per))


def test_the_largest_pages(cuda_device):
    """65536 tokens to a page: written, read back and attended to on both sides of the
    boundary of two pages."""
    page, Hq, Hkv, D = 65536, 4, 2, 64
    g = gen(9)
    raw = ref4.random_cache(g, 3, Hkv, page, D)
    table = torch.tensor([[2, 0], [1, 2]], dtype=torch.int32)
    at = torch.tensor([0, 1, page - 1, page, page + 1, 2 * page - 1])
    slots = table[0].long()[at // page] * page + at % page
    qkv = normal(g, len(at), (Hq + 2 * Hkv) * D)
    cache = raw.cuda()
    kvq.paged_kv4_rope_append(qkv.cuda(), Hq, Hkv, D, None, True, None, slots.cuda(), cache)
    torch.cuda.synchronize()
    k, v = qkv.view(-1, Hq + 2 * Hkv, D)[:, Hq:].split(Hkv, 1)
    codes = ref4.Cache(raw).codes.clone()
    got = ref4.Cache(cache.cpu())
    for which, rows in ((0, k), (1, v)):
        codes[slots // page, which, :, slots % page] = ref4.quantise(rows)[0]
    assert torch.equal(got.codes, codes)
    back = kvq.paged_kv4_gather(cache, slots.cuda())
    for x, want in zip(back, ref4.gather(cache.cpu(), slots)):
        assert torch.equal(x.cpu(), want)
    q = normal(g, 6, Hq, D)
    lens = torch.tensor([page - 1, page, page + 1, 2 * page, 17, 0], dtype=torch.int32)
    out = kvq.paged_kv4_attention(q.cuda(), cache, table.cuda(), lens.cuda(), tokens_per_request=3)
    torch.cuda.synchronize()
    ref.check(out, *ref4.attention(q, cache.cpu(), table, lens, D ** -0.5, per_request=3))


@pytest.mark.parametrize("D,per,G", [(64, 1, 8), (64, 3, 8), (64, 4, 8), (128, 1, 4), (128, 2, 8),
                                     (128, 3, 8), (256, 1, 4), (256, 2, 8)])
def test_pages_outside_the_cache_among_seen_keys(cuda_device, D, per, G):
    """Every seventh page or so lies outside the cache, behind each other and alone, in
    long ranges that every row sees: they are left out, and counted."""
    q, raw, table, lens = kv4_case(2, per, 2 * G, 2, D, 16, 300, seed=D + per)
    g = gen(10)
    table[torch.rand(2, 300, generator=g) < 0.15] = raw.shape[0]
    table[0, 40:48] = -1
    lens[:] = torch.randint(4600, 4801, (2 * per,), generator=g, dtype=torch.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = kvq.paged_kv4_attention(q.cuda(), raw.cuda(), table.cuda(), lens.cuda(),
                                  tokens_per_request=per, errors=err)
    torch.cuda.synchronize()
    assert int(err.item()) > 0
    ref.check(got, *ref4.attention(q, raw, table, lens, D ** -0.5, per_request=per))
