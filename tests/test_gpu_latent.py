"""Attention over the FP8 latent entries on the GPU against the fp64 form, and
behind the insert that writes them."""
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


def counter():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def case(T, H, K, block, seed, std=1.0):
    g = gen(seed)
    blocks = -(-T * K // block) + 2
    cache = ref4.entries(normal(g, blocks * block, 512)).view(blocks, block, 584)
    slots = torch.randperm(blocks * block, generator=g)[:T * K].view(T, K).int()
    lens = torch.randint(0, K + 1, (T,), generator=g, dtype=torch.int32)
    lens[0] = K
    return normal(g, T, H, 512, std=std), cache, slots, lens


def run(q, cache, slots, lens, **kw):
    out = kvq.dsv4_latent_attention(q.cuda(), cache.cuda(), slots.cuda(), lens.cuda(), **kw)
    torch.cuda.synchronize()
    return out


SHAPES = [(1, 1, 1, 1), (1, 64, 300, 64), (3, 16, 130, 16), (2, 128, 257, 64), (5, 20, 64, 1),
          (2, 8, 1000, 64), (40, 64, 70, 64), (1, 33, 129, 64), (2, 80, 500, 16), (1, 64, 5000, 64),
          (200, 16, 40, 64), (3, 200, 128, 64)]


@pytest.mark.parametrize("T,H,K,block", SHAPES)
def test_latent_attention(cuda_device, T, H, K, block):
    args = case(T, H, K, block, seed=T + H + K)
    err = counter()
    out = run(*args, errors=err)
    assert int(err.item()) == 0
    ref.check(out, *ref4.latent_attention(*args, 512 ** -0.5))


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("length", [0, 1, 2, 63, 64, 65, 127, 128, 129, 191, 256, 257])
def test_lengths(cuda_device, length, H):
    q, cache, slots, lens = case(3, H, 300, 64, seed=length)
    lens[:] = torch.tensor([length, 300, 1])
    out = run(q, cache, slots, lens)
    ref.check(out, *ref4.latent_attention(q, cache, slots, lens, 512 ** -0.5))
    if length == 0:
        assert bool((out[0] == 0).all())


@pytest.mark.parametrize("H", [16, 64])
def test_lists_with_gaps_and_repeats(cuda_device, H):
    q, cache, slots, lens = case(4, H, 400, 64, seed=7)
    g = gen(8)
    slots[torch.rand(4, 400, generator=g) < 0.3] = -1
    slots[1] = -1
    slots[2, :128] = -1      # a first tile without any entry
    slots[3, 5:300] = 17     # one entry many times
    lens[:] = torch.tensor([400, 400, 390, 333])
    err = counter()
    out = run(q, cache, slots, lens, errors=err)
    assert int(err.item()) == 0 and bool((out[1] == 0).all())
    ref.check(out, *ref4.latent_attention(q, cache, slots, lens, 512 ** -0.5))


def test_rejects_bad_indices(cuda_device):
    q, cache, slots, lens = case(5, 64, 200, 64, seed=9)
    n = cache.shape[0] * 64
    slots[0, 3], slots[0, 150], slots[1, 0], slots[2, 199] = n, -2, 2 ** 31 - 1, -2 ** 31
    lens[:] = torch.tensor([200, 200, 201, -1, 2 ** 31 - 1])
    err = counter()
    out = run(q, cache, slots, lens, errors=err)
    assert int(err.item()) > 0
    ref.check(out, *ref4.latent_attention(q, cache, slots, lens, 512 ** -0.5))
    assert torch.equal(bits(run(q, cache, slots, lens)), bits(out))
    # what lies behind a list's length is not read
    lens[:] = 100
    slots[:] = slots.clamp(0, n - 1)
    slots[:, 100:] = 2 ** 30
    err = counter()
    out = run(q, cache, slots, lens, errors=err)
    assert int(err.item()) == 0
    ref.check(out, *ref4.latent_attention(q, cache, slots, lens, 512 ** -0.5))


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("std,scale", [(1.0, 0.0), (1.0, -0.1), (8.0, None), (1e-4, None),
                                       (1.0, 1.0)])
def test_scales_of_scores(cuda_device, std, scale, H):
    q, cache, slots, lens = case(2, H, 500, 64, seed=11, std=std)
    out = run(q, cache, slots, lens, scale=scale)
    ref.check(out, *ref4.latent_attention(q, cache, slots, lens,
                                          512 ** -0.5 if scale is None else scale))


@pytest.mark.parametrize("H", [16, 64])
def test_every_code_and_exponent(cuda_device, H):
    """All finite e4m3 codes under exponents from the least to the greatest that
    leaves the products finite, entry by entry: with one entry the output is the
    entry."""
    n = 60
    cache = torch.zeros(n, 1, 584, dtype=torch.uint8)
    codes = torch.tensor([c for c in range(256) if c & 127 != 127], dtype=torch.uint8)
    for i in range(n):
        cache[i, 0, :448] = codes[(torch.arange(448) + 37 * i) % len(codes)]
        cache[i, 0, 448:576] = normal(gen(i), 64).view(torch.uint8)
        cache[i, 0, 576:583] = torch.tensor([(b * 11 + 3 * i) % 240 for b in range(7)],
                                            dtype=torch.uint8)
    q = torch.zeros(n, H, 512, dtype=torch.bfloat16)
    slots = torch.arange(n).view(n, 1).int()
    out = run(q, cache, slots, torch.ones(n, dtype=torch.int32)).cpu()
    rows = kvq.dsv4_kv_cache_gather(cache.cuda(), torch.arange(n).cuda()).cpu()
    assert torch.equal(out, rows[:, None].expand(n, H, 512))


@pytest.mark.parametrize("H", [16, 64])
def test_nonfinite_entries_reach_their_readers_alone(cuda_device, H):
    q, cache, slots, lens = case(3, H, 200, 64, seed=13)
    lens[:] = 200
    want, tol = ref4.latent_attention(q, cache, slots, lens, 512 ** -0.5)
    flat = cache.view(-1, 584)
    flat[int(slots[1, 150]), 70] = 0x7f  # a NaN code
    out = run(q, cache, slots, lens).cpu()
    assert bool(out[1].isnan().all())
    for t in (0, 2):
        ref.check(out[t], want[t], tol[t])
    # behind the length it is not seen
    lens[1] = 150
    out = run(q, cache, slots, lens)
    ref.check(out, *ref4.latent_attention(q, cache, slots, lens, 512 ** -0.5))
    assert not bool(out.isnan().any())


def test_strided_queries_workspace_stream_and_graph(cuda_device):
    q, cache, slots, lens = case(2, 64, 4000, 64, seed=15)
    want = ref4.latent_attention(q, cache, slots, lens, 512 ** -0.5)
    wide = torch.zeros(2, 70, 512, dtype=torch.bfloat16)
    wide[:, :64] = q
    dc, ds, dl = cache.cuda(), slots.cuda(), lens.cuda()
    view = wide.cuda()[:, :64]
    need = kvq.lib().dsv4_latent_attention_workspace(2, 64, 4000)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN throughout
    out = torch.empty(2, 64, 512, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kvq.dsv4_latent_attention(view, dc, ds, dl, out=out, workspace=ws)
    side.synchronize()
    ref.check(out, *want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = kvq.dsv4_latent_attention(view, dc, ds, dl, workspace=ws)
    for n in ((4000, 3999), (0, 1), (2000, 64)):
        dl.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        ref.check(captured, *ref4.latent_attention(q, cache, slots, dl.cpu(), 512 ** -0.5))


def test_empty_calls(cuda_device):
    cache = torch.zeros(2, 4, 584, dtype=torch.uint8, device="cuda")
    none = torch.empty(0, 5, dtype=torch.int32, device="cuda")
    lens = torch.empty(0, dtype=torch.int32, device="cuda")
    q = torch.empty(0, 8, 512, dtype=torch.bfloat16, device="cuda")
    assert kvq.dsv4_latent_attention(q, cache, none, lens).shape == (0, 8, 512)
    q = normal(gen(1), 2, 8, 512).cuda()
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    slots = torch.empty(2, 0, dtype=torch.int32, device="cuda")
    assert bool((kvq.dsv4_latent_attention(q, cache, slots, lens) == 0).all())


def test_behind_the_insert(cuda_device):
    """Prompt tokens are inserted, then decode steps insert one token each and
    attend, through q_out, to all entries so far."""
    g = gen(17)
    H, block, prompt, more = 64, 16, 50, 3
    total = prompt + more
    cache = torch.zeros(6, block, 584, dtype=torch.uint8, device="cuda")
    qw, kw = (1 + 0.1 * torch.randn(2, 512, generator=g)).bfloat16().cuda()
    cs = wl.cos_sin_table(128, 64, 1e4).cuda()
    order = torch.randperm(6 * block, generator=g)[:total].cuda()
    list_ = order.int().view(1, total)
    for lo, hi in [(0, prompt)] + [(p, p + 1) for p in range(prompt, total)]:
        n = hi - lo
        q, kv = normal(g, n, H, 512).cuda(), normal(g, n, 512).cuda()
        kvq.dsv4_qnorm_rope_kv_rope_quant_insert(
            q, kv, 1e-6, qw, kw, cs, torch.arange(lo, hi, device="cuda"),
            order[lo:hi].contiguous(), cache)
        # every token of the chunk sees those before it
        lens = torch.arange(lo + 1, hi + 1, dtype=torch.int32, device="cuda")
        out = kvq.dsv4_latent_attention(q, cache, list_.expand(n, total).contiguous(), lens)
        torch.cuda.synchronize()
        ref.check(out, *ref4.latent_attention(q.cpu(), cache.cpu(), list_.cpu().expand(n, total),
                                              lens.cpu(), 512 ** -0.5))
