"""What a 4-bit cache holds after appends, whole: the slots that were written, codes, scales
and zeros, and those that were not."""
import pytest
import torch

import kv4_ref as ref4
import kv_quant_cache_gb300 as kvq
import workloads as wl

pytestmark = pytest.mark.gpu


def written(parts, slots, k, v, page):
    """``parts`` (codes, scale, zero of the cache before) after k and v [n, Hkv, D] at ``slots``."""
    for which, rows in ((0, k), (1, v)):
        for held, new in zip(parts, ref4.quantise(rows)):
            held[slots // page, which, :, slots % page] = new
    return ref4.raw_of(*parts)


def taken_apart(raw):
    c = ref4.Cache(raw)
    return [x.contiguous() for x in (c.codes, c.scale.bfloat16(), c.zero.bfloat16())]


@pytest.mark.parametrize("D,page,rot,neox", [(128, 16, 128, True), (64, 32, 16, False), (256, 48, 128, True)])
def test_a_prompt_and_decode_steps(cuda_device, D, page, rot, neox):
    """A prompt and tokens one by one into a cache that holds others already: after each step
    its bytes are those of the plain form, in the slots of that step and everywhere else."""
    g = torch.Generator().manual_seed(D)
    B, Hq, Hkv, prompt = 3, 8, 2, 37
    width = -(-(prompt + 4) // page)
    N = B * width + 2
    raw = ref4.random_cache(g, N, Hkv, page, D)
    parts, cache = taken_apart(raw), raw.cuda()
    assert torch.equal(ref4.raw_of(*parts), raw)
    table = torch.randperm(N, generator=g)[:B * width].view(B, width)
    cs = wl.cos_sin_table(64, rot, 1e4)
    for pos in [list(range(prompt))] + [[p] for p in range(prompt, prompt + 4)]:
        at = torch.tensor(pos).repeat(B)
        slots = table[torch.arange(B).repeat_interleave(len(pos)), at // page] * page + at % page
        qkv = torch.randn(len(at), (Hq + 2 * Hkv) * D, generator=g).bfloat16()
        kvq.paged_kv4_rope_append(qkv.cuda(), Hq, Hkv, D, cs.cuda(), neox, at.cuda(), slots.cuda(),
                                  cache)
        torch.cuda.synchronize()
        x = qkv.view(len(at), -1, D)
        k = ref4.rotated_keys(x[:, Hq:Hq + Hkv], cs, at, rot, neox)
        assert torch.equal(cache.cpu(), written(parts, slots, k, x[:, Hq + Hkv:], page))


def test_the_largest_pages(cuda_device):
    """65536 tokens to a page: codes, scales and zeros on both sides of the boundary of two pages,
    and nothing else written."""
    page, Hq, Hkv, D = 65536, 4, 2, 64
    g = torch.Generator().manual_seed(9)
    raw = ref4.random_cache(g, 3, Hkv, page, D)
    at = torch.tensor([0, 1, page - 1, page, page + 1, 2 * page - 1])
    slots = torch.tensor([2, 0])[at // page] * page + at % page
    qkv = torch.randn(len(at), (Hq + 2 * Hkv) * D, generator=g).bfloat16()
    cache = raw.cuda()
    kvq.paged_kv4_rope_append(qkv.cuda(), Hq, Hkv, D, None, True, None, slots.cuda(), cache)
    torch.cuda.synchronize()
    k, v = qkv.view(-1, Hq + 2 * Hkv, D)[:, Hq:].split(Hkv, 1)
    assert torch.equal(cache.cpu(), written(taken_apart(raw), slots, k, v, page))
