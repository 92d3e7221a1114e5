"""Tensor-core tiles behind tiles that gave up: a CTA whose wait runs out ends only when
its own copies and matrix instructions have landed, so that the CTAs which get its
shared and tensor memory next, of a call that is enqueued right behind, compute what they
always do.  Limits are set so low that waits which would end well are given up; nothing is
broken to get there."""
import pytest
import torch

import kv4_ref as ref4
import kv_quant_cache_gb300 as kvq

pytestmark = pytest.mark.gpu

LIMITS = [0, 1, 2, 3, 5, 8, 16, 40, 100, 300, 600, 1000, 2000]


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16)


def behind_calls_that_give_up(first, second):
    """``second``'s bits each time it is enqueued behind ``first`` under a low limit."""
    torch.cuda.synchronize()
    want = bits(second())
    got = []
    for limit in LIMITS:
        for _ in range(4):
            old = kvq.set_tile_wait_limit(limit)
            try:
                first()
            finally:
                assert kvq.set_tile_wait_limit(old) == limit
            got.append(second())
    torch.cuda.synchronize()
    assert all(torch.equal(bits(x), want) for x in got)


def latent(T, H, K, seed):
    g = torch.Generator().manual_seed(seed)
    cache = ref4.entries(torch.randn(1000, 512, generator=g).bfloat16()).view(1000, 1, 584)
    q = torch.randn(T, H, 512, generator=g).bfloat16()
    slots = torch.randint(0, 1000, (T, K), generator=g, dtype=torch.int32)
    lens = torch.randint(0, K + 1, (T,), generator=g, dtype=torch.int32)
    args = [q.cuda(), cache.cuda(), slots.cuda(), lens.cuda()]
    return lambda: kvq.dsv4_latent_attention(*args)


@pytest.mark.parametrize("T,H,K", [(3, 64, 1500), (60, 64, 700), (40, 20, 129), (620, 2, 300),
                                   (620, 40, 100)])
def test_latent_tiles(cuda_device, T, H, K):
    behind_calls_that_give_up(latent(T, H, K, seed=T), latent(150, 64, 256, seed=2))


def prefix(D, T, H, keys, seed):
    g = torch.Generator().manual_seed(seed + D)
    page, pages = 64, -(-keys // 64)
    q = torch.randn(T, H, D, generator=g).bfloat16()
    cache = torch.randn(pages + T, 2, H, page, D, generator=g).bfloat16()
    ids = torch.randperm(pages + T, generator=g).int()
    lens = torch.randint(0, 9, (T,), generator=g, dtype=torch.int32)
    args = [q.cuda(), cache.cuda(), ids[:pages].cuda(), keys, ids[pages:].view(T, 1).cuda(),
            lens.cuda()]
    return lambda: kvq.paged_shared_prefix_attention(*args)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefix_tiles(cuda_device, D):
    """Whole blocks of keys, which the copy engine brings, few and many to a CTA."""
    old = kvq.set_config("prefix", 1)
    try:
        for T, H, keys in ((20, 200, 256), (40, 4, 3000)):
            behind_calls_that_give_up(prefix(D, T, H, keys, seed=1), prefix(D, 30, 160, 384, seed=2))
    finally:
        kvq.set_config("prefix", old)
