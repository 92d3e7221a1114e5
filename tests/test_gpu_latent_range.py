"""Attention over latent entries where scores lie far apart or far out: exact
answers, as a row of weights is then ones and zeros."""
import pytest
import torch

import kv4_ref as ref4
import kv_quant_cache_gb300 as kvq
import paged_ref as ref

pytestmark = pytest.mark.gpu

# Scores (the first rotary dim's products, exact in fp32) by their place in a list;
# further ones repeat the one before. Tiles are 128 entries, so most of these raise the
# maximum of a tile that has begun or of tiles before it.
RISING = {0: -2.0 ** 100, 1: -2.0 ** 90, 5: 0.0, 100: 64.0, 130: 128.0, 300: 256.0, 301: -512.0,
          520: 1024.0, 640: 2.0 ** 20, 777: 2.0 ** 50, 900: 2.0 ** 100, 901: 2.0 ** 99}


@pytest.mark.parametrize("T,H", [(1, 64), (1, 20), (3, 16), (160, 64), (170, 30)])
def test_rising_scores(cuda_device, T, H):
    """Of every prefix the output is the mean of the entries with the greatest score:
    all others are 50 or more below. The sums are of at most 400 bf16 values times
    one, divided once: (400 + 8) 2^-24 of the largest, and the output's rounding."""
    K = 1000
    g = torch.Generator().manual_seed(T + H)
    x = torch.randn(K, 512, generator=g).bfloat16()
    score = torch.empty(K)
    at = -2.0 ** 100
    for j in range(K):
        at = RISING.get(j, at)
        score[j] = at
    x[:, 448] = (score.double() * 2.0 ** -60).bfloat16()
    cache = ref4.entries(x).view(K, 1, 584)
    rows = ref4.entry_rows(cache.view(K, 584))
    order = torch.randperm(K, generator=g)
    moved = torch.empty_like(cache)
    moved[order] = cache
    slots = order.int().expand(T, K).contiguous()
    ends = [1, 2, 5, 6, 100, 101, 130, 131, 300, 301, 302, 520, 521, 640, 641, 777, 778, 900, 901, 902,
            1000]
    lens = torch.tensor([ends[(7 * t + 3) % len(ends)] for t in range(T)], dtype=torch.int32)
    if T == 1:
        todo = ends
    else:
        todo = [None]
    q = torch.zeros(T, H, 512, dtype=torch.bfloat16)
    q[:, :, 448] = 2.0 ** 60
    for end in todo:
        if end is not None:
            lens[0] = end
        out = kvq.dsv4_latent_attention(q.cuda(), moved.cuda(), slots.cuda(), lens.cuda(), scale=1.0)
        torch.cuda.synchronize()
        want = torch.empty(T, H, 512).double()
        tol = torch.empty(T, H, 512).double()
        for t in range(T):
            n = int(lens[t])
            top = rows[:n][score[:n] == score[:n].max()]
            want[t] = top.mean(0)
            tol[t] = ref4.EPS_BF16 * want[t].abs() + 408 * 2.0 ** -24 * top.abs().amax(0)
        ref.check(out, want, tol, f"length {end}")
