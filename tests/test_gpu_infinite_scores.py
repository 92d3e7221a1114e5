"""Scores that overflow fp32: -inf weighs nothing wherever it comes, and rows without
another score are zeros; +inf makes its row NaN; rows beside them are as always."""
import math

import pytest
import torch

import kv4_ref as ref4
import kv_quant_cache_gb300 as kvq
import paged_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("where", ["first", "last", "some", "all", "steps of one warp", "but one"])
@pytest.mark.parametrize("D,per", [(64, 1), (64, 2), (64, 4), (128, 1), (128, 2), (128, 3), (256, 1),
                                   (256, 2)])
def test_4_bit_attention(cuda_device, D, per, where):
    """The keys of ``where`` are 3e38 in the first 64 dims, exactly; head 0 has a sum of -8 there,
    head 1 zeros, head 2 a sum of 8."""
    B, G, page, n = 2, 8, 16, 1200
    g = torch.Generator().manual_seed(D + per)
    width = n // page
    codes, scale, zero = ref4.quantise(torch.randn(width, 2, 1, page, D, generator=g).bfloat16())
    at = torch.arange(n)
    hit = {"first": at < 700, "last": at >= 500, "some": torch.rand(n, generator=g) < 0.5, "all": at >= 0,
           "steps of one warp": at // 16 % 4 == 2, "but one": at != 333}[where]
    page_of, off = at[hit] // page, at[hit] % page
    codes[page_of, 0, 0, off, :64], scale[page_of, 0, 0, off, 0] = 8, 0
    zero[page_of, 0, 0, off, 0] = 3e38
    raw = ref4.raw_of(codes, scale, zero)
    q = torch.randn(B * per, G, D, generator=g).bfloat16()
    q[:, :3, :64] = 0
    q[:, 0, 5], q[:, 2, 5] = -8, 8
    q[:, 3:, :64] = -q[:, 3:, :64].abs()
    table = torch.arange(width).int().expand(B, width).contiguous()
    lens = torch.randint(900, n + 1, (B * per,), generator=g, dtype=torch.int32)
    lens[0] = n
    got = kvq.paged_kv4_attention(q.cuda(), raw.cuda(), table.cuda(), lens.cuda(), scale=1.0,
                                  tokens_per_request=per).cpu()
    sn, z, s = ref4.Cache(raw).terms(at // page, at % page, 0)
    for t, m in enumerate(lens.tolist()):
        keep = ~hit[:m]
        for h, of in ((0, keep), (1, torch.ones(m, dtype=torch.bool)), (4, keep)):
            ref.check(got[t, h:h + 1], *ref4.attend(q[t, h:h + 1], sn[:m][of], z[:m][of], s[:m][of], 1.0),
                      f"token {t} head {h}")
        assert bool(got[t, 2].isnan().all()) == bool(hit[:m].any())


@pytest.mark.parametrize("T,H", [(2, 16), (3, 64), (160, 20)])
def test_latent_attention(cuda_device, T, H):
    """The same with entries of 2^100 in the first rotary dim, and heads with -2^40, 0 and 2^40
    there."""
    K = 300
    g = torch.Generator().manual_seed(T + H)
    x = torch.randn(2 * K, 512, generator=g).bfloat16()
    x[:, 448] = 0
    x[K:, 448] = 2.0 ** 100
    cache = ref4.entries(x).view(2 * K, 1, 584)
    slots = torch.randint(0, 2 * K, (T, K), generator=g, dtype=torch.int32)
    slots[0, :200] = torch.arange(K, K + 200)  # the first tile's all, and more
    slots[1] = torch.arange(K, 2 * K)
    lens = torch.full((T,), K, dtype=torch.int32)
    q = torch.randn(T, H, 512, generator=g).bfloat16()
    q[:, :, 448] = 0
    q[:, 0, 448], q[:, 2, 448] = -2.0 ** 40, 2.0 ** 40
    got = kvq.dsv4_latent_attention(q.cuda(), cache.cuda(), slots.cuda(), lens.cuda()).cpu()
    rows = ref4.entry_rows(cache.view(-1, 584))
    for t in list(range(min(T, 8))) + [T - 1]:
        at = slots[t].long()
        for h, of in ((0, at[at < K]), (1, at)):
            want, tol = ref.attend(q[t, h:h + 1], rows[of], rows[of], 512 ** -0.5)
            ref.check(got[t, h:h + 1], want, tol, f"token {t} head {h}")
        assert bool(got[t, 2].isnan().all()) == bool((at >= K).any())


@pytest.mark.parametrize("low", [-0.25, -2.0, -2.0 ** 20])
@pytest.mark.parametrize("T,H", [(2, 16), (3, 64), (160, 20)])
def test_latent_scores_far_below_behind_infinite_ones(cuda_device, T, H, low):
    """A first tile of scores of -inf, then finite ones however low: every other product is
    ``low`` times 512, so that the mean of those entries is due: 100 values with weights of one
    added and divided, (100 + 8) 2^-24 of the largest, and the output's rounding."""
    K = 300
    g = torch.Generator().manual_seed(T + H)
    x = torch.randn(K, 512, generator=g).bfloat16()
    x[:, 448], x[:, 449] = 0, 512
    x[:200, 448] = 2.0 ** 100
    cache = ref4.entries(x).view(K, 1, 584)
    slots = torch.arange(K).int().expand(T, K).contiguous()
    lens = torch.full((T,), K, dtype=torch.int32)
    q = torch.zeros(T, H, 512, dtype=torch.bfloat16)
    q[:, :, 448], q[:, :, 449] = -2.0 ** 40, low
    got = kvq.dsv4_latent_attention(q.cuda(), cache.cuda(), slots.cuda(), lens.cuda(), scale=1.0)
    rows = ref4.entry_rows(cache.view(-1, 584))[200:]
    want = rows.mean(0).expand(T, H, 512)
    tol = ref4.EPS_BF16 * want.abs() + 108 * 2.0 ** -24 * rows.abs().amax(0)
    ref.check(got, want, tol)


@pytest.mark.parametrize("low", [-0.25, -2.0, -2.0 ** 20])
@pytest.mark.parametrize("D,per", [(64, 1), (64, 3), (128, 1), (128, 2), (256, 2)])
def test_4_bit_scores_far_below_behind_infinite_ones(cuda_device, D, per, low):
    """The same with keys of one value, whose scores are ``low`` times 512: the mean of the
    values with weights of one, each times its scale rounded once, and the output's rounding.
    Parts of the keys are joined by the log2 of their sums, score included, in fp32: each is off
    by 2^-24 of itself, the ratio of two parts' weights by a factor of 2^(2^-23 of that), and
    the mean by this factor less one of twice the largest value, or, the output being a mean
    of the parts' means whatever their weights, by twice that value at most."""
    page, n = 16, 1200
    width = n // page
    g = torch.Generator().manual_seed(D + per)
    codes, scale, zero = ref4.quantise(torch.randn(width, 2, 1, page, D, generator=g).bfloat16())
    codes[:, 0], scale[:, 0], zero[:, 0] = 8, 0, 0
    zero[:, 0, ..., 0] = 512
    zero[:50, 0, ..., 0] = 3e38
    raw = ref4.raw_of(codes, scale, zero)
    q = torch.zeros(per, 4, D, dtype=torch.bfloat16)
    q[..., 7] = low
    table = torch.arange(width).int()[None]
    lens = torch.full((per,), n, dtype=torch.int32)
    got = kvq.paged_kv4_attention(q.cuda(), raw.cuda(), table.cuda(), lens.cuda(), scale=64.0,
                                  tokens_per_request=per)
    at = torch.arange(800, n)
    sn, z, _ = ref4.Cache(raw).terms(at // page, at % page, 0)
    v = sn[:, 1] + z[:, 1]
    want = v.mean(0).expand(per, 4, D)
    tol = (ref4.EPS_BF16 * (sn[:, 1].abs().mean(0) + want.abs())
           + 408 * 2.0 ** -24 * (sn[:, 1].abs() + z[:, 1].abs()).amax(0) * 2)
    log2_sum = -low * 512 * 64 * math.log2(math.e) + 11
    ratio = min(2.0 ** min(2.0 ** -23 * log2_sum, 64) - 1, 1)
    tol = tol + ratio * 2 * (sn[:, 1].abs() + z[:, 1].abs()).amax(0)
    ref.check(got, want, tol)
