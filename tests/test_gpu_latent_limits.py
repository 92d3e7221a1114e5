"""Attention over latent entries when a wait on one of its kernel's barriers runs
out: the launch's limit is set so low that waits which would end well are given up.
Nothing is broken to get there."""
import time

import pytest
import torch

import kv4_ref as ref4
import kv_quant_cache_gb300 as kvq
import paged_ref as ref

pytestmark = pytest.mark.gpu

LIMITS = [0, 1, 2, 3, 5, 8, 16, 40, 100, 300, 600, 1000, 2000]


def case(T, H, K, seed=1):
    """-> (arguments, the outputs' exact values, their bounds)"""
    g = torch.Generator().manual_seed(seed + T)
    cache = ref4.entries(torch.randn(1000, 512, generator=g).bfloat16()).view(1000, 1, 584)
    q = torch.randn(T, H, 512, generator=g).bfloat16()
    slots = torch.randint(0, 1000, (T, K), generator=g, dtype=torch.int32)
    lens = torch.randint(0, K + 1, (T,), generator=g, dtype=torch.int32)
    want = ref4.latent_attention(q, cache, slots, lens, 512 ** -0.5)
    return [q.cuda(), cache.cuda(), slots.cuda(), lens.cuda()], *want


@pytest.mark.parametrize("T,H,K", [(3, 64, 1500), (40, 20, 700), (60, 64, 700), (620, 2, 300)])
def test_rows_of_a_wait_that_ran_out_are_marked(cuda_device, T, H, K):
    """A call ends in time; what a CTA that gave up has not computed becomes NaN and is
    counted, nothing that the workspace held gets out, and the next call is whole.
    (620 tokens are more than are shared out: a CTA each, and no workspace.)"""
    args, want, tol = case(T, H, K)
    need = kvq.lib().dsv4_latent_attention_workspace(T, H, K)
    assert (need == 0) == (T == 620)
    for limit in LIMITS:
        workspace = torch.full((max(need, 16) // 4,), 3.0, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        old = kvq.set_tile_wait_limit(limit)
        try:
            start = time.monotonic()
            got = kvq.dsv4_latent_attention(*args, workspace=workspace, errors=err).cpu()
            assert time.monotonic() - start < 20
        finally:
            assert kvq.set_tile_wait_limit(old) == limit
        lost = got.isnan().all(-1)
        ref.check(got[~lost], want[~lost], tol[~lost], f"limit {limit}")
        assert int(err.item()) > 0 or not bool(lost.any())
        if limit == 0:
            assert bool(lost.all())
        err.zero_()
        ref.check(kvq.dsv4_latent_attention(*args, errors=err), want, tol, f"after limit {limit}")
        assert int(err.item()) == 0
