"""The tensor-core tiles of the shared prefix when a wait on one of their
barriers runs out: the launch's limit is set so low that waits which would end
well are given up.  Nothing is broken to get there."""
import time

import pytest
import torch

import kv_quant_cache_gb300 as kvq
import paged_ref as ref

pytestmark = pytest.mark.gpu

LIMITS = [0, 1, 2, 3, 5, 8, 16, 40, 100, 300]


@pytest.fixture
def tiles():
    old = kvq.set_config("prefix", 1)
    yield
    kvq.set_config("prefix", old)


def many_items(D, seed=1):
    """200 kv heads behind 200 keys: the blocks of each CTA are those of two or
    three heads, every second one partly filled.  -> (arguments, the outputs'
    exact values, their bounds)"""
    g = torch.Generator().manual_seed(seed + D)
    T, H, page, prefix = 20, 200, 64, 200
    q = torch.randn(T, H, D, generator=g).bfloat16()
    cache = torch.randn(4 + T, 2, H, page, D, generator=g).bfloat16()
    ids = torch.randperm(4 + T, generator=g).int()
    lens = torch.randint(0, 9, (T,), generator=g, dtype=torch.int32)
    pages, table = ids[:4], ids[4:].view(T, 1)
    want = ref.prefix_attention(q, cache, pages, prefix, table, lens, D ** -0.5)
    return [q.cuda(), cache.cuda(), pages.cuda(), prefix, table.cuda(), lens.cuda()], *want


def run_out(args, limit):
    """(outputs, errors) of a call under ``limit``, which has to end in time."""
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    old = kvq.set_tile_wait_limit(limit)
    try:
        start = time.monotonic()
        out = kvq.paged_shared_prefix_attention(*args, errors=err)
        torch.cuda.synchronize()
        assert time.monotonic() - start < 20
    finally:
        assert kvq.set_tile_wait_limit(old) == limit
    return out.cpu(), int(err.item())


@pytest.mark.parametrize("D", [64, 128])
def test_a_wait_that_runs_out_ends_the_call(cuda_device, tiles, D):
    args, want, tol = many_items(D)
    for limit in LIMITS:
        run_out(args, limit)
        ref.check(kvq.paged_shared_prefix_attention(*args), want, tol)  # and none after it


def test_a_wait_that_runs_out_ends_the_call_with_heads_of_256(cuda_device, tiles):
    """Two blocks' scores are under way at once there: a warp whose partner has
    given up on the first finds the second's ready, and must not wait for it."""
    args, want, tol = many_items(256)
    for limit in LIMITS + [600, 1000, 2000]:
        run_out(args, limit)
        ref.check(kvq.paged_shared_prefix_attention(*args), want, tol)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_of_a_wait_that_ran_out_are_marked(cuda_device, tiles, D):
    """What a CTA that gave up has not computed becomes NaN and is counted, in
    its later heads as well; nothing that the workspace held before gets out."""
    args, want, tol = many_items(D, seed=2)
    T, H, _ = args[0].shape
    need = kvq.lib().paged_shared_prefix_attention_workspace(T, H, H, D, 64, args[3], 1)
    for limit in LIMITS + [600, 1000, 2000, 1 << 24]:
        workspace = torch.full((need // 4,), 3.0, device="cuda")  # sums and outputs alike
        old = kvq.set_tile_wait_limit(limit)
        try:
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            got = kvq.paged_shared_prefix_attention(*args, workspace=workspace, errors=err).cpu()
        finally:
            kvq.set_tile_wait_limit(old)
        lost = got.isnan().all(-1)
        ref.check(got[~lost], want[~lost], tol[~lost])
        # (warps that have none of the 20 rows may be those that give up)
        assert int(err.item()) > 0 or not bool(lost.any())
        if limit == 0:
            assert bool(lost.all())
    assert int(err.item()) == 0 and not bool(lost.any())  # the default limit
