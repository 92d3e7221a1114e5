"""Calls of the paged operators as a server makes them beside other work:
settings that change meanwhile, pinned buffers, other allocators, batches of
thousands of rows."""
import threading

import pytest
import torch

import kv_quant_cache_gb300 as kvq
import paged_ref as ref

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape):
    return torch.randn(*shape, generator=g).bfloat16()


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16)


def batch(g, T, Hq, Hkv, D, page, prefix, width, most):
    """Inputs of a shared-prefix call, on the host: q, cache, prefix pages,
    prefix length, table, lens (up to ``most``)."""
    P = -(-prefix // page)
    N = T * width + P
    ids = torch.randperm(N, generator=g).int()
    lens = torch.randint(0, most + 1, (T,), generator=g, dtype=torch.int32)
    return [normal(g, T, Hq, D), normal(g, N, 2, Hkv, page, D), ids[:P].contiguous(), prefix,
            ids[P:].view(T, width).contiguous(), lens]


def to(args, move):
    return [move(x) if isinstance(x, torch.Tensor) else x for x in args]


def exact(args):
    return ref.prefix_attention(*args, args[0].shape[2] ** -0.5)


def test_configuration_that_changes_during_calls(cuda_device):
    """A call decides once: without a workspace it is refused where the tiles
    are asked for, and never takes them with the workspace of the others."""
    args = batch(gen(1), 40, 8, 2, 128, 64, 500, 1, 64)
    want, tol = exact(args)
    q, cache, pages, prefix, table, lens = to(args, lambda t: t.cuda())
    out = torch.empty_like(q)
    L = kvq.lib()
    old = kvq.set_config("prefix", 0)
    stop = threading.Event()

    def change():
        while not stop.is_set():
            L.kvq_set_prefix_config(1)
            L.kvq_set_prefix_config(0)

    other = threading.Thread(target=change)
    other.start()
    seen = set()
    try:
        for i in range(3000):
            status = L.paged_shared_prefix_attention(
                q.data_ptr(), 8 * 128, 40, 8, 2, 128, cache.data_ptr(), cache.shape[0], 64,
                pages.data_ptr(), prefix, table.data_ptr(), 40, 1, None, lens.data_ptr(),
                128 ** -0.5, out.data_ptr(), None, 0, None, torch.cuda.current_stream().cuda_stream)
            seen.add(status)
            if i % 100 == 0:
                torch.cuda.synchronize()
    finally:
        stop.set()
        other.join()
        kvq.set_config("prefix", old)
    assert seen <= {kvq.KVQ_OK, kvq.KVQ_ERR_NULL} and kvq.KVQ_OK in seen
    ref.check(out, want, tol)
