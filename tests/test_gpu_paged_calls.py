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


@pytest.mark.parametrize("raw", [True, False])
def test_pinned_calls_whose_range_is_split(cuda_device, monkeypatch, raw):
    """Every tensor in pinned host memory, a range long enough for partials:
    pinned memory that the program takes and fills as soon as the call returns,
    with the kernels still to come, is not the call's workspace."""
    if not raw:
        monkeypatch.setattr(kvq, "_raw_free", None)
    T, Hq, Hkv, D, page, prefix, topk = 1, 4, 1, 128, 64, 40000, 700
    L = kvq.lib()
    needs = [L.paged_shared_prefix_attention_workspace(T, Hq, Hkv, D, page, prefix, 1),
             L.paged_block_sparse_attention_workspace(T, Hq, Hkv, D, page, topk)]
    assert min(needs) > 0
    host = batch(gen(2), T, Hq, Hkv, D, page, prefix, 1, page)
    blocks = torch.arange(topk, dtype=torch.int32).expand(T, Hkv, topk).contiguous()
    some = torch.full((T,), (topk - 1) * page + 5, dtype=torch.int32)
    long_table = host[2].repeat(2)[:topk].view(T, topk).contiguous()
    want, tol = exact(host)
    sparse = ref.sparse_attention(host[0], host[1], long_table, blocks, some, D ** -0.5)
    args = to(host, lambda t: t.pin_memory())
    blocks, some, long_table = blocks.pin_memory(), some.pin_memory(), long_table.pin_memory()
    old = kvq.set_config("prefix", 0)  # the tiles take device memory alone
    try:
        for _ in range(2):
            torch.cuda.synchronize()
            torch.cuda._sleep(10000000)  # about five milliseconds
            a = kvq.paged_shared_prefix_attention(*args)
            b = kvq.paged_block_sparse_attention(args[0], args[1], long_table, blocks, some)
            taken = [torch.empty(n, dtype=torch.uint8, pin_memory=True) for n in needs * 2]
            for x in taken:
                x.fill_(7)
            torch.cuda.synchronize()
            assert a.is_pinned() and b.is_pinned()
            ref.check(a, want, tol)
            ref.check(b, *sparse)
            assert all(bool((x == 7).all()) for x in taken)
        # a workspace of the caller's may be device memory there
        ws = torch.empty(needs[0], dtype=torch.uint8, device="cuda")
        c = kvq.paged_shared_prefix_attention(*args, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(bits(c), bits(a))
    finally:
        kvq.set_config("prefix", old)


def test_append_with_its_positions_alone_on_the_device(cuda_device):
    """One device tensor among pinned ones decides the device, whichever it is."""
    g = gen(3)
    T, Hq, Hkv, D, page = 6, 4, 2, 64, 16
    qkv, cache = normal(g, T, (Hq + 2 * Hkv) * D), normal(g, 3, 2, Hkv, page, D)
    slots, pos = torch.randperm(3 * page, generator=g)[:T], torch.arange(T)
    table = torch.randn(8, D, generator=g)
    got = []
    for move in (lambda t: t.cuda(), lambda t: t.pin_memory()):
        x, kv = move(qkv.clone()), move(cache.clone())
        kvq.paged_kv_rope_append(x, Hq, Hkv, D, move(table), True, pos.cuda(), move(slots), kv)
        torch.cuda.synchronize()
        got.append((bits(x), bits(kv)))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def against_exact(g, host, bad_page=False, **k):
    """A call against the exact values, and repeated bit for bit."""
    if bad_page:
        host[2][1] = host[1].shape[0]
    want, tol = exact(host)
    args = to(host, lambda t: t.cuda())
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = kvq.paged_shared_prefix_attention(*args, errors=err, **k)
    ref.check(got, want, tol)
    assert (int(err.item()) > 0) == bad_page
    assert torch.equal(bits(got), bits(kvq.paged_shared_prefix_attention(*args, **k)))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("prefix", [70, 1100])
def test_hundreds_of_row_tiles_behind_a_prefix(cuda_device, D, prefix):
    """640 row tiles with few keys of their own each: a warp takes a tile and
    joins the parts of the prefix to it; tokens without own keys as well."""
    old = kvq.set_config("prefix", 1)
    try:
        g = gen(4 + D)
        against_exact(g, batch(g, 640, 16, 2, D, 16, prefix, 3, 44), bad_page=prefix > 1000)
    finally:
        kvq.set_config("prefix", old)


@pytest.mark.parametrize("T,Hkv,D,prefix", [
    (613, 2, 256, 400),    # 39 row tiles of a head
    (1240, 2, 128, 300),   # 39
    (1240, 1, 64, 700),    # 39
    (980, 1, 256, 129),    # 62: these stay in step
    (2500, 1, 128, 260),   # 79
    (2460, 1, 256, 128),   # 154, more than there are SMs
    (4950, 1, 64, 200)])   # 155
def test_row_tiles_that_fill_the_sms_unevenly(cuda_device, T, Hkv, D, prefix):
    """Where CTAs in step would leave many SMs idle, each takes its share of a
    head's row tiles one after the other."""
    old = kvq.set_config("prefix", 1)
    try:
        g = gen(5 + T)
        against_exact(g, batch(g, T, 8 * Hkv, Hkv, D, 64, prefix, 1, 5), bad_page=prefix == 300)
    finally:
        kvq.set_config("prefix", old)


def test_workspaces_without_the_allocator_by_itself(cuda_device, monkeypatch):
    """A torch whose allocator is not reached by itself: tensors are the
    workspaces, with the same results, on a stream of the call's own too."""
    host = batch(gen(6), 70, 8, 1, 128, 64, 3000, 1, 64)
    args = to(host, lambda t: t.cuda())
    want = kvq.paged_shared_prefix_attention(*args)
    ref.check(want, *exact(host))
    monkeypatch.setattr(kvq, "_raw_free", None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, side.cuda_stream):
        got = kvq.paged_shared_prefix_attention(*args, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(bits(got), bits(want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kvq.paged_shared_prefix_attention(*args)
    got.zero_()
    graph.replay()
    assert torch.equal(bits(got), bits(want))


@pytest.mark.parametrize("way", [-1, 0, 1])
def test_the_largest_pages(cuda_device, way):
    """Pages of 65536 tokens through every operator: the last slot of one, a
    full page, a few keys of one, a prefix that ends inside its second."""
    g = gen(7)
    T, Hq, Hkv, D, page = 20, 4, 1, 64, 65536
    cache = normal(g, 4, 2, Hkv, page, D)
    qkv = normal(g, 2, (Hq + 2 * Hkv) * D)
    slots = torch.tensor([page - 1, 4 * page - 1])
    d = cache.cuda()
    kvq.paged_kv_rope_append(qkv.cuda(), Hq, Hkv, D, None, True, None, slots.cuda(), d)
    rows = qkv.view(2, Hq + 2 * Hkv, D)
    for i, p in enumerate((0, 3)):
        cache[p, 0, 0, -1], cache[p, 1, 0, -1] = rows[i, Hq], rows[i, Hq + 1]
    assert torch.equal(bits(d), bits(cache))
    fill = torch.tensor([page, 1, page - 1, page], dtype=torch.int32)
    bounds = torch.zeros(4, Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
    kvq.paged_kv_page_bounds(d, torch.arange(4, device="cuda"), fill.cuda(), bounds)
    keys = [cache[p, 0, 0, :fill[p]] for p in range(4)]
    want = torch.stack([torch.stack([k.amin(0), k.amax(0)]) for k in keys])[:, None]
    assert torch.equal(bits(bounds), bits(want))
    q = normal(g, T, Hq, D)
    table = torch.tensor([[0, 1, 3]], dtype=torch.int32)
    requests = torch.zeros(T, dtype=torch.int32)
    lens = torch.full((T,), 3, dtype=torch.int32)
    lens[0], lens[1], lens[2] = 2 * page + 7, page, 0
    blocks = kvq.paged_kv_block_select(q.cuda(), bounds, table.cuda(), lens.cuda(), page, 2,
                                       requests=requests.cuda())
    assert torch.equal(blocks.cpu(), ref.select(q, want, table, lens, page, 2, 0, 0, requests))
    got = kvq.paged_block_sparse_attention(q.cuda(), d, table.cuda(), blocks, lens.cuda(),
                                           requests=requests.cuda())
    ref.check(got, *ref.sparse_attention(q, cache, table, blocks.cpu(), lens, D ** -0.5, requests))
    old = kvq.set_config("prefix", way)
    try:
        pages = torch.tensor([2, 3], dtype=torch.int32)
        got = kvq.paged_shared_prefix_attention(q.cuda(), d, pages.cuda(), page + 77, table.cuda(),
                                                lens.cuda(), requests=requests.cuda())
    finally:
        kvq.set_config("prefix", old)
    ref.check(got, *ref.prefix_attention(q, cache, pages, page + 77, table, lens, D ** -0.5,
                                         requests))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_selection_from_the_widest_table(cuda_device, D):
    """16384 blocks, of which a third are equal and a third differ in a dim
    whose query is tiny; half of them selected, or few, or all but one."""
    g = gen(8 + D)
    T, Hq, Hkv, page, width, some = 2, 4, 1, 4, 16384, 5000
    mid, half = torch.randn(some, Hkv, 1, D, generator=g) * 0.5, torch.rand(some, Hkv, 2, D, generator=g)
    half[:, :, 0] *= -1
    bounds = (mid + half).bfloat16()
    bounds[:1700] = bounds[0]
    bounds[1700:3400] = bounds[1700]
    bounds[1700:3400, :, 1, 5] = (1 + torch.arange(1700)[:, None] / 2048).bfloat16()
    q = normal(g, T, Hq, D)
    q[:, :, 5] = 2.0 ** -22
    table = torch.randint(0, some, (T, width), generator=g, dtype=torch.int32)
    lens = torch.tensor([width * page, width * page - page - 1], dtype=torch.int32)
    for topk, first, last in ((8192, 0, 0), (33, 2, 2), (16383, 0, 1), (6000, 0, 0)):
        got = kvq.paged_kv_block_select(q.cuda(), bounds.cuda(), table.cuda(), lens.cuda(), page,
                                        topk, first, last)
        assert torch.equal(got.cpu(), ref.select(q, bounds, table, lens, page, topk, first, last))


def test_pinned_calls_with_empty_lists(cuda_device):
    """No prefix, no pages of their own, no tokens, with everything pinned."""
    T, Hq, Hkv, D, page = 5, 4, 2, 64, 16
    host = batch(gen(9), T, Hq, Hkv, D, page, 0, 2, 2 * page)
    want, tol = exact(host)
    args = to(host, lambda t: t.pin_memory())
    got = kvq.paged_shared_prefix_attention(*args)
    torch.cuda.synchronize()
    ref.check(got, want, tol)
    args[4], args[5] = args[4][:, :0], torch.zeros(T, dtype=torch.int32).pin_memory()
    got = kvq.paged_shared_prefix_attention(*args)
    torch.cuda.synchronize()
    assert not bool(bits(got).any())
    args[0], args[5] = args[0][:0], args[5][:0]
    assert kvq.paged_shared_prefix_attention(*args).shape == (0, Hq, D)
