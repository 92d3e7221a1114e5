"""The paged grouped-query operators on the GPU against plain fp64 forms
(paged_ref.py): the append with rotation, the page bounds, the block
selection, block-sparse and shared-prefix attention, and a run of them
together."""
import math

import pytest
import torch

import kv_quant_cache_gb300 as kvq
import paged_ref as ref
import workloads as wl

pytestmark = pytest.mark.gpu

NAN = float("nan")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).bfloat16()


def ints(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g, dtype=torch.int32)


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16)


def counter():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---- append -----------------------------------------------------------------------

def append_case(T, Hq, Hkv, D, rot, neox, page, seed):
    g = gen(seed)
    pages = -(-T // page) + 3
    cache = normal(g, pages, 2, Hkv, page, D)
    qkv = normal(g, T, (Hq + 2 * Hkv) * D)
    slots = torch.randperm(pages * page, generator=g)[:T]
    if T > 2:
        slots[T // 2] = -1
    pos = torch.randint(0, 512, (T,), generator=g)
    table = wl.cos_sin_table(512, rot, 1e4) if rot else None
    return qkv, cache, slots, pos, table


def run_append(case, Hq, Hkv, D, neox, in_place, stream=None, errors=None):
    qkv, cache, slots, pos, table = (None if x is None else x.cuda() for x in case)
    T = qkv.shape[0]
    q_out = None if in_place else torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    kvq.paged_kv_rope_append(qkv, Hq, Hkv, D, table, neox, pos, slots, cache, q_out=q_out,
                             stream=stream, errors=errors)
    torch.cuda.synchronize()
    return qkv.view(T, Hq + 2 * Hkv, D), q_out, cache


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,neox,page", [
    (1, 4, 1, 128, 128, True, 64), (17, 16, 8, 128, 128, True, 64), (5, 8, 8, 64, 64, False, 16),
    (33, 6, 2, 64, 16, False, 16), (40, 5, 5, 128, 32, True, 1), (19, 7, 1, 256, 256, True, 7),
    (23, 4, 2, 256, 64, False, 128), (300, 3, 3, 64, 48, True, 5), (64, 28, 4, 128, 64, False, 64),
    (9, 4, 2, 128, 0, True, 64), (700, 32, 8, 128, 128, True, 64), (31, 0, 3, 64, 64, True, 16),
    (21, 40, 40, 64, 64, False, 32)])
def test_append(cuda_device, T, Hq, Hkv, D, rot, neox, page, in_place):
    case = append_case(T, Hq, Hkv, D, rot, neox, page, seed=T + D + rot)
    qkv, cache, slots, pos, table = case
    err = counter()
    x, q_out, kv = run_append(case, Hq, Hkv, D, neox, in_place, errors=err)
    q, q_tol, want, tol = ref.append(qkv, Hq, Hkv, D, table, rot, neox, pos, slots, cache)
    ref.check(x[:, :Hq] if in_place else q_out, q, q_tol, "q")
    ref.check(kv, want, tol, "cache")
    # what is not an output is as it was, bit for bit
    before = bits(qkv.view(T, Hq + 2 * Hkv, D))
    assert torch.equal(bits(x)[:, Hq:], before[:, Hq:])
    if not in_place:
        assert torch.equal(bits(x), before)
    assert int(err.item()) == 0


def test_append_rejects_bad_indices(cuda_device):
    T, Hq, Hkv, D, page = 50, 4, 2, 128, 16
    case = append_case(T, Hq, Hkv, D, D, True, page, seed=3)
    qkv, cache, slots, pos, table = case
    pos[[0, 7]] = torch.tensor([-1, 512])
    pos[20] = 2 ** 40
    slots[[9, 10]] = torch.tensor([cache.shape[0] * page, -2])
    slots[30] = 2 ** 45
    err = counter()
    x, q_out, kv = run_append(case, Hq, Hkv, D, True, False, errors=err)
    assert int(err.item()) == 6
    q, q_tol, want, tol = ref.append(qkv, Hq, Hkv, D, table, D, True, pos, slots, cache)
    bad = (pos < 0) | (pos >= 512)
    assert bool((q_out[bad.cuda()] == 7.0).all())
    ref.check(q_out.cpu()[~bad], q[~bad], q_tol[~bad], "q")
    ref.check(kv, want, tol, "cache")
    # without a counter the same tokens are rejected all the same
    _, q2, kv2 = run_append(case, Hq, Hkv, D, True, False)
    assert torch.equal(bits(q2), bits(q_out)) and torch.equal(bits(kv2), bits(kv))


def test_append_passes_nonfinite_values_through(cuda_device):
    T, Hq, Hkv, D, page = 4, 2, 1, 64, 16
    case = append_case(T, Hq, Hkv, D, 0, True, page, seed=5)
    case[0][1, 3 * D + 5] = NAN
    case[0][1, 2 * D + 1] = math.inf
    case[2][:] = torch.tensor([3, 1, 9, 4])
    _, _, kv = run_append(case, Hq, Hkv, D, True, True)
    assert math.isnan(float(kv[0, 1, 0, 1, 5])) and float(kv[0, 0, 0, 1, 1]) == math.inf


# ---- page bounds ---------------------------------------------------------------------

@pytest.mark.parametrize("n,Hkv,D,page", [(1, 1, 64, 16), (9, 3, 128, 64), (40, 2, 256, 17),
                                          (130, 8, 128, 1), (64, 1, 64, 130), (7, 5, 256, 300)])
def test_page_bounds(cuda_device, n, Hkv, D, page):
    g = gen(n + D + page)
    total = n + 5
    cache = normal(g, total, 2, Hkv, page, D)
    pages = torch.randperm(total, generator=g)[:n]
    lens = ints(g, 1, page, n)
    lens[0] = page
    bounds = normal(g, total, Hkv, 2, D)
    want = bounds.clone()
    for i in range(n):
        k = cache[pages[i], 0, :, :lens[i]]
        want[pages[i], :, 0], want[pages[i], :, 1] = k.amin(1), k.amax(1)
        cache[pages[i], 0, :, lens[i]:] = NAN  # past the page's fill: not to be seen
    err = counter()
    got = bounds.cuda()
    out = kvq.paged_kv_page_bounds(cache.cuda(), pages.cuda(), lens.cuda(), got, errors=err)
    assert out is got and int(err.item()) == 0
    assert torch.equal(got.cpu(), want)


def test_page_bounds_skips_and_rejects(cuda_device):
    g = gen(8)
    cache = normal(g, 6, 2, 2, 16, 64)
    cache[4, 0, 1, 3, 9] = NAN
    bounds = normal(g, 6, 2, 2, 64)
    pages = torch.tensor([0, -1, 1, 2, 6, -2, 3, 4, 4])
    lens = torch.tensor([16, 4, 0, 17, 3, 3, -1, 16, 16], dtype=torch.int32)
    err = counter()
    got = kvq.paged_kv_page_bounds(cache.cuda(), pages.cuda(), lens.cuda(), bounds.cuda(),
                                   errors=err).cpu()
    assert int(err.item()) == 4
    want = bounds.clone()
    for p in (0, 4):
        want[p, :, 0], want[p, :, 1] = cache[p, 0].amin(1), cache[p, 0].amax(1)
    assert torch.equal(got.isnan(), want.isnan()) and bool(want.isnan().sum() == 2)
    assert torch.equal(got.nan_to_num(), want.nan_to_num())


# ---- block selection -------------------------------------------------------------------

def bounds_of(g, pages, Hkv, D):
    mid = normal(g, pages, Hkv, 1, D, std=0.5)
    half = torch.rand(pages, Hkv, 2, D, generator=g) + 1.0
    half[:, :, 0] *= -1
    return (mid + half).bfloat16()


def run_select(q, bounds, table, lens, page, topk, first=0, last=0, requests=None, errors=None):
    return kvq.paged_kv_block_select(q.cuda(), bounds.cuda(), table.cuda(), lens.cuda(), page,
                                     topk, first, last,
                                     requests=None if requests is None else requests.cuda(),
                                     errors=errors).cpu()


@pytest.mark.parametrize("T,Hq,Hkv,D,page,width,topk,first,last", [
    (1, 8, 2, 128, 64, 700, 16, 1, 1), (3, 4, 4, 64, 16, 33, 8, 0, 0), (1, 4, 1, 256, 16, 2100, 64, 2, 3),
    (5, 14, 2, 128, 32, 130, 1, 0, 0), (2, 64, 1, 64, 1, 300, 7, 0, 1), (40, 8, 8, 128, 64, 65, 64, 1, 0),
    (2, 2, 1, 64, 16, 500, 499, 0, 0), (2, 4, 2, 128, 16, 40, 5, 9, 9), (200, 2, 1, 128, 16, 90, 12, 1, 1)])
def test_block_select(cuda_device, T, Hq, Hkv, D, page, width, topk, first, last):
    g = gen(T + D + width)
    N = T * width + 3
    table = torch.randperm(N, generator=g)[:T * width].view(T, width).int()
    lens = ints(g, 0, width * page, T)
    lens[0] = width * page
    q, bounds = normal(g, T, Hq, D), bounds_of(g, N, Hkv, D)
    err = counter()
    got = run_select(q, bounds, table, lens, page, topk, first, last, errors=err)
    assert torch.equal(got, ref.select(q, bounds, table, lens, page, topk, first, last))
    assert int(err.item()) == 0


def test_block_select_close_scores_and_ties(cuda_device):
    """Scores that fp32 cannot order: equal blocks (lowest index first), and
    blocks whose scores differ by less than the fp32 error of a score."""
    g = gen(12)
    T, Hq, Hkv, D, page, width = 3, 4, 1, 128, 16, 400
    bounds = bounds_of(g, width, Hkv, D)
    bounds[100:200] = bounds[100]  # equal
    # copies that differ in a dim with a tiny query value only
    bounds[200:300] = bounds[200]
    bounds[200:300, 0, 1, 5] = (1 + torch.arange(100) / 128).bfloat16()
    q = normal(g, T, Hq, D)
    q[:, :, 5] = 2.0 ** -22
    q[2] = 0  # every score zero
    table = torch.arange(width).expand(T, width).contiguous().int()
    lens = torch.full((T,), width * page, dtype=torch.int32)
    for topk in (1, 30, 150, 250, 399):
        got = run_select(q, bounds, table, lens, page, topk)
        assert torch.equal(got, ref.select(q, bounds, table, lens, page, topk, 0, 0)), topk


def test_block_select_nonfinite_and_bad_pages(cuda_device):
    g = gen(13)
    T, Hq, Hkv, D, page, width = 2, 2, 1, 64, 16, 120
    bounds = bounds_of(g, 130, Hkv, D)
    bounds[7, 0, 0, 3] = NAN
    bounds[9, 0, 1] = math.inf
    q = normal(g, T, Hq, D).abs() + 0.25  # no zero: inf * 0 stays out
    table = torch.randperm(130, generator=g)[:T * 60].repeat(2).view(T, width).int()
    table[0, 11] = 130
    table[0, 12] = -1
    table[1, 3] = 7
    table[1, 4] = 9
    lens = torch.full((T,), width * page, dtype=torch.int32)
    for topk in (4, 117, 119):
        err = counter()
        got = run_select(q, bounds, table, lens, page, topk, errors=err)
        assert torch.equal(got, ref.select(q, bounds, table, lens, page, topk, 0, 0)), topk
        assert int(err.item()) > 0
    nan_q = q.clone()
    nan_q[0, 0, 0] = NAN
    got = run_select(nan_q, bounds, table, lens, page, 5)
    assert got[0, 0].tolist() == [0, 1, 2, 3, 4]


def test_block_select_requests_lengths_and_strides(cuda_device):
    g = gen(14)
    R, width, page, Hq, Hkv, D, T = 3, 50, 16, 8, 2, 128, 9
    bounds = bounds_of(g, R * width, Hkv, D)
    table = torch.randperm(R * width, generator=g).view(R, width).int()
    requests = torch.tensor([2, 0, 1, 1, 3, -1, 0, 2, 2], dtype=torch.int32)
    lens = torch.tensor([800, 0, 1, 799, 800, 800, -3, 10 ** 6, 333], dtype=torch.int32)
    wide = normal(g, T, (Hq + 2 * Hkv) * D).cuda()
    q = wide.view(T, Hq + 2 * Hkv, D)[:, :Hq]  # a view into packed QKV
    err = counter()
    got = kvq.paged_kv_block_select(q, bounds.cuda(), table.cuda(), lens.cuda(), page, 6, 1, 1,
                                    requests=requests.cuda(), errors=err).cpu()
    want = ref.select(q.cpu(), bounds, table, lens, page, 6, 1, 1, requests)
    assert torch.equal(got, want)
    assert int(err.item()) >= 4


# ---- attention ------------------------------------------------------------------------------

def paged_inputs(g, T, Hq, Hkv, D, page, R, width, extra=2, std=1.5):
    N = R * width + extra
    ids = torch.randperm(N, generator=g)
    table = ids[:R * width].view(R, width).int()
    return normal(g, T, Hq, D, std=std), normal(g, N, 2, Hkv, page, D), table, ids[R * width:]


def random_blocks(g, T, Hkv, topk, width, lens, page):
    out = torch.full((T, Hkv, topk), -1, dtype=torch.int32)
    for t in range(T):
        n = -(-int(lens[t]) // page)
        for h in range(Hkv):
            b = torch.randperm(n, generator=g)[:topk].sort().values
            out[t, h, :len(b)] = b.int()
    return out


def hide_unseen(cache, seen):
    """NaN in every token place of the cache that no row may look at."""
    c = cache.clone()
    c.transpose(2, 3)[~seen.unsqueeze(1).expand(-1, 2, -1)] = NAN
    return c


@pytest.mark.parametrize("T,Hq,Hkv,D,page,width,topk", [
    (1, 4, 1, 128, 64, 40, 8), (3, 8, 2, 128, 16, 30, 9), (2, 4, 4, 64, 64, 5, 5),
    (2, 14, 2, 64, 1, 90, 50), (1, 32, 1, 128, 32, 20, 20), (5, 20, 1, 256, 16, 12, 4),
    (4, 6, 3, 256, 7, 33, 11), (2, 40, 2, 128, 128, 9, 6), (1, 2, 2, 64, 300, 7, 3),
    (70, 8, 8, 64, 16, 17, 6), (1, 8, 1, 128, 64, 160, 150)])
def test_sparse_attention(cuda_device, T, Hq, Hkv, D, page, width, topk):
    g = gen(T + Hq + D + page)
    q, cache, table, _ = paged_inputs(g, T, Hq, Hkv, D, page, T, width)
    lens = ints(g, 0, width * page, T)
    lens[0] = width * page - (page > 1)
    blocks = random_blocks(g, T, Hkv, topk, width, lens, page)
    if T > 1:
        blocks[1] = blocks[1, :, torch.randperm(topk, generator=g)]  # -1 anywhere, any order
    seen = torch.zeros(cache.shape[0], page, dtype=torch.bool)
    for t in range(T):
        for b in blocks[t].unique().tolist():
            if b >= 0:
                seen[table[t, b].long(), :max(0, int(lens[t]) - b * page)] = True
    err = counter()
    got = kvq.paged_block_sparse_attention(q.cuda(), hide_unseen(cache, seen).cuda(), table.cuda(),
                                           blocks.cuda(), lens.cuda(), errors=err)
    want, tol = ref.sparse_attention(q, cache, table, blocks, lens, D ** -0.5)
    ref.check(got, want, tol)
    assert int(err.item()) == 0


def test_sparse_attention_rows_without_keys_and_bad_indices(cuda_device):
    g = gen(30)
    T, Hq, Hkv, D, page, R, width, topk = 8, 4, 2, 128, 16, 3, 10, 4
    q, cache, table, _ = paged_inputs(g, T, Hq, Hkv, D, page, R, width)
    requests = torch.tensor([0, 1, 2, 3, -1, 0, 1, 2], dtype=torch.int32)
    lens = torch.tensor([160, 0, 50, 160, 160, -5, 10 ** 7, 1], dtype=torch.int32)
    blocks = ints(g, 0, 9, T, Hkv, topk)
    blocks[0, 0] = -1                                       # nothing selected
    blocks[0, 1] = torch.tensor([3, 3, 3, 5])               # the same block three times
    blocks[2] = torch.tensor([0, 3, 4, -7])                 # one past the length, one negative
    blocks[7] = torch.tensor([0, -1, -1, 2 ** 30])
    table[1, 2] = 10 ** 6                                   # a page outside the cache
    blocks[6, 0, 0] = 2
    err = counter()
    got = kvq.paged_block_sparse_attention(q.cuda(), cache.cuda(), table.cuda(), blocks.cuda(),
                                           lens.cuda(), scale=0.3, requests=requests.cuda(),
                                           errors=err).cpu()
    assert int(err.item()) > 0
    want, tol = ref.sparse_attention(q, cache, table, blocks, lens, 0.3, requests)
    ref.check(got, want, tol)
    for t in (1, 3, 4, 5):
        assert torch.equal(bits(got[t]), torch.zeros(Hq, D, dtype=torch.int16))
    assert not bool(bits(got[0, :2]).any())


@pytest.fixture(params=["auto", "rows", "tiles"])
def prefix_way(request):
    """Both kernels that can take a prefix, and the choice between them."""
    ids = {"auto": -1, "rows": 0, "tiles": 1}
    old = kvq.set_config("prefix", ids[request.param])
    yield request.param
    kvq.set_config("prefix", old)


@pytest.mark.parametrize("T,Hq,Hkv,D,page,prefix,width,q_len", [
    (1, 4, 1, 128, 64, 64, 3, 1), (4, 8, 2, 128, 64, 1000, 4, 1), (6, 4, 4, 64, 16, 257, 9, 2),
    (9, 14, 2, 128, 16, 1, 2, 3), (40, 8, 1, 64, 32, 2048, 1, 1), (3, 32, 1, 128, 7, 500, 30, 1),
    (5, 6, 3, 256, 16, 333, 20, 5), (70, 16, 2, 128, 64, 4100, 2, 1), (33, 4, 1, 256, 64, 700, 1, 3),
    (130, 8, 2, 64, 64, 129, 3, 2), (64, 8, 1, 128, 128, 1024, 0, 1), (257, 8, 4, 128, 16, 2049, 1, 1),
    (100, 5, 1, 64, 1, 600, 5, 1), (20, 16, 1, 128, 300, 1500, 2, 4), (600, 8, 2, 64, 8, 1000, 1, 1),
    (33, 8, 1, 128, 1024, 2500, 1, 1), (150, 4, 2, 128, 64, 9000, 2, 1), (21, 64, 1, 64, 64, 130, 1, 1)])
def test_prefix_attention(cuda_device, prefix_way, T, Hq, Hkv, D, page, prefix, width, q_len):
    g = gen(T + Hq + D + prefix)
    R, P = -(-T // q_len), -(-prefix // page)
    q, cache, table, spare = paged_inputs(g, T, Hq, Hkv, D, page, R, width, extra=P + 2)
    requests = (torch.arange(T) // q_len).int()
    lens = ints(g, 0, width * page, T)
    pages = spare[:P].int()
    seen = torch.zeros(cache.shape[0], page, dtype=torch.bool)
    seen[pages.long()] = True
    if prefix % page:
        seen[pages[-1].long(), prefix % page:] = False
    for t in range(T):
        for b in range(-(-int(lens[t]) // page)):
            seen[table[requests[t], b].long(), :int(lens[t]) - b * page] = True
    err = counter()
    got = kvq.paged_shared_prefix_attention(q.cuda(), hide_unseen(cache, seen).cuda(),
                                            pages.cuda(), prefix, table.cuda(), lens.cuda(),
                                            requests=requests.cuda(), errors=err)
    want, tol = ref.prefix_attention(q, cache, pages, prefix, table, lens, D ** -0.5, requests)
    ref.check(got, want, tol)
    assert int(err.item()) == 0


def test_prefix_attention_without_prefix_or_keys(cuda_device, prefix_way):
    g = gen(40)
    T, Hq, Hkv, D, page, width = 3, 8, 2, 128, 16, 4
    q, cache, table, spare = paged_inputs(g, T, Hq, Hkv, D, page, T, width)
    lens = torch.tensor([0, 64, 5], dtype=torch.int32)
    none = torch.zeros(0, dtype=torch.int32)
    got = kvq.paged_shared_prefix_attention(q.cuda(), cache.cuda(), none.cuda(), 0, table.cuda(),
                                            lens.cuda()).cpu()
    want, tol = ref.prefix_attention(q, cache, none, 0, table, lens, D ** -0.5)
    ref.check(got, want, tol)
    assert not bool(bits(got[0]).any())
    empty = torch.zeros(T, 0, dtype=torch.int32)
    out = torch.full((T, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    kvq.paged_shared_prefix_attention(q.cuda(), cache.cuda(), none.cuda(), 0, empty.cuda(),
                                      (lens * 0).cuda(), out=out)
    assert not bool(bits(out).any())


@pytest.mark.parametrize("T", [2, 40, 300])
def test_prefix_attention_bad_pages(cuda_device, prefix_way, T):
    g = gen(41)
    Hq, Hkv, D, page, width, prefix = 4, 1, 128, 64, 2, 700
    q, cache, table, spare = paged_inputs(g, T, Hq, Hkv, D, page, T, width, extra=11)
    pages = spare[:11].int()
    pages[3], pages[10] = cache.shape[0], -1
    lens = ints(g, 1, width * page, T)
    lens[1] = 10 ** 6
    table[0, 0] = -4
    err = counter()
    got = kvq.paged_shared_prefix_attention(q.cuda(), cache.cuda(), pages.cuda(), prefix,
                                            table.cuda(), lens.cuda(), errors=err)
    want, tol = ref.prefix_attention(q, cache, pages, prefix, table, lens, D ** -0.5)
    ref.check(got, want, tol)
    assert int(err.item()) > 0


def test_prefix_attention_large_scores_and_nonfinite_values(cuda_device, prefix_way):
    """Logits of a thousand and more (no exponential may overflow), a NaN
    value and an infinite one that one request each sees (the infinite one
    gives NaN where its weight is zero)."""
    g = gen(42)
    T, Hq, Hkv, D, page, width, prefix = 160, 4, 1, 128, 64, 2, 300
    q, cache, table, spare = paged_inputs(g, T, Hq, Hkv, D, page, T, width, extra=5, std=400.0)
    lens = ints(g, 1, width * page, T)
    cache[table[1, 0].long(), 1, 0, 0, 7] = NAN
    cache[table[2, 0].long(), 1, 0, 0, 7] = math.inf
    got = kvq.paged_shared_prefix_attention(q.cuda(), cache.cuda(), spare.int().cuda(), prefix,
                                            table.cuda(), lens.cuda()).cpu()
    want, tol = ref.prefix_attention(q, cache, spare, prefix, table, lens, D ** -0.5)
    assert bool(got[1, :, 7].isnan().all()) and not bool(got[2, :, 7].isfinite().any())
    ok = torch.ones(T, Hq, D, dtype=torch.bool)
    ok[1:3, :, 7] = False
    ref.check(got[ok], want[ok], tol[ok])


@pytest.mark.parametrize("T,Hq,Hkv,page,q_len,prefix", [
    (9, 4, 4, 16, 1, 40), (6, 8, 2, 64, 2, 0), (16, 1, 1, 1, 1, 5), (12, 6, 2, 5, 3, 33),
    (40, 8, 1, 16, 1, 300), (50, 3, 1, 8, 2, 129)])
def test_nonfinite_values_stay_with_their_request(cuda_device, prefix_way, T, Hq, Hkv, page, q_len, prefix):
    """Requests share a CTA's rows; NaN and infinite keys and values of one
    reach no row of another."""
    g = gen(T + page)
    D, width, R, P = 64, -(-40 // page), -(-T // q_len), -(-prefix // page)
    q, cache, table, spare = paged_inputs(g, T, Hq, Hkv, D, page, R, width, extra=P + 1)
    requests = (torch.arange(T) // q_len).int()
    lens = ints(g, 1, width * page, T)
    args = (spare[:P].int().cuda(), prefix, table.cuda(), lens.cuda())
    bad = R // 2
    spoiled = cache.clone()
    spoiled[table[bad].long(), 0, :, :, 3] = NAN
    spoiled[table[bad].long(), 1, :, :, 5] = math.inf
    spoiled[table[bad].long(), 1, :, :, 6] = NAN
    a = kvq.paged_shared_prefix_attention(q.cuda(), cache.cuda(), *args,
                                          requests=requests.cuda()).cpu()
    b = kvq.paged_shared_prefix_attention(q.cuda(), spoiled.cuda(), *args,
                                          requests=requests.cuda()).cpu()
    ok = requests != bad
    assert torch.equal(bits(a[ok]), bits(b[ok]))
    assert bool(b[~ok].isnan().all())  # NaN scores: every output of these rows
    want, tol = ref.prefix_attention(q, cache, spare[:P], prefix, table, lens, D ** -0.5, requests)
    ref.check(a, want, tol)


def test_attention_of_a_strided_query_and_given_buffers(cuda_device, prefix_way):
    g = gen(43)
    T, Hq, Hkv, D, page, width, prefix = 5, 8, 2, 128, 16, 20, 100
    _, cache, table, spare = paged_inputs(g, T, Hq, Hkv, D, page, T, width, extra=9)
    packed = normal(g, T, (Hq + 2 * Hkv) * D)
    q = packed.cuda().view(T, Hq + 2 * Hkv, D)[:, :Hq]
    lens = ints(g, 1, width * page, T)
    L = kvq.lib()
    ws = torch.full((L.paged_shared_prefix_attention_workspace(T, Hq, Hkv, D, page, prefix, width),),
                    255, dtype=torch.uint8, device="cuda")
    out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    kvq.paged_shared_prefix_attention(q, cache.cuda(), spare.int().cuda(), prefix, table.cuda(),
                                      lens.cuda(), out=out, workspace=ws, stream=stream)
    stream.synchronize()
    want, tol = ref.prefix_attention(q.cpu(), cache, spare, prefix, table, lens, D ** -0.5)
    ref.check(out, want, tol)


def test_cache_offsets_past_32_bits(cuda_device, prefix_way):
    """A cache of 9 GB: element offsets past 2^32 for the append, the bounds
    and the attentions."""
    T, Hq, Hkv, D, page = 4, 8, 8, 128, 64
    N = 34500
    assert (N - 8) * 2 * Hkv * page * D > 2 ** 32
    cache = torch.zeros(N, 2, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    g = gen(50)
    ids = torch.arange(N - 8, N)
    small = normal(g, 8, 2, Hkv, page, D)
    cache[ids.cuda()] = small.cuda()
    qkv = normal(g, T, (Hq + 2 * Hkv) * D)
    slots = (ids[:T] * page + 5)
    kvq.paged_kv_rope_append(qkv.cuda(), Hq, Hkv, D, None, True, None, slots.cuda(), cache)
    x = qkv.view(T, Hq + 2 * Hkv, D)
    small[torch.arange(T), 0, :, 5], small[torch.arange(T), 1, :, 5] = x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    assert torch.equal(bits(cache[ids.cuda()]), bits(small))
    bounds = torch.zeros(N, Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
    kvq.paged_kv_page_bounds(cache, ids.cuda(), torch.full((8,), page, dtype=torch.int32).cuda(),
                             bounds)
    assert torch.equal(bounds[ids.cuda(), :, 0].cpu(), small[:, 0].amin(2))
    q = x[:, :Hq].contiguous()
    lens = torch.full((T,), 2 * page - 3, dtype=torch.int32)
    table = ids[:8].view(T, 2).int()
    local = torch.arange(8).view(T, 2).int()
    blocks = torch.tensor([0, 1], dtype=torch.int32).expand(T, Hkv, 2).contiguous()
    got = kvq.paged_block_sparse_attention(q.cuda(), cache, table.cuda(), blocks.cuda(),
                                           lens.cuda())
    ref.check(got, *ref.sparse_attention(q, small, local, blocks, lens, D ** -0.5))
    for rep in (1, 40):  # few rows, and enough for the tiled prefix kernel
        qq = q.repeat(rep, 1, 1)
        got = kvq.paged_shared_prefix_attention(qq.cuda(), cache, ids.int().cuda(), 8 * page - 9,
                                                table.repeat(rep, 1).cuda(),
                                                lens.repeat(rep).cuda())
        want, tol = ref.prefix_attention(q, small, torch.arange(8), 8 * page - 9, local, lens,
                                         D ** -0.5)
        ref.check(got, want.repeat(rep, 1, 1), tol.repeat(rep, 1, 1))


# ---- a run of them together ------------------------------------------------------------------

def decode_state(seed, B=6, Hq=8, Hkv=2, D=128, page=16, width=24, prefix=200):
    """A batch in the middle of its answers, and the buffers a server keeps."""
    g = gen(seed)
    P = -(-prefix // page)
    N = B * width + P + 1
    ids = torch.randperm(N, generator=g)
    s = dict(B=B, Hq=Hq, Hkv=Hkv, D=D, page=page, prefix=prefix,
             table=ids[:B * width].view(B, width).int(), prefix_pages=ids[B * width:][:P].int(),
             cache=normal(g, N, 2, Hkv, page, D), cos_sin=wl.cos_sin_table(4096, D, 1e4),
             lens=ints(g, page * 8, width * page - 8, B))
    s["bounds"] = torch.zeros(N, Hkv, 2, D, dtype=torch.bfloat16)
    return s


def step(s, qkv, topk=5):
    """One decode step on the device state ``s``: append, refresh the last
    pages' bounds, select, attend sparsely and over the shared prefix."""
    T, page = s["B"], s["page"]
    at = s["lens"].long()
    last = s["table"].long().gather(1, (at // page)[:, None])[:, 0]
    q = torch.empty(T, s["Hq"], s["D"], dtype=torch.bfloat16, device="cuda")
    kvq.paged_kv_rope_append(qkv, s["Hq"], s["Hkv"], s["D"], s["cos_sin"], True, at,
                             last * page + at % page, s["cache"], q_out=q)
    kvq.paged_kv_page_bounds(s["cache"], last, (at % page + 1).int(), s["bounds"])
    s["lens"] += 1
    blocks = kvq.paged_kv_block_select(q, s["bounds"], s["table"], s["lens"], page, topk, 1, 1)
    sparse = kvq.paged_block_sparse_attention(q, s["cache"], s["table"], blocks, s["lens"])
    full = kvq.paged_shared_prefix_attention(q, s["cache"], s["prefix_pages"], s["prefix"],
                                             s["table"], s["lens"])
    return q, blocks, sparse, full


def on_gpu(s):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}


def fill_bounds(d):
    n = d["cache"].shape[0]
    full = torch.full((n,), d["page"], dtype=torch.int32, device="cuda")
    kvq.paged_kv_page_bounds(d["cache"], torch.arange(n, device="cuda"), full, d["bounds"])


def test_decode_steps_together(cuda_device):
    s = decode_state(60)
    d = on_gpu(s)
    fill_bounds(d)
    lens = s["lens"].clone()
    for i in range(4):
        qkv = normal(gen(61 + i), s["B"], (s["Hq"] + 2 * s["Hkv"]) * s["D"])
        q, blocks, sparse, full = step(d, qkv.cuda())
        lens += 1
        assert torch.equal(d["lens"].cpu(), lens)
        cache, bounds, qh = d["cache"].cpu(), d["bounds"].cpu(), q.cpu()
        assert torch.equal(blocks.cpu(), ref.select(qh, bounds, s["table"], lens, s["page"], 5, 1, 1))
        scale = s["D"] ** -0.5
        ref.check(sparse, *ref.sparse_attention(qh, cache, s["table"], blocks.cpu(), lens, scale))
        ref.check(full, *ref.prefix_attention(qh, cache, s["prefix_pages"], s["prefix"],
                                              s["table"], lens, scale))


def test_decode_steps_in_a_graph(cuda_device, prefix_way):
    """The same steps captured once and replayed give the eager results, bit
    for bit, also when two captured graphs are replayed in turn."""
    s = decode_state(70)
    eager, graphs = on_gpu(s), []
    fill_bounds(eager)
    for _ in range(2):
        d = on_gpu(s)
        fill_bounds(d)
        x = torch.zeros(s["B"], (s["Hq"] + 2 * s["Hkv"]) * s["D"], dtype=torch.bfloat16,
                        device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(on_gpu(s), x)  # set-up of the kernels, outside the capture
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step(d, x)
        graphs.append((graph, x, outs, d))
    for i in range(3):
        qkv = normal(gen(71 + i), s["B"], (s["Hq"] + 2 * s["Hkv"]) * s["D"]).cuda()
        want = step(eager, qkv)
        for graph, x, outs, d in graphs:
            x.copy_(qkv)
            graph.replay()
        torch.cuda.synchronize()
        for graph, x, outs, d in graphs:
            for a, b in zip(outs, want):
                assert torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))
            assert torch.equal(bits(d["cache"]), bits(eager["cache"]))


def test_same_call_twice_is_the_same(cuda_device, prefix_way):
    g = gen(80)
    T, Hq, Hkv, D, page, width, prefix = 90, 8, 2, 128, 64, 3, 2000
    q, cache, table, spare = paged_inputs(g, T, Hq, Hkv, D, page, T, width, extra=32)
    lens = ints(g, 1, width * page, T).cuda()
    q, cache, table, pages = q.cuda(), cache.cuda(), table.cuda(), spare.int().cuda()
    a = kvq.paged_shared_prefix_attention(q, cache, pages, prefix, table, lens)
    for _ in range(5):
        b = kvq.paged_shared_prefix_attention(q, cache, pages, prefix, table, lens)
        assert torch.equal(bits(a), bits(b))


def test_two_streams_at_once(cuda_device, prefix_way):
    """Calls on two streams, each with its own workspace, do not disturb each
    other."""
    g = gen(81)
    T, Hq, Hkv, D, page, width, prefix = 40, 8, 2, 128, 64, 3, 4000
    q, cache, table, spare = paged_inputs(g, T, Hq, Hkv, D, page, T, width, extra=63)
    lens = ints(g, 1, width * page, T).cuda()
    qs = [q.cuda(), q.flip(0).cuda()]
    cache, table, pages = cache.cuda(), table.cuda(), spare.int().cuda()
    want = [kvq.paged_shared_prefix_attention(x, cache, pages, prefix, table, lens) for x in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for x, st in zip(qs, streams):
            with torch.cuda.stream(st):
                got.append(kvq.paged_shared_prefix_attention(x, cache, pages, prefix, table, lens))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(bits(a), bits(b))


def test_long_lists_of_small_pages(cuda_device, prefix_way):
    """More pages than a CTA lists at a time, in the prefix, in a request and
    in a selection."""
    g = gen(90)
    T, Hq, Hkv, D, page, width, prefix = 3, 4, 1, 64, 1, 5000, 20000
    N = 6000
    q, cache = normal(g, T, Hq, D), normal(g, N, 2, Hkv, page, D)
    table = ints(g, 0, N - 1, T, width)   # pages listed several times
    pages = ints(g, 0, N - 1, prefix)
    lens = torch.tensor([width, 4500, 3], dtype=torch.int32)
    got = kvq.paged_shared_prefix_attention(q.cuda(), cache.cuda(), pages.cuda(), prefix,
                                            table.cuda(), lens.cuda())
    ref.check(got, *ref.prefix_attention(q, cache, pages, prefix, table, lens, D ** -0.5))
    blocks = torch.arange(width, dtype=torch.int32).expand(T, Hkv, width).contiguous()
    blocks[2, 0, 3:] = -1
    got = kvq.paged_block_sparse_attention(q.cuda(), cache.cuda(), table.cuda(), blocks.cuda(),
                                           lens.cuda())
    blocks[1, 0, 4500:] = -1
    ref.check(got, *ref.sparse_attention(q, cache, table, blocks, lens, D ** -0.5))


def test_many_rows_with_long_small_pages(cuda_device):
    """Many row tiles, so that a CTA has a whole long list to itself."""
    g = gen(91)
    T, Hq, Hkv, D, page, width = 700, 1, 1, 64, 16, 300
    N = 400
    q, cache = normal(g, T, Hq, D), normal(g, N, 2, Hkv, page, D)
    table = ints(g, 0, N - 1, T, width)
    lens = ints(g, 0, 40, T)
    lens[5], lens[699] = width * page, 3000
    none = torch.zeros(0, dtype=torch.int32)
    got = kvq.paged_shared_prefix_attention(q.cuda(), cache.cuda(), none.cuda(), 0, table.cuda(),
                                            lens.cuda())
    ref.check(got, *ref.prefix_attention(q, cache, none, 0, table, lens, D ** -0.5))


def test_many_tokens_with_few_blocks(cuda_device):
    """Row tiles in their hundreds with a short selection each: a warp a tile."""
    g = gen(92)
    for T, Hq, Hkv, D, page in ((330, 8, 2, 128, 16), (90, 14, 7, 64, 64), (40, 32, 16, 256, 32)):
        width = 12
        q, cache, table, _ = paged_inputs(g, T, Hq, Hkv, D, page, T, width)
        lens = ints(g, 0, width * page, T)
        blocks = random_blocks(g, T, Hkv, 512 // page if page < 64 else 5, width, lens, page)
        got = kvq.paged_block_sparse_attention(q.cuda(), cache.cuda(), table.cuda(), blocks.cuda(),
                                               lens.cuda())
        ref.check(got, *ref.sparse_attention(q, cache, table, blocks, lens, D ** -0.5))


def test_no_tokens(cuda_device):
    cache = torch.zeros(4, 2, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    bounds = torch.zeros(4, 2, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    i64 = torch.zeros(0, dtype=torch.int64, device="cuda")
    kvq.paged_kv_rope_append(torch.zeros(0, 512, dtype=torch.bfloat16, device="cuda"), 4, 2, 64,
                             None, True, None, i64, cache)
    kvq.paged_kv_page_bounds(cache, i64, i32(0), bounds)
    assert kvq.paged_kv_block_select(q, bounds, i32(3, 5), i32(0), 16, 2).shape == (0, 2, 2)
    assert kvq.paged_block_sparse_attention(q, cache, i32(3, 5), i32(0, 2, 2),
                                            i32(0)).shape == (0, 4, 64)
    assert kvq.paged_shared_prefix_attention(q, cache, i32(2), 20, i32(3, 5),
                                             i32(0)).shape == (0, 4, 64)


def test_pinned_host_tensors(cuda_device, prefix_way):
    """The cache and the inputs in pinned host memory: the same results, bit
    for bit, as from device memory (the tiles take device memory alone)."""
    g = gen(93)
    T, Hq, Hkv, D, page, width, prefix, topk = 20, 8, 2, 64, 16, 8, 90, 3
    q, cache, table, spare = paged_inputs(g, T, Hq, Hkv, D, page, T, width, extra=6)
    bounds = bounds_of(g, cache.shape[0], Hkv, D)
    lens = ints(g, 1, width * page, T)
    pages = spare.int()
    old = kvq.set_config("prefix", 0) if prefix_way == "tiles" else None

    def run(where):
        x = [where(t) for t in (q, cache, table, bounds, lens, pages)]
        blocks = kvq.paged_kv_block_select(x[0], x[3], x[2], x[4], page, topk)
        a = kvq.paged_block_sparse_attention(x[0], x[1], x[2], blocks, x[4])
        b = kvq.paged_shared_prefix_attention(x[0], x[1], x[5], prefix, x[2], x[4])
        torch.cuda.synchronize()
        return blocks.cpu(), bits(a), bits(b)

    want = run(lambda t: t.cuda())
    if old is not None:
        kvq.set_config("prefix", old)
    for a, b in zip(run(lambda t: t.pin_memory()), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("page,q_len,Hq,Hkv,D", [(16, 4, 4, 1, 64), (64, 3, 8, 2, 128), (5, 4, 2, 1, 64),
                                                 (16, 2, 16, 1, 256), (128, 16, 1, 1, 64)])
def test_causal_chunk_of_a_request(cuda_device, prefix_way, page, q_len, Hq, Hkv, D):
    """Tokens of one request that see different lengths of it share its pages
    in a CTA; what only a later one sees (here NaN) stays with that one."""
    g = gen(page + q_len)
    R, width, prefix = 7, -(-90 // page), 40
    T = R * q_len
    q, cache, table, spare = paged_inputs(g, T, Hq, Hkv, D, page, R, width,
                                          extra=-(-prefix // page))
    requests = (torch.arange(T) // q_len).int()
    lens = ints(g, 1, 60, R).repeat_interleave(q_len) + (torch.arange(T) % q_len).int()
    lens[q_len:2 * q_len] = lens[q_len:2 * q_len].flip(0)  # any order of the lengths
    last = int(lens[2 * q_len - 1 + q_len])                # request 2's longest length
    spoiled = cache.clone()
    at = last - 1
    spoiled[table[2, at // page].long(), :, :, at % page] = NAN
    args = (spare.int().cuda(), prefix, table.cuda(), lens.cuda())
    got = [kvq.paged_shared_prefix_attention(q.cuda(), c.cuda(), *args,
                                             requests=requests.cuda()).cpu()
           for c in (cache, spoiled)]
    want, tol = ref.prefix_attention(q, cache, spare, prefix, table, lens, D ** -0.5, requests)
    ref.check(got[0], want, tol)
    sees = (requests == 2) & (lens >= last)
    assert int(sees.sum()) == 1 and bool(got[1][sees].isnan().all())
    assert torch.equal(bits(got[0][~sees]), bits(got[1][~sees]))


def test_without_programmatic_launches(cuda_device, prefix_way):
    """Ordinary launches give the same results, bit for bit."""
    s = decode_state(95, B=40)
    qkv = normal(gen(96), s["B"], (s["Hq"] + 2 * s["Hkv"]) * s["D"]).cuda()
    results = []
    for programmatic in (True, False):
        d = on_gpu(s)
        fill_bounds(d)
        old = kvq.set_programmatic_launch(programmatic)
        try:
            outs = [step(d, qkv) for _ in range(3)]
        finally:
            kvq.set_programmatic_launch(old)
        torch.cuda.synchronize()
        results.append([bits(t.view(torch.int16)) for out in outs for t in out] + [bits(d["cache"])])
    for a, b in zip(*results):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,Hq,Hkv,page,prefix", [
    (70, 16, 2, 64, 3000), (300, 4, 2, 8, 1290), (17, 1, 1, 16, 128), (129, 2, 2, 32, 129),
    (64, 2, 1, 128, 20000), (257, 5, 1, 1024, 1500), (700, 2, 1, 64, 640), (40, 32, 8, 256, 77)])
@pytest.mark.parametrize("std", [1.0, 100.0])
def test_prefix_attention_of_heads_of_256(cuda_device, prefix_way, T, Hq, Hkv, page, prefix, std):
    """A row tile, several, and a row more; a block of the prefix, a key more,
    and many; with large scores, whose maxima keep moving, as well."""
    g = gen(97 + T + prefix)
    D, width, P = 256, 2 if page < 64 else 1, -(-prefix // page)
    q, cache, table, spare = paged_inputs(g, T, Hq, Hkv, D, page, T, width, extra=P + 1, std=std)
    lens = ints(g, 0, min(width * page, 40), T)
    pages = spare[:P].int()
    outside = P > 4
    if outside:
        pages[2] = cache.shape[0] + 1
    err = counter()
    args = (q.cuda(), cache.cuda(), pages.cuda(), prefix, table.cuda(), lens.cuda())
    got = kvq.paged_shared_prefix_attention(*args, scale=-0.05, errors=err)
    again = kvq.paged_shared_prefix_attention(*args, scale=-0.05)
    want, tol = ref.prefix_attention(q, cache, pages, prefix, table, lens, -0.05)
    ref.check(got, want, tol)
    assert torch.equal(bits(got), bits(again))
    assert (int(err.item()) > 0) == outside


@pytest.mark.parametrize("T,Hkv,D,width,topk", [
    (40, 8, 128, 1024, 32), (160, 1, 256, 130, 16), (62, 5, 64, 600, 300), (310, 1, 128, 300, 200),
    (77, 4, 64, 1025, 7), (153, 1, 256, 16, 15)])
def test_block_select_of_many_tokens(cuda_device, T, Hkv, D, width, topk):
    """More tokens and heads than CTAs that run at once, for some of them with
    equal blocks, with scores that fp32 cannot order, and with zero queries."""
    g = gen(98 + T + width)
    page = 16
    bounds = bounds_of(g, width + 40, Hkv, D)
    few = width // 3
    bounds[:few] = bounds[0]  # equal
    bounds[few:2 * few] = bounds[few]  # these differ where the query is tiny
    bounds[few:2 * few, :, 1, 5] = (1 + torch.arange(few)[:, None] / 1024).bfloat16()
    q = normal(g, T, 2 * Hkv, D)
    q[:, :, 5] = 2.0 ** -22
    q[1::7] = 0
    rows = torch.stack([torch.randperm(width, generator=g) for _ in range(3)]).int()
    spread = torch.randperm(width + 40, generator=g)[:width].int()
    table = torch.cat([rows, spread[None]])
    requests = ints(g, 0, 3, T)
    lens = ints(g, 0, width * page, T)
    lens[:T // 2] = width * page
    err = counter()
    got = run_select(q, bounds, table, lens, page, topk, 1, 1, requests=requests, errors=err)
    assert torch.equal(got, ref.select(q, bounds, table, lens, page, topk, 1, 1, requests))
    assert int(err.item()) == 0


@pytest.mark.parametrize("scale", [0.0, 1e-42, -1e-42])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefix_attention_with_no_or_hardly_any_scale(cuda_device, prefix_way, D, scale):
    """A scale of zero: the mean of the values that exist, in a partly filled
    block and beside a page outside the cache as well."""
    g = gen(99 + D)
    T, Hq, Hkv, page, width, prefix = 40, 4, 1, 16, 2, 300
    q, cache, table, spare = paged_inputs(g, T, Hq, Hkv, D, page, T, width, extra=19)
    pages = spare.int()
    pages[5] = -2
    lens = ints(g, 0, width * page, T)
    got = kvq.paged_shared_prefix_attention(q.cuda(), cache.cuda(), pages.cuda(), prefix,
                                            table.cuda(), lens.cuda(), scale=scale)
    ref.check(got, *ref.prefix_attention(q, cache, pages, prefix, table, lens, scale))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_lists_longer_than_a_cta_keeps(cuda_device, D):
    """More row tiles than CTAs that are resident, and of a few tokens more
    pages than a CTA lists at a time."""
    g = gen(100 + D)
    T, Hq, Hkv, page, topk = 165, 4, 2, 16, 2600
    N = 500
    q, cache = normal(g, T, Hq, D), normal(g, N, 2, Hkv, page, D)
    table = ints(g, 0, N - 1, T, topk)
    lens = ints(g, 0, 40, T)
    lens[3], lens[100], lens[164] = topk * page, 513 * page, 2048 * page + 1
    blocks = torch.full((T, Hkv, topk), -1, dtype=torch.int32)
    for t in range(T):
        n = -(-int(lens[t]) // page)
        for h in range(Hkv):
            blocks[t, h, topk - n:] = torch.randperm(n, generator=g).int()
    got = kvq.paged_block_sparse_attention(q.cuda(), cache.cuda(), table.cuda(), blocks.cuda(),
                                           lens.cuda())
    ref.check(got, *ref.sparse_attention(q, cache, table, blocks, lens, D ** -0.5))


@pytest.mark.parametrize("raw", [False, True])
def test_memory_of_a_call_on_a_given_stream(cuda_device, prefix_way, raw):
    """What a call on a stream of its own allocates is not memory that work of
    the current stream, which is behind, still writes."""
    g = gen(101)
    T, Hq, Hkv, D, page, width, prefix = 70, 8, 1, 128, 64, 1, 3000
    q, cache, table, spare = paged_inputs(g, T, Hq, Hkv, D, page, T, width, extra=47)
    lens = ints(g, 0, page, T)
    want, tol = ref.prefix_attention(q, cache, spare, prefix, table, lens, D ** -0.5)
    args = [t.cuda() for t in (q, cache, spare.int())] + [prefix] + [t.cuda() for t in (table, lens)]
    blocks = torch.zeros(T, Hkv, 1, dtype=torch.int32, device="cuda")
    bounds = torch.zeros(cache.shape[0], Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
    need = kvq.lib().paged_shared_prefix_attention_workspace(T, Hq, Hkv, D, page, prefix, width)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    for _ in range(3):
        torch.cuda.synchronize()
        junk = [torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
                for n in (need, T * Hq * D * 2, T * Hkv * 4) for _ in range(2)]
        torch.cuda._sleep(10000000)  # about five milliseconds, in front of the filling
        for x in junk:
            x.fill_(255)
        del x, junk  # back to the current stream's memory, the filling still to come
        out = kvq.paged_shared_prefix_attention(*args, stream=stream)
        sparse = kvq.paged_block_sparse_attention(args[0], args[1], args[4], blocks, args[5],
                                                  stream=stream)
        picked = kvq.paged_kv_block_select(args[0], bounds, args[4], args[5], page, 1,
                                           stream=stream)
        torch.cuda.synchronize()
        ref.check(out, want, tol)
        ref.check(sparse, *ref.sparse_attention(q, cache, table, blocks.cpu(), lens, D ** -0.5))
        assert bool((picked.cpu().view(T) == torch.where(lens > 0, 0, -1)).all())
    with torch.cuda.stream(side):  # the default stream, asked for by its handle
        blocks = kvq.paged_kv_block_select(args[0], bounds, args[4], args[5], page, 1, stream=0)
        again = kvq.paged_shared_prefix_attention(*args, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(blocks.cpu(), picked.cpu()) and torch.equal(bits(again), bits(out))
