"""Attention over a 4-bit cache where there are too many rows for clusters and the keys
are cut in parts of 2048 or 4096, each a CTA's, joined by a second launch."""
import pytest
import torch

import kv4_ref as ref4
import kv_quant_cache_gb300 as kvq
import paged_ref as ref

pytestmark = pytest.mark.gpu


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16)


def case(B, per, Hq, Hkv, D, page, width, seed, pool=300):
    """Requests that share the pages of a small cache, in orders of their own."""
    g = torch.Generator().manual_seed(seed)
    raw = ref4.random_cache(g, pool, Hkv, page, D)
    table = torch.randint(0, pool, (B, width), generator=g, dtype=torch.int32)
    return torch.randn(B * per, Hq, D, generator=g).bfloat16(), raw, table


def parts(q, raw, table, per):
    """Parts that the call's workspace has room for (0: none)."""
    T, Hq, D = q.shape
    need = kvq.lib().paged_kv4_attention_workspace(T, per, Hq, raw.shape[2], D, raw.shape[3],
                                                   table.shape[1])
    assert need % (T * Hq * (D + 1) * 4) == 0
    return need // (T * Hq * (D + 1) * 4)


def check(out, q, raw, table, lens, per, some):
    """The tokens ``some`` against the fp64 form."""
    want = ref4.attention(q[some], raw, table[some // per], lens[some], q.shape[2] ** -0.5)
    ref.check(out[some.cuda()], *want)


# size of a part, parts, and the call
CASES = [(2048, 5, (160, 2, 8, 1, 256, 16, 563)), (2048, 3, (400, 1, 8, 1, 64, 48, 100)),
         (2048, 3, (160, 3, 4, 1, 128, 64, 70)), (2048, 3, (80, 5, 8, 1, 64, 64, 70)),
         (2048, 3, (160, 1, 10, 2, 128, 32, 150)), (4096, 13, (160, 1, 8, 1, 256, 64, 800))]


@pytest.mark.parametrize("size,count,sizes", CASES)
def test_parts_of_a_fixed_size(cuda_device, size, count, sizes):
    """Lengths around the borders of parts, of steps within them and of the table, tokens of
    a request with different ones; the workspace holds NaN before."""
    B, per, Hq, Hkv, D, page, width = sizes
    q, raw, table = case(*sizes, seed=D + width)
    assert parts(q, raw, table, per) == count == -(-width * page // size)
    most = width * page
    ends = [most, 0, size - 1, size, size + 1, 1, 2 * size - 1, 2 * size, 2 * size + 1, size + 16,
            most - 1, size + 17, (count - 1) * size, (count - 1) * size + 1, 2 * size - 16, 777]
    T = B * per
    lens = torch.tensor([ends[t % len(ends)] for t in range(T)], dtype=torch.int32)
    need = kvq.lib().paged_kv4_attention_workspace(T, per, Hq, Hkv, D, page, width)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    args = [x.cuda() for x in (q, raw, table, lens)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = kvq.paged_kv4_attention(*args, tokens_per_request=per, workspace=ws, errors=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    some = torch.arange(len(ends)) + T // 2
    check(out, q, raw, table, lens, per, some)
    assert bool((out[lens.cuda() == 0] == 0).all()) and not bool(out.isnan().any())
    again = kvq.paged_kv4_attention(*args, tokens_per_request=per)
    assert torch.equal(bits(again), bits(out))


def test_bad_pages_and_lengths_in_later_parts(cuda_device):
    """Pages outside the cache, lengths past the table and below zero, in a graph that is
    replayed after the lengths have changed."""
    B, width, page = 400, 100, 48
    q, raw, table = case(B, 1, 8, 1, 64, page, width, seed=7)
    assert parts(q, raw, table, 1) == 3
    g = torch.Generator().manual_seed(8)
    table[torch.rand(B, width, generator=g) < 0.1] = raw.shape[0]
    table[3, 42:] = -1  # the whole second part and the third
    args = [x.cuda() for x in (q, raw, table, torch.zeros(B, dtype=torch.int32))]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = kvq.paged_kv4_attention(*args, errors=err)
    for shift in (0, 1900):
        lens = (torch.arange(B, dtype=torch.int32) * 37 + shift) % (width * page + 1)
        lens[5], lens[6], lens[7] = width * page + 1, -5, 2 ** 31 - 1
        lens[3] = width * page
        args[3].copy_(lens)
        err.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert int(err.item()) > 0
        check(out, q, raw, table, lens, 1, torch.tensor([0, 1, 3, 5, 6, 7, 100, 128, 200, 399]))


@pytest.mark.parametrize("D,per,G,B,page,count", [(64, 1, 8, 400, 64, 30), (128, 2, 8, 160, 64, 30),
                                                  (256, 1, 8, 320, 128, 15)])
def test_a_table_much_wider_than_the_requests(cuda_device, D, per, G, B, page, count):
    """A table for 131072 keys over requests of a few thousand, and some as long as it: 16
    waves of parts, which the longest requests fill with larger ones. Parts past a request's
    end leave their place in the workspace as it was."""
    width = 131072 // page
    q, raw, table = case(B, per, G, 1, D, page, width, seed=D + per)
    assert parts(q, raw, table, per) == count
    T = B * per
    g = torch.Generator().manual_seed(9)
    lens = torch.randint(0, 4097, (T,), generator=g, dtype=torch.int32)
    some = torch.arange(12) + T // 2
    lens[some] = torch.tensor([131072, 131071, count * 4096, count * 4096 - 1, 0, 0, 4096, 4096, 60000,
                               60000, 8, 3000], dtype=torch.int32)
    if per == 1:
        lens[T // 3], some = count * 4096 + 1, torch.cat([some, torch.tensor([T // 3])])
    need = kvq.lib().paged_kv4_attention_workspace(T, per, G, 1, D, page, width)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    args = [x.cuda() for x in (q, raw, table, lens)]
    out = kvq.paged_kv4_attention(*args, tokens_per_request=per, workspace=ws)
    torch.cuda.synchronize()
    check(out, q, raw, table, lens, per, some)
    assert bool((out[lens.cuda() == 0] == 0).all()) and not bool(out.isnan().any())
    # rows of requests of up to 4096 keys: the first part's alone are written
    held = ws.view(torch.int32)[:count * T * G * D].view(count, T, G * D)
    short = (lens.view(B, per).amax(1) <= 4096).repeat_interleave(per).cuda()
    assert bool((held[1:, short] == -1).all())
    # the same requests behind a table that ends with them
    short = short.nonzero()[:, 0]
    n = len(short) // per
    tight = args[2][short[::per] // per, :4096 // page].contiguous()
    again = kvq.paged_kv4_attention(args[0][short], args[1], tight, args[3][short],
                                    tokens_per_request=per)
    assert tight.shape[0] == n
    want = ref4.attention(q[short.cpu()][:8], raw, table[short.cpu()[:8] // per], lens[short.cpu()[:8]],
                          D ** -0.5)
    ref.check(again[:8], *want)
    ref.check(out[short[:8]], *want)
