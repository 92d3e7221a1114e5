"""The paged grouped-query operators on the host: validation by the C ABI and
by the Python binding, workspace sizes, and the plain fp64 forms the GPU tests
compare with.  No call here reaches a kernel launch."""
import ctypes
import math

import pytest
import torch

import kv_quant_cache_gb300 as kvq
import paged_ref as ref
from kv_quant_cache_gb300 import _build

A = 0x10000    # fake, never-dereferenced device addresses
MIS = 0x10002


@pytest.fixture(scope="module")
def L():
    _build.build()
    return kvq.lib()


def rejected(status):
    """The call came back from validation (and launched nothing)."""
    assert status not in (kvq.KVQ_OK, kvq.KVQ_ERR_CUDA)
    return status


def append(L, qkv=A, q_out=None, T=4, Hq=4, Hkv=2, D=128, cs=A, max_pos=16, rot=128, neox=1,
           pos=A, slots=A, cache=A, pages=8, page=16, err=None):
    return L.paged_kv_rope_append(qkv, q_out, T, Hq, Hkv, D, cs, max_pos, rot, neox, pos, slots,
                                  cache, pages, page, err, None)


def test_append_validation(L):
    bad = lambda **k: rejected(append(L, **k))  # noqa: E731
    for name in ("qkv", "cs", "pos", "slots", "cache"):
        assert bad(**{name: None}) == kvq.KVQ_ERR_NULL
        assert bad(**{name: MIS}) == kvq.KVQ_ERR_ALIGN
    assert bad(q_out=MIS) == kvq.KVQ_ERR_ALIGN
    assert bad(err=MIS + 1) == kvq.KVQ_ERR_ALIGN
    for k in (dict(T=-1), dict(Hq=-1), dict(Hkv=0), dict(page=0), dict(page=65537),
              dict(pages=-1), dict(pages=2 ** 31), dict(max_pos=-1), dict(T=2 ** 31),
              dict(T=2 ** 30), dict(T=2 ** 62), dict(Hq=2 ** 31 - 1), dict(Hkv=2 ** 31 - 1)):
        assert bad(**k) == kvq.KVQ_ERR_SHAPE, k
    for k in (dict(D=96), dict(D=512), dict(neox=2), dict(rot=8), dict(rot=24), dict(rot=144),
              dict(rot=-16)):
        assert bad(**k) == kvq.KVQ_ERR_UNSUPPORTED, k
    # q_out within, across the end and across the start of qkv
    nbytes = 4 * 8 * 128 * 2
    for at in (A, A + 16, A + nbytes - 16, A - 16):
        assert bad(q_out=at) == kvq.KVQ_ERR_VALUE
    assert append(L, T=0, qkv=None, cs=None, pos=None, slots=None, cache=None) == kvq.KVQ_OK
    # without a rotation the table and the positions are not asked for
    assert bad(rot=0, cs=None, pos=None, cache=None) == kvq.KVQ_ERR_NULL


def test_page_bounds_validation(L):
    def call(cache=A, pages=8, Hkv=2, page=16, D=64, ids=A, lens=A, n=3, bounds=A, err=None):
        return L.paged_kv_page_bounds(cache, pages, Hkv, page, D, ids, lens, n, bounds, err, None)
    for name in ("cache", "ids", "lens", "bounds"):
        assert rejected(call(**{name: None})) == kvq.KVQ_ERR_NULL
        assert rejected(call(**{name: MIS})) == kvq.KVQ_ERR_ALIGN
    for k in (dict(n=-1), dict(n=2 ** 31), dict(n=2 ** 30), dict(Hkv=0), dict(page=0),
              dict(pages=-1)):
        assert rejected(call(**k)) == kvq.KVQ_ERR_SHAPE, k
    assert rejected(call(D=32)) == kvq.KVQ_ERR_UNSUPPORTED
    assert call(n=0, cache=None, ids=None, lens=None, bounds=None) == kvq.KVQ_OK


QUERY = dict(q=A, stride=512, T=4, Hq=4, Hkv=2, D=128, cache=A, pages=8, page=16, table=A, R=4,
             width=5, req=None, lens=A)
BAD_QUERY = [
    (dict(q=None), 1), (dict(cache=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(T=-1), 2), (dict(T=2 ** 31), 2), (dict(T=2 ** 62), 2), (dict(Hq=3), 2), (dict(Hq=0), 2),
    (dict(Hkv=0), 2), (dict(page=0), 2), (dict(pages=-1), 2), (dict(R=-1), 2), (dict(width=-1), 2),
    (dict(width=2 ** 22 + 1), 2), (dict(R=3), 2), (dict(stride=511), 2), (dict(stride=2 ** 40), 2),
    (dict(D=96), 3), (dict(q=A + 8), 4), (dict(stride=516), 4), (dict(cache=A + 8), 4),
    (dict(table=MIS), 4), (dict(req=MIS), 4), (dict(lens=MIS), 4), (dict(err=MIS), 4)]


def select(L, topk=3, first=0, last=0, blocks=A, err=None, **k):
    x = {**QUERY, **k}
    return L.paged_kv_block_select(x["q"], x["stride"], x["T"], x["Hq"], x["Hkv"], x["D"],
                                   x["cache"], x["pages"], x["page"], x["table"], x["R"],
                                   x["width"], x["req"], x["lens"], topk, first, last, blocks, err,
                                   None)


def sparse(L, blocks=A, topk=3, scale=0.1, out=0x900000, ws=0x800000, ws_bytes=1 << 40, err=None,
           **k):
    x = {**QUERY, **k}
    return L.paged_block_sparse_attention(x["q"], x["stride"], x["T"], x["Hq"], x["Hkv"], x["D"],
                                          x["cache"], x["pages"], x["page"], x["table"], x["R"],
                                          x["width"], x["req"], x["lens"], blocks, topk, scale,
                                          out, ws, ws_bytes, err, None)


def prefix(L, ids=A, length=50, scale=0.1, out=0x900000, ws=0x800000, ws_bytes=1 << 40, err=None,
           **k):
    x = {**QUERY, **k}
    return L.paged_shared_prefix_attention(x["q"], x["stride"], x["T"], x["Hq"], x["Hkv"], x["D"],
                                           x["cache"], x["pages"], x["page"], ids, length,
                                           x["table"], x["R"], x["width"], x["req"], x["lens"],
                                           scale, out, ws, ws_bytes, err, None)


@pytest.mark.parametrize("call", [select, sparse, prefix])
def test_query_validation(L, call):
    for k, want in BAD_QUERY:
        if call is select and k == dict(width=2 ** 22 + 1):
            continue
        assert rejected(call(L, **k)) == want, k
    assert call(L, T=0, q=None, cache=None, table=None, lens=None) == kvq.KVQ_OK


def test_select_validation(L):
    for k in (dict(topk=0), dict(topk=-1), dict(first=-1), dict(last=-1), dict(T=2 ** 28),
              dict(width=2 ** 22 + 1)):
        assert rejected(select(L, **k)) == kvq.KVQ_ERR_SHAPE, k
    assert rejected(select(L, width=16385)) == kvq.KVQ_ERR_UNSUPPORTED
    assert rejected(select(L, blocks=None)) == kvq.KVQ_ERR_NULL
    assert rejected(select(L, blocks=MIS)) == kvq.KVQ_ERR_ALIGN


@pytest.mark.parametrize("call", [sparse, prefix])
def test_attention_validation(L, call):
    # sizes whose call needs a workspace: a long range that few rows see
    big = dict(T=1, R=1, Hq=4, Hkv=1, stride=512, page=64, width=2048)
    big.update(topk=2048) if call is sparse else big.update(length=131072)
    need = (L.paged_block_sparse_attention_workspace(1, 4, 1, 128, 64, 2048) if call is sparse else
            L.paged_shared_prefix_attention_workspace(1, 4, 1, 128, 64, 131072, 2048))
    assert need > 0 and need % 16 == 0
    assert rejected(call(L, ws=None, **big)) == kvq.KVQ_ERR_NULL
    assert rejected(call(L, ws=MIS, **big)) == kvq.KVQ_ERR_ALIGN
    assert rejected(call(L, ws_bytes=need - 1, **big)) == kvq.KVQ_ERR_SHAPE
    assert rejected(call(L, out=None, **big)) == kvq.KVQ_ERR_NULL
    assert rejected(call(L, out=A + 8, **big)) == kvq.KVQ_ERR_ALIGN
    for at in (A, A + 512, A - 512):  # out over q
        assert rejected(call(L, out=at, **big)) == kvq.KVQ_ERR_VALUE
    for scale in (math.nan, math.inf):
        assert rejected(call(L, scale=scale, **big)) == kvq.KVQ_ERR_VALUE


def test_key_list_validation(L):
    assert rejected(sparse(L, blocks=None)) == kvq.KVQ_ERR_NULL
    assert rejected(sparse(L, blocks=MIS)) == kvq.KVQ_ERR_ALIGN
    assert rejected(sparse(L, topk=0)) == kvq.KVQ_ERR_SHAPE
    assert rejected(sparse(L, topk=2 ** 22 + 1)) == kvq.KVQ_ERR_SHAPE
    assert rejected(prefix(L, ids=None)) == kvq.KVQ_ERR_NULL
    assert rejected(prefix(L, ids=MIS)) == kvq.KVQ_ERR_ALIGN
    for length in (-1, 2 ** 31, 2 ** 22 * 16 + 1, 2 ** 62):
        assert rejected(prefix(L, length=length)) == kvq.KVQ_ERR_SHAPE


def test_workspace_of_sizes_that_no_call_takes(L):
    f, g = L.paged_block_sparse_attention_workspace, L.paged_shared_prefix_attention_workspace
    for args in ((0, 4, 2, 128, 16, 3), (4, 3, 2, 128, 16, 3), (4, 4, 0, 128, 16, 3),
                 (4, 4, 2, 96, 16, 3), (4, 4, 2, 128, 0, 3), (4, 4, 2, 128, 16, 0)):
        assert f(*args) == 0
    for args in ((0, 4, 2, 128, 16, 3, 3), (4, 4, 2, 128, 16, -1, 3), (4, 4, 2, 128, 16, 3, -1),
                 (4, 4, 2, 128, 16, 2 ** 62, 3)):
        assert g(*args) == 0
    assert g(4, 4, 2, 128, 16, 0, 0) == 0


def test_binding_checks():
    cache = torch.zeros(4, 2, 2, 16, 64, dtype=torch.bfloat16)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    blocks = torch.zeros(3, 2, 2, dtype=torch.int32)
    bounds = torch.zeros(4, 2, 2, 64, dtype=torch.bfloat16)
    ids = torch.zeros(3, dtype=torch.int64)
    qkv = torch.zeros(3, 8 * 64, dtype=torch.bfloat16)
    cs = torch.zeros(9, 64)
    calls = [
        lambda: kvq.paged_kv_rope_append(qkv[:, 64:], 4, 2, 64, cs, True, ids, ids, cache),
        lambda: kvq.paged_kv_rope_append(qkv, 4, 2, 64, cs, True, ids, ids, cache[:, :1]),
        lambda: kvq.paged_kv_rope_append(qkv, 4, 2, 64, cs, True, ids[:2], ids, cache),
        lambda: kvq.paged_kv_rope_append(qkv, 4, 2, 64, cs, True, ids, ids[:2], cache),
        lambda: kvq.paged_kv_rope_append(qkv, 4, 2, 64, cs, True, ids, ids, cache, q_out=q[:2]),
        lambda: kvq.paged_kv_rope_append(qkv, 4, 2, 64, cs, True, ids, ids, cache, rotary_dim=32),
        lambda: kvq.paged_kv_rope_append(qkv, 4, 2, 64, None, True, ids, ids, cache, rotary_dim=32),
        lambda: kvq.paged_kv_page_bounds(cache, ids, lens[:2], bounds),
        lambda: kvq.paged_kv_page_bounds(cache, ids, lens, bounds[:3]),
        lambda: kvq.paged_kv_block_select(q, bounds[..., :32], table, lens, 16, 2),
        lambda: kvq.paged_kv_block_select(q.float(), bounds, table, lens, 16, 2),
        lambda: kvq.paged_kv_block_select(q, bounds, table[:2], lens, 16, 2),
        lambda: kvq.paged_kv_block_select(q, bounds, table, lens[:2], 16, 2),
        lambda: kvq.paged_block_sparse_attention(q, cache, table, blocks[:2], lens),
        lambda: kvq.paged_block_sparse_attention(q, cache, table, blocks[:, :1], lens),
        lambda: kvq.paged_shared_prefix_attention(q, cache, lens, 49, table, lens),
        # everything in order, but on the host and not pinned
        lambda: kvq.paged_kv_rope_append(qkv, 4, 2, 64, cs, True, ids, ids, cache),
        lambda: kvq.paged_kv_page_bounds(cache, ids, lens, bounds),
        lambda: kvq.paged_kv_block_select(q, bounds, table, lens, 16, 2),
        lambda: kvq.paged_block_sparse_attention(q, cache, table, blocks, lens),
        lambda: kvq.paged_shared_prefix_attention(q, cache, lens, 48, table, lens),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was accepted")


def test_plain_forms_agree_with_torch():
    """The fp64 forms against independent torch formulas on one small case."""
    g = torch.Generator().manual_seed(1)
    q = torch.randn(2, 4, 64, generator=g).bfloat16()
    cache = torch.randn(6, 2, 2, 8, 64, generator=g).bfloat16()
    table = torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=torch.int32)
    lens = torch.tensor([20, 24], dtype=torch.int32)
    blocks = torch.tensor([0, 1, 2], dtype=torch.int32).expand(2, 2, 3)
    a, tol = ref.sparse_attention(q, cache, table, blocks, lens, 0.125)
    b, _ = ref.prefix_attention(q, cache, table[0, :0], 0, table, lens, 0.125)
    assert torch.allclose(a, b, rtol=0, atol=1e-12) and bool((tol > 0).all())
    k = cache[3:6, 0].transpose(0, 1).reshape(2, 24, 64).double()
    v = cache[3:6, 1].transpose(0, 1).reshape(2, 24, 64).double()
    w = torch.softmax(q[1].double().view(2, 2, 64) @ k.transpose(1, 2) * 0.125, -1)
    assert torch.allclose((w @ v).view(4, 64), a[1], rtol=0, atol=1e-12)
    # a rotation by zero angle leaves a row alone, one by a quarter turn swaps pairs
    x = torch.randn(3, 64, generator=g).double()
    flat = torch.cat([torch.ones(32), torch.zeros(32)]).double()
    assert torch.equal(ref.rotate(x, flat, 64, True)[0], x)
    y, _ = ref.rotate(x, flat.flip(0), 64, False)
    assert torch.equal(y[:, 0::2], -x[:, 1::2]) and torch.equal(y[:, 1::2], x[:, 0::2])
    # the score is the sum over heads of the larger product, dim by dim
    lo, hi = torch.randn(2, 1, 64, generator=g).sort(0).values.double()
    direct = torch.maximum(q[0].double() * lo, q[0].double() * hi).sum()
    got = ref.scores(q[0], torch.stack([lo, hi], 1), torch.tensor([0]))
    assert torch.allclose(got, direct[None], rtol=1e-12)


def test_prefix_configurations(L):
    assert [n.split("<")[0] for n in kvq.configs("prefix")] == ["rows", "tiles"]
    assert L.kvq_prefix_config_name(2) is None and L.kvq_prefix_config_name(-1) is None
    with pytest.raises(ValueError):
        kvq.set_config("prefix", 2)
    # few rows need no workspace; forced through the tiles they do, sizes the
    # tiles cannot take do not
    f = L.paged_shared_prefix_attention_workspace
    small, odd = (40, 8, 2, 128, 64, 500, 4), (40, 8, 2, 128, 24, 500, 4)
    assert f(*small) == 0 and f(*odd) == 0
    assert kvq.set_config("prefix", 1) == -1
    try:
        assert f(*small) > 0 and f(*odd) == 0
    finally:
        assert kvq.set_config("prefix", -1) == 1
    assert f(256, 64, 8, 128, 64, 32768, 8) > 0


def test_status_of_the_new_symbols(L):
    assert ctypes.sizeof(ctypes.c_int64) == 8
    for n in ("paged_kv_rope_append", "paged_kv_page_bounds", "paged_kv_block_select",
              "paged_block_sparse_attention", "paged_shared_prefix_attention"):
        assert hasattr(L, n) and callable(getattr(kvq, n))


def test_tile_wait_limit_round_trip(L):
    """The limit of the tiles' waits: returns the one before, 2^24 to start with."""
    old = kvq.set_tile_wait_limit(17)
    try:
        assert old == 1 << 24
        assert kvq.set_tile_wait_limit(0) == 17
        assert kvq.set_tile_wait_limit(2 ** 32 - 1) == 0
    finally:
        assert kvq.set_tile_wait_limit(old) == 2 ** 32 - 1


def test_size_found_while_the_configuration_changes(L, monkeypatch):
    """A workspace size that was computed under the setting before a change is
    not what later calls are given."""
    name, sizes = "paged_shared_prefix_attention_workspace", (40, 8, 2, 128, 64, 501, 4)

    class Changing:
        def __getattr__(self, symbol):
            f = getattr(L, symbol)
            if symbol != name:
                return f

            def size(*args):
                need = f(*args)
                kvq.set_config("prefix", 1)  # as another thread might
                return need
            return size

    assert kvq.set_config("prefix", -1) == -1
    try:
        with monkeypatch.context() as m:
            m.setattr(kvq, "lib", Changing)
            assert kvq._workspace_bytes(name, *sizes) == 0
        assert kvq._workspace_bytes(name, *sizes) == getattr(L, name)(*sizes) > 0
    finally:
        kvq.set_config("prefix", -1)


@pytest.mark.parametrize("raw", [True, False])
def test_workspace_of_a_call_on_pinned_tensors(monkeypatch, raw):
    """No device among the call's tensors: the workspace is the current
    device's, in the order of the call's stream, with torch's allocator by
    itself (``raw``) and with tensors from it."""
    made, calls = [], []

    def fn(*args):
        calls.append(args)
        return 0

    def new(shape, dtype, dev, stream):
        made.append((shape, dev, stream))
        return torch.zeros(shape, dtype=dtype)

    monkeypatch.setattr(kvq, "_current_device", lambda: 3)
    monkeypatch.setattr(kvq, "_stream", lambda stream, dev: 77)
    monkeypatch.setattr(kvq, "_new", new)
    monkeypatch.setattr(kvq, "_raw_alloc", lambda n, stream: made.append((n, stream)) or 4096)
    monkeypatch.setattr(kvq, "_raw_free", (lambda p: made.append(p)) if raw else None)
    kvq._launch_attention(-1, None, fn, (1, 2), None, 640, None)
    assert made == ([(640, 77), 4096] if raw else [(640, 3, None)])
    assert len(calls) == 1 and calls[0][:2] + calls[0][3:] == (1, 2, 640, None, 77)
    assert not raw or calls[0][2] == 4096
    kvq._launch_attention(-1, None, fn, (1, 2), None, 0, None)  # none needed, none made
    assert calls[1] == (1, 2, None, 0, None, 77) and len(made) == (2 if raw else 1)


@pytest.mark.parametrize("call", [sparse, prefix])
def test_scale_whose_logarithmic_form_overflows(L, call):
    """scale * log2(e) past the largest float: a score of zero would be NaN."""
    for scale in (2.5e38, -2.5e38, 3.4e38, math.nan, -math.inf):
        assert rejected(call(L, scale=scale)) == kvq.KVQ_ERR_VALUE


def test_host_tensors_without_elements():
    """torch calls no empty tensor pinned; a list without entries has to be
    taken all the same, of the right type only."""
    for dev in (-1, 0):
        assert kvq._ptr(torch.empty(0, dtype=torch.int32), torch.int32, dev, "pages") == 0
        with pytest.raises(ValueError):
            kvq._ptr(torch.empty(0, dtype=torch.int64), torch.int32, dev, "pages")
        with pytest.raises(ValueError):
            kvq._ptr(torch.zeros(1, dtype=torch.int32), torch.int32, dev, "pages")
    assert kvq._paged_q(torch.empty(0, 4, 64, dtype=torch.bfloat16), 64, -1)[1:] == (0, 4, 256)
