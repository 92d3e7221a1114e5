"""What the attentions over quantised caches make of a call's sizes, on the host: seen
through the workspace that they ask for.  No call here reaches a kernel launch."""
import pytest

import kv_quant_cache_gb300 as kvq
from kv_quant_cache_gb300 import _build


@pytest.fixture(scope="module")
def L():
    _build.build()
    return kvq.lib()


def test_tiles_that_are_shared_out_are_counted_in_32_bits(L):
    """Blocks of 64 heads times tiles of 128 entries past 2^31 - 1 are a CTA to a unit, which
    needs no workspace; up to there they are shared out."""
    f = L.dsv4_latent_attention_workspace
    shared = 152 * 2 * 64 * 514 * 4
    wide = 2 ** 30  # entries, 2^23 tiles
    assert f(1, 64 * 256, wide) == 0 and f(1, 64 * 608, wide) == 0 and f(8, 64 * 76, wide) == 0
    assert f(1, 64 * 256, wide - 128) == f(1, 64 * 255, wide) == f(51, 64 * 5, wide) == shared
    assert f(608, 64, wide) == 0 and f(255, 64, wide) == f(608, 64, 2 ** 28) == shared
    assert f(1, 64 * 609, 4096) == 0  # more units than are shared out
