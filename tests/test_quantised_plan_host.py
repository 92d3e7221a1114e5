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


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,per", [(1, 1), (8, 1), (4, 3), (8, 4), (16, 19)])
def test_a_wide_table_costs_no_more_than_waves_of_partials(L, D, G, per):
    """The partials of a 4-bit cache's attention are those of 16 waves of CTAs at most (at most
    5 x 152 CTAs of 8 rows, 4 x 152 of 16 (64 dims) or 8, 2 x 152 of 32, of 16 with 256 dims),
    however wide the table: 256 tokens of 64 query and 8 kv heads asked for 270 MB with a table
    for 131072 keys, 300 tokens for 2.6 GB with the widest."""
    most = 16 * 2 * 152 * (16 if D == 256 else 32) * (D + 1) * 4
    assert most < 81 * 10 ** 6
    for tokens in (1, 7, 64, 256, 300, 3000, 50000):
        for Hkv in (1, 2, 8):
            for width in (1, 32, 64, 128, 1000, 2048, 8192, 2 ** 17, 2 ** 22):
                need = L.paged_kv4_attention_workspace(tokens * per, per, G * Hkv, Hkv, D, 64, width)
                assert need <= most, (tokens, Hkv, width)
