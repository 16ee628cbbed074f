"""Host-side checks of the cache, attention, rotary and norm calls at the ends of their ranges (no GPU)."""
import ctypes

import pytest

from test_layer_ops_host import E, F, SHAPE, cache, lib  # noqa: F401 (lib is a fixture)


@pytest.mark.parametrize("batch,q_heads", [(1, 65536), (1, 1 << 31), (1, 1 << 32), (1, 3 << 32), (65536, 1), (32768, 65535)])
def test_workspace_of_sizes_that_the_attention_refuses(lib, batch, q_heads):  # noqa: F811
    c = cache(heads=1)
    p = ctypes.addressof(c)
    assert lib.nf4_attention_workspace_bytes(p, batch, q_heads) == -1
    assert lib.nf4_attention_decode(p, E, F, 4, F + 4096, batch, q_heads, 1.0, 0, E + 65536, F + (1 << 30), 1 << 30,
                                    None) == SHAPE
    assert lib.nf4_attention_workspace_bytes(p, 65535, 16384) > 0 and lib.nf4_attention_workspace_bytes(p, 0, 65535) > 0


@pytest.mark.parametrize("pages,heads,page", [((1 << 31) - 1, 65535, 65536), (1 << 30, 8192, 65536), ((1 << 31) - 1, 33, 16),
                                              ((1 << 24) + 1, 1, 65536)])
def test_caches_of_more_bytes_than_64_bits_count(lib, pages, heads, page):  # noqa: F811
    """Each size is in its range; their product is not."""
    for fmt in (0, 1, 2):
        p = ctypes.addressof(cache(fmt=fmt, pages=pages, heads=heads, page=page, dim=256))
        assert lib.nf4_kv_append(p, E, E + 65536, F, 4, None) == SHAPE
        assert lib.nf4_kv_read(p, F, 4, E, E + 65536, None) == SHAPE
        assert lib.nf4_attention_workspace_bytes(p, 2, heads) == -1
    fits = cache(pages=1 << 24, heads=1, page=65536, dim=256)  # 2^40 vectors
    assert lib.nf4_attention_workspace_bytes(ctypes.addressof(fits), 2, 4) > 0
