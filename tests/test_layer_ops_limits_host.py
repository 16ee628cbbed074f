"""Host-side checks of the cache, attention, rotary and norm calls at the ends of their ranges (no GPU)."""
import ctypes

import pytest
import torch

from test_layer_ops_host import A, ALIGN, B, C, D, E, F, SHAPE, cache, lib  # noqa: F401 (lib is a fixture)


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
        c = cache(fmt=fmt, pages=pages, heads=heads, page=page, dim=256)
        p = ctypes.addressof(c)
        assert lib.nf4_kv_append(p, E, E + 65536, F, 4, None) == SHAPE
        assert lib.nf4_kv_read(p, F, 4, E, E + 65536, None) == SHAPE
        assert lib.nf4_attention_workspace_bytes(p, 2, heads) == -1
    fits = cache(pages=1 << 24, heads=1, page=65536, dim=256)  # 2^40 vectors
    assert lib.nf4_attention_workspace_bytes(ctypes.addressof(fits), 2, 4) > 0


def test_integers_of_a_cut_batch(lib):  # noqa: F811
    """lengths, page_table and positions that begin at any element are taken: with no GPU here, refused for that alone."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    c = cache()
    p = ctypes.addressof(c)
    ws = lib.nf4_attention_workspace_bytes(p, 3, 4)

    def attention(table, lengths):
        return lib.nf4_attention_decode(p, E, table, 5, lengths, 3, 4, 1.0, 0, E + 65536, F + (1 << 30), ws, None)

    def rope(positions):
        return lib.nf4_rope(A, 4, B, 2, 3, 128, positions, 1, (ctypes.c_int32 * 1)(64), D, 128, 0, 1.0, E, F, None)

    for off in (4, 8, 12):
        assert attention(F + off, F + 4096) in (5, 6) and attention(F, F + 4096 + off) in (5, 6)
        assert rope(C + off) in (5, 6)
    for off in (1, 2, 6):
        assert attention(F + off, F + 4096) == ALIGN and attention(F, F + 4096 + off) == ALIGN and rope(C + off) == ALIGN


def test_outputs_that_are_left_out(monkeypatch):
    """A missing output is a ValueError that names it."""
    import nf4_weight_only_gb300 as nf4
    from nf4_weight_only_gb300 import build
    build.build()
    q, f = torch.zeros(1, 2, 64, dtype=torch.bfloat16), torch.zeros(32)
    positions = torch.zeros(1, 1, dtype=torch.int32)
    real = nf4._expect
    # CPU tensors pass, so that the missing one is what is met
    monkeypatch.setattr(nf4, "_expect", lambda t, *a: 0 if isinstance(t, torch.Tensor) else real(t, *a))
    with pytest.raises(ValueError, match="q_out: want a tensor"):
        nf4.nf4_rope(q, None, positions, f, None, None)
    with pytest.raises(ValueError, match="k_out: want a tensor"):
        nf4.nf4_rope(None, q, positions, f, None, None)
    with pytest.raises(ValueError, match="out: want a tensor"):
        cache = type("Cache", (), {"_address": 0, "head_dim": 64})
        nf4.nf4_attention_decode(cache, q, positions, positions[0], None, torch.zeros(16, dtype=torch.uint8))
