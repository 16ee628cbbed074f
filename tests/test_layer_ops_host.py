"""Host-side checks of the cache, attention, rotary and norm calls (no GPU): argument errors come back
before any device work, and the binding refuses tensors of the wrong type, shape or device."""
import ctypes
import os

import pytest
import torch

A, B, C, D, E, F = (0x7F0000000000 + (i << 36) for i in range(6))  # fake device addresses, never read
vp = ctypes.c_void_p
OK, NULL, SHAPE, ALIGN, ALIAS = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    from nf4_weight_only_gb300 import build
    import nf4_weight_only_gb300 as nf4
    return nf4.load(build.build())


def cache(fmt=2, k=A, v=B, ks=C, vs=D, pages=4, heads=2, page=16, dim=128):
    import nf4_weight_only_gb300 as nf4
    return nf4._KvCacheStruct(k, v, ks, vs, pages, heads, page, dim, fmt)


BAD_CACHES = [
    (dict(fmt=3), SHAPE), (dict(fmt=-1), SHAPE), (dict(dim=96), SHAPE), (dict(dim=512), SHAPE), (dict(page=8), SHAPE),
    (dict(page=24), SHAPE), (dict(page=0), SHAPE), (dict(page=65552), SHAPE), (dict(heads=0), SHAPE),
    (dict(heads=65536), SHAPE), (dict(pages=-1), SHAPE), (dict(pages=1 << 31), SHAPE), (dict(k=0), NULL),
    (dict(vs=0), NULL), (dict(ks=0, fmt=1), NULL), (dict(k=A + 8), ALIGN), (dict(vs=D + 2), ALIGN),
]


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_cache_descriptions(lib, kw, want):
    c = cache(**kw)
    p = ctypes.addressof(c)
    assert lib.nf4_kv_append(p, E, E + 65536, F, 4, None) == want
    assert lib.nf4_kv_read(p, F, 4, E, E + 65536, None) == want
    assert lib.nf4_attention_decode(p, E, F, 4, F + 4096, 2, 4, 1.0, 0, E + 65536, F + (1 << 30), 1 << 30, None) == want
    if want == SHAPE:
        assert lib.nf4_attention_workspace_bytes(p, 2, 4) == -1


def test_append_and_read(lib):
    c = cache()
    p = ctypes.addressof(c)
    app, read = lib.nf4_kv_append, lib.nf4_kv_read
    assert app(None, E, E + 65536, F, 4, None) == NULL
    assert app(p, E, E, F, 0, None) == OK and read(p, F, 0, E, E, None) == OK
    assert read(p, F, 4, None, None, None) == OK  # nothing asked for
    assert app(p, E, E, F, -1, None) == SHAPE and read(p, F, 1 << 31, E, E + 65536, None) == SHAPE
    assert app(p, None, E, F, 4, None) == NULL and app(p, E, E, None, 4, None) == NULL
    assert app(p, E + 2, E, F, 4, None) == ALIGN and app(p, E, E, F + 8, 4, None) == ALIGN
    assert app(p, A + 64, E, F, 4, None) == ALIAS and app(p, E, E, C, 4, None) == ALIAS  # inputs inside the cache
    shared = cache(v=A + 64)
    assert app(ctypes.addressof(shared), E, E, F, 4, None) == ALIAS  # k and v arrays overlap
    assert read(p, F, 4, E, E + 64, None) == ALIAS                   # outputs overlap
    assert read(p, F, 4, B + 64, None, None) == ALIAS and read(p, F, 4, F, None, None) == ALIAS


def test_attention(lib):
    c = cache()
    p = ctypes.addressof(c)
    ws = lib.nf4_attention_workspace_bytes(p, 3, 4)
    assert ws > 0 and lib.nf4_attention_workspace_bytes(p, 3, 3) == -1
    assert lib.nf4_attention_workspace_bytes(None, 3, 4) == -1

    def call(q=E, table=F, max_pages=4, lengths=F + 4096, b=3, heads=4, window=0, out=E + 65536, work=F + (1 << 30),
             size=ws):
        return lib.nf4_attention_decode(p, q, table, max_pages, lengths, b, heads, 1.0, window, out, work, size, None)

    assert call(b=0) == OK
    assert call(b=-1) == SHAPE and call(b=65536) == SHAPE and call(heads=3) == SHAPE and call(heads=0) == SHAPE
    assert call(window=-1) == SHAPE and call(max_pages=-1) == SHAPE and call(max_pages=1 << 28) == SHAPE
    assert call(size=ws - 1) == SHAPE
    assert call(q=None) == NULL and call(table=None) == NULL and call(lengths=None) == NULL and call(work=None) == NULL
    assert call(q=E + 2) == ALIGN and call(lengths=F + 4098) == ALIGN and call(work=F + (1 << 30) + 8) == ALIGN
    assert call(out=E) == ALIAS and call(out=A) == ALIAS and call(work=C) == ALIAS and call(work=E + 65536) == ALIAS


def test_rope(lib):
    def call(q=A, hq=4, k=B, hk=2, t=3, d=128, pos=C, axes=2, sections=(40, 24), freq=D, rotary=128, qo=E, ko=F):
        s = None if sections is None else (ctypes.c_int32 * max(1, len(sections)))(*sections)
        return lib.nf4_rope(q, hq, k, hk, t, d, pos, axes, s, freq, rotary, 0, 1.0, qo, ko, None)

    assert call(t=0) == OK and call(hq=0, hk=0) == OK
    assert call(t=-1) == SHAPE and call(d=120) == SHAPE and call(d=0) == SHAPE and call(rotary=136) == SHAPE
    assert call(rotary=8, sections=(2, 2)) == SHAPE and call(d=512, rotary=512, sections=(128, 128)) == SHAPE
    assert call(axes=0, sections=()) == SHAPE and call(axes=5, sections=(16, 16, 16, 8, 8)) == SHAPE
    assert call(sections=(40, 23)) == SHAPE and call(sections=(65, -1)) == SHAPE
    assert call(hq=65535, d=1024) == SHAPE
    assert call(sections=None) == NULL and call(pos=None) == NULL and call(freq=None) == NULL and call(ko=None) == NULL
    assert call(q=A + 2) == ALIGN and call(qo=E + 8) == ALIGN
    assert call(qo=A + 16) == ALIAS and call(qo=B) == ALIAS and call(ko=E) == ALIAS and call(ko=C) == ALIAS


def test_rmsnorm(lib):
    def call(x=A, r=B, w=C, t=3, h=256, ro=D, y=E, y8=F, s=F + 65536):
        return lib.nf4_rmsnorm(x, r, w, t, h, 1e-6, ro, y, y8, s, None)

    assert call(t=0) == OK
    assert call(t=-1) == SHAPE and call(h=0) == SHAPE and call(h=252) == SHAPE
    assert call(x=None) == NULL and call(w=None) == NULL and call(y=None, y8=None, s=None) == NULL
    assert call(s=None) == NULL and call(y8=None) == NULL
    assert call(x=A + 2) == ALIGN and call(y8=F + 8) == ALIGN
    assert call(ro=B + 16) == ALIAS and call(y=B) == ALIAS and call(y=D) == ALIAS and call(y8=A) == ALIAS
    assert call(y=C) == ALIAS and call(s=F + 16) == ALIAS


def test_valid_calls_without_gpu_fail_cleanly(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    c = cache()
    p = ctypes.addressof(c)
    assert lib.nf4_kv_append(p, E, E + 65536, F, 4, None) in (5, 6)
    assert lib.nf4_kv_read(p, F, 4, E, E + 65536, None) in (5, 6)
    assert lib.nf4_rmsnorm(A, None, C, 3, 256, 1e-6, None, E, None, None, None) in (5, 6)


def test_binding_refuses_wrong_tensors():
    import nf4_weight_only_gb300 as nf4
    bf = torch.zeros(2, 2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        nf4.KVCache("bf16", bf, bf)
    with pytest.raises(ValueError, match="format"):
        nf4.KVCache("int3", bf, bf)
    with pytest.raises(ValueError, match="k: want"):
        nf4.KVCache("fp8", bf, bf)
    with pytest.raises(ValueError, match="k: want"):
        nf4.KVCache("bf16", bf[0], bf[0])
    with pytest.raises(ValueError, match="both None"):
        nf4.nf4_rope(None, None, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(64), None, None)
    with pytest.raises(ValueError, match="contiguous"):
        nf4.nf4_rmsnorm(bf.view(64, 128).t(), torch.zeros(64, dtype=torch.bfloat16), 1e-6, y=bf)
