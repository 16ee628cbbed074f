"""The build where only the library can be built, and the binding without its compiled calls (no GPU)."""
import os
import sysconfig

import pytest
import torch

import nf4_weight_only_gb300 as nf4
from nf4_weight_only_gb300 import build


@pytest.fixture
def no_headers(tmp_path, monkeypatch):
    """Build outputs in a folder of their own, no Python.h, and an nvcc that only leaves its output."""
    include = tmp_path / "include"
    include.mkdir()
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: {"include": str(include)})
    out = tmp_path / "_build"
    monkeypatch.setattr(build, "BUILD_DIR", str(out))
    monkeypatch.setattr(build, "LIB_PATH", str(out / "libnf4.so"))
    monkeypatch.setattr(build, "CALLS_PATH", str(out / os.path.basename(build.CALLS_PATH)))
    nvcc = tmp_path / "nvcc"
    nvcc.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\necho built > "$2"\n')
    nvcc.chmod(0o755)
    monkeypatch.setattr(build, "_nvcc", lambda: str(nvcc))
    return out


def test_the_library_builds_without_pythons_headers(no_headers):
    assert build.build() == build.LIB_PATH
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.CALLS_PATH)
    assert not build.is_stale()


def test_the_compiled_calls_are_named_after_their_interpreter():
    assert build.CALLS_PATH.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    build.build()
    assert os.path.exists(build.CALLS_PATH)


def test_the_binding_works_without_them(monkeypatch):
    build.build()
    monkeypatch.setattr(nf4, "_calls", None)
    monkeypatch.setattr(build, "CALLS_PATH", build.CALLS_PATH + ".gone")
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.warns(RuntimeWarning, match="ctypes"):
        with pytest.raises(ValueError, match="CUDA"):  # the wrapper's own checks
            nf4.nf4_rmsnorm(x, w, 1e-6, y=x)
    with pytest.raises(ValueError, match="both None"):
        nf4.nf4_rope(None, None, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(64), None, None)


@pytest.mark.gpu
def test_results_are_the_same_without_them(monkeypatch):
    from test_layer_ops_gpu import new_cache, randn
    dev = "cuda:0"
    c = new_cache("nf4", 8, 2, 16, 64, seed=1)
    q, k, w = randn((3, 4, 64), 2), randn((3, 2, 64), 3), randn((64,), 4)
    table = torch.arange(8, dtype=torch.int32, device=dev).view(1, 8).repeat(3, 1)
    lengths = torch.tensor([100, 3, 0], dtype=torch.int32, device=dev)
    positions, freq = torch.arange(3, dtype=torch.int32, device=dev)[None], torch.rand(32, device=dev)
    slots = torch.tensor([5, -1, 100], device=dev)

    def everything():
        ws = nf4.attention_workspace(c, 3, 4)
        out = [nf4.attention_decode(c, q, table, lengths, ws, window=50), *nf4.rope(q, k, positions, freq),
               *nf4.rmsnorm(q.view(-1, 64), w, 1e-6, residual=q.view(-1, 64))]
        nf4.nf4_kv_append(c, k, k, slots)
        return out + list(nf4.kv_read(c, slots))

    want = everything()
    monkeypatch.setattr(nf4, "_calls", nf4._NoCalls)
    for a, b in zip(everything(), want):
        assert torch.equal(a, b)
