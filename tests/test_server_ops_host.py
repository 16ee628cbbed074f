"""Host-side checks of the calls that plan a step, apply adapters and sample (no GPU): argument errors come back before
any device work, and the binding refuses tensors of the wrong type, shape or device."""
import ctypes
import os
import sys

import pytest
import torch

A, B, C, D, E, F, G, H, I, J, K = (0x7F0000000000 + (i << 36) for i in range(11))  # fake device addresses, never read
vp = ctypes.c_void_p
OK, NULL, SHAPE, ALIGN, ALIAS = 0, 1, 2, 3, 4
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from nf4_weight_only_gb300 import build
    import nf4_weight_only_gb300 as nf4
    return nf4.load(build.build())


PLAN = dict(lengths=A, new_tokens=B, batch=4, page_size=16, pages=64, table=C, max_pages=8, ring=D, free_in=E, free_out=F,
            lengths_out=G, starts=H, t=32, slots=I, positions=J, sequences=K)


def plan(lib, **change):
    return lib.nf4_plan_step(*{**PLAN, **change}.values(), None)


@pytest.mark.parametrize("change,want", [
    (dict(batch=-1), SHAPE), (dict(batch=8193), SHAPE), (dict(t=-1), SHAPE), (dict(t=1 << 31), SHAPE),
    (dict(pages=-1), SHAPE), (dict(pages=1 << 31), SHAPE), (dict(pages=(1 << 31) - 1), SHAPE), (dict(page_size=8), SHAPE), (dict(page_size=24), SHAPE),
    (dict(page_size=131072), SHAPE), (dict(page_size=0), SHAPE), (dict(max_pages=-1), SHAPE),
    (dict(batch=8192, max_pages=(1 << 31) - 1), SHAPE),
    (dict(lengths=0), NULL), (dict(new_tokens=0), NULL), (dict(table=0), NULL), (dict(ring=0), NULL),
    (dict(free_in=0), NULL), (dict(free_out=0), NULL), (dict(lengths_out=0), NULL), (dict(starts=0), NULL),
    (dict(slots=0), NULL), (dict(positions=0), NULL), (dict(sequences=0), NULL),
    (dict(lengths=A + 2), ALIGN), (dict(free_in=E + 4), ALIGN), (dict(free_out=F + 4), ALIGN),
    (dict(slots=I + 4), ALIGN), (dict(positions=J + 1), ALIGN), (dict(table=C + 2), ALIGN),
    (dict(starts=A), ALIAS), (dict(lengths_out=A + 4), ALIAS), (dict(lengths_out=B), ALIAS), (dict(free_out=E + 8), ALIAS),
    (dict(table=D), ALIAS), (dict(slots=C), ALIAS), (dict(positions=I + 128), ALIAS), (dict(sequences=J + 124), ALIAS),
    (dict(free_out=A), ALIAS), (dict(table=B), ALIAS),
])
def test_plan_step_refusals(lib, change, want):
    assert plan(lib, **change) == want


@pytest.mark.parametrize("t,adapters,want", [(-1, 1, -1), (1 << 24, 8192, 0), ((1 << 24) + 1, 1, -1), (1, -1, -1),
                                             (1, 8193, -1), (0, 0, 0)])
def test_lora_plan_sizes(lib, t, adapters, want):
    n = lib.nf4_lora_plan_bytes(t, adapters)
    assert (n == -1) if want < 0 else n > 0
    if want < 0:
        assert lib.nf4_lora_plan(vp(A), None, 0, t, adapters, vp(B), 1 << 40, None) == SHAPE


def test_lora_plan_refusals(lib):
    need = lib.nf4_lora_plan_bytes(100, 8)
    assert lib.nf4_lora_plan(vp(A), None, 0, 100, 8, vp(B), need - 1, None) == SHAPE
    assert lib.nf4_lora_plan(vp(A), vp(C), -1, 100, 8, vp(B), need, None) == SHAPE
    assert lib.nf4_lora_plan(None, None, 0, 100, 8, vp(B), need, None) == NULL
    assert lib.nf4_lora_plan(None, vp(C), 3, 100, 8, vp(B), need, None) == NULL
    assert lib.nf4_lora_plan(vp(A), None, 0, 100, 8, None, need, None) == NULL
    assert lib.nf4_lora_plan(vp(A), None, 0, 100, 8, vp(B + 8), need, None) == ALIGN
    assert lib.nf4_lora_plan(vp(A + 2), None, 0, 100, 8, vp(B), need, None) == ALIGN
    assert lib.nf4_lora_plan(vp(B + 16), None, 0, 100, 8, vp(B), need, None) == ALIAS
    assert lib.nf4_lora_plan(vp(A), vp(B + need - 4), 5, 100, 8, vp(B), need, None) == ALIAS


def lora(lib, x=A, t=4, k=128, plan=B, plan_bytes=None, adapters=3, rank=16, scales=C, a=(D, D + 65536), b=(E, E + 65536),
         bases=None, ys=(F, F + 65536), ns=(64, 24), workspace=G, room=None, count=None):
    arr = vp * len(ns)
    pick = lambda v: None if v is None else ctypes.cast(arr(*v), vp)  # noqa: E731
    if plan_bytes is None:
        plan_bytes = lib.nf4_lora_plan_bytes(t, adapters)
    if room is None:
        room = lib.nf4_lora_workspace_bytes(t, adapters, rank, len(ns))
    return lib.nf4_lora(x, t, k, plan, plan_bytes, adapters, rank, scales, len(ns) if count is None else count, pick(a),
                        pick(b), pick(bases), pick(ys), ctypes.cast((ctypes.c_int64 * len(ns))(*ns), vp), workspace, room,
                        None)


@pytest.mark.parametrize("change,want", [
    (dict(k=100), SHAPE), (dict(k=0), SHAPE), (dict(rank=0), SHAPE), (dict(rank=12), SHAPE), (dict(rank=136), SHAPE),
    (dict(adapters=8193), SHAPE), (dict(t=-1), SHAPE), (dict(count=0), SHAPE), (dict(count=9), SHAPE),
    (dict(ns=(-1, 24)), SHAPE), (dict(ns=((1 << 31) - 1, 24)), SHAPE), (dict(plan_bytes=8), SHAPE), (dict(room=8), SHAPE),
    (dict(x=0), NULL), (dict(plan=0), NULL), (dict(scales=0), NULL), (dict(workspace=0), NULL), (dict(a=None), NULL),
    (dict(b=None), NULL), (dict(ys=None), NULL), (dict(a=(D, 0)), NULL), (dict(b=(0, E)), NULL), (dict(ys=(F, 0)), NULL),
    (dict(bases=(H, 0)), NULL),
    (dict(x=A + 8), ALIGN), (dict(plan=B + 4), ALIGN), (dict(scales=C + 2), ALIGN), (dict(a=(D + 8, D + 65536)), ALIGN),
    (dict(ys=(F, F + 65528)), ALIGN), (dict(bases=(H + 2, H + 65536)), ALIGN), (dict(workspace=G + 8), ALIGN),
    (dict(ys=(A, F)), ALIAS), (dict(ys=(F, F + 16)), ALIAS), (dict(ys=(D + 16, F)), ALIAS), (dict(ys=(F, E + 32)), ALIAS),
    (dict(bases=(F + 65536, H)), ALIAS), (dict(bases=(F + 16, H)), ALIAS), (dict(workspace=A), ALIAS),
    (dict(workspace=D), ALIAS), (dict(workspace=E), ALIAS), (dict(ys=(G, F)), ALIAS), (dict(ys=(B, F)), ALIAS),
    (dict(bases=(G, H)), ALIAS), (dict(t=0), OK), (dict(ns=(0, 0)), OK),
])
def test_lora_refusals(lib, change, want):
    assert lora(lib, **change) == want


def test_lora_workspace_sizes(lib):
    assert lib.nf4_lora_workspace_bytes(1, 1, 16, 3) > 0
    for bad in ((-1, 1, 16, 1), (1, 9000, 16, 1), (1, 1, 4, 1), (1, 1, 20, 1), (1, 1, 256, 1), (1, 1, 16, 0), (1, 1, 16, 9)):
        assert lib.nf4_lora_workspace_bytes(*bad) == -1


SAMPLE = dict(logits=A, bf16=1, batch=4, vocab=100, stride=128, temperature=B, top_k=C, top_p=D, min_p=E, random=F,
              tokens=G, logprobs=H)


@pytest.mark.parametrize("change,want", [
    (dict(batch=-1), SHAPE), (dict(batch=(1 << 24) + 1), SHAPE), (dict(vocab=0), SHAPE),
    (dict(vocab=262145, stride=300000), SHAPE), (dict(stride=99), SHAPE), (dict(stride=1 << 31), SHAPE),
    (dict(logits=0), NULL), (dict(random=0), NULL), (dict(tokens=0), NULL),
    (dict(logits=A + 1), ALIGN), (dict(logits=A + 2, bf16=0), ALIGN), (dict(random=F + 2), ALIGN), (dict(tokens=G + 1), ALIGN), (dict(logprobs=H + 2), ALIGN),
    (dict(tokens=A + 16), ALIAS), (dict(tokens=C), ALIAS), (dict(logprobs=G + 12), ALIAS), (dict(logprobs=F), ALIAS),
    (dict(logprobs=A + 3 * 256 + 196), ALIAS), (dict(batch=0, logits=0), OK),
])
def test_sample_refusals(lib, change, want):
    assert lib.nf4_sample(*{**SAMPLE, **change}.values(), None) == want


def test_valid_calls_without_gpu_fail_cleanly(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert plan(lib) in (5, 6)
    assert plan(lib, lengths_out=A, free_out=E) in (5, 6)  # in place
    assert plan(lib, batch=0, t=0) in (5, 6)
    assert lora(lib) in (5, 6)
    assert lora(lib, bases=(F, H)) in (5, 6)
    assert lora(lib, adapters=0, a=(0, 0), b=(0, 0), scales=0) in (5, 6)
    assert lib.nf4_sample(*SAMPLE.values(), None) in (5, 6)
    assert lib.nf4_sample(*{**SAMPLE, **dict(temperature=0, top_k=0, top_p=0, min_p=0, logprobs=0)}.values(), None) in (5, 6)


@pytest.mark.parametrize("compiled", [True, False])
def test_binding_refuses_wrong_tensors(lib, compiled, monkeypatch):
    """Both ways into the library refuse before any call."""
    import nf4_weight_only_gb300 as nf4
    if not compiled:
        monkeypatch.setattr(nf4, "_calls", nf4._NoCalls)
    i32, i64, bf = torch.int32, torch.int64, torch.bfloat16
    z = torch.zeros
    good = [z(2, dtype=i32), z(2, dtype=i32), 16, z((2, 3), dtype=i32), z(9, dtype=i32), z(2, dtype=i64), z(2, dtype=i64),
            z(2, dtype=i32), z(3, dtype=i32), z(5, dtype=i64), z(5, dtype=i32), z(5, dtype=i32)]
    with pytest.raises(ValueError, match="CUDA tensor"):
        nf4.nf4_plan_step(*good)
    for at, bad in ((0, z(2, dtype=i64)), (1, z(3, dtype=i32)), (3, z((3, 3), dtype=i32)), (5, z(2, dtype=i32)),
                    (8, z(2, dtype=i32)), (9, z(5, dtype=i32)), (11, z(4, dtype=i32)), (4, None)):
        args = list(good)
        args[at] = bad
        with pytest.raises((ValueError, AttributeError)):
            nf4.nf4_plan_step(*args)
    with pytest.raises(ValueError):
        nf4.nf4_lora_plan(z(4, dtype=i64), 2, z(100, dtype=torch.uint8))
    with pytest.raises(ValueError, match="same length"):
        nf4.nf4_lora(z((2, 64), dtype=bf), z(9, dtype=torch.uint8), z(3), [z((3, 8, 64), dtype=bf)], [], [],
                     z(9, dtype=torch.uint8))
    with pytest.raises(ValueError):
        nf4.nf4_lora(z((2, 64), dtype=bf), z(9, dtype=torch.uint8), z(3), [z((3, 8, 32), dtype=bf)],
                     [z((3, 16, 8), dtype=bf)], [z((2, 16), dtype=bf)], z(9, dtype=torch.uint8))
    with pytest.raises(ValueError, match="1 to 8"):
        nf4.nf4_lora(z((2, 64), dtype=bf), z(9, dtype=torch.uint8), z(3), [], [], [], z(9, dtype=torch.uint8))
    with pytest.raises(ValueError, match="logits"):
        nf4.nf4_sample(z((2, 9), dtype=torch.float16), z(2), z(2, dtype=i32))
    with pytest.raises(ValueError, match="CUDA tensor"):
        nf4.nf4_sample(z((2, 9)), z(2), z(2, dtype=i32))
    with pytest.raises(ValueError):
        nf4.nf4_sample(z((2, 9)), z(3), z(2, dtype=i32))


def test_sizes_past_the_limits_are_errors(lib):
    import nf4_weight_only_gb300 as nf4
    with pytest.raises(nf4.NF4Error):
        nf4.nf4_lora_plan_bytes(-1, 4)
    with pytest.raises(nf4.NF4Error):
        nf4.nf4_lora_workspace_bytes(4, 4, 20, 1)


def test_plain_forms_and_definitions_agree_on_the_cpu(monkeypatch):
    """The measured cases' plain forms against their 64-bit definitions, on small cases."""
    import random
    sys.path.insert(0, os.path.join(ROOT, "perf"))
    import more_operators as m
    monkeypatch.setattr(m, "DEV", "cpu")
    rng, seen = random.Random(4), set()
    for n in range(400):
        case = m.draw(rng)
        if m.work(case)["bytes"] > 300000 or case.get("loaded", 0) * case.get("k", 0) > 20000:
            continue
        seen.add(case["op"])
        want, got = m.exact(case, n), m.run(m.prepare(case, n))
        if case["op"] == "plan":
            assert all(torch.equal(got[name], want[name]) for name in want)
        elif case["op"] == "sample":
            assert torch.equal(got[0], want[0])
        else:
            for g, w in zip(got, want):
                assert float((g.double() - w).abs().max()) <= 2.0 ** -8 * float(w.abs().max()) * 1.01
    assert seen == {"plan", "lora", "sample"}
