"""Calls on a stream that is not the current one: their results' memory is that stream's (GPU)."""
import pytest
import torch

import nf4_weight_only_gb300 as nf4
from gpu_util import DEV
from test_layer_ops_gpu import new_cache, paged, randn

pytestmark = pytest.mark.gpu


def operators():
    """name -> (call, shape of its first result): the call takes a stream."""
    c = new_cache("bf16", 8, 2, 64, 64, seed=3)
    slots = torch.arange(512, device=DEV)
    q = randn((4, 8, 64), 4)
    table, lengths = paged([100] * 4, 64, 8, 2, 5).to(DEV), torch.full((4,), 100, dtype=torch.int32, device=DEV)
    ws = nf4.attention_workspace(c, 4, 8)
    positions = torch.arange(512, dtype=torch.int32, device=DEV).view(1, 512)
    freq = torch.rand(32, device=DEV)
    x, k, w = randn((512, 4, 64), 6), randn((512, 2, 64), 7), randn((64,), 8)
    return {
        "read": (lambda s: nf4.kv_read(c, slots, stream=s)[0], (512, 2, 64)),
        "attention": (lambda s: nf4.attention_decode(c, q, table, lengths, ws, stream=s), (4, 8, 64)),
        "rope": (lambda s: nf4.rope(x, k, positions, freq, stream=s)[0], (512, 4, 64)),
        "norm": (lambda s: nf4.rmsnorm(x.view(-1, 64), w, 1e-6, stream=s), (2048, 64)),
    }


@pytest.mark.parametrize("name", ["read", "attention", "rope", "norm"])
@pytest.mark.parametrize("raw", [False, True])
def test_results_belong_to_their_stream(name, raw):
    call, shape = operators()[name]
    want = call(None).clone()
    assert want.shape == shape
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # memory that the current stream will still write to, and that torch may hand out again on it
    old = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    torch.cuda._sleep(50_000_000)
    old.fill_(7)
    del old
    got = call(side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_workspace_is_zeroed_on_its_stream():
    c = new_cache("nf4", 8, 2, 64, 64, seed=3)
    side = torch.cuda.Stream()
    size = nf4.nf4_attention_workspace_bytes(c, 4, 8)
    torch.cuda.synchronize()
    old = torch.empty(size, dtype=torch.uint8, device=DEV)
    torch.cuda._sleep(50_000_000)
    old.fill_(1)
    del old
    ws = nf4.attention_workspace(c, 4, 8, stream=side)
    torch.cuda.synchronize()
    assert ws.numel() == size and not ws.any()
