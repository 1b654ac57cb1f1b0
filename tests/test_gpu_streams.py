"""Outputs allocated by a call on another stream do not take memory that queued work still uses, and
their memory is not given on while the current stream reads them."""
import pytest
import torch

from sparse_attention_lightning_indexer_gb300 import ds4idx

pytestmark = pytest.mark.gpu


def test_memory_of_outputs_on_another_stream():
    n = 20000                                        # 23 MB a tensor: blocks of their own
    x = torch.randn(n, 576, device="cuda").to(torch.bfloat16)
    cache = torch.empty(n, 416, dtype=torch.uint8, device="cuda")
    ds4idx.quantize_latents(x, cache)
    want = ds4idx.read_latents(cache).cpu()
    s = torch.cuda.Stream()
    freed = torch.full((n, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    copy = freed.clone()                             # queued behind the sleep
    del freed
    out = ds4idx.read_latents(cache, stream=s)       # runs at once
    torch.cuda.synchronize()
    assert bool((copy == 3).all())
    torch.cuda._sleep(50_000_000)
    copy.copy_(out)                                  # queued behind the sleep
    del out
    with torch.cuda.stream(s):
        other = torch.zeros(n, 576, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(copy.cpu(), want) and not bool(other.any())
