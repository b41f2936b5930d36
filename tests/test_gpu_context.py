"""A context just made is ready for any stream (needs a gfx950 GPU)."""
import pytest
import torch

from newton_schulz_amd import Context

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def test_a_new_context_waits_for_nothing_on_the_null_stream():
    """The words that workgroups exchange through are zeros when the context is
    there, also where the null stream is busy at that time: nothing of the
    creation is still queued on it, and a first call on a side stream, which
    does not wait for the null stream, gives what a later one gives."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    x, y = torch.randn(4, 9, 50257, device=DEV), torch.zeros(4, 9, dtype=torch.int64, device=DEV)
    first, later = torch.empty(4, 9, device=DEV), torch.empty(4, 9, device=DEV)
    side = torch.cuda.Stream(DEV)
    big = torch.randn(4096, 4096, device=DEV)
    for _ in range(3):
        torch.cuda.synchronize()
        for _ in range(40):
            big = big @ big * 1e-2
        null = torch.cuda.default_stream(DEV)
        ctx = Context(DEV, 1 << 20)
        assert null.query()
        ctx.token_logps(x, y, first, stream=side)
        side.synchronize()
        ctx.token_logps(x, y, later)
        torch.cuda.synchronize()
        assert torch.equal(first, later)
        ctx.close()
