"""A context just made is ready for any stream (needs a gfx950 GPU)."""
import ctypes

import pytest
import torch

from newton_schulz_amd import Context, _lib

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


class Exchange(ctypes.Structure):
    _fields_ = [("words", ctypes.c_void_p), ("dirty", ctypes.c_bool)]


def test_a_recorded_clearing_counts_only_when_it_runs():
    """After a call that failed half way the next one empties the words.  Where
    that one is being recorded, nothing has been emptied yet: calls before the
    replay still have to."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    clear = getattr(ctypes.CDLL(_lib.LIB_PATH), "_Z14clear_exchangeP12ihipStream_tR8Exchange")
    clear.argtypes = [ctypes.c_void_p, ctypes.POINTER(Exchange)]
    words = torch.ones(40000, dtype=torch.int64, device=DEV)  # (the launch empties the first 33824)
    count = 32768 + 33 * 32
    x = Exchange(words.data_ptr(), True)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.graph(graph, stream=side):
        assert clear(side.cuda_stream, ctypes.byref(x)) == 0
    torch.cuda.current_stream(DEV).wait_stream(side)
    torch.cuda.synchronize()
    assert x.dirty and (words == 1).all()
    assert clear(torch.cuda.current_stream(DEV).cuda_stream, ctypes.byref(x)) == 0
    torch.cuda.synchronize()
    assert not x.dirty and (words[:count] == 0).all() and (words[count:] == 1).all()
    for _ in range(3):
        words.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert (words[:count] == 0).all() and (words[count:] == 1).all()
