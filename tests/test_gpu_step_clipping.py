"""MuonStep with clipping: whose gradients the norm is of (needs a gfx950 GPU)."""
import gc
import weakref

import pytest
import torch

from newton_schulz_amd import MuonStep

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32 = torch.float32


def make(shapes, **kw):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return MuonStep(shapes, DEV, max_grad_norm=1.0, grad_dtype=F32, **kw)


def close(step):
    for c in step.contexts:
        c.close()


def size(*tensors):
    return sum(t.double().square().sum() for t in tensors).sqrt().item()


def test_norm_of_a_gradient_buffer_put_in_place_of_the_first():
    """A step reads the buffer that `grad` is at the time, its norm too."""
    a, b = make([(128, 256, 0)]), make([(128, 256, 0)])
    g = torch.randn(128 * 256, device=DEV)
    b.grad.copy_(g)
    a.grad = g
    for s in (a, b):
        s.step()
    torch.cuda.synchronize()
    # 2^15 squares, each sum within a few 2^-53 a term
    assert a.grad_norm[1].item() == pytest.approx(size(g), rel=2 ** 16 * 2.0 ** -53)
    assert torch.equal(a.grad_norm, b.grad_norm) and torch.equal(a.momentum, b.momentum)
    close(a)
    close(b)


@pytest.mark.parametrize("sizes", [[5] * 9000, [(1 << 26) + 5] * 3], ids=["many", "large"])
def test_norm_over_far_more_than_the_step_itself(sizes):
    """Other gradients whose partial sums the step's own workspace has no room
    for, eager and recorded."""
    a = make([(64, 64, 0)], keep_bf16_weights=False)
    g = torch.Generator(device=DEV).manual_seed(1)
    others = [torch.empty(n, device=DEV).normal_(generator=g) for n in sizes]
    assert a.ctx.tensor_list(others).norm_workspace_bytes() > a.ctx.workspace_bytes
    before = [t.clone() for t in others]
    a.grad.normal_(generator=g)
    want = size(a.grad, *others)
    total = a.numel + sum(sizes)

    def check():
        torch.cuda.synchronize()
        assert a.grad_norm[1].item() == pytest.approx(want, rel=total * 2.0 ** -53)
        coef = a.grad_norm[2].float()
        assert 0 < coef < 1
        for t, b in zip(others, before):
            assert torch.equal(t, b * coef)
            t.copy_(b)

    a.capture(other_grads=others)  # before any eager step
    for _ in range(3):
        a.replay()
        check()
        a.step(other_grads=others)
        check()
    a.step(other_grads=a.ctx.tensor_list(others))
    check()
    assert len(a.contexts) == 2
    close(a)


# the rejected call records nothing, so torch reports an empty graph
@pytest.mark.filterwarnings("ignore:The CUDA Graph is empty")
def test_an_allocation_is_refused_while_a_graph_is_recorded():
    a = make([(64, 64, 0)])
    others = [torch.ones(3, device=DEV) for _ in range(9000)]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with pytest.raises(RuntimeError, match="once before"):
        with torch.cuda.graph(graph, stream=side):
            a.step(stream=side, other_grads=others)
    torch.cuda.synchronize()
    a.step(other_grads=others)
    torch.cuda.synchronize()
    # 27000 ones and a gradient of zeros
    assert a.grad_norm[0].item() == 27000
    close(a)


def test_a_recorded_step_keeps_the_gradients_it_scales():
    """Replays write to the other gradients' memory: it stays theirs although the
    caller lets go of them, and of the step's own gradient buffer."""
    a = make([(64, 64, 0)])
    others = [torch.ones(1 << 20, device=DEV), torch.ones(77, device=DEV)]
    a.capture(other_grads=others)
    at = [t.data_ptr() for t in (a.grad, *others)]
    kept = [weakref.ref(t) for t in (a.grad, *others)]
    del others
    a.grad = torch.zeros_like(a.grad)
    gc.collect()
    assert [t().data_ptr() for t in kept] == at
    fresh = [torch.full((1 << 20,), 3.0, device=DEV) for _ in range(4)]
    for _ in range(3):
        a.replay()
        torch.cuda.synchronize()
        assert all((t == 3).all() for t in fresh)
    close(a)
