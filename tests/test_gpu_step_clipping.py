"""MuonStep with clipping: whose gradients the norm is of (needs a gfx950 GPU)."""
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
