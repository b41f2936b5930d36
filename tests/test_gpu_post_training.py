"""The operators together: the example's training steps, the gradient of a
small model through the losses against torch's own, and MuonStep with
clipping (needs a gfx950 GPU)."""
import os
import sys

import numpy as np
import pytest
import torch

import oracle
from newton_schulz_amd import Context, MuonStep, synth
from newton_schulz_amd.offload import MuonOffloadStep
from oracle import loss_oracle as lo

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("loss", ["policy", "preference"])
def test_example_lowers_the_loss(loss):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import post_training_step
    history = post_training_step.train(loss, steps=6, say=lambda *a: print(*a, file=sys.stderr, flush=True))
    assert np.isfinite(history).all() and history[-1] < history[0] - 0.01


def test_weight_gradients_follow_the_formula():
    """fp32 logits x W^T: the weights' gradient from policy_loss's gradient
    equals the one computed in binary64 from the oracle's."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator().manual_seed(4)
    x, w = torch.randn(2, 9, 32, generator=g), torch.randn(517, 32, generator=g) * 0.3
    y = torch.randint(517, (2, 9), generator=g)
    y[0, :4] = -1
    adv, old = torch.randn(2, generator=g), -6 + torch.randn(2, 9, generator=g)
    wd = w.to(DEV).requires_grad_()
    logits = x.to(DEV) @ wd.t()
    ctx, out, grad = Context(DEV, 1 << 20), torch.empty(4, device=DEV), torch.empty(2, 9, 517, device=DEV)
    ctx.policy_loss(logits.detach(), y.to(DEV), adv.to(DEV), out, old_logps=old.to(DEV), grad_logits=grad)
    logits.backward(grad)
    z = logits.detach().double().cpu().numpy()
    lp = lo.token_logps_ref(z, y.numpy())
    _, gl = lo.policy_ref(lp, y.numpy(), adv.double().numpy(), old.double().numpy(), None, float(np.float32(0.2)),
                          float(np.float32(0.2)))
    gz = lo.logits_grad_ref(z, y.numpy(), gl)
    want = np.einsum("btv,bth->vh", gz, x.double().numpy())
    # 18 products summed in fp32 and the logits' gradient good to a few 2^-21
    assert oracle.rel_fro(wd.grad.cpu().numpy(), want) < 18 * 2.0 ** -23 + 2.0 ** -20
    ctx.close()


SHAPES = [(256, 512, 0), (512, 256, 0), (130, 202, 0), (128, 640, 64)]


@pytest.mark.parametrize("inflight", [1, 2])
def test_muon_step_with_clipping(inflight):
    """A step with max_grad_norm equals a step on the gradient multiplied
    beforehand by the coefficient, for gradients that the product keeps exact
    (fp32 gradients, a coefficient of a power of two), bit for bit."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    kw = dict(cap_bytes=1 << 20, inflight=inflight, grad_dtype=torch.float32)
    a = MuonStep(SHAPES, DEV, max_grad_norm=1.0, **kw)
    b = MuonStep(SHAPES, DEV, **kw)
    g = torch.Generator(device=DEV).manual_seed(5)
    w0 = synth.normal((a.numel,), 2e-2, g, DEV, torch.float32)
    gr = synth.normal((a.numel,), 1.0, g, DEV, torch.float32)
    other = [torch.randn(1000, device=DEV), torch.randn(77, device=DEV).bfloat16()]
    # a limit that makes the coefficient 1/4 (but for eps, far below a rounding)
    size = (gr.double().square().sum() + sum(t.double().square().sum() for t in other)).sqrt().item()
    a.max_grad_norm = 0.25 * size + 0.25e-6
    for s in (a, b):
        s.master.copy_(w0)
    a.grad.copy_(gr)
    b.grad.copy_(gr * 0.25)
    before = [t.clone() for t in other]
    a.step(other_grads=other)
    b.step()
    torch.cuda.synchronize()
    assert a.grad_norm[1].item() == pytest.approx(size, rel=1e-12) and np.float32(a.grad_norm[2].item()) == 0.25
    assert torch.equal(a.momentum, b.momentum) and torch.equal(a.master, b.master)
    assert torch.equal(a.grad, gr)
    for t, u in zip(other, before):
        assert torch.equal(t, (u.float() * 0.25).to(t.dtype))
    # recorded, and without other gradients: the eager step's bits
    a.max_grad_norm = 1.0
    state = {n: getattr(a, n).clone() for n in ("momentum", "master")}
    a.step()
    torch.cuda.synchronize()
    eager = {n: getattr(a, n).clone() for n in state}
    a.capture()
    for _ in range(3):
        for n, v in state.items():
            getattr(a, n).copy_(v)
        torch.randn(1 << 16, device=DEV).sum()
        a.replay()
        torch.cuda.synchronize()
        for n, v in eager.items():
            assert torch.equal(getattr(a, n), v), n
    assert a.grad_norm[2] < 1
    with pytest.raises(ValueError):
        b.step(other_grads=other)
    for s in (a, b):
        for c in s.contexts:
            c.close()


def test_offloaded_step_refuses_clipping():
    with pytest.raises(ValueError):
        MuonOffloadStep([(64, 64, 0)], DEV, max_grad_norm=1.0)
