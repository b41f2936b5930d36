"""The operators around the layers one after the other, as a round of sampling
and training uses them: scores out of 8-bit weights, a draft verified against
them, the loss on what came out, the gradients out of the kept 8-bit
activations into the step's buffer, the step, and its new 8-bit weights.

Every stage is compared with the formula in 64 bits on what the stage before
left on the device."""
import numpy as np
import pytest
import torch

from newton_schulz_amd import Context, MuonStep
from oracle import linear8_oracle as lo

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("grad_dtype", [BF, F32])
@pytest.mark.parametrize("batch,draft,vocab,hidden,t", [(5, 3, 384, 128, 1.0), (3, 4, 2500, 72, 0.8), (12, 1, 131, 200, 1.2)])
def test_round(grad_dtype, batch, draft, vocab, hidden, t):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ctx = Context(DEV, 64 << 20)
    gen = torch.Generator().manual_seed(vocab)
    step = MuonStep([(vocab, hidden, 0)], DEV, lr=0.02, grad_dtype=grad_dtype, keep_int8_weights=True)
    step.view(step.master, 0).copy_(torch.randn(vocab, hidden, generator=gen) * 2 * hidden ** -0.5)
    step.quantize_weights()
    rows = batch * (draft + 1)
    x = torch.randn(batch, draft + 1, hidden, generator=gen).to(BF).to(DEV)
    x8, gx = ctx.rows8(rows, hidden), torch.empty(batch, draft + 1, hidden, dtype=BF, device=DEV)
    logits = torch.empty(batch, draft + 1, vocab, dtype=BF, device=DEV)
    ctx.linear8(x, step.weight8(0), logits, x8=x8)
    w = lo.values_ref(step.weight8(0).q.cpu().numpy(), step.weight8(0).scale.cpu().numpy())
    xs = lo.values_ref(x8.q.cpu().numpy(), x8.scale.cpu().numpy())
    want = xs @ w.T
    # (three roundings of the scales' product and the sum, then to bf16)
    off = np.abs(logits.double().cpu().numpy().reshape(rows, vocab) - want)
    assert (off <= (2.0 ** -8 + 2.0 ** -21) * np.abs(want)).all()

    # a draft from scores of its own, one sequence's shorter
    d = (logits[:, :draft].float() + 0.5 * torch.randn(batch, draft, vocab, generator=gen).to(DEV)).to(BF)
    noise = torch.rand(batch, draft, vocab, generator=gen).clamp(min=1e-30).to(DEV)
    y = (d.float() / t - torch.log(-torch.log(noise))).argmax(-1)
    y[0, draft - 1:] = -1
    u = torch.rand(batch, draft + 1, generator=gen).to(DEV)
    tokens = torch.empty(batch, draft + 1, dtype=torch.int64, device=DEV)
    accepted = torch.empty(batch, dtype=torch.int64, device=DEV)
    old = torch.empty(batch, draft + 1, device=DEV)
    ctx.verify_draft(logits, y, tokens, accepted, draft_logits=d, uniforms=u, logps=old, temperature=t)
    ref = lo.verify_ref(*[v.double().cpu().numpy() if v.is_floating_point() else v.cpu().numpy() for v in (logits, y, d, u)], t)
    assert np.array_equal(tokens.cpu().numpy(), ref[0]) and np.array_equal(accepted.cpu().numpy(), ref[1])
    assert (np.abs(old.double().cpu().numpy() - ref[2]) <= 2.0 ** -22 + 2.0 ** -21 * np.abs(ref[2])).all()

    # the loss on the tokens that came out (-1 behind them: left out), its own policy's
    a = torch.randn(batch, generator=gen).to(DEV)
    out, g = torch.empty(4, device=DEV), torch.empty_like(logits)
    ctx.policy_loss(logits, tokens, a, out, old_logps=old, grad_logits=g, temperature=t)
    counted = (tokens >= 0).double().cpu()
    n = counted.sum().item()
    ad = a.double().cpu()
    # ratios are 1 up to both log-probabilities' roundings
    assert abs(out[1].item() + (ad[:, None] * counted).sum().item() / n) <= 2.0 ** -17 * ad.abs().max().item()
    assert out[3].item() == 0.0
    p = torch.softmax(logits.double().cpu() / t, -1)
    hot = torch.nn.functional.one_hot(tokens.cpu().clamp(min=0), vocab).double()
    scale = (ad[:, None] * counted / (n * t))[..., None]
    gd = g.double().cpu()
    assert ((gd + scale * (hot - p)).abs() <= 2.0 ** -8 * gd.abs() + scale.abs() * (2.0 ** -17 * (hot + p)) + 2.0 ** -126).all()

    # gradients out of the 8-bit rows, into the step's buffer
    ctx.input_grad8(g, step.weight8(0), gx)
    gw = step.view(step.grad, 0)
    ctx.weight_grad8(g.view(rows, vocab), x8, gw)
    gm = gd.numpy().reshape(rows, vocab)
    for got, m, v, dtype in ((gx.view(rows, hidden), gm, w, BF), (gw, gm.T, xs, grad_dtype)):
        want, size, half = m @ v, np.abs(m) @ np.abs(v), torch.finfo(dtype).eps / 2
        tol = size * ((2.0 ** -8 if dtype == BF else 0.0) + 2.0 ** -24 + (m.shape[1] + 8) * 2.0 ** -23)
        tol = tol * (1 + half) + (half + 2.0 ** -24) * np.abs(want) + 2.0 ** -130
        assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()

    # the step moves the weights, and their 8-bit rows with them
    before = step.view(step.master, 0).clone()
    step.step()
    again = ctx.rows8(vocab, hidden)
    ctx.quantize_rows(step.view(step.master, 0), again)
    assert not torch.equal(before, step.view(step.master, 0))
    assert torch.equal(again.q, step.weight8(0).q) and torch.equal(again.scale, step.weight8(0).scale)
    ctx.close()
