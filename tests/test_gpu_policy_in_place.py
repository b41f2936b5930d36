"""The policy loss in place over many more rows than the device works on at once,
with and without waiting: the same bits as out of place (needs a gfx950 GPU).

Workgroups that do not wait overwrite their scores while others of their row
have not started yet."""
import pytest
import torch

from newton_schulz_amd import Context, loss_workspace_bytes

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("seq,vocab,dtype", [
    (2000, 151936, BF),     # 8 slices a row, 16000 workgroups
    (1500, 41001, F32),     # 5 slices, rows at odd addresses
    (17000, 20488, BF),     # 2 slices; more slots than the context keeps: words in the workspace
])
def test_in_place_over_many_generations(seq, vocab, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator(device=DEV).manual_seed(vocab)
    x = torch.empty(1, seq, vocab, dtype=dtype, device=DEV).normal_(0.0, 2.0, generator=g)
    y = torch.randint(vocab, (1, seq), generator=g, device=DEV)
    y[0, ::7] = -1
    y[0, 5], y[0, 11] = 0, vocab - 1
    lp = torch.cat([torch.log_softmax(r.double(), -1).gather(-1, k.clamp(min=0)[:, None])[:, 0]
                    for r, k in zip(x[0].split(256), y[0].split(256))])[None]
    old = (lp + 0.3 * torch.randn(1, seq, generator=g, device=DEV)).float()
    ref = (lp + 0.3 * torch.randn(1, seq, generator=g, device=DEV)).float()
    adv = torch.randn(1, seq, generator=g, device=DEV)
    kw = dict(old_logps=old, ref_logps=ref, kl_coef=0.05, reduce="sum")
    ctx = Context(DEV, loss_workspace_bytes(1, seq, vocab, dtype))

    def call(scores, grad):
        out, logps = torch.empty(4, device=DEV), torch.empty(1, seq, device=DEV)
        ctx.policy_loss(scores, y, adv, out, logps=logps, grad_logits=grad, **kw)
        return out, logps

    grad = torch.empty_like(x)
    out, logps = call(x, grad)
    # far above the error of lp, far below what a gradient in a score's place makes
    assert (logps.double() - lp).masked_fill(y < 0, 0.0).abs().max() < 1e-4
    own = torch.empty_like(x)
    for polls in (0, 1, 1 << 14):
        ctx.set_loss_polls(polls)
        own.copy_(x)
        out2, logps2 = call(own, own)
        print(f"{seq} x {vocab}, {polls} polls", flush=True)
        assert torch.equal(logps2, logps), polls
        assert torch.equal(out2, out), polls
        assert torch.equal(own, grad), polls
    ctx.close()
