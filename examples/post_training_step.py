"""Post-training steps of a small policy, on one device: the loss on the logits
with its gradient, clipping by the global norm, and the Muon step.

    python examples/post_training_step.py                      # clipped policy loss with a KL term
    python examples/post_training_step.py --loss preference    # paired preference loss

The policy is an embedding, two hidden matrices and an output matrix.  Per step

    logits = policy(tokens)                        torch
    ctx.policy_loss / ctx.preference_loss          loss, and its gradient in the logits
    logits.backward(gradient)                      torch
    ctx.clip_grads(..., out=views of step.grad)    norm, and the clipped gradients where Muon reads them
    step.step()                                    momentum -> Newton-Schulz -> apply

The reference's and the old policy's log-probabilities come from
ctx.token_logps on the same kind of logits, without a gradient.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from newton_schulz_amd import Context, MuonStep, loss_workspace_bytes  # noqa: E402


class Policy:
    """tokens -> logits; the hidden and output matrices are Muon's, the
    embedding takes plain steps."""

    def __init__(self, vocab: int, hidden: int, device, seed: int = 0):
        g = torch.Generator().manual_seed(seed)

        def make(*shape, std):
            return (torch.randn(*shape, generator=g) * std).to(device).requires_grad_()

        self.embedding = make(vocab, hidden, std=1.0)
        self.matrices = [make(hidden, hidden, std=hidden ** -0.5), make(hidden, hidden, std=hidden ** -0.5),
                         make(vocab, hidden, std=hidden ** -0.5)]

    def logits(self, tokens: torch.Tensor) -> torch.Tensor:
        x = self.embedding[tokens]
        for w in self.matrices[:-1]:
            x = x + torch.tanh(x @ w.t())
        return (x @ self.matrices[-1].t()).to(torch.bfloat16)


def train(loss: str = "policy", steps: int = 8, batch: int = 8, seq: int = 24, vocab: int = 1009, hidden: int = 128,
          prompt: int = 6, lr: float = 0.004, max_norm: float = 1.0, device="cuda:0", say=print):
    """The loss of each step, as floats."""
    device = torch.device(device)
    policy = Policy(vocab, hidden, device)
    shapes = [(*w.shape, 0) for w in policy.matrices]
    muon = MuonStep(shapes, device, lr=lr, keep_bf16_weights=False)
    for i, w in enumerate(policy.matrices):
        muon.view(muon.master, i).copy_(w.detach())
    ctx = Context(device, max(loss_workspace_bytes(batch, seq, vocab), 1 << 20))

    # sampled sequences; the loss counts what follows the prompt
    g = torch.Generator().manual_seed(1)
    tokens = torch.randint(vocab, (batch, seq + 1), generator=g).to(device)
    inputs, labels = tokens[:, :-1], tokens[:, 1:].contiguous()
    labels[:, :prompt] = -100
    advantages = torch.randn(batch, generator=g).to(device)

    def buffer(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device=device)

    with torch.no_grad():  # reference and old policy: the policy before the first step
        ref = buffer(batch, seq)
        ctx.token_logps(policy.logits(inputs), labels, ref)
    old = ref.clone()
    out, norm = buffer(4 if loss == "policy" else 3), buffer(3, dtype=torch.float64)
    grad = buffer(batch, seq, vocab, dtype=torch.bfloat16)
    history = []
    for k in range(steps):
        logits = policy.logits(inputs)
        if loss == "policy":
            ctx.policy_loss(logits.detach(), labels, advantages, out, old_logps=old, ref_logps=ref, grad_logits=grad,
                            kl_coef=0.02, reduce="sequence")
        else:
            ctx.preference_loss(logits.detach(), labels, ref, out, grad_logits=grad, beta=0.2)
        for p in (policy.embedding, *policy.matrices):
            p.grad = None
        logits.backward(grad)
        # one norm over everything; Muon's matrices go clipped into its flat
        # buffer (in its dtype), the embedding's gradient is clipped in place
        grads = [policy.embedding.grad, *(w.grad for w in policy.matrices)]
        ctx.clip_grads(grads, norm, max_norm,
                       out=[grads[0], *(muon.view(muon.grad, i) for i in range(len(policy.matrices)))])
        muon.step()
        with torch.no_grad():
            policy.embedding -= 0.5 * policy.embedding.grad
            for i, w in enumerate(policy.matrices):
                w.copy_(muon.view(muon.master, i))
        history.append(out[0].item())
        say(f"step {k}: loss {history[-1]:.5f}  gradient norm {norm[1].item():.4f}  coefficient {norm[2].item():.4f}")
    ctx.close()
    for c in muon.contexts:
        c.close()
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--loss", choices=("policy", "preference"), default="policy")
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    train(a.loss, a.steps)
