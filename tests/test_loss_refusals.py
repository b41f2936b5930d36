"""Refusals of the loss and clipping calls, without a GPU: the arguments are
checked before the context, so every refusal can be provoked with addresses
that are never read.  No compute call is made here."""
import ctypes

import pytest
import torch

from newton_schulz_amd import _lib, loss_workspace_bytes
from newton_schulz_amd._lib import (
    MUON_BF16, MUON_EDTYPE, MUON_EINVAL, MUON_ESHAPE, MUON_F32, Logits, PolicyParams, PreferenceParams, Tensor,
)

B, S, V = 2, 3, 100
LOGITS, GRAD, LABELS, ADV, OLD, REF, OUT, LOGPS, STATS, NORM, REWARDS = (0x10000 * (i + 1) for i in range(11))


def text():
    return _lib.load().muon_last_error(None).decode()


def logits(data=LOGITS, dtype=MUON_BF16, batch=B, seq=S, vocab=V, bs=S * V, rs=V):
    return Logits(data, dtype, batch, seq, vocab, bs, rs)


def policy(x=None, labels=LABELS, params=(), adv=ADV, old=OLD, ref=REF, out=OUT, logps=LOGPS, grad="own"):
    p = dict(temperature=1.0, clip_low=0.2, clip_high=0.2, kl_coef=0.1, weight=1.0, reduce=0, advantage_per_token=0)
    p.update(params)
    x = x if x is not None else logits()
    g = logits(GRAD, x.dtype, x.batch, x.seq, x.vocab, x.batch_stride, x.row_stride) if grad == "own" else grad
    return _lib.load().muon_policy_loss(
        None, None, ctypes.byref(x), labels, ctypes.byref(PolicyParams(**p)), adv, old, ref, out, logps,
        ctypes.byref(g) if g is not None else None)


def preference(x=None, params=(), ref=REF, out=OUT, rewards=REWARDS, logps=LOGPS, grad=None):
    p = dict(beta=0.1, label_smoothing=0.0, temperature=1.0, weight=1.0, kind=0, average=0)
    p.update(params)
    x = x if x is not None else logits()
    return _lib.load().muon_preference_loss(
        None, None, ctypes.byref(x), LABELS, ctypes.byref(PreferenceParams(**p)), ref, out, rewards, logps,
        ctypes.byref(grad) if grad is not None else None)


def refused(st, want, words):
    assert st == want and words in text(), (st, text())


def test_only_the_context_is_missing():
    for st in (policy(), policy(grad=None), preference(), policy(ref=None, params=dict(kl_coef=0.0)),
               policy(grad=logits()),                                   # in place
               policy(x=logits(batch=0), labels=None, adv=None, old=None, ref=None, logps=None, grad=None),
               policy(x=logits(bs=0, rs=0), grad=logits(GRAD))):        # broadcast scores
        refused(st, MUON_EINVAL, "context NULL")


def test_logits_are_checked():
    refused(policy(x=logits(dtype=7), grad=None), MUON_EDTYPE, "dtype")
    refused(policy(x=logits(vocab=0), grad=None), MUON_ESHAPE, "vocab")
    refused(policy(x=logits(vocab=(1 << 19) + 1, rs=1 << 20), grad=None), MUON_ESHAPE, "vocab")
    refused(policy(x=logits(vocab=(1 << 30) + 1), grad=None), MUON_ESHAPE, "vocab")
    refused(policy(x=logits(batch=-1), grad=None), MUON_ESHAPE, "batch")
    refused(policy(x=logits(batch=1 << 20, seq=1 << 20), grad=None), MUON_ESHAPE, "batch")
    refused(policy(x=logits(rs=-V), grad=None), MUON_ESHAPE, "stride")
    refused(policy(x=logits(bs=1 << 60), grad=None), MUON_ESHAPE, "stride")
    refused(policy(x=logits(data=None), grad=None), MUON_EINVAL, "data NULL")
    refused(policy(x=logits(data=LOGITS + 1), grad=None), MUON_EINVAL, "misaligned")
    refused(policy(x=logits(data=LOGITS + 2, dtype=MUON_F32), grad=None), MUON_EINVAL, "misaligned")


def test_gradient_is_checked():
    refused(policy(grad=logits(GRAD, dtype=MUON_F32)), MUON_EDTYPE, "differ in dtype")
    refused(policy(grad=logits(GRAD, vocab=V - 1)), MUON_ESHAPE, "differ in shape")
    refused(policy(grad=logits(GRAD, rs=V - 1)), MUON_EINVAL, "rows of the gradient")
    refused(policy(grad=logits(GRAD, bs=S * V - 1)), MUON_EINVAL, "rows of the gradient")
    refused(policy(grad=logits(GRAD, bs=0)), MUON_EINVAL, "rows of the gradient")
    refused(policy(grad=logits(LOGITS + 2)), MUON_EINVAL, "overlaps")
    refused(policy(grad=logits(LOGITS, bs=S * V + 8)), MUON_EINVAL, "overlaps")
    # sequence-major rows are disjoint too
    refused(policy(grad=logits(GRAD, bs=V, rs=B * V)), MUON_EINVAL, "context NULL")
    refused(policy(grad=logits(GRAD, bs=V, rs=B * V - 1)), MUON_EINVAL, "rows of the gradient")


@pytest.mark.parametrize("params", [
    dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("inf")), dict(temperature=float("nan")),
    dict(temperature=1e-45), dict(temperature=1e31), dict(clip_low=-0.1), dict(clip_low=1.5), dict(clip_high=-0.1), dict(clip_high=float("nan")),
    dict(kl_coef=-1.0), dict(kl_coef=float("inf")), dict(weight=float("nan")), dict(reduce=3), dict(reduce=-1)])
def test_policy_parameters(params):
    st = policy(params=params)
    assert st == MUON_EINVAL and "context" not in text(), text()


@pytest.mark.parametrize("params", [
    dict(beta=0.0), dict(beta=-1.0), dict(beta=float("inf")), dict(label_smoothing=0.6), dict(label_smoothing=-0.1),
    dict(kind=2), dict(kind=1, label_smoothing=0.1), dict(weight=float("inf")), dict(temperature=0.0)])
def test_preference_parameters(params):
    st = preference(params=params)
    assert st == MUON_EINVAL and "context" not in text(), text()


def test_pointers_and_overlaps():
    refused(policy(labels=None), MUON_EINVAL, "null pointer")
    refused(policy(adv=None), MUON_EINVAL, "null pointer")
    refused(policy(out=None), MUON_EINVAL, "null pointer")
    refused(policy(ref=None), MUON_EINVAL, "kl_coef needs")
    refused(policy(labels=LABELS + 4), MUON_EINVAL, "misaligned")
    refused(policy(out=OUT + 2), MUON_EINVAL, "misaligned")
    refused(policy(logps=OLD), MUON_EINVAL, "overlaps")
    refused(policy(out=LOGPS), MUON_EINVAL, "overlaps")
    refused(policy(logps=LOGITS), MUON_EINVAL, "overlaps")
    refused(policy(logps=GRAD + 4), MUON_EINVAL, "overlaps")
    refused(preference(x=logits(batch=3)), MUON_ESHAPE, "odd")
    refused(preference(rewards=REF), MUON_EINVAL, "overlaps")


def test_token_logps_arguments():
    f = _lib.load().muon_token_logps
    x = logits()
    refused(f(None, None, ctypes.byref(x), LABELS, 1.0, LOGPS, STATS), MUON_EINVAL, "context NULL")
    refused(f(None, None, ctypes.byref(x), LABELS, 1.0, LOGPS, None), MUON_EINVAL, "context NULL")
    refused(f(None, None, None, LABELS, 1.0, LOGPS, STATS), MUON_EINVAL, "logits NULL")
    refused(f(None, None, ctypes.byref(x), LABELS, 0.0, LOGPS, STATS), MUON_EINVAL, "temperature")
    refused(f(None, None, ctypes.byref(x), LABELS, 1.0, None, STATS), MUON_EINVAL, "null pointer")
    refused(f(None, None, ctypes.byref(x), LABELS, 1.0, LOGPS, STATS + 4), MUON_EINVAL, "misaligned")
    refused(f(None, None, ctypes.byref(x), LABELS, 1.0, LOGPS, LOGPS + 8), MUON_EINVAL, "overlaps")
    b = _lib.load().muon_token_logps_backward
    g = logits(GRAD)
    refused(b(None, None, ctypes.byref(x), LABELS, 1.0, STATS, ADV, ctypes.byref(g)), MUON_EINVAL, "context NULL")
    refused(b(None, None, ctypes.byref(x), LABELS, 1.0, None, ADV, ctypes.byref(g)), MUON_EINVAL, "null pointer")
    refused(b(None, None, ctypes.byref(x), LABELS, 1.0, STATS, ADV, None), MUON_EINVAL, "grad_logits NULL")
    refused(b(None, None, ctypes.byref(x), LABELS, 1.0, GRAD, ADV, ctypes.byref(g)), MUON_EINVAL, "overlaps")


def tensors(*entries):
    return (Tensor * max(1, len(entries)))(*[Tensor(*e) for e in entries]), len(entries)


def test_gradient_list_arguments():
    lib = _lib.load()
    good = tensors((0x10000, 10, MUON_BF16), (0x20000, 7, MUON_F32), (None, 0, MUON_F32))
    refused(lib.muon_grad_norm(None, None, *good, 1.0, 1e-6, NORM), MUON_EINVAL, "context NULL")
    refused(lib.muon_grad_norm(None, None, *good, float("inf"), 0.0, NORM), MUON_EINVAL, "context NULL")
    refused(lib.muon_grad_norm(None, None, None, 0, 1.0, 1e-6, NORM), MUON_EINVAL, "context NULL")
    refused(lib.muon_grad_norm(None, None, None, 2, 1.0, 1e-6, NORM), MUON_EINVAL, "list NULL")
    refused(lib.muon_grad_norm(None, None, None, -1, 1.0, 1e-6, NORM), MUON_EINVAL, "count")
    for m, e in ((0.0, 0.0), (-1.0, 0.0), (float("nan"), 0.0), (1.0, -1.0), (1.0, float("nan")), (1.0, float("inf"))):
        st = lib.muon_grad_norm(None, None, *good, m, e, NORM)
        assert st == MUON_EINVAL and ("max_norm" in text() or "eps" in text())
    refused(lib.muon_grad_norm(None, None, *good, 1.0, 1e-6, None), MUON_EINVAL, "norm NULL")
    refused(lib.muon_grad_norm(None, None, *good, 1.0, 1e-6, NORM + 4), MUON_EINVAL, "misaligned")
    refused(lib.muon_grad_norm(None, None, *good, 1.0, 1e-6, 0x20000), MUON_EINVAL, "overlaps")
    for entry, st, words in (((0x10000, 10, 5), MUON_EDTYPE, "dtype"), ((0x10000, -1, 0), MUON_ESHAPE, "numel"),
                             ((0x10000, 1 << 41, 0), MUON_ESHAPE, "numel"), ((None, 3, 0), MUON_EINVAL, "NULL"),
                             ((0x10002, 3, 0), MUON_EINVAL, "misaligned")):
        refused(lib.muon_grad_norm(None, None, *tensors(entry), 1.0, 1e-6, NORM), st, words)
        assert lib.muon_grad_norm_workspace_bytes(*tensors(entry)) == 0
    refused(lib.muon_clip_coef(None, None, 1.0, 1e-6, NORM), MUON_EINVAL, "context NULL")
    refused(lib.muon_clip_coef(None, None, 0.0, 1e-6, NORM), MUON_EINVAL, "max_norm")


def test_scaled_outputs_are_checked():
    lib = _lib.load()
    grads, n = tensors((0x10000, 16, MUON_BF16), (0x20000, 16, MUON_F32))

    def scale(out, norm=NORM):
        return lib.muon_scale_grads(None, None, grads, tensors(*out)[0] if out else None, n, norm)

    refused(scale(None), MUON_EINVAL, "context NULL")
    refused(scale([(0x10000, 16, MUON_BF16), (0x30000, 16, MUON_BF16)]), MUON_EINVAL, "context NULL")
    refused(scale([(0x10000, 16, MUON_F32), (0x30000, 16, MUON_BF16)]), MUON_EINVAL, "overlap")
    refused(scale([(0x10010, 16, MUON_BF16), (0x30000, 16, MUON_BF16)]), MUON_EINVAL, "overlap")
    refused(scale([(0x30000, 16, MUON_BF16), (0x30010, 16, MUON_BF16)]), MUON_EINVAL, "overlap")
    refused(scale([(0x30000, 16, MUON_BF16), (0x40000, 15, MUON_BF16)]), MUON_ESHAPE, "numel")
    refused(scale(None, norm=0x20008), MUON_EINVAL, "overlap")
    refused(scale(None, norm=None), MUON_EINVAL, "norm NULL")
    twice, _ = tensors((0x10000, 16, MUON_BF16), (0x10000, 16, MUON_BF16))
    refused(lib.muon_scale_grads(None, None, twice, None, 2, NORM), MUON_EINVAL, "overlap")


def test_polls():
    lib = _lib.load()
    refused(lib.muon_loss_set_polls(None, 5), MUON_EINVAL, "context NULL")
    refused(lib.muon_loss_set_polls(None, -1), MUON_EINVAL, "polls")


def test_clipped_momentum_without_context():
    assert _lib.load().muon_momentum_update_clipped(None, None, None, 1, None, None, 1, 8, 0.9, 1, NORM,
                                                    None) == MUON_EINVAL


def test_workspace_sizes():
    lib = _lib.load()
    bf, f32 = torch.bfloat16, torch.float32
    assert loss_workspace_bytes(-1, 4, 100) == 0 and loss_workspace_bytes(1 << 20, 1 << 20, 100) == 0
    assert loss_workspace_bytes(2, 4, 0) == 0 and loss_workspace_bytes(2, 4, 100, torch.float16) == 0
    # per token two floats, a double and two words, a word for each slice of
    # at most 2560 pieces of 16 bytes; per sequence a double, per pair three
    for dtype, slices in ((bf, 8), (f32, 15)):
        need = 4096 * (8 + 8 + 16 + 8 * slices) + 8 * 5 + 24 * 2 + 24 * 64
        assert need <= loss_workspace_bytes(4, 1024, 151936, dtype) <= need + 7 * 256
    assert loss_workspace_bytes(0, 0, 100) > 0
    # one double per chunk of 8192 elements, and 32 more
    t, n = tensors((0x10000, 1 << 30, MUON_BF16))
    assert lib.muon_grad_norm_workspace_bytes(t, n) == 8 * ((1 << 17) + 32)
    assert lib.muon_grad_norm_workspace_bytes(None, 0) == 0
