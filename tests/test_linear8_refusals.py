"""Refusals of the 8-bit layer and draft verification calls, without a GPU: the
arguments are checked before the context, so every refusal can be provoked
with addresses that are never read.  No compute call is made here."""
import ctypes

import pytest
import torch

from newton_schulz_amd import Rows8, _lib, linear8_workspace_bytes, verify_workspace_bytes
from newton_schulz_amd._lib import MUON_BF16, MUON_EDTYPE, MUON_EINVAL, MUON_ESHAPE, MUON_F32, Logits, Rows
from newton_schulz_amd._lib import Rows8 as R8

T, N, K, P = 6, 10, 40, 48  # tokens, channels, inputs, padded inputs
X, W, WS, Q, QS, Y, GX, GW, DRAFT, DL, U, TOK, ACC, LP = (0x100000 * (i + 1) for i in range(14))


def text():
    return _lib.load().muon_last_error(None).decode()


def refused(st, want, words):
    assert st == want and words in text(), (st, text())


def rows(data, r, c, dtype=MUON_BF16, stride=None):
    return Rows(data, dtype, r, c, c if stride is None else stride)


def rows8(data=W, scale=WS, r=N, c=K, stride=P):
    return R8(data, scale, r, c, stride)


def ref(v):
    return None if v is None else ctypes.byref(v)


def quantize(x=None, q=None):
    return _lib.load().muon_quantize_rows(None, None, ref(x or rows(X, T, K)), ref(q or rows8(Q, QS, T)))


def dequantize(q=None, out=None):
    return _lib.load().muon_dequantize_rows(None, None, ref(q or rows8(Q, QS, T)), ref(out or rows(X, T, K)))


def matmul(a=None, b=None, out=None):
    return _lib.load().muon_matmul8(None, None, ref(a or rows8(Q, QS, T)), ref(b or rows8()), ref(out or rows(Y, T, N)))


def linear(x=None, w=None, x8=None, out=None):
    return _lib.load().muon_linear8(None, None, ref(x or rows(X, T, K)), ref(w or rows8()), ref(x8), ref(out or rows(Y, T, N)))


def input_grad(y=None, w=None, out=None):
    return _lib.load().muon_input_grad8(None, None, ref(y or rows(Y, T, N)), ref(w or rows8()), ref(out or rows(GX, T, K)), 0)


def weight_grad(y=None, x=None, out=None):
    return _lib.load().muon_weight_grad8(None, None, ref(y or rows(Y, T, N)), ref(x or rows8(Q, QS, T)),
                                         ref(out or rows(GW, N, K)), 0)


def test_only_the_context_is_missing():
    for st in (quantize(), dequantize(), matmul(), linear(), linear(x8=rows8(Q, QS, T)), input_grad(), weight_grad(),
               quantize(rows(X, T, K, stride=0)), quantize(rows(X, T, K, MUON_F32, K + 1)),
               matmul(a=rows8(Q, QS, T, stride=0)),                                       # one row for every token
               matmul(a=rows8(Q, QS, 1, stride=3), out=rows(Y, 1, N, stride=-5)),         # a single row's stride
               quantize(rows(None, 0, K), rows8(None, None, 0)), input_grad(rows(None, 0, N), out=rows(None, 0, K)),
               weight_grad(rows(None, 0, N), rows8(None, None, 0))):
        refused(st, MUON_EINVAL, "context NULL")


BAD_ROWS = [
    (dict(dtype=7), MUON_EDTYPE, "dtype"), (dict(r=-1), MUON_ESHAPE, "out of range"), (dict(c=0), MUON_ESHAPE, "out of range"),
    (dict(r=(1 << 24) + 1), MUON_ESHAPE, "out of range"), (dict(c=(1 << 22) + 1), MUON_ESHAPE, "out of range"),
    (dict(stride=-1), MUON_ESHAPE, "stride"), (dict(stride=1 << 41), MUON_ESHAPE, "stride"), (dict(data=None), MUON_EINVAL, "NULL"),
    (dict(data=X + 1), MUON_EINVAL, "misaligned"), (dict(data=X + 2, dtype=MUON_F32), MUON_EINVAL, "misaligned"),
]


@pytest.mark.parametrize("change,status,words", BAD_ROWS)
def test_rows_are_checked(change, status, words):
    a = dict(data=X, r=T, c=K)
    a.update(change)
    refused(quantize(rows(**a)), status, words)
    refused(linear(rows(**a)), status, words)
    refused(dequantize(out=rows(**a)), status, words)
    a = dict(data=Y, r=T, c=N)
    a.update(change)
    refused(matmul(out=rows(**a)), status, words)
    if "dtype" not in change or change["dtype"] == 7:
        refused(input_grad(rows(**a)), status, words)
        refused(weight_grad(rows(**a)), status, words)


@pytest.mark.parametrize("change,status,words", [
    (dict(r=-1), MUON_ESHAPE, "out of range"), (dict(c=0), MUON_ESHAPE, "out of range"), (dict(c=131072, stride=131072), MUON_ESHAPE, "out of range"),
    (dict(r=(1 << 24) + 1), MUON_ESHAPE, "out of range"), (dict(stride=-16), MUON_ESHAPE, "stride"), (dict(stride=1 << 41), MUON_ESHAPE, "stride"),
    (dict(data=None), MUON_EINVAL, "NULL"), (dict(scale=None), MUON_EINVAL, "NULL"), (dict(data=Q + 8), MUON_EINVAL, "16 bytes"),
    (dict(stride=K), MUON_EINVAL, "16 bytes"), (dict(scale=QS + 2), MUON_EINVAL, "scale"),
])
def test_8_bit_rows_are_checked(change, status, words):
    a = dict(data=Q, scale=QS, r=T, c=K, stride=P)
    a.update(change)
    refused(quantize(q=rows8(**a)), status, words)
    refused(dequantize(rows8(**a)), status, words)
    refused(matmul(a=rows8(**a)), status, words)
    refused(matmul(b=rows8(**a)), status, words)
    refused(linear(w=rows8(**a)), status, words)
    refused(linear(x8=rows8(**a)), status, words)
    refused(weight_grad(x=rows8(**a)), status, words)
    refused(input_grad(w=rows8(**a)), status, words)


def test_shapes_have_to_match():
    for st in (quantize(q=rows8(Q, QS, T + 1)), quantize(q=rows8(Q, QS, T, K - 1)), dequantize(out=rows(X, T, K + 1)),
               linear(x8=rows8(Q, QS, T + 1)), linear(x8=rows8(Q, QS, T, K - 1))):
        refused(st, MUON_ESHAPE, "differ in shape")
    for st in (matmul(out=rows(Y, T, N + 1)), matmul(out=rows(Y, T + 1, N)), matmul(a=rows8(Q, QS, T, K - 1)),
               linear(rows(X, T, K - 1)), linear(out=rows(Y, T + 1, N)), input_grad(w=rows8(r=N + 1)), input_grad(out=rows(GX, T, K + 1)),
               input_grad(out=rows(GX, T + 1, K)), weight_grad(x=rows8(Q, QS, T + 1)), weight_grad(out=rows(GW, N + 1, K)),
               weight_grad(out=rows(GW, N, K - 1))):
        refused(st, MUON_ESHAPE, "do not match")
    refused(matmul(b=rows8(None, None, 0), out=rows(Y, T, N)), MUON_ESHAPE, "no columns")
    big = 1 << 20
    refused(matmul(rows8(0x10000000, 0x9000000000, big), rows8(0xA000000000, 0xB000000000, big), rows(0x100000000000, big, big)),
            MUON_ESHAPE, "too many")


def test_outputs_stand_alone():
    refused(quantize(q=rows8(Q, QS, T, stride=32)), MUON_EINVAL, "overlap")
    refused(dequantize(out=rows(X, T, K, stride=K - 1)), MUON_EINVAL, "overlap")
    for st in (quantize(q=rows8(X, QS, T)), quantize(q=rows8(Q, Q + 16, T)), quantize(q=rows8(Q, X + 4, T)),
               dequantize(out=rows(Q, T, K)), dequantize(out=rows(QS, T, K)), matmul(out=rows(W + 2, T, N)), matmul(out=rows(QS, T, N)),
               linear(out=rows(X, T, N)), linear(out=rows(WS, T, N)), linear(x8=rows8(W, QS, T)), linear(x8=rows8(Q, Y, T)),
               linear(x8=rows8(X, QS, T)), input_grad(out=rows(Y, T, K)), input_grad(out=rows(W, T, K)),
               weight_grad(out=rows(QS, N, K)), weight_grad(out=rows(Q, N, K))):
        refused(st, MUON_EINVAL, "overlaps")


def test_gradients_are_of_bf16():
    refused(input_grad(rows(Y, T, N, MUON_F32)), MUON_EDTYPE, "bf16")
    refused(weight_grad(rows(Y, T, N, MUON_F32)), MUON_EDTYPE, "bf16")


B, D, V = 3, 4, 100


def logits(data=X, dtype=MUON_BF16, batch=B, seq=D + 1, vocab=V, bs=None, rs=V):
    return Logits(data, dtype, batch, seq, vocab, seq * rs if bs is None else bs, rs)


def verify(x=None, draft=DRAFT, dl="own", u=U, t=1.0, tokens=TOK, accepted=ACC, logps=LP):
    x = x or logits()
    d = logits(DL, MUON_F32, x.batch, x.seq - 1, x.vocab) if dl == "own" else dl
    return _lib.load().muon_verify_draft(None, None, ref(x), draft, ref(d), u, t, tokens, accepted, logps)


def test_verification_is_checked():
    for st in (verify(), verify(dl=None), verify(logps=None), verify(t=0.0, u=None), verify(logits(bs=0, rs=0)),
               verify(logits(seq=1), draft=None, dl=None), verify(logits(seq=1), draft=None, dl=logits(None, seq=0)),
               verify(logits(batch=0), draft=None, u=None, tokens=None, accepted=None, logps=None)):
        refused(st, MUON_EINVAL, "context NULL")
    refused(verify(logits(seq=0), dl=None), MUON_ESHAPE, "no row")
    refused(verify(logits(seq=1026), dl=None), MUON_ESHAPE, "too long")
    refused(verify(logits(vocab=0), dl=None), MUON_ESHAPE, "vocab")
    refused(verify(logits(dtype=5), dl=None), MUON_EDTYPE, "dtype")
    refused(verify(logits(rs=-V), dl=None), MUON_ESHAPE, "stride")
    for t in (-1.0, float("nan"), float("inf"), 1e-31, 1e31):
        refused(verify(t=t), MUON_EINVAL, "temperature")
    for d in (logits(DL, batch=B + 1, seq=D), logits(DL, seq=D + 1), logits(DL, seq=D, vocab=V + 1)):
        refused(verify(dl=d), MUON_ESHAPE, "differ in shape")
    for st in (verify(draft=None), verify(u=None), verify(tokens=None), verify(accepted=None)):
        refused(st, MUON_EINVAL, "null pointer")
    for st in (verify(draft=DRAFT + 4), verify(u=U + 2), verify(tokens=TOK + 4), verify(accepted=ACC + 4), verify(logps=LP + 1)):
        refused(st, MUON_EINVAL, "misaligned")
    for st in (verify(tokens=DRAFT), verify(accepted=TOK + 8), verify(logps=U), verify(tokens=X), verify(logps=DL + 4)):
        refused(st, MUON_EINVAL, "overlaps")


def test_workspace_sizes():
    assert linear8_workspace_bytes(1, 9728, 2560) >= 2560 + 4 and linear8_workspace_bytes(0, 1, 1) >= 0
    assert linear8_workspace_bytes(100, 64, 1000) >= 100 * 1008 + 400
    for bad in ((-1, 1, 1), ((1 << 24) + 1, 1, 1), (1, -1, 1), (1, 1, 0), (1, 1, 131072)):
        assert linear8_workspace_bytes(*bad) == 0
    assert verify_workspace_bytes(1, 0, 1) > 0 and verify_workspace_bytes(64, 8, 151936) > 0
    for bad in ((-1, 1, 1), (1, -1, 1), (1, 1025, 5), (1, 1, 0), (1, 1, (1 << 19) + 1), (1 << 29, 8, 5)):
        assert verify_workspace_bytes(*bad) == 0


def test_rows8_of_tensors():
    q, s = torch.zeros(3, 32, dtype=torch.int8), torch.zeros(3)
    r = Rows8(q[:, :20], s)
    assert r.shape == (3, 20) and r.struct.row_stride == 32 and r[1:].struct.rows == 2
    with pytest.raises(TypeError):
        Rows8(q.int(), s)
    with pytest.raises(TypeError):
        Rows8(q, s.double())
    with pytest.raises(ValueError):
        Rows8(q.t(), torch.zeros(32))
    with pytest.raises(ValueError):
        Rows8(q, torch.zeros(4))
    with pytest.raises(ValueError):
        Rows8(q, torch.zeros(6)[::2])
    with pytest.raises(ValueError):
        Rows8(q[0], s)
