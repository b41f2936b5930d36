"""Python binding of libmuon: argument marshalling only.

Every step of the optimizer runs in the HIP kernels behind include/muon.h;
PyTorch supplies device memory and the current HIP stream.  When libmuon.so
is missing the calls raise instead of falling back to any other code.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import List, Optional, Sequence, Tuple

import torch

from . import _lib
from ._lib import (
    MUON_BF16, MUON_CAP_FULL_BYTES, MUON_CAP_WORKSPACE, MUON_F32, Logits, NsParams, PolicyParams,
    PreferenceParams, Rows, Shape, Tensor,
)


class MuonError(RuntimeError):
    def __init__(self, status: int, msg: str = ""):
        lib = _lib.load()
        text = lib.muon_status_string(status).decode()
        super().__init__(f"libmuon status {status} ({text}){': ' + msg if msg else ''}")
        self.status = status


_DT = {torch.float32: MUON_F32, torch.bfloat16: MUON_BF16}


def _dtype(t: torch.Tensor) -> int:
    dt = _DT.get(t.dtype)
    if dt is None:
        raise TypeError(f"unsupported dtype {t.dtype}; libmuon takes float32 or bfloat16")
    return dt


def _stream(device: torch.device, stream) -> int:
    # the raw handle of the current stream: building a torch.cuda.Stream for it
    # costs 2 us a call
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


def _check(t: torch.Tensor, name: str, device: torch.device):
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


NS_FUSE = {"auto": 0, "off": 1, "on": 2}
SQ_BLOCK = 4096  # MUON_SQ_BLOCK
NS_METHODS = {"quintic": 0, "gram": 1}


def minimax_coeffs(steps: int, lo: float = 1e-3, margin: float = 0.05) -> Tuple[list, float]:
    """Per-iteration (a, b, c) rows from libmuon's muon_ns_minimax_coeffs and
    the bound E after the last one (every singular value of X_0 in [lo, 1]
    ends in [1 - E, 1 + E] in exact arithmetic)."""
    lib = _lib.load()
    out = (ctypes.c_float * (3 * steps))()
    bound = ctypes.c_double()
    st = lib.muon_ns_minimax_coeffs(steps, lo, margin, out, ctypes.byref(bound))
    if st != _lib.MUON_OK:
        raise MuonError(st, "muon_ns_minimax_coeffs")
    return [tuple(out[3 * k:3 * k + 3]) for k in range(steps)], bound.value


def ns_params(steps: int = 5, a: float = 3.4445, b: float = -4.7750, c: float = 2.0315,
              eps: float = 1e-7, compute: str = "bf16", method: str = "quintic",
              fuse: str = "auto", coeffs=None, lo: float = 1e-3,
              margin: float = 0.05) -> NsParams:
    """Newton-Schulz parameters.  coeffs: None (the fixed a, b, c), "minimax"
    (libmuon's per-iteration schedule for `lo`, `margin`), or `steps` rows of
    (a, b, c).  The returned structure keeps its coefficient table alive."""
    p = NsParams(steps, a, b, c, eps, MUON_BF16 if compute == "bf16" else MUON_F32,
                 NS_METHODS[method], NS_FUSE[fuse], None)
    if coeffs is not None:
        if isinstance(coeffs, str) and coeffs != "minimax":
            raise ValueError(f"unknown coefficient schedule {coeffs!r}")
        rows = minimax_coeffs(steps, lo, margin)[0] if isinstance(coeffs, str) else coeffs
        flat = [float(v) for r in rows for v in r]
        if len(flat) != 3 * steps:
            raise ValueError("coeffs must hold `steps` rows of (a, b, c)")
        table = (ctypes.c_float * len(flat))(*flat)
        p.coeffs = ctypes.cast(table, ctypes.POINTER(ctypes.c_float))
        p._table = table  # owned by the structure for as long as it lives
    return p


def sq_blocks(numel: int) -> int:
    """Sum-of-squares partials a momentum pass over `numel` elements writes."""
    return (int(numel) + SQ_BLOCK - 1) // SQ_BLOCK


def ns_workspace_bytes(rows: int, cols: int, count: int, head_rows: int = 0,
                       compute: str = "bf16") -> int:
    return int(_lib.load().muon_ns_workspace_bytes(
        Shape(rows, cols, head_rows), count, MUON_BF16 if compute == "bf16" else MUON_F32))


def workspace_bytes(shapes: Sequence[Tuple[int, int, int]], compute: str = "bf16") -> int:
    """muon_workspace_bytes: workspace for Newton-Schulz over mixed shapes, one
    call per shape group, one after another on one context."""
    arr = (Shape * max(len(shapes), 1))(*[Shape(r, c, h) for (r, c, h) in shapes])
    return int(_lib.load().muon_workspace_bytes(arr, len(shapes),
                                                MUON_BF16 if compute == "bf16" else MUON_F32))


def newton_schulz_noalloc(mats: Sequence[torch.Tensor], out: Optional[Sequence[torch.Tensor]] = None,
                          head_rows: int = 0, params: Optional[NsParams] = None,
                          nonfinite_flag: Optional[torch.Tensor] = None, stream=None):
    """muon_newton_schulz_batched_noalloc: the batched Newton-Schulz without a
    context or any allocation (static device scratch of
    MUON_NOALLOC_SCRATCH_BYTES per GPU).  Matrices evenly spaced; out None
    (in place), the inputs, or disjoint from them."""
    lib = _lib.load()
    device = mats[0].device
    if params is None:
        params = ns_params(compute="bf16" if mats[0].dtype == torch.bfloat16 else "f32")
    shape, dt = mats[0].shape, mats[0].dtype
    for i, m in enumerate(mats):
        _check(m, f"mats[{i}]", device)
        if m.dim() != 2 or m.shape != shape or m.dtype != dt:
            raise ValueError("all matrices of one call must be 2D with one shape and dtype")
    arr_t = ctypes.c_void_p * len(mats)
    pin = arr_t(*[m.data_ptr() for m in mats])
    pout = None
    if out is not None:
        for i, o in enumerate(out):
            _check(o, f"out[{i}]", device)
        pout = arr_t(*[o.data_ptr() for o in out])
    flag = ctypes.c_void_p(nonfinite_flag.data_ptr()) if nonfinite_flag is not None else None
    st = lib.muon_newton_schulz_batched_noalloc(
        device.index, _stream(device, stream), pin, len(mats), Shape(shape[0], shape[1], head_rows),
        _dtype(mats[0]), ctypes.byref(params), pout, flag)
    if st != _lib.MUON_OK:
        raise MuonError(st, f"muon_newton_schulz_batched_noalloc: {lib.muon_noalloc_last_error().decode()}")


LOSS_REDUCE = {"token": 0, "sequence": 1, "sum": 2}
PREFERENCE_KINDS = {"sigmoid": 0, "ipo": 1}


def loss_workspace_bytes(batch: int, seq: int, vocab: int, dtype: torch.dtype = torch.bfloat16) -> int:
    """Workspace a context needs for any loss call on batch x seq rows of
    `vocab` scores."""
    return int(_lib.load().muon_loss_workspace_bytes(batch, seq, vocab, _DT.get(dtype, -1)))


def grad_norm_workspace_bytes(tensors: Sequence[torch.Tensor]) -> int:
    """Workspace a context needs for grad_norm over these tensors."""
    arr = (Tensor * max(len(tensors), 1))(*[Tensor(t.data_ptr(), t.numel(), _dtype(t)) for t in tensors])
    return int(_lib.load().muon_grad_norm_workspace_bytes(arr, len(tensors)))


def _logits(t: torch.Tensor, name: str, device: torch.device) -> Logits:
    """Scores as [batch, seq, vocab] or [rows, vocab]: any strides, the
    vocabulary contiguous."""
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    shape, stride = t.shape, t.stride()
    if len(shape) == 2:
        shape, stride = (1, *shape), (0, *stride)
    elif len(shape) != 3:
        raise ValueError(f"{name} must be [batch, seq, vocab] or [rows, vocab]")
    if shape[2] > 1 and stride[2] != 1:
        raise ValueError(f"the vocabulary of {name} must be contiguous")
    return Logits(t.data_ptr(), _dtype(t), shape[0], shape[1], shape[2], stride[0], stride[1])


def _tokens(t: Optional[torch.Tensor], name: str, shape, dtype: torch.dtype, device: torch.device):
    """Device address of a dense per-token (or per-sequence) array, or None."""
    if t is None:
        return None
    _check(t, name, device)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}")
    return t.data_ptr()


class TensorList:
    """A list of tensors as libmuon takes it (Context.tensor_list): made once
    for tensors that stay where they are, kept while they live."""

    def __init__(self, tensors: Sequence[torch.Tensor], device: torch.device):
        for i, t in enumerate(tensors):
            _check(t, f"tensors[{i}]", device)
        self.tensors = list(tensors)
        self.array = (Tensor * max(len(self.tensors), 1))(
            *[Tensor(t.data_ptr(), t.numel(), _dtype(t)) for t in self.tensors])

    def __len__(self):
        return len(self.tensors)

    def norm_workspace_bytes(self) -> int:
        """Workspace a context needs for grad_norm over the list."""
        return int(_lib.load().muon_grad_norm_workspace_bytes(self.array, len(self)))


def linear8_workspace_bytes(tokens: int, n: int, k: int) -> int:
    """Workspace a context needs for any call on a layer of n x k 8-bit weights
    and up to `tokens` tokens."""
    return int(_lib.load().muon_linear8_workspace_bytes(tokens, n, k))


def verify_workspace_bytes(batch: int, draft: int, vocab: int) -> int:
    """Workspace a context needs for verify_draft."""
    return int(_lib.load().muon_verify_workspace_bytes(batch, draft, vocab))


def _rows(t: torch.Tensor, name: str, device: torch.device) -> Rows:
    """Values as [rows, cols], or [..., cols] whose leading dimensions are rows
    at one stride; the columns contiguous."""
    if t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 2:
        if len(shape) < 2:
            raise ValueError(f"{name} must be [rows, cols]")
        try:
            t = t.flatten(0, -2) if t.numel() == 0 else t.view(-1, shape[-1])
        except RuntimeError:
            raise ValueError(f"the rows of {name} lie at no one stride") from None
        shape, stride = t.shape, t.stride()
    rows, cols = shape
    if stride[1] != 1 and cols > 1:
        raise ValueError(f"the columns of {name} must be contiguous")
    return Rows(t.data_ptr(), _dtype(t), rows, cols, stride[0])


class Rows8:
    """8-bit rows: values scale[r] * q[r, c].  q: int8 [rows, cols], rows at
    multiples of 16 bytes (Context.rows8 makes such ones); scale: float32
    [rows].  Made once for tensors that stay where they are, kept while they
    live."""

    def __init__(self, q: torch.Tensor, scale: torch.Tensor):
        if q.dtype != torch.int8:
            raise TypeError("q must be int8")
        if q.dim() != 2 or (q.shape[1] > 1 and q.stride(1) != 1):
            raise ValueError("q must be [rows, cols], the columns contiguous")
        if scale.device != q.device or not scale.is_contiguous():
            raise ValueError("scale must be contiguous and on q's device")
        if scale.dtype != torch.float32:
            raise TypeError("scale must be float32")
        if scale.shape != q.shape[:1]:
            raise ValueError("scale must hold one number per row")
        self.q, self.scale, self.device = q, scale, q.device
        self.struct = _lib.Rows8(q.data_ptr(), scale.data_ptr(), q.shape[0], q.shape[1], q.stride(0))

    @property
    def shape(self):
        return self.q.shape

    def __getitem__(self, rows: slice) -> "Rows8":
        """Some of the rows, in place."""
        return Rows8(self.q[rows], self.scale[rows])


class Context:
    """A libmuon context: one device and one preallocated workspace slab."""

    def __init__(self, device=None, workspace_bytes: int = 0):
        self.lib = _lib.load()
        self.device = torch.device(device if device is not None else "cuda", )
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        h = ctypes.c_void_p()
        st = self.lib.muon_create(self.device.index, int(workspace_bytes), ctypes.byref(h))
        if st != _lib.MUON_OK:
            raise MuonError(st, "muon_create")
        self.handle = h
        self.workspace_bytes = int(workspace_bytes)

    def close(self):
        if getattr(self, "handle", None):
            self.lib.muon_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _raise(self, st: int, what: str):
        if st != _lib.MUON_OK:
            raise MuonError(st, f"{what}: {self.lib.muon_last_error(self.handle).decode()}")

    # -- the three steps ----------------------------------------------------
    def momentum_update(self, grad: torch.Tensor, momentum: torch.Tensor, update_out: torch.Tensor,
                        beta: float = 0.95, nesterov: bool = True, stream=None,
                        sq_partials: Optional[torch.Tensor] = None,
                        grad_scale: Optional[torch.Tensor] = None):
        """Momentum step; with `sq_partials` (float64, ceil(numel / 4096)
        elements) also the per-block sums of squares of the stored update;
        with `grad_scale` (grad_norm's float64 triple) on the gradient times
        the clip coefficient in it."""
        for t, n in ((grad, "grad"), (momentum, "momentum"), (update_out, "update_out")):
            _check(t, n, self.device)
        if momentum.dtype != torch.float32:
            raise TypeError("momentum must be float32")
        numel = grad.numel()
        if momentum.numel() != numel or update_out.numel() != numel:
            raise ValueError("grad, momentum and update_out must have the same numel")
        args = (self.handle, _stream(self.device, stream), ctypes.c_void_p(grad.data_ptr()), _dtype(grad),
                ctypes.c_void_p(momentum.data_ptr()), ctypes.c_void_p(update_out.data_ptr()),
                _dtype(update_out), numel, float(beta), 1 if nesterov else 0)
        sq = None
        if sq_partials is not None:
            _check(sq_partials, "sq_partials", self.device)
            if sq_partials.dtype != torch.float64 or sq_partials.numel() < sq_blocks(numel):
                raise ValueError(f"sq_partials must be float64 with at least {sq_blocks(numel)} elements")
            sq = ctypes.c_void_p(sq_partials.data_ptr())
        if grad_scale is not None:
            st = self.lib.muon_momentum_update_clipped(*args, self._norm(grad_scale), sq)
        elif sq is not None:
            st = self.lib.muon_momentum_update_sq(*args, sq)
        else:
            st = self.lib.muon_momentum_update(*args)
        self._raise(st, "muon_momentum_update")

    def newton_schulz(self, mats: Sequence[torch.Tensor], out: Optional[Sequence[torch.Tensor]] = None,
                      head_rows: int = 0, params: Optional[NsParams] = None,
                      nonfinite_flag: Optional[torch.Tensor] = None, stream=None,
                      _ptrs: Optional[Tuple] = None, sq: Optional[Tuple] = None):
        """Orthogonalise a same-shape group of matrices (in place when out is None).

        sq = (partials, base): norms from a momentum pass's sum-of-squares
        partials (float64 tensor) written for the update buffer `base` (a
        tensor, or its device address) that the matrices are views of."""
        if params is None:
            params = ns_params(compute="bf16" if mats[0].dtype == torch.bfloat16 else "f32")
        if sq is not None:
            partials, base = sq
            p = NsParams()
            ctypes.memmove(ctypes.byref(p), ctypes.byref(params), ctypes.sizeof(NsParams))
            p.sq_partials = partials.data_ptr()
            p.sq_base = base if isinstance(base, int) else base.data_ptr()
            p.sq_count = partials.numel()
            params = p
        if _ptrs is None:
            _ptrs = self.pointer_arrays(mats, out)
        rows, cols = mats[0].shape[-2], mats[0].shape[-1]
        flag = ctypes.c_void_p(nonfinite_flag.data_ptr()) if nonfinite_flag is not None else None
        pin, pout, count = _ptrs
        st = self.lib.muon_newton_schulz_batched(
            self.handle, _stream(self.device, stream), pin, count, Shape(rows, cols, head_rows),
            _dtype(mats[0]), ctypes.byref(params), pout, flag)
        self._raise(st, "muon_newton_schulz_batched")

    def pointer_arrays(self, mats: Sequence[torch.Tensor], out: Optional[Sequence[torch.Tensor]] = None):
        """Host pointer arrays for newton_schulz (cacheable while the tensors live)."""
        if isinstance(mats, torch.Tensor) and mats.dim() == 3:
            mats = list(mats.unbind(0))
        if out is not None and isinstance(out, torch.Tensor) and out.dim() == 3:
            out = list(out.unbind(0))
        shape, dt = mats[0].shape, mats[0].dtype
        for i, m in enumerate(mats):
            _check(m, f"mats[{i}]", self.device)
            if m.dim() != 2 or m.shape != shape or m.dtype != dt:
                raise ValueError("all matrices of one call must be 2D with one shape and dtype")
        arr_t = ctypes.c_void_p * len(mats)
        pin = arr_t(*[m.data_ptr() for m in mats])
        pout = None
        if out is not None:
            if len(out) != len(mats):
                raise ValueError("out must have one matrix per input")
            for i, o in enumerate(out):
                _check(o, f"out[{i}]", self.device)
                if o.shape != shape or o.dtype != dt:
                    raise ValueError("out matrices must match the inputs")
            pout = arr_t(*[o.data_ptr() for o in out])
        return pin, pout, len(mats)

    def apply(self, master: torch.Tensor, update: torch.Tensor, lr: float, scale: float = 1.0,
              weight_decay: float = 0.0, weight_bf16: Optional[torch.Tensor] = None, stream=None):
        _check(master, "master", self.device)
        _check(update, "update", self.device)
        if master.dtype != torch.float32:
            raise TypeError("master must be float32")
        numel = master.numel()
        if update.numel() != numel:
            raise ValueError("master and update must have the same numel")
        wb = None
        if weight_bf16 is not None:
            _check(weight_bf16, "weight_bf16", self.device)
            if weight_bf16.dtype != torch.bfloat16 or weight_bf16.numel() != numel:
                raise ValueError("weight_bf16 must be bfloat16 with the master's numel")
            wb = ctypes.c_void_p(weight_bf16.data_ptr())
        st = self.lib.muon_apply(self.handle, _stream(self.device, stream),
                                 ctypes.c_void_p(master.data_ptr()), ctypes.c_void_p(update.data_ptr()),
                                 _dtype(update), wb, numel, float(lr), float(scale), float(weight_decay))
        self._raise(st, "muon_apply")

    # -- the losses in front of the step --------------------------------------
    def token_logps(self, logits: torch.Tensor, labels: torch.Tensor, logps: torch.Tensor,
                    row_stats: Optional[torch.Tensor] = None, temperature: float = 1.0, stream=None):
        """Log-probability of every row's label under softmax(logits /
        temperature) into `logps` (float32, the labels' shape; 0 where the
        label is negative).  `row_stats` (float32, [..., 2]) keeps what
        token_logps_backward needs of each row.  As every call here this one
        is no autograd function: logits that require a gradient are read like
        any others and nothing is recorded."""
        x, shape = _logits(logits, "logits", self.device), logits.shape[:-1]
        st = self.lib.muon_token_logps(
            self.handle, _stream(self.device, stream), ctypes.byref(x),
            _tokens(labels, "labels", shape, torch.int64, self.device), temperature,
            _tokens(logps, "logps", shape, torch.float32, self.device),
            _tokens(row_stats, "row_stats", (*shape, 2), torch.float32, self.device))
        self._raise(st, "muon_token_logps")

    def token_logps_backward(self, logits: torch.Tensor, labels: torch.Tensor, row_stats: torch.Tensor,
                             grad_logps: torch.Tensor, grad_logits: torch.Tensor,
                             temperature: float = 1.0, stream=None):
        """Gradient of token_logps into `grad_logits` (the logits' dtype; may
        be the logits themselves, unless autograd saved them for a backward
        pass of its own)."""
        x, shape = _logits(logits, "logits", self.device), logits.shape[:-1]
        gx = self._grad(logits, grad_logits)
        st = self.lib.muon_token_logps_backward(
            self.handle, _stream(self.device, stream), ctypes.byref(x),
            _tokens(labels, "labels", shape, torch.int64, self.device), temperature,
            _tokens(row_stats, "row_stats", (*shape, 2), torch.float32, self.device),
            _tokens(grad_logps, "grad_logps", shape, torch.float32, self.device), ctypes.byref(gx))
        self._raise(st, "muon_token_logps_backward")

    def policy_loss(self, logits: torch.Tensor, labels: torch.Tensor, advantages: torch.Tensor,
                    out: torch.Tensor, old_logps: Optional[torch.Tensor] = None,
                    ref_logps: Optional[torch.Tensor] = None, logps: Optional[torch.Tensor] = None,
                    grad_logits: Optional[torch.Tensor] = None, clip_low: float = 0.2,
                    clip_high: float = 0.2, kl_coef: float = 0.0, reduce: str = "token",
                    weight: float = 1.0, temperature: float = 1.0, stream=None):
        """Clipped policy loss with a KL term, and the gradient of weight *
        loss in the logits (`grad_logits`; None: none is formed; may be the
        logits themselves, as in token_logps_backward); hand it on with
        logits.backward(grad_logits), no graph is recorded here.  advantages: float32, one per sequence ([batch])
        or per token.  old_logps None: the logits' own policy.  out: four
        float32 {weight * loss, policy term, KL, share clipped}.  reduce:
        "token", "sequence" or "sum"."""
        x, shape = _logits(logits, "logits", self.device), logits.shape[:-1]
        gx = self._grad(logits, grad_logits)
        if reduce not in LOSS_REDUCE:
            raise ValueError(f"unknown reduction {reduce!r}; one of {list(LOSS_REDUCE)}")
        # 2-D logits are one sequence of rows
        sequences = (x.batch,)
        per_token = advantages.shape != sequences
        p = PolicyParams(temperature, clip_low, clip_high, kl_coef, weight, LOSS_REDUCE[reduce], 1 if per_token else 0)
        st = self.lib.muon_policy_loss(
            self.handle, _stream(self.device, stream), ctypes.byref(x),
            _tokens(labels, "labels", shape, torch.int64, self.device), ctypes.byref(p),
            _tokens(advantages, "advantages", shape if per_token else sequences, torch.float32, self.device),
            _tokens(old_logps, "old_logps", shape, torch.float32, self.device),
            _tokens(ref_logps, "ref_logps", shape, torch.float32, self.device),
            _tokens(out, "out", (4,), torch.float32, self.device),
            _tokens(logps, "logps", shape, torch.float32, self.device),
            None if gx is None else ctypes.byref(gx))
        self._raise(st, "muon_policy_loss")

    def preference_loss(self, logits: torch.Tensor, labels: torch.Tensor,
                        ref_logps: Optional[torch.Tensor], out: torch.Tensor,
                        rewards: Optional[torch.Tensor] = None, logps: Optional[torch.Tensor] = None,
                        grad_logits: Optional[torch.Tensor] = None, kind: str = "sigmoid",
                        beta: float = 0.1, label_smoothing: float = 0.0, average: bool = False,
                        weight: float = 1.0, temperature: float = 1.0, stream=None):
        """Preference loss over batch / 2 pairs (sequence i was preferred over
        sequence batch / 2 + i), and the gradient of weight * loss in the
        logits.  ref_logps None: no reference.  out: three float32 {weight *
        loss, mean of beta * margin, share of pairs ranked right}.
        grad_logits: as for policy_loss.  rewards:
        float32 [batch], beta times each sequence's score.  kind: "sigmoid" or
        "ipo"; average: scores are means over a sequence's tokens."""
        x, shape = _logits(logits, "logits", self.device), logits.shape[:-1]
        gx = self._grad(logits, grad_logits)
        if kind not in PREFERENCE_KINDS:
            raise ValueError(f"unknown preference loss {kind!r}; one of {list(PREFERENCE_KINDS)}")
        p = PreferenceParams(temperature, beta, label_smoothing, weight, PREFERENCE_KINDS[kind], 1 if average else 0)
        st = self.lib.muon_preference_loss(
            self.handle, _stream(self.device, stream), ctypes.byref(x),
            _tokens(labels, "labels", shape, torch.int64, self.device), ctypes.byref(p),
            _tokens(ref_logps, "ref_logps", shape, torch.float32, self.device),
            _tokens(out, "out", (3,), torch.float32, self.device),
            _tokens(rewards, "rewards", (x.batch,), torch.float32, self.device),
            _tokens(logps, "logps", shape, torch.float32, self.device),
            None if gx is None else ctypes.byref(gx))
        self._raise(st, "muon_preference_loss")

    def _grad(self, logits: torch.Tensor, grad_logits: Optional[torch.Tensor]) -> Optional[Logits]:
        if grad_logits is None:
            return None
        if grad_logits.shape != logits.shape or grad_logits.dtype != logits.dtype:
            raise ValueError("grad_logits must have the logits' shape and dtype")
        return _logits(grad_logits, "grad_logits", self.device)

    # -- linear layers in 8 bits ------------------------------------------------
    def rows8(self, rows: int, cols: int) -> Rows8:
        """Room for 8-bit rows, each at a multiple of 16 bytes."""
        q = torch.empty(rows, (cols + 15) // 16 * 16, dtype=torch.int8, device=self.device)
        return Rows8(q[:, :cols], torch.empty(rows, dtype=torch.float32, device=self.device))

    # (where a pointer is asked for ctypes takes the struct itself, 0.5 us a call
    # faster than its byref)
    def _rows8(self, x: Rows8, name: str):
        if x.device != self.device:
            raise ValueError(f"{name} must be on {self.device}")
        return x.struct

    def quantize_rows(self, x: torch.Tensor, x8: Rows8, stream=None):
        """The rows of x (bf16 or float32, any row stride) in 8 bits with a scale
        each: the largest magnitude becomes 127."""
        r = _rows(x, "x", self.device)
        self._raise(self.lib.muon_quantize_rows(self.handle, _stream(self.device, stream), r,
                                                self._rows8(x8, "x8")), "muon_quantize_rows")

    def dequantize_rows(self, x8: Rows8, out: torch.Tensor, stream=None):
        """The values that 8-bit rows stand for (bf16 or float32)."""
        r = _rows(out, "out", self.device)
        self._raise(self.lib.muon_dequantize_rows(self.handle, _stream(self.device, stream), self._rows8(x8, "x8"),
                                                  r), "muon_dequantize_rows")

    def matmul8(self, a: Rows8, b: Rows8, out: torch.Tensor, stream=None):
        """out = a b^T, summed in integers (bf16 or float32)."""
        r = _rows(out, "out", self.device)
        self._raise(self.lib.muon_matmul8(self.handle, _stream(self.device, stream), self._rows8(a, "a"),
                                          self._rows8(b, "b"), r), "muon_matmul8")

    def linear8(self, x: torch.Tensor, w: Rows8, out: torch.Tensor, x8: Optional[Rows8] = None, stream=None):
        """out = x w^T in 8 bits: x [tokens, k] is quantised by token, w holds a
        row per channel.  `x8` (tokens x k) keeps the quantised activations for
        the backward pass (weight_grad8); None: they are not kept.  As every
        call here no autograd function."""
        r, o = _rows(x, "x", self.device), _rows(out, "out", self.device)
        self._raise(self.lib.muon_linear8(self.handle, _stream(self.device, stream), r, self._rows8(w, "w"),
                                          None if x8 is None else self._rows8(x8, "x8"), o), "muon_linear8")

    def input_grad8(self, grad_y: torch.Tensor, w: Rows8, grad_x: torch.Tensor, accumulate: bool = False, stream=None):
        """Gradient of linear8 in x: grad_x (+)= grad_y w.  grad_y: bf16
        [tokens, n]; grad_x: bf16 or float32."""
        y, o = _rows(grad_y, "grad_y", self.device), _rows(grad_x, "grad_x", self.device)
        self._raise(self.lib.muon_input_grad8(self.handle, _stream(self.device, stream), y, self._rows8(w, "w"),
                                              o, 1 if accumulate else 0), "muon_input_grad8")

    def weight_grad8(self, grad_y: torch.Tensor, x8: Rows8, grad_w: torch.Tensor, accumulate: bool = False, stream=None):
        """Gradient of linear8 in the weights, out of the kept activations:
        grad_w (+)= grad_y^T x8.  grad_w: bf16 or float32 [n, k], e.g. a view of
        MuonStep.grad."""
        y, o = _rows(grad_y, "grad_y", self.device), _rows(grad_w, "grad_w", self.device)
        self._raise(self.lib.muon_weight_grad8(self.handle, _stream(self.device, stream), y,
                                               self._rows8(x8, "x8"), o, 1 if accumulate else 0),
                    "muon_weight_grad8")

    # -- verification of drafted tokens -----------------------------------------
    def verify_draft(self, logits: torch.Tensor, draft_tokens: torch.Tensor, tokens: torch.Tensor,
                     accepted: torch.Tensor, draft_logits: Optional[torch.Tensor] = None,
                     uniforms: Optional[torch.Tensor] = None, logps: Optional[torch.Tensor] = None,
                     temperature: float = 1.0, stream=None):
        """Keeps the drafted tokens that the target's scores allow and takes the
        token behind them.  logits: [batch, draft + 1, vocab]; draft_tokens:
        int64 [batch, draft], a negative one ends a sequence's draft;
        draft_logits: [batch, draft, vocab] that the tokens were sampled from,
        None: a deterministic draft; uniforms: float32 [batch, draft + 1] in
        [0, 1).  tokens (int64 [batch, draft + 1]) receives the kept tokens, the
        one taken, then -1; accepted (int64 [batch]) how many were kept; logps
        (float32 like tokens) their log-probabilities under the target.
        temperature 0: the most likely tokens, uniforms and draft_logits unused."""
        if logits.dim() != 3:
            raise ValueError("logits must be [batch, draft + 1, vocab]")
        x, dev = _logits(logits, "logits", self.device), self.device
        places = logits.shape[:2]
        draft = (places[0], places[1] - 1)
        d = None
        if draft_logits is not None:
            if draft_logits.shape != (*draft, logits.shape[2]):
                raise ValueError("draft_logits must be [batch, draft, vocab]")
            d = _logits(draft_logits, "draft_logits", dev)
        st = self.lib.muon_verify_draft(
            self.handle, _stream(dev, stream), x, _tokens(draft_tokens, "draft_tokens", draft, torch.int64, dev), d,
            _tokens(uniforms, "uniforms", places, torch.float32, dev), temperature,
            _tokens(tokens, "tokens", places, torch.int64, dev), _tokens(accepted, "accepted", places[:1], torch.int64, dev),
            _tokens(logps, "logps", places, torch.float32, dev))
        self._raise(st, "muon_verify_draft")

    # -- gradient norm and clipping -------------------------------------------
    def tensor_list(self, tensors: Sequence[torch.Tensor]) -> TensorList:
        """`tensors` as grad_norm and scale_grads take them, described once
        (those take a plain sequence too and describe it at each call)."""
        return TensorList(tensors, self.device)

    def _list(self, tensors) -> TensorList:
        return tensors if isinstance(tensors, TensorList) else TensorList(tensors, self.device)

    def _norm(self, norm: torch.Tensor) -> int:
        return _tokens(norm, "norm", (3,), torch.float64, self.device)

    def grad_norm(self, grads, norm: torch.Tensor, max_norm: float = float("inf"), eps: float = 1e-6, stream=None):
        """Global norm of a list of tensors: `norm` (float64 [3]) receives the
        sum of squares, its root, and min(1, max_norm / (root + eps))."""
        grads = self._list(grads)
        st = self.lib.muon_grad_norm(self.handle, _stream(self.device, stream), grads.array, len(grads),
                                     max_norm, eps, self._norm(norm))
        self._raise(st, "muon_grad_norm")

    def clip_coef(self, norm: torch.Tensor, max_norm: float, eps: float = 1e-6, stream=None):
        """norm[1:] from norm[0], e.g. after it was summed over ranks."""
        st = self.lib.muon_clip_coef(self.handle, _stream(self.device, stream), max_norm, eps, self._norm(norm))
        self._raise(st, "muon_clip_coef")

    def scale_grads(self, grads, norm: torch.Tensor, out=None, stream=None):
        """grads times the coefficient in `norm`, in place or into the tensors
        `out` (either dtype)."""
        grads = self._list(grads)
        dst = None
        if out is not None:
            out = self._list(out)
            if len(out) != len(grads):
                raise ValueError("out must have one tensor per gradient")
            dst = out.array
        st = self.lib.muon_scale_grads(self.handle, _stream(self.device, stream), grads.array, dst, len(grads),
                                       self._norm(norm))
        self._raise(st, "muon_scale_grads")

    def clip_grads(self, grads, norm: torch.Tensor, max_norm: float, eps: float = 1e-6, out=None, stream=None):
        """grad_norm, then scale_grads."""
        grads = self._list(grads)
        self.grad_norm(grads, norm, max_norm, eps, stream)
        self.scale_grads(grads, norm, out, stream)

    def set_loss_polls(self, polls: int):
        """muon_loss_set_polls: how long a workgroup of policy_loss waits for
        its row's others before it does their part itself."""
        self._raise(self.lib.muon_loss_set_polls(self.handle, polls), "muon_loss_set_polls")

    # -- timing ---------------------------------------------------------------
    def timing_enable(self, enable: bool = True, capacity: int = 8192):
        self._raise(self.lib.muon_timing_enable(self.handle, 1 if enable else 0, capacity), "timing_enable")

    def timing_select(self, classes=None):
        """Time only the named kernel classes (names of timing_read); None: all."""
        names = list(_lib.KERNEL_CLASSES)
        if classes is None:
            mask = (1 << len(names)) - 1
        else:
            mask = 0
            for c in classes:
                if c not in names:
                    raise ValueError(f"unknown kernel class {c!r}; one of {names}")
                mask |= 1 << names.index(c)
        self._raise(self.lib.muon_timing_select(self.handle, mask), "timing_select")

    def timing_reset(self):
        self._raise(self.lib.muon_timing_reset(self.handle), "timing_reset")

    def timing_read(self) -> dict:
        res = {}
        for k, name in enumerate(_lib.KERNEL_CLASSES):
            ms, n = ctypes.c_double(), ctypes.c_int64()
            self._raise(self.lib.muon_timing_read(self.handle, k, ctypes.byref(ms), ctypes.byref(n)),
                        "timing_read")
            res[name] = (ms.value, n.value)
        return res


@dataclass
class BucketInfo:
    m: int
    n: int
    count: int
    units: int
    numel: int
    full_bytes: int
    workspace_bytes: int
    over_cap: bool
    shape_groups: int
    indices: List[int]
    elem_offset: int = 0
    offsets: List[int] = None


class Plan:
    """Host scheduler result: micro-buckets of whole matrices under a cap."""

    def __init__(self, shapes: Sequence[Tuple[int, int, int]], cap_bytes: int, cap_kind: str = "full",
                 compute: str = "bf16", compute_units: int = 0):
        lib = _lib.load()
        arr = (Shape * len(shapes))(*[Shape(r, c, h) for (r, c, h) in shapes])
        h = ctypes.c_void_p()
        kind = MUON_CAP_FULL_BYTES if cap_kind == "full" else MUON_CAP_WORKSPACE
        st = lib.muon_plan_create(arr, len(shapes), int(cap_bytes), kind,
                                  MUON_BF16 if compute == "bf16" else MUON_F32, int(compute_units),
                                  ctypes.byref(h))
        if st != _lib.MUON_OK:
            raise MuonError(st, "muon_plan_create")
        try:
            self.buckets: List[BucketInfo] = []
            for b in range(lib.muon_plan_num_buckets(h)):
                info = _lib.BucketInfo()
                lib.muon_plan_bucket(h, b, ctypes.byref(info), None, None)
                idx = (ctypes.c_int64 * info.count)()
                off = (ctypes.c_int64 * info.count)()
                lib.muon_plan_bucket(h, b, ctypes.byref(info), idx, off)
                self.buckets.append(BucketInfo(info.m, info.n, info.count, info.units, info.numel,
                                               info.full_bytes, info.workspace_bytes,
                                               bool(info.over_cap), info.shape_groups, list(idx),
                                               info.elem_offset, list(off)))
            self.max_workspace = int(lib.muon_plan_max_workspace(h))
            self.total_elems = int(lib.muon_plan_total_elems(h))
        finally:
            lib.muon_plan_destroy(h)
