"""Tensor helpers of the distillation loss on a teacher's top logits.

They check and marshal arguments; the loss and its gradients run in the
library's kernels (cce_distill_forward, cce_distill_backward).
"""
from __future__ import annotations

from typing import Optional

import torch

from . import IGNORE_INDEX, Workspace
from ._native import (CCE_BWD_ACCUMULATE, CCE_BWD_BF16_GRADS, CCE_BWD_DETERMINISTIC, CCE_DTYPE_BF16, CCE_DTYPE_F32,
                      CCEError, cce_distill_backward, cce_distill_backward_workspace_size, cce_distill_forward,
                      cce_distill_forward_workspace_size)


def check_head(E, C):
    """E [N, D] and C [V, D]: contiguous CUDA bfloat16 matrices on one device."""
    if E.dtype != torch.bfloat16 or C.dtype != torch.bfloat16:
        raise TypeError("E and C must be torch.bfloat16")
    if E.dim() != 2 or C.dim() != 2 or E.shape[1] != C.shape[1]:
        raise ValueError("shapes must be E [N, D], C [V, D]")
    for t, n in ((E, "E"), (C, "C")):
        check_tensor(t, n, t.shape, torch.bfloat16, E.device)
    return E.shape[0], E.shape[1], C.shape[0]


def check_tensor(t, name, shape, dtype, device):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a contiguous CUDA tensor of shape {list(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, E on {device}")


class Launch:
    """Device, stream and scratch of one call: the tensors' device is made
    current, and what the call allocates is kept from reuse until `stream`
    has passed it when that is not the allocating stream."""

    __slots__ = ("device", "workspace", "stream", "foreign", "guard")

    def __init__(self, device, stream, workspace: Optional[Workspace]):
        self.device = device
        self.workspace = workspace or Workspace(device)
        self.stream = stream
        self.guard = None

    def __enter__(self):
        if self.device.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(self.device)
            self.guard.__enter__()
        current = torch.cuda.current_stream(self.device)
        if self.stream is None:
            self.stream = current
        self.foreign = self.stream != current
        return self

    def __exit__(self, *exc):
        return self.guard.__exit__(*exc) if self.guard is not None else None

    @property
    def ptr(self) -> int:
        return int(self.stream.cuda_stream)

    def empty(self, shape, dtype):
        t = torch.empty(shape, dtype=dtype, device=self.device)
        if self.foreign:
            t.record_stream(self.stream)
        return t

    def scratch(self, nbytes: int, what: str):
        if nbytes == 0:
            raise CCEError(1, f"{what}: invalid sizes or no sm_100 device")
        buf = self.workspace.get(nbytes)
        if buf.device != self.device:
            raise ValueError(f"the workspace is on {buf.device}, E on {self.device}")
        if self.foreign:
            buf.record_stream(self.stream)
        return buf


def _check_targets(ids, teacher, N, device):
    if ids.dim() != 2:
        raise ValueError("ids must be [N, K]")
    check_tensor(ids, "ids", (N, ids.shape[1]), torch.int64, device)
    if teacher.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("teacher must be torch.float32 or torch.bfloat16")
    check_tensor(teacher, "teacher", ids.shape, teacher.dtype, device)
    return ids.shape[1], (CCE_DTYPE_BF16 if teacher.dtype == torch.bfloat16 else CCE_DTYPE_F32)


def distill_forward(E, C, ids, teacher, temperature: float = 1.0, ignore_index: int = IGNORE_INDEX,
                    workspace: Optional[Workspace] = None, stream=None, out=None, mean=None):
    """Per-token distillation loss and log-sum-exp (fp32 [N]).

    ids [N, K] int64 and teacher [N, K] (float32 or bfloat16) hold a teacher's
    top logits, e.g. from top_logits; entries whose id is ignore_index or
    whose logit is -inf are absent, and a row without entries has loss 0.
    With p the softmax of a row's teacher logits over its entries at
    `temperature` T and q the student's softmax of E C^T / T over all of the
    vocabulary, loss = T^2 sum_k p_k log(p_k / q_{ids_k}).  lse is the
    log-sum-exp of the logits divided by T, which distill_backward needs.  T is
    from 1e-3 to 1e6.
    mean: optionally two fp32 scalar tensors that receive the mean loss over
    the rows with an entry and one over their number."""
    N, D, V = check_head(E, C)
    K, dtype = _check_targets(ids, teacher, N, E.device)
    with Launch(E.device, stream, workspace) as run:
        if out is None:
            loss, lse = run.empty((N,), torch.float32), run.empty((N,), torch.float32)
        else:
            loss, lse = out
            check_tensor(loss, "loss", (N,), torch.float32, E.device)
            check_tensor(lse, "lse", (N,), torch.float32, E.device)
        means = (0, 0)
        if mean is not None:
            for t in mean:
                check_tensor(t, "mean", (), torch.float32, E.device)
            means = (mean[0].data_ptr(), mean[1].data_ptr())
        ws = run.scratch(cce_distill_forward_workspace_size(N, D, V, K), "cce_distill_forward_workspace_size")
        cce_distill_forward(E.data_ptr(), C.data_ptr(), ids.data_ptr(), teacher.data_ptr(), dtype, N, D, V, K,
                            ignore_index, float(temperature), loss.data_ptr(), lse.data_ptr(), *means,
                            ws.data_ptr(), ws.numel(), run.ptr)
    return loss, lse


def distill_backward(E, C, ids, teacher, lse, dloss, temperature: float = 1.0, ignore_index: int = IGNORE_INDEX,
                     workspace: Optional[Workspace] = None, stream=None, out=None, deterministic: bool = False,
                     bf16_grads: bool = False, accumulate: bool = False, dloss_scale=None):
    """dE [N, D] and dC [V, D] of sum_i dloss[i] * loss[i] for the loss of
    distill_forward (every entry of the softmax's gradient; no filter): fp32,
    or bf16 with bf16_grads.  dloss is [N], or a scalar tensor for all rows;
    dloss_scale, a scalar tensor, multiplies it (with distill_forward's second
    mean: the gradient of dloss times the mean).  deterministic=True sums dE in
    a fixed order (linear_distillation does); accumulate=True adds to the tensors given in `out`
    (required).  The
    logits are formed again on chip; the scratch is 24 KB per token (of at most
    16384) or, for few tokens, up to 128 MB, a copy of E, and the fp32 sums of
    dE for bf16 outputs (and of dC with accumulate or more than 16384 tokens);
    with deterministic and few tokens, up to 39 MB of parts of dE.
    What E, lse and dloss hold for a row without entries is not looked at."""
    N, D, V = check_head(E, C)
    K, dtype = _check_targets(ids, teacher, N, E.device)
    check_tensor(lse, "lse", (N,), torch.float32, E.device)
    check_tensor(dloss, "dloss", (N,) if dloss.dim() else (), torch.float32, E.device)
    if dloss_scale is not None:
        check_tensor(dloss_scale, "dloss_scale", (), torch.float32, E.device)
    if accumulate and out is None:
        raise ValueError("accumulate=True adds into existing gradients: pass them as out=(dE, dC)")
    flags = ((CCE_BWD_DETERMINISTIC if deterministic else 0) | (CCE_BWD_BF16_GRADS if bf16_grads else 0) |
             (CCE_BWD_ACCUMULATE if accumulate else 0))
    gdt = torch.bfloat16 if bf16_grads else torch.float32
    with Launch(E.device, stream, workspace) as run:
        if out is None:
            dE, dC = run.empty((N, D), gdt), run.empty((V, D), gdt)
        else:
            dE, dC = out
            check_tensor(dE, "dE", (N, D), gdt, E.device)
            check_tensor(dC, "dC", (V, D), gdt, E.device)
        ws = run.scratch(cce_distill_backward_workspace_size(N, D, V, K, flags), "cce_distill_backward_workspace_size")
        cce_distill_backward(E.data_ptr(), C.data_ptr(), ids.data_ptr(), teacher.data_ptr(), dtype, lse.data_ptr(),
                             dloss.data_ptr(), 1 if dloss.dim() else 0,
                             0 if dloss_scale is None else dloss_scale.data_ptr(), N, D, V, K, ignore_index,
                             float(temperature), flags, dE.data_ptr(), dC.data_ptr(), ws.data_ptr(), ws.numel(),
                             run.ptr)
    return dE, dC
