"""Tensor helpers that choose among the head's logits.

They check and marshal arguments; the work is done by the library's kernels
(cce_top_logits, cce_sample).
"""
from __future__ import annotations

from typing import Optional

import torch

from . import Workspace
from ._distill import Launch, check_head, check_tensor
from ._native import CCEError, CCESampleSettings, cce_head_workspace_size, cce_sample, cce_top_logits


def top_logits(E, C, k: int, workspace: Optional[Workspace] = None, stream=None, out=None):
    """Each token's k largest logits of E C^T in falling order (equal ones:
    lowest id first): values [N, k] fp32, ids [N, k] int64, and lse [N] fp32,
    the log-sum-exp over the vocabulary.  values and ids are what
    distill_forward takes of a teacher.  k is at most 1024 (and V).  The
    scratch holds the logits of min(N, 512) tokens."""
    N, D, V = check_head(E, C)
    if not 0 < k <= min(V, 1024):      # (before anything of its size is allocated)
        raise CCEError(1, f"cce_top_logits: k must be in 1 .. min(V, 1024), not {k}")
    with Launch(E.device, stream, workspace) as run:
        if out is None:
            values, ids = run.empty((N, k), torch.float32), run.empty((N, k), torch.int64)
            lse = run.empty((N,), torch.float32)
        else:
            values, ids, lse = out
            check_tensor(values, "values", (N, k), torch.float32, E.device)
            check_tensor(ids, "ids", (N, k), torch.int64, E.device)
            check_tensor(lse, "lse", (N,), torch.float32, E.device)
        ws = run.scratch(cce_head_workspace_size(N, D, V), "cce_head_workspace_size")
        cce_top_logits(E.data_ptr(), C.data_ptr(), N, D, V, k, values.data_ptr(), ids.data_ptr(), lse.data_ptr(),
                       ws.data_ptr(), ws.numel(), run.ptr)
    return values, ids, lse


def sample(E, C, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, workspace: Optional[Workspace] = None,
           stream=None, out=None):
    """One token per row of hidden states: (token [N] int64, logp [N] fp32).

    u [N] fp32 holds a random number in [0, 1) per row.  temperature (0: the
    largest logit), top_k (0: off), top_p (1: off) and min_p (0: off) are
    numbers, or tensors [N] (top_k int32, the others float32) with one value
    per row.  The filters are applied in that order: the k largest; of these
    the shortest prefix in falling order with at least top_p of their mass; of
    these the ones with at least min_p of the largest one's probability.  The
    token is the first id, in the order of ids, whose cumulated kept mass is
    above u times the whole.  logp is the token's log-probability at the
    row's temperature (1 where that is 0) before the filters; with
    temperature 1 it is -forward(E, C, token)[0].  A row whose largest logit
    is infinite or NaN gets token -1."""
    N, D, V = check_head(E, C)
    check_tensor(u, "u", (N,), torch.float32, E.device)
    settings = CCESampleSettings()
    for name, value, dtype in (("temperature", temperature, torch.float32), ("top_k", top_k, torch.int32),
                               ("top_p", top_p, torch.float32), ("min_p", min_p, torch.float32)):
        if torch.is_tensor(value):
            check_tensor(value, name, (N,), dtype, E.device)
            setattr(settings, name, value.data_ptr())
        else:
            setattr(settings, name + "_all", min(max(int(value), -1), 2 ** 31 - 1) if name == "top_k" else float(value))
    with Launch(E.device, stream, workspace) as run:
        if out is None:
            token, logp = run.empty((N,), torch.int64), run.empty((N,), torch.float32)
        else:
            token, logp = out
            check_tensor(token, "token", (N,), torch.int64, E.device)
            check_tensor(logp, "logp", (N,), torch.float32, E.device)
        ws = run.scratch(cce_head_workspace_size(N, D, V), "cce_head_workspace_size")
        cce_sample(E.data_ptr(), C.data_ptr(), N, D, V, u.data_ptr(), settings, token.data_ptr(), logp.data_ptr(),
                   ws.data_ptr(), ws.numel(), run.ptr)
    return token, logp
