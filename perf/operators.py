"""Measured cases of the operators around the classifier head that answer and distil.

sample        tokens drawn from the head: the logits E C^T of N hidden states, temperature,
              top-k, top-p and min-p, and one given random number per row
top_logits    each row's k largest logits with their ids, and its log-sum-exp (what a teacher
              hands to a student)
distill       forward: KL(teacher's top-K distribution || student's softmax) at a temperature
step          the distillation loss of a batch with the gradients of E and C

Every case holds the sizes; `prepare` makes the tensors a program has in hand, `run` is one
pass, in plain torch operations or (own) through the package.

Inputs of sample and top_logits lie on a binary grid (E on multiples of 2^-5, C on multiples of
2^-11), on which every partial sum of a logit fits in the 24 bits of a float: the logits do not
depend on the order of summation, so the chosen ids can be compared for equality.  Ties among
the logits are frequent on that grid; they go to the lowest id.
"""
import math

import torch

own = False

IGNORE = -100


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # smallest call: one token of a small test model, where the launches count
        dict(name="sample-1-tiny", op="sample", N=1, D=256, V=4096, how="nucleus"),
        # single-stream decoding with the usual chat settings on a 256k vocabulary
        dict(name="sample-1-256k", op="sample", N=1, D=2304, V=256000, how="nucleus"),
        # a serving batch whose requests bring their own settings: greedy, plain, top-k, top-p, min-p
        dict(name="sample-64-mixed", op="sample", N=64, D=4096, V=128256, how="mixed"),
        # rollouts for on-policy training: temperature 1, no filter, an odd batch
        dict(name="sample-193-plain", op="sample", N=193, D=896, V=151936, how="plain"),
        # a teacher scores a short reply
        dict(name="top-37", op="top_logits", N=37, D=2048, V=262144, k=20),
        # a teacher scores a batch of replies for a student with a 256k vocabulary
        dict(name="top-1024", op="top_logits", N=1024, D=2304, V=256000, k=64),
        # evaluation of a distilled small model: odd batch, bf16 teacher logits, soft temperature
        dict(name="distill-300", op="distill", N=300, D=896, V=151936, K=32, T=2.0, t_dtype="bf16"),
        # validation loss on a packed batch
        dict(name="distill-4096", op="distill", N=4096, D=2304, V=256000, K=64, T=1.0, t_dtype="fp32"),
        # a micro-batch of a small test model
        dict(name="step-256-tiny", op="step", N=256, D=256, V=4096, K=8, T=2.0, t_dtype="fp32"),
        # ragged everything: odd vocabulary, odd K, tokens that are not a multiple of a tile
        dict(name="step-1000-ragged", op="step", N=1000, D=2040, V=100003, K=101, T=1.5, t_dtype="bf16"),
        # wide hidden size, few teacher logits
        dict(name="step-2048-wide", op="step", N=2048, D=4096, V=128256, K=20, T=1.0, t_dtype="fp32"),
        # a full training micro-batch on the 256k vocabulary
        dict(name="step-8192-256k", op="step", N=8192, D=2304, V=256000, K=64, T=1.0, t_dtype="fp32"),
    ]


_LARGEST = 8192 * 2304 * 256000


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "top_logits", "distill", "step"])
    D = 8 * _log_int(rng, 16, 512)
    V = _log_int(rng, 4096, 262144)
    # a distillation step does three products of this size
    room = _LARGEST // (D * V) // (1 if op == "step" else 2)
    if op == "sample":
        return dict(op=op, N=_log_int(rng, 1, 256), D=D, V=V, how=rng.choice(["nucleus", "mixed", "plain"]))
    if op == "top_logits":
        return dict(op=op, N=_log_int(rng, 1, 1024), D=D, V=V, k=_log_int(rng, 1, 128))
    return dict(op=op, N=min(_log_int(rng, 1, 8192), room), D=D, V=V, K=_log_int(rng, 1, 128),
                T=rng.choice([1.0, 1.5, 2.0, 4.0]), t_dtype=rng.choice(["fp32", "bf16"]))


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _grid(x, step):
    return (x / step).round_().mul_(step).to(torch.bfloat16)


def _head(g, N, D, V, spread, boost, grid):
    """Hidden states and a classifier whose logits have the standard deviation `spread`, with up to
    eight ids a row whose logits stand out by 0 .. boost."""
    std = spread / math.sqrt(D)
    C = torch.randn(V, D, generator=g, device="cuda", dtype=torch.float32).mul_(std)
    C = _grid(C, 2.0 ** -11) if grid else C.to(torch.bfloat16)
    ids = torch.randint(0, V, (N, 8), generator=g, device="cuda")
    up = torch.rand(N, 8, generator=g, device="cuda").mul_(boost)
    E = torch.randn(N, D, generator=g, device="cuda", dtype=torch.float32)
    for j in range(8):
        E.addcmul_(up[:, j:j + 1], C[ids[:, j]].float(), value=1.0 / (D * std * std))
    E = _grid(E, 2.0 ** -5) if grid else E.to(torch.bfloat16)
    return E, C, ids, up


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 11)
    N, D, V, op = case["N"], case["D"], case["V"], case["op"]
    s = dict(op=op)
    if op in ("sample", "top_logits"):
        # logits of a trained head: a bulk of about 1.5 and a few candidates well above it
        s["E"], s["C"], _, _ = _head(g, N, D, V, 1.5, 18.0, True)
        if op == "top_logits":
            s["k"] = case["k"]
        else:
            one = torch.ones(N, device="cuda")
            s["u"] = torch.rand(N, generator=g, device="cuda")
            how = case["how"]
            kind = torch.arange(N, device="cuda") % 5
            if how == "nucleus":
                s.update(temperature=0.75 * one, top_k=torch.full((N,), 50, dtype=torch.int32, device="cuda"),
                         top_p=0.95 * one, min_p=0 * one)
            elif how == "plain":
                s.update(temperature=one, top_k=torch.zeros(N, dtype=torch.int32, device="cuda"),
                         top_p=one.clone(), min_p=0 * one)
            else:  # rows in turn: greedy, plain, top-k 40, top-p 0.9 at 0.5, min-p 0.05 at 1.25
                s.update(temperature=torch.tensor([0.0, 1.0, 0.875, 0.5, 1.25], device="cuda")[kind],
                         top_k=torch.tensor([0, 0, 40, 0, 0], dtype=torch.int32, device="cuda")[kind],
                         top_p=torch.tensor([1.0, 1.0, 1.0, 0.9, 1.0], device="cuda")[kind],
                         min_p=torch.tensor([0.0, 0.0, 0.0, 0.0, 0.05], device="cuda")[kind])
    else:
        K = case["K"]
        E, C, ids8, up = _head(g, N, D, V, 1.0, 12.0, False)
        # the teacher agrees with the student on some of the ids that stand out
        ids = torch.randint(0, V, (N, K), generator=g, device="cuda")
        n8 = min(8, K)
        ids[:, :n8] = ids8[:, :n8]
        t = torch.rand(N, K, generator=g, device="cuda").mul_(6.0).add_(6.0)
        t[:, :n8] = up[:, :n8] + torch.randn(N, n8, generator=g, device="cuda")
        t, order = t.sort(1, descending=True)
        ids = ids.gather(1, order)
        # short lists: one row in nine ends early, one row in 31 has no target (padding tokens)
        row = torch.arange(N, device="cuda")[:, None]
        at = torch.arange(K, device="cuda")[None, :]
        pad = ((row % 9 == 4) & (at > K // 2)) | (row % 31 == 17)
        ids = torch.where(pad, torch.full_like(ids, IGNORE), ids).contiguous()
        t = torch.where(pad, torch.full_like(t, -math.inf), t)
        t = t.to(torch.bfloat16 if case["t_dtype"] == "bf16" else torch.float32).contiguous()
        s.update(E=E, C=C, ids=ids, t=t, T=float(case["T"]))
    return s


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------

def _plain_sample(E, C, u, temperature, top_k, top_p, min_p):
    """Temperature, then top-k, top-p and min-p in the order of falling logits (ties: lowest id
    first), then the first id, in the order of ids, whose cumulated mass passes u times the whole."""
    z = E.float() @ C.float().t()
    N, V = z.shape
    greedy = temperature <= 0
    tau = torch.where(greedy, torch.ones_like(temperature), temperature).double()[:, None]
    zs, order = z.sort(dim=1, descending=True, stable=True)
    x = z.double() / tau
    xs = zs.double() / tau
    lse = xs[:, 0] + (x - xs[:, :1]).exp().sum(1).log()
    mass = (xs - xs[:, :1]).exp()
    rank = torch.arange(V, device=z.device)[None, :]
    k = torch.where(top_k <= 0, torch.full_like(top_k, V), top_k)[:, None]
    k = torch.where(greedy[:, None], torch.ones_like(k), k)
    keep = rank < k
    mass_k = mass * keep
    before = mass_k.cumsum(1) - mass_k
    p = top_p.double()[:, None]
    keep &= (p >= 1) | (before < p * mass_k.sum(1, keepdim=True)) | (rank == 0)
    keep &= mass >= min_p.double()[:, None]
    kept = torch.zeros_like(mass).scatter_(1, order, mass * keep)
    total = kept.cumsum(1)
    token = (total <= u.double()[:, None] * total[:, -1:]).sum(1)
    # u so near 1 that rounding leaves nothing above it: the last kept id
    last = torch.where(kept > 0, torch.arange(V, device=z.device)[None, :], torch.zeros_like(order)).amax(1)
    token = torch.minimum(token, last)
    logp = x.gather(1, token[:, None])[:, 0] - lse
    return token, logp.float()


def _plain_top(E, C, k):
    z = E.float() @ C.float().t()
    zs, order = z.sort(dim=1, descending=True, stable=True)
    lse = zs[:, 0].double() + (z.double() - zs[:, :1].double()).exp().sum(1).log()
    return zs[:, :k].contiguous(), order[:, :k].contiguous(), lse.float()


def _targets(ids, t, T):
    """The teacher's distribution over its valid entries (0 elsewhere), ids safe to index with, and
    which rows have any target."""
    live = (ids != IGNORE) & (t > -math.inf)
    x = torch.where(live, t.double() / T, torch.full_like(t, -math.inf, dtype=torch.float64))
    top = x.amax(1, keepdim=True)
    has = top[:, 0] > -math.inf
    w = (x - torch.where(has[:, None], top, torch.zeros_like(top))).exp()
    total = w.sum(1, keepdim=True)
    p = w / torch.where(has[:, None], total, torch.ones_like(total))
    return p, torch.where(live, ids, torch.zeros_like(ids)), has


def _plain_distill(E, C, ids, t, T):
    z = (E.float() @ C.float().t()).div_(T)
    p, at, has = _targets(ids, t, T)
    top = z.amax(1, keepdim=True)
    picked = z.gather(1, at).double()
    lse = top[:, 0].double() + (z.sub_(top)).exp_().sum(1, dtype=torch.float64).log()
    logp = torch.where(p > 0, p, torch.ones_like(p)).log()
    loss = T * T * (p * (logp - picked + lse[:, None])).sum(1)
    return torch.where(has, loss, torch.zeros_like(loss)).float(), lse.float()


def _plain_step(E, C, ids, t, T):
    Ef, Cf = E.float(), C.float()
    z = (Ef @ Cf.t()).div_(T)
    p, at, has = _targets(ids, t, T)
    top = z.amax(1, keepdim=True)
    picked = z.gather(1, at).double()
    z.sub_(top).exp_()
    total = z.sum(1, keepdim=True, dtype=torch.float64)
    lse = top.double() + total.log()
    logp = torch.where(p > 0, p, torch.ones_like(p)).log()
    loss = T * T * (p * (logp - picked + lse)).sum(1)
    n = has.sum()
    mean = torch.where(has, loss, torch.zeros_like(loss)).sum() / n
    # G = dloss T (softmax - p), dloss = 1 / n on the rows with a target
    scale = (has.double() * (T / n))[:, None]
    z.mul_((scale / total).float())
    z.scatter_add_(1, at, (-scale * p).float())
    return mean.float(), (z @ Cf).to(E.dtype), (z.t() @ Ef).to(C.dtype)


def run(s):
    op = s["op"]
    if own:
        import linear_cross_entropy_05_b200 as L
        if op == "sample":
            return L.sample(s["E"], s["C"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                            min_p=s["min_p"])
        if op == "top_logits":
            return L.top_logits(s["E"], s["C"], s["k"])
        if op == "distill":
            return L.distill_forward(s["E"], s["C"], s["ids"], s["t"], temperature=s["T"])
        E, C = s["E"].detach().requires_grad_(), s["C"].detach().requires_grad_()
        loss = L.linear_distillation(E, C, s["ids"], s["t"], temperature=s["T"])
        dE, dC = torch.autograd.grad(loss, (E, C))
        return loss.detach(), dE, dC
    if op == "sample":
        return _plain_sample(s["E"], s["C"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])
    if op == "top_logits":
        return _plain_top(s["E"], s["C"], s["k"])
    if op == "distill":
        return _plain_distill(s["E"], s["C"], s["ids"], s["t"], s["T"])
    return _plain_step(s["E"], s["C"], s["ids"], s["t"], s["T"])


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    N, D, V, op = case["N"], case["D"], case["V"], case["op"]
    head = 2 * (N * D + V * D)
    if op == "sample":
        return dict(bytes=head + N * (4 * 5 + 12), flops=2 * N * D * V)
    if op == "top_logits":
        return dict(bytes=head + N * (12 * case["k"] + 4), flops=2 * N * D * V)
    teacher = N * case["K"] * (8 + (2 if case["t_dtype"] == "bf16" else 4))
    if op == "distill":
        return dict(bytes=head + teacher + 8 * N, flops=2 * N * D * V)
    # logits, dE and dC: three products (the logits again in the backward are this path's choice)
    return dict(bytes=2 * head + teacher + 4, flops=6 * N * D * V)


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

def _exact_row_token(z, u, tau, k, p, m):
    """One row of numpy doubles: the chosen id and its log-probability."""
    import numpy as np
    if tau <= 0:
        x = z
        token = int(np.argmax(z))
    else:
        x = z / tau
        order = np.lexsort((np.arange(z.size), -z))
        w = np.exp(x[order] - x[order[0]])
        count = z.size if k <= 0 else min(k, z.size)
        w = w[:count]
        if p < 1:
            count = max(1, int(np.searchsorted(np.cumsum(w), p * w.sum(), side="left")) + 1)
            w = w[:count]
        count = min(count, int((w >= m).sum()))
        ids = np.sort(order[:count])
        c = np.cumsum(np.exp(x[ids] - x[order[0]]))
        token = int(ids[min(count - 1, int(np.searchsorted(c, u * c[-1], side="right")))])
    top = x.max()
    return token, float(x[token] - top - np.log(np.exp(x - top).sum()))


def exact(case, seed):
    s = prepare(case, seed)
    E, C = s["E"].double(), s["C"].double()
    op = s["op"]
    if op == "sample":
        z = (E @ C.T).cpu().numpy()
        cols = [s[n].double().cpu().numpy() for n in ("u", "temperature", "top_k", "top_p", "min_p")]
        rows = [_exact_row_token(z[i], cols[0][i], cols[1][i], int(cols[2][i]), cols[3][i], cols[4][i])
                for i in range(z.shape[0])]
        return None, torch.tensor([r[1] for r in rows], dtype=torch.float64)
    if op == "top_logits":
        values, lse = [], []
        for at in range(0, E.shape[0], 256):
            z = E[at:at + 256] @ C.T
            values.append(torch.topk(z, s["k"], dim=1).values)
            lse.append(torch.logsumexp(z, 1))
        return torch.cat(values), None, torch.cat(lse)
    T, N, K = s["T"], E.shape[0], s["ids"].shape[1]
    loss = torch.zeros(N, dtype=torch.float64, device=E.device)
    lse = torch.zeros_like(loss)
    count = int(((s["ids"] != IGNORE) & (s["t"].double() != -math.inf)).any(1).sum())
    dE, dC = torch.zeros_like(E), torch.zeros_like(C)
    for at in range(0, N, 1024):
        rows = slice(at, min(N, at + 1024))
        n = rows.stop - at
        logq = torch.log_softmax(E[rows] @ C.T / T, 1)
        z0 = E[rows] @ C[0]
        lse[rows] = z0 / T - logq[:, 0]
        gone = s["ids"][rows] == IGNORE
        teacher = s["t"][rows].double().masked_fill(gone, -math.inf) / T
        empty = torch.isinf(teacher).all(1)
        p = torch.softmax(teacher, 1).masked_fill(empty[:, None], 0.0)
        dense = torch.zeros_like(logq)  # the teacher's distribution over the whole vocabulary
        flat = torch.arange(n, device=E.device)[:, None].expand(n, K)
        dense.index_put_((flat[~gone], s["ids"][rows][~gone]), p[~gone], accumulate=True)
        plogp = torch.special.xlogy(p, p).sum(1)
        loss[rows] = T * T * (plogp - (dense * logq).sum(1))
        if op == "step":
            grad = (logq.exp_().masked_fill_(empty[:, None], 0.0) - dense) * (T / count)
            dE[rows] = grad @ C
            dC += grad.T @ E[rows]
    if op == "distill":
        return loss, lse
    return loss.sum() / count, dE, dC
