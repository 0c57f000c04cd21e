"""Distillation from a teacher's top logits on the GPU against the fp64
definition, at the sizes, masks and orders where it can go wrong."""
import numpy as np
import pytest

import oracle

from _gpu_helpers import IGN

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24   # half a step of fp32, relative
U16 = 2.0 ** -8    # half a step of bf16, relative


def make(seed, N, D, V, K, t_dtype="fp32", spread=2.0):
    """Device tensors and the same values as fp64 arrays."""
    import torch
    g = torch.Generator().manual_seed(seed)
    E = torch.randn(N, D, generator=g).to(torch.bfloat16)
    C = (torch.randn(V, D, generator=g) * (spread / D ** 0.5)).to(torch.bfloat16)
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(N)]) if V >= K else \
        torch.randint(0, V, (N, K), generator=g)
    t = torch.randn(N, K, generator=g) * 3
    t = t.to(torch.bfloat16 if t_dtype == "bf16" else torch.float32)
    return E, C, ids, t, torch.rand(N, generator=g) + 0.5


def mask(ids, t):
    """Short rows, -inf entries, rows without any entry, values behind masked ids, duplicates."""
    N, K = ids.shape
    if N > 3:
        ids[1, K // 2:] = IGN
        t[1, K // 2:] = float("nan")          # behind ignore_index: never looked at
        ids[2] = IGN                           # no entry
        t[2, :] = float("inf")
        t[3, 0] = float("-inf")                # absent, and its id is not looked at
        ids[3, 0] = 1 << 40
    if N > 5:
        ids[4, -1] = ids[4, 0]                 # the same id twice (thrice with K = 1: one entry)
        t[5] = float("-inf")                   # no entry
    return ids, t


def f64(x):
    return x.double().numpy()


def reference(E, C, ids, t, T, dl=None):
    ids, t = ids.numpy().copy(), f64(t)
    ids[t == -np.inf] = IGN
    t = np.where(ids == IGN, -np.inf, t)
    return oracle.distill(f64(E), f64(C), ids, t, T, IGN, None if dl is None else f64(dl))


def forward_bound(E, C, T, K):
    """Largest error of (loss, lse) by rounding.  A logit is D products summed
    in fp32, K = 16 at a time: (D / 16 + 1) additions, each off by at most one
    step (2 U32) of the sum of magnitudes.  exp2's argument is rounded (the
    shift and the product: 2 U32 of the largest |z / T|, twice) and exp2, the
    running sums (rescaled once a tile: under 64 steps) and the final
    logarithm are off by a few steps of 1; the weights by U32 each."""
    S = np.abs(f64(E)) @ np.abs(f64(C)).T
    dz = (E.shape[1] / 16 + 1) * 2 * U32 * S.max(axis=1) / T
    zmax = np.abs(f64(E) @ f64(C).T).max(axis=1) / T
    dlse = dz + 8 * U32 * zmax + 96 * U32 + 2 * U32 * (zmax + 12)
    dloss = T * T * (dz + dlse + (K + 4) * U32 * (zmax + 1) + U32 * (zmax + 24))
    return dloss + 1e-30, dlse


SHAPES = [
    (1, 8, 1, 1), (1, 64, 300, 5), (2, 2304, 700, 3), (3, 264, 4173, 1), (257, 136, 1000, 33), (300, 256, 5000, 128),
    (7, 96, 1500, 1024), (130, 896, 3001, 1000), (520, 128, 257, 200),
]


@pytest.mark.parametrize("T", [0.5, 1.0, 4.0])
@pytest.mark.parametrize("N,D,V,K", SHAPES)
def test_forward_and_backward_match_the_definition(N, D, V, K, T):
    import torch
    import linear_cross_entropy_05_b200 as L
    t_dtype = "bf16" if (K + N) % 2 else "fp32"
    E, C, ids, t, dl = make(N + D + V + K, N, D, V, K, t_dtype)
    ids, t = mask(ids, t)
    loss, lse, dE, dC, G = reference(E, C, ids, t, T, dl)
    dev = [x.cuda() for x in (E, C, ids, t)]
    ws = L.Workspace("cuda")
    got_loss, got_lse = L.distill_forward(*dev, temperature=T, workspace=ws)
    st = L.read_status(ws)
    assert st["status"] == 0, st
    bl, bs = forward_bound(E, C, T, K)
    assert (np.abs(got_lse.double().cpu().numpy() - lse) <= bs).all()
    assert (np.abs(got_loss.double().cpu().numpy() - loss) <= bl).all()
    # G is rounded to bf16 (U16); its softmax carries the logits' and the
    # log-sum-exp's error, e = exp(.) (1 + d), d <= dz + dlse
    q = np.abs(G) + 0.0
    d = (2 * bs.max() + 16 * U32)
    P = np.abs(f64(dl)[:, None] * T * np.exp(f64(E) @ f64(C).T / T - lse[:, None]))
    dG = (U16 + 4 * U32) * q + d * P * 1.01
    for bf16 in (False, True):
        gE, gC = L.distill_backward(*dev, got_lse, dl.cuda(), temperature=T, bf16_grads=bf16, workspace=ws)
        st = L.read_status(ws)
        assert st["status"] == 0, st
        for got, want, bound in ((gE, dE, dG @ np.abs(f64(C))), (gC, dC, dG.T @ np.abs(f64(E)))):
            n_sum = max(N, V)
            bound = bound + (n_sum / 16 + 64) * 2 * U32 * (bound / U16) + (1.01 * U16 * np.abs(want) if bf16 else 0)
            assert got.dtype == (torch.bfloat16 if bf16 else torch.float32)
            err = np.abs(got.double().cpu().numpy() - want)
            assert (err <= bound + 1e-30).all(), (err.max(), bound.max())


def test_ids_on_tile_borders_in_any_order():
    import linear_cross_entropy_05_b200 as L
    N, D, V = 40, 64, 2051
    E, C, _, _, dl = make(5, N, D, V, 4)
    import torch
    borders = [0, 31, 32, 127, 128, 255, 256, 511, 512, 2047, 2048, 2050]
    g = torch.Generator().manual_seed(6)
    ids = torch.stack([torch.tensor(borders)[torch.randperm(len(borders), generator=g)] for _ in range(N)])
    t = torch.randn(N, len(borders), generator=g)
    loss, lse, dE, dC, G = reference(E, C, ids, t, 1.0, dl)
    dev = [x.cuda() for x in (E, C, ids, t)]
    got, gl = L.distill_forward(*dev)
    bl, _ = forward_bound(E, C, 1.0, len(borders))
    assert (np.abs(got.double().cpu().numpy() - loss) <= bl).all()
    gE, gC = L.distill_backward(*dev, gl, dl.cuda())
    for a, b in ((gE, dE), (gC, dC)):
        assert np.linalg.norm(a.double().cpu().numpy() - b) <= U16 * np.linalg.norm(b)


def test_bad_entries_make_their_row_nan_and_leave_the_others():
    import torch
    import linear_cross_entropy_05_b200 as L
    N, D, V, K = 9, 72, 600, 6
    E, C, ids, t, dl = make(11, N, D, V, K)
    keep = [i for i in range(N) if i not in (2, 4, 6, 7)]
    loss, lse, dE, dC, _ = reference(E, C, ids, t, 2.0, dl * torch.tensor([float(i in keep) for i in range(N)]))
    ids[2, 3] = V            # outside the vocabulary
    ids[4, 0] = -1
    t[6, 1] = float("nan")
    t[7, 5] = float("inf")
    dev = [x.cuda() for x in (E, C, ids, t)]
    ws = L.Workspace("cuda")
    got, gl = L.distill_forward(*dev, temperature=2.0, workspace=ws)
    st = L.read_status(ws)
    assert st["status"] == 7 and st["flags"] == 2
    got = got.cpu().numpy()
    assert np.isnan(got[[2, 4, 6, 7]]).all() and np.allclose(got[keep], loss[keep], rtol=1e-5, atol=1e-5)
    assert np.allclose(gl.cpu().numpy(), lse, rtol=1e-5)
    gE, gC = L.distill_backward(*dev, gl, dl.cuda(), temperature=2.0, workspace=ws)
    assert L.read_status(ws)["status"] == 7
    assert (gE[[2, 4, 6, 7]] == 0).all()
    for a, b in ((gE, dE), (gC, dC)):
        assert np.linalg.norm(a.double().cpu().numpy() - b) <= U16 * np.linalg.norm(b)


@pytest.mark.parametrize("bf16", [False, True])
def test_deterministic_accumulate_and_several_launches(bf16):
    import torch
    import linear_cross_entropy_05_b200 as L
    N, D, V, K = 700, 264, 9001, 17
    E, C, ids, t, dl = make(21, N, D, V, K)
    ids, t = mask(ids, t)
    _, _, dE, dC, _ = reference(E, C, ids, t, 1.0, dl)
    dev = [x.cuda() for x in (E, C, ids, t)]
    _, lse = L.distill_forward(*dev)
    kw = dict(bf16_grads=bf16)
    one = L.distill_backward(*dev, lse, dl.cuda(), deterministic=True, **kw)
    for _ in range(3):
        two = L.distill_backward(*dev, lse, dl.cuda(), deterministic=True, **kw)
        assert all(torch.equal(a, b) for a, b in zip(one, two))
    # bf16 sums: dE's and dC's rounding, then the sum's
    tol = U16 if not bf16 else 3 * U16
    base = [torch.ones_like(g) for g in one]
    acc = L.distill_backward(*dev, lse, dl.cuda(), accumulate=True, out=tuple(base), **kw)
    for a, b in zip(acc, (dE, dC)):
        assert np.linalg.norm(a.double().cpu().numpy() - (b + 1)) <= tol * np.linalg.norm(b + 1)
    L.cce_debug_set_stripe_params(tokens_per_launch=256)   # three launches, dC added to
    try:
        more = L.distill_backward(*dev, lse, dl.cuda(), **kw)
    finally:
        L.cce_debug_set_stripe_params()
    for a, b in zip(more, (dE, dC)):
        assert np.linalg.norm(a.double().cpu().numpy() - b) <= tol * np.linalg.norm(b)


def test_autograd_mean_over_rows_with_a_target():
    import torch
    import linear_cross_entropy_05_b200 as L
    N, D, V, K = 65, 128, 3001, 9
    E, C, ids, t, _ = make(31, N, D, V, K, "bf16")
    ids, t = mask(ids, t)
    has = oracle.distill_targets(np.where(f64(t) == -np.inf, IGN, ids.numpy()), f64(t), 1.5, IGN)[1]
    n = int(has.sum())
    assert n == N - 2
    dl = torch.full((N,), 3.0 / n)
    loss, _, dE, dC, _ = reference(E, C, ids, t, 1.5, dl)
    Eg, Cg = E.cuda().requires_grad_(), C.cuda().requires_grad_()
    out = L.linear_distillation(Eg, Cg, ids.cuda(), t.cuda(), temperature=1.5)
    assert abs(out.item() - loss.sum() / n) <= 1e-5 * abs(loss.sum() / n)
    (3 * out).backward()
    for g, b in ((Eg.grad, dE), (Cg.grad, dC)):
        assert g.dtype == torch.bfloat16
        assert np.linalg.norm(g.double().cpu().numpy() - b) <= 2 * U16 * np.linalg.norm(b)
    # a frozen head
    E2 = E.cuda().requires_grad_()
    L.linear_distillation(E2, C.cuda(), ids.cuda(), t.cuda(), temperature=1.5).backward()
    assert np.linalg.norm(E2.grad.double().cpu().numpy() - dE / 3) <= 2 * U16 * np.linalg.norm(dE / 3)


def test_means_and_one_dloss_for_all_rows():
    import torch
    import linear_cross_entropy_05_b200 as L
    for N, V in ((1, 50), (33, 300), (2100, 777)):
        E, C, ids, t, _ = [x.cuda() for x in make(N, N, 64, V, 7)]
        if N > 1:
            ids[::3] = IGN
        mean, inv = torch.zeros((), device="cuda"), torch.zeros((), device="cuda")
        loss, lse = L.distill_forward(E, C, ids, t, mean=(mean, inv))
        kept = (ids != IGN).any(1)
        n = int(kept.sum())
        # one rounding each of a double sum
        assert inv.item() == float(np.float32(1.0 / n))
        want = loss.double()[kept].sum().item() / n
        assert abs(mean.item() - want) <= 1.01 * U32 * abs(want) + 1e-12
        a = L.distill_backward(E, C, ids, t, lse, torch.tensor(0.7, device="cuda"), dloss_scale=inv, deterministic=True)
        b = L.distill_backward(E, C, ids, t, lse, (0.7 * inv).expand(N).contiguous(), deterministic=True)
        for p, q in zip(a, b):   # the factors are multiplied in another order: a last bit of G
            assert (p - q).norm() <= U16 * q.norm()
    ids[:] = IGN
    E.requires_grad_()
    out = L.linear_distillation(E, C, ids, t)
    out.backward()
    assert torch.isnan(out) and (E.grad == 0).all()


def test_one_entry_at_temperature_one_is_the_cross_entropy():
    import torch
    import linear_cross_entropy_05_b200 as L
    N, D, V = 300, 264, 9001
    E, C, ids, t, dl = make(41, N, D, V, 1)
    ids[7] = IGN
    y = ids[:, 0].contiguous()
    dev = [x.cuda() for x in (E, C)]
    loss, lse = L.distill_forward(*dev, ids.cuda(), t.cuda())
    ref, ref_lse = L.forward(*dev, y.cuda())
    assert torch.allclose(loss, ref, rtol=0, atol=4e-6) and torch.allclose(lse, ref_lse, rtol=0, atol=4e-6)
    a = L.distill_backward(*dev, ids.cuda(), t.cuda(), lse, dl.cuda())
    b = L.backward(*dev, y.cuda(), ref_lse, dl.cuda())
    for p, q in zip(a, b):
        assert (p - q).norm() <= U16 * q.norm()


def test_other_streams_graphs_and_two_calls_at_once():
    import torch
    import linear_cross_entropy_05_b200 as L
    N, D, V, K = 300, 256, 5000, 20
    sets = []
    for seed in (51, 52):
        E, C, ids, t, dl = [x.cuda() for x in make(seed, N, D, V, K)]
        loss, lse = L.distill_forward(E, C, ids, t)
        sets.append(((E, C, ids, t), dl, loss, lse, L.distill_backward(E, C, ids, t, lse, dl, deterministic=True)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for (args, dl, _, lse, _), s in zip(sets, streams):       # both at once, through stream=
        s.wait_stream(torch.cuda.current_stream())
        loss, l2 = L.distill_forward(*args, stream=s)
        outs.append((loss, l2) + tuple(L.distill_backward(*args, l2, dl, deterministic=True, stream=s)))
    torch.cuda.synchronize()
    for (args, dl, loss, lse, grads), got in zip(sets, outs):
        assert torch.equal(got[0], loss) and torch.equal(got[1], lse)
        assert torch.equal(got[2], grads[0]) and torch.equal(got[3], grads[1])
    # captured once, replayed on other inputs
    (args, dl, _, _, _) = sets[0]
    held = [x.clone() for x in args]
    hdl = dl.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, lse = L.distill_forward(*held)
        gE, gC = L.distill_backward(*held, lse, hdl, deterministic=True)
    for args, dl, want, wlse, grads in reversed(sets):
        for h, a in zip(held, args):
            h.copy_(a)
        hdl.copy_(dl)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want) and torch.equal(gE, grads[0]) and torch.equal(gC, grads[1])


@pytest.mark.parametrize("D", [256, 1032])
def test_a_wait_that_gives_up_yields_nan(D):
    import torch
    import linear_cross_entropy_05_b200 as L
    E, C, ids, t, dl = [x.cuda() for x in make(61, 300, D, 5000, 20)]
    ws = L.Workspace("cuda")
    L.cce_debug_set_wait_limit_ns(20_000_000)
    L.cce_debug_withhold_loads(True)
    try:
        loss, lse = L.distill_forward(E, C, ids, t, workspace=ws)
        torch.cuda.synchronize()
    finally:
        L.cce_debug_withhold_loads(False)
        L.cce_debug_set_wait_limit_ns(1_000_000_000)
    assert L.read_status(ws)["status"] == 6
    assert torch.isnan(loss).all() and torch.isnan(lse).all()
    loss, _ = L.distill_forward(E, C, ids, t, workspace=ws)
    assert torch.isfinite(loss).all()


def test_refusals():
    import torch
    import linear_cross_entropy_05_b200 as L
    E, C, ids, t, dl = [x.cuda() for x in make(71, 20, 64, 300, 4)]
    with pytest.raises(TypeError):
        L.distill_forward(E.float(), C, ids, t)
    with pytest.raises(TypeError):
        L.distill_forward(E, C, ids.int(), t)
    with pytest.raises(TypeError):
        L.distill_forward(E, C, ids, t.half())
    with pytest.raises(ValueError):
        L.distill_forward(E, C, ids[:, :3], t)
    with pytest.raises(ValueError):
        L.distill_forward(E, C, ids, t.t().contiguous().t())   # not contiguous
    with pytest.raises(ValueError):
        L.distill_forward(E, C, ids.cpu(), t)
    for T in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(L.CCEError):
            L.distill_forward(E, C, ids, t, temperature=T)
    many = torch.zeros(20, 1025, device="cuda")
    with pytest.raises(L.CCEError):
        L.distill_forward(E, C, many.long(), many)
    with pytest.raises(ValueError):
        L.distill_backward(E, C, ids, t, dl, dl, accumulate=True)
    with pytest.raises(L.CCEError):
        L.distill_forward(E[:0], C, ids[:0], t[:0])


@pytest.mark.parametrize("bf16", [False, True])
def test_rows_without_a_gradient_may_hold_anything(bf16):
    """NaN and inf in E, lse and dloss of padded and of bad rows reach nothing."""
    import torch
    import linear_cross_entropy_05_b200 as L
    N, D, V, K = 140, 136, 1000, 5
    E, C, ids, t, dl = make(81, N, D, V, K)
    dead = [0, 3, 64, 131, 139]
    ids[dead] = IGN
    ids[3, 2] = V + 5                                # bad, not empty
    clean = [x.cuda() for x in (E, C, ids, t)]
    want_loss, lse = L.distill_forward(*clean, temperature=2.0)
    want = L.distill_backward(*clean, lse, dl.cuda(), temperature=2.0, deterministic=True, bf16_grads=bf16)
    E[dead[::2]] = float("nan")
    E[dead[1::2]] = float("inf")
    dl[dead] = float("nan")
    dirty = [x.cuda() for x in (E, C, ids, t)]
    loss, lse = L.distill_forward(*dirty, temperature=2.0)
    assert torch.equal(loss.nan_to_num(nan=-1), want_loss.nan_to_num(nan=-1))
    got = L.distill_backward(*dirty, lse, dl.cuda(), temperature=2.0, deterministic=True, bf16_grads=bf16)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (got[0][dead] == 0).all() and torch.isfinite(got[1].float()).all()


@pytest.mark.parametrize("D", [1016, 1024, 1032, 2048, 4104])
def test_long_rows_are_summed_in_parts(D):
    """The lse of one-signed logits, where every truncation of a running sum
    goes the same way.  A part of 1024 is 65 additions as in forward_bound, each
    off by at most one step (2 U32) of the part's sum, and the parts' sums make
    up the logit; they are added rounded to nearest (U32 of the logit each);
    exp2's argument, exp2 and the sums as in forward_bound."""
    import torch
    import linear_cross_entropy_05_b200 as L
    N, V, K = 130, 700, 3
    g = torch.Generator().manual_seed(D)
    E = torch.rand(N, D, generator=g).to(torch.bfloat16)
    C = (torch.rand(V, D, generator=g) * (64.0 / D)).to(torch.bfloat16)
    ids, t = torch.randint(0, V, (N, K), generator=g), torch.randn(N, K, generator=g)
    loss, lse, _, _, _ = reference(E, C, ids, t, 1.0, torch.ones(N))
    _, got = L.distill_forward(*(x.cuda() for x in (E, C, ids, t)))
    parts = -(-D // 1024)
    zmax = np.abs(f64(E) @ f64(C).T).max(axis=1)
    bound = (65 * 2 + parts + 8 + 2) * U32 * zmax + (96 + 24) * U32
    assert (np.abs(got.double().cpu().numpy() - lse) <= bound).all()


def test_a_second_derivative_is_refused():
    import torch
    import linear_cross_entropy_05_b200 as L
    E, C, ids, t, _ = [x.cuda() for x in make(91, 20, 64, 300, 4)]
    E.requires_grad_()
    g, = torch.autograd.grad(L.linear_distillation(E, C, ids, t), E, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


@pytest.mark.parametrize("N,D,V,K", [(256, 256, 4096, 8), (700, 264, 9001, 17), (1500, 1032, 20011, 4)])
def test_a_step_repeats_itself(N, D, V, K):
    import torch
    import linear_cross_entropy_05_b200 as L
    E, C, ids, t, _ = [x.cuda() for x in make(101, N, D, V, K)]
    first = None
    for _ in range(6):
        a, b = E.detach().requires_grad_(), C.detach().requires_grad_()
        loss = L.linear_distillation(a, b, ids, t, temperature=1.5)
        got = (loss.detach(),) + torch.autograd.grad(loss, (a, b))
        first = first or got
        assert all(torch.equal(x, y) for x, y in zip(first, got))


@pytest.mark.parametrize("N,D,V", [(1, 8, 300), (7, 192, 23568), (33, 264, 5000), (520, 1032, 60011), (600, 40, 100003)])
@pytest.mark.parametrize("per_launch", [None, 256])
def test_the_deterministic_sums_are_the_others(N, D, V, per_launch):
    """Only the order of fp32 additions of dE differs (one for each stripe, each
    off by U32 of a partial sum): fp32 gradients agree to 1e-5 of their norm,
    bf16 ones to the few values that round the other way."""
    import torch
    import linear_cross_entropy_05_b200 as L
    E, C, ids, t, dl = make(111, N, D, V, 3)
    dev = [x.cuda() for x in (E, C, ids, t)]
    _, lse = L.distill_forward(*dev)
    dl = dl.cuda()
    if per_launch:
        L.cce_debug_set_stripe_params(tokens_per_launch=per_launch)
    try:
        for bf16 in (False, True):
            for acc in (False, True):
                gdt = torch.bfloat16 if bf16 else torch.float32
                runs = []
                for det in (False, True, True):
                    out = tuple(torch.full(s, 0.25, dtype=gdt, device="cuda") for s in ((N, D), (V, D)))
                    runs.append(L.distill_backward(*dev, lse, dl, bf16_grads=bf16, accumulate=acc, deterministic=det,
                                                   out=out))
                for a, b, c in zip(*runs):
                    assert torch.equal(b, c)
                    a, b = a.float(), b.float()
                    assert (a - b).norm() <= (U16 if bf16 else 1e-5) * a.norm()
    finally:
        L.cce_debug_set_stripe_params()


def records(z, tiles):
    """Upper bound, per row, on how often the running maximum of a share of the
    vocabulary grows: shares are at most `tiles` tiles of 256, folded 32 columns
    at a time."""
    N, V = z.shape
    pad = -V % 256
    m = np.pad(z, ((0, 0), (0, pad)), constant_values=-np.inf).reshape(N, -1, 32).max(axis=2)
    most = np.zeros(N, dtype=int)
    for s in range(0, m.shape[1], 8):
        run = np.maximum.accumulate(m[:, s:s + 8 * tiles], axis=1)
        most = np.maximum(most, 1 + (np.diff(run, axis=1) > 0).sum(axis=1))
    return most


@pytest.mark.parametrize("T", [1e-3, 0.05, 1.0, 3.0, 1e6])
@pytest.mark.parametrize("N,D,V", [(40, 64, 100003), (9, 1088, 100100), (300, 96, 60001)])
def test_lse_of_exact_logits(N, D, V, T):
    """On a binary grid every partial sum of a logit is exact in fp32, so only
    the log-sum-exp's own roundings are left, none of which may grow with the
    number of columns folded.  With R = 2^-22 (exp2's relative error) and
    U = U32, the sum's relative error is at most
      3 U ln V      the argument of exp2 is rounded and its scale twice: 3 U of
                    a term's distance (M - z) / T, whose mean is below ln V
      R             exp2
      (64 + 16) U   additions: at most 64 chunks of 32 to a share, 9 within one, and
                    the shares' (in more bits)
      (R + 2 U) n   a new maximum rescales: n of them at most
      R + 2 U       the shares' join
    and the result is rounded once."""
    import torch
    import linear_cross_entropy_05_b200 as L
    # the temperature is a float: 1e-3 stands for one 4.7e-8 larger (relatively),
    # which alone moves an lse of 30900 by 1.5e-3
    T = float(np.float32(T))
    g = torch.Generator().manual_seed(N + D)
    se, sc, K = 2.0 ** -5, 2.0 ** -11, 5
    E = ((torch.randn(N, D, generator=g) / se).round() * se).to(torch.bfloat16)
    C = ((torch.randn(V, D, generator=g) * (6.0 / D ** 0.5) / sc).round() * sc).to(torch.bfloat16)
    z = (E.double() @ C.double().T).numpy()
    assert (E.abs().double() @ C[:500].abs().double().T).max() * 1.5 < 2.0 ** 24 * se * sc
    ids = torch.randint(0, V, (N, K), generator=g)
    ids[:, 0] = torch.from_numpy(z.argmax(axis=1))
    t = torch.randn(N, K, generator=g)
    x = z / T
    top = x.max(axis=1)
    lse = top + np.log(np.exp(x - top[:, None]).sum(axis=1))
    p, _ = oracle.distill_targets(ids.numpy(), f64(t), T, IGN)
    q = np.take_along_axis(x, ids.numpy(), 1) - lse[:, None]
    loss = T * T * (np.where(p > 0, p * np.log(np.maximum(p, 1e-300)), 0.0) - p * q).sum(axis=1)
    R, U = 2.0 ** -22, U32
    dlse = 3 * U * np.log(V) + R + 80 * U + (R + 2 * U) * records(z, 8) + R + 2 * U
    got, gl = L.distill_forward(*(a.cuda() for a in (E, C, ids, t)), temperature=T)
    err = np.abs(gl.double().cpu().numpy() - lse)
    assert (err <= dlse + 1.01 * U * np.abs(lse)).all(), (err / (dlse + U * np.abs(lse))).max()
    # the loss: lse before it is rounded, each weight rounded once, one rounding
    # of the result (and T to float for T^2: 2 U)
    err = np.abs(got.double().cpu().numpy() - loss)
    bound = T * T * (dlse + U * (p * np.abs(q)).sum(axis=1)) + 4 * U * np.abs(loss) + 4 * U * T * np.abs(p * q).sum(axis=1) * T
    assert (err <= bound).all(), (err / bound).max()


@pytest.mark.parametrize("D", [256, 264])
@pytest.mark.parametrize("how", [dict(), dict(bf16_grads=True), dict(deterministic=True), dict(accumulate=True),
                                 dict(bf16_grads=True, accumulate=True)])
def test_a_backward_whose_wait_gives_up_yields_nan(D, how):
    import torch
    import linear_cross_entropy_05_b200 as L
    N, V, K = 300, 5000, 20
    E, C, ids, t, dl = [x.cuda() for x in make(62, N, D, V, K)]
    gdt = torch.bfloat16 if how.get("bf16_grads") else torch.float32
    ws = L.Workspace("cuda")
    _, lse = L.distill_forward(E, C, ids, t, workspace=ws)

    def call():
        out = tuple(torch.zeros(s, dtype=gdt, device="cuda") for s in ((N, D), (V, D)))
        return L.distill_backward(E, C, ids, t, lse, dl, workspace=ws, out=out, **how)

    want = call()
    assert L.read_status(ws)["status"] == 0
    L.cce_debug_set_wait_limit_ns(20_000_000)
    L.cce_debug_withhold_loads(True)
    try:
        got = call()
        torch.cuda.synchronize()
    finally:
        L.cce_debug_withhold_loads(False)
        L.cce_debug_set_wait_limit_ns(1_000_000_000)
    assert L.read_status(ws)["status"] == 6
    assert all(torch.isnan(g).all() for g in got)
    got = call()
    assert L.read_status(ws)["status"] == 0
    for a, b in zip(got, want):
        assert torch.isfinite(a).all() and (a.float() - b.float()).norm() <= U16 * b.float().norm()
