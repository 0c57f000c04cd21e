"""The k largest logits and drawn tokens on the GPU against the fp64
definition.

E and C lie on a binary grid on which every partial sum of a logit is exact in
fp32, so the GPU's logits are the definition's and ids are compared for
equality; ties are frequent."""
import numpy as np
import pytest

import oracle

from _gpu_helpers import IGN

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24

# Rows whose token does not hang on it get their log-sum-exp from float
# exponentials 2^t, t <= 0, within each group of 32 (summed in double from
# there); the largest logit's own is exact and kept apart.  Of the others' sum
# the relative error is at most
#   2^-22      ex2's own
#   45 U32     t = (z - top) c: the difference, c and the product are rounded,
#              3 U32 |t| ln 2 of 2^t, and sum |t| ln 2 2^t / sum 2^t <= ln V + 1
#              < 15
#   6 U32      the others of a group are summed in six additions
# and S = 1 + others (where 1 is the largest), so log S is off by at most
# FLOAT_SUMS * others / S <= FLOAT_SUMS * log S.
FLOAT_SUMS = 2.0 ** -22 + 51 * U32


def make(seed, N, D, V, spread=2.0, coarse=False):
    """E on multiples of 2^-5, C on multiples of 2^-11 (coarse: 2^-2 and 2^-4,
    many ties); |z| partial sums stay under 2^24 steps."""
    import torch
    g = torch.Generator().manual_seed(seed)
    se, sc = (2.0 ** -2, 2.0 ** -4) if coarse else (2.0 ** -5, 2.0 ** -11)
    E = (torch.randn(N, D, generator=g) / se).round() * se
    C = (torch.randn(V, D, generator=g) * spread / D ** 0.5 / sc).round() * sc
    E, C = E.to(torch.bfloat16), C.to(torch.bfloat16)
    z = E.double().numpy() @ C.double().numpy().T
    assert (E.abs().double() @ C.abs().double().T).max() < 2.0 ** 24 * se * sc
    return E, C, z, torch.rand(N, generator=g)


def check_top(got, z, k):
    values, ids, lse = (t.cpu().numpy() for t in got)
    for i in range(z.shape[0]):
        order = oracle.falling_order(z[i])[:k]
        assert np.array_equal(ids[i], order), i
        assert np.array_equal(values[i], z[i][order].astype(np.float32))
    top = z.max(axis=1)
    want = top + np.log(np.exp(z - top[:, None]).sum(axis=1))
    assert (np.abs(lse - want) <= FLOAT_SUMS * (want - top) + 1.01 * U32 * np.abs(want) + 1e-12).all()


@pytest.mark.parametrize("N,D,V,k", [
    (1, 8, 1, 1), (1, 64, 31, 31), (3, 264, 257, 20), (33, 128, 1000, 1000), (70, 896, 4097, 64), (5, 64, 40000, 1024),
    (300, 64, 20000, 7), (2, 2304, 30011, 129), (4, 16, 300000, 50), (257, 40, 2000, 100),
])
@pytest.mark.parametrize("coarse", [False, True])
def test_top_logits(N, D, V, k, coarse):
    import linear_cross_entropy_05_b200 as L
    E, C, z, _ = make(N + V + k, N, D, V, coarse=coarse)
    ws = L.Workspace("cuda")
    got = L.top_logits(E.cuda(), C.cuda(), k, workspace=ws)
    assert L.read_status(ws)["status"] == 0
    check_top(got, z, k)


def test_top_logits_of_rows_full_of_ties():
    import linear_cross_entropy_05_b200 as L
    E, C, z, _ = make(3, 6, 64, 20000, coarse=True)
    E[1] = 0                       # every logit equal
    C[:, 1:] = 0                   # rows of a few distinct values
    C[:, 0] = C[:, 0].sign() * 0.5
    z = E.double().numpy() @ C.double().numpy().T
    for k in (1, 33, 1024):
        check_top(L.top_logits(E.cuda(), C.cuda(), k), z, k)


SETTINGS = [
    dict(temperature=0.0), dict(temperature=1.0), dict(temperature=0.25), dict(temperature=8.0), dict(top_k=1),
    dict(top_k=50), dict(top_k=2000), dict(top_k=1 << 30), dict(top_p=0.0), dict(top_p=0.5), dict(top_p=0.9),
    dict(top_p=0.9990), dict(min_p=0.1), dict(min_p=1.0), dict(min_p=1e-3), dict(top_k=40, top_p=0.8),
    dict(top_k=200, min_p=0.02), dict(top_p=0.95, min_p=0.01, temperature=1.5),
    dict(top_k=100, top_p=0.9, min_p=0.05, temperature=0.7), dict(temperature=1e-30), dict(temperature=1e30),
    dict(temperature=1e30, top_p=0.75), dict(temperature=0.0, top_k=5, min_p=0.5),
]


def check_draw(got, z, u, settings):
    token, logp = (t.cpu().numpy() for t in got)
    for i in range(z.shape[0]):
        s = {n: (v[i] if hasattr(v, "__len__") else v) for n, v in settings.items()}
        s = {n: (int(v) if n == "top_k" else float(np.float32(v))) for n, v in s.items()}
        want, lp = oracle.sample_row(z[i], float(u[i]), **s)
        assert token[i] == want, (i, s, float(u[i]))
        k = s.get("top_k", 0)
        exact = (s.get("temperature", 1.0) > 0 and not 0 < k < z.shape[1] and
                 (s.get("top_p", 1.0) < 1 or s.get("min_p", 0.0) == 0))
        # double sums: one rounding of the result; else log S <= -lp is off too
        assert abs(logp[i] - lp) <= (1.01 * U32 + (0 if exact else FLOAT_SUMS)) * abs(lp) + 1e-12, (i, s)


@pytest.mark.parametrize("N,D,V", [(1, 8, 1), (2, 64, 31), (40, 264, 257), (33, 128, 3000), (21, 96, 20000),
                                   (300, 64, 5000), (3, 16, 300000)])
def test_draws_match_the_definition(N, D, V):
    import torch
    import linear_cross_entropy_05_b200 as L
    E, C, z, u = make(N + V, N, D, V, spread=3.0)
    u[0] = 0.0
    u[-1] = 1.0 - 2.0 ** -24
    ws = L.Workspace("cuda")
    for s in SETTINGS:
        if V > 100000 and s.get("temperature", 1.0) < 1e-20:
            continue
        check_draw(L.sample(E.cuda(), C.cuda(), u.cuda(), workspace=ws, **s), z, u, s)
        assert L.read_status(ws)["status"] == 0
    # every row with settings of its own
    pick = [SETTINGS[i % len(SETTINGS)] for i in range(N)]
    rows = {n: [s.get(n, d) for s in pick] for n, d in
            (("temperature", 1.0), ("top_k", 0), ("top_p", 1.0), ("min_p", 0.0))}
    dev = {n: torch.tensor(v, dtype=torch.int32 if n == "top_k" else torch.float32, device="cuda")
           for n, v in rows.items()}
    check_draw(L.sample(E.cuda(), C.cuda(), u.cuda(), workspace=ws, **dev), z, u, rows)


@pytest.mark.parametrize("V,spread", [(20000, 0.5), (70001, 2.5)])
@pytest.mark.parametrize("coarse", [False, True])
def test_wide_prefixes_and_rows_full_of_ties(coarse, V, spread):
    """Kept sets of more entries than the sorted ones, and ties across every border."""
    import linear_cross_entropy_05_b200 as L
    E, C, z, u = make(8, 12, 32, V, spread=spread, coarse=coarse)
    E[3] = 0
    E[4] = 0
    E[5] = 0
    z = E.double().numpy() @ C.double().numpy().T
    u[3], u[4], u[5] = 0.0, 0.5, 1.0 - 2.0 ** -24
    for s in (dict(top_p=0.9), dict(top_k=6000), dict(top_k=6000, top_p=0.8), dict(min_p=0.2), dict(top_p=0.7, min_p=0.3),
              dict(top_k=7001, top_p=0.95, min_p=0.1, temperature=1.25), dict(top_k=50), dict(), dict(temperature=0.0),
              dict(top_p=0.01), dict(top_p=1.0 - 2.0 ** -24), dict(top_p=0.6, temperature=50.0), dict(top_k=4097),
              dict(top_k=V - 1, top_p=0.99), dict(top_p=0.97, temperature=3.0, min_p=1e-5)):
        check_draw(L.sample(E.cuda(), C.cuda(), u.cuda(), **s), z, u, s)


def test_a_log_probability_near_zero_keeps_its_relative_precision():
    import torch
    import linear_cross_entropy_05_b200 as L
    E, C, z, u = make(13, 9, 128, 30000, spread=1.5)
    up = torch.tensor([6.0, 8.0, 10.0, 12.0, 14.0, 16.0, 18.0, 20.0, 22.0])
    for i in range(9):   # one id stands out
        E[i] = (E[i].float() + up[i] * C[100 * i].float() / C[100 * i].float().square().sum()).mul(32).round().div(32)
    z = E.double().numpy() @ C.double().numpy().T
    for s in (dict(temperature=0.0), dict(top_k=3), dict(top_p=0.9), dict(), dict(min_p=0.5)):
        check_draw(L.sample(E.cuda(), C.cuda(), u.cuda(), **s), z, u, s)


def test_a_row_that_is_not_finite_is_marked_and_the_others_are_right():
    import torch
    import linear_cross_entropy_05_b200 as L
    E, C, z, u = make(9, 7, 64, 900)
    E[2, 5] = float("nan")
    E[4, 0] = float("inf")
    keep = [0, 1, 3, 5, 6]
    ws = L.Workspace("cuda")
    for s in (dict(temperature=0.0), dict(), dict(top_k=9), dict(top_p=0.5)):
        token, logp = L.sample(E.cuda(), C.cuda(), u.cuda(), workspace=ws, **s)
        st = L.read_status(ws)
        assert st["status"] == 8 and st["flags"] == 4
        assert (token[[2, 4]] == -1).all() and torch.isnan(logp[[2, 4]]).all()
        check_draw((token[keep], logp[keep]), z[keep], u[keep], s)
    values, ids, lse = L.top_logits(E.cuda(), C.cuda(), 5, workspace=ws)
    assert L.read_status(ws)["status"] == 8
    assert (ids[[2, 4]] == -1).all() and torch.isnan(values[[2, 4]]).all() and torch.isnan(lse[[2, 4]]).all()
    check_top((values[keep], ids[keep], lse[keep]), z[keep], 5)


def test_settings_outside_their_range_per_row():
    import torch
    import linear_cross_entropy_05_b200 as L
    E, C, z, u = make(10, 8, 64, 900)
    nan = float("nan")
    t = torch.tensor([nan, -1.0, 1, 1, 1, 1, 1, 1], device="cuda")
    k = torch.tensor([0, 0, -3, 0, 0, 0, 0, 0], dtype=torch.int32, device="cuda")
    p = torch.tensor([1, 1, 1, nan, 7.0, -1.0, 1, 1], device="cuda")
    m = torch.tensor([0, 0, 0, 0, 0, 0, 5.0, nan], device="cuda")
    got = L.sample(E.cuda(), C.cuda(), u.cuda(), temperature=t, top_k=k, top_p=p, min_p=m)
    check_draw(got, z, u, dict(temperature=[0.0, 0.0] + [1.0] * 6, top_p=[1.0] * 5 + [0.0, 1.0, 1.0],
                               min_p=[0.0] * 6 + [1.0, 0.0]))
    odd = torch.tensor([nan, -2.0, 1.0, 3.0, float("inf"), 0.0, 0.0, 0.0])
    want = torch.tensor([0.0, 0.0] + [1.0 - 2.0 ** -53] * 3 + [0.0] * 3, dtype=torch.float64)
    for s in (dict(), dict(top_k=30), dict(top_p=0.9)):
        check_draw(L.sample(E.cuda(), C.cuda(), odd.cuda(), **s), z, want, s)


def test_teacher_student_and_rollout_together():
    """As they are used: the teacher's top logits teach the student, whose
    drawn tokens have the log-probability that the loss gives them."""
    import torch
    import linear_cross_entropy_05_b200 as L
    N, V, K = 300, 5003, 24
    Et, Ct, zt, _ = make(11, N, 192, V)
    Es, Cs, zs, u = make(12, N, 128, V)
    values, ids, lse_t = L.top_logits(Et.cuda(), Ct.cuda(), K)
    E, C = Es.cuda().requires_grad_(), Cs.cuda().requires_grad_()
    loss = L.linear_distillation(E, C, ids, values, temperature=2.0)
    loss.backward()
    order = np.stack([oracle.falling_order(r)[:K] for r in zt])
    t = np.take_along_axis(zt, order, 1)
    dl = np.full(N, 1.0 / N)
    ref, _, dE, dC, _ = oracle.distill(Es.double().numpy(), Cs.double().numpy(), order, t, 2.0, IGN, dl)
    assert abs(loss.item() - ref.mean()) <= 1e-5 * ref.mean()
    for g, b in ((E.grad, dE), (C.grad, dC)):
        assert np.linalg.norm(g.double().cpu().numpy() - b) <= 2 * 2.0 ** -8 * np.linalg.norm(b)
    token, logp = L.sample(Es.cuda(), Cs.cuda(), u.cuda(), top_k=40, top_p=0.9)
    check_draw((token, logp), zs, u, dict(top_k=40, top_p=0.9))
    ce, _ = L.forward(Es.cuda(), Cs.cuda(), token)
    assert torch.allclose(logp, -ce, rtol=0, atol=2e-5)
    # without logits the student learns the same from the token alone
    one = L.distill_forward(Es.cuda(), Cs.cuda(), token[:, None].contiguous(), torch.zeros(N, 1, device="cuda"))[0]
    assert torch.allclose(one, ce, rtol=0, atol=2e-5)


def test_streams_graphs_and_two_calls_at_once():
    import torch
    import linear_cross_entropy_05_b200 as L
    sets = []
    for seed in (21, 22):
        E, C, z, u = make(seed, 290, 64, 5000)
        sets.append((E.cuda(), C.cuda(), u.cuda(), z, u))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for (E, C, ug, _, _), st in zip(sets, streams):
        outs.append((L.sample(E, C, ug, top_k=30, stream=st), L.top_logits(E, C, 9, stream=st)))
    torch.cuda.synchronize()
    for (E, C, ug, z, u), (drawn, top) in zip(sets, outs):
        check_draw(drawn, z, u, dict(top_k=30))
        check_top(top, z, 9)
    held = [t.clone() for t in sets[0][:3]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        drawn = L.sample(*held, top_p=0.8)
        top = L.top_logits(held[0], held[1], 9)
    for E, C, ug, z, u in reversed(sets):
        for h, x in zip(held, (E, C, ug)):
            h.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        check_draw(drawn, z, u, dict(top_p=0.8))
        check_top(top, z, 9)


def test_a_wait_that_gives_up_marks_every_row():
    import torch
    import linear_cross_entropy_05_b200 as L
    E, C, z, u = make(31, 40, 64, 5000)
    ws = L.Workspace("cuda")
    check_draw(L.sample(E.cuda(), C.cuda(), u.cuda(), workspace=ws), z, u, {})
    L.cce_debug_set_wait_limit_ns(20_000_000)
    L.cce_debug_withhold_loads(True)
    try:
        token, logp = L.sample(E.cuda(), C.cuda(), u.cuda(), workspace=ws)
        torch.cuda.synchronize()
    finally:
        L.cce_debug_withhold_loads(False)
        L.cce_debug_set_wait_limit_ns(1_000_000_000)
    assert L.read_status(ws)["status"] == 6
    assert (token == -1).all() and torch.isnan(logp).all()
    check_draw(L.sample(E.cuda(), C.cuda(), u.cuda(), workspace=ws), z, u, {})


def test_refusals():
    import torch
    import linear_cross_entropy_05_b200 as L
    E, C, z, u = make(41, 6, 64, 300)
    E, C, u = E.cuda(), C.cuda(), u.cuda()
    for k in (0, -1, 301, 1025):
        with pytest.raises(L.CCEError):
            L.top_logits(E, C, k)
    with pytest.raises(TypeError):
        L.sample(E.half(), C, u)
    with pytest.raises(TypeError):
        L.sample(E, C, u.double())
    with pytest.raises(ValueError):
        L.sample(E, C, u[:5])
    with pytest.raises(ValueError):
        L.sample(E, C.t().contiguous().t(), u)
    with pytest.raises(TypeError):
        L.sample(E, C, u, top_k=torch.zeros(6, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        L.sample(E, C, u, temperature=torch.ones(5, device="cuda"))
    for bad in (dict(temperature=-0.5), dict(temperature=float("nan")), dict(top_k=-1), dict(top_p=-0.1),
                dict(min_p=1.5), dict(min_p=float("nan"))):
        with pytest.raises(L.CCEError):
            L.sample(E, C, u, **bad)
    with pytest.raises(L.CCEError):
        L.sample(E, C, u, top_k=5 - 2 ** 32)      # not 5


def test_wide_prefixes_of_two_blocks_of_tokens():
    """More than 256 tokens: fewer bins a row than head_select has threads."""
    import linear_cross_entropy_05_b200 as L
    E, C, z, u = make(15, 261, 16, 21001, spread=1.0)
    for s in (dict(top_p=0.9), dict(top_k=5000, top_p=0.5)):
        check_draw(L.sample(E.cuda(), C.cuda(), u.cuda(), **s), z, u, s)


@pytest.mark.parametrize("V", [31, 257, 900, 1024, 5003])
def test_an_infinite_temperature_draws_evenly(V):
    """x = z / inf: 0 for every logit but one of -inf, which has no weight."""
    import torch
    import linear_cross_entropy_05_b200 as L
    E, C, z, u = make(51, 40, 64, V)
    E[:, 0] = 0
    E[7, 0] = 2.0 ** 100
    C[:, 0] = 0
    C[[0, V // 2, V - 1], 0] = -(2.0 ** 100)     # these logits of row 7 are -inf
    z = E.double().numpy() @ C.double().numpy().T
    z[z < -1e38] = -np.inf
    live = np.flatnonzero(z[7] > -np.inf)
    assert live.size == V - 3 and np.isfinite(np.delete(z, 7, 0)).all()
    inf = float("inf")
    for s in (dict(top_k=9), dict(top_k=V - 1), dict(min_p=0.5), dict(top_k=20, top_p=0.5), dict(),
              dict(top_p=0.6), dict(top_k=12, min_p=0.25)):
        for rows in (False, True):
            t = torch.full((40,), inf, device="cuda") if rows else inf
            token, logp = L.sample(E.cuda(), C.cuda(), u.cuda(), temperature=t, **s)
            keep = np.delete(np.arange(40), 7)
            check_draw((token[keep], logp[keep]), z[keep], u[keep], dict(temperature=inf, **s))
            if s.get("top_k", 0) != V - 1:       # row 7 over the entries with any weight
                at = torch.from_numpy(np.searchsorted(live, token[[7]].cpu().numpy()))
                assert live[at.item()] == token[7].item()
                check_draw((at, logp[[7]]), z[[7]][:, live], u[[7]], dict(temperature=inf, **s))


@pytest.mark.parametrize("V", [31, 900, 9001])
def test_min_p_of_one_at_temperatures_that_level_the_masses(V):
    """Where exp((z - max) / T) rounds to 1 in double, every entry is as likely
    as the largest."""
    import linear_cross_entropy_05_b200 as L
    E, C, z, u = make(52, 10, 64, V)
    for t in (1e18, 1e30, float("inf")):
        for s in (dict(min_p=1.0), dict(min_p=1.0, top_k=12), dict(min_p=1.0, top_p=0.5)):
            s["temperature"] = t
            check_draw(L.sample(E.cuda(), C.cuda(), u.cuda(), **s), z, u, s)


@pytest.mark.parametrize("D", [136, 896, 2304, 8192])
def test_ordinary_inputs(D):
    """Inputs on no grid: the tensor cores add 16 products at a time to a fp32
    sum, D / 16 additions that each truncate by at most one step (2 U32) of the
    sum of the magnitudes S, so a logit is off by at most
    dz = (D / 16 + 1) 2 U32 S; log-sum-exps by that and FLOAT_SUMS."""
    import torch
    import linear_cross_entropy_05_b200 as L
    N, V, k = 70, 9001, 40
    g = torch.Generator().manual_seed(D)
    E = torch.randn(N, D, generator=g).to(torch.bfloat16)
    C = (torch.randn(V, D, generator=g) * 2.0 / D ** 0.5).to(torch.bfloat16)
    for i in range(N):   # a few candidates stand out, as in a trained head
        E[i] = (E[i].float() + 3.0 * C[7 * i:7 * i + 3].float().sum(0)).to(torch.bfloat16)
    z = (E.double() @ C.double().T).numpy()
    dz = ((D / 16 + 1) * 2 * U32 * (E.double().abs() @ C.double().abs().T)).numpy()
    most = dz.max(axis=1)
    top = z.max(axis=1)
    wide = np.log(np.exp(z - top[:, None]).sum(axis=1))       # lse - largest
    dlse = most + FLOAT_SUMS * wide + 1.01 * U32 * np.abs(top + wide) + 1e-12
    values, ids, lse = (t.cpu().numpy() for t in L.top_logits(E.cuda(), C.cuda(), k))
    rows = np.arange(N)[:, None]
    assert (np.abs(values - z[rows, ids]) <= dz[rows, ids] + U32 * np.abs(values)).all()
    assert (np.diff(values, axis=1) <= 0).all()
    kth = np.sort(z, axis=1)[:, -k]
    assert all(np.unique(r).size == k for r in ids) and (z[rows, ids] >= (kth - 2 * most)[:, None]).all()
    assert (np.abs(lse - (top + wide)) <= dlse).all()
    u = torch.rand(N, generator=g).cuda()
    token, logp = (t.cpu().numpy() for t in L.sample(E.cuda(), C.cuda(), u, temperature=0.0))
    assert np.array_equal(token, ids[:, 0])
    got = z[np.arange(N), token]
    assert (np.abs(logp - (got - top - wide)) <= 2 * most + dlse).all()
    token, logp = (t.cpu().numpy() for t in L.sample(E.cuda(), C.cuda(), u, top_k=k, top_p=0.9))
    assert all(token[i] in ids[i] for i in range(N))
    got = z[np.arange(N), token]
    assert (np.abs(logp - (got - top - wide)) <= 2 * most + dlse).all()


def test_a_k_out_of_range_allocates_nothing():
    import torch
    import linear_cross_entropy_05_b200 as L
    E, C, _, _ = make(53, 6, 64, 300)
    E, C = E.cuda(), C.cuda()
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    held = torch.cuda.memory_allocated()
    for k in (301, 1 << 24, 1 << 50, -(1 << 50)):
        with pytest.raises(L.CCEError):
            L.top_logits(E, C, k)
    assert torch.cuda.max_memory_allocated() == held


def test_a_token_is_chosen_alike_in_any_batch():
    import torch
    import linear_cross_entropy_05_b200 as L
    g = torch.Generator().manual_seed(54)
    N, D, V = 600, 2304, 9001
    E = torch.randn(N, D, generator=g).to(torch.bfloat16).cuda()
    C = (torch.randn(V, D, generator=g) * 3.0 / D ** 0.5).to(torch.bfloat16).cuda()
    values, ids, _ = L.top_logits(E, C, 50)
    for rows in ([0], [599], list(range(100, 133)), list(range(0, 600, 2)), list(range(40, 552))):
        v, i, _ = L.top_logits(E[rows].contiguous(), C, 50)
        assert torch.equal(v, values[rows]) and torch.equal(i, ids[rows])
