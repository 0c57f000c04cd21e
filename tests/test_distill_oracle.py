"""The fp64 definition of the distillation loss: pinned by torch autograd,
finite differences and the cases that have a closed form."""
import numpy as np
import pytest

import oracle


def _case(seed, N=5, D=16, V=37, K=6):
    rng = np.random.default_rng(seed)
    E, C = rng.standard_normal((N, D)), rng.standard_normal((V, D)) * 0.5
    ids = np.stack([rng.permutation(V)[:K] for _ in range(N)])
    return E, C, ids, rng.standard_normal((N, K)) * 2, rng.standard_normal(N)


@pytest.mark.parametrize("T", [0.5, 1.0, 3.0])
def test_gradient_matches_torch_and_differences(T):
    import torch
    E, C, ids, t, dl = _case(1)
    ids[1, 3:] = -100          # a short row
    t[2, 0] = -np.inf          # an absent entry
    ids[3] = -100              # a row without a target
    ids[4, 1] = ids[4, 0]      # the same id twice
    loss, lse, dE, dC, _ = oracle.distill(E, C, ids, t, T, dloss=dl)
    Et, Ct = (torch.tensor(v, requires_grad=True) for v in (E, C))
    logq = torch.log_softmax(Et @ Ct.T / T, 1)
    total = 0.0
    for i in range(E.shape[0]):
        live = [k for k in range(ids.shape[1]) if ids[i, k] != -100 and t[i, k] != -np.inf]
        if not live:
            assert loss[i] == 0
            continue
        p = torch.softmax(torch.tensor(t[i, live]) / T, 0)
        one = T * T * (p * (p.log() - logq[i, ids[i, live]])).sum()
        assert abs(float(one) - loss[i]) < 1e-12 * max(1, abs(loss[i]))
        total = total + dl[i] * one
    total.backward()
    assert np.allclose(Et.grad.numpy(), dE, atol=1e-12) and np.allclose(Ct.grad.numpy(), dC, atol=1e-12)
    rng = np.random.default_rng(2)
    for M, dM in ((E, dE), (C, dC)):
        step = rng.standard_normal(M.shape)
        h = 1e-5
        at = []
        for s in (h, -h):
            M += s * step
            at.append((oracle.distill(E, C, ids, t, T)[0] * dl).sum())
            M -= s * step
        assert abs((at[0] - at[1]) / (2 * h) - (dM * step).sum()) < 1e-7 * max(1, abs((dM * step).sum()))


def test_a_teacher_that_is_the_student_gives_no_loss_and_no_gradient():
    E, C, _, _, dl = _case(3, V=24)
    ids = np.tile(np.arange(24), (5, 1))
    loss, _, dE, dC, _ = oracle.distill(E, C, ids, E @ C.T, 2.0, dloss=dl)
    assert np.abs(loss).max() < 1e-12 and np.abs(dE).max() < 1e-12 and np.abs(dC).max() < 1e-12


def test_one_entry_is_the_cross_entropy_of_its_id():
    E, C, ids, t, dl = _case(4, K=1)
    loss, lse, dE, dC, _ = oracle.distill(E, C, ids, t, 1.0, dloss=dl)
    z = E @ C.T
    want = np.log(np.exp(z).sum(1)) - z[np.arange(5), ids[:, 0]]
    assert np.allclose(loss, want, atol=1e-12)
