"""The draw's definition, and the host-side checks of cce_top_logits and cce_sample."""
import ctypes

import numpy as np
import pytest

import oracle

P = 1 << 20


def test_draw_by_hand():
    z = np.log(np.array([0.1, 0.4, 0.05, 0.4, 0.05]))
    assert [oracle.sample_row(z, u)[0] for u in (0.0, 0.0999, 0.1001, 0.4999, 0.5001, 0.5499, 0.5501, 0.9499, 0.9501)] == \
        [0, 0, 1, 1, 2, 2, 3, 3, 4]
    assert abs(oracle.sample_row(z, 0.2)[1] - np.log(0.4)) < 1e-12
    assert oracle.sample_row(z, 0.9, temperature=0.0)[0] == 1          # a tie: the lowest id
    assert oracle.sample_row(z, 0.999, top_k=1)[0] == 1
    assert [oracle.sample_row(z, u, top_k=2)[0] for u in (0.49, 0.51)] == [1, 3]
    assert [oracle.sample_row(z, u, top_k=4)[0] for u in (0.999, 0.0)] == [3, 0]   # the second 0.05 is out
    assert oracle.sample_row(z, 0.999, top_p=0.39)[0] == 1
    assert oracle.sample_row(z, 0.999, top_p=0.41)[0] == 3
    assert oracle.sample_row(z, 0.0, top_p=0.85)[0] == 0
    assert oracle.sample_row(z, 0.0, min_p=0.3)[0] == 1
    assert oracle.sample_row(z, 0.0, min_p=0.2)[0] == 0


@pytest.fixture(scope="module")
def L():
    from linear_cross_entropy_05_b200 import build
    build.build()
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake pointers are only passed where no GPU could be touched")
    import linear_cross_entropy_05_b200 as L
    return L


def test_workspace(L):
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    for N, V in ((1, 1), (5, 4096), (256, 256000), (513, 100003), (100000, 33)):
        rows, grp = min(N, 512), -(-V // 32)
        want = 256 + 8 * (1024 + 512) + up(4 * rows * 32 * grp) + up(8 * rows * grp) + up(4 * rows * grp) + 12 * 1024 * rows
        assert L.cce_head_workspace_size(N, 64, V) == want
    for bad in ((0, 64, 100), (5, 60, 100), (5, 64, 0), (5, 8, (1 << 31) - 1)):
        assert L.cce_head_workspace_size(*bad) == 0


def test_top_logits(L):
    ok = [P, P, 16, 64, 1000, 10, P, P, P, P, 1 << 30, 0]

    def call(**at):
        a = list(ok)
        for k, v in at.items():
            a[int(k[1:])] = v
        return L.cce_top_logits(*a, check=False)

    for i in (0, 1, 6, 7, 8, 9):
        assert call(**{f"a{i}": 0}) == 1
    for k in (0, -1, 1001, 1025):
        assert call(a5=k) == 1
    assert call(a4=5000, a5=1025) == 1
    assert call(a0=P + 8) == 2 and call(a7=P + 4) == 2 and call(a9=P + 16) == 2
    assert call() == 4


def test_sample(L):
    def call(i=None, v=None, **settings):
        s = L.CCESampleSettings(temperature_all=1.0, top_p_all=1.0)
        for n, x in settings.items():
            setattr(s, n, x)
        a = [P, P, 16, 64, 1000, P, s, P, P, P, 1 << 30, 0]
        if i is not None:
            a[i] = v
        return L.cce_sample(*a, check=False)

    for i in (0, 1, 5, 7, 8, 9):
        assert call(i, 0) == 1
    nan = float("nan")
    for bad in (dict(temperature_all=-1.0), dict(temperature_all=nan), dict(top_k_all=-1), dict(top_p_all=-0.5),
                dict(top_p_all=nan), dict(min_p_all=1.5), dict(min_p_all=nan)):
        assert call(**bad) == 1
        name = next(iter(bad))[:-4]
        assert call(**bad, **{name: P}) == 4       # not looked at where an array is given
    assert call(temperature=P + 2) == 2 and call(7, P + 4) == 2
    assert call() == 4


def test_settings_layout(L):
    assert ctypes.sizeof(L.CCESampleSettings) == 48
