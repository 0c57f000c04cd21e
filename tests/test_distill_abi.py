"""Host-side argument checks of the distillation entry points."""
import pytest


@pytest.fixture(scope="module")
def L():
    from linear_cross_entropy_05_b200 import build
    build.build()
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake pointers are only passed where no GPU could be touched")
    import linear_cross_entropy_05_b200 as L
    return L


P = 1 << 20


def test_forward(L):
    ok = [P, P, P, P, 0, 256, 256, 4096, 8, -100, 1.0, P, P, P, P, P, 1 << 30, 0]

    def call(**at):
        a = list(ok)
        for k, v in at.items():
            a[int(k[1:])] = v
        return L.cce_distill_forward(*a, check=False)

    for i in (0, 1, 2, 3, 11, 12, 13, 14, 15):                        # (13, 14: both or neither)
        assert call(**{f"a{i}": 0}) == 1
    assert call(a13=0, a14=0) == 4
    assert call(a4=2) == 1 and call(a4=-1) == 1                       # unknown teacher type
    assert call(a5=0) == 1 and call(a6=252) == 1 and call(a7=0) == 1
    assert call(a8=0) == 1 and call(a8=1025) == 1                     # K
    assert call(a7=(1 << 31) - 1, a6=8) == 1                          # ids of a tile's end must fit int32
    for T in (0.0, -2.0, float("nan"), float("inf"), 1e-45, 0.9e-3, 1.1e6):
        assert call(a10=T) == 1
    assert call(a0=P + 8) == 2 and call(a2=P + 4) == 2 and call(a3=P + 2) == 2 and call(a15=P + 128) == 2
    assert call(a3=P + 2, a4=1) == 4                                  # bf16 logits on 2-byte addresses
    assert call() == 4                                                # valid, no device here


def test_backward(L):
    ok = [P, P, P, P, 0, P, P, 1, P, 256, 256, 4096, 8, -100, 1.0, 0, P, P, P, 1 << 40, 0]

    def call(**at):
        a = list(ok)
        for k, v in at.items():
            a[int(k[1:])] = v
        return L.cce_distill_backward(*a, check=False)

    for i in (0, 1, 2, 3, 5, 6, 16, 17, 18):
        assert call(**{f"a{i}": 0}) == 1
    for flags in (8, 16, 32, 64):
        assert call(a15=flags) == 1
    for flags in range(8):
        assert call(a15=flags) == 4
    assert call(a16=P + 8) == 2 and call(a5=P + 2) == 2
    assert call(a7=2) == 1 and call(a7=0) == 4 and call(a8=0) == 4 and call(a8=P + 2) == 2


def test_backward_workspace(L):
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    size = L.cce_distill_backward_workspace_size
    N, D, V, K = 8192, 2304, 256000, 64
    stripes = (L.cce_backward_workspace_size_ex(N, D, V, 16) - L.cce_backward_workspace_size(N, D, V))
    base = 256 + up(4 * N) + up(16 * N) + 2 * up(4 * N * K) + up(2 * N * D) + stripes
    assert size(N, D, V, K, 0) == size(N, D, V, K, 1) == size(N, D, V, K, 4) == base
    assert size(N, D, V, K, 2) == base + up(4 * N * D)                        # dC is rounded where it is formed
    assert size(N, D, V, K, 6) == base + up(4 * N * D) + up(4 * V * D)        # accumulated: fp32 sums first
    assert size(N, D, V, 0, 0) == 0 and size(N, D, V, 1025, 0) == 0 and size(N, D, V, K, 16) == 0
    # few dE tiles: narrower stripes, as many columns of buffers
    assert size(256, 256, 4096, 8, 0) == 256 + up(4 * 256) + up(16 * 256) + 2 * up(4 * 256 * 8) + \
        up(2 * 256 * 256) + up(8 + 4 * (16 + 16 + 16 + 1) + 16) + up(16 * 256 * 256 * 2)
    big = size(16385, 256, 4096, 4, 2)
    assert big >= up(4 * 16385 * 256) + up(4 * 4096 * 256)                    # several launches: fp32 sums first
    assert L.cce_distill_forward_workspace_size(N, D, V, K) == 0              # no device here
