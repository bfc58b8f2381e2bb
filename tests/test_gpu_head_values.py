"""Head norm with rotation at values where its arithmetic could leave the definition: infinities and NaN in
channels that nothing turns, norms without eps, norms far below 1.  Every path of the kernels: heads held by lanes
(halves, halves inside a vector, neighbouring pairs) and channel by channel.

Tolerance of finite fp32 values, relative 2-norm: a few roundings of 2^-24 and approximations of 2^-22 a value: 2e-6."""
import numpy as np
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
FLAT = 2e-6
INF, NAN = float("inf"), float("nan")


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def same(got, want, what):
    """NaN and infinities in the same places, finite values within the tolerance."""
    g = np64(got)
    assert g.shape == want.shape, (what, g.shape, want.shape)
    assert np.array_equal(np.isnan(g), np.isnan(want)), f"{what}: NaN elsewhere"
    far = np.isinf(want)
    assert np.array_equal(np.isinf(g), far) and np.array_equal(g[far], want[far]), f"{what}: infinities elsewhere"
    ok = np.isfinite(want)
    rel = np.linalg.norm(g[ok] - want[ok]) / max(np.linalg.norm(want[ok]), 1e-30)
    assert rel <= FLAT, f"{what}: rel {rel:.2e}"


def rand(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *shape: torch.randn(*shape, generator=g, device="cuda")


@pytest.mark.parametrize("d", [128, 40, 7])
def test_gradient_without_a_norm(d):
    """No norm: dx is dy w, whatever x holds and whatever the head's other channels hold."""
    import kda_recurrent_state_gb300 as kda

    r = rand(d)
    x, dy, w = r(9, 3, d), r(9, 3, d), r(d)
    x[1, 0, 2], x[2, 1, 3], x[3, 2, 0] = INF, -INF, NAN
    dy[4, 0, 1], dy[5, 1, 4], dy[6, 2, 5] = INF, NAN, -INF
    g = kda.kda_qk_norm_bwd(x, None, dy, None, w, norm=kda.KDA_NORM_NONE)
    same(g["dq"], np64(dy) * np64(w), "dq")
    with np.errstate(invalid="ignore"):
        same(g["dq_weight"], (np64(dy) * np64(x)).sum((0, 1)), "dq_weight")
