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


ANGLES = 50
HEADS = [  # d, rot, half: one path each
    (128, 64, True),   # halves of whole lanes
    (40, 10, True),    # a half inside a lane's channels
    (128, 60, False),  # neighbouring pairs, the last of them inside a lane's channels
    (7, 4, True),      # channel by channel
    (7, 4, False),
]


@pytest.mark.parametrize("d,rot,half", HEADS)
@pytest.mark.parametrize("norm", ["none", "rms"])
def test_what_is_not_turned_stays(d, rot, half, norm):
    """Infinities and NaN in channels past the turned ones, and anywhere in a head whose position is outside the
    tables, touch no other channel of a head that has no norm, and come out as they are; with a norm they spoil their
    own head alone."""
    import kda_recurrent_state_gb300 as kda
    from kda_recurrent_state_gb300 import binding

    r = rand(d + rot)
    x, dy, w, ang = r(12, 3, d), r(12, 3, d), r(d), r(ANGLES, rot // 2) * 3
    cos, sin = ang.cos(), ang.sin()
    pos = torch.arange(12, device="cuda") * 4
    pos[3], pos[7] = ANGLES, -1
    for t in (x, dy):
        t[0, 0, rot], t[1, 1, rot + 1], t[2, 2, d - 1] = INF, NAN, -INF  # past the turned channels
        t[3, 0, 0], t[3, 1, rot - 1], t[3, 2, rot // 2] = INF, NAN, -INF  # outside the tables
        t[7, 1, 1] = NAN
    kw = dict(norm=kda.KDA_NORM_NONE if norm == "none" else kda.KDA_NORM_RMS, eps=1e-5,
              layout=kda.KDA_ROT_HALF if half else kda.KDA_ROT_PAIRS)
    assert kda.kda_get_device_status() == 0
    out, _ = kda.kda_qk_norm_fwd(x, None, w, None, cos, sin, pos, **kw)
    g = kda.kda_qk_norm_bwd(x, None, dy, None, w, None, cos, sin, pos, **kw)
    assert kda.kda_get_device_status() == binding.KDA_STATUS_POSITION_RANGE
    at = pos.cpu().numpy()
    with np.errstate(invalid="ignore"):
        n64 = lambda t: ref.head_fwd(np64(t), np64(w), np64(cos), np64(sin), at, half, norm, 1e-5)
        turned_back = ref._turn(np64(dy), np64(cos), np64(sin), at, half, back=True)
        if norm == "none":
            same(out, n64(x), "out")
            same(g["dq"], turned_back * np64(w), "dq")
            same(g["dq_weight"], (turned_back * np64(x)).sum((0, 1)), "dq_weight")
            return
        keep = np.isfinite(np64(x)).all(-1)
        same(out[torch.from_numpy(keep)], n64(x)[keep], "heads without one")
        want, _ = ref.head_bwd(np64(x), np64(w), np64(cos), np64(sin), at, half, norm, 1e-5, np64(dy))
        same(g["dq"][torch.from_numpy(keep)], want[keep], "dq of heads without one")


NO_EPS = [  # tokens, Hq, Hk, d
    (5, 3, 1, 64),     # lanes past the last head
    (3, 1, 1, 40),     # and past the head's channels
    (8000, 5, 3, 64),  # several heads a unit, the last unit of a token not full
    (5, 3, 1, 7),      # channel by channel
]


@pytest.mark.parametrize("tokens,Hq,Hk,d", NO_EPS)
@pytest.mark.parametrize("norm", ["rms", "l2"])
def test_no_eps(tokens, Hq, Hk, d, norm):
    """eps = 0: what a launch has beyond its heads adds nothing to the weights' gradients."""
    import kda_recurrent_state_gb300 as kda

    r = rand(tokens)
    q, k, wq, wk = r(tokens, Hq, d), r(tokens, Hk, d), r(d), r(d)
    dq, dk = r(tokens, Hq, d), r(tokens, Hk, d)
    kw = dict(norm=kda.KDA_NORM_RMS if norm == "rms" else kda.KDA_NORM_L2, eps=0.0)
    qo, ko = kda.kda_qk_norm_fwd(q, k, wq, wk, **kw)
    g = kda.kda_qk_norm_bwd(q, k, dq, dk, wq, wk, **kw)
    for name, x, w, dy, out in (("q", q, wq, dq, qo), ("k", k, wk, dk, ko)):
        same(out, ref.head_fwd(np64(x), np64(w), None, None, None, True, norm, 0.0), name)
        dx, dw = ref.head_bwd(np64(x), np64(w), None, None, None, True, norm, 0.0, np64(dy))
        same(g["d" + name], dx, "d" + name)
        same(g[f"d{name}_weight"], dw, f"d{name}_weight")


FAR = [(d, scale, eps) for d in (128, 40, 7, 1)
       for scale, eps in ((2.0 ** -50, 0.0), (2.0 ** -50, 2.0 ** -98), (2.0 ** 40, 1e-6))
       if d > 1 or scale < 1]  # one large channel: eps r^3 is below fp32's smallest ordinary number


@pytest.mark.parametrize("d,scale,eps", FAR)
@pytest.mark.parametrize("norm", ["rms", "l2"])
def test_norms_far_from_one(d, scale, eps, norm):
    """Heads whose norm is far from 1 (its square is still an ordinary fp32 number, its cube's inverse is not): the
    gradients are those of the definition.  One channel without eps has no gradient: exactly 0."""
    import kda_recurrent_state_gb300 as kda

    r = rand(d)
    x, w, dy = (1 + r(30, 3, d).abs()) * scale, r(d), r(30, 3, d)
    kw = dict(norm=kda.KDA_NORM_RMS if norm == "rms" else kda.KDA_NORM_L2, eps=eps)
    out, _ = kda.kda_qk_norm_fwd(x, None, w, **kw)
    g = kda.kda_qk_norm_bwd(x, None, dy, None, w, **kw)
    same(out, ref.head_fwd(np64(x), np64(w), None, None, None, True, norm, eps), "out")
    dx, dw = ref.head_bwd(np64(x), np64(w), None, None, None, True, norm, eps, np64(dy))
    if d == 1:  # r h - x r^3 <h, x> is eps r^3 h: the definition's own difference cancels even in 64 bits
        m = np64(x) ** 2 + eps
        dx = np64(dy) * np64(w) * eps * m ** -1.5
    same(g["dq"], dx, "dq")
    same(g["dq_weight"], dw, "dq_weight")
