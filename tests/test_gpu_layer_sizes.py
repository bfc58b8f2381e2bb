"""Parity of the operators around the recurrence at sizes that reach what their launch rules choose for large calls:
several heads a unit and more units than blocks, pieces of many tokens, whole sequences a CTA, several sessions a
thread -- each with remainders, against the 64-bit definitions.

Tolerances (relative 2-norm) as for the small sizes: fp32 without a recurrence 2e-6, the scan 2e-5, bf16 outputs
(rounded once, 2^-9.2 in the mean square) 2e-3.  Sums over n tokens or heads of random signs carry a rounding error of
2^-24 times the size of their partial sums, which a tree of short runs keeps below the flat bound."""
import numpy as np
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
FLAT, SCAN, BF16 = 2e-6, 2e-5, 2e-3
bf16, f32 = torch.bfloat16, torch.float32


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def check(got, want, tol, what):
    g = np64(got).reshape(want.shape)
    rel = np.linalg.norm(g - want) / np.linalg.norm(want)
    assert rel <= tol, f"{what}: rel {rel:.2e} (<= {tol})"


def rand(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *shape: torch.randn(*shape, generator=g, device="cuda")


def tol_of(dtype, tol):
    return BF16 if dtype == bf16 else tol


def cu_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int64, device="cuda")


# ---------------------------------------------------------------- head norm and rotation
@pytest.mark.parametrize("tokens,Hq,Hk,d,rot,half,dt,gt", [
    (25001, 5, 2, 128, 64, True, bf16, bf16),    # four heads a unit, 5 = 4 + 1; gradient units past one per block
    (25001, 5, 2, 128, 128, False, bf16, f32),
    (5003, 3, 2, 64, 40, True, f32, f32),        # two heads a unit, halves inside a lane's channels
    (9001, 9, 0, 80, 32, True, f32, bf16),       # 10 of 16 lanes, no keys
    (9001, 6, 7, 31, 10, False, f32, f32),       # channel by channel
])
def test_heads(tokens, Hq, Hk, d, rot, half, dt, gt):
    import kda_recurrent_state_gb300 as kda

    r = rand(tokens + d)
    q, k = r(tokens, Hq, d).to(dt), r(tokens, Hk, d).to(dt) if Hk else None
    wq, wk = r(d), r(d) if Hk else None
    ang = r(99, rot // 2) * 3
    cos, sin = ang.cos(), ang.sin()
    pos = torch.arange(tokens, device="cuda") * 7 % 99
    dq, dk = r(tokens, Hq, d).to(gt), r(tokens, Hk, d).to(gt) if Hk else None
    kw = dict(norm=kda.KDA_NORM_RMS, layout=kda.KDA_ROT_HALF if half else kda.KDA_ROT_PAIRS, eps=1e-5)
    qo, ko = kda.kda_qk_norm_fwd(q, k, wq, wk, cos, sin, pos, out_dtype=gt, **kw)
    g = kda.kda_qk_norm_bwd(q, k, dq, dk, wq, wk, cos, sin, pos, **kw)
    at = pos.cpu().numpy()
    for n, x, w, dy, out in (("q", q, wq, dq, qo), ("k", k, wk, dk, ko)):
        if x is None:
            continue
        a = (np64(x), np64(w), np64(cos), np64(sin), at, half, "rms", 1e-5)
        check(out, ref.head_fwd(*a), tol_of(gt, FLAT), n)
        dx, dw = ref.head_bwd(*a, np64(dy))
        check(g["d" + n], dx, tol_of(gt, FLAT), "d" + n)
        check(g[f"d{n}_weight"], dw, FLAT, f"d{n}_weight")
    assert kda.kda_get_device_status() == 0


# ---------------------------------------------------------------- convolution
def pieces(total, seed):
    """Sequence lengths of very different sizes that fill `total` tokens, empty ones among them."""
    r = np.random.default_rng(seed)
    lens = [0, 1]
    while sum(lens) < total:
        lens.append(min(total - sum(lens), int(np.exp(r.uniform(0, np.log(total / 3))))))
    return lens + [0]


@pytest.mark.parametrize("total,D,W,dt,gt", [
    (15000, 1024, 4, bf16, bf16),  # 25 rows a thread; gradients in 300 pieces
    (15000, 1024, 4, bf16, f32),
    (30000, 256, 4, f32, f32),     # gradients in more than 1000 pieces, summed in 32 runs
    (30000, 258, 3, bf16, f32),    # two channels a thread
    (30000, 257, 2, f32, bf16),    # one
])
def test_convolution(total, D, W, dt, gt):
    import kda_recurrent_state_gb300 as kda

    r = rand(total + D)
    lens = pieces(total, D)
    x, w, b, st = r(total, D).to(dt), r(D, W) * 0.5, r(D), r(len(lens), W - 1, D).to(dt)
    dy, dl = r(total, D).to(gt), r(len(lens), W - 1, D)
    cu = cu_of(lens)
    y, last = kda.kda_conv_fwd(x, w, b, st, cu_seqlens=cu, out_dtype=gt)
    ry, rl = ref.conv_fwd(np64(x), np64(w), np64(b), np64(st), lens, True)
    check(y, ry, tol_of(gt, FLAT), "y")
    assert np.array_equal(np64(last), rl)
    g = kda.kda_conv_bwd(x, w, b, dy, st, dl, cu_seqlens=cu)
    want = ref.conv_bwd(np64(x), np64(w), np64(b), np64(st), lens, True, np64(dy), np64(dl))
    check(g["dx"], want["dx"], tol_of(gt, FLAT), "dx")
    for n in ("dweight", "dbias", "d_init"):
        check(g[n], want[n], FLAT, n)


@pytest.mark.parametrize("B,D,W,dt", [
    (67, 40008, 4, bf16),  # 8 sessions a thread, 3 in the last one
    (67, 9001, 3, f32),
    (21, 16384, 2, f32),   # 2
])
def test_convolution_step(B, D, W, dt):
    import kda_recurrent_state_gb300 as kda

    r = rand(B + D)
    x, w, b, st = r(B, D).to(dt), r(D, W) * 0.5, r(D), r(B, W - 1, D).to(dt)
    ry, rl = ref.conv_fwd(np64(x), np64(w), np64(b), np64(st), [1] * B, True)
    y = kda.kda_conv_step(x, w, b, st, out_dtype=f32)
    check(y, ry, FLAT, "y")
    assert np.array_equal(np64(st), rl)


# ---------------------------------------------------------------- scan
@pytest.mark.parametrize("B,T,D,N,G,dt,gt", [
    (12, 70, 1024, 16, 1, bf16, bf16),  # 96 (sequence, 128 channels): fewer channels a CTA fill the last wave better
    (7, 45, 1000, 24, 2, f32, f32),     # 112 (sequence, 64 channels)
    (20, 37, 160, 64, 1, f32, bf16),    # 100 (sequence, 32 channels)
    (33, 30, 520, 5, 1, bf16, f32),     # 99 (sequence, 256 channels), the last of 8
])
def test_scan_whole_sequences(B, T, D, N, G, dt, gt):
    import kda_recurrent_state_gb300 as kda

    r = rand(B + D)
    v = dict(u=r(B, T, D).to(dt), delta=(r(B, T, D) - 2).to(dt), A=-torch.exp(r(D, N)), B=r(B, T, G, N).to(dt),
             C=r(B, T, G, N).to(dt), skip=r(D), z=r(B, T, D).to(dt), bias=r(D) * 0.3, init=r(B, D, N))
    dout, dl = r(B, T, D).to(gt), r(B, D, N)
    want = {k: np64(t) for k, t in v.items()}
    for k in ("u", "delta", "z"):
        want[k] = want[k].reshape(-1, D)
    for k in ("B", "C"):
        want[k] = want[k].reshape(-1, G, N)
    want.update(softplus=True, lens=[T] * B)
    x, rest = [v[k] for k in ("u", "delta", "A", "B", "C")], [v[k] for k in ("skip", "z", "bias", "init")]
    out, last = kda.kda_ssm_fwd(*x, *rest, out_dtype=gt)
    ro, rl, _, _ = ref.scan_fwd(want)
    check(out, ro, tol_of(gt, SCAN), "out")
    check(last, rl, SCAN, "final state")
    g = kda.kda_ssm_bwd(*x, dout, *rest, dl)
    w = ref.scan_bwd(want, np64(dout).reshape(-1, D), np64(dl))
    for n in ("du", "ddelta", "dz"):
        check(g[n], w[n], tol_of(gt, SCAN), n)
    for n in ("dA", "dB", "dC", "dD", "ddelta_bias", "d_init"):
        check(g[n], w[n], SCAN, n)


@pytest.mark.parametrize("S,D,N,G,dt", [
    (77, 8200, 4, 1, f32),  # four sessions a thread, one in the last one, for every number of lanes a channel
    (66, 5000, 7, 1, bf16),
    (70, 2500, 16, 2, bf16),
    (71, 1300, 32, 1, f32),
    (70, 650, 64, 1, bf16),
])
def test_scan_step(S, D, N, G, dt):
    import kda_recurrent_state_gb300 as kda

    r = rand(S + D)
    v = dict(u=r(S, D).to(dt), delta=r(S, D).to(dt), A=-torch.exp(r(D, N)), B=r(S, G, N).to(dt), C=r(S, G, N).to(dt),
             skip=r(D), z=r(S, D).to(dt), bias=r(D), init=r(S, D, N))
    ro, rl, _, _ = ref.scan_fwd(dict({k: np64(t) for k, t in v.items()}, softplus=True, lens=[1] * S))
    state = v["init"].clone()
    out = kda.kda_ssm_step(v["u"], v["delta"], v["A"], v["B"], v["C"], v["skip"], v["z"], v["bias"], state, out_dtype=f32)
    check(out, ro, SCAN, "out")
    check(state, rl, SCAN, "state")
