"""The selective scan with decay rates down to fp32's lowest value, and steps of exactly 0: exp(0 A) is 1 for every
finite A, whatever A log2 e is.

Tolerance (relative 2-norm): as for ordinary rates, 2e-5 over at most 300 tokens."""
import numpy as np
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
SCAN = 2e-5
LOWEST = torch.finfo(torch.float32).min


def np64(t):
    return t.detach().double().cpu().numpy()


def check(got, want, what):
    g = np64(got).reshape(want.shape)
    rel = np.linalg.norm(g - want) / np.linalg.norm(want)
    assert rel <= SCAN, f"{what}: rel {rel:.2e}"


@pytest.mark.parametrize("T", [300, 37])  # in segments, and whole
@pytest.mark.parametrize("D,N", [(40, 16), (33, 5), (16, 64)])
def test_lowest_rates(T, D, N):
    import kda_recurrent_state_gb300 as kda

    g = torch.Generator(device="cuda").manual_seed(T + D)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    u, B, C, init, dout = r(1, T, D), r(1, T, 1, N), r(1, T, 1, N), r(1, D, N), r(1, T, D)
    A = -torch.exp(r(D, N))
    A[:, ::2] = LOWEST
    delta = torch.rand(1, T, D, generator=g, device="cuda") * 0.1
    delta[0, torch.rand(T, generator=g, device="cuda") < 0.7] = 0  # most tokens leave the states alone
    delta[0, :, 0] = 0                                              # one channel keeps its initial state to the end
    v = dict(u=np64(u)[0], delta=np64(delta)[0], A=np64(A), B=np64(B)[0], C=np64(C)[0], skip=None, z=None, bias=None,
             init=np64(init), softplus=False, lens=[T])
    ro, rl, _, _ = ref.scan_fwd(v)
    out, last = kda.kda_ssm_fwd(u, delta, A, B, C, init_state=init, delta_softplus=False)
    check(out, ro, "out")
    check(last, rl, "final state")
    assert torch.equal(last[:, 0], init[:, 0])
    state = init.clone()
    steps = torch.stack([kda.kda_ssm_step(u[:, t], delta[:, t], A, B[:, t], C[:, t], None, None, None, state,
                                          delta_softplus=False) for t in range(T)], 1)
    check(steps, ro, "single tokens")
    check(state, rl, "their state")
    got = kda.kda_ssm_bwd(u, delta, A, B, C, dout, init_state=init, delta_softplus=False)
    w = ref.scan_bwd(v, np64(dout)[0], None)
    for n in ("du", "dA", "dB", "dC", "d_init"):  # a step's own gradient is A times the state: past fp32's range
        check(got[n], w[n], n)
