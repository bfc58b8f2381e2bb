"""Out-of-bounds writes of the operators around the recurrence, without a sanitizer: every output and workspace of a C
call lies between guard regions of NaN, which must be unchanged; every output value must have been written."""
import pytest
import torch

pytestmark = pytest.mark.gpu
GUARD = 4096  # elements on each side, a multiple of 16 bytes
bf16, f32 = torch.bfloat16, torch.float32


class Guards:
    def __init__(self):
        self.all = []

    def __call__(self, *shape, dtype=f32, like=None, written=True):
        """The address of an array between guards, holding NaN (or a copy of `like`)."""
        n = 1
        for d in shape:
            n *= d
        buf = torch.full((GUARD + n + GUARD,), float("nan"), dtype=dtype, device="cuda")
        if like is not None:
            buf[GUARD:GUARD + n] = like.reshape(-1)
        self.all.append((buf, n, written))
        return buf.data_ptr() + GUARD * buf.element_size()

    def workspace(self, size):
        return self((size + 3) // 4, written=False)

    def intact(self):
        torch.cuda.synchronize()
        for i, (buf, n, written) in enumerate(self.all):
            assert torch.isnan(buf[:GUARD]).all() and torch.isnan(buf[GUARD + n:]).all(), i
            assert not written or not torch.isnan(buf[GUARD:GUARD + n]).any(), i


def setup(seed, dt, lens):
    from kda_recurrent_state_gb300 import binding

    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    code = lambda t: binding.KDA_BF16 if t == bf16 else binding.KDA_F32
    return binding.lib(), r, torch.tensor(cu, dtype=torch.int64, device="cuda"), cu[-1], code(dt), code


P = lambda t: t.data_ptr()


@pytest.mark.parametrize("D,W", [(257, 4), (66, 3), (264, 2), (1, 4)])
@pytest.mark.parametrize("dt,ot", [(bf16, bf16), (bf16, f32), (f32, bf16), (f32, f32)])
def test_convolution(D, W, dt, ot):
    lens = [5, 0, 1, 130, 2]
    L, r, cu, T, i, code = setup(D, dt, lens)
    N, o = len(lens), code(ot)
    x, w, b, st = r(T, D).to(dt), r(D, W), r(D), r(N, W - 1, D).to(dt)
    dy, dl = r(T, D).to(ot), r(N, W - 1, D)
    g = Guards()
    assert L.kda_conv_fwd(P(x), D, P(w), P(b), P(st), g(T, D, dtype=ot), g(N, W - 1, D, dtype=dt), P(cu), N, T, D, W, 1, i, o,
                          None) == 0
    assert L.kda_conv_step(P(x), D, P(w), P(b), g(N, W - 1, D, dtype=dt, like=st), g(N, D, dtype=ot), N, D, W, 1, i, o, None) == 0
    size = L.kda_conv_bwd_workspace_size(T, D, W)
    assert L.kda_conv_bwd(P(x), D, P(w), P(b), P(st), P(dy), P(dl), P(cu), N, T, D, W, 1, g(T, D, dtype=ot), g(D, W), g(D),
                          g(N, W - 1, D), i, o, g.workspace(size), size, None) == 0
    g.intact()


@pytest.mark.parametrize("D,N,G", [(37, 5, 1), (40, 16, 1), (72, 24, 3), (9, 64, 9), (130, 33, 2), (8, 4, 1)])
@pytest.mark.parametrize("dt,ot", [(bf16, bf16), (f32, f32), (f32, bf16)])
def test_scan(D, N, G, dt, ot):
    lens = [5, 0, 1, 330, 66]
    L, r, cu, T, i, code = setup(D, dt, lens)
    S, o = len(lens), code(ot)
    u, delta, z, B, C = r(T, D).to(dt), (r(T, D) - 2).to(dt), r(T, D).to(dt), r(T, G, N).to(dt), r(T, G, N).to(dt)
    A, skip, bias, init, dy, dl = -torch.exp(r(D, N)), r(D), r(D), r(S, D, N), r(T, D).to(ot), r(S, D, N)
    head = (P(u), D, P(delta), D, P(A), P(B), G * N, P(C), G * N, P(skip), P(z), D, P(bias), 1)
    g = Guards()
    size = L.kda_ssm_fwd_workspace_size(S, T, D, N, G, 1)
    assert L.kda_ssm_fwd(*head, P(init), g(T, D, dtype=ot), g(S, D, N), P(cu), S, T, D, N, G, i, o, g.workspace(size), size,
                         None) == 0
    assert L.kda_ssm_step(*head, g(S, D, N, like=init), g(S, D, dtype=ot), S, D, N, G, i, o, None) == 0
    size = L.kda_ssm_bwd_workspace_size(S, T, D, N, G, 1)
    assert L.kda_ssm_bwd(*head, P(init), P(dy), P(dl), P(cu), S, T, D, N, G, g(T, D, dtype=ot), g(T, D, dtype=ot), g(D, N),
                         g(T, G, N), g(T, G, N), g(D), g(T, D, dtype=ot), g(D), g(S, D, N), i, o, g.workspace(size), size,
                         None) == 0
    g.intact()


@pytest.mark.parametrize("d,rot,layout", [(128, 64, 0), (40, 10, 0), (80, 30, 1), (7, 4, 0), (256, 256, 1), (8, 0, 0)])
@pytest.mark.parametrize("dt,ot", [(bf16, bf16), (f32, f32), (bf16, f32)])
@pytest.mark.parametrize("norm", [0, 1])
def test_heads(d, rot, layout, dt, ot, norm):
    T, Hq, Hk = 333, 5, 3
    L, r, _, _, i, code = setup(d, dt, [])
    o = code(ot)
    q, k, wq, wk, ang = r(T, Hq, d).to(dt), r(T, Hk, d).to(dt), r(d), r(d), r(50, max(rot // 2, 1))
    cos, sin, pos = ang.cos(), ang.sin(), torch.arange(T, device="cuda") % 50
    dq, dk = r(T, Hq, d).to(ot), r(T, Hk, d).to(ot)
    x = (P(q), Hq * d, P(k), Hk * d)
    tables = (P(wq), P(wk), P(cos), P(sin), P(pos), 50)
    tail = (T, Hq, Hk, d, rot, layout, norm, 1e-6, i, o)
    g = Guards()
    assert L.kda_qk_norm_fwd(*x, *tables, g(T, Hq, d, dtype=ot), g(T, Hk, d, dtype=ot), *tail, None) == 0
    size = L.kda_qk_norm_bwd_workspace_size(d)
    assert L.kda_qk_norm_bwd(*x, P(dq), P(dk), *tables, g(T, Hq, d, dtype=ot), g(T, Hk, d, dtype=ot), g(d), g(d), *tail,
                             g.workspace(size), size, None) == 0
    g.intact()
