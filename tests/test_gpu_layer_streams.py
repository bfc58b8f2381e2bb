"""The operators around the recurrence run on the stream that is current when they are called."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def rand(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *shape: torch.randn(*shape, generator=g, device="cuda")


def test_launches_follow_the_current_stream():
    """Every call on a side stream whose inputs are filled there only after a while: a launch on any other stream
    would read the NaN that the buffers hold until then."""
    import kda_recurrent_state_gb300 as kda

    r = rand(11)
    L = (3, 260)
    src = dict(x=r(*L, 256), w=r(256, 4), b=r(256), rows=r(3, 3, 256), dy=r(*L, 256), delta=r(*L, 256) - 2,
               A=-torch.exp(r(256, 16)), B=r(*L, 1, 16), C=r(*L, 1, 16), D=r(256), h=r(3, 256, 16), q=r(780, 2, 128),
               k=r(780, 1, 128), wq=r(128), dq=r(780, 2, 128), dk=r(780, 1, 128))

    def calls(v):
        one = lambda n: v[n][:, 0]
        y, last = kda.kda_conv_fwd(v["x"], v["w"], v["b"], v["rows"])
        out, state = kda.kda_ssm_fwd(v["x"], v["delta"], v["A"], v["B"], v["C"], v["D"], v["dy"], v["b"], v["h"])
        q, k = kda.kda_qk_norm_fwd(v["q"], v["k"], v["wq"])
        g = [kda.kda_conv_bwd(v["x"], v["w"], v["b"], v["dy"], v["rows"]),
             kda.kda_ssm_bwd(v["x"], v["delta"], v["A"], v["B"], v["C"], v["dy"], v["D"], None, v["b"], v["h"]),
             kda.kda_qk_norm_bwd(v["q"], v["k"], v["dq"], v["dk"], v["wq"])]
        steps = [kda.kda_conv_step(one("x"), v["w"], v["b"], v["rows"]),
                 kda.kda_ssm_step(one("x"), one("delta"), v["A"], one("B"), one("C"), v["D"], one("dy"), v["b"], v["h"])]
        return [y, last, out, state, q, k, *steps, v["rows"], v["h"],
                *(t for d in g for t in d.values() if t is not None)]

    want = calls({n: t.clone() for n, t in src.items()})
    late = {n: torch.full_like(t, float("nan")) for n, t in src.items()}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)  # about 0.1 s: longer than all the calls take to be made
        for n, t in src.items():
            late[n].copy_(t)
        got = calls(late)
    s.synchronize()
    assert len(got) == len(want) == 25
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), i
