"""The 64-bit definitions that the gated linear recurrence and the verification of
drafts are tested against: gradients against differences, and the tokens'
distribution against the target's."""
import pytest
import torch

from glr_ref import gradients, make_inputs, mixer, verify


def loss(i, cu):
    o, S = mixer(i, cu)
    return float((o * i["do"].double()).sum() + (0 if i["dS"] is None else (S * i["dS"].double()).sum()))


@pytest.mark.parametrize("state, bias, gate", [(True, True, True), (False, False, False)])
def test_gradients_are_those_of_differences(state, bias, gate):
    """Central differences along one random direction per input: with steps of 1e-5 in 64 bits they
    are good to about 1e-10 (step^2) + 1e-11 (rounding / step)."""
    cu = [0, 9, 9, 10, 31]
    i = make_inputs(31, 4, 5, torch.float32, 1, state, bias, gate)
    i = {k: v.double() if torch.is_tensor(v) else v for k, v in i.items()}
    want = gradients(i, cu)
    g = torch.Generator().manual_seed(2)
    for name, grad in (("x", "dx"), ("r", "dr"), ("i", "di"), ("z", "dz"), ("S", "dS_in"), ("A_log", "dA_log"),
                       ("r_bias", "dr_bias"), ("i_bias", "di_bias")):
        if i[name] is None:
            continue
        d, e = torch.randn(i[name].shape, generator=g, dtype=torch.float64), 1e-5
        diff = (loss({**i, name: i[name] + e * d}, cu) - loss({**i, name: i[name] - e * d}, cu)) / (2 * e)
        assert abs(diff - float((want[grad] * d).sum())) < 1e-7 * max(1.0, abs(diff)), name


@pytest.mark.parametrize("drawn", [True, False])
def test_verified_tokens_follow_the_target(drawn):
    """Two siblings and the token behind them: the first emitted token has the target's
    distribution whatever the drafter's.  20000 rounds; a count's deviation is below 5 standard
    deviations, sqrt(n p (1 - p)), but for odds of 6e-7 each."""
    n, V = 20000, 5
    g = torch.Generator().manual_seed(3)
    p0 = torch.tensor([0.4, 0.3, 0.15, 0.1, 0.05])
    q0 = torch.tensor([0.1, 0.2, 0.3, 0.15, 0.25])
    p = p0.expand(n, 2, V)
    tokens = torch.multinomial(q0.expand(2 * n, V), 1, generator=g).view(n, 2) if drawn else torch.tensor([[3, 1]]).expand(n, 2)
    q = q0.expand(n, 2, V) if drawn else None
    paths, nxt = verify(p, tokens.int(), torch.tensor([[-1, -1]]).expand(n, 2), torch.rand(n, 2, generator=g),
                        torch.rand(n, generator=g), q=q, p_last=p[:, 0], q_last=None if q is None else q[:, 0], max_len=1)
    first = torch.tensor([int(tokens[s, path[0]]) if path else nxt[s] for s, path in enumerate(paths)])
    count = torch.bincount(first, minlength=V).double()
    sd = (n * p0.double() * (1 - p0.double())).sqrt()
    assert ((count - n * p0.double()).abs() < 5 * sd).all(), (count / n, p0)
    assert any(paths) and not all(paths)
