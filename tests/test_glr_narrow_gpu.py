"""The gated linear recurrence over many tiles whose rows are no tensor copies: a warp's own copies take the
place of rows that its lanes have just read, tile after tile in the same CTA.  Tokens whose channels are taken one
by one."""
import pytest
import torch

import gated_delta_rule_04_gb300 as kda
from glr_ref import SUM_TOL, close, make_inputs
from test_glr_gpu import GRADS, IO, cumsum, dev, forward64, params, tokens_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_04_gb300 import build as kbuild
    kbuild.build()
    kda.lib()


def gradients64(i, n, s, j, before, h):
    """As glr_ref.gradients on the GPU for n sequences of one length, side by side."""
    C = i["C"]
    z, G, a = j["z"].double(), j["do"].double(), s["a"].view(n, -1, C)
    e = torch.sigmoid(z)
    out = {"dz": G * h * (e + z * e * torch.sigmoid(-z))}
    G = G * z * e
    by, carry = G.view(n, -1, C), j["dS"].double().clone()
    for t in range(by.shape[1] - 1, -1, -1):
        by[:, t] += carry
        carry = a[:, t] * by[:, t]
    dA = G * (s["a"] * before * s["la"] - s["a"] ** 2 * s["v"] * j["x"].double() * s["la"] / s["m"])
    out.update(dx=G * s["m"] * s["v"], di=G * s["b"] * s["v_"], dr=dA * s["w_"], dS_in=carry)
    out.update(dA_log=dA.sum(0), dr_bias=out["dr"].sum(0), di_bias=out["di"].sum(0))
    return out


@pytest.mark.parametrize("io, C, pad", [("f32", 40, 0), ("f32", 63, 1), ("f32", 64, 1), ("bf16", 40, 0), ("bf16", 63, 0), ("bf16", 65, 0),
                                        ("bf16", 64, 2)])
def test_rows_that_follow_one_another(io, C, pad):
    """At least six tiles a CTA, whole and partial ones, with an output gate; the same bits whatever ran before in the
    workspace.  The parameters' gradients are sums of T terms: (T / 700)^1/2 times the usual tolerance."""
    T, n = 140000, 40
    cu = cumsum([T // n] * n)
    i = make_inputs(T, n, C, IO[io], 60 + C + pad)
    wide = {k: torch.full((T, C + pad), float("nan"), dtype=IO[io], device=DEV)[:, :C].copy_(i[k]) for k in ("x", "r", "i", "z", "do")}
    p, S = params(i, io), dev(i["S"])
    st = torch.empty(-(-T // kda.KDA_GLR_CHUNK), C, device=DEV)
    ws = torch.empty(kda.kda_glr_backward_workspace_bytes(p, n, T), dtype=torch.uint8, device=DEV)
    runs = []
    for fill in (255, 0, 1):
        ws.fill_(fill)
        o, So = kda.kda_glr_prefill(p, wide["x"], wide["r"], wide["i"], cu, z=wide["z"], S_in=S, states=st, workspace=ws)
        g = kda.kda_glr_backward(p, wide["x"], wide["r"], wide["i"], cu, st, wide["do"], z=wide["z"], S_in=S, dS_out=dev(i["dS"]),
                                 workspace=ws)
        assert kda.kda_workspace_status(ws) == kda.KDA_OK
        runs.append([o, So, st.clone()] + [getattr(g, k) for k in GRADS])
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)
    s, j, wo, wS, before, h = forward64(i, cu)
    close("o", o, wo.cpu())
    close("S", So, wS.cpu())
    close("states", st, before[::kda.KDA_GLR_CHUNK].cpu())
    want = gradients64(i, n, s, j, before, h)
    for k in GRADS:
        close(k, getattr(g, k), want[k].cpu(), SUM_TOL * (T / 700) ** 0.5 if k in ("dA_log", "dr_bias", "di_bias") else None)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("C", [1, 31, 129])
@pytest.mark.parametrize("faster", [False, True])
def test_tokens_of_single_channels(io, C, faster):
    """Channels that are taken one by one (odd rows): decays that no exponential is needed for, and one channel
    among them whose decay may need it."""
    n, R = 3, 5
    i = make_inputs(n * R, n, C, IO[io], 80 + C)
    i["A_log"] -= 1.0                                    # exp(A_log) is at most e^-1
    if faster:
        i["A_log"][C // 2] = 1.5
    x, r, s, z = (dev(i[k]).view(n, R, C) for k in ("x", "r", "i", "z"))
    wo, wS = tokens_ref(i, n, R, i["S"], [range(R)] * n)
    S = dev(i["S"])
    o = kda.kda_glr_decode(params(i, io), x, r, s, S, z=z)
    close("o", o, wo)
    close("S", S, wS)
