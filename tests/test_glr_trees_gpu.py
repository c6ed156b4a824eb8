"""A round over draft trees with the gated linear recurrence: the tree's rows as straight runs from one state, its
verification, and the commit of the accepted paths."""
import pytest
import torch

import gated_delta_rule_04_gb300 as kda
from glr_ref import close, make_draft, make_inputs, steps, verify
from test_glr_gpu import IO, dev, params

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_04_gb300 import build as kbuild
    kbuild.build()
    kda.lib()


def ways(parents):
    """The nodes from the root to each leaf."""
    out = []
    for leaf in set(range(len(parents))) - set(parents):
        way = [leaf]
        while parents[way[0]] >= 0:
            way.insert(0, parents[way[0]])
        out.append(way)
    return out


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", ["bushy", "star"])
@pytest.mark.parametrize("C", [40, 129])
def test_a_round_over_trees(io, shape, C):
    n, R, slots_n, V = 7, 11, 10, 50
    i = make_inputs(n * R, slots_n, C, IO[io], 90 + C)
    d = make_draft(n, R, V, torch.float32, 91, shape)
    d["u"] *= 0.5
    slots = torch.tensor([4, 9, 0, 7, 1, 3, 8], dtype=torch.int32)
    # rows: every run reads its session's state
    runs = [(s, way) for s in range(n) for way in ways(d["parents"][s].tolist())]
    depth = max(len(way) for _, way in runs)
    assert len(runs) > n
    at = torch.tensor([[s * R + r for r in way] + [s * R] * (depth - len(way)) for s, way in runs], device=DEV)
    x, r, g, z = (dev(i[k])[at] for k in ("x", "r", "i", "z"))
    S, of = dev(i["S"]), dev(slots[[s for s, _ in runs]])
    o = kda.kda_glr_decode(params(i, io), x, r, g, S, z=z, slots=of, keep_state=True)
    assert torch.equal(S.cpu(), i["S"])
    # each node from its parent's state, in 64 bits
    t, h = steps(i), torch.empty(n, R, C, dtype=torch.float64)
    for s in range(n):
        for node, parent in enumerate(d["parents"][s].tolist()):
            before = i["S"][slots[s]].double() if parent < 0 else h[s, parent]
            h[s, node] = t["a"][s * R + node] * before + t["b"][s * R + node]
    zz = i["z"].double().view(n, R, C)
    want = h * zz * torch.sigmoid(zz)
    got = torch.full((n, R, C), float("nan"), dtype=IO[io])
    for k, (s, way) in enumerate(runs):
        for j, node in enumerate(way):
            assert torch.isnan(got[s, node]).all() or torch.equal(got[s, node], o[k, j].cpu())    # of two runs: the same
            got[s, node] = o[k, j].cpu()
    close("o", got, want)
    # the accepted paths
    on = {k: dev(v) for k, v in d.items()}
    path, length, token = kda.kda_draft_verify(on["p"], on["tokens"], on["parents"], on["u"], on["u_next"], q=on["q"],
                                               p_last=on["p_last"], q_last=on["q_last"])
    wp, wn = verify(**d)
    assert length.tolist() == [len(w) for w in wp] and token.tolist() == wn and max(map(len, wp)) > (shape == "bushy")
    rows = [dev(i[k]).view(n, R, C) for k in ("x", "r", "i")]
    kda.kda_glr_commit(params(i, io), *rows, path, length, S, slots=dev(slots))
    end = i["S"].double()
    for s, way in enumerate(wp):
        if way:
            end[slots[s]] = h[s, way[-1]]
    close("S", S, end)
    untouched = [k for k in range(slots_n) if k not in slots.tolist()]
    assert torch.equal(S[untouched].cpu(), i["S"][untouched])
