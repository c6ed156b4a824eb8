"""Drawn calls of kda_draft_verify against the walk in 64 bits: sizes over their logarithms, any shape of tree,
rows off 16 bytes, shared or apart, entries that count as zero."""
import math
import random

import pytest
import torch

import gated_delta_rule_04_gb300 as kda
from glr_ref import make_draft, verify

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_04_gb300 import build as kbuild
    kbuild.build()
    kda.lib()


def log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def placed(rng, t):
    """The rows on the device, with a gap behind each and from any element on."""
    if t is None:
        return None
    gap, off = rng.choice([0, 0, 1, 3, 8]), rng.choice([0, 0, 1, 5, 8])
    *lead, V = t.shape
    flat = torch.full((off + math.prod(lead) * (V + gap),), float("nan"), dtype=t.dtype, device=DEV)
    view = flat[off:].view(*lead, V + gap)[..., :V]
    view.copy_(t)
    return view


@pytest.mark.parametrize("seed", range(40))
def test_drawn_calls(seed):
    rng = random.Random(seed)
    for _ in range(10):
        V, R = log_int(rng, 1, 60000), log_int(rng, 1, 64)
        n = log_int(rng, 1, max(1, min(1500, 300000 // (V * R))))
        drawn, last = rng.random() < 0.7, rng.random() < 0.6
        d = make_draft(n, R, V, rng.choice([torch.float32, torch.bfloat16]), rng.randrange(1 << 30),
                       rng.choice(["chain", "bushy", "star"]), drawn, last)
        d["u"] = d["u"] ** rng.choice([0.2, 1, 3])
        if rng.random() < 0.3:
            for k in ("p", "p_last", "q", "q_last"):
                if d[k] is not None:
                    bad = torch.rand(d[k].shape, generator=torch.Generator().manual_seed(rng.randrange(1 << 30)))
                    d[k][bad < 0.01], d[k][bad > 0.98] = float("nan"), -0.5
        max_len = rng.choice([None, None, 1, R, 64])
        p = placed(rng, d["p"])
        path, length, nxt = kda.kda_draft_verify(p, d["tokens"].to(DEV), d["parents"].to(DEV), d["u"].to(DEV), d["u_next"].to(DEV),
                                                 q=placed(rng, d["q"]), p_last=placed(rng, d["p_last"]),
                                                 q_last=placed(rng, d["q_last"]), max_len=max_len)
        wp, wn = verify(**d, max_len=max_len)
        what = dict(n=n, R=R, V=V, drawn=drawn, last=last, max_len=max_len)
        assert length.tolist() == [len(w) for w in wp], what
        assert path.tolist() == [w + [-1] * (path.shape[1] - len(w)) for w in wp], what
        assert nxt.tolist() == wn, what
