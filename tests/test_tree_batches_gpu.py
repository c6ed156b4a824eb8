"""Draft trees and commits of more (session, head) items than CTAs run at once,
so that every CTA walks several: what it holds of an item (planes, barrier
phases, slots and paths read ahead) is used again for the next, with skipped
sessions between live ones.  Against the fp64 oracle, tolerances of
``test_tree_gpu``."""
import random

import numpy as np
import pytest
import torch

import gated_delta_rule_04_gb300 as kda
from kda_testlib import kda_params, rel_l2
from test_tree_gpu import DEV, TOL, Round, check_rows, path_to, tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_04_gb300 import build as kbuild
    kbuild.build()
    kda.lib()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n, R, H", [(131, 6, 7), (66, 24, 10), (50, 40, 7), (24, 64, 13)])
def test_several_trees_a_cta(io, n, R, H):
    assert n * H > 2 * (304 if R <= 32 else 152)
    rd = Round(io, n, R, H=H, seed=100 + R)
    rng = random.Random(R)
    parents = [tree(("bushy", "bushy", "chain", "star")[s % 4], R, rng) for s in range(n)]
    sent = rd.slots.clone()
    out = [s for s in range(n) if s % 5 == 3]                 # no slot: their rows stay as they are
    for s in out:
        sent[s] = (-1, n + 2, 2 ** 31 - 1)[s % 3]
    rows = [x.clone() for x in rd.rows]
    for x in rows:
        x[out] = float("nan")
    o = kda.kda_decode_tree(rd.kp, *rows, torch.tensor(parents, dtype=torch.int32, device=DEV), rd.S.to(DEV), rd.ring.to(DEV),
                            slots=sent.int().to(DEV), o=torch.full_like(rows[0], 7.0))
    assert bool((o[out] == 7.0).all())
    check_rows(rd, o, parents, skip={(s, r) for s in out for r in range(R)})


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("separate", [True, False])
def test_several_commits_a_cta(io, separate):
    n, R, H = 140, 12, 5
    assert n * H > 2 * 304
    rd = Round(io, n, R, H=H, seed=9)
    rng = random.Random(9)
    lens = [rng.choice([0, 1, 2, 3, 7, 8, 9, 12]) for _ in range(n)]
    paths = [(s, sorted(rng.sample(range(R), L))) for s, L in enumerate(lens)]
    path, sent = torch.full((n, R), -1, dtype=torch.int32), rd.slots.clone()
    for s, p in paths:
        path[s, :len(p)] = torch.tensor(p, dtype=torch.int32)
    skipped = set()
    for s in range(n):
        if s % 6 == 2 and lens[s]:                            # a bad node, a bad length, no slot
            path[s, rng.randrange(lens[s])] = rng.choice([-1, R, 99])
            skipped.add(s)
        elif s % 6 == 4:
            lens[s] = rng.choice([-1, R + 1, 2 ** 31 - 1, -2 ** 31])
            skipped.add(s)
        elif s % 6 == 5:
            sent[s] = rng.choice([-1, n + 2])
            skipped.add(s)
    S, ring = rd.S.to(DEV), rd.ring.to(DEV)
    out = dict(S_out=torch.full_like(S, 9.0), ring_out=torch.full_like(ring, 9.0)) if separate else {}
    q, k, v, z, b, _ = rd.rows
    S2, r2 = kda.kda_tree_commit(rd.kp, q, k, v, z, b, path.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), S, ring,
                                 slots=sent.int().to(DEV), **out)
    live = [p for p in paths if p[0] not in skipped]
    at = rd.slots[[s for s, _ in live]]
    ref = rd.oracle(live)
    assert rel_l2(S2.cpu()[at].double().numpy(), ref["S"]) <= TOL["f32"]
    np.testing.assert_array_equal(r2.cpu()[at].double().numpy(), ref["ring"])
    rest = sorted(set(range(n + 2)) - set(at.tolist()))
    if separate:
        assert bool((S2[rest] == 9.0).all()) and bool((r2[rest] == 9.0).all())
    else:
        assert torch.equal(S2[rest].cpu(), rd.S[rest]) and torch.equal(r2[rest].cpu(), rd.ring[rest])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("q_scale", [1e-6, 1.0, 3000.0, 1e12])
def test_any_q_scale(io, q_scale):
    """q^ is a unit vector times q_scale, whatever its size; the output's norm takes its eps
    from outside the range of the squares, so that the scale is seen."""
    rd = Round(io, 2, 11, seed=31)
    rd.p.q_scale, rd.p.norm_eps = q_scale, 1e-5 * q_scale * q_scale
    rd.kp = kda_params(rd.p, io)
    rng = random.Random(31)
    parents = [tree("bushy", 11, rng) for _ in range(2)]
    check_rows(rd, rd.decode(parents), parents)
