"""Draft trees over the KDA state (kda_decode_tree, kda_tree_commit): every
node against the fp64 oracle run over the node's path, and the state after an
accepted path.

Tolerances (relative 2-norm): fp32 outputs and states 2e-5, a few hundred
roundings of 2^-24 along a value's history; bf16 outputs 2^-8 for the final
rounding plus 4 * 2^-11 for 11-bit operands of tensor-core products."""
import random

import numpy as np
import pytest
import torch

import gated_delta_rule_04_gb300 as kda
import kda_synth
from kda_testlib import kda_params, oracle_run, rel_l2

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = {"f32": 2e-5, "bf16": 2 ** -8 + 4 * 2 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_04_gb300 import build as kbuild
    kbuild.build()
    kda.lib()


def tree(kind, R, rng):
    if kind == "chain":
        return list(range(-1, R - 1))
    if kind == "star":
        return [-1] * R
    return [-1] + [rng.randint(-1, r - 1) for r in range(1, R)]


def path_to(parents, r):
    p = []
    while r >= 0:
        p.append(r)
        r = parents[r]
    return p[::-1]


class Round:
    """A round of n sessions x R nodes at slots of a pool."""

    def __init__(self, io, n, R, H=2, seed=1, gate_kind=0, spare=2):
        self.io, self.n, self.R, self.H = io, n, R, H
        self.p = kda_synth.draw_params(H, seed)
        self.p.gate_kind = gate_kind
        self.tk = kda_synth.draw_tokens(n * R, H, seed + 1, kda_synth.io_dtype(io))
        g = torch.Generator().manual_seed(seed + 2)
        self.S = torch.randn(n + spare, H, 128, 128, generator=g) * 0.05
        self.ring = torch.randn(n + spare, 3, 3, H * 128, generator=g).to(kda_synth.io_dtype(io))
        self.slots = torch.randperm(n + spare, generator=g)[:n]
        self.kp = kda_params(self.p, io)
        self.rows = [t.reshape(n, R, -1).to(DEV) for t in self.tk.fields()]

    def decode(self, parents, **kw):
        return kda.kda_decode_tree(self.kp, *self.rows, torch.tensor(parents, dtype=torch.int32, device=DEV), self.S.to(DEV),
                                   self.ring.to(DEV), slots=self.slots.int().to(DEV), **kw)

    def oracle(self, paths):
        """The oracle over paths [(session, [nodes])]: one sequence each."""
        idx = torch.tensor([s * self.R + r for s, p in paths for r in p], dtype=torch.long)
        tk = kda_synth.Tokens(*[t[idx] for t in self.tk.fields()])
        at = self.slots[[s for s, _ in paths]]
        return oracle_run(self.p, tk, kda_synth.cumsum0([len(p) for _, p in paths]), S_in=self.S[at], ring_in=self.ring[at])


def check_rows(rd, o, parents, skip=()):
    paths = [(s, path_to(parents[s], r)) for s in range(rd.n) for r in range(rd.R) if (s, r) not in skip]
    ref = rd.oracle(paths)
    ends = np.cumsum([len(p) for _, p in paths]) - 1
    got = np.stack([o[s, p[-1]].double().cpu().numpy() for s, p in paths])
    assert np.isfinite(got).all()
    err = rel_l2(got, ref["o"].reshape(-1, rd.H * 128)[ends])
    assert err <= TOL[rd.io], f"relative error {err:.3e}"


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate_kind", [0, 1])
@pytest.mark.parametrize("kind, R", [("bushy", 1), ("bushy", 2), ("bushy", 7), ("chain", 9), ("star", 13), ("bushy", 16),
                                     ("bushy", 17), ("bushy", 33), ("chain", 64), ("bushy", 64)])
def test_every_node_matches_the_oracle(io, gate_kind, kind, R):
    rd = Round(io, 2, R, seed=10 + R, gate_kind=gate_kind)
    rng = random.Random(R)
    parents = [tree(kind, R, rng) for _ in range(rd.n)]
    check_rows(rd, rd.decode(parents), parents)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_many_sessions(io):
    rd = Round(io, 40, 5, H=3, seed=3)
    rng = random.Random(3)
    parents = [tree("bushy", 5, rng) for _ in range(rd.n)]
    check_rows(rd, rd.decode(parents), parents)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_unused_nodes_keep_their_rows(io):
    """Entries that are no parent (below -1, itself, a later node) leave their
    node and everything under it out, whatever their inputs hold."""
    rd = Round(io, 2, 12, seed=5)
    parents = [[-1, 0, -2, 2, 4, 0, 9, 1, 6, -1, 9, 500], [0, -1, 1, 2, 3, 4, -7, 6, 7, 8, 9, 10]]
    unused = {(0, r) for r in (2, 3, 4, 6, 8, 11)} | {(1, 0), *((1, r) for r in range(6, 12))}
    for x in rd.rows:
        for s, r in unused:
            x[s, r] = float("nan")
    o = rd.decode(parents, o=torch.full_like(rd.rows[0], 7.0))
    for s, r in unused:
        assert (o[s, r] == 7.0).all()
    check_rows(rd, o, parents, skip=unused)


def test_chain_equals_a_straight_round_and_state_is_kept():
    rd = Round("f32", 3, 11, seed=6)
    S, ring = rd.S.to(DEV), rd.ring.to(DEV)
    slots = rd.slots.int().to(DEV)
    par = torch.tensor([tree("chain", 11, None)] * 3, dtype=torch.int32, device=DEV)
    o = kda.kda_decode_tree(rd.kp, *rd.rows, par, S, ring, slots=slots)
    assert torch.equal(S.cpu(), rd.S) and torch.equal(ring.cpu(), rd.ring)
    want = kda.kda_decode_multi(rd.kp, *rd.rows, S, ring, slots=slots)
    assert rel_l2(o.double().cpu().numpy(), want.double().cpu().numpy()) <= 2 * TOL["f32"]


def test_a_slot_twice_and_slots_out_of_range():
    """Two trees over one session's state; sessions without a slot keep their rows."""
    rd = Round("bf16", 4, 6, seed=7)
    rd.slots = torch.tensor([3, 3, 0, 1])
    rng = random.Random(7)
    parents = [tree("bushy", 6, rng) for _ in range(4)]
    full = rd.decode(parents)
    check_rows(rd, full, parents)
    sent = rd.slots.clone()
    sent[1], sent[3] = -1, 6
    o = kda.kda_decode_tree(rd.kp, *rd.rows, torch.tensor(parents, dtype=torch.int32, device=DEV), rd.S.to(DEV),
                            rd.ring.to(DEV), slots=sent.int().to(DEV), o=torch.full_like(rd.rows[0], 7.0))
    assert torch.equal(o[[0, 2]], full[[0, 2]]) and (o[[1, 3]] == 7.0).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate_kind", [0, 1])
@pytest.mark.parametrize("separate", [True, False])
def test_commit(io, gate_kind, separate):
    """Paths of every length around the groups of eight, none among them."""
    R, lens = 20, [0, 1, 2, 3, 8, 9, 17, 20]
    rd = Round(io, len(lens), R, seed=8, gate_kind=gate_kind)
    rng = random.Random(8)
    paths = [(s, sorted(rng.sample(range(R), L))) for s, L in enumerate(lens)]
    path = torch.full((rd.n, R), -1, dtype=torch.int32)
    for s, p in paths:
        path[s, :len(p)] = torch.tensor(p, dtype=torch.int32)
    S, ring = rd.S.to(DEV), rd.ring.to(DEV)
    out = dict(S_out=torch.full_like(S, 9.0), ring_out=torch.full_like(ring, 9.0)) if separate else {}
    q, k, v, z, b, _ = rd.rows
    S2, r2 = kda.kda_tree_commit(rd.kp, q, k, v, z, b, path.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), S, ring,
                                 slots=rd.slots.int().to(DEV), **out)
    ref = rd.oracle(paths)
    assert rel_l2(S2.cpu()[rd.slots].double().numpy(), ref["S"]) <= TOL["f32"]
    np.testing.assert_array_equal(r2.cpu()[rd.slots].double().numpy(), ref["ring"])
    rest = [s for s in range(rd.n + 2) if s not in rd.slots.tolist()]
    if separate:
        assert torch.equal(S.cpu(), rd.S) and torch.equal(ring.cpu(), rd.ring)
        assert (S2[rest] == 9.0).all() and (r2[rest] == 9.0).all()
    else:
        assert torch.equal(S2[rest].cpu(), rd.S[rest]) and torch.equal(r2[rest].cpu(), rd.ring[rest])


def test_commit_skips_bad_paths():
    """A length or an accepted node out of range, or a slot, skips its session;
    what lies behind a path's end is not looked at."""
    rd = Round("bf16", 6, 5, seed=9)
    path = torch.tensor([[0, 1, 2], [0, 5, 1], [-1, 0, 1], [2, 99, -5], [0, 1, 2], [0, 1, 2]], dtype=torch.int32)
    lens = torch.tensor([-1, 2, 1, 1, 4, 3], dtype=torch.int32)
    S, ring = rd.S.to(DEV), rd.ring.to(DEV)
    slots = rd.slots.clone()
    slots[5] = 8
    q, k, v, z, b, _ = rd.rows
    kda.kda_tree_commit(rd.kp, q, k, v, z, b, path.to(DEV), lens.to(DEV), S, ring, slots=slots.int().to(DEV))
    ref = rd.oracle([(3, [2])])
    at = int(rd.slots[3])
    assert rel_l2(S[at:at + 1].cpu().double().numpy(), ref["S"]) <= TOL["f32"]
    np.testing.assert_array_equal(ring[at:at + 1].cpu().double().numpy(), ref["ring"])
    rest = [s for s in range(8) if s != at]
    assert torch.equal(S[rest].cpu(), rd.S[rest]) and torch.equal(ring[rest].cpu(), rd.ring[rest])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prompt_tree_commit_tokens(io):
    """A session's life: prompt, a tree round, the accepted path, a single
    token; against the oracle over the tokens that were kept."""
    H, R, T = 2, 9, 70
    p = kda_synth.draw_params(H, 41)
    kp = kda_params(p, io)
    dt = kda_synth.io_dtype(io)
    prompt, nodes, last = (kda_synth.draw_tokens(m, H, 42 + m, dt) for m in (T, R, 1))
    parents = [-1, 0, 0, 1, 1, 2, 4, 4, 6]
    kept = path_to(parents, 7)
    _, S, ring = kda.kda_prefill(kp, *[t.to(DEV) for t in prompt.fields()], [0, T])
    rows = [t[None].to(DEV) for t in nodes.fields()]
    o = kda.kda_decode_tree(kp, *rows, torch.tensor([parents], dtype=torch.int32, device=DEV), S, ring)
    q, k, v, z, b, _ = rows
    kda.kda_tree_commit(kp, q, k, v, z, b, torch.tensor([kept], dtype=torch.int32, device=DEV),
                        torch.tensor([len(kept)], dtype=torch.int32, device=DEV), S, ring)
    o1 = kda.kda_decode(kp, *[t.to(DEV) for t in last.fields()], S, ring)
    every = kda_synth.Tokens(*[torch.cat([a, n[kept], l]) for a, n, l in zip(prompt.fields(), nodes.fields(), last.fields())])
    ref = oracle_run(p, every, [0, T + len(kept) + 1])
    tol = 1e-4 if io == "f32" else 2e-2     # the prompt's own tolerance
    got = torch.cat([o[0, kept], o1]).double().cpu().numpy()
    assert rel_l2(got, ref["o"].reshape(-1, H * 128)[T:]) <= tol
    assert rel_l2(S.cpu().double().numpy(), ref["S"]) <= tol
    np.testing.assert_array_equal(ring.double().cpu().numpy(), ref["ring"])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_deterministic_on_any_stream_and_in_a_graph(io):
    rd = Round(io, 3, 24, seed=12)
    rng = random.Random(12)
    parents = [tree("bushy", 24, rng) for _ in range(3)]
    par = torch.tensor(parents, dtype=torch.int32, device=DEV)
    path = torch.tensor([path_to(p, 23)[:4] + [-1] * (4 - len(path_to(p, 23)[:4])) for p in parents], dtype=torch.int32, device=DEV)
    lens = (path >= 0).sum(1).int()
    S, ring, slots = rd.S.to(DEV), rd.ring.to(DEV), rd.slots.int().to(DEV)
    q, k, v, z, b, gout = rd.rows

    def call(o, S2, r2, stream=None):
        kda.kda_decode_tree(rd.kp, q, k, v, z, b, gout, par, S, ring, slots=slots, o=o, stream=stream)
        kda.kda_tree_commit(rd.kp, q, k, v, z, b, path, lens, S, ring, S_out=S2, ring_out=r2, slots=slots, stream=stream)

    def buffers():
        return torch.zeros_like(q), torch.zeros_like(S), torch.zeros_like(ring)

    want = buffers()
    call(*want)
    side = torch.cuda.Stream()
    got = buffers()
    side.wait_stream(torch.cuda.current_stream())
    call(*got, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    out = buffers()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(*out)
    for _ in range(2):
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))
