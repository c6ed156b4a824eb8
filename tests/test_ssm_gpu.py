"""The state space mixer (kda_ssm_prefill, kda_ssm_decode) against its
definition token by token in 64 bits."""
import pytest
import torch

import gated_delta_rule_04_gb300 as kda
from ssm_ref import close, make_inputs, mixer

pytestmark = pytest.mark.gpu
DEV = "cuda"
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_04_gb300 import build as kbuild
    kbuild.build()
    kda.lib()


def dev(x):
    return None if x is None else x.to(DEV)


def params(i, io, algo="auto"):
    return kda.make_ssm_params(dev(i["conv_w"]), dev(i["A_log"]), dev(i["dt_bias"]), head_dim=i["P"], state_dim=i["N"],
                               num_groups=i["G"], D=dev(i["D"]), conv_b=dev(i["conv_b"]), io_dtype=io, algo=algo)


def cumsum(lens):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return cu


def prefill(i, io, cu, gate=True, algo="auto", **kw):
    return kda.kda_ssm_prefill(params(i, io, algo), dev(i["xbc"]), dev(i["dt"]), cu, z=dev(i["z"]) if gate else None,
                               S_in=dev(i["S"]), ring_in=dev(i["ring"]), **kw)


def check(i, io, cu, gate=True, algo="auto"):
    o, S, ring = prefill(i, io, cu, gate, algo)
    wo, wS, wr = mixer(i, cu, gate)
    close("o", o, wo)
    close("S", S, wS)
    assert torch.equal(ring.cpu(), wr)
    return o, S, ring


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("H, P, N, G", [(2, 64, 64, 1), (3, 64, 128, 3), (6, 64, 128, 2), (2, 128, 64, 1), (3, 128, 128, 1),
                                        (5, 64, 64, 1)])
def test_prefill_layouts(io, H, P, N, G):
    """Head and state widths, shared and single groups, an odd number of heads in a group."""
    cu = cumsum([70, 0, 1, 130])
    check(make_inputs(cu[-1], 4, H, P, N, G, IO[io], 11 + H), io, cu)


@pytest.mark.parametrize("io, algo", [("f32", "auto"), ("bf16", "auto"), ("bf16", "scan")])
@pytest.mark.parametrize("lens", [[1], [2], [3], [15, 16, 17], [63], [64], [65], [0, 0, 5, 0], [129, 64, 200, 1]])
def test_prefill_lengths(io, algo, lens):
    cu = cumsum(lens)
    check(make_inputs(cu[-1], len(lens), 2, 64, 128, 1, IO[io], 5 + len(lens)), io, cu, algo=algo)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("state, bias, skip, gate", [(False, True, True, True), (True, False, True, True),
                                                     (True, True, False, True), (True, True, True, False),
                                                     (False, False, False, False)])
def test_prefill_optional_inputs(io, state, bias, skip, gate):
    cu = cumsum([100, 30])
    check(make_inputs(cu[-1], 2, 4, 64, 64, 2, IO[io], 3, state, bias, skip), io, cu, gate)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prefill_longer(io):
    """A sequence of many blocks, whose state carries over all of them."""
    cu = cumsum([1100, 37])
    i = make_inputs(cu[-1], 2, 2, 64, 128, 1, IO[io], 8)
    i["A_log"] -= 3.0          # slow decay: early tokens still count at the end
    check(i, io, cu)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prefill_strong_decay(io):
    """Steps so large that a state vanishes within a token, next to tiny ones."""
    cu = cumsum([150])
    i = make_inputs(150, 1, 2, 64, 64, 1, IO[io], 9)
    i["dt"] = (i["dt"].float() * 8).to(IO[io])
    i["dt_bias"] += 3.0
    check(i, io, cu)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-4, 1e4])
def test_prefill_scales(io, scale):
    """Inputs far from unit size keep their relative precision."""
    cu = cumsum([140, 20])
    i = make_inputs(cu[-1], 2, 2, 64, 128, 1, IO[io], 10, bias=False)
    if scale < 1:        # SiLU is linear here: keep x, B, C small and the step ordinary
        i["S"] *= scale ** 2
    i["xbc"] = (i["xbc"].float() * scale).to(IO[io])
    i["ring"] = (i["ring"].float() * scale).to(IO[io])
    check(i, io, cu)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prefill_column_ranges_of_one_projection(io):
    """xbc, dt and z as strided views of one row, and the buffers reused in place."""
    H, P, N, G, T = 4, 64, 64, 2, 90
    cu = cumsum([T - 7, 7])
    i = make_inputs(T, 2, H, P, N, G, IO[io], 12)
    ch, W = H * P + 2 * G * N, H * P
    row = torch.full((T, W + ch + 16), float("nan"), dtype=IO[io], device=DEV)
    row[:, :W], row[:, W:W + ch], row[:, W + ch:W + ch + H] = dev(i["z"]), dev(i["xbc"]), dev(i["dt"])
    S, ring = dev(i["S"]), dev(i["ring"])
    o, S2, r2 = kda.kda_ssm_prefill(params(i, io), row[:, W:W + ch], row[:, W + ch:W + ch + H], cu, z=row[:, :W], S_in=S,
                                    S_out=S, ring_in=ring, ring_out=ring)
    wo, wS, wr = mixer(i, cu)
    close("o", o, wo)
    close("S", S, wS)
    assert S2 is S and r2 is ring and torch.equal(ring.cpu(), wr)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prefill_keeps_sequences_apart(io):
    """A sequence of NaN and infinities beside others: they do not see it, nor
    does what lies around the rows in memory."""
    lens = [20, 70, 33]
    cu = cumsum(lens)
    i = make_inputs(cu[-1], 3, 3, 64, 128, 1, IO[io], 13)
    want = prefill(i, io, cu)
    bad = {**i, **{k: i[k].clone() for k in ("xbc", "dt", "z")}}
    for k in ("xbc", "dt", "z"):
        bad[k][cu[1]:cu[2]] = float("nan")
        bad[k][cu[1] + 3] = float("inf")
    got = prefill(bad, io, cu)
    for a, b in ((0, cu[1]), (cu[2], cu[3])):
        assert torch.equal(got[0][a:b], want[0][a:b])
    for s in (0, 2):
        assert torch.equal(got[1][s], want[1][s]) and torch.equal(got[2][s], want[2][s])
    assert torch.isnan(got[1][1]).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("where", ["x", "B", "C", "dt", "S"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_prefill_non_finite_inputs_never_look_finite(io, where, value):
    """Where the definition gives a finite value, the output has that value or
    (the chunked form, from that chunk on) is not finite; an output the
    definition has no finite value for is not finite either."""
    H, P, N, G = 2, 64, 64, 1
    i = make_inputs(140, 1, H, P, N, G, IO[io], 16)
    at = {"x": 5, "B": H * P + 7, "C": H * P + N + 9}.get(where)
    if at is not None:
        i["xbc"][70, at] = value
    elif where == "dt":
        i["dt"][70, 1] = value
    else:
        i["S"][0, 1, 3, 4] = value
    o, S, _ = prefill(i, io, [0, 140])
    wo, wS, _ = mixer(i, [0, 140])
    for got, want in ((o.cpu(), wo), (S.cpu(), wS)):
        assert not (torch.isfinite(got) & ~torch.isfinite(want)).any()
        both = torch.isfinite(got) & torch.isfinite(want)
        assert both.any() or want is wS      # (the chunked form may lose a group's whole state)
        close("finite part", torch.where(both, got, torch.zeros_like(got)), torch.where(both, want, torch.zeros_like(want)))
    if where != "S":
        assert torch.isfinite(o[:64]).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prefill_in_parts_and_then_tokens(io):
    """A prompt whole, in two parts, and its tail as single tokens."""
    T, H, P, N, G = 150, 4, 64, 128, 2
    i = make_inputs(T, 1, H, P, N, G, IO[io], 14)
    wo, wS, wr = mixer(i, [0, T])
    p = params(i, io)
    x, d, z = dev(i["xbc"]), dev(i["dt"]), dev(i["z"])
    o1, S, ring = kda.kda_ssm_prefill(p, x[:77], d[:77], [0, 77], z=z[:77], S_in=dev(i["S"]), ring_in=dev(i["ring"]))
    o2, S, ring = kda.kda_ssm_prefill(p, x[77:140], d[77:140], [0, 63], z=z[77:140], S_in=S, ring_in=ring)
    outs = [o1, o2] + [kda.kda_ssm_decode(p, x[t:t + 1], d[t:t + 1], S, ring, z=z[t:t + 1]) for t in range(140, T)]
    close("o", torch.cat(outs), wo)
    close("S", S, wS)
    assert torch.equal(ring.cpu(), wr)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prefill_is_deterministic_on_any_stream_and_in_a_graph(io):
    cu = cumsum([260, 64, 3])
    i = make_inputs(cu[-1], 3, 4, 64, 128, 2, IO[io], 15)
    p = params(i, io)
    args = [dev(i[k]) for k in ("xbc", "dt", "z", "S", "ring")]
    ws = torch.empty(kda.kda_ssm_prefill_workspace_bytes(p, 3, cu[-1]), dtype=torch.uint8, device=DEV)

    def call(**kw):
        return kda.kda_ssm_prefill(p, args[0], args[1], cu, z=args[2], S_in=args[3], ring_in=args[4], **kw)

    want = call(workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = dict(o=torch.zeros_like(want[0]), S_out=torch.zeros_like(want[1]), ring_out=torch.zeros_like(want[2]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(workspace=ws, **out)
    for _ in range(2):
        for t in out.values():
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out.values(), want))
    assert kda.kda_workspace_status(ws) == kda.KDA_OK


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("H, P, N, G, n", [(2, 64, 64, 1, 1), (6, 64, 128, 3, 5), (3, 128, 64, 1, 3), (4, 128, 128, 2, 2),
                                           (1, 64, 128, 1, 2), (12, 64, 64, 1, 2), (17, 64, 64, 1, 1), (32, 64, 128, 1, 1),
                                           (33, 64, 64, 1, 2), (80, 64, 64, 2, 1)])
@pytest.mark.parametrize("gate, bias", [(True, True), (False, False)])
def test_decode(io, H, P, N, G, n, gate, bias):
    i = make_inputs(n, n, H, P, N, G, IO[io], 21, bias=bias, skip=bias)
    S, ring = dev(i["S"]), dev(i["ring"])
    o = kda.kda_ssm_decode(params(i, io), dev(i["xbc"]), dev(i["dt"]), S, ring, z=dev(i["z"]) if gate else None)
    wo, wS, wr = mixer(i, list(range(n + 1)), gate)
    close("o", o, wo)
    close("S", S, wS)
    assert torch.equal(ring.cpu(), wr)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_decode_pool_and_skipped_sessions(io):
    """Sessions at slots of a pool; a slot out of range leaves its session,
    its output row (and the rest of the pool) as they were, whatever its inputs hold."""
    n, slots, H, P, N, G = 5, 9, 4, 64, 128, 2
    i = make_inputs(n, slots, H, P, N, G, IO[io], 22)
    i["xbc"][1] = float("nan")
    i["dt"][3] = float("inf")
    at = torch.tensor([7, -1, 0, 9, 4], dtype=torch.int32)
    S, ring = dev(i["S"]), dev(i["ring"])
    o = torch.full((n, H * P), 3.0, dtype=IO[io], device=DEV)
    kda.kda_ssm_decode(params(i, io), dev(i["xbc"]), dev(i["dt"]), S, ring, z=dev(i["z"]), slots=at.to(DEV), o=o)
    live = [0, 2, 4]
    sub = {**i, **{k: i[k][live] for k in ("xbc", "dt", "z")}, "S": i["S"][at[live].long()], "ring": i["ring"][at[live].long()]}
    wo, wS, wr = mixer(sub, [0, 1, 2, 3])
    close("o", o[live], wo)
    close("S", S[at[live].long().to(DEV)], wS)
    assert torch.equal(ring[at[live].long().to(DEV)].cpu(), wr)
    assert (o[[1, 3]] == 3.0).all()
    for s in set(range(slots)) - {7, 0, 4}:
        assert torch.equal(S[s].cpu(), i["S"][s]) and torch.equal(ring[s].cpu(), i["ring"][s])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("P, N, H, n", [(64, 128, 16, 70), (128, 128, 8, 80), (64, 64, 40, 60)])
def test_decode_larger_batches(io, P, N, H, n):
    """More than 32 MB of states (two kernels), more items than resident CTAs."""
    i = make_inputs(n, n, H, P, N, 4, IO[io], 23)
    i["slots"] = torch.randperm(n, generator=torch.Generator().manual_seed(1))
    p = params(i, io)
    assert kda.kda_ssm_decode_workspace_bytes(p, n) > 0
    S, ring = dev(i["S"]), dev(i["ring"])
    o = kda.kda_ssm_decode(p, dev(i["xbc"]), dev(i["dt"]), S, ring, z=dev(i["z"]), slots=i["slots"].int().to(DEV))
    wo, wS, wr = mixer({**i, "S": i["S"][i["slots"]], "ring": i["ring"][i["slots"]]}, list(range(n + 1)))
    close("o", o, wo)
    close("S", S.cpu()[i["slots"]], wS)
    assert torch.equal(ring.cpu()[i["slots"]], wr)


@pytest.mark.parametrize("H, G", [(4, 2), (40, 1)])
def test_decode_in_a_graph_with_its_own_workspace(H, G):
    """Two captured calls, each with its workspace, replayed in turn."""
    P, N = 64, 128
    graphs = []
    for seed in (31, 32):
        i = make_inputs(2, 2, H, P, N, G, torch.bfloat16, seed)
        p = params(i, "bf16")
        x, d, z, S, ring = (dev(i[k]) for k in ("xbc", "dt", "z", "S", "ring"))
        ws = torch.empty(kda.kda_ssm_decode_workspace_bytes(p, 2), dtype=torch.uint8, device=DEV)
        o = torch.zeros(2, H * P, dtype=torch.bfloat16, device=DEV)
        S0, r0 = S.clone(), ring.clone()
        kda.kda_ssm_decode(p, x, d, S, ring, z=z, o=o, workspace=ws)
        want = o.clone(), S.clone(), ring.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kda.kda_ssm_decode(p, x, d, S, ring, z=z, o=o, workspace=ws)
        graphs.append((g, p, x, d, z, ws, o, S, ring, S0, r0, want))
    for g, *_, o, S, ring, S0, r0, want in graphs:
        S.copy_(S0)
        ring.copy_(r0)
        o.zero_()
    for g, *_ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for g, *_, o, S, ring, S0, r0, want in graphs:
        assert all(torch.equal(a, b) for a, b in zip((o, S, ring), want))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("H, P, N, lens", [
    (2, 64, 128, [1500, 30, 700, 0, 300]),                     # one unit: many pieces, of several sequences
    (3, 128, 64, [1100, 1000, 980]),                           # close lengths
    (2, 64, 64, [5, 900, 64, 128] + [20 * k for k in range(16)]),   # more sequences than travel with the launch
    (40, 64, 64, [600, 8, 8, 8])])                             # the longest one alone at the end
def test_prefill_cut_sequences_in_place(io, H, P, N, lens):
    """Sequences cut into pieces, whose starts are composed; state and ring updated in place; the
    rows behind the last sequence are neither read nor written."""
    cu = cumsum(lens)
    T, n = cu[-1], len(lens)
    i = make_inputs(T, n, H, P, N, 1, IO[io], 31 + H)
    i["A_log"] -= 2.0
    wo, wS, wr = mixer(i, cu, True)
    pad = {k: torch.full((T + 70, dev(i[k]).shape[1]), float("nan"), dtype=IO[io], device=DEV) for k in ("xbc", "dt", "z")}
    for k, t in pad.items():
        t[:T] = dev(i[k])
    S, ring = dev(i["S"]), dev(i["ring"])
    buf = torch.full((T + 70, H * P), 7.0, dtype=IO[io], device=DEV)
    p = params(i, io)
    ws = torch.empty(kda.kda_ssm_prefill_workspace_bytes(p, n, T), dtype=torch.uint8, device=DEV)
    o, S_out, ring_out = kda.kda_ssm_prefill(p, pad["xbc"][:T], pad["dt"][:T], cu, z=pad["z"][:T], S_in=S, S_out=S, ring_in=ring,
                                             ring_out=ring, o=buf[:T], workspace=ws)
    assert kda.kda_workspace_status(ws) == kda.KDA_OK
    assert S_out is S and ring_out is ring
    close("o", o, wo)
    close("S", S, wS)
    assert torch.equal(ring.cpu(), wr)
    assert bool((buf[T:] == 7.0).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prefill_two_at_once_and_two_graphs_with_one_workspace(io):
    sizes = ([700, 65], [33] * 18)
    cases = []
    for k, lens in enumerate(sizes):
        cu = cumsum(lens)
        i = make_inputs(cu[-1], len(lens), 4, 64, 128, 2, IO[io], 50 + k)
        p = params(i, io)
        t = [dev(i[x]) for x in ("xbc", "dt", "z", "S", "ring")]
        cases.append((p, cu, t, kda.kda_ssm_prefill_workspace_bytes(p, len(lens), cu[-1])))

    def call(c, ws, **kw):
        p, cu, t, _ = c
        return kda.kda_ssm_prefill(p, t[0], t[1], cu, z=t[2], S_in=t[3], ring_in=t[4], workspace=ws, **kw)

    space = [torch.empty(c[3], dtype=torch.uint8, device=DEV) for c in cases]
    want = [call(c, w) for c, w in zip(cases, space)]
    torch.cuda.synchronize()
    # two streams, a workspace each
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        for k in range(2):
            got[k].append(call(cases[k], space[k], stream=streams[k]))
    for s in streams:
        s.synchronize()
    for k in range(2):
        for g in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[k]))
    # two graphs that share a workspace, replayed in turn on one stream
    shared = torch.empty(max(c[3] for c in cases), dtype=torch.uint8, device=DEV)
    graphs, outs = [], []
    for k, c in enumerate(cases):
        out = dict(o=torch.zeros_like(want[k][0]), S_out=torch.zeros_like(want[k][1]), ring_out=torch.zeros_like(want[k][2]))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(c, shared, **out)
        graphs.append(g)
        outs.append(out)
    for k in (0, 1, 0, 1, 1, 0):
        for t in outs[k].values():
            t.zero_()
        graphs[k].replay()
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(a, b) for a, b in zip(outs[k].values(), want[k]))
