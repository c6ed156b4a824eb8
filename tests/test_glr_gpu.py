"""The gated linear recurrence (kda_glr_prefill, kda_glr_backward, kda_glr_decode,
kda_glr_commit) against its definition token by token in 64 bits."""
import math

import pytest
import torch

import gated_delta_rule_04_gb300 as kda
from glr_ref import SUM_TOL, close, gradients, make_inputs, mixer, states, steps

pytestmark = pytest.mark.gpu
DEV = "cuda"
IO = {"f32": torch.float32, "bf16": torch.bfloat16}
GRADS = ("dx", "dr", "di", "dz", "dS_in", "dA_log", "dr_bias", "di_bias")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_04_gb300 import build as kbuild
    kbuild.build()
    kda.lib()


def dev(x):
    return None if x is None else x.to(DEV)


def params(i, io):
    return kda.make_glr_params(dev(i["A_log"]), r_bias=dev(i["r_bias"]), i_bias=dev(i["i_bias"]), io_dtype=io)


def cumsum(lens):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return cu


def empty_states(i, cu):
    return torch.full((-(-cu[-1] // kda.KDA_GLR_CHUNK), i["C"]), float("nan"), device=DEV)


def prefill(i, io, cu, **kw):
    return kda.kda_glr_prefill(params(i, io), dev(i["x"]), dev(i["r"]), dev(i["i"]), cu, z=dev(i["z"]), S_in=dev(i["S"]), **kw)


def backward(i, io, cu, st, **kw):
    return kda.kda_glr_backward(params(i, io), dev(i["x"]), dev(i["r"]), dev(i["i"]), cu, st, dev(i["do"]), z=dev(i["z"]),
                                S_in=dev(i["S"]), dS_out=dev(i["dS"]), **kw)


def check(i, io, cu, scale=1.0):
    """Both directions; ``scale`` widens the tolerances."""
    st = empty_states(i, cu)
    o, S = prefill(i, io, cu, states=st)
    wo, wS = mixer(i, cu)
    tol = lambda t: {torch.float32: 2e-5, torch.bfloat16: 2 ** -8 + 2e-5}[t] * scale
    close("o", o, wo, tol(o.dtype))
    close("S", S, wS, tol(S.dtype))
    before = states(i, cu)[0]
    close("states", st, before[::kda.KDA_GLR_CHUNK], tol(st.dtype))
    got, want = backward(i, io, cu, st), gradients(i, cu)
    for k in GRADS:
        if k == "dz" and i["z"] is None:
            assert got.dz is None
            continue
        g = getattr(got, k)
        close(k, g, want[k], SUM_TOL * scale if k in ("dA_log", "dr_bias", "di_bias") else tol(g.dtype))
    return o, S, st, got


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("C", [1, 2, 3, 8, 31, 32, 33, 40, 63, 64, 65, 96, 127, 128, 130, 200, 257])
def test_widths(io, C):
    cu = cumsum([70, 0, 1, 130])
    check(make_inputs(cu[-1], 4, C, IO[io], 11 + C), io, cu)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[1], [2], [3], [7, 8, 9], [15, 16, 17], [63], [64], [65], [128], [129], [0, 0, 5, 0],
                                  [64, 64], [63, 1, 64, 1], [1] * 40, [129, 64, 200, 1], [0, 1] * 9 + [0] * 5, [3] * 100])
def test_lengths(io, lens):
    cu = cumsum(lens)
    check(make_inputs(cu[-1], len(lens), 24, IO[io], 5 + len(lens)), io, cu)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("state, bias, gate", [(False, True, True), (True, False, True), (True, True, False), (False, False, False)])
def test_optional_inputs(io, state, bias, gate):
    cu = cumsum([100, 30, 0])
    check(make_inputs(cu[-1], 3, 72, IO[io], 3, state, bias, gate), io, cu)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("C, lens", [(24, [700]), (200, [650, 37]), (8, [1, 500, 0, 199])])
def test_longer(io, C, lens):
    """Sequences over many 64-token chunks, a state that carries over several of them."""
    cu = cumsum(lens)
    i = make_inputs(cu[-1], len(lens), C, IO[io], 8)
    i["A_log"] -= 1.0
    check(i, io, cu)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_long_memory(io):
    """5000 tokens whose decays are 1 - 1e-4 to 1 - 1e-3: the first tokens still count at the end.
    The rounding of a decay next to 1 is up to 2^-25 of it, and a value takes part in up to 1 / (1 - a)
    = 10^4 of them, worst case 10^4 * 2^-25 = 3e-4 (15 times the usual tolerance) if all had one sign."""
    cu = [0, 4900, 5000]
    i = make_inputs(5000, 2, 16, IO[io], 9)
    i["A_log"] = torch.log(torch.logspace(-3.7, -2.7, 16))
    o, S = prefill(i, io, cu)
    wo, wS = mixer(i, cu)
    close("S", S, wS, 15 * 2e-5)
    close("o", o, wo, 15 * 2e-5 + (2 ** -8 if io == "bf16" else 0))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [-30.0, -12.0, 12.0, 30.0])
def test_gates_far_from_zero(io, shift):
    """Gates that are nearly shut or open: 1 - a^2 of a decay next to 1, a decay of e^-50.  The
    output gate's argument is as far out."""
    cu = cumsum([150, 20])
    for which in ("r", "i", "z"):
        i = make_inputs(cu[-1], 2, 40, IO[io], 10, state=which != "r")
        i[which] = (i[which].float() + shift).to(IO[io])
        if which == "r":
            i["A_log"] += math.log(50.0)
        check(i, io, cu)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_infinite_gate_logits(io):
    """A shut gate (-inf) and an open one (+inf) have finite values and gradients: w = 0 keeps the state
    and takes nothing in, v = 0 takes nothing in."""
    cu = [0, 90]
    i = make_inputs(90, 1, 24, IO[io], 12)
    i["r"][20], i["r"][40], i["i"][30], i["i"][50] = -math.inf, math.inf, -math.inf, math.inf
    check(i, io, cu)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-4, 1e4])
def test_scales(io, scale):
    cu = cumsum([140, 20])
    i = make_inputs(cu[-1], 2, 40, IO[io], 13)
    for k in ("x", "do"):
        i[k] = (i[k].float() * scale).to(IO[io])
    i["S"], i["dS"] = i["S"] * scale, i["dS"] * scale
    check(i, io, cu)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("C, pad, off", [(64, 64, 0), (40, 8, 8), (40, 3, 1), (33, 31, 0), (130, 7, 5)])
def test_column_ranges_of_projections(io, C, pad, off):
    """x, z and r, i as strided views of wider rows, on 16 bytes or not, with NaN around them; the
    gradients into views as well, whose surroundings stay; the states in place."""
    cu = cumsum([83, 7, 41])
    T = cu[-1]
    i = make_inputs(T, 3, C, IO[io], 14)
    nan = lambda: torch.full((T, 2 * C + pad + off), float("nan"), dtype=IO[io], device=DEV)
    xz, ri, dxz, dri, do = nan(), nan(), nan(), nan(), nan()
    a, b = slice(off, off + C), slice(off + C, off + 2 * C)
    xz[:, a], xz[:, b], ri[:, a], ri[:, b], do[:, b] = (dev(i[k]) for k in ("x", "z", "r", "i", "do"))
    S, st, p = dev(i["S"]), empty_states(i, cu), params(i, io)
    start = S.clone()
    o, S2 = kda.kda_glr_prefill(p, xz[:, a], ri[:, a], ri[:, b], cu, z=xz[:, b], S_in=S, S_out=S, states=st)
    wo, wS = mixer(i, cu)
    close("o", o, wo)
    close("S", S, wS)
    assert S2 is S
    dS = dev(i["dS"])
    got = kda.kda_glr_backward(p, xz[:, a], ri[:, a], ri[:, b], cu, st, do[:, b], z=xz[:, b], S_in=start, dS_out=dS, dx=dxz[:, a],
                               dz=dxz[:, b], dr=dri[:, a], di=dri[:, b])
    want = gradients(i, cu)
    for k in GRADS:
        close(k, getattr(got, k), want[k], SUM_TOL if k in ("dA_log", "dr_bias", "di_bias") else None)
    assert torch.equal(dS.cpu(), i["dS"])
    for t in (dxz, dri):
        assert torch.isnan(t[:, :off]).all() and torch.isnan(t[:, off + 2 * C:]).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_sequences_and_channels_stay_apart(io):
    """NaN and infinities of a sequence or a channel leave the others bit for bit, both ways."""
    cu = cumsum([20, 70, 33])
    i = make_inputs(cu[-1], 3, 72, IO[io], 15)
    o, S, st, g = check(i, io, cu)
    bad = {k: v.clone() if torch.is_tensor(v) else v for k, v in i.items()}
    for k in ("x", "r", "i", "z", "do"):
        bad[k][cu[1]:cu[2], :] = float("nan")
        bad[k][cu[1] + 3] = float("inf")
    st2 = empty_states(i, cu)
    o2, S2 = prefill(bad, io, cu, states=st2)
    st2 = torch.where(torch.isnan(st2), st2, st2)
    g2 = backward(bad, io, cu, st2)
    for a, b in ((0, cu[1]), (cu[2], cu[3])):
        assert torch.equal(o2[a:b], o[a:b])
        for k in ("dx", "dr", "di", "dz"):
            assert torch.equal(getattr(g2, k)[a:b], getattr(g, k)[a:b])
    for s in (0, 2):
        assert torch.equal(S2[s], S[s]) and torch.equal(g2.dS_in[s], g.dS_in[s])
    assert torch.isnan(S2[1]).all()
    bad = {k: v.clone() if torch.is_tensor(v) else v for k, v in i.items()}
    bad["x"][25, 7] = float("nan")
    bad["S"][1, 9] = float("inf")
    o2, S2 = prefill(bad, io, cu, states=st2)
    g2 = backward(bad, io, cu, st2)
    ok = [c for c in range(72) if c not in (7, 9)]
    assert torch.equal(o2[:, ok], o[:, ok]) and torch.equal(g2.dr[:, ok], g.dr[:, ok]) and torch.equal(g2.dA_log[ok], g.dA_log[ok])
    assert torch.isfinite(o2[:25, 7]).all() and torch.isnan(o2[25:cu[2], 7]).all() and torch.equal(o2[cu[2]:], o[cu[2]:])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_in_parts_and_then_tokens(io):
    """A prompt whole, in two parts, and its tail as single tokens and runs."""
    T, C = 150, 72
    i = make_inputs(T, 1, C, IO[io], 16)
    wo, wS = mixer(i, [0, T])
    p = params(i, io)
    x, r, s, z = (dev(i[k]) for k in ("x", "r", "i", "z"))
    o1, S = kda.kda_glr_prefill(p, x[:77], r[:77], s[:77], [0, 77], z=z[:77], S_in=dev(i["S"]))
    o2, S = kda.kda_glr_prefill(p, x[77:140], r[77:140], s[77:140], [0, 63], z=z[77:140], S_in=S)
    outs = [o1, o2]
    for a, b in ((140, 141), (141, 142), (142, 146), (146, 150)):
        outs.append(kda.kda_glr_decode(p, x[None, a:b], r[None, a:b], s[None, a:b], S, z=z[None, a:b])[0])
    close("o", torch.cat(outs), wo)
    close("S", S, wS)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_many_sequences(io):
    """5000 sequences of 0 to 3 tokens (their offsets are built on the device)."""
    g = torch.Generator().manual_seed(17)
    cu = cumsum(torch.randint(0, 4, (5000,), generator=g).tolist())
    i = make_inputs(cu[-1], 5000, 5, IO[io], 17)
    check(i, io, cu, scale=4.0)    # sums of 7500 terms: (7500 / 700)^1/2 = 3.3 times the usual tolerance


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[], [0], [0, 0, 0], [0] * 40])
def test_no_tokens(io, lens):
    cu = cumsum(lens)
    i = make_inputs(0, len(lens), 24, IO[io], 18)
    st = empty_states(i, cu)
    o, S = prefill(i, io, cu, states=st)
    assert o.shape == (0, 24) and torch.equal(S.cpu(), i["S"])
    g = backward(i, io, cu, st)
    assert torch.equal(g.dS_in.cpu(), i["dS"])
    for k in ("dA_log", "dr_bias", "di_bias"):
        assert not getattr(g, k).any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gradients_are_those_of_differences(io):
    """The kernel's gradients against differences of the 64-bit loss along random directions.  Steps of
    1e-5 in 64 bits are good to 1e-9 of the loss' scale; the kernel's error along a direction is that of its
    outputs (2e-5 or 2^-8) times the sizes of gradient and direction."""
    cu = cumsum([66, 0, 9, 130])
    i = make_inputs(cu[-1], 4, 24, IO[io], 19)
    st = empty_states(i, cu)
    prefill(i, io, cu, states=st)
    got = backward(i, io, cu, st)
    i64 = {k: v.double() if torch.is_tensor(v) else v for k, v in i.items()}

    def loss(j):
        o, S = mixer(j, cu)
        return float((o * i64["do"]).sum() + (S * i64["dS"]).sum())

    g = torch.Generator().manual_seed(20)
    for name, grad in (("x", "dx"), ("r", "dr"), ("i", "di"), ("z", "dz"), ("S", "dS_in"), ("A_log", "dA_log"),
                       ("r_bias", "dr_bias"), ("i_bias", "di_bias")):
        d, e = torch.randn(i64[name].shape, generator=g, dtype=torch.float64), 1e-5
        diff = (loss({**i64, name: i64[name] + e * d}) - loss({**i64, name: i64[name] - e * d})) / (2 * e)
        k = getattr(got, grad).cpu().double()
        tol = (2 ** -8 if getattr(got, grad).dtype == torch.bfloat16 else 0) + (SUM_TOL if k.dim() == 1 else 2e-5)
        assert abs(float((k * d).sum()) - diff) <= tol * float(k.norm()) * float(d.norm()) / math.sqrt(d.numel()) * 4 + 1e-6, name
        # (a random direction meets an error vector at 1 / sqrt(numel) of its length; 4 standard deviations)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_deterministic_on_any_stream_and_in_a_graph(io):
    cu = cumsum([260, 64, 3, 700])
    i = make_inputs(cu[-1], 4, 136, IO[io], 21)
    p = params(i, io)
    x, r, s, z, S, do, dS = (dev(i[k]) for k in ("x", "r", "i", "z", "S", "do", "dS"))
    size = max(kda.kda_glr_prefill_workspace_bytes(p, 4, cu[-1]), kda.kda_glr_backward_workspace_bytes(p, 4, cu[-1]))
    ws, ws2 = (torch.full((size,), 255, dtype=torch.uint8, device=DEV) for _ in range(2))
    st = empty_states(i, cu)

    def both(st, ws, **kw):
        o, So = kda.kda_glr_prefill(p, x, r, s, cu, z=z, S_in=S, states=st, workspace=ws, **kw)
        g = kda.kda_glr_backward(p, x, r, s, cu, st, do, z=z, S_in=S, dS_out=dS, workspace=ws, **kw)
        return [o, So, st] + [getattr(g, k) for k in GRADS]

    want = both(st, ws)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    # two calls at once, each on its stream with its own workspace
    runs = [both(empty_states(i, cu), ws, stream=side), both(empty_states(i, cu), ws2, stream=other)]
    torch.cuda.synchronize()
    runs.append(both(empty_states(i, cu), None))
    # two graphs that share one workspace, replayed in turn
    graphs, outs = [], []
    for _ in range(2):
        stg = empty_states(i, cu)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(both(stg, ws))
        graphs.append(gr)
    for k in (0, 1, 0):
        graphs[k].replay()
    torch.cuda.synchronize()
    for run in runs + outs:
        for a, b in zip(run, want):
            assert torch.equal(a, b)
    assert kda.kda_workspace_status(ws) == kda.KDA_OK


# ---- tokens over a pool -------------------------------------------------------------------

def tokens_ref(i, n, R, S, paths):
    """Outputs of every taken row and the states, in 64 bits; i's rows are [n * R]."""
    s = steps(i)
    S, o = S.double().clone(), torch.zeros(n, R, i["C"], dtype=torch.float64)
    for k, path in enumerate(paths):
        for j in path:
            S[k] = s["a"][k * R + j] * S[k] + s["b"][k * R + j]
            o[k, j] = S[k]
    if i["z"] is not None:
        z = i["z"].double().view(n, R, -1)
        o = o * z * torch.sigmoid(z)
    return o, S


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("C", [1, 7, 8, 64, 129, 1024])
@pytest.mark.parametrize("n, R", [(1, 1), (5, 1), (3, 4), (2, 64)])
def test_decode(io, C, n, R):
    i = make_inputs(n * R, n, C, IO[io], 30 + C + R, gate=C != 7)
    v = {k: None if i[k] is None else dev(i[k]).view(n, R, C) for k in ("x", "r", "i", "z")}
    wo, wS = tokens_ref(i, n, R, i["S"], [range(R)] * n)
    S = dev(i["S"])
    o = kda.kda_glr_decode(params(i, io), v["x"], v["r"], v["i"], S, z=v["z"])
    close("o", o, wo)
    close("S", S, wS)
    S = dev(i["S"])
    o2 = kda.kda_glr_decode(params(i, io), v["x"], v["r"], v["i"], S, z=v["z"], keep_state=True)
    assert torch.equal(o2, o) and torch.equal(S.cpu(), i["S"])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_decode_slots_and_pools(io):
    """Slots in any order, some out of range (their rows and everything else stay), other output pools,
    strided rows."""
    n, R, C, slots_n = 6, 3, 40, 9
    i = make_inputs(n * R, slots_n, C, IO[io], 31)
    slots = torch.tensor([7, 2, -1, 0, 9, 5], dtype=torch.int32)
    start = torch.stack([i["S"][s] if 0 <= s < slots_n else torch.zeros(C) for s in slots.tolist()])
    wo, wS = tokens_ref(i, n, R, start, [range(R)] * n)
    wide = torch.full((n, R, 4 * C + 5), float("nan"), dtype=IO[io], device=DEV)
    parts = [wide[..., k * C + k:(k + 1) * C + k] for k in range(4)]
    for part, k in zip(parts, ("x", "r", "i", "z")):
        part.copy_(dev(i[k]).view(n, R, C))
    S, S_out = dev(i["S"]), torch.full((slots_n, C), 77.0, device=DEV)
    o = torch.full((n, R, C), 55.0, dtype=IO[io], device=DEV)
    out = kda.kda_glr_decode(params(i, io), *parts[:3], S, z=parts[3], slots=dev(slots), S_out=S_out, o=o)
    assert out is o and torch.equal(S.cpu(), i["S"])
    used = [k for k in range(n) if 0 <= slots[k] < slots_n]
    close("o", o[used], wo[used])
    close("S", S_out[slots[used].long()], wS[used])
    assert (o[[2, 4]] == 55).all()
    rest = [k for k in range(slots_n) if k not in slots.tolist()]
    assert (S_out[rest] == 77).all()
    kda.kda_glr_decode(params(i, io), *parts[:3], S, z=parts[3], slots=dev(slots), o=o)    # in place
    assert torch.equal(S[slots[used].long()], S_out[slots[used].long()]) and torch.equal(S[rest].cpu(), i["S"][rest])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("C", [5, 64, 200])
def test_commit(io, C):
    """Paths of any length, empty and out of range: those sessions are skipped."""
    n, R, slots_n = 8, 7, 11
    i = make_inputs(n * R, slots_n, C, IO[io], 33)
    paths = [[0, 1, 2], [], [6], [3, 1, 1, 5], [0, 7], [2, -1], [1, 2, 3, 4], [0]]
    m = 4
    path = torch.tensor([p + [99] * (m - len(p)) for p in paths], dtype=torch.int32)
    lens = torch.tensor([len(p) for p in paths], dtype=torch.int32)
    lens[7] = 5                                                  # more than max_len
    slots = torch.tensor([4, 3, 2, 1, 0, 10, 11, 9], dtype=torch.int32)     # the seventh's is out of range
    skip = {4, 5, 6, 7}
    start = torch.stack([i["S"][min(s, slots_n - 1)] for s in slots.tolist()])
    _, wS = tokens_ref(i, n, R, start, [[] if k in skip else p for k, p in enumerate(paths)])
    rows = [dev(i[k]).view(n, R, C) for k in ("x", "r", "i")]
    S, S_out = dev(i["S"]), torch.full((slots_n, C), 77.0, device=DEV)
    out = kda.kda_glr_commit(params(i, io), *rows, dev(path), dev(lens), S, S_out=S_out, slots=dev(slots))
    assert out is S_out and torch.equal(S.cpu(), i["S"])
    used = [k for k in range(n) if k not in skip]
    close("S", S_out[slots[used].long()], wS[used])
    assert torch.equal(S_out[3].cpu(), i["S"][3])                # an empty path copies
    assert (S_out[[0, 5, 6, 7, 8, 9, 10]] == 77).all()
    assert kda.kda_glr_commit(params(i, io), *rows, dev(path), dev(lens), S, slots=dev(slots)) is S
    assert torch.equal(S[slots[used].long()], S_out[slots[used].long()])
    rest = [0, 5, 6, 7, 8, 9, 10]
    assert torch.equal(S[rest].cpu(), i["S"][rest])


def test_commit_is_decode_of_the_path():
    """A straight path of all tokens and the same tokens decoded leave the same bytes."""
    n, R, C = 5, 6, 136
    i = make_inputs(n * R, n, C, torch.bfloat16, 34)
    rows = [dev(i[k]).view(n, R, C) for k in ("x", "r", "i")]
    S, S2 = dev(i["S"]), dev(i["S"])
    kda.kda_glr_decode(params(i, "bf16"), *rows, S)
    path = torch.arange(R, dtype=torch.int32, device=DEV).expand(n, R).contiguous()
    kda.kda_glr_commit(params(i, "bf16"), *rows, path, torch.full((n,), R, dtype=torch.int32, device=DEV), S2)
    assert torch.equal(S, S2)


# ---- batches of many tiles: set up by a kernel of their own, tickets over several rounds ----

def forward64(i, cu):
    """As glr_ref.mixer on the GPU: (o, S, state before each token), sequences side by side."""
    j = {k: v.to(DEV) if torch.is_tensor(v) else v for k, v in i.items()}
    s = steps(j)
    n, T, C = len(cu) - 1, cu[-1], i["C"]
    order = sorted(range(n), key=lambda k: cu[k] - cu[k + 1])
    S = torch.zeros(n, C, dtype=torch.float64, device=DEV) if j["S"] is None else j["S"].double()[order].clone()
    start, h, before = torch.tensor([cu[k] for k in order], device=DEV), *(torch.empty(T, C, dtype=torch.float64, device=DEV) for _ in range(2))
    for t in range(max(cu[k + 1] - cu[k] for k in range(n))):
        m = sum(cu[k + 1] - cu[k] > t for k in order)
        at = start[:m] + t
        before[at] = S[:m]
        S[:m] = s["a"][at] * S[:m] + s["b"][at]
        h[at] = S[:m]
    o = h if j["z"] is None else h * j["z"].double() * torch.sigmoid(j["z"].double())
    return s, j, o, S[torch.argsort(torch.tensor(order, device=DEV))], before, h


def gradients64(i, cu):
    s, j, _, _, before, h = forward64(i, cu)
    n, T, C = len(cu) - 1, cu[-1], i["C"]
    z = j["z"].double()
    e = torch.sigmoid(z)
    G = j["do"].double()
    out = {"dz": G * h * (e + z * e * torch.sigmoid(-z))}
    G = G * z * e
    carry = j["dS"].double().clone()
    for k in range(n):
        for t in range(cu[k + 1] - 1, cu[k] - 1, -1):
            G[t] += carry[k]
            carry[k] = s["a"][t] * G[t]
    dA = G * (s["a"] * before * s["la"] - s["a"] ** 2 * s["v"] * j["x"].double() * s["la"] / s["m"])
    out.update(dx=G * s["m"] * s["v"], di=G * s["b"] * s["v_"], dr=dA * s["w_"], dS_in=carry)
    out.update(dA_log=dA.sum(0), dr_bias=out["dr"].sum(0), di_bias=out["di"].sum(0))
    return out


@pytest.mark.parametrize("io, T, C, pad", [("bf16", 9000, 1024, 0), ("bf16", 20500, 300, 0), ("bf16", 9000, 1023, 1),
                                           ("bf16", 9000, 1000, 2), ("f32", 6000, 512, 0), ("f32", 6000, 519, 1)])
def test_many_tiles(io, T, C, pad):
    """Every way of copying rows (tensor copies, 4 bytes at a time, odd rows: `pad` widens the rows), over
    several rounds of tiles, with sequence borders in some of them."""
    cu = [0, 1, 77, 77, 4000, T - 13, T]
    i = make_inputs(T, len(cu) - 1, C, IO[io], 40 + C)
    i["A_log"] -= 0.7
    wide = {k: torch.empty(T, C + pad, dtype=IO[io], device=DEV)[:, :C].copy_(i[k]) for k in ("x", "r", "i", "z", "do")}
    p, S = params(i, io), dev(i["S"])
    st = torch.empty(-(-T // kda.KDA_GLR_CHUNK), C, device=DEV)
    ws = torch.full((kda.kda_glr_backward_workspace_bytes(p, len(cu) - 1, T),), 255, dtype=torch.uint8, device=DEV)
    _, _, wo, wS, before, _ = forward64(i, cu)
    runs = []
    for fill in (255, 0):                       # whatever the workspace holds
        ws.fill_(fill)
        o, So = kda.kda_glr_prefill(p, wide["x"], wide["r"], wide["i"], cu, z=wide["z"], S_in=S, states=st, workspace=ws)
        ws.fill_(fill)
        g = kda.kda_glr_backward(p, wide["x"], wide["r"], wide["i"], cu, st, wide["do"], z=wide["z"], S_in=S, dS_out=dev(i["dS"]),
                                 workspace=ws)
        assert kda.kda_workspace_status(ws) == kda.KDA_OK
        runs.append([o, So, st.clone()] + [getattr(g, k) for k in GRADS])
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    close("o", o, wo.cpu())
    close("S", So, wS.cpu())
    close("states", st, before[::kda.KDA_GLR_CHUNK].cpu())
    want = gradients64(i, cu)
    for k in GRADS:   # sums of T terms: (T / 700)^1/2 times the usual tolerance of a sum
        close(k, getattr(g, k), want[k].cpu(), SUM_TOL * (T / 700) ** 0.5 if k in ("dA_log", "dr_bias", "di_bias") else None)


def test_two_large_calls_at_once():
    """Two walks of several rounds and a cooperative one beside them, each on its stream."""
    T, C = 6000, 2048
    i = make_inputs(T, 2, C, torch.bfloat16, 50)
    cu = [0, 2500, T]
    p = params(i, "bf16")
    x, r, s, z, S, do, dS = (dev(i[k]) for k in ("x", "r", "i", "z", "S", "do", "dS"))
    small = [t[:300].contiguous() for t in (x, r, s, z)]
    st = torch.empty(-(-T // 64), C, device=DEV)
    want = kda.kda_glr_prefill(p, x, r, s, cu, z=z, S_in=S, states=st)
    gw = kda.kda_glr_backward(p, x, r, s, cu, st, do, z=z, S_in=S, dS_out=dS)
    sw = kda.kda_glr_prefill(p, *small[:3], [0, 300], z=small[3])
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        outs.append((kda.kda_glr_prefill(p, x, r, s, cu, z=z, S_in=S, stream=streams[0]),
                     kda.kda_glr_backward(p, x, r, s, cu, st, do, z=z, S_in=S, dS_out=dS, stream=streams[1]),
                     kda.kda_glr_prefill(p, *small[:3], [0, 300], z=small[3], stream=streams[2])))
    torch.cuda.synchronize()
    for a, g, b in outs:
        assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1]) and torch.equal(b[0], sw[0]) and torch.equal(b[1], sw[1])
        for k in GRADS:
            assert torch.equal(getattr(g, k), getattr(gw, k))


def test_rows_past_32_bits_of_elements():
    """Row offsets past 2^31 elements and 2^32 bytes: the last of 600000 tokens whose rows lie 4100 elements apart."""
    T, C, stride = 600000, 64, 4100
    base = torch.zeros(T * stride, dtype=torch.bfloat16, device=DEV).view(T, stride)
    i = make_inputs(2000, 1, C, torch.bfloat16, 51, state=False)
    parts = {k: base[:, j * 64:(j + 1) * 64] for j, k in enumerate(("x", "r", "i", "z", "do"))}
    for k, t in parts.items():
        t[-2000:] = dev(i[k])
        if k == "r":
            t[-2001] = float("inf")            # a token whose decay is e^-1 or less, and whose input is zero, like all before
    p = params(i, "bf16")
    st = torch.empty(-(-T // 64), C, device=DEV)
    o, S = kda.kda_glr_prefill(p, parts["x"], parts["r"], parts["i"], [0, T], z=parts["z"], states=st)
    wo, wS = mixer(i, [0, 2000])
    close("o", o[-2000:], wo)
    close("S", S, wS)
    assert not o[:-2000].any()
    g = kda.kda_glr_backward(p, parts["x"], parts["r"], parts["i"], [0, T], st, parts["do"], z=parts["z"])
    want = gradients(i, [0, 2000])
    for k in ("dx", "dr", "di", "dz"):
        close(k, getattr(g, k)[-2000:], want[k])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("C", [77, 128, 130])
@pytest.mark.parametrize("most", [5, 40, 90])
def test_many_short_sequences(io, C, most):
    """More sequences than travel in a launch's arguments, several borders to a warp's tokens or a few to a tile;
    borders on the tiles', sequences without tokens; the states in place."""
    g = torch.Generator().manual_seed(most)
    lens = torch.randint(0, most, (60,), generator=g).tolist()
    lens += [-sum(lens) % 64, 64, 0, 63, 1, 64 - 8, 8]
    cu = cumsum(lens)
    i = make_inputs(cu[-1], len(lens), C, IO[io], 31 + most)
    _, S, _, _ = check(i, io, cu)
    own = i["S"].to(DEV)
    prefill({**i, "S": None}, io, cu)                                   # (another call in between)
    o, same = kda.kda_glr_prefill(params(i, io), dev(i["x"]), dev(i["r"]), dev(i["i"]), cu, z=dev(i["z"]), S_in=own, S_out=own)
    assert same is own and torch.equal(own, S)
