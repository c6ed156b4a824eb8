"""The state space mixer away from inputs of ordinary size: large and tiny
values, states that only pass through, decays without bound, tokens of very
unlike size in one chunk.  Against its definition token by token in 64 bits,
with the tolerances of ``ssm_ref`` unless a test derives its own."""
import math

import pytest
import torch

import gated_delta_rule_04_gb300 as kda
from ssm_ref import TOL, close, make_inputs, mixer

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


def prefill(i, io, cu, rows=slice(None), **kw):
    kw = {"S_in": dev(i["S"]), "ring_in": dev(i["ring"]), **kw}
    return kda.kda_ssm_prefill(params(i, io), dev(i["xbc"][rows]), dev(i["dt"][rows]), cu, z=dev(i["z"][rows]), **kw)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [2.0 ** 22, 2.0 ** 25])
def test_large_states_of_cut_and_continued_sequences(io, scale):
    """Inputs whose states pass 2^44: every piece of a cut sequence and every continued
    prompt starts from one, and its first chunk's outputs read it."""
    cu = cumsum([1500, 40])
    i = make_inputs(cu[-1], 2, 2, 64, 128, 1, IO[io], 61, bias=False)
    i["A_log"] -= 2.0
    i["xbc"] = (i["xbc"].float() * scale).to(IO[io])
    i["ring"] = (i["ring"].float() * scale).to(IO[io])
    i["S"] *= scale ** 2
    wo, wS, _ = mixer(i, cu)
    assert float(wS.abs().max()) > 2.0 ** 44
    o, S, _ = prefill(i, io, cu)
    close("o", o, wo)
    close("S", S, wS)
    # the same sequence in two parts, the second from the first one's state
    T = 300
    o1, S1, ring = prefill(i, io, [0, T], slice(0, T), S_in=dev(i["S"][:1]), ring_in=dev(i["ring"][:1]))
    o2, S2, _ = prefill(i, io, [0, 1500 - T], slice(T, 1500), S_in=S1, ring_in=ring)
    close("o in parts", torch.cat([o1, o2]), wo[:1500])
    close("S in parts", S2, wS[:1])


@pytest.mark.parametrize("io, algo", [("f32", "auto"), ("bf16", "auto"), ("bf16", "scan")])
@pytest.mark.parametrize("lens", [[0, 5, 0], [0], [0, 0] + [3] * 16])
def test_states_of_empty_sequences_pass_through_bit_by_bit(io, algo, lens):
    H, P, N = 3, 64, 64
    cu = cumsum(lens)
    i = make_inputs(cu[-1], len(lens), H, P, N, 1, IO[io], 62)
    empty = [s for s, n in enumerate(lens) if n == 0]
    for s in empty:
        i["S"][s, 0, 3, 5] = float("inf")
        i["S"][s, 1, 60, 7] = float("nan")
        i["S"][s, 2, 1, :] = 1e-42        # below fp32's normal range
        i["S"][s, 2, 2, :] = 3e38
    S_in, ring_in = dev(i["S"]), dev(i["ring"])
    _, S, ring = kda.kda_ssm_prefill(params(i, io, algo), dev(i["xbc"]), dev(i["dt"]), cu, z=dev(i["z"]), S_in=S_in,
                                     ring_in=ring_in)
    for s in empty:
        assert torch.equal(S[s].view(torch.int32), S_in[s].view(torch.int32))
        assert torch.equal(ring[s].view(torch.uint8), ring_in[s].view(torch.uint8))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[64], [70, 3], [1], [200]])
def test_a_decay_without_bound(io, lens):
    """exp(A_log) past fp32's range: each of that head's tokens leaves only its own update,
    in a chunk that the sequence fills and in one that it does not."""
    cu = cumsum(lens)
    i = make_inputs(cu[-1], len(lens), 4, 64, 64, 2, IO[io], 63)
    i["A_log"][1] = 90.0
    wo, wS, _ = mixer(i, cu)
    o, S, _ = prefill(i, io, cu)
    close("o", o, wo)
    close("S", S, wS)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("skip", [True, False])
def test_small_matrices_beside_large_rows(io, skip):
    """B and C near 2^-38, x near 2^20: without the skip term the outputs are the scan's alone,
    whose weights are near 2^-76."""
    H, P, N = 2, 64, 128
    cu = cumsum([140, 20])
    i = make_inputs(cu[-1], 2, H, P, N, 1, IO[io], 64, bias=False, skip=skip)
    scale = torch.full((H * P + 2 * N,), 2.0 ** -38)
    scale[:H * P] = 2.0 ** 20
    for k in ("xbc", "ring"):
        i[k] = (i[k].float() * scale).to(IO[io])
    i["S"] *= 2.0 ** -18
    wo, wS, _ = mixer(i, cu)
    o, S, _ = prefill(i, io, cu)
    close("o", o, wo)
    close("S", S, wS)


def test_outputs_past_the_range_never_look_finite():
    """C and state so large that their product passes fp32's range: what the definition puts
    past it comes out infinite or NaN, and the tokens of ordinary size in its chunk as they are."""
    H, P, N, T = 2, 64, 64, 80
    i = make_inputs(T, 1, H, P, N, 1, torch.bfloat16, 65, bias=False)
    i["A_log"] -= 6.0
    i["S"] *= 2.0 ** 108
    i["xbc"][:, H * P + N:] = (i["xbc"][:, H * P + N:].float() * 2.0 ** 22).to(torch.bfloat16)
    i["xbc"][66:, H * P + N:] = 0.25                     # (from token 69 on the whole conv window)
    wo, wS, _ = mixer(i, [0, T])
    o, S, _ = prefill(i, "bf16", [0, T])
    top = float(torch.finfo(torch.bfloat16).max)
    o = o.cpu().double()
    assert not (torch.isfinite(o) & (wo.abs() > 1.01 * top)).any()
    assert torch.isfinite(wo[69:].bfloat16()).all()
    close("o", o[69:], wo[69:], TOL[torch.bfloat16])
    close("S", S, wS)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("at", [0, 17, 63, 64, 90])
@pytest.mark.parametrize("what", ["B", "C", "BC", "x"])
def test_one_large_token_leaves_the_others_their_digits(io, at, what):
    """A token whose B or x is 2^10, whose C 2^18, or B and C 2^9 each larger than the others' of
    its chunk.  Outputs of the other tokens are held to the tolerance each by itself, where
    the large one has not reached them (C: nowhere; x and B: before it)."""
    H, P, N, T = 2, 64, 128, 130
    i = make_inputs(T, 1, H, P, N, 1, IO[io], 66, bias=False)
    i["conv_w"][:, :3] = 0.0                              # (a token's rows are its own)
    cols = {"x": [slice(0, H * P)], "B": [slice(H * P, H * P + N)], "C": [slice(H * P + N, H * P + 2 * N)]}
    for w in what:
        for c in cols[w]:
            i["xbc"][at, c] = (i["xbc"][at, c].float() * {'C': 2 ** 18, 'BC': 2 ** 9}.get(what, 2 ** 10)).to(IO[io])
    wo, wS, _ = mixer(i, [0, T])
    o, S, _ = prefill(i, io, [0, T])
    close("S", S, wS)
    o = o.cpu()
    for t in range(T):
        if t != at and (what == "C" or t < at):
            close(f"o[{t}]", o[t], wo[t])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_a_large_token_that_decays_leaves_the_state_its_digits(io):
    """The first token's B is 2^10 larger, and gone after a few steps: what the later ones
    leave in the state keeps an fp32 state's precision."""
    H, P, N, T = 2, 64, 64, 64
    i = make_inputs(T, 1, H, P, N, 1, IO[io], 67, state=False)
    i["A_log"][:] = 2.0
    i["dt_bias"][:] = 0.5                                 # a step's decay is about e^-7
    i["conv_w"][:, :3] = 0.0
    c = slice(H * P, H * P + N)
    i["xbc"][0, c] = (i["xbc"][0, c].float() * 1024).to(IO[io])
    wo, wS, _ = mixer(i, [0, T])
    o, S, _ = prefill(i, io, [0, T])
    close("S", S, wS)
    for t in (0, 20, 40, 63):
        close(f"o[{t}]", o[t], wo[t])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("at", [17, 63, 90])
def test_an_x_far_larger_than_those_before_it(io, at):
    """The same with an x 2^18 larger, whose channels' earlier values share its scale.

    The state: an operand pair ends at 2^-25 where the state is scaled to below 2^14, by a
    bound of at most 4 max|x| max|B| sum(dt) beside what there was: 64 tokens of it, times a
    B of less than 2^5, are 2^-25 max|x| max|B| sum(dt) an element."""
    H, P, N, T = 2, 64, 64, 130
    i = make_inputs(T, 1, H, P, N, 1, IO[io], 69, bias=False)
    i["conv_w"][:, :3] = 0.0
    i["xbc"][at, :H * P] = (i["xbc"][at, :H * P].float() * 2 ** 18).to(IO[io])
    wo, wS, _ = mixer(i, [0, T])
    o, S, _ = prefill(i, io, [0, T])
    u = i["xbc"].double() * i["conv_w"][:, 3].double()
    u = (u * torch.sigmoid(u)).abs()
    steps = torch.nn.functional.softplus(i["dt"].double() + i["dt_bias"].double())[64 * (at // 64):][:64].sum(0).max()
    most = float(u[:, :H * P].max() * u[:, H * P:H * P + N].max() * steps)
    close("S", S, wS, TOL[torch.float32] + 2.0 ** -25 * most * math.sqrt(wS.numel()) / float(wS.norm()))
    o = o.cpu()
    for t in range(at):
        close(f"o[{t}]", o[t], wo[t])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_a_large_x_that_decays_leaves_the_state_its_digits(io):
    """As with B above, of an x: the bound that scales the state knows the decay."""
    H, P, N, T = 2, 64, 64, 64
    i = make_inputs(T, 1, H, P, N, 1, IO[io], 70, state=False)
    i["A_log"][:] = 2.0
    i["dt_bias"][:] = 0.5
    i["conv_w"][:, :3] = 0.0
    i["xbc"][0, :H * P] = (i["xbc"][0, :H * P].float() * 1024).to(IO[io])
    wo, wS, _ = mixer(i, [0, T])
    o, S, _ = prefill(i, io, [0, T])
    close("S", S, wS)
    for t in (0, 20, 40, 63):
        close(f"o[{t}]", o[t], wo[t])


@pytest.mark.parametrize("call", ["prefill", "token", "tokens in two kernels"])
def test_silu_to_fp32_rounding(call):
    """fp32 I/O, one token from a zero state: every element of the state is dt * SiLU(b) * SiLU(x).

    Roundings of 2^-24 each, at most: SiLU 8 (exp 2 ulp = 4, the sum 1, a reciprocal of 1 ulp = 2,
    the product 1), of B and of x; softplus 8 (exp 4, log1p 2 ulp = 4); two products 2: 26."""
    H, P, N = 2, 64, 64
    i = make_inputs(1, 1, H, P, N, 1, torch.float32, 68, state=False, bias=False)
    i["conv_w"][:] = torch.tensor([0.0, 0.0, 0.0, 1.0])
    i["xbc"][0, :H * P] = torch.linspace(-40, 40, H * P)
    i["xbc"][0, H * P:H * P + N] = torch.linspace(-30, 30, N)
    _, want, _ = mixer(i, [0, 1])
    n = 1100 if call == "tokens in two kernels" else 1     # (more than 32 MB of states)
    p = params(i, "f32")
    if call == "prefill":
        _, S, _ = prefill(i, "f32", [0, 1])
    else:
        assert (kda.kda_ssm_decode_workspace_bytes(p, n) > 0) == (n > 1)
        S = torch.zeros(n, H, N, P, device=DEV)
        ring = torch.zeros(n, 3, H * P + 2 * N, device=DEV)
        kda.kda_ssm_decode(p, dev(i["xbc"]).repeat(n, 1), dev(i["dt"]).repeat(n, 1), S, ring, z=dev(i["z"]).repeat(n, 1))
    err = ((S.cpu().double() - want) / want).abs().max()
    assert float(err) <= 26 * 2.0 ** -24


@pytest.mark.parametrize("call", ["prefill f32", "prefill bf16", "prefill bf16 scan", "tokens f32", "tokens bf16",
                                  "tokens f32 in two kernels"])
def test_a_slow_decay_over_many_tokens(call):
    """A decay of about 1.5e-4 a token: its distance from 1 is a few thousand steps of fp32, so a
    rounding of one sign would show in a state that is multiplied by it 3000 times."""
    H, P, N, T = 33 if "two" in call else 2, 64, 64, 3000
    io = "f32" if "f32" in call else "bf16"
    i = make_inputs(T, 1, H, P, N, 1, IO[io], 72)
    i["A_log"][:] = -3.0
    i["dt_bias"][:] = math.log(math.expm1(0.003))
    _, wS, _ = mixer(i, [0, T])
    if "prefill" in call:
        p = params(i, io, "scan" if "scan" in call else "auto")
        _, S, _ = kda.kda_ssm_prefill(p, dev(i["xbc"]), dev(i["dt"]), [0, T], S_in=dev(i["S"]), ring_in=dev(i["ring"]))
    else:
        p, S, ring, x, d = params(i, io), dev(i["S"]), dev(i["ring"]), dev(i["xbc"]), dev(i["dt"])
        assert (kda.kda_ssm_decode_workspace_bytes(p, 1) > 0) == ("two" in call)
        for t in range(T):
            kda.kda_ssm_decode(p, x[t:t + 1], d[t:t + 1], S, ring)
    for h in range(H):
        close(f"S[{h}]", S[:, h], wS[:, h])
