"""The state space prefill's kernel variants by size: wide scans, cut sequences
over several groups, chunk walks that wait for a long preparation.  Against
the definition token by token in 64 bits."""
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


def check(i, io, lens, algo="auto"):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    p = kda.make_ssm_params(dev(i["conv_w"]), dev(i["A_log"]), dev(i["dt_bias"]), head_dim=i["P"], state_dim=i["N"],
                            num_groups=i["G"], D=dev(i["D"]), conv_b=dev(i["conv_b"]), io_dtype=io, algo=algo)
    ws = torch.empty(kda.kda_ssm_prefill_workspace_bytes(p, len(lens), cu[-1]), dtype=torch.uint8, device=DEV)
    o, S, ring = kda.kda_ssm_prefill(p, dev(i["xbc"]), dev(i["dt"]), cu, z=dev(i["z"]), S_in=dev(i["S"]),
                                     ring_in=dev(i["ring"]), workspace=ws)
    wo, wS, wr = mixer(i, cu)
    assert kda.kda_workspace_status(ws) == kda.KDA_OK
    close("o", o, wo)
    close("S", S, wS)
    assert torch.equal(ring.cpu(), wr)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("P, N, H, G", [(64, 64, 40, 4), (64, 128, 40, 1), (128, 64, 21, 3), (128, 128, 20, 2)])
@pytest.mark.parametrize("lens", [[9, 0, 1, 37], [8, 16, 64, 7]])
def test_wide_scans(io, P, N, H, G, lens):
    """More (sequence, head, 16 columns) slices than four an SM: the scan takes 64 columns a CTA."""
    assert len(lens) * H * (P // 16) > 608
    check(make_inputs(sum(lens), len(lens), H, P, N, G, IO[io], 71 + H), io, lens, "scan")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("H, P, N, G, lens", [
    (6, 64, 128, 2, [1500, 30, 700, 0]),         # three heads a group: the second unit holds one
    (3, 128, 128, 3, [1300, 64]),
    (10, 64, 64, 2, [900, 900] + [5] * 16)])     # more sequences than travel with the launch
def test_cut_sequences_of_several_groups(io, H, P, N, G, lens):
    i = make_inputs(sum(lens), len(lens), H, P, N, G, IO[io], 81 + H)
    i["A_log"] -= 2.0
    check(i, io, lens)


@pytest.mark.parametrize("lens", [[1300], [700, 0, 1, 600]])
def test_walks_behind_a_long_preparation(lens):
    """More preparation blocks (17 a chunk) than run at once, so the walks start behind it."""
    H = G = 16
    assert sum(lens) // 64 * (G + H // 32 + 1) > 304
    check(make_inputs(sum(lens), len(lens), H, 64, 64, G, torch.bfloat16, 91), "bf16", lens)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_more_sequences_than_a_grid_dimension(io):
    """70001 sequences of 0 to 2 tokens, state and ring in place, against the token calls."""
    H, P, N, n, t = 1, 64, 64, 70001, IO[io]
    ch = H * P + 2 * N
    g = torch.Generator(device=DEV).manual_seed(7)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)
    p = kda.make_ssm_params(rn(ch, 4) * 0.5, torch.zeros(H, device=DEV), rn(H) * 0.1 - 3, head_dim=P, state_dim=N, D=rn(H),
                            io_dtype=io)
    lens = torch.tensor([i * 7919 % 3 for i in range(n)])
    cu = [0] + lens.cumsum(0).tolist()
    x, d, z = rn(cu[-1], ch).to(t), rn(cu[-1], H).to(t), rn(cu[-1], H * P).to(t)
    S, ring = rn(n, H, N, P) * 0.3, rn(n, 3, ch).to(t)
    S1, r1, S2, r2 = S.clone(), ring.clone(), S.clone(), ring.clone()
    o, _, _ = kda.kda_ssm_prefill(p, x, d, cu, z=z, S_in=S1, S_out=S1, ring_in=r1, ring_out=r1)
    want = torch.zeros_like(o)
    start, lens = torch.tensor(cu[:-1], device=DEV), lens.to(DEV)
    for k in range(2):
        live = (lens > k).nonzero()[:, 0]
        want[start[live] + k] = kda.kda_ssm_decode(p, x[start[live] + k], d[start[live] + k], S2, r2, z=z[start[live] + k],
                                                   slots=live.int())
    close("o", o, want.double().cpu())
    close("S", S1, S2.double().cpu())
    assert torch.equal(r1, r2) and torch.equal(S1[lens == 0], S[lens == 0])


def test_state_pools_past_2_to_31_elements():
    """The last slots of a pool of 2.3 G state values: single tokens (both forms), a tree and a commit
    there equal the same calls on a pool of their own."""
    import kda_synth
    from kda_testlib import kda_params
    H, slots = 64, 2200
    pool = torch.empty(slots, H, 128, 128, device=DEV)
    assert pool.numel() > 2 ** 31
    at = torch.tensor([slots - 1, 3, slots - 2], dtype=torch.int32, device=DEV)
    own = torch.arange(3, dtype=torch.int32, device=DEV)
    S = torch.randn(3, H, 128, 128, generator=torch.Generator(device=DEV).manual_seed(8), device=DEV) * 0.1

    def both(call, ring):
        big = torch.zeros(slots, *ring.shape[1:], dtype=ring.dtype, device=DEV)
        pool[at.long()], big[at.long()] = S, ring
        small, r = S.clone(), ring.clone()
        a, b = call(pool, big, at), call(small, r, own)
        assert torch.equal(a, b)
        assert torch.equal(pool[at.long()], small) and torch.equal(big[at.long()], r)

    for G in (1, 2):                                       # (one group of 64 heads: two kernels)
        i = make_inputs(3, 3, H, 128, 128, G, torch.bfloat16, 95 + G)
        p = kda.make_ssm_params(dev(i["conv_w"]), dev(i["A_log"]), dev(i["dt_bias"]), head_dim=128, state_dim=128, num_groups=G,
                                D=dev(i["D"]), conv_b=dev(i["conv_b"]))
        assert (kda.kda_ssm_decode_workspace_bytes(p, 3) > 0) == (G == 1)
        both(lambda s, r, k: kda.kda_ssm_decode(p, dev(i["xbc"]), dev(i["dt"]), s, r, z=dev(i["z"]), slots=k), dev(i["ring"]))
    kp = kda_params(kda_synth.draw_params(H, 9), "bf16")
    q, k, v, z, b, gout = (t.reshape(3, 5, -1).to(DEV) for t in kda_synth.draw_tokens(15, H, 10, torch.bfloat16).fields())
    ring = torch.randn(3, 3, 3, H * 128, generator=torch.Generator(device=DEV).manual_seed(11), device=DEV).bfloat16()
    par = torch.tensor([[-1, 0, 0, 1, 2]] * 3, dtype=torch.int32, device=DEV)
    both(lambda s, r, k_: kda.kda_decode_tree(kp, q, k, v, z, b, gout, par, s, r, slots=k_), ring)
    path, lens = torch.tensor([[0, 1, 3]] * 3, dtype=torch.int32, device=DEV), torch.tensor([3, 2, 1], dtype=torch.int32, device=DEV)

    def commit(s, r, k_):
        kda.kda_tree_commit(kp, q, k, v, z, b, path, lens, s, r, slots=k_)
        return lens
    both(commit, ring)


@pytest.mark.parametrize("io, algo", [("f32", "auto"), ("bf16", "auto"), ("bf16", "scan")])
def test_rows_past_2_to_31_elements(io, algo):
    """Rows so far apart that the last ones lie past 2^31 elements equal the same rows packed."""
    H, P, N, T, stride = 2, 64, 64, 200, 12_000_000
    lens, ch, W = [70, 1, 129], H * P + 2 * N, H * P
    i = make_inputs(T, 3, H, P, N, 1, IO[io], 99)
    far = torch.empty(T * stride, dtype=IO[io], device=DEV).view(T, stride)
    assert far[-1].storage_offset() > 2 ** 31
    at = stride - W - ch - 8
    far[:, at:at + W], far[:, at + W:at + W + ch], far[:, -8:-8 + H] = dev(i["z"]), dev(i["xbc"]), dev(i["dt"])
    p = kda.make_ssm_params(dev(i["conv_w"]), dev(i["A_log"]), dev(i["dt_bias"]), head_dim=P, state_dim=N, D=dev(i["D"]),
                            conv_b=dev(i["conv_b"]), io_dtype=io, algo=algo)
    cu = [0, 70, 71, 200]
    kw = dict(S_in=dev(i["S"]), ring_in=dev(i["ring"]))
    got = kda.kda_ssm_prefill(p, far[:, at + W:at + W + ch], far[:, -8:-8 + H], cu, z=far[:, at:at + W], **kw)
    want = kda.kda_ssm_prefill(p, dev(i["xbc"]), dev(i["dt"]), cu, z=dev(i["z"]), **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    S, ring = torch.zeros(T, H, N, P, device=DEV), torch.zeros(T, 3, ch, dtype=IO[io], device=DEV)
    S2, ring2 = S.clone(), ring.clone()
    o = kda.kda_ssm_decode(p, far[:, at + W:at + W + ch], far[:, -8:-8 + H], S, ring, z=far[:, at:at + W])
    o2 = kda.kda_ssm_decode(p, dev(i["xbc"]), dev(i["dt"]), S2, ring2, z=dev(i["z"]))
    assert torch.equal(o, o2) and torch.equal(S, S2) and torch.equal(ring, ring2)
