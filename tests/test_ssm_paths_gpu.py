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
