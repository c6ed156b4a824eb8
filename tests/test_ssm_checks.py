"""Workspace sizes and argument checks of the state space and draft-tree calls
on the host: nothing here reaches a GPU."""
import ctypes
import itertools

import pytest

import gated_delta_rule_04_gb300 as kda
from gated_delta_rule_04_gb300 import build as kbuild
from test_ssm_tree_abi import struct


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kda.lib()


@pytest.mark.parametrize("H, P, N, G", [(64, 64, 128, 4), (96, 64, 128, 8), (1, 128, 128, 1), (6, 64, 64, 2), (2000, 64, 64, 1)])
def test_prefill_workspace_grows_with_the_batch(L, H, P, N, G):
    """A workspace for the largest call serves every smaller one: the size falls neither with
    more sequences (around the number from which sequences are no longer cut) nor with
    more tokens."""
    for io in (kda.KDA_DTYPE_BF16, kda.KDA_DTYPE_F32):
        p = struct(num_heads=H, head_dim=P, state_dim=N, num_groups=G, io_dtype=io)
        size = lambda n, T: L.kda_ssm_prefill_workspace_bytes(ctypes.byref(p), n, T)
        for T in (0, 63, 8192):
            sizes = [size(n, T) for n in itertools.chain(range(1, 160), range(160, 3000, 97), (70000,))]
            assert sizes == sorted(sizes)
        for n in (1, 25, 26, 37, 38, 39, 200):
            sizes = [size(n, T) for T in sorted((0, 1, n - 1, n, 63, 64, 65, 1000, 8192, 100000))]
            assert sizes == sorted(sizes)


def test_decode_workspace_grows_with_the_batch(L):
    for H, G in ((32, 1), (33, 1), (64, 8), (80, 2)):
        p = struct(num_heads=H, num_groups=G)
        sizes = [L.kda_ssm_decode_workspace_bytes(ctypes.byref(p), n) for n in range(0, 600)]
        assert sizes == sorted(sizes)


# ---- the binding's own checks (CPU and meta tensors: nothing reaches the library) ----

def ssm_params(device="cpu", **kw):
    import torch
    t = dict(conv_w=torch.zeros(768, 4, device=device), A_log=torch.zeros(4, device=device), dt_bias=torch.zeros(4, device=device))
    t.update(kw)
    return kda.make_ssm_params(**t, head_dim=64, state_dim=128, num_groups=2)


def kda_params(**kw):
    import torch
    t = dict(conv_w=torch.zeros(3, 256, 4), A_log=torch.zeros(2), dt_bias=torch.zeros(256), norm_w=torch.zeros(128))
    t.update(kw)
    return kda.make_params(**t)


@pytest.mark.parametrize("name, shape", [("conv_w", (768, 4)), ("conv_b", (768,)), ("A_log", (4,)), ("dt_bias", (4,)), ("D", (4,))])
def test_ssm_parameters_lie_on_one_device(name, shape):
    import torch
    with pytest.raises(ValueError, match="one device"):
        ssm_params(**{name: torch.zeros(shape, device="meta")})


@pytest.mark.parametrize("name, shape", [("conv_w", (3, 256, 4)), ("A_log", (2,)), ("dt_bias", (256,)), ("norm_w", (128,))])
def test_kda_parameters_lie_on_one_device(name, shape):
    import torch
    with pytest.raises(ValueError, match="one device"):
        kda_params(**{name: torch.zeros(shape, device="meta")})


def test_parameters_lie_on_the_device_of_the_call():
    """Parameters of another device (their struct says so here) are refused before anything else
    is looked at."""
    import torch
    bf = torch.bfloat16
    p, k = ssm_params(), kda_params()
    assert p.device == -1 and k.device == -1
    p.device = k.device = 1
    x, d = torch.zeros(5, 768, dtype=bf), torch.zeros(5, 4, dtype=bf)
    rows = {n: torch.zeros(2, 5, 256, dtype=bf) for n in ("q", "k", "v", "z")}
    b, par = torch.zeros(2, 5, 2, dtype=bf), torch.zeros(2, 5, dtype=torch.int32)
    S, ring = torch.zeros(2, 2, 128, 128), torch.zeros(2, 3, 3, 256, dtype=bf)
    for call in (lambda: kda.kda_ssm_prefill(p, x, d, [0, 5]),
                 lambda: kda.kda_ssm_decode(p, x, d, torch.zeros(5, 4, 128, 64), torch.zeros(5, 3, 768, dtype=bf)),
                 lambda: kda.kda_decode_tree(k, **rows, b=b, gout=rows["q"], parents=par, S=S, ring=ring),
                 lambda: kda.kda_tree_commit(k, **rows, b=b, path=par, path_len=par[:, 0].contiguous(), S_in=S, ring_in=ring)):
        with pytest.raises(ValueError, match="on cuda:1"):
            call()


def test_workspaces_are_dense():
    """An expanded or strided workspace has more bytes by its shape than it owns."""
    import torch
    like = torch.zeros(1)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(512, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            kda._workspace(ws, like, None, None)
    ws = torch.zeros(512, dtype=torch.uint8)
    assert kda._workspace(ws, like, None, None) == (ws, ws.data_ptr(), 512)
