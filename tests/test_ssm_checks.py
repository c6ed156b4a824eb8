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
