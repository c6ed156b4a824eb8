"""The bounded wait between a session's CTAs in kda_draft_verify, made to run out: nothing faults or hangs.

The library's own entry for this takes the limit of the wait.  A minus in the first entries of a row makes the CTA
that sums them go over its piece a second time, one entry a lane and turn, which takes it a large part of a
millisecond; the others wait one microsecond and give up, and the one they wait for does not."""
import ctypes

import pytest
import torch

import gated_delta_rule_04_gb300 as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
V = 1 << 23


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_04_gb300 import build as kbuild
    kbuild.build()
    kda.lib()


def call(n, limit_ns, row, u_next, q=None):
    f = kda.lib().kda_draft_verify_wait
    f.argtypes, f.restype = kda.lib().kda_draft_verify.argtypes + [ctypes.c_uint64], ctypes.c_int
    i32 = dict(dtype=torch.int32, device=DEV)
    tokens, parents = torch.zeros(n, 2, **i32), torch.full((n, 2), -1, **i32)
    parents[:, 1] = 0                                    # the chosen token, and a child (token 0, whose p is no number: refused)
    path, length, nxt = torch.full((n, 2), 9, **i32), torch.full((n,), 9, **i32), torch.full((n,), 9, **i32)
    u = torch.full((n, 2), 0.5, device=DEV)
    st = f(kda.KDA_DTYPE_F32, n, 2, V, row.data_ptr(), 0, 0, None, 0, None if q is None else q.data_ptr(), 0, 0, None, 0,
           tokens.data_ptr(), parents.data_ptr(), u.data_ptr(), u_next.data_ptr(), 2, path.data_ptr(), length.data_ptr(),
           nxt.data_ptr(), torch.cuda.current_stream().cuda_stream, limit_ns)
    assert st == kda.KDA_OK
    torch.cuda.synchronize()
    return path.tolist(), length.tolist(), nxt.tolist()


@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("n", [1, 6])
def test_a_wait_that_runs_out_leaves_no_token(n, drawn):
    row = torch.full((V,), 2.0 ** -23, device=DEV)
    q = row * 0.5 if drawn else None
    row[0] = -1.0
    u_next = torch.linspace(0.03, 0.97, n, device=DEV)   # the token in the CTA that is late, and in those that gave up
    path, length, nxt = call(n, 1000, row, u_next, q)
    assert nxt == [-1] * n
    assert length == [1] * n and path == [[0, -1]] * n
    # the same call with the usual limit: V - 1 entries are equal, and u_next (V - 1) of them lie before the token
    path, length, nxt = call(n, 2 * 10 ** 9, row, u_next, q)
    assert length == [1] * n and path == [[0, -1]] * n
    assert nxt == [1 + int(u * (V - 1)) for u in u_next.double().tolist()]
