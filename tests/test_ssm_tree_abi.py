"""Argument checks of the state space and draft-tree entry points, on the
host: every call here is refused (or empty) before anything is enqueued."""
import ctypes

import pytest
import torch

import gated_delta_rule_04_gb300 as kda
from gated_delta_rule_04_gb300 import build as kbuild
from test_abi import params as kda_struct

FAKE = 0x10000  # aligned non-null address; never dereferenced on these paths


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kda.lib()


def struct(**kw):
    d = dict(num_heads=4, head_dim=64, state_dim=128, num_groups=2, conv_kernel=4, io_dtype=kda.KDA_DTYPE_BF16,
             algo=kda.KDA_ALGO_AUTO, conv_w=FAKE, conv_b=None, A_log=FAKE, dt_bias=FAKE, D=None)
    d.update(kw)
    return kda.kda_ssm_params(**d)


def prefill(L, p, cu=(0, 64), T=None, sx=0, sd=0, sz=0, ws=FAKE, ws_bytes=1 << 40, null_cu=False, **ptrs):
    arr = (ctypes.c_int64 * len(cu))(*cu)
    a = dict(xbc=FAKE, dt=FAKE, z=FAKE, S_in=None, S_out=FAKE, ring_in=None, ring_out=FAKE, o=FAKE)
    a.update(ptrs)
    return L.kda_ssm_prefill(ctypes.byref(p), a["xbc"], sx, a["dt"], sd, a["z"], sz, None if null_cu else arr, len(cu) - 1,
                             cu[-1] if T is None else T, a["S_in"], a["S_out"], a["ring_in"], a["ring_out"], a["o"], ws,
                             ws_bytes, None)


def decode(L, p, n=3, sx=0, sd=0, sz=0, slots=None, n_slots=3, ws=FAKE, ws_bytes=1 << 40, **ptrs):
    a = dict(xbc=FAKE, dt=FAKE, z=FAKE, S=FAKE, ring=FAKE, o=FAKE)
    a.update(ptrs)
    return L.kda_ssm_decode(ctypes.byref(p), n, a["xbc"], sx, a["dt"], sd, a["z"], sz, slots, n_slots, a["S"], a["ring"],
                            a["o"], ws, ws_bytes, None)


BAD_PARAMS = [
    (dict(num_heads=0), kda.KDA_ERR_INVALID_ARG),
    (dict(num_groups=0), kda.KDA_ERR_INVALID_ARG),
    (dict(num_groups=3), kda.KDA_ERR_INVALID_ARG),
    (dict(head_dim=32), kda.KDA_ERR_UNSUPPORTED),
    (dict(state_dim=256), kda.KDA_ERR_UNSUPPORTED),
    (dict(conv_kernel=3), kda.KDA_ERR_UNSUPPORTED),
    (dict(io_dtype=5), kda.KDA_ERR_INVALID_ARG),
    (dict(algo=9), kda.KDA_ERR_INVALID_ARG),
    (dict(algo=kda.KDA_ALGO_CHUNKED_SEGMENTS), kda.KDA_ERR_UNSUPPORTED),
    (dict(conv_w=None), kda.KDA_ERR_INVALID_ARG),
    (dict(conv_w=FAKE + 4), kda.KDA_ERR_INVALID_ARG),
    (dict(conv_b=FAKE + 4), kda.KDA_ERR_INVALID_ARG),
    (dict(A_log=None), kda.KDA_ERR_INVALID_ARG),
    (dict(dt_bias=None), kda.KDA_ERR_INVALID_ARG),
    (dict(D=FAKE + 1), kda.KDA_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw, want", BAD_PARAMS)
def test_bad_params(L, kw, want):
    p = struct(**kw)
    assert prefill(L, p) == want and decode(L, p) == want
    assert L.kda_ssm_prefill_algo(ctypes.byref(p)) == -1
    assert L.kda_ssm_prefill_workspace_bytes(ctypes.byref(p), 1, 64) == 0
    assert L.kda_ssm_decode_workspace_bytes(ctypes.byref(p), 1) == 0


def test_chunked_needs_bf16(L):
    assert prefill(L, struct(algo=kda.KDA_ALGO_CHUNKED, io_dtype=kda.KDA_DTYPE_F32)) == kda.KDA_ERR_UNSUPPORTED
    assert L.kda_ssm_prefill_algo(ctypes.byref(struct(io_dtype=kda.KDA_DTYPE_F32))) == kda.KDA_ALGO_SCAN


@pytest.mark.parametrize("cu, T", [((1, 64), 64), ((0, 64, 32), 32), ((0, 64), 65), ((0, 10), -1)])
def test_bad_cu_seqlens(L, cu, T):
    assert prefill(L, struct(), cu, T) == kda.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(null_cu=True), dict(xbc=None), dict(dt=None), dict(o=None), dict(S_out=None),
                                dict(xbc=FAKE + 8), dict(z=FAKE + 2), dict(o=FAKE + 4), dict(dt=FAKE + 1), dict(S_in=FAKE + 8),
                                dict(S_out=FAKE + 8), dict(ring_in=FAKE + 8), dict(ring_out=FAKE + 8),
                                dict(sx=760), dict(sx=772), dict(sz=255), dict(sz=260), dict(sd=3), dict(sx=-8), dict(sz=-8)])
def test_prefill_refusals(L, kw):
    """Channels 4*64 + 2*2*128 = 768: strides below the row, or off 16 bytes, among them."""
    assert prefill(L, struct(), **kw) == kda.KDA_ERR_INVALID_ARG


def test_prefill_workspace(L):
    p = struct()
    need = L.kda_ssm_prefill_workspace_bytes(ctypes.byref(p), 1, 64)
    assert need > 0
    assert prefill(L, p, ws_bytes=need - 1) == kda.KDA_ERR_WORKSPACE
    assert prefill(L, p, ws=None) == kda.KDA_ERR_WORKSPACE
    assert prefill(L, p, ws=FAKE + 16) == kda.KDA_ERR_WORKSPACE
    for T in (1, 63, 64, 65, 1000):     # the size never shrinks with more tokens or sequences
        sizes = [L.kda_ssm_prefill_workspace_bytes(ctypes.byref(p), n, T) for n in (1, 2, 5)]
        assert sizes == sorted(sizes) and sizes[0] <= L.kda_ssm_prefill_workspace_bytes(ctypes.byref(p), 1, T + 1)
    assert L.kda_ssm_prefill_workspace_bytes(ctypes.byref(p), -1, 64) == 0
    assert prefill(L, p, cu=(0,), T=0, ws=None) == kda.KDA_OK       # no sequences: nothing to do


@pytest.mark.parametrize("kw", [dict(n=-1), dict(n_slots=-1), dict(n_slots=2), dict(slots=FAKE + 2), dict(xbc=None),
                                dict(dt=None), dict(S=None), dict(ring=None), dict(o=None), dict(S=FAKE + 8),
                                dict(ring=FAKE + 8), dict(z=FAKE + 8), dict(sx=8), dict(sx=772), dict(sd=1), dict(sz=4)])
def test_decode_refusals(L, kw):
    assert decode(L, struct(), **kw) == kda.KDA_ERR_INVALID_ARG


def test_decode_workspace_and_empty(L):
    assert L.kda_ssm_decode_workspace_bytes(ctypes.byref(struct(num_heads=32, num_groups=1)), 3) == 0
    p = struct(num_heads=33, num_groups=1)
    need = L.kda_ssm_decode_workspace_bytes(ctypes.byref(p), 3)
    assert need >= 3 * (33 * 64 + 2 * 128) * 4
    assert decode(L, p, ws_bytes=need - 1) == kda.KDA_ERR_WORKSPACE
    assert decode(L, p, ws=None) == kda.KDA_ERR_WORKSPACE
    assert decode(L, p, n=0, ws=None) == kda.KDA_OK


def tree(L, p, n=2, R=8, slots=None, n_slots=2, **ptrs):
    a = dict.fromkeys(("q", "k", "v", "z", "b", "gout", "parents", "S", "ring", "o"), FAKE)
    a.update(ptrs)
    return L.kda_decode_tree(ctypes.byref(p), n, R, a["q"], a["k"], a["v"], a["z"], a["b"], a["gout"], a["parents"], slots,
                             n_slots, a["S"], a["ring"], a["o"], None)


def commit(L, p, n=2, R=8, m=4, slots=None, n_slots=2, **ptrs):
    a = dict.fromkeys(("q", "k", "v", "z", "b", "path", "path_len", "S_in", "S_out", "ring_in", "ring_out"), FAKE)
    a.update(ptrs)
    return L.kda_tree_commit(ctypes.byref(p), n, R, a["q"], a["k"], a["v"], a["z"], a["b"], a["path"], a["path_len"], m, slots,
                             n_slots, a["S_in"], a["S_out"], a["ring_in"], a["ring_out"], None)


SIZES = [dict(n=-1), dict(R=0), dict(R=65), dict(n_slots=-1), dict(n_slots=1)]


@pytest.mark.parametrize("kw", SIZES + [{k: None} for k in ("q", "k", "v", "z", "b", "gout", "parents", "S", "ring", "o")]
                         + [{k: FAKE + 8} for k in ("q", "z", "gout", "S", "ring", "o")])
def test_tree_refusals(L, kw):
    assert tree(L, kda_struct(), **kw) == kda.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", SIZES + [dict(m=0), dict(m=65)]
                         + [{k: None} for k in ("q", "k", "v", "z", "b", "path", "path_len", "S_in", "S_out", "ring_in", "ring_out")]
                         + [{k: FAKE + 8} for k in ("q", "v", "S_in", "S_out", "ring_in", "ring_out")])
def test_commit_refusals(L, kw):
    assert commit(L, kda_struct(), **kw) == kda.KDA_ERR_INVALID_ARG


def test_tree_params_and_empty(L):
    assert tree(L, kda_struct(head_dim=64)) == kda.KDA_ERR_UNSUPPORTED
    assert commit(L, kda_struct(conv_kernel=2)) == kda.KDA_ERR_UNSUPPORTED
    assert tree(L, kda_struct(), n=0) == kda.KDA_OK and commit(L, kda_struct(), n=0) == kda.KDA_OK


# ---- the binding's own checks (CPU tensors: nothing reaches the library) ----

def ssm_params(**kw):
    d = dict(head_dim=64, state_dim=128, num_groups=2)
    d.update(kw)
    return kda.make_ssm_params(torch.zeros(768, 4), torch.zeros(4), torch.zeros(4), **d)


@pytest.mark.parametrize("kw", [dict(num_groups=1), dict(head_dim=128), dict(D=torch.zeros(3)), dict(conv_b=torch.zeros(4)),
                                dict(D=torch.zeros(4, dtype=torch.float64))])
def test_binding_params(kw):
    with pytest.raises(ValueError):
        ssm_params(**kw)


def test_binding_ssm_tensors():
    p, bf = ssm_params(), torch.bfloat16
    x, d, z = torch.zeros(5, 768, dtype=bf), torch.zeros(5, 4, dtype=bf), torch.zeros(5, 256, dtype=bf)
    S, ring = torch.zeros(1, 4, 128, 64), torch.zeros(1, 3, 768, dtype=bf)
    bad = [dict(xbc=x.float()), dict(xbc=x[:, :700]), dict(xbc=x[:4]), dict(dt=d.float()), dict(z=z[:, ::2].repeat(1, 2)[:, :255]),
           dict(S_in=S.double()), dict(S_in=S.transpose(2, 3)), dict(ring_in=ring.float()), dict(o=torch.zeros(5, 255, dtype=bf)),
           dict(xbc=torch.zeros(768, 5, dtype=bf).T), dict(xbc=torch.zeros(1, 768, dtype=bf).expand(5, 768)), {}]
    for kw in bad:        # the last: CPU tensors
        with pytest.raises(ValueError):
            a = dict(xbc=x, dt=d, z=z)
            a.update(kw)
            kda.kda_ssm_prefill(p, a.pop("xbc"), a.pop("dt"), [0, 5], **a)
    for kw in (dict(S=S.half()), dict(ring=ring[:, :2]), dict(slots=torch.zeros(5)), dict(z=z[:2]), {}):
        a = dict(S=S.expand(5, 4, 128, 64).contiguous(), ring=ring.expand(5, 3, 768).contiguous())
        a.update(kw)
        with pytest.raises(ValueError):
            kda.kda_ssm_decode(p, x, d, **a)


def test_binding_tree_tensors():
    p = kda.make_params(torch.zeros(3, 256, 4), torch.zeros(2), torch.zeros(256), torch.zeros(128))
    bf = torch.bfloat16
    rows = dict.fromkeys(("q", "k", "v", "z", "gout"), torch.zeros(2, 5, 256, dtype=bf))
    rows["b"] = torch.zeros(2, 5, 2, dtype=bf)
    S, ring = torch.zeros(2, 2, 128, 128), torch.zeros(2, 3, 3, 256, dtype=bf)
    par = torch.zeros(2, 5, dtype=torch.int32)
    for kw in (dict(q=rows["q"][0]), dict(k=rows["q"].float()), dict(b=rows["q"]), dict(parents=par.long()), dict(parents=par[:, :4]),
               dict(S=S[:, :1]), dict(ring=ring[:1]), dict(slots=par), dict(o=rows["b"]), {}):
        a = {**rows, "parents": par, "S": S, "ring": ring, **kw}
        with pytest.raises(ValueError):
            kda.kda_decode_tree(p, **a)
    del rows["gout"]
    for kw in (dict(path=par.long()), dict(path=par[0]), dict(path_len=par), dict(S_out=S[:1]), dict(ring_out=ring.float()),
               dict(v=rows["v"][:, :4]), {}):
        a = {**rows, "path": par, "path_len": par[:, 0].contiguous(), "S_in": S, "ring_in": ring, **kw}
        with pytest.raises(ValueError):
            kda.kda_tree_commit(p, **a)


@pytest.mark.parametrize("name", ["parents", "slots", "b"])
def test_tree_refuses_misaligned_indices(L, name):
    assert tree(L, kda_struct(), **{name: FAKE + 1}) == kda.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["path", "path_len", "slots", "b"])
def test_commit_refuses_misaligned_indices(L, name):
    assert commit(L, kda_struct(), **{name: FAKE + 1}) == kda.KDA_ERR_INVALID_ARG
