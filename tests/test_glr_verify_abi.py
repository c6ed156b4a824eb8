"""Argument checks of the gated linear recurrence and of the verification of
drafts, on the host: every call here is refused (or empty) before anything is enqueued."""
import ctypes

import pytest
import torch

import gated_delta_rule_04_gb300 as kda
from gated_delta_rule_04_gb300 import build as kbuild

FAKE = 0x10000  # aligned non-null address; never dereferenced on these paths


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kda.lib()


def struct(**kw):
    d = dict(channels=40, io_dtype=kda.KDA_DTYPE_BF16, A_log=FAKE, r_bias=FAKE, i_bias=None)
    d.update(kw)
    return kda.kda_glr_params(**d)


def tensors(names, kw, **defaults):
    """Pointers and strides (name_s) of a call, with some replaced."""
    a = {n: FAKE for n in names}
    a.update({n + "_s": 0 for n in names})
    a.update(defaults)
    a.update(kw)
    return a


def batch(cu, T, null_cu):
    return [None if null_cu else (ctypes.c_int64 * len(cu))(*cu), len(cu) - 1, cu[-1] if T is None else T]


def prefill(L, p, cu=(0, 64), T=None, ws=FAKE, ws_bytes=1 << 40, null_cu=False, **kw):
    a = tensors("x r i z S_in S_out states o".split(), kw)
    rows = [v for n in "xriz" for v in (a[n], a[n + "_s"])]
    return L.kda_glr_prefill(ctypes.byref(p), *rows, *batch(cu, T, null_cu), a["S_in"], a["S_out"], a["states"], a["o"], ws,
                             ws_bytes, None)


def backward(L, p, cu=(0, 64), T=None, ws=FAKE, ws_bytes=1 << 40, null_cu=False, **kw):
    a = tensors("x r i z S_in states do dS_out dx dr di dz dS_in dA_log dr_bias di_bias".split(), kw, dS_in=kw.get("dS_in"))
    two = lambda *names: [v for n in names for v in (a[n], a[n + "_s"])]
    return L.kda_glr_backward(ctypes.byref(p), *two(*"xriz"), *batch(cu, T, null_cu), a["S_in"], a["states"], *two("do"),
                              a["dS_out"], *two("dx", "dr", "di", "dz"), a["dS_in"], a["dA_log"], a["dr_bias"], a["di_bias"], ws,
                              ws_bytes, None)


def decode(L, p, n=3, R=2, n_slots=3, **kw):
    a = tensors("x r i z slots S_in S_out o".split(), kw, slots=kw.get("slots"))
    rows = [v for n_ in "xriz" for v in (a[n_], a[n_ + "_s"])]
    return L.kda_glr_decode(ctypes.byref(p), n, R, *rows, a["slots"], n_slots, a["S_in"], a["S_out"], a["o"], None)


def commit(L, p, n=3, R=2, m=2, n_slots=3, **kw):
    a = tensors("x r i path path_len slots S_in S_out".split(), kw, slots=kw.get("slots"))
    rows = [v for n_ in "xri" for v in (a[n_], a[n_ + "_s"])]
    return L.kda_glr_commit(ctypes.byref(p), n, R, *rows, a["path"], a["path_len"], m, a["slots"], n_slots, a["S_in"],
                            a["S_out"], None)


def verify(L, dtype=kda.KDA_DTYPE_BF16, n=2, R=3, V=100, m=3, **kw):
    a = dict(p=FAKE, pss=300, prs=100, p_last=FAKE, pls=100, q=FAKE, qss=300, qrs=100, q_last=FAKE, qls=100, tokens=FAKE,
             parents=FAKE, u=FAKE, u_next=FAKE, path=FAKE, path_len=FAKE, next_token=FAKE)
    a.update(kw)
    return L.kda_draft_verify(dtype, n, R, V, a["p"], a["pss"], a["prs"], a["p_last"], a["pls"], a["q"], a["qss"], a["qrs"],
                              a["q_last"], a["qls"], a["tokens"], a["parents"], a["u"], a["u_next"], m, a["path"], a["path_len"],
                              a["next_token"], None)


@pytest.mark.parametrize("kw", [dict(channels=0), dict(channels=-5), dict(channels=(1 << 24) + 1), dict(io_dtype=2),
                                dict(A_log=None), dict(A_log=FAKE + 2), dict(r_bias=FAKE + 1), dict(i_bias=FAKE + 2)])
def test_bad_params(L, kw):
    p = struct(**kw)
    for call in (prefill, backward, decode, commit):
        assert call(L, p) == kda.KDA_ERR_INVALID_ARG
    for size in (L.kda_glr_prefill_workspace_bytes, L.kda_glr_backward_workspace_bytes):
        assert size(ctypes.byref(p), 1, 64) == 0


@pytest.mark.parametrize("kw", [dict(cu=(1, 64)), dict(cu=(0, 64, 32), T=32), dict(T=65), dict(cu=(0, 10), T=-1), dict(null_cu=True)])
def test_bad_cu_seqlens(L, kw):
    assert prefill(L, struct(), **kw) == kda.KDA_ERR_INVALID_ARG
    assert backward(L, struct(), **kw) == kda.KDA_ERR_INVALID_ARG


ROWS = [dict(x=None), dict(r=None), dict(i=None), dict(x=FAKE + 1), dict(r=FAKE + 1), dict(i=FAKE + 1), dict(z=FAKE + 1),
        dict(x_s=39), dict(r_s=-40), dict(i_s=1 << 31), dict(x_s=1 << 30), dict(z_s=1)]


@pytest.mark.parametrize("kw", ROWS + [dict(o=None), dict(o=FAKE + 1), dict(S_out=None), dict(S_out=FAKE + 2),
                                       dict(S_in=FAKE + 2), dict(states=FAKE + 2)])
def test_prefill_refusals(L, kw):
    assert prefill(L, struct(), **kw) == kda.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", ROWS + [dict(do=None), dict(dx=None), dict(dr=None), dict(di=None), dict(dz=None), dict(z=None),
                                       dict(states=None), dict(dA_log=None), dict(do_s=39), dict(dx_s=3), dict(dr_s=39),
                                       dict(di_s=-1), dict(dz_s=39), dict(do=FAKE + 1), dict(dx=FAKE + 1), dict(dz=FAKE + 1),
                                       dict(dS_out=FAKE + 2), dict(dS_in=FAKE + 1), dict(dA_log=FAKE + 2), dict(dr_bias=FAKE + 2),
                                       dict(di_bias=FAKE + 2), dict(states=FAKE + 2), dict(S_in=FAKE + 2), dict(dS_in=FAKE)])
def test_backward_refusals(L, kw):
    """dz without z (z=None here) is among them, z without dz, and dS_in in the place of dS_out."""
    assert backward(L, struct(), **{"dS_in": FAKE + 4096, **kw}) == kda.KDA_ERR_INVALID_ARG


def test_too_many_tokens(L):
    T = (1 << 31) + 5
    assert prefill(L, struct(), cu=(0, T)) == kda.KDA_ERR_UNSUPPORTED
    assert backward(L, struct(), cu=(0, T)) == kda.KDA_ERR_UNSUPPORTED
    assert L.kda_glr_prefill_workspace_bytes(ctypes.byref(struct()), 1, T) == 0


def test_fp32_rows_need_their_elements_alignment(L):
    p = struct(io_dtype=kda.KDA_DTYPE_F32)
    assert prefill(L, p, x=FAKE + 2) == kda.KDA_ERR_INVALID_ARG
    assert backward(L, p, dx=FAKE + 2) == kda.KDA_ERR_INVALID_ARG
    assert decode(L, p, z=FAKE + 2) == kda.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("call, size", [(prefill, "kda_glr_prefill_workspace_bytes"), (backward, "kda_glr_backward_workspace_bytes")])
def test_workspace(L, call, size):
    f = getattr(L, size)
    for C in (1, 40, 4096):
        p = struct(channels=C)
        need = f(ctypes.byref(p), 1, 64)
        assert need > 0
        assert call(L, p, ws_bytes=need - 1) == kda.KDA_ERR_WORKSPACE
        assert call(L, p, ws=None) == kda.KDA_ERR_WORKSPACE
        assert call(L, p, ws=FAKE + 16) == kda.KDA_ERR_WORKSPACE
        for T in (0, 1, 63, 64, 65, 1000, 8192, 100000):
            sizes = [f(ctypes.byref(p), n, T) for n in (*range(1, 40), 100, 1023, 1024, 1025, 70000)]
            assert sizes == sorted(sizes)
        for n in (1, 16, 17, 500):
            sizes = [f(ctypes.byref(p), n, T) for T in (0, 1, 63, 64, 65, 127, 128, 129, 1000, 8191, 8192, 100000, 1 << 20)]
            assert sizes == sorted(sizes)
    assert f(ctypes.byref(struct()), -1, 64) == 0 and f(ctypes.byref(struct()), 1, -1) == 0 and f(ctypes.byref(struct()), 0, 0) == 0
    assert prefill(L, struct(), cu=(0,), T=0, ws=None) == kda.KDA_OK       # no sequences: nothing to do


@pytest.mark.parametrize("kw", ROWS + [dict(n=-1), dict(R=0), dict(R=65), dict(n_slots=-1), dict(n_slots=2), dict(slots=FAKE + 2),
                                       dict(S_in=None), dict(S_in=FAKE + 2), dict(S_out=FAKE + 2), dict(o=None), dict(o=FAKE + 1)])
def test_decode_refusals(L, kw):
    assert decode(L, struct(), **kw) == kda.KDA_ERR_INVALID_ARG
    assert decode(L, struct(), n=0) == kda.KDA_OK


@pytest.mark.parametrize("kw", [k for k in ROWS if "z" not in k and "z_s" not in k] +
                         [dict(n=-1), dict(R=0), dict(R=65), dict(m=0), dict(m=65), dict(n_slots=-1), dict(n_slots=2),
                          dict(slots=FAKE + 2), dict(S_in=None), dict(S_out=None), dict(S_in=FAKE + 2), dict(S_out=FAKE + 2),
                          dict(path=None), dict(path_len=None), dict(path=FAKE + 2), dict(path_len=FAKE + 1)])
def test_commit_refusals(L, kw):
    assert commit(L, struct(), **kw) == kda.KDA_ERR_INVALID_ARG
    assert commit(L, struct(), n=0) == kda.KDA_OK


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(n=-1), dict(R=0), dict(R=65), dict(V=0), dict(m=0), dict(m=65), dict(p=None),
                                dict(tokens=None), dict(parents=None), dict(u=None), dict(u_next=None), dict(path=None),
                                dict(path_len=None), dict(next_token=None), dict(p=FAKE + 1), dict(q=FAKE + 1),
                                dict(p_last=FAKE + 1), dict(q_last=FAKE + 1), dict(tokens=FAKE + 2), dict(parents=FAKE + 2),
                                dict(u=FAKE + 2), dict(u_next=FAKE + 2), dict(path=FAKE + 2), dict(path_len=FAKE + 2),
                                dict(next_token=FAKE + 2), dict(q_last=None), dict(p_last=None), dict(q=None),
                                dict(pss=-1), dict(prs=-1), dict(pls=-1), dict(qss=-1), dict(qrs=-1), dict(qls=-1)])
def test_verify_refusals(L, kw):
    """q_last is there if and only if p_last and q are."""
    assert verify(L, **kw) == kda.KDA_ERR_INVALID_ARG


def test_verify_limits(L):
    assert verify(L, V=(1 << 30) + 1) == kda.KDA_ERR_UNSUPPORTED
    assert verify(L, n=0) == kda.KDA_OK
    assert verify(L, dtype=kda.KDA_DTYPE_F32, p=FAKE + 2) == kda.KDA_ERR_INVALID_ARG


# ---- the binding's own checks (CPU tensors: nothing reaches the library) ----

def glr_params(**kw):
    t = dict(A_log=torch.zeros(40), r_bias=torch.zeros(40), i_bias=torch.zeros(40))
    t.update(kw)
    return kda.make_glr_params(t.pop("A_log"), **t)


def test_parameters():
    for bad in (dict(A_log=torch.zeros(40, 1)), dict(A_log=torch.zeros(40).double()), dict(r_bias=torch.zeros(39)),
                dict(i_bias=torch.zeros(40).half())):
        with pytest.raises(ValueError):
            glr_params(**bad)
    for name in ("A_log", "r_bias", "i_bias"):
        with pytest.raises(ValueError, match="one device"):
            glr_params(**{name: torch.zeros(40, device="meta")})
    with pytest.raises(KeyError):
        glr_params(io_dtype="f16")


def test_host_tensors_are_refused():
    """Nothing runs on the CPU, and parameters of another device are refused first."""
    p, bf = glr_params(), torch.bfloat16
    x, S, path = torch.zeros(5, 40, dtype=bf), torch.zeros(5, 40), torch.zeros(5, 1, dtype=torch.int32)
    prob, tok, u = torch.zeros(2, 3, 7), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)
    calls = (lambda: kda.kda_glr_prefill(p, x, x, x, [0, 5]),
             lambda: kda.kda_glr_backward(p, x, x, x, [0, 5], S[:1], x),
             lambda: kda.kda_glr_decode(p, x[:, None], x[:, None], x[:, None], S),
             lambda: kda.kda_glr_commit(p, x[:, None], x[:, None], x[:, None], path, path[:, 0].contiguous(), S))
    for call in (*calls, lambda: kda.kda_draft_verify(prob, tok, tok, u, u[:, 0].contiguous())):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    p.device = 1
    for call in calls:
        with pytest.raises(ValueError, match="on cuda:1"):
            call()


def test_round_rows_lie_evenly_apart():
    t = torch.zeros(4, 3, 80, dtype=torch.bfloat16)
    ok = lambda x, dev=-1: kda._run_rows("x", x, torch.bfloat16, *x.shape, dev)
    with pytest.raises(ValueError, match="CUDA device"):
        ok(t)
    class On:                                    # a tensor that says it is on a device
        def __init__(self, t): self.t = t
        def get_device(self): return 0
        def __getattr__(self, k): return getattr(self.t, k)
    rows = lambda x: kda._run_rows("x", On(x), torch.bfloat16, *x.shape, 0)
    assert rows(t)[1] == 0 and rows(t[..., :40])[1] == 80 and rows(t[:, :1, :40])[1] == 240
    assert rows(t[:1, :1, :40])[1] == 0
    for bad in (t[:, :2], t[..., ::2], t[:, :1].expand(4, 3, 80), t.transpose(0, 1)):
        with pytest.raises(ValueError):
            rows(bad)
