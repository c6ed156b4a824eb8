"""Python binding of the GB300 KDA mixer-core library (``libkda.so``).

Argument marshalling only: every step of the mixer runs in the CUDA kernels
behind the C ABI declared in ``include/kda.h``; PyTorch supplies device
memory and the stream.  The functions carry the C names:

    kda_prefill_algo, kda_prefill_workspace_bytes, kda_prefill_windows, kda_prefill_segments, kda_prefill,
    kda_prefill_with_events (as kda_prefill(..., stage_events=...)),
    kda_prefill_host_scratch_bytes, kda_prefill_host, kda_decode, kda_decode_multi,
    kda_decode_tree, kda_tree_commit, kda_workspace_status, kda_status_str,
    kda_ssm_prefill_algo, kda_ssm_prefill_workspace_bytes, kda_ssm_prefill,
    kda_ssm_decode_workspace_bytes, kda_ssm_decode

There is no fallback: if ``libkda.so`` is missing the import of this package
still succeeds, but the first call raises ``KdaLibraryMissing``.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Sequence

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkda.so")

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_WORKSPACE, KDA_ERR_CUDA, KDA_ERR_TIMEOUT = range(6)
KDA_DTYPE_F32, KDA_DTYPE_BF16 = 0, 1
KDA_ALGO_AUTO, KDA_ALGO_SCAN, KDA_ALGO_CHUNKED, KDA_ALGO_CHUNKED_SEGMENTS = 0, 1, 2, 3
_ALGOS = {"auto": KDA_ALGO_AUTO, "scan": KDA_ALGO_SCAN, "chunked": KDA_ALGO_CHUNKED,
          "chunked_segments": KDA_ALGO_CHUNKED_SEGMENTS}

_vp = ctypes.c_void_p


class KdaLibraryMissing(RuntimeError):
    pass


class KdaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {kda_status_str(status)} (status {status})")


class kda_params(ctypes.Structure):
    _fields_ = [
        ("num_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("conv_kernel", ctypes.c_int32),
        ("io_dtype", ctypes.c_int32),
        ("algo", ctypes.c_int32),
        ("gate_lower_bound", ctypes.c_float),
        ("l2_eps", ctypes.c_float),
        ("norm_eps", ctypes.c_float),
        ("q_scale", ctypes.c_float),
        ("conv_w", _vp),
        ("A_log", _vp),
        ("dt_bias", _vp),
        ("norm_w", _vp),
        ("gate_kind", ctypes.c_int32),
        ("wait_limit_us", ctypes.c_uint32),
    ]


class kda_ssm_params(ctypes.Structure):
    _fields_ = [
        ("num_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("state_dim", ctypes.c_int32),
        ("num_groups", ctypes.c_int32),
        ("conv_kernel", ctypes.c_int32),
        ("io_dtype", ctypes.c_int32),
        ("algo", ctypes.c_int32),
        ("conv_w", _vp),
        ("conv_b", _vp),
        ("A_log", _vp),
        ("dt_bias", _vp),
        ("D", _vp),
    ]


_lib = None


def lib():
    """The loaded ``libkda.so`` (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise KdaLibraryMissing(
                f"{LIB_PATH} is missing; build it with `python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(kda_params)
        i32, i64, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        L.kda_prefill_algo.argtypes = [P]
        L.kda_prefill_algo.restype = i32
        L.kda_prefill_workspace_bytes.argtypes = [P, i32, i64]
        L.kda_prefill_workspace_bytes.restype = sz
        L.kda_prefill_windows.argtypes = [P, i32, i64, sz]
        L.kda_prefill_windows.restype = i32
        L.kda_prefill_segments.argtypes = [P, i32, i64, sz]
        L.kda_prefill_segments.restype = i32
        L.kda_prefill.argtypes = [P] + [_vp] * 6 + [ctypes.POINTER(ctypes.c_int64), i32, i64] + [_vp] * 5 + [_vp, sz, _vp]
        L.kda_prefill.restype = ctypes.c_int
        L.kda_prefill_with_events.argtypes = L.kda_prefill.argtypes + [ctypes.POINTER(_vp)]
        L.kda_prefill_with_events.restype = ctypes.c_int
        L.kda_decode.argtypes = [P, i32] + [_vp] * 6 + [_vp] * 3 + [_vp]
        L.kda_decode.restype = ctypes.c_int
        L.kda_decode_multi.argtypes = [P, i32, i32] + [_vp] * 6 + [_vp, i32] + [_vp] * 5 + [_vp]
        L.kda_decode_multi.restype = ctypes.c_int
        L.kda_prefill_host_scratch_bytes.argtypes = [P, ctypes.POINTER(ctypes.c_int64), i32, i64, i64]
        L.kda_prefill_host_scratch_bytes.restype = sz
        L.kda_prefill_host.argtypes = ([P] + [_vp] * 6 + [ctypes.POINTER(ctypes.c_int64), i32, i64] + [_vp] * 5
                                       + [i64, _vp, sz, _vp, _vp, _vp])
        L.kda_prefill_host.restype = ctypes.c_int
        L.kda_decode_tree.argtypes = [P, i32, i32] + [_vp] * 6 + [_vp, _vp, i32] + [_vp] * 4
        L.kda_decode_tree.restype = ctypes.c_int
        L.kda_tree_commit.argtypes = [P, i32, i32] + [_vp] * 5 + [_vp, _vp, i32, _vp, i32] + [_vp] * 5
        L.kda_tree_commit.restype = ctypes.c_int
        SP = ctypes.POINTER(kda_ssm_params)
        L.kda_ssm_prefill_algo.argtypes = [SP]
        L.kda_ssm_prefill_algo.restype = i32
        L.kda_ssm_prefill_workspace_bytes.argtypes = [SP, i32, i64]
        L.kda_ssm_prefill_workspace_bytes.restype = sz
        L.kda_ssm_prefill.argtypes = ([SP] + [_vp, i64] * 3 + [ctypes.POINTER(ctypes.c_int64), i32, i64] + [_vp] * 5
                                      + [_vp, sz, _vp])
        L.kda_ssm_prefill.restype = ctypes.c_int
        L.kda_ssm_decode_workspace_bytes.argtypes = [SP, i32]
        L.kda_ssm_decode_workspace_bytes.restype = sz
        L.kda_ssm_decode.argtypes = [SP, i32] + [_vp, i64] * 3 + [_vp, i32] + [_vp] * 3 + [_vp, sz, _vp]
        L.kda_ssm_decode.restype = ctypes.c_int
        L.kda_workspace_status.argtypes = [_vp, _vp]
        L.kda_workspace_status.restype = ctypes.c_int
        L.kda_status_str.argtypes = [ctypes.c_int]
        L.kda_status_str.restype = ctypes.c_char_p
        _lib = L
    return _lib


def kda_status_str(status: int) -> str:
    return lib().kda_status_str(int(status)).decode()


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


@dataclass
class Params:
    """Holds the device parameter tensors and the C struct that points at them."""

    struct: kda_params
    tensors: tuple
    num_heads: int
    io_dtype: int
    device: int           # CUDA device of the tensors (-1: none)

    @property
    def ref(self):
        return ctypes.byref(self.struct)


def _params_device(tensors):
    """The CUDA device (-1: none) that all of the parameter tensors are on, or ValueError."""
    devs = {t.device for t in tensors if t is not None}
    if len(devs) > 1:
        raise ValueError(f"parameters: expected one device, got {sorted(map(str, devs))}")
    return tensors[0].get_device()


KDA_GATE_BOUNDED, KDA_GATE_SOFTPLUS = 0, 1
_GATES = {"bounded": KDA_GATE_BOUNDED, "softplus": KDA_GATE_SOFTPLUS}


def make_params(conv_w, A_log, dt_bias, norm_w, *, io_dtype: str = "bf16", algo: str = "auto",
                gate_lower_bound: float = -5.0, l2_eps: float = 1e-6, norm_eps: float = 1e-5,
                q_scale: float = 0.0, gate: str = "bounded", wait_limit_us: int = 0) -> Params:
    """conv_w [3][H*128][4], A_log [H], dt_bias [H*128], norm_w [128]: fp32 CUDA tensors.
    gate: "bounded" (g = lb sigmoid(e^A (z + dt_bias))) or "softplus"
    (g = -e^A softplus(z + dt_bias), unbounded below).  wait_limit_us: the
    test hook of kda_params (0 in normal use)."""
    H = int(A_log.shape[0])
    dt = {"f32": KDA_DTYPE_F32, "bf16": KDA_DTYPE_BF16}[io_dtype]
    tensors = tuple(t.contiguous() for t in (conv_w, A_log, dt_bias, norm_w))
    st = kda_params(H, 128, 4, dt, _ALGOS[algo], gate_lower_bound, l2_eps, norm_eps, q_scale,
                    *[t.data_ptr() for t in tensors], _GATES[gate], int(wait_limit_us))
    return Params(st, tensors, H, dt, _params_device(tensors))


def kda_prefill_algo(params: Params) -> str:
    """'scan' or 'chunked': the prefill algorithm these parameters select."""
    a = int(lib().kda_prefill_algo(params.ref))
    if a < 0:
        raise KdaError(KDA_ERR_INVALID_ARG, "kda_prefill_algo")
    return {KDA_ALGO_SCAN: "scan", KDA_ALGO_CHUNKED: "chunked"}[a]


def kda_prefill_workspace_bytes(params: Params, n_seqs: int, total_tokens: int) -> int:
    return int(lib().kda_prefill_workspace_bytes(params.ref, int(n_seqs), int(total_tokens)))


def kda_prefill_windows(params: Params, n_seqs: int, total_tokens: int, workspace_bytes: int) -> int:
    """How many overlapped windows kda_prefill runs (1 = single pass)."""
    return int(lib().kda_prefill_windows(params.ref, int(n_seqs), int(total_tokens), int(workspace_bytes)))


def kda_prefill_segments(params: Params, n_seqs: int, total_tokens: int, workspace_bytes: int) -> int:
    """How many segments kda_prefill runs one sequence's recurrence as (0 = none)."""
    return int(lib().kda_prefill_segments(params.ref, int(n_seqs), int(total_tokens), int(workspace_bytes)))


def _cu_array(cu_seqlens: Sequence[int]):
    vals = [int(x) for x in cu_seqlens]
    return (ctypes.c_int64 * len(vals))(*vals), len(vals) - 1, vals[-1]


KDA_PREFILL_EVENTS = 6


def kda_prefill(params: Params, q, k, v, z, b, gout, cu_seqlens, S_in=None, S_out=None,
                ring_in=None, ring_out=None, o=None, workspace=None, stream=None, stage_events=None):
    """Varlen prefill.  Tensors are CUDA tensors in the layouts of ``include/kda.h``;
    ``cu_seqlens`` is a host sequence of n+1 ints.  Missing outputs and the
    workspace are allocated with torch.  ``stage_events`` (optional) is a list
    of KDA_PREFILL_EVENTS torch.cuda.Event objects recorded at the stage
    boundaries (kda_prefill_with_events).  Returns (o, S_out, ring_out)."""
    import torch
    cu, n, T = _cu_array(cu_seqlens)
    H = params.num_heads
    dev = q.device
    if o is None:
        o = torch.empty_like(q)
    if S_out is None:
        S_out = torch.empty(n, H, 128, 128, dtype=torch.float32, device=dev)
    if ring_out is None:
        ring_out = torch.empty(n, 3, 3, H * 128, dtype=q.dtype, device=dev)
    if workspace is None:
        nbytes = kda_prefill_workspace_bytes(params, n, T)
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
    args = (params.ref, _ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(b), _ptr(gout),
            cu, n, T, _ptr(S_in), _ptr(S_out), _ptr(ring_in), _ptr(ring_out), _ptr(o),
            _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    if stage_events is None:
        st = lib().kda_prefill(*args)
    else:
        handles = []
        for e in stage_events:
            if e is not None and not e.cuda_event:
                e.record()  # torch creates the underlying cudaEvent_t lazily
            handles.append(None if e is None else e.cuda_event)
        evs = (_vp * KDA_PREFILL_EVENTS)(*handles)
        st = lib().kda_prefill_with_events(*args, evs)
    if st != KDA_OK:
        raise KdaError(st, "kda_prefill")
    return o, S_out, ring_out


def kda_prefill_host_scratch_bytes(params: Params, cu_seqlens, segment_tokens: int) -> int:
    cu, n, T = _cu_array(cu_seqlens)
    return int(lib().kda_prefill_host_scratch_bytes(params.ref, cu, n, T, int(segment_tokens)))


def kda_prefill_host(params: Params, q, k, v, z, b, gout, cu_seqlens, S_in=None, S_out=None,
                     ring_in=None, ring_out=None, o=None, segment_tokens: int = 4096, scratch=None,
                     stream=None, h2d_stream=None, d2h_stream=None, device=None):
    """Prefill from HOST tensors (page-locked for the copies to overlap): the
    library copies token segments in on ``h2d_stream``, runs them on
    ``stream`` and copies the output back on ``d2h_stream``.  S_in / ring_in /
    S_out / ring_out and ``scratch`` are CUDA tensors; missing ones are
    allocated (``o`` as pinned host memory).  Synchronise ``stream`` before
    reading ``o``.  Returns (o, S_out, ring_out)."""
    import torch
    cu, n, T = _cu_array(cu_seqlens)
    H = params.num_heads
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if o is None:
        o = torch.empty(q.shape, dtype=q.dtype).pin_memory()
    if S_out is None:
        S_out = torch.empty(n, H, 128, 128, dtype=torch.float32, device=dev)
    if ring_out is None:
        ring_out = torch.empty(n, 3, 3, H * 128, dtype=q.dtype, device=dev)
    if scratch is None:
        nbytes = int(lib().kda_prefill_host_scratch_bytes(params.ref, cu, n, T, int(segment_tokens)))
        scratch = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
    st = lib().kda_prefill_host(params.ref, _ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(b), _ptr(gout),
                                cu, n, T, _ptr(S_in), _ptr(S_out), _ptr(ring_in), _ptr(ring_out), _ptr(o),
                                int(segment_tokens), _ptr(scratch), scratch.numel() * scratch.element_size(),
                                _stream(stream), None if h2d_stream is None else _stream(h2d_stream),
                                None if d2h_stream is None else _stream(d2h_stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_prefill_host")
    return o, S_out, ring_out


def kda_decode(params: Params, q, k, v, z, b, gout, S, ring, o=None, stream=None):
    """One token per session; S and ring are updated in place.  Returns o."""
    import torch
    n = int(q.shape[0])
    if o is None:
        o = torch.empty_like(q)
    st = lib().kda_decode(params.ref, n, _ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(b), _ptr(gout),
                          _ptr(S), _ptr(ring), _ptr(o), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_decode")
    return o


KDA_DECODE_MAX_TOKENS = 64


def kda_decode_multi(params: Params, q, k, v, z, b, gout, S_in, ring_in, S_out=None, ring_out=None,
                     slots=None, o=None, stream=None):
    """n_tokens consecutive tokens per session (a speculative verify round).
    q, k, v, z, gout: [n][n_tokens][H*128]; b: [n][n_tokens][H].  S_in /
    ring_in are state / ring pools [n_slots][...]; S_out / ring_out default to
    them (in-place).  ``slots`` (int32 CUDA tensor [n]) maps sessions to pool
    slots.  Keeping S_in / ring_in (separate outputs) allows a rollback: call
    again with the accepted prefix of the tokens.  Returns o."""
    import torch
    n, n_tok = int(q.shape[0]), int(q.shape[1])
    S_out = S_in if S_out is None else S_out
    ring_out = ring_in if ring_out is None else ring_out
    if o is None:
        o = torch.empty_like(q)
    n_slots = int(S_in.shape[0])
    st = lib().kda_decode_multi(params.ref, n, n_tok, _ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(b), _ptr(gout),
                                _ptr(slots), n_slots, _ptr(S_in), _ptr(S_out), _ptr(ring_in), _ptr(ring_out),
                                _ptr(o), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_decode_multi")
    return o


def kda_workspace_status(workspace, stream=None) -> int:
    return int(lib().kda_workspace_status(_ptr(workspace), _stream(stream)))


# ---- draft trees and the state space mixer -------------------------------------------

# These run before every launch of a serving loop's smallest calls, whose kernels take a
# few microseconds: one comparison each where the argument is right.

def _shaped(name, t, dtype, shape, dev):
    """The address of a dense tensor of this type and shape on CUDA device ``dev``, or ValueError."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != dev or dev < 0:
        raise ValueError(f"{name}: expected a contiguous tensor {dtype} {list(shape)} on CUDA device {max(dev, 0)}, got "
                         f"{'' if t.is_contiguous() else 'non-contiguous '}{t.dtype} {list(t.shape)} on {t.device}")
    return t.data_ptr()


def _pool(name, t, dtype, rest, dev):
    """(address, slots) of a dense tensor [slots][*rest] of this type."""
    n = t.shape[0] if t.dim() else 0
    return _shaped(name, t, dtype, (n, *rest), dev), n


def _empty(like, shape, dtype, stream):
    """A new tensor on ``like``'s device that belongs to ``stream`` (default: the current one), so
    that its memory is neither still in use there nor reused before the call's kernels are done."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)   # (1 us less than like.new_empty)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, like.device) if isinstance(stream, int) else stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _output(name, o, like, shape, dtype, dev, stream):
    """(tensor, address) of the caller's output tensor, or of a new one."""
    if o is None:
        o = _empty(like, shape, dtype, stream)
        return o, o.data_ptr()
    return o, _shaped(name, o, dtype, shape, dev)


def _workspace(t, like, nbytes, params, *sizes, stream=None):
    """(tensor, address, bytes) of the caller's workspace, or of a new one of ``nbytes(params, *sizes)``."""
    if t is None:
        import torch
        t = _empty(like, max(nbytes(params, *sizes), 256), torch.uint8, stream)
    elif t.get_device() != like.get_device() or not t.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on {like.device}, got "
                         f"{'' if t.is_contiguous() else 'a non-contiguous one '}on {t.device}")
    return t, t.data_ptr(), t.nbytes


def _rows(name, t, dtype, n, width, dev):
    """(address, row stride in elements) of a [n][width] tensor whose rows may lie apart."""
    if t.dtype is not dtype or t.shape != (n, width) or t.get_device() != dev or dev < 0:
        raise ValueError(f"{name}: expected a tensor {dtype} {[n, width]} on CUDA device {max(dev, 0)}, got {t.dtype} "
                         f"{list(t.shape)} on {t.device}")
    stride, inner = t.stride()
    if width > 1 and inner != 1:
        raise ValueError(f"{name}: the elements of a row have to lie side by side")
    if n <= 1:
        return t.data_ptr(), 0
    if stride < width:
        raise ValueError(f"{name}: rows overlap (stride {stride} < {width})")
    return t.data_ptr(), stride


def _same_device(params, dev):
    if params.device != dev:
        raise ValueError(f"parameters: they are on {'no CUDA device' if params.device < 0 else f'cuda:{params.device}'}, the "
                         f"call's tensors on {'none' if dev < 0 else f'cuda:{dev}'}")


def _call(name, dev, f, *args, stream=None):
    """Calls ``f`` with CUDA device ``dev`` current, on ``stream`` (default: that device's current stream)."""
    import torch
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            st = f(*args, _stream(stream))
    else:
        st = f(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, name)


def _io_torch(io_dtype):
    import torch
    return torch.float32 if io_dtype == KDA_DTYPE_F32 else torch.bfloat16


KDA_TREE_MAX_NODES = 64


def kda_decode_tree(params: Params, q, k, v, z, b, gout, parents, S, ring, slots=None, o=None, stream=None):
    """The output rows of a tree of drafted tokens per session; state and ring
    stay as they are.  q, k, v, z, gout: [n][n_nodes][H*128]; b:
    [n][n_nodes][H]; parents: int32 [n][n_nodes], -1 under the session's last
    token, parents before children (any other entry leaves the node and those
    under it out, their rows untouched).  S / ring: pools [n_slots][...];
    ``slots``: int32 [n].  Returns o."""
    import torch
    t = _io_torch(params.io_dtype)
    if q.dim() != 3:
        raise ValueError(f"q: expected [n][n_nodes][H*128], got {list(q.shape)}")
    n, R, _ = q.shape
    H, dev = params.num_heads, q.get_device()
    _same_device(params, dev)
    rows = (n, R, H * 128)
    S_p, slots_n = _pool("S", S, torch.float32, (H, 128, 128), dev)
    args = (params.ref, n, R, _shaped("q", q, t, rows, dev), _shaped("k", k, t, rows, dev), _shaped("v", v, t, rows, dev),
            _shaped("z", z, t, rows, dev), _shaped("b", b, t, (n, R, H), dev), _shaped("gout", gout, t, rows, dev),
            _shaped("parents", parents, torch.int32, (n, R), dev), None if slots is None else _shaped("slots", slots, torch.int32, (n,), dev), slots_n, S_p,
            _shaped("ring", ring, t, (slots_n, 3, 3, H * 128), dev))
    o, o_p = _output("o", o, q, rows, t, dev, stream)
    _call("kda_decode_tree", dev, lib().kda_decode_tree, *args, o_p, stream=stream)
    return o


def kda_tree_commit(params: Params, q, k, v, z, b, path, path_len, S_in, ring_in, S_out=None, ring_out=None, slots=None,
                    stream=None):
    """Advances each session's state and ring by its accepted path: ``path``
    int32 [n][max_len] node indices in order, ``path_len`` int32 [n].  The
    token tensors are those of the kda_decode_tree round.  S_out / ring_out
    default to the input pools (in place).  Returns (S_out, ring_out)."""
    import torch
    t = _io_torch(params.io_dtype)
    if q.dim() != 3 or path.dim() != 2:
        raise ValueError(f"q, path: expected [n][n_nodes][H*128] and [n][max_len], got {list(q.shape)}, {list(path.shape)}")
    n, R, _ = q.shape
    H, m, dev = params.num_heads, path.shape[1], q.get_device()
    _same_device(params, dev)
    S_out = S_in if S_out is None else S_out
    ring_out = ring_in if ring_out is None else ring_out
    rows = (n, R, H * 128)
    S_p, slots_n = _pool("S_in", S_in, torch.float32, (H, 128, 128), dev)
    ring = (slots_n, 3, 3, H * 128)
    _call("kda_tree_commit", dev, lib().kda_tree_commit, params.ref, n, R, _shaped("q", q, t, rows, dev), _shaped("k", k, t, rows, dev),
          _shaped("v", v, t, rows, dev), _shaped("z", z, t, rows, dev), _shaped("b", b, t, (n, R, H), dev),
          _shaped("path", path, torch.int32, (n, m), dev), _shaped("path_len", path_len, torch.int32, (n,), dev), m,
          None if slots is None else _shaped("slots", slots, torch.int32, (n,), dev), slots_n, S_p,
          _shaped("S_out", S_out, torch.float32, (slots_n, H, 128, 128), dev), _shaped("ring_in", ring_in, t, ring, dev),
          _shaped("ring_out", ring_out, t, ring, dev), stream=stream)
    return S_out, ring_out


@dataclass
class SsmParams:
    """The state space mixer's parameter tensors and the C struct that points at them."""

    struct: kda_ssm_params
    tensors: tuple
    num_heads: int
    head_dim: int
    state_dim: int
    num_groups: int
    io_dtype: int
    channels: int         # conv channels of a token: x (H*P) | B (G*N) | C (G*N)
    torch_dtype: object   # torch type of xbc, dt, z, o and the ring
    device: int           # CUDA device of the parameter tensors (-1: none)
    ref: object           # pointer to the struct


def make_ssm_params(conv_w, A_log, dt_bias, *, head_dim: int, state_dim: int, num_groups: int = 1, D=None, conv_b=None,
                    io_dtype: str = "bf16", algo: str = "auto") -> SsmParams:
    """conv_w [H*P + 2*G*N][4], conv_b [H*P + 2*G*N] or None, A_log, dt_bias, D
    (or None) [H]: fp32 CUDA tensors.  head_dim P and state_dim N are 64 or
    128; num_groups G divides H."""
    import torch
    H = int(A_log.shape[0])
    ch = H * int(head_dim) + 2 * int(num_groups) * int(state_dim)
    for name, x, shape in (("conv_w", conv_w, (ch, 4)), ("conv_b", conv_b, (ch,)), ("A_log", A_log, (H,)),
                           ("dt_bias", dt_bias, (H,)), ("D", D, (H,))):
        if x is not None and (x.dtype != torch.float32 or tuple(x.shape) != shape):
            raise ValueError(f"{name}: expected float32 {list(shape)}, got {x.dtype} {list(x.shape)}")
    dt = {"f32": KDA_DTYPE_F32, "bf16": KDA_DTYPE_BF16}[io_dtype]
    tensors = tuple(None if x is None else x.contiguous() for x in (conv_w, conv_b, A_log, dt_bias, D))
    st = kda_ssm_params(H, int(head_dim), int(state_dim), int(num_groups), 4, dt, _ALGOS[algo], *[_ptr(x) for x in tensors])
    return SsmParams(st, tensors, H, int(head_dim), int(state_dim), int(num_groups), dt, ch, _io_torch(dt), _params_device(tensors),
                     ctypes.byref(st))


def kda_ssm_prefill_algo(params: SsmParams) -> str:
    """'scan' or 'chunked': the prefill algorithm these parameters select."""
    a = int(lib().kda_ssm_prefill_algo(params.ref))
    if a < 0:
        raise KdaError(KDA_ERR_INVALID_ARG, "kda_ssm_prefill_algo")
    return {KDA_ALGO_SCAN: "scan", KDA_ALGO_CHUNKED: "chunked"}[a]


def kda_ssm_prefill_workspace_bytes(params: SsmParams, n_seqs: int, total_tokens: int) -> int:
    return int(lib().kda_ssm_prefill_workspace_bytes(params.ref, int(n_seqs), int(total_tokens)))


def kda_ssm_prefill(params: SsmParams, xbc, dt, cu_seqlens, z=None, S_in=None, S_out=None, ring_in=None, ring_out=None,
                    o=None, workspace=None, stream=None):
    """Varlen prefill of the state space mixer.  xbc [T][H*P + 2*G*N], dt
    [T][H] and z [T][H*P] (or None: no gate) may be column ranges of one
    projection tensor; ``cu_seqlens`` is a host sequence of n+1 ints.  S_in /
    S_out: [n][H][N][P] fp32, ring_in / ring_out: [n][3][H*P + 2*G*N].
    Missing outputs and the workspace are allocated with torch.  Returns
    (o, S_out, ring_out)."""
    import torch
    cu, n, T = _cu_array(cu_seqlens)
    t, H, P, N, ch = params.torch_dtype, params.num_heads, params.head_dim, params.state_dim, params.channels
    dev, f32 = xbc.get_device(), torch.float32
    _same_device(params, dev)
    x_p, sx = _rows("xbc", xbc, t, T, ch, dev)
    d_p, sd = _rows("dt", dt, t, T, H, dev)
    z_p, sz = (None, 0) if z is None else _rows("z", z, t, T, H * P, dev)
    S_p = None if S_in is None else _shaped("S_in", S_in, f32, (n, H, N, P), dev)
    r_p = None if ring_in is None else _shaped("ring_in", ring_in, t, (n, 3, ch), dev)
    o, o_p = _output("o", o, xbc, (T, H * P), t, dev, stream)
    S_out, So_p = _output("S_out", S_out, xbc, (n, H, N, P), f32, dev, stream)
    ring_out, ro_p = _output("ring_out", ring_out, xbc, (n, 3, ch), t, dev, stream)
    _, w_p, w_bytes = _workspace(workspace, xbc, kda_ssm_prefill_workspace_bytes, params, n, T, stream=stream)
    _call("kda_ssm_prefill", dev, lib().kda_ssm_prefill, params.ref, x_p, sx, d_p, sd, z_p, sz, cu, n, T, S_p, So_p,
          r_p, ro_p, o_p, w_p, w_bytes, stream=stream)
    return o, S_out, ring_out


def kda_ssm_decode_workspace_bytes(params: SsmParams, n_sessions: int) -> int:
    return int(lib().kda_ssm_decode_workspace_bytes(params.ref, int(n_sessions)))


def kda_ssm_decode(params: SsmParams, xbc, dt, S, ring, z=None, slots=None, o=None, workspace=None, stream=None):
    """One token per session; the pools S [n_slots][H][N][P] and ring
    [n_slots][3][H*P + 2*G*N] are updated in place.  xbc, dt and z hold one row
    per session, ``slots`` (int32 [n]) its pool slot.  Returns o."""
    import torch
    n = xbc.shape[0]
    t, H, P, N, ch = params.torch_dtype, params.num_heads, params.head_dim, params.state_dim, params.channels
    dev = xbc.get_device()
    _same_device(params, dev)
    x_p, sx = _rows("xbc", xbc, t, n, ch, dev)
    d_p, sd = _rows("dt", dt, t, n, H, dev)
    z_p, sz = (None, 0) if z is None else _rows("z", z, t, n, H * P, dev)
    S_p, slots_n = _pool("S", S, torch.float32, (H, N, P), dev)
    r_p = _shaped("ring", ring, t, (slots_n, 3, ch), dev)
    s_p = None if slots is None else _shaped("slots", slots, torch.int32, (n,), dev)
    o, o_p = _output("o", o, xbc, (n, H * P), t, dev, stream)
    _, w_p, w_bytes = _workspace(workspace, xbc, kda_ssm_decode_workspace_bytes, params, n, stream=stream)
    _call("kda_ssm_decode", dev, lib().kda_ssm_decode, params.ref, n, x_p, sx, d_p, sd, z_p, sz, s_p, slots_n, S_p, r_p,
          o_p, w_p, w_bytes, stream=stream)
    return o
