"""Measured cases of the gated linear recurrence and of the verification of drafts.

Five operators, each as a user calls it and in a plain form of elementary
torch operations:

* ``prefill``   packed prompts through an elementwise gated linear recurrence
  with its output gate, the state carried in and out;
* ``backward``  the gradients of such a pass, from the states it left at the
  start of every 64 tokens;
* ``decode``    one token or a straight run of tokens per session over a pool
  of states;
* ``commit``    the states after each session's accepted tokens of a round;
* ``verify``    which of the drafted tokens of a round are accepted, and the
  token that follows, from the target's and the drafter's probabilities and
  given random numbers.

Projections have unit variance, as in the repository's own workloads.  The
decays are those of a trained layer: exp(A_log) spread so that at a zero gate
logit a channel forgets within 10 to 1000 tokens.  The target's probabilities
are a softmax of logits of standard deviation 2.5, the drafter's those of the
same logits with noise of 0.7, and drafts are drawn from the drafter's.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
CHUNK = 64       # tokens between two states that the backward pass starts from
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases

def _scan(op, name, io, C, tokens, seqs, split=0, state=True, gate=True, bias=True):
    return {"name": name, "op": op, "io": io, "C": C, "tokens": tokens, "seqs": seqs, "split": split, "state": state,
            "gate": gate, "bias": bias}


def _decode(name, io, C, sessions, tokens, spare, keep=False, gate=True):
    return {"name": name, "op": "decode", "io": io, "C": C, "sessions": sessions, "tokens": tokens, "spare": spare,
            "keep": keep, "gate": gate}


def _commit(name, io, C, sessions, tokens, longest, spare):
    return {"name": name, "op": "commit", "io": io, "C": C, "sessions": sessions, "tokens": tokens, "longest": longest,
            "spare": spare}


def _verify(name, io, V, sessions, nodes, shape, drawn=True, last=False):
    return {"name": name, "op": "verify", "io": io, "V": V, "sessions": sessions, "nodes": nodes, "shape": shape,
            "drawn": drawn, "last": last}


def listed():
    return [
        # a few short prompts in fp32, as a numerics check or a tiny model runs them
        _scan("prefill", "prompts f32 601x512", "f32", 512, 601, 5, split=1, gate=False),
        # one prompt of ordinary length on a layer of 32 x 128 channels
        _scan("prefill", "prompt 4096x4096", "bf16", 4096, 4096, 1, state=False),
        # a packed batch of ragged prompts that continue their sessions
        _scan("prefill", "prompts packed 65273x8192", "bf16", 8192, 65273, 8, split=4),
        # a gradient check's size
        _scan("backward", "backward f32 777x321", "f32", 321, 777, 4, split=2),
        # a training batch of packed documents on a layer of 32 x 128 channels
        _scan("backward", "backward 32768x4096", "bf16", 4096, 32768, 5, split=3, state=False),
        # one user, one token: latency
        _decode("token x1", "bf16", 4096, 1, 1, 3),
        # a verify round of a full serving batch, the states kept until the paths are known
        _decode("round x256, 5 tokens", "bf16", 8192, 256, 5, 19, keep=True),
        # the accepted tokens of a small fp32 batch
        _commit("commit x5 f32", "f32", 768, 5, 11, 4, 2),
        # the accepted paths of a serving batch's draft trees
        _commit("commit x256", "bf16", 8192, 256, 24, 6, 11),
        # one user's straight draft of chosen tokens behind the last one: latency
        _verify("verify x1, 6 nodes", "bf16", 32000, 1, 6, "chain", drawn=False),
        # small trees over a vocabulary of odd size
        _verify("verify x37, 23 nodes f32", "f32", 50021, 37, 23, "bushy", last=True),
        # straight drafts of a full serving batch
        _verify("verify x256, 5 nodes", "f32", 131072, 256, 5, "chain"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "backward", "backward", "decode", "commit", "verify", "verify"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op in ("prefill", "backward"):
        C = rng.choice([_log_int(rng, 1, 8192), 8 * _log_int(rng, 1, 1024), 128 * _log_int(rng, 1, 64)])
        most = (65273 * 8192 if op == "prefill" else 32768 * 4096) // (C if io == "bf16" else 4 * C)
        c = _scan(op, "", io, C, _log_int(rng, 1, max(1, min(32768, most))), rng.randint(1, 12), rng.randint(0, 999),
                  rng.random() < 0.6, rng.random() < 0.7, rng.random() < 0.5)
    elif op == "decode":
        C = 4 * _log_int(rng, 1, 2048)
        n = _log_int(rng, 1, max(1, 256 * 8192 // C // 2))
        c = _decode("", io, C, min(n, 512), rng.choice([1, 1, 2, 4, rng.randint(1, 16)]), rng.randint(0, 20),
                    rng.random() < 0.4, rng.random() < 0.7)
    elif op == "commit":
        C, tokens = 4 * _log_int(rng, 1, 2048), _log_int(rng, 1, 64)
        c = _commit("", io, C, min(512, _log_int(rng, 1, max(1, 256 * 8192 // C // 2))), tokens, rng.randint(1, min(tokens, 12)),
                    rng.randint(0, 20))
    else:
        V, nodes = _log_int(rng, 200, 200000), _log_int(rng, 1, 64)
        most = (256 * 5 * 131072) // (V * nodes)
        c = _verify("", io, V, _log_int(rng, 1, max(1, min(256, most))), nodes, rng.choice(["chain", "bushy", "bushy", "star"]),
                    rng.random() < 0.7, rng.random() < 0.5)
    del c["name"]
    return c


def _lens(case):
    """The packed sequences' lengths: ragged, now and then empty or a single token."""
    rng, n, T = random.Random(case["split"] * 7919 + case["tokens"]), case["seqs"], case["tokens"]
    if n == 1:
        return [T]
    cuts = sorted(rng.randint(0, T) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [T])]


# --------------------------------------------------------------- the inputs

def _maker(seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    return (lambda *s: torch.randn(*s, generator=g, device=DEV)), (lambda *s: torch.rand(*s, generator=g, device=DEV)), g


def _gates(n, u, C, bias):
    # sigma(0) exp(A_log) = 1 / (tokens until a channel has forgotten)
    forget = torch.exp(u(C) * math.log(100) + math.log(10))
    return {"A_log": torch.log(2 / forget), "r_bias": n(C) * 0.3 if bias else None, "i_bias": n(C) * 0.3 if bias else None}


def _prepare_scan(case, seed):
    n, u, _ = _maker(seed)
    C, T, t = case["C"], case["tokens"], TYPES[case["io"]]
    # r and i are the halves of one projection's rows, x and z those of another
    ri, xz = n(T, 2 * C).to(t), n(T, 2 * C).to(t)
    s = {"case": dict(case), "r": ri[:, :C], "i": ri[:, C:], "x": xz[:, :C], "z": xz[:, C:] if case["gate"] else None,
         **_gates(n, u, C, case["bias"])}
    lens = _lens(case)
    s["cu"] = [0]
    for L in lens:
        s["cu"].append(s["cu"][-1] + L)
    s["S_in"] = n(len(lens), C) if case["state"] else None
    if case["op"] == "backward":
        s["do"] = n(T, C).to(t)
        s["dS_out"] = n(len(lens), C) if case["state"] else None
        # what the forward pass left: the state before every 64th token
        s["states"] = _forward(s)["h_before"][::CHUNK].contiguous()
        s["dri"] = torch.empty(T, 2 * C, dtype=t, device=DEV)
    return s


def _prepare_tokens(case, seed):
    n, u, g = _maker(seed)
    C, B, R, t = case["C"], case["sessions"], case["tokens"], TYPES[case["io"]]
    slots = B + case["spare"]
    s = {"case": dict(case), **_gates(n, u, C, True), "S": n(slots, C), "x": n(B, R, C).to(t), "r": n(B, R, C).to(t),
         "i": n(B, R, C).to(t), "slots": torch.randperm(slots, generator=g, device=DEV)[:B].to(torch.int32)}
    if case["op"] == "decode":
        s["z"] = n(B, R, C).to(t) if case["gate"] else None
    else:
        rng = random.Random(int(seed) * 31 + R)
        lens = [rng.randint(0, case["longest"]) for _ in range(B)]
        path = [sorted(rng.sample(range(R), k)) + [-1] * (case["longest"] - k) for k in lens]
        s["path"] = torch.tensor(path, dtype=torch.int32, device=DEV)
        s["path_len"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["S_out"] = s["S"].clone()
    return s


def _prepare_verify(case, seed):
    n, u, g = _maker(seed)
    B, R, V, t = case["sessions"], case["nodes"], case["V"], TYPES[case["io"]]
    rng = random.Random(int(seed) * 37 + R)
    parents = []
    for _ in range(B):
        row = [-1]
        for r in range(1, R):
            root = -1 if case["last"] else 0       # without p_last the root node is the session's last token
            low = max(root, (r - 1) // 3 - 1)
            row.append({"chain": r - 1, "star": root, "bushy": rng.randint(low, r - 1)}[case["shape"]])
        parents.append(row)
    # rows: behind the session's last token (where it is not the root node itself), then behind each node
    logits = n(B, R + 1, V) * 2.5
    p = torch.softmax(logits, -1)
    logits += n(B, R + 1, V) * 0.7
    q = torch.softmax(logits, -1)
    s = {"case": dict(case), "p": p[:, 1:].to(t), "p_last": p[:, 0].to(t) if case["last"] else None,
         "parents": torch.tensor(parents, dtype=torch.int32, device=DEV), "u": u(B, R), "u_next": u(B)}
    del p
    if case["drawn"]:
        s["q"], s["q_last"] = q[:, 1:].to(t), q[:, 0].to(t) if case["last"] else None
        rows = torch.gather(q.cumsum(-1, dtype=torch.float64).view(B * (R + 1), V), 0,
                            (torch.arange(B, device=DEV)[:, None] * (R + 1) + s["parents"].long() + 1).view(-1, 1).expand(B * R, V))
        drawn = torch.searchsorted(rows, u(B * R, 1).double() * rows[:, -1:])
        s["tokens"] = drawn.clamp(max=V - 1).view(B, R).to(torch.int32)
    else:
        s["q"] = s["q_last"] = None
        # each child is one of the drafter's best at its parent, a different one for each
        best = torch.topk(logits, min(V, R + 1), -1)[1]
        nth = torch.tensor([[sum(row[k] == row[r] for k in range(r)) for r in range(R)] for row in parents], device=DEV)
        at = best[torch.arange(B, device=DEV)[:, None], s["parents"].long() + 1]
        s["tokens"] = torch.gather(at, 2, nth[..., None])[..., 0].to(torch.int32)
    return s


def prepare(case, seed):
    if case["op"] in ("prefill", "backward"):
        return _prepare_scan(case, seed)
    return _prepare_verify(case, seed) if case["op"] == "verify" else _prepare_tokens(case, seed)


# ------------------------------------------------ one pass, the user's calls

def _own(s):
    import gated_delta_rule_04_gb300 as kda
    c = s["case"]
    op = c["op"]
    if op == "verify":
        path, length, token = kda.kda_draft_verify(s["p"], s["tokens"], s["parents"], s["u"], s["u_next"], q=s["q"],
                                                   p_last=s["p_last"], q_last=s["q_last"])
        return {"path": path, "path_len": length, "next": token}
    if "handle" not in s:
        s["handle"] = kda.make_glr_params(s["A_log"], r_bias=s["r_bias"], i_bias=s["i_bias"], io_dtype=c["io"])
        if op in ("prefill", "backward"):
            size = kda.kda_glr_prefill_workspace_bytes if op == "prefill" else kda.kda_glr_backward_workspace_bytes
            s["workspace"] = torch.empty(max(size(s["handle"], len(s["cu"]) - 1, c["tokens"]), 256), dtype=torch.uint8, device=DEV)
    if op == "prefill":
        o, S = kda.kda_glr_prefill(s["handle"], s["x"], s["r"], s["i"], s["cu"], z=s["z"], S_in=s["S_in"],
                                   workspace=s["workspace"])
        return {"o": o, "S": S}
    if op == "backward":
        C = c["C"]
        g = kda.kda_glr_backward(s["handle"], s["x"], s["r"], s["i"], s["cu"], s["states"], s["do"], z=s["z"], S_in=s["S_in"],
                                 dS_out=s["dS_out"], dr=s["dri"][:, :C], di=s["dri"][:, C:], workspace=s["workspace"])
        return {"dx": g.dx, "dri": s["dri"], "dz": g.dz, "dS_in": g.dS_in if c["state"] else None, "dA_log": g.dA_log,
                "dr_bias": g.dr_bias if c["bias"] else None, "di_bias": g.di_bias if c["bias"] else None}
    if op == "decode":
        o = kda.kda_glr_decode(s["handle"], s["x"], s["r"], s["i"], s["S"], z=s["z"], slots=s["slots"], keep_state=c["keep"])
        return {"o": o, "S": s["S"]}
    return kda.kda_glr_commit(s["handle"], s["x"], s["r"], s["i"], s["path"], s["path_len"], s["S"], S_out=s["S_out"],
                              slots=s["slots"])


# --------------------------------------------------- one pass, plainly written

def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _biased(x, b):
    return x.float() if b is None else x.float() + b


def _steps(s, x, r, i):
    """Decays a, their logarithms, inputs b and the factors of b, in 32 bits."""
    w, v = _sigmoid(_biased(r, s["r_bias"])), _sigmoid(_biased(i, s["i_bias"]))
    la = -torch.exp(s["A_log"]) * w
    m = torch.sqrt(-torch.expm1(2 * la))
    return torch.exp(la), la, w, v, m, m * v * x.float()


def _linear_scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis from zero: doubling steps within 64 rows, then over the 64-row blocks."""
    T, C = a.shape
    K = -(-T // CHUNK)
    pad = K * CHUNK - T
    A = torch.cat([a, a.new_ones(pad, C)]).view(K, CHUNK, C)
    B = torch.cat([b, b.new_zeros(pad, C)]).view(K, CHUNK, C)
    d = 1
    while d < CHUNK:
        B = torch.cat([B[:, :d], B[:, d:] + A[:, d:] * B[:, :-d]], 1)
        A = torch.cat([A[:, :d], A[:, d:] * A[:, :-d]], 1)
        d *= 2
    eA, eB, d = A[:, -1], B[:, -1], 1
    while d < K:
        eB = torch.cat([eB[:d], eB[d:] + eA[d:] * eB[:-d]])
        eA = torch.cat([eA[:d], eA[d:] * eA[:-d]])
        d *= 2
    B[1:] += A[1:] * eB[:-1, None]
    return B.view(K * CHUNK, C)[:T]


def _marks(s):
    """Per sequence with tokens: its index, first and last token."""
    live = [(n, a, b - 1) for n, (a, b) in enumerate(zip(s["cu"], s["cu"][1:])) if b > a]
    return tuple(torch.tensor(v, device=DEV, dtype=torch.long) for v in (zip(*live) if live else ((), (), ())))


def _forward(s):
    a, la, w, v, m, b = _steps(s, s["x"], s["r"], s["i"])
    seq, first, last = _marks(s)
    start = torch.zeros(len(s["cu"]) - 1, a.shape[1], device=DEV) if s["S_in"] is None else s["S_in"]
    a2, b2 = a.clone(), b.clone()
    b2[first] += a[first] * start[seq]
    a2[first] = 0
    h = _linear_scan(a2, b2)
    S = start.clone()
    S[seq] = h[last]
    before = torch.cat([h.new_zeros(1, h.shape[1]), h[:-1]])
    before[first] = start[seq]
    return {"a": a, "la": la, "w": w, "v": v, "m": m, "b": b, "h": h, "h_before": before, "S": S, "first": first, "last": last,
            "seq": seq}


def _plain_prefill(s):
    f = _forward(s)
    o = f["h"]
    if s["z"] is not None:
        z = s["z"].float()
        o = o * z * _sigmoid(z)
    return {"o": o.to(TYPES[s["case"]["io"]]), "S": f["S"]}


def _plain_backward(s):
    f, t, case = _forward(s), TYPES[s["case"]["io"]], s["case"]
    T = case["tokens"]
    do = s["do"].float()
    dz, G = None, do
    if s["z"] is not None:
        z = s["z"].float()
        e = _sigmoid(z)
        dz = (do * f["h"] * e * (1 + z * (1 - e))).to(t)
        G = do * z * e
    if s["dS_out"] is not None:
        G = G.clone()
        G[f["last"]] += s["dS_out"][f["seq"]]
    nxt = torch.cat([f["a"][1:], f["a"].new_zeros(1, case["C"])])     # the decay between a token and the next one
    nxt[f["last"]] = 0
    g = _linear_scan(nxt.flip(0), G.flip(0)).flip(0)
    a, la, w, v, m, b = (f[k] for k in ("a", "la", "w", "v", "m", "b"))
    dla = g * (a * f["h_before"] - a * a / (m * m) * b)
    dr, di = dla * la * (1 - w), g * b * (1 - v)
    out = {"dx": (g * m * v).to(t), "dri": torch.cat([dr, di], 1).to(t), "dz": dz}
    dS = None
    if case["state"]:
        dS = s["dS_out"].clone()
        dS[f["seq"]] = (a * g)[f["first"]]
    out["dS_in"] = dS
    # sums over all tokens in 64 bits
    out["dA_log"] = (dla * la).sum(0, dtype=torch.float64).float()
    out["dr_bias"] = dr.sum(0, dtype=torch.float64).float() if case["bias"] else None
    out["di_bias"] = di.sum(0, dtype=torch.float64).float() if case["bias"] else None
    return out


def _plain_decode(s):
    c, idx = s["case"], s["slots"].long()
    a, _, _, _, _, b = _steps(s, s["x"], s["r"], s["i"])
    h, rows = s["S"][idx], []
    for j in range(c["tokens"]):
        h = a[:, j] * h + b[:, j]
        rows.append(h)
    o = torch.stack(rows, 1)
    if s["z"] is not None:
        z = s["z"].float()
        o = o * z * _sigmoid(z)
    if not c["keep"]:
        s["S"][idx] = h
    return {"o": o.to(TYPES[c["io"]]), "S": s["S"]}


def _plain_commit(s):
    c, idx = s["case"], s["slots"].long()
    at = s["path"].long().clamp(min=0)[..., None].expand(c["sessions"], c["longest"], c["C"])
    a, _, _, _, _, b = _steps(s, *(torch.gather(s[k], 1, at) for k in ("x", "r", "i")))
    h = s["S"][idx]
    for j in range(c["longest"]):
        h = torch.where((j < s["path_len"])[:, None], a[:, j] * h + b[:, j], h)
    s["S_out"][idx] = h
    return s["S_out"]


def _plain_verify(s):
    c = s["case"]
    B, R = c["sessions"], c["nodes"]
    each = torch.arange(B, device=DEV)
    # rows of the last token first; in 64 bits: sums over a vocabulary next to a random border
    blank = torch.zeros(B, 1, c["V"], dtype=s["p"].dtype, device=DEV)
    p = torch.cat([blank if s["p_last"] is None else s["p_last"][:, None], s["p"]], 1)
    q = None if s["q"] is None else torch.cat([blank if s["q_last"] is None else s["q_last"][:, None], s["q"]], 1)
    cur = torch.full((B,), -1, device=DEV)
    coef, T = torch.zeros(B, dtype=torch.float64, device=DEV), torch.ones(B, dtype=torch.float64, device=DEV)
    gone = torch.zeros(B, c["V"], dtype=torch.bool, device=DEV)       # tokens refused at the current node
    path, length = torch.full((B, R), -1, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.long, device=DEV)
    for r in range(R):
        x, test = s["tokens"][:, r].long(), s["parents"][:, r] == cur
        W = p[each, cur + 1, x].double()
        if q is None:
            W = torch.where(gone[each, x], 0.0, W)
            yes = s["u"][:, r].double() * T < W
        else:
            qx = q[each, cur + 1, x].double()
            W = (W - coef * qx).clamp(min=0)
            yes = s["u"][:, r].double() * T * qx < W
        yes = yes & (W > 0)
        if s["p_last"] is None:
            yes = yes | (cur < 0)
        yes, no = yes & test, test & ~yes
        if q is None:
            T = torch.where(no, T - W, T)
            gone[each, x] |= no
        else:
            coef = torch.where(no, coef + T, coef)
            left = (p[each, cur + 1].double() - coef[:, None] * q[each, cur + 1].double()).clamp(min=0).sum(1)
            T = torch.where(no, left, T)
        end = length.clamp(max=R - 1)
        path[each, end] = torch.where(yes, torch.full_like(path[:, 0], r), path[each, end])
        length = length + yes
        cur, coef, T = torch.where(yes, r, cur), torch.where(yes, 0.0, coef), torch.where(yes, 1.0, T)
        gone &= ~yes[:, None]
    row = p[each, cur + 1].double()
    W = torch.where(gone, 0.0, row) if q is None else (row - coef[:, None] * q[each, cur + 1].double()).clamp(min=0)
    W = torch.where((W.sum(1) > 0)[:, None], W, row)
    cum = W.cumsum(1)
    over = (cum > s["u_next"].double()[:, None] * cum[:, -1:]) & (W > 0)
    at = torch.arange(c["V"], device=DEV)
    first = torch.where(over, at, c["V"]).amin(1)
    last = torch.where(W > 0, at, -1).amax(1)
    return {"path": path, "path_len": length.to(torch.int32), "next": torch.where(first < c["V"], first, last).to(torch.int32)}


def run(state):
    if own:
        return _own(state)
    return {"prefill": _plain_prefill, "backward": _plain_backward, "decode": _plain_decode, "commit": _plain_commit,
            "verify": _plain_verify}[state["case"]["op"]](state)


# ------------------------------------------------------- what a pass needs

def work(case):
    e = 2 if case["io"] == "bf16" else 4
    if case["op"] == "verify":
        B, R, V = case["sessions"], case["nodes"], case["V"]
        # one row of the target's probabilities a session, and one of the drafter's where a draft was refused (two in three)
        rows = B * V * (5 / 3 if case["drawn"] else 1)
        return {"bytes": int(rows * e + B * R * (16 + 2 * e) + B * 12), "flops": int(rows * 4)}
    C = case["C"]
    if case["op"] in ("prefill", "backward"):
        T, n = case["tokens"], case["seqs"]
        rows = (5 if case["gate"] else 4) if case["op"] == "prefill" else (9 if case["gate"] else 7)
        states = n * (2 if case["state"] else 1) * 4 + (0 if case["op"] == "prefill" else (T + CHUNK - 1) // CHUNK * 4)
        return {"bytes": C * (rows * T * e + states + 16), "flops": T * C * (60 if case["op"] == "prefill" else 110)}
    B = case["sessions"]
    if case["op"] == "decode":
        return {"bytes": C * (B * case["tokens"] * (5 if case["gate"] else 4) * e + B * (4 if case["keep"] else 8) + 12),
                "flops": B * case["tokens"] * C * 60}
    rows = B * (case["longest"] + 1) // 2
    return {"bytes": C * (rows * 3 * e + B * 8 + 12), "flops": rows * C * 45}


# ------------------------------- the definitions, token by token in 64 bits

def _exact_token(s, x, r, i):
    """a, m sigma(i), and what the gradients need, of one token's rows."""
    zr = r.double() + (0 if s["r_bias"] is None else s["r_bias"].double())
    zi = i.double() + (0 if s["i_bias"] is None else s["i_bias"].double())
    ea = s["A_log"].double().exp()
    la = -ea * torch.sigmoid(zr)
    m = (-torch.special.expm1(la + la)).sqrt()
    return la.exp(), la, m, torch.sigmoid(zi), torch.sigmoid(-zr), torch.sigmoid(-zi)


def _exact_scan(case, s):
    """States token by token, sequences side by side, longest first."""
    lens, C, T = _lens(case), case["C"], case["tokens"]
    order = sorted(range(len(lens)), key=lambda k: -lens[k])
    start = torch.tensor([s["cu"][k] for k in order], device=DEV)
    S = torch.zeros(len(lens), C, dtype=torch.float64, device=DEV) if s["S_in"] is None else s["S_in"].double()[order].clone()
    back = [order.index(k) for k in range(len(lens))]
    want = case["op"] == "prefill"
    out = torch.empty(T, C, dtype=torch.float64, device=DEV)
    for t in range(max(lens)):
        m = sum(L > t for L in lens)
        at = start[:m] + t
        if not want:
            out[at] = S[:m]                                           # the state before the token
        a, _, scale, v, _, _ = _exact_token(s, s["x"][at], s["r"][at], s["i"][at])
        S[:m] = a * S[:m] + scale * v * s["x"][at].double()
        if want:
            out[at] = S[:m]
    if want:
        if s["z"] is not None:
            z = s["z"].double()
            out *= z * torch.sigmoid(z)
        return {"o": out, "S": S[back]}
    f64 = dict(dtype=torch.float64, device=DEV)
    dx, dri, dz = torch.empty(T, C, **f64), torch.empty(T, 2 * C, **f64), torch.empty(T, C, **f64)
    dA, dr_b, di_b = torch.zeros(C, **f64), torch.zeros(C, **f64), torch.zeros(C, **f64)
    carry = torch.zeros(len(lens), C, **f64) if s["dS_out"] is None else s["dS_out"].double()[order].clone()
    for t in range(max(lens) - 1, -1, -1):
        n = sum(L > t for L in lens)
        at = start[:n] + t
        x = s["x"][at].double()
        a, la, m, v, w_, v_ = _exact_token(s, s["x"][at], s["r"][at], s["i"][at])
        do = s["do"][at].double()
        if s["z"] is not None:
            z = s["z"][at].double()
            sz = torch.sigmoid(z)
            h = a * out[at] + m * v * x
            dz[at] = do * h * (sz + z * sz * torch.sigmoid(-z))
            do = do * z * sz
        g = do + carry[:n]
        dx[at] = g * m * v
        # h_t = a h + m v x: by a and by m(a), both functions of la
        dla = g * out[at] * a - g * v * x * a * a / m
        step = dla * la
        dr, di = step * w_, g * m * x * v * v_
        dri[at] = torch.cat([dr, di], 1)
        dA += step.sum(0)
        dr_b += dr.sum(0)
        di_b += di.sum(0)
        carry[:n] = a * g
    return {"dx": dx, "dri": dri, "dz": dz if s["z"] is not None else None, "dS_in": carry[back] if case["state"] else None,
            "dA_log": dA, "dr_bias": dr_b if case["bias"] else None, "di_bias": di_b if case["bias"] else None}


def _exact_tokens(case, s):
    S, out = s["S"].double(), None
    if case["op"] == "decode":
        out = torch.empty(case["sessions"], case["tokens"], case["C"], dtype=torch.float64, device=DEV)
    for b, slot in enumerate(s["slots"].tolist()):
        taken = range(case["tokens"]) if out is not None else s["path"][b, :int(s["path_len"][b])].tolist()
        h = S[slot].clone()
        for j in taken:
            a, _, m, v, _, _ = _exact_token(s, s["x"][b, j], s["r"][b, j], s["i"][b, j])
            h = a * h + m * v * s["x"][b, j].double()
            if out is not None:
                out[b, j] = h
        if out is None or not case["keep"]:
            S[slot] = h
    if out is None:
        return S
    if s["z"] is not None:
        z = s["z"].double()
        out *= z * torch.sigmoid(z)
    return {"o": out, "S": S}


def _exact_verify(case, s):
    B, R, V = case["sessions"], case["nodes"], case["V"]
    path, lens, nxt = torch.full((B, R), -1, dtype=torch.int32), [], []
    for b in range(B):
        parents, tokens, u = s["parents"][b].tolist(), s["tokens"][b].tolist(), s["u"][b].tolist()

        def dist(of, last, node):
            row = of[b, node] if node >= 0 else (None if last is None else last[b])
            return None if row is None else row.double()

        node, taken, left = -1, [], dist(s["p"], s["p_last"], -1)      # left: what the target still has to give here, normalised
        while True:
            for r in [r for r in range(R) if parents[r] == node]:
                x = tokens[r]
                if left is None:
                    ok = True
                else:
                    draft = torch.zeros(V, dtype=torch.float64, device=DEV) if s["q"] is None else dist(s["q"], s["q_last"], node)
                    if s["q"] is None:
                        draft[x] = 1
                    have = float(left[x])
                    ok = have > 0 and u[r] * float(draft[x]) < have
                if ok:
                    node = r
                    break
                rest = (left - draft).clamp(min=0)
                if s["q"] is None:                                     # p's own sum may be off 1 by its rounding
                    rest, total = torch.where(draft > 0, 0.0, left), 1 - have
                else:
                    total = float(rest.sum())
                left = rest / total if total > 0 else rest
            else:
                break
            taken.append(node)
            left = dist(s["p"], s["p_last"], node)
        if left is None:
            left = torch.zeros(V, dtype=torch.float64, device=DEV)
        if not bool((left > 0).any()):
            row = dist(s["p"], s["p_last"], node)
            left = left if row is None else row
        cum = torch.cumsum(left, 0)
        hit = ((cum > float(s["u_next"][b]) * cum[-1]) & (left > 0)).nonzero()
        live = (left > 0).nonzero()
        nxt.append(int(hit[0]) if len(hit) else int(live[-1]) if len(live) else -1)
        lens.append(len(taken))
        path[b, :len(taken)] = torch.tensor(taken, dtype=torch.int32)
    return {"path": path.to(DEV), "path_len": torch.tensor(lens, dtype=torch.int32, device=DEV),
            "next": torch.tensor(nxt, dtype=torch.int32, device=DEV)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("prefill", "backward"):
        return _exact_scan(case, s)
    return _exact_verify(case, s) if case["op"] == "verify" else _exact_tokens(case, s)
