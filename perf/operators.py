"""Measured cases of the state-space mixer and of draft trees over the KDA state.

Four operators, each as a user calls it and in a plain form of elementary
torch operations:

* ``ssm_prefill``  packed prompts through the short conv, the selective state
  space scan and the output gate, with state and conv ring carried in and out;
* ``ssm_decode``   one token per session over a pool of states, in place;
* ``tree``         the outputs of every node of a tree of drafted tokens
  against each session's KDA state, which stays as it is;
* ``commit``       the KDA state and ring after each session's accepted path.

The random numbers follow the distributions that the repository's own
workloads use (unit-variance projections, conv weights of variance 0.25,
A_log = log U(1, 16), gate bound -5); the state-space step sizes are those of
a trained layer's range, 0.001 to 0.1 at a zero logit.
"""
from __future__ import annotations

import math
import random

import torch
import torch.nn.functional as F

own = False

DEV = "cuda"
D = 128          # head width of the KDA mixer
CHUNK = 64       # tokens per block of the plain scan
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases

def _prefill(name, io, H, P, N, G, tokens, seqs, split=0, state=True, gate=True, bias=True):
    return {"name": name, "op": "ssm_prefill", "io": io, "H": H, "P": P, "N": N, "G": G, "tokens": tokens, "seqs": seqs,
            "split": split, "state": state, "gate": gate, "bias": bias}


def _decode(name, io, H, P, N, G, sessions, spare, gate=True, bias=True):
    return {"name": name, "op": "ssm_decode", "io": io, "H": H, "P": P, "N": N, "G": G, "sessions": sessions,
            "spare": spare, "gate": gate, "bias": bias}


def _tree(name, io, H, sessions, nodes, shape, spare=0, softplus=False):
    return {"name": name, "op": "tree", "io": io, "H": H, "sessions": sessions, "nodes": nodes, "shape": shape,
            "spare": spare, "softplus": softplus}


def _commit(name, io, H, sessions, nodes, longest, spare=0, softplus=False):
    return {"name": name, "op": "commit", "io": io, "H": H, "sessions": sessions, "nodes": nodes, "longest": longest,
            "spare": spare, "softplus": softplus}


def listed():
    return [
        # a few short prompts in fp32, as a numerics check or a tiny model runs them
        _prefill("ssm prompts f32 8x64", "f32", 8, 64, 64, 2, 601, 5, split=1),
        # one prompt of ordinary length on a 32-head layer
        _prefill("ssm prompt 4096", "bf16", 32, 128, 128, 1, 4096, 1, state=False),
        # one long document on a 96-head layer
        _prefill("ssm prompt 32768", "bf16", 96, 64, 128, 8, 32768, 1, state=False),
        # a packed batch of ragged prompts that continue their sessions
        _prefill("ssm prompts packed", "bf16", 64, 64, 128, 4, 65273, 8, split=4),
        # one user, one token: latency
        _decode("ssm token x1", "bf16", 32, 64, 128, 1, 1, 3),
        # an fp32 service with an odd batch
        _decode("ssm token x37 f32", "f32", 20, 64, 64, 5, 37, 4, gate=False, bias=False),
        # a full serving batch over a pool of states
        _decode("ssm token x256", "bf16", 64, 64, 128, 8, 256, 19),
        # one user's draft tree: latency
        _tree("tree x1, 16 nodes", "bf16", 32, 1, 16, "bushy", spare=2),
        # an odd batch of small trees in fp32 with the softplus gate
        _tree("tree x7, 11 nodes f32", "f32", 6, 7, 11, "bushy", softplus=True),
        # a serving batch of wide trees
        _tree("tree x64, 64 nodes", "bf16", 32, 64, 64, "bushy", spare=9),
        # the accepted paths of a small fp32 batch
        _commit("commit x5 f32", "f32", 6, 5, 11, 4),
        # the accepted paths of a serving batch
        _commit("commit x256", "bf16", 32, 256, 24, 6, spare=11),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ssm_prefill", "ssm_prefill", "ssm_decode", "tree", "commit"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("ssm_prefill", "ssm_decode"):
        P, N, G = rng.choice([64, 128]), rng.choice([64, 128]), rng.choice([1, 1, 2, 3, 8])
        H = G * _log_int(rng, 1, max(1, (96 * 64) // (P * G)))
        gate, bias = rng.random() < 0.7, rng.random() < 0.5
        if op == "ssm_prefill":
            most = (65273 * 64 * 64 if io == "bf16" else 2048 * 64 * 64) // (H * P)
            tokens = _log_int(rng, 1, max(1, min(32768, most)))
            c = _prefill("", io, H, P, N, G, tokens, rng.randint(1, 12), rng.randint(0, 999), rng.random() < 0.6, gate, bias)
        else:
            most = (256 * 64 * 64 * 128) // (H * P * N)
            c = _decode("", io, H, P, N, G, _log_int(rng, 1, max(1, min(512, most))), rng.randint(0, 20), gate, bias)
    else:
        H = _log_int(rng, 1, 40)
        softplus = rng.random() < 0.3
        if op == "tree":
            nodes = _log_int(rng, 1, 64)
            most = (64 * 32 * 64) // (H * nodes)
            c = _tree("", io, H, _log_int(rng, 1, max(1, min(256, most))), nodes, rng.choice(["bushy", "bushy", "chain", "star"]),
                      rng.randint(0, 9), softplus)
        else:
            nodes = _log_int(rng, 2, 64)
            c = _commit("", io, H, _log_int(rng, 1, max(1, (256 * 32) // H // 2)), nodes, rng.randint(1, min(nodes, 12)),
                        rng.randint(0, 9), softplus)
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


def _prepare_ssm(case, seed):
    n, u, g = _maker(seed)
    H, P, N, G, t = case["H"], case["P"], case["N"], case["G"], TYPES[case["io"]]
    W, C = H * P, H * P + 2 * G * N
    rows = case["tokens"] if case["op"] == "ssm_prefill" else case["sessions"]
    # one projection row per token, as the layer's input product leaves it: gate | conv channels | step logits
    width = (W + C + H + 7) // 8 * 8
    proj = n(rows, width).to(t)
    step = torch.exp(u(H) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
    s = {"case": dict(case), "proj": proj, "z": proj[:, :W] if case["gate"] else None, "xbc": proj[:, W:W + C],
         "dt": proj[:, W + C:W + C + H], "conv_w": n(C, 4) * 0.5, "conv_b": n(C) * 0.1 if case["bias"] else None,
         "A_log": torch.log(u(H) * 15 + 1), "dt_bias": step + torch.log(-torch.expm1(-step)),
         "D": 1 + 0.1 * n(H)}
    if case["op"] == "ssm_prefill":
        lens = _lens(case)
        s["cu"] = [0]
        for L in lens:
            s["cu"].append(s["cu"][-1] + L)
        s["S_in"] = n(len(lens), H, N, P) * 0.3 if case["state"] else None
        s["ring_in"] = n(len(lens), 3, C).to(t) if case["state"] else None
    else:
        slots = rows + case["spare"]
        s["S"], s["ring"] = n(slots, H, N, P) * 0.3, n(slots, 3, C).to(t)
        s["slots"] = torch.randperm(slots, generator=g, device=DEV)[:rows].to(torch.int32)
    return s


def _parents(case, rng):
    """A tree per session, parents before children; -1 hangs a node on the session's last token."""
    out = []
    for _ in range(case["sessions"]):
        m = case.get("shape", "bushy")
        row = [-1]
        for i in range(1, case["nodes"]):
            row.append(i - 1 if m == "chain" else -1 if m == "star" else rng.randint(max(-1, (i - 1) // 3 - 1), i - 1))
        out.append(row)
    return out


def _prepare_kda(case, seed):
    n, u, g = _maker(seed)
    H, t, B, R = case["H"], TYPES[case["io"]], case["sessions"], case["nodes"]
    W, slots = H * D, case["sessions"] + case["spare"]
    rng = random.Random(int(seed) * 31 + R)
    parents = _parents(case, rng)
    s = {"case": dict(case), "conv_w": n(3, W, 4) * 0.5, "A_log": torch.log(u(H) * 15 + 1), "dt_bias": n(W) * math.sqrt(0.5),
         "norm_w": 1 + n(D) * math.sqrt(0.1), "parents": torch.tensor(parents, dtype=torch.int32, device=DEV),
         "S": n(slots, H, D, D) * 0.05, "ring": n(slots, 3, 3, W).to(t),
         "slots": torch.randperm(slots, generator=g, device=DEV)[:B].to(torch.int32)}
    for name in ("q", "k", "v", "z", "gout"):
        s[name] = n(B, R, W).to(t)
    s["b"] = n(B, R, H).to(t)
    if case["op"] == "commit":
        # each session accepted a path from the root's side: 0 to `longest` nodes deep
        path, lens = [], []
        for row in parents:
            leaf, p = rng.randrange(R), []
            while leaf >= 0:
                p.append(leaf)
                leaf = row[leaf]
            p = p[::-1][:rng.randint(0, case["longest"])]
            lens.append(len(p))
            path.append(p + [-1] * (case["longest"] - len(p)))
        s["path"] = torch.tensor(path, dtype=torch.int32, device=DEV)
        s["path_len"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["S_out"], s["ring_out"] = s["S"].clone(), s["ring"].clone()
    return s


def prepare(case, seed):
    return _prepare_ssm(case, seed) if case["op"] in ("ssm_prefill", "ssm_decode") else _prepare_kda(case, seed)


# ------------------------------------------------ one pass, the user's calls

def _own(s):
    import gated_delta_rule_04_gb300 as kda
    c = s["case"]
    if c["op"] in ("ssm_prefill", "ssm_decode"):
        if "handle" not in s:
            s["handle"] = kda.make_ssm_params(s["conv_w"], s["A_log"], s["dt_bias"], head_dim=c["P"], state_dim=c["N"],
                                              num_groups=c["G"], D=s["D"], conv_b=s["conv_b"], io_dtype=c["io"])
            nbytes = (kda.kda_ssm_prefill_workspace_bytes(s["handle"], len(s["cu"]) - 1, s["cu"][-1])
                      if c["op"] == "ssm_prefill" else kda.kda_ssm_decode_workspace_bytes(s["handle"], c["sessions"]))
            s["workspace"] = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=DEV)
        if c["op"] == "ssm_prefill":
            o, S, ring = kda.kda_ssm_prefill(s["handle"], s["xbc"], s["dt"], s["cu"], z=s["z"], S_in=s["S_in"],
                                             ring_in=s["ring_in"], workspace=s["workspace"])
            return {"o": o, "S": S, "ring": ring}
        o = kda.kda_ssm_decode(s["handle"], s["xbc"], s["dt"], s["S"], s["ring"], z=s["z"], slots=s["slots"],
                               workspace=s["workspace"])
        return {"o": o, "S": s["S"], "ring": s["ring"]}
    if "handle" not in s:
        s["handle"] = kda.make_params(s["conv_w"], s["A_log"], s["dt_bias"], s["norm_w"], io_dtype=c["io"],
                                      gate="softplus" if c["softplus"] else "bounded")
    if c["op"] == "tree":
        return kda.kda_decode_tree(s["handle"], s["q"], s["k"], s["v"], s["z"], s["b"], s["gout"], s["parents"], s["S"],
                                   s["ring"], slots=s["slots"])
    kda.kda_tree_commit(s["handle"], s["q"], s["k"], s["v"], s["z"], s["b"], s["path"], s["path_len"], s["S"], s["ring"],
                        S_out=s["S_out"], ring_out=s["ring_out"], slots=s["slots"])
    return {"S": s["S_out"], "ring": s["ring_out"]}


# --------------------------------------------------- one pass, plainly written

def _silu(x):
    return x / (1 + torch.exp(-x))


def _conv4(rows, w, b):
    """rows [..., 3 + L, C] -> [..., L, C]: the causal conv of four taps, then SiLU."""
    L = rows.shape[-2] - 3
    y = rows[..., :L, :] * w[:, 0] + rows[..., 1:L + 1, :] * w[:, 1] + rows[..., 2:L + 2, :] * w[:, 2] + rows[..., 3:, :] * w[:, 3]
    return _silu(y if b is None else y + b)


def _plain_prefill(s):
    c = s["case"]
    H, P, N, G, t = c["H"], c["P"], c["N"], c["G"], TYPES[c["io"]]
    W, C, n = H * P, H * P + 2 * G * N, len(s["cu"]) - 1
    cu = torch.tensor(s["cu"], device=DEV)
    lens = cu[1:] - cu[:-1]
    K = max(1, -(-(max(b - a for a, b in zip(s["cu"], s["cu"][1:]))) // CHUNK))
    at = torch.arange(K * CHUNK, device=DEV)
    live = at[None] < lens[:, None]                                    # [n, L]
    rows = (cu[:-1, None] + at[None]).clamp(max=c["tokens"] - 1)
    raw = s["xbc"][rows] * live[..., None].to(t)                       # [n, L, C]
    ring = s["ring_in"] if s["ring_in"] is not None else torch.zeros(n, 3, C, dtype=t, device=DEV)
    raw = torch.cat([ring, raw], 1)
    last = (lens[:, None] + torch.arange(3, device=DEV))[..., None].expand(n, 3, C)
    ring_out = torch.gather(raw, 1, last)
    u = _conv4(raw.float(), s["conv_w"], s["conv_b"])
    del raw
    x = u[..., :W].reshape(n, K, CHUNK, H, P)
    Bm = u[..., W:W + G * N].reshape(n, K, CHUNK, G, N)
    Cm = u[..., W + G * N:].reshape(n, K, CHUNK, G, N)
    dt = F.softplus(s["dt"][rows].float() + s["dt_bias"]) * live[..., None]
    # cumulative log decays in 64 bits: differences of long sums
    lam = (-torch.exp(s["A_log"].double()) * dt.double()).reshape(n, K, CHUNK, H).cumsum(2)
    dt = dt.reshape(n, K, CHUNK, H)
    hg = torch.arange(H, device=DEV) // (H // G)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()
    lt = lam.permute(0, 1, 3, 2)                                       # [n, K, H, C]
    M = torch.exp((lt[..., :, None] - lt[..., None, :]).masked_fill(~low, -math.inf)).float()
    M = M * dt.permute(0, 1, 3, 2)[..., None, :]
    CB = torch.einsum("bkigd,bkjgd->bkgij", Cm, Bm)
    M = M * CB[:, :, hg]
    xh = x.permute(0, 1, 3, 2, 4)                                      # [n, K, H, C, P]
    y = M @ xh
    del M
    out_w = (torch.exp(lt[..., -1:] - lt).float() * dt.permute(0, 1, 3, 2))[..., None]
    Bh = Bm.permute(0, 1, 3, 4, 2)[:, :, hg]                           # [n, K, H, N, C]
    local = Bh @ (xh * out_w)                                          # [n, K, H, N, P]
    del Bh
    # states before each block and after the last: sums over the earlier blocks
    tot = torch.cat([torch.zeros(n, 1, H, dtype=torch.float64, device=DEV), lt[..., -1].cumsum(1)], 1)
    early = torch.ones(K + 1, K, dtype=torch.bool, device=DEV).tril(-1)
    gap = (tot[:, :, None] - tot[:, None, 1:]).masked_fill(~early[None, :, :, None], -math.inf)
    gap = torch.exp(gap).float().permute(0, 3, 1, 2)                   # [n, H, K+1, K]
    S = (gap @ local.permute(0, 2, 1, 3, 4).reshape(n, H, K, N * P)).reshape(n, H, K + 1, N, P)
    del local
    if s["S_in"] is not None:
        S = S + torch.exp(tot).float().permute(0, 2, 1)[..., None, None] * s["S_in"][:, :, None]
    Ch = Cm.permute(0, 1, 3, 2, 4)[:, :, hg]                           # [n, K, H, C, N]
    y = y + torch.exp(lt).float()[..., None] * (Ch @ S[:, :, :-1].transpose(1, 2))
    y = y + s["D"][:, None, None] * xh
    y = y.permute(0, 1, 3, 2, 4).reshape(n, K * CHUNK, W)[live]
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return {"o": y.to(t), "S": S[:, :, -1].contiguous(), "ring": ring_out}


def _plain_decode(s):
    c = s["case"]
    H, P, N, G, t = c["H"], c["P"], c["N"], c["G"], TYPES[c["io"]]
    W, B, idx = H * P, c["sessions"], s["slots"].long()
    rows = torch.cat([s["ring"][idx], s["xbc"][:, None]], 1)
    u = _conv4(rows.float(), s["conv_w"], s["conv_b"])[:, 0]
    hg = torch.arange(H, device=DEV) // (H // G)
    x = u[:, :W].reshape(B, H, P)
    Bm, Cm = (v.reshape(B, G, N)[:, hg] for v in u[:, W:].split(G * N, 1))
    dt = F.softplus(s["dt"].float() + s["dt_bias"])
    S = s["S"][idx] * torch.exp(-torch.exp(s["A_log"]) * dt)[..., None, None] + (dt[..., None] * Bm)[..., None] * x[:, :, None]
    y = (S * Cm[..., None]).sum(2) + s["D"][:, None] * x
    y = y.reshape(B, W)
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["S"][idx] = S
    s["ring"][idx] = rows[:, 1:]
    return {"o": y.to(t), "S": s["S"], "ring": s["ring"]}


def _kda_gate(s, z):
    """The log decays of the gate logits z [..., H*128], in 64 bits."""
    a = torch.exp(s["A_log"].double()).repeat_interleave(D)
    zb = z.double() + s["dt_bias"].double()
    if s["case"]["softplus"]:
        return -a * F.softplus(zb)
    return -5.0 / (1 + torch.exp(-a * zb))


def _kda_rows(s, win):
    """Conv, SiLU and norms of the nodes whose windows (rows of ring | nodes) are win [B, R, 4]."""
    c = s["case"]
    B, R, H = win.shape[0], win.shape[1], c["H"]
    W = H * D
    ring = s["ring"][s["slots"].long()]

    def plane(p, x):
        rows = torch.cat([ring[:, p], x], 1).float()
        taken = torch.gather(rows, 1, win.reshape(B, R * 4, 1).expand(B, R * 4, W)).reshape(B, R, 4, W)
        return _silu((taken * s["conv_w"][p].T).sum(2)).reshape(B, R, H, D).transpose(1, 2)

    q, k, v = plane(0, s["q"]), plane(1, s["k"]), plane(2, s["v"])
    q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6) * D ** -0.5
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    return q, k, v


def _windows(before):
    """The four-row windows, oldest first: `before` [B, 3 + R] is the row before each row of ring | nodes."""
    B, R = before.shape[0], before.shape[1] - 3
    w3 = torch.arange(3, 3 + R, device=DEV).expand(B, R)
    w2 = torch.gather(before, 1, w3)
    w1 = torch.gather(before, 1, w2)
    return torch.stack([torch.gather(before, 1, w1), w1, w2, w3], -1)


def _kda_solve(S0, k, v, gam, beta, strict):
    """u of every node: (1 + beta A)^-1 beta (v - (k e^gam)^T S0), A over the strict ancestors; and the pairs' decays."""
    gap = (gam[:, :, :, None] - gam[:, :, None]).masked_fill(~(strict | torch.eye(k.shape[2], dtype=torch.bool, device=DEV))[..., None], -math.inf)
    gap = torch.exp(gap).float()
    A = torch.where(strict, ((k[:, :, :, None] * k[:, :, None]) * gap).sum(-1), 0.0).double()
    rhs = beta[..., None] * (v - (k * torch.exp(gam).float()) @ S0)
    m = -beta[..., None].double() * A                                  # nilpotent: at most 64 nodes deep
    one = torch.eye(k.shape[2], dtype=torch.float64, device=DEV)
    m2 = m @ m
    m4 = m2 @ m2
    m8 = m4 @ m4
    m16 = m8 @ m8
    inv = (one + m) @ (one + m2) @ (one + m4) @ (one + m8) @ (one + m16) @ (one + m16 @ m16)
    return (inv @ rhs.double()).float(), gap


def _plain_tree(s):
    c = s["case"]
    H, B, R, t = c["H"], c["sessions"], c["nodes"], TYPES[c["io"]]
    par = s["parents"].long()
    before = torch.cat([torch.tensor([0, 0, 1], device=DEV).expand(B, 3), torch.where(par >= 0, par + 3, 2)], 1)
    q, k, v = _kda_rows(s, _windows(before))
    up = (par[..., None] == torch.arange(R, device=DEV)).double()
    anc = torch.linalg.matrix_power(up + torch.eye(R, dtype=torch.float64, device=DEV), R) > 0.5   # ancestors and itself
    strict = (anc & ~torch.eye(R, dtype=torch.bool, device=DEV))[:, None]
    g = _kda_gate(s, s["z"])
    gam = (anc.double() @ g).reshape(B, R, H, D).transpose(1, 2)
    beta = 1 / (1 + torch.exp(-s["b"].float().transpose(1, 2)))
    S0 = s["S"][s["slots"].long()]
    uu, gap = _kda_solve(S0, k, v, gam, beta, strict)
    att = torch.where(anc[:, None], ((q[:, :, :, None] * k[:, :, None]) * gap).sum(-1), 0.0)
    o = (q * torch.exp(gam).float()) @ S0 + att @ uu
    o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + 1e-5) * s["norm_w"]
    o = o.transpose(1, 2).reshape(B, R, H * D) / (1 + torch.exp(-s["gout"].float()))
    return o.to(t)


def _plain_commit(s):
    c = s["case"]
    H, B, L = c["H"], c["sessions"], c["longest"]
    idx, lens, path = s["slots"].long(), s["path_len"].long(), s["path"].long().clamp(min=0)
    at = torch.arange(L, device=DEV)
    live = at[None] < lens[:, None]
    chosen = {k: torch.gather(s[k], 1, path[..., None].expand(B, L, s[k].shape[-1])) for k in ("q", "k", "v", "z", "b")}
    t = {**s, **chosen}
    before = torch.cat([torch.tensor([0, 0, 1], device=DEV).expand(B, 3), (at + 2).expand(B, L)], 1)
    _, k, v = _kda_rows(t, _windows(before))
    g = _kda_gate(s, t["z"]) * live[..., None]
    gam = g.cumsum(1).reshape(B, L, H, D).transpose(1, 2)
    beta = (live[..., None] / (1 + torch.exp(-t["b"].float()))).transpose(1, 2)
    S0 = s["S"][idx]
    strict = torch.ones(L, L, dtype=torch.bool, device=DEV).tril(-1)[None, None]
    uu, _ = _kda_solve(S0, k, v, gam, beta, strict)
    end = gam[:, :, -1]
    w = k * torch.exp(end[:, :, None] - gam).float()
    s["S_out"][idx] = torch.exp(end).float()[..., None] * S0 + w.transpose(-1, -2) @ uu
    raw = torch.cat([s["ring"][idx], torch.stack([t["q"], t["k"], t["v"]], 1)], 2)      # [B, 3, 3 + L, W]
    last = (lens[:, None] + torch.arange(3, device=DEV))[:, None, :, None].expand(B, 3, 3, H * D)
    s["ring_out"][idx] = torch.gather(raw, 2, last)
    return {"S": s["S_out"], "ring": s["ring_out"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "ssm_prefill":
        return _plain_prefill(state)
    if op == "ssm_decode":
        return _plain_decode(state)
    return _plain_tree(state) if op == "tree" else _plain_commit(state)


# ------------------------------------------------------- what a pass needs

def work(case):
    e, H = (2 if case["io"] == "bf16" else 4), case["H"]
    if case["op"] in ("ssm_prefill", "ssm_decode"):
        P, N, G = case["P"], case["N"], case["G"]
        W, C = H * P, H * P + 2 * G * N
        if case["op"] == "ssm_prefill":
            T, n, ins = case["tokens"], case["seqs"], 2 if case["state"] else 1
        else:
            T, n, ins = case["sessions"], case["sessions"], 2
        bytes_ = T * (C + H + W * (2 if case["gate"] else 1)) * e + n * ins * (H * N * P * 4 + 3 * C * e) + C * 20
        return {"bytes": bytes_, "flops": T * (H * N * P * 5 + C * 12)}
    W = H * D
    if case["op"] == "tree":
        rows, B = case["sessions"] * case["nodes"], case["sessions"]
        return {"bytes": B * (H * D * D * 4 + 9 * W * e) + rows * (6 * W + H) * e + rows * 4 + W * 52,
                "flops": rows * H * (4 * D * D + 60 * D)}
    rows, B = case["sessions"] * (case["longest"] + 1) // 2, case["sessions"]
    return {"bytes": B * (2 * H * D * D * 4 + 18 * W * e) + rows * (4 * W + H) * e + W * 52, "flops": rows * H * 7 * D * D}


# ------------------------------- the definitions, token by token in 64 bits

def _exact_prefill(case, s):
    H, P, N, G = case["H"], case["P"], case["N"], case["G"]
    W, lens = H * P, _lens(case)
    order = sorted(range(len(lens)), key=lambda i: -lens[i])           # longest first: the running ones are a prefix
    C = W + 2 * G * N
    zero = s["S_in"] is None
    S = torch.zeros(len(lens), H, N, P, dtype=torch.float64, device=DEV) if zero else s["S_in"].double()[order].clone()
    ring = torch.zeros(len(lens), 3, C, dtype=s["xbc"].dtype, device=DEV) if zero else s["ring_in"][order].clone()
    w, cb = s["conv_w"].double(), 0 if s["conv_b"] is None else s["conv_b"].double()
    A, bias, skip = -s["A_log"].double().exp(), s["dt_bias"].double(), s["D"].double()[:, None]
    start = torch.tensor([s["cu"][i] for i in order], device=DEV)
    out = torch.empty(case["tokens"], W, dtype=torch.float64, device=DEV)
    for i in range(max(lens)):
        m = sum(L > i for L in lens)
        at = start[:m] + i
        new = s["xbc"][at]
        a = (ring[:m].double() * w[:, :3].T).sum(1) + new.double() * w[:, 3] + cb
        a = a * torch.sigmoid(a)
        ring[:m] = torch.cat([ring[:m, 1:], new[:, None]], 1)
        x = a[:, :W].view(m, H, P)
        Bt = a[:, W:W + G * N].view(m, G, 1, N).expand(m, G, H // G, N).reshape(m, H, N)
        Ct = a[:, W + G * N:].view(m, G, 1, N).expand(m, G, H // G, N).reshape(m, H, N)
        dt = s["dt"][at].double() + bias
        dt = torch.clamp(dt, min=0) + torch.log1p(torch.exp(-dt.abs()))
        S[:m].mul_(torch.exp(A * dt)[..., None, None]).addcmul_((Bt * dt[..., None])[..., None], x[:, :, None])
        y = torch.matmul(Ct[:, :, None], S[:m])[:, :, 0] + skip * x
        out[at] = y.reshape(m, W)
    if s["z"] is not None:
        out *= s["z"].double() * torch.sigmoid(s["z"].double())
    back = [order.index(i) for i in range(len(lens))]
    return {"o": out, "S": S[back], "ring": ring[back]}


def _exact_decode(case, s):
    H, P, N, G, B = case["H"], case["P"], case["N"], case["G"], case["sessions"]
    W = H * P
    S, ring = s["S"].double(), s["ring"].clone()
    out = torch.empty(B, W, dtype=torch.float64, device=DEV)
    for i, slot in enumerate(s["slots"].tolist()):
        a = (torch.cat([ring[slot], s["xbc"][i:i + 1]]).double() * s["conv_w"].double().T).sum(0)
        a = a if s["conv_b"] is None else a + s["conv_b"].double()
        a = a * torch.sigmoid(a)
        dt = torch.log1p(torch.exp(s["dt"][i].double() + s["dt_bias"].double()))
        x = a[:W].view(H, P)
        Bt, Ct = a[W:].view(2, G, N).repeat_interleave(H // G, 1)
        S[slot] = S[slot] * torch.exp(-s["A_log"].double().exp() * dt)[:, None, None] + torch.einsum("h,hn,hp->hnp", dt, Bt, x)
        y = torch.einsum("hn,hnp->hp", Ct, S[slot]) + s["D"].double()[:, None] * x
        out[i] = y.reshape(W)
        ring[slot] = torch.cat([ring[slot, 1:], s["xbc"][i:i + 1]])
    if s["z"] is not None:
        out *= s["z"].double() * torch.sigmoid(s["z"].double())
    return {"o": out, "S": S, "ring": ring}


def _exact_step(s, S, rows, z, b):
    """One token on states S [B, H, 128, 128] from the raw rows [3 planes][B, 4, W]: the new states and the outputs before the norm."""
    B, H = S.shape[:2]
    q, k, v = ((r.double() * s["conv_w"][p].double().T).sum(1) for p, r in enumerate(rows))
    q, k, v = ((a * torch.sigmoid(a)).view(B, H, D) for a in (q, k, v))
    q = q * torch.rsqrt(q.square().sum(-1, keepdim=True) + 1e-6) / math.sqrt(D)
    k = k * torch.rsqrt(k.square().sum(-1, keepdim=True) + 1e-6)
    ea = s["A_log"].double().exp()[:, None]
    zb = (z.double() + s["dt_bias"].double()).view(B, H, D)
    g = -ea * torch.where(zb > 0, zb + torch.log1p(torch.exp(-zb.abs())), torch.log1p(torch.exp(-zb.abs()))) if s["case"]["softplus"] else -5.0 * torch.sigmoid(ea * zb)
    S = g.exp()[..., None] * S
    S = S + torch.sigmoid(b.double())[..., None, None] * k[..., None] * (v - (k[:, :, None] @ S)[:, :, 0])[:, :, None]
    return S, (q[:, :, None] @ S)[:, :, 0]


def _exact_tree(case, s):
    H, B, R = case["H"], case["sessions"], case["nodes"]
    idx, par = s["slots"].long(), s["parents"].long()
    each = torch.arange(B, device=DEV)
    states = torch.empty(B, R + 1, H, D, D, dtype=torch.float64, device=DEV)      # the last one: the session's own
    states[:, R] = s["S"][idx].double()
    rows = [torch.cat([s["ring"][idx][:, p], s[n]], 1) for p, n in enumerate(("q", "k", "v"))]
    o = torch.empty(B, R, H, D, dtype=torch.float64, device=DEV)
    for r in range(R):
        at = [torch.full((B,), 3 + r, device=DEV)]
        for _ in range(3):
            p = par[each, (at[-1] - 3).clamp(min=0)]
            at.append(torch.where(at[-1] >= 3, torch.where(p >= 0, p + 3, 2), (at[-1] - 1).clamp(min=0)))
        win = torch.stack(at[::-1], 1)
        S, y = _exact_step(s, states[each, par[:, r] % (R + 1)], [x[each[:, None], win] for x in rows], s["z"][:, r], s["b"][:, r])
        states[:, r] = S
        o[:, r] = y
    o = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + 1e-5) * s["norm_w"].double()
    return o.reshape(B, R, H * D) * torch.sigmoid(s["gout"].double())


def _exact_commit(case, s):
    idx, L = s["slots"].long(), case["longest"]
    S, ring = s["S"][idx].double(), s["ring"][idx].clone()
    each = torch.arange(case["sessions"], device=DEV)
    for i in range(L):
        on = (i < s["path_len"])
        node = s["path"][:, i].long().clamp(min=0)
        new = torch.stack([s[n][each, node] for n in ("q", "k", "v")], 1)[:, :, None]
        rows = torch.cat([ring, new], 2)
        S2, _ = _exact_step(s, S, [rows[:, p] for p in range(3)], s["z"][each, node], s["b"][each, node])
        S = torch.where(on[:, None, None, None], S2, S)
        ring = torch.where(on[:, None, None, None], rows[:, :, 1:], ring)
    out, rout = s["S"].double(), s["ring"].clone()
    out[idx], rout[idx] = S, ring
    return {"S": out, "ring": rout}


def exact(case, seed):
    s = prepare(case, seed)
    return {"ssm_prefill": _exact_prefill, "ssm_decode": _exact_decode, "tree": _exact_tree, "commit": _exact_commit}[case["op"]](case, s)
