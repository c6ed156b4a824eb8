"""The gated linear recurrence token by token in 64 bits, its gradients by the
formulas, the verification of drafts in 64 bits, and seeded inputs for them.

Tolerances of the tests that use this module (relative 2-norm over an output):
  fp32 outputs: 2e-5, the sum of at most a few hundred fp32 roundings of 2^-24
    each along one value's history (300 * 2^-24 = 1.8e-5; the decays below
    forget within 100 tokens, and the errors with them);
  bf16 outputs: 2^-8 for the final rounding (half a step is 2^-8 of the value)
    plus the same 2e-5;
  parameter gradients: sums of up to T = 700 terms of either sign, each good to 2e-5.  A
    sum of T random terms is about T^-1/2 of the sum of their sizes, so its relative
    error is up to T^1/2 = 27 times theirs: 5.4e-4.
"""
import math

import torch

TOL = {torch.float32: 2e-5, torch.bfloat16: 2 ** -8 + 2e-5}
SUM_TOL = 5.4e-4


def make_inputs(T, n, C, dtype, seed, state=True, bias=True, gate=True):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)
    forget = torch.exp(torch.rand(C, generator=g) * math.log(50) + math.log(2))
    i = dict(C=C, x=rn(T, C).to(dtype), r=rn(T, C).to(dtype), i=rn(T, C).to(dtype), A_log=torch.log(2 / forget))
    z, rb, ib, S = rn(T, C).to(dtype), rn(C) * 0.5, rn(C) * 0.5, rn(n, C)
    i.update(z=z if gate else None, r_bias=rb if bias else None, i_bias=ib if bias else None, S=S if state else None)
    i.update(do=rn(T, C).to(dtype), dS=rn(n, C) if state else None)
    return i


def steps(i):
    """(w, v, la, a, m, b) of every token, in 64 bits; w_ and v_ are 1 - w and 1 - v."""
    r, s = i["r"].double(), i["i"].double()
    r = r if i["r_bias"] is None else r + i["r_bias"].double()
    s = s if i["i_bias"] is None else s + i["i_bias"].double()
    w, v = torch.sigmoid(r), torch.sigmoid(s)
    la = -torch.exp(i["A_log"].double()) * w
    m = torch.sqrt(-torch.expm1(2 * la))
    return dict(w=w, v=v, w_=torch.sigmoid(-r), v_=torch.sigmoid(-s), la=la, a=torch.exp(la), m=m, b=m * v * i["x"].double())


def states(i, cu):
    """(h before each token, h after it, the final states), in 64 bits."""
    n, C, T = len(cu) - 1, i["C"], cu[-1]
    s = steps(i)
    S = torch.zeros(n, C, dtype=torch.float64) if i["S"] is None else i["S"].double().clone()
    before, h = torch.empty(T, C, dtype=torch.float64), torch.empty(T, C, dtype=torch.float64)
    for k in range(n):
        for t in range(cu[k], cu[k + 1]):
            before[t] = S[k]
            S[k] = s["a"][t] * S[k] + s["b"][t]
            h[t] = S[k]
    return before, h, S


def mixer(i, cu):
    """(o [T][C], S [n][C]) in 64 bits."""
    _, h, S = states(i, cu)
    if i["z"] is not None:
        z = i["z"].double()
        h = h * z * torch.sigmoid(z)
    return h, S


def gradients(i, cu):
    """The gradients by the formulas, in 64 bits."""
    s = steps(i)
    before, h, _ = states(i, cu)
    n, T, C = len(cu) - 1, cu[-1], i["C"]
    G, out = i["do"].double(), {}
    if i["z"] is not None:
        z = i["z"].double()
        e = torch.sigmoid(z)
        out["dz"] = G * h * (e + z * e * torch.sigmoid(-z))
        G = G * z * e
    carry = torch.zeros(n, C, dtype=torch.float64) if i["dS"] is None else i["dS"].double().clone()
    g = torch.empty(T, C, dtype=torch.float64)
    for k in range(n):
        for t in range(cu[k + 1] - 1, cu[k] - 1, -1):
            g[t] = G[t] + carry[k]
            carry[k] = s["a"][t] * g[t]
    # m = (1 - a^2)^1/2: dm/dla = -a^2 / m, where m is zero nothing is left of it (la / m -> 0)
    la_m = torch.where(s["m"] > 0, s["la"] / s["m"].clamp(min=1e-300), torch.zeros_like(s["la"]))
    dA = g * (s["a"] * before * s["la"] - s["a"] ** 2 * s["v"] * i["x"].double() * la_m)
    out["dx"], out["di"], out["dr"] = g * s["m"] * s["v"], g * s["b"] * s["v_"], dA * s["w_"]
    out.update(dS_in=carry, dA_log=dA.sum(0), dr_bias=out["dr"].sum(0), di_bias=out["di"].sum(0))
    return out


def close(name, got, want, tol=None):
    got = got.detach().cpu()
    tol = TOL[got.dtype] if tol is None else tol
    assert got.shape == want.shape, f"{name}: {tuple(got.shape)} != {tuple(want.shape)}"
    assert torch.isfinite(got).all(), f"{name}: non-finite values"
    if got.numel() == 0:
        return
    err = float((got.double() - want.double()).norm() / max(float(want.double().norm()), 1e-30))
    assert err <= tol, f"{name}: relative error {err:.3e} > {tol:.3e}"


# ---- verification of drafts -------------------------------------------------------------

def verify(p, tokens, parents, u, u_next, q=None, p_last=None, q_last=None, max_len=None):
    """(paths, next tokens): the walk of one distribution after another in 64 bits, each refusal
    applied to what the target has left and normalised (not the one-coefficient form)."""
    n, R, V = p.shape
    max_len = R if max_len is None else max_len

    def clean(row):
        row = row.double().clone()
        row[~(torch.isfinite(row) & (row > 0))] = 0
        return row

    paths, nxt = [], []
    for s in range(n):
        row = lambda of, last, r: clean(of[s, r]) if r >= 0 else None if last is None else clean(last[s])
        cur, path, left, mass = -1, [], row(p, p_last, -1), 1.0
        go = True
        while go and len(path) < max_len:
            go = False
            for r in range(R):
                x = int(tokens[s, r])
                if int(parents[s, r]) != cur or not 0 <= x < V or r <= cur:
                    continue
                if left is None:
                    ok = True
                else:
                    if q is None:
                        draft = torch.zeros(V, dtype=torch.float64)
                        draft[x] = 1
                    else:
                        draft = row(q, q_last, cur)
                    have = float(left[x])
                    ok = have > 0 and float(u[s, r]) * mass * float(draft[x]) < have
                if ok:
                    cur, left, mass, go = r, row(p, p_last, r), 1.0, True
                    path.append(r)
                    break
                if q is None:
                    mass -= have
                    left[x] = 0
                else:
                    left = (left - mass * draft).clamp(min=0)
                    mass = float(left.sum())
        if left is None:
            nxt.append(-1)
        else:
            if not bool((left > 0).any()):
                left = row(p, p_last, cur)
            cum = left.cumsum(0)
            live = (left > 0).nonzero().flatten()
            over = ((cum > float(u_next[s]) * float(cum[-1])) & (left > 0)).nonzero().flatten()
            nxt.append(int(over[0]) if len(over) else int(live[-1]) if len(live) else -1)
        paths.append(path)
    return paths, nxt


def make_draft(n, R, V, dtype, seed, shape="bushy", drawn=True, last=True):
    """A round's probabilities, tokens, trees and random numbers."""
    g = torch.Generator().manual_seed(seed)
    rn, ru = (lambda *s: torch.randn(*s, generator=g)), (lambda *s: torch.rand(*s, generator=g))
    parents = torch.empty(n, R, dtype=torch.int32)
    root = -1 if last else 0
    for s in range(n):
        parents[s, 0] = -1
        for r in range(1, R):
            parents[s, r] = {"chain": r - 1, "star": root}.get(shape, int(torch.randint(max(root, r // 3 - 2), r, (1,), generator=g)))
    logits = rn(n, R + 1, V) * 2
    p, q = torch.softmax(logits, -1), torch.softmax(logits + 0.8 * rn(n, R + 1, V), -1)
    at = parents.long() + 1
    rows = q[torch.arange(n)[:, None], at]                                 # [n, R, V]: what each node was drawn from
    tokens = torch.multinomial(rows.view(n * R, V), 1, generator=g).view(n, R).to(torch.int32)
    d = dict(p=p[:, 1:].to(dtype).contiguous(), tokens=tokens, parents=parents, u=ru(n, R), u_next=ru(n),
             p_last=p[:, 0].to(dtype).contiguous() if last else None)
    d.update(q=q[:, 1:].to(dtype).contiguous() if drawn else None,
             q_last=q[:, 0].to(dtype).contiguous() if drawn and last else None)
    return d
