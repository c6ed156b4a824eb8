"""The state space mixer token by token in 64 bits, and seeded inputs for it.

Tolerances of the tests that use this module (relative 2-norm over an output):
  fp32 outputs (o of fp32 I/O, every state): 2e-5, the sum of at most a few
    hundred fp32 roundings of 2^-24 each along one value's history;
  bf16 outputs: 2^-8 for the final rounding (half a step is 2^-8 of the value)
    plus 4 * 2^-11 for 11-bit operands of the tensor-core products.
"""
import math

import torch

TOL = {torch.float32: 2e-5, torch.bfloat16: 2 ** -8 + 4 * 2 ** -11}


def make_inputs(T, n, H, P, N, G, dtype, seed, state=True, bias=True, skip=True):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)
    ch = H * P + 2 * G * N
    step = torch.exp(torch.rand(H, generator=g) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
    return dict(
        H=H, P=P, N=N, G=G,
        xbc=rn(T, ch).to(dtype), dt=rn(T, H).to(dtype), z=rn(T, H * P).to(dtype),
        conv_w=rn(ch, 4) * 0.5, conv_b=rn(ch) * 0.1 if bias else None,
        A_log=torch.log(torch.rand(H, generator=g) * 15 + 1), dt_bias=step + torch.log(-torch.expm1(-step)),
        D=1 + 0.1 * rn(H) if skip else None,
        S=rn(n, H, N, P) * 0.3 if state else None, ring=rn(n, 3, ch).to(dtype) if state else None)


def softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def mixer(i, cu, gate=True):
    """(o [T][H*P], S [n][H][N][P], ring [n][3][ch]) in 64 bits (the ring in its own type)."""
    H, P, N, G = i["H"], i["P"], i["N"], i["G"]
    W, ch, n = H * P, H * P + 2 * G * N, len(cu) - 1
    grp = torch.arange(H) // (H // G)
    w = i["conv_w"].double()
    S = torch.zeros(n, H, N, P, dtype=torch.float64) if i["S"] is None else i["S"].double().clone()
    ring = torch.zeros(n, 3, ch, dtype=i["xbc"].dtype) if i["ring"] is None else i["ring"].clone()
    o = torch.zeros(cu[-1], W, dtype=torch.float64)
    for s in range(n):
        for t in range(cu[s], cu[s + 1]):
            rows = torch.cat([ring[s], i["xbc"][t:t + 1]])
            u = (rows.double() * w.T).sum(0)
            if i["conv_b"] is not None:
                u = u + i["conv_b"].double()
            u = u * torch.sigmoid(u)
            ring[s] = rows[1:]
            x = u[:W].view(H, P)
            B, C = u[W:W + G * N].view(G, N)[grp], u[W + G * N:].view(G, N)[grp]
            dt = softplus(i["dt"][t].double() + i["dt_bias"].double())
            a = torch.exp(-torch.exp(i["A_log"].double()) * dt)
            S[s] = a[:, None, None] * S[s] + (dt[:, None] * B)[:, :, None] * x[:, None, :]
            y = (C[:, :, None] * S[s]).sum(1)
            if i["D"] is not None:
                y = y + i["D"].double()[:, None] * x
            y = y.reshape(W)
            if gate:
                z = i["z"][t].double()
                y = y * z * torch.sigmoid(z)
            o[t] = y
    return o, S, ring


def close(name, got, want, tol=None):
    got = got.detach().cpu()
    tol = TOL[got.dtype] if tol is None else tol
    assert got.shape == want.shape, f"{name}: {tuple(got.shape)} != {tuple(want.shape)}"
    assert torch.isfinite(got).all(), f"{name}: non-finite values"
    if got.numel() == 0:
        return
    err = float((got.double() - want.double()).norm() / max(float(want.double().norm()), 1e-30))
    assert err <= tol, f"{name}: relative error {err:.3e} > {tol:.3e}"
