"""Sums of the verification of drafts (kda_draft_verify) that decide the next token: pieces of
a row whose parts are marked, products next to the target, long rows."""
import pytest
import torch

import gated_delta_rule_04_gb300 as kda
from glr_ref import verify

pytestmark = pytest.mark.gpu
DEV = "cuda"
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_04_gb300 import build as kbuild
    kbuild.build()
    kda.lib()


def dev(x):
    return x.to(DEV)


def one_row(row, n, off=0):
    """The row for n sessions (they share its memory), `off` elements behind a 256-byte boundary."""
    at = torch.zeros(row.numel() + off, dtype=row.dtype, device=DEV)
    at[off:] = row.to(DEV)
    return at[off:].expand(n, row.numel())


def draft(n, tokens, u):
    """n sessions of the same children of the last token."""
    R = len(tokens)
    return (torch.tensor(tokens, dtype=torch.int32, device=DEV).expand(n, R).contiguous(),
            torch.full((n, R), -1, dtype=torch.int32, device=DEV), torch.full((n, R), u, device=DEV))


@pytest.mark.parametrize("io, V, n", [("f32", 8961, 700), ("f32", 128257, 256), ("f32", 33793, 256), ("bf16", 32769, 256),
                                      ("bf16", 9729, 1300), ("bf16", 9735, 1300),
                                      ("f32", 16381, 700), ("bf16", 16381, 1300)])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("off", [0, 3])
def test_tokens_behind_the_last_whole_16_bytes(io, V, n, drawn, off):
    """Pieces whose whole steps end with a marked part and entries behind them (a part of their own), or in the middle of
    the last part: half of the rest lies on the row's last 7 tokens, the other half all over it.  One refused child."""
    g = torch.Generator().manual_seed(V + off)
    w = torch.rand(V, generator=g) + 0.1
    w[-7:] = 0
    p = w / w.sum() * 0.5
    p[-7:] = 0.5 / 7
    q = p * (0.5 + torch.rand(V, generator=g))
    q[-7:] *= 0.25
    p[11] = 0                                            # the child's token: refused
    p, q = p.to(IO[io]), q.to(IO[io])
    u_next = torch.rand(n, generator=g)
    u_next[:64] = 1 - torch.rand(64, generator=g) * 0.1
    tokens, parents, u = draft(n, [11], 0.5)
    rows = one_row(p, n, off)
    path, length, nxt = kda.kda_draft_verify(torch.zeros(1, 1, V, dtype=IO[io], device=DEV).expand(n, 1, V), tokens, parents, u,
                                             dev(u_next), p_last=rows,
                                             q=torch.zeros(1, 1, V, dtype=IO[io], device=DEV).expand(n, 1, V) if drawn else None,
                                             q_last=one_row(q, n, off) if drawn else None)
    W = (p.double() - q.double()).clamp(min=0) if drawn else p.double()
    cum = W.cumsum(0)
    goal = u_next.double() * cum[-1]
    want = torch.searchsorted(cum, goal, right=True)
    assert not length.any() and bool((path == -1).all())
    assert nxt.tolist() == want.tolist()
    assert len(set(want[want >= V - 7].tolist())) == 7


@pytest.mark.parametrize("V", [8, 5000])
@pytest.mark.parametrize("accept", [False, True])
def test_a_product_rounded_to_the_target(V, accept):
    """c q just below p, by less than half a step of fp32: what is left of that token is positive, 2^-25 of p or
    less, and all that is left after two refusals.  The next token is that one; a third child with it is accepted."""
    import random
    from fractions import Fraction as F
    rng = random.Random(V)
    f32 = lambda x: float(torch.tensor(float(x)))
    found = []
    while len(found) < 40:
        q = f32(rng.uniform(2 ** -6, 2 ** -5))
        p = q
        for _ in range(50):                              # p = c q rounded, where c = 1 + T and T = (5/4 - 1) + (p - q)
            c = 1 + F(1, 4) + F(p) - F(q)
            p = f32(c * F(q))
        c = 1 + F(1, 4) + F(p) - F(q)
        if p == f32(c * F(q)) and F(p) - c * F(q) > F(p) / 2 ** 36:
            found.append((p, q))
    n = len(found)
    P, Q = torch.zeros(n, V), torch.zeros(n, V)
    P[:, 1], Q[:, 1] = 1.25, 1.0                         # left of it after the first refusal: 1/4, after the second: nothing
    Q[:, 2], Q[:, 3] = 0.5, 0.25                         # the refused ones
    at = V - 2
    P[:, at], Q[:, at] = torch.tensor([x for x, _ in found]), torch.tensor([y for _, y in found])
    tokens, parents, u = draft(n, [2, 3, at] if accept else [2, 3], 0.9)
    R = tokens.shape[1]
    none = torch.zeros(n, R, V)
    none[:, :, 5] = 1.0
    u_next = torch.linspace(0, 0.99, n)
    path, length, nxt = kda.kda_draft_verify(dev(none), tokens, parents, u, dev(u_next), q=dev(none), p_last=dev(P), q_last=dev(Q))
    wp, wn = verify(none, tokens.cpu(), parents.cpu(), u.cpu(), u_next, q=none, p_last=P, q_last=Q)
    assert wp == ([[2]] * n if accept else [[]] * n) and wn == [5 if accept else at] * n
    assert length.tolist() == [len(w) for w in wp]
    assert nxt.tolist() == wn


@pytest.mark.parametrize("io, value", [("f32", 0.1), ("f32", 1e-5), ("bf16", 0.1)])
@pytest.mark.parametrize("V, n", [(1 << 22, 700), (1 << 24, 300), (1 << 24, 1)])
@pytest.mark.parametrize("off", [0, 1])
def test_even_rows(io, value, V, n, off):
    """Rows of one value: every sum is a multiple of it, and u_next times the whole is a whole number of entries, so
    the next token is u_next V exactly.

    A sum is a pair hi + lo of fp32.  Behind a lane's own sum (settled: |lo| is half a step U of hi at most) 32 lanes are
    joined in five additions: their lo and the additions' errors come to at most 1.5 U + 5 U / 2 = 4 U before the
    sum is settled, warps and CTAs to less.  A sum below 2^46 units of the value's last place has U <= 2^22 units, so
    lo stays within 2^24 of them and no addition rounds: with 24 bits for the value up to V = 2^22 the token is exact.
    Above, each of fewer than 24 additions rounds lo by 2^-24 4 U <= 2^-45 of the sum, together less than 2^-40 of it,
    where an entry is 2^-24 of it: u_next V is a border between two tokens, and either may follow."""
    row = torch.full((V,), value, dtype=IO[io])
    k = torch.arange(n) * 1021 % 1024 if n > 1 else torch.tensor([341])
    u_next = k.float() / 1024
    tokens = torch.zeros(n, 1, dtype=torch.int32, device=DEV)
    parents = torch.full((n, 1), -1, dtype=torch.int32, device=DEV)
    rows = one_row(row, n, off)
    nxt = kda.kda_draft_verify(rows[:, None], tokens, parents, torch.zeros(n, 1, device=DEV), dev(u_next))[2].cpu()
    want = k * (V // 1024)
    if V <= 1 << 22 or io == "bf16":                     # (bf16: 8 bits for the value)
        assert nxt.tolist() == want.tolist()
    else:
        assert bool(((nxt == want) | (nxt == (want - 1).clamp(min=0))).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("V, n, small", [(1 << 17, 8, 1e-13), (1 << 17, 200, 1e-13), (1 << 15, 700, 1e-12), (1 << 20, 3, 1e-14), (1 << 10, 30, 1e-16)])
def test_a_rest_beside_large_refused_tokens(io, V, n, small):
    """Chosen tokens that hold nearly all of the target are refused: the others have next to nothing each, all the same,
    so their sums are exact, and u_next times the whole is a whole number of them."""
    R = 6
    tokens = torch.tensor([0, 3, V // 2, V // 2 + 1, V + R - 2, V + R - 1])
    row = torch.full((V + R,), small, dtype=IO[io])
    row[tokens] = (torch.tensor([0.3, 0.2, 0.3, 0.1, 0.05, 0.04])).to(IO[io])
    t, parents, u = draft(n, tokens.tolist(), 1.0)   # (u T is at least what the target has)
    k = torch.arange(n) * 1021 % 1024
    nothing = torch.zeros(1, 1, V + R, dtype=IO[io], device=DEV).expand(n, R, V + R)
    path, length, nxt = kda.kda_draft_verify(nothing, t, parents, u, dev(k.float() / 1024), p_last=one_row(row, n))
    left = torch.ones(V + R)
    left[tokens] = 0
    want = torch.searchsorted(left.cumsum(0), (k * (V // 1024)).float(), right=True)
    assert not length.any()
    assert nxt.tolist() == want.tolist()
