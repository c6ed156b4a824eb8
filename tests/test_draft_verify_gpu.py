"""Verification of drafted tokens (kda_draft_verify) against the walk in 64 bits,
and a whole round: outputs, verification and commit."""
import pytest
import torch

import gated_delta_rule_04_gb300 as kda
from glr_ref import make_draft, verify

pytestmark = pytest.mark.gpu
DEV = "cuda"
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_04_gb300 import build as kbuild
    kbuild.build()
    kda.lib()


def dev(x):
    return None if x is None else x.to(DEV)


def run(d, **kw):
    on = {k: v.to(DEV) if torch.is_tensor(v) and v.device.type == "cpu" else v for k, v in d.items()}
    return kda.kda_draft_verify(on["p"], on["tokens"], on["parents"], on["u"], on["u_next"], q=on["q"], p_last=on["p_last"],
                                q_last=on["q_last"], **kw)


def check(d, max_len=None):
    path, length, nxt = run(d, max_len=max_len)
    wp, wn = verify(**d, max_len=max_len)
    m = d["p"].shape[1] if max_len is None else max_len
    assert path.shape == (d["p"].shape[0], m)
    assert length.tolist() == [len(p) for p in wp]
    assert path.tolist() == [p + [-1] * (m - len(p)) for p in wp]
    assert nxt.tolist() == wn
    return wp, wn


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", ["chain", "bushy", "star"])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("last", [True, False])
def test_shapes(io, shape, drawn, last):
    for V, n, R in ((50, 9, 12), (1000, 5, 7), (33, 4, 64), (7, 30, 1)):
        check(make_draft(n, R, V, IO[io], V + R, shape, drawn, last))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 3, 8, 31, 255, 256, 257, 1023, 4096, 4099, 20011, 70001])
def test_vocabularies(io, V):
    """From one token to many, odd sizes (rows off 16 bytes) among them."""
    check(make_draft(6, 5, V, IO[io], V, "bushy"))
    check(make_draft(3, 4, V, IO[io], V + 1, "chain", drawn=False, last=False))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 37, 160, 400, 1300])
def test_batches(io, n):
    check(make_draft(n, 4, 600, IO[io], n, "bushy"))


@pytest.mark.parametrize("max_len", [1, 2, 5, 64])
def test_longest_path(max_len):
    """The walk ends at max_len nodes, and the next token follows the last of them."""
    d = make_draft(12, 9, 40, torch.float32, 5, "chain")
    d["u"] *= 0.3
    wp, _ = check(d, max_len)
    assert max(map(len, wp)) == min(max_len, max(map(len, verify(**d)[0])))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("drawn", [True, False])
def test_many_refused_siblings(io, drawn):
    """A star of 64 children whose draws are unlikely ones, the same token more than once among them."""
    d = make_draft(10, 64, 300, IO[io], 6, "star", drawn)
    d["u"] = 0.7 + 0.3 * d["u"]
    d["tokens"][:, 10:20] = d["tokens"][:, :10]
    wp, _ = check(d)
    d["u"][:] = 0.999
    d["u"][:, -1] = 0.0
    check(d)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("drawn", [True, False])
def test_left_out_nodes(io, drawn):
    """Tokens outside the vocabulary and parents out of range leave a node, and those under it, out."""
    d = make_draft(14, 11, 60, IO[io], 7, "bushy", drawn)
    d["u"] *= 0.5
    d["tokens"][::2, 1], d["tokens"][1::3, 0], d["tokens"][3, 4] = -1, 60, 2 ** 31 - 1
    d["parents"][2, 3], d["parents"][4, 2], d["parents"][5, 6], d["parents"][6, 0] = 3, 10, -2, -5
    check(d)
    d["parents"][:] = -7                      # no tree at all
    assert all(p == [] for p in check(d)[0])
    d = make_draft(4, 3, 60, IO[io], 8, "chain", drawn, last=False)
    d["parents"][:, 0] = 5                    # not even the chosen token: nothing to follow
    assert check(d)[1] == [-1] * 4


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_rows_without_anything(io):
    """Zero, negative, NaN and infinite entries count as zero; an empty rest is the target itself, an empty target -1."""
    d = make_draft(12, 4, 90, IO[io], 9, "chain")
    d["p_last"][0] = 0                        # nothing to accept, nothing to draw
    d["p_last"][1, ::2] = float("nan")
    d["p_last"][2, 1::2] = float("inf")
    d["p_last"][3, :80] = -1.0
    d["q_last"][4] = float("nan")
    d["q_last"][5, ::3] = float("inf")
    d["p_last"][6] = d["q_last"][6] * 0.25    # all refused: the rest is empty
    d["u"][6] = 0.9
    d["p"][7, 0] = 0
    d["u"][7] = 0.0
    d["p_last"][8] = float("nan")
    d["p_last"][9] = -float("inf")
    d["p_last"][10] = 0
    d["p_last"][10, 89] = 1e-30
    d["q_last"][10] = 0
    wp, wn = check(d)
    assert wn[0] == wn[8] == wn[9] == -1 and wn[10] == 89


def test_random_numbers_at_the_ends():
    """0 takes the first entry above zero, the largest float below 1 one near the end, 1 and NaN the last above zero."""
    d = make_draft(8, 2, 500, torch.float32, 10, "chain")
    d["u"][:] = 1.0                           # refuse (but where the target gives more than the drafter)
    d["p_last"][:, :3] = 0
    d["p_last"][:, 495:] = 0
    d["u_next"] = torch.tensor([0.0, 1 - 2 ** -24, 1.0, float("nan"), 0.0, 2 ** -30, 5.0, 0.5])
    path, length, nxt = run(d)
    wp, wn = verify(**d)
    assert length.tolist() == [len(p) for p in wp] and nxt.tolist() == wn


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_strided_rows(io):
    """Rows of a padded vocabulary, sessions apart, one drafter's distribution for all; NaN in the padding."""
    d = make_draft(5, 4, 77, IO[io], 11, "bushy")
    want = run(d)
    nan = lambda *s: torch.full(s, float("nan"), dtype=IO[io], device=DEV)
    p, q, pl, ql = nan(5, 6, 83), nan(4, 5, 96), nan(5, 81), nan(5, 77)
    p[:, :4, :77], q[:, :, :77], pl[:, :77], ql[:] = dev(d["p"]), dev(d["q"]).transpose(0, 1), dev(d["p_last"]), dev(d["q_last"])
    got = run({**d, "p": p[:, :4, :77], "q": q[:, :, :77].transpose(0, 1), "p_last": pl[:, :77], "q_last": ql})
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    one = d["q"][:1, :1].expand(5, 4, 77)
    e = {**d, "q": one, "q_last": d["q"][0, :1].expand(5, 77)}
    got = kda.kda_draft_verify(dev(d["p"]), dev(d["tokens"]), dev(d["parents"]), dev(d["u"]), dev(d["u_next"]), p_last=dev(d["p_last"]),
                               q=dev(d["q"])[:1, :1].expand(5, 4, 77), q_last=dev(d["q"])[0, :1].expand(5, 77))
    wp, wn = verify(**e)
    assert got[1].tolist() == [len(x) for x in wp] and got[2].tolist() == wn


def test_given_outputs_streams_and_graphs():
    d = make_draft(20, 6, 5000, torch.bfloat16, 12, "bushy")
    on = {k: dev(v) for k, v in d.items()}
    want = run(on)
    out = dict(path=torch.full((20, 6), 9, dtype=torch.int32, device=DEV), path_len=torch.full((20,), 9, dtype=torch.int32, device=DEV),
               next_token=torch.full((20,), 9, dtype=torch.int32, device=DEV))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = run(on, **out, stream=side)
    torch.cuda.synchronize()
    assert all(a is b for a, b in zip(got, out.values()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = run(on)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(got, cap, want):
        assert torch.equal(a, c) and torch.equal(b, c)


def test_a_round_of_both_mixers():
    """A round as a server runs it: a draft of a straight run per session through a KDA layer and a
    gated linear recurrence, verification, and the commit of the accepted paths to both; the states equal those of
    the accepted tokens alone, decoded one after the other."""
    torch.manual_seed(0)
    n, R, H, C, V, bf = 6, 5, 2, 256, 97, torch.bfloat16
    rn = lambda *s: torch.randn(*s, device=DEV)
    kp = kda.make_params(rn(3, H * 128, 4) * 0.5, torch.log(torch.rand(H, device=DEV) * 15 + 1), rn(H * 128) * 0.7, 1 + 0.3 * rn(128))
    gp = kda.make_glr_params(rn(C) - 2, r_bias=rn(C), i_bias=rn(C))
    q, k, v, z, gout = (rn(n, R, H * 128).to(bf) for _ in range(5))
    b = rn(n, R, H).to(bf)
    x, r, i, gz = (rn(n, R, C).to(bf) for _ in range(4))
    S, ring, hS = rn(n, H, 128, 128) * 0.05, rn(n, 3, 3, H * 128).to(bf), rn(n, C)
    d = make_draft(n, R, V, torch.float32, 13, "chain", last=False)
    d["u"] *= 0.6
    on = {key: dev(val) for key, val in d.items()}
    keep = S.clone(), ring.clone(), hS.clone()
    rows = kda.kda_decode_tree(kp, q, k, v, z, b, gout, on["parents"], S, ring)
    hrows = kda.kda_glr_decode(gp, x, r, i, hS, z=gz, keep_state=True)
    assert torch.isfinite(rows).all() and torch.isfinite(hrows).all() and torch.equal(hS, keep[2])
    path, length, token = run(on)
    wp, wn = verify(**d)
    assert length.tolist() == [len(w) for w in wp] and token.tolist() == wn and len(set(length.tolist())) > 1
    kda.kda_tree_commit(kp, q, k, v, z, b, path, length, S, ring)
    kda.kda_glr_commit(gp, x, r, i, path, length, hS)
    for s in range(n):
        S1, r1, h1 = keep[0][s:s + 1].clone(), keep[1][s:s + 1].clone(), keep[2][s:s + 1].clone()
        for j in wp[s]:
            at = lambda t: t[s:s + 1, j].contiguous()
            o1 = kda.kda_decode(kp, at(q), at(k), at(v), at(z), at(b), at(gout), S1, r1)
            h = kda.kda_glr_decode(gp, *(at(t)[:, None] for t in (x, r, i)), h1, z=at(gz)[:, None])
            assert (o1.float() - rows[s:s + 1, j].float()).norm() <= 2e-2 * o1.float().norm()
            assert torch.equal(h[0, 0], hrows[s, j])
        assert (S[s] - S1[0]).norm() <= 1e-4 * S1.norm() and torch.equal(ring[s], r1[0])
        assert (hS[s] - h1[0]).norm() <= 2e-5 * h1.norm()


@pytest.mark.parametrize("V", [100, 5000, 40001])
def test_a_rest_lost_in_rounding(V):
    """Chosen tokens that hold all of the target but nothing or a trace, of very different sizes: what is left
    of the sums once they are refused is rounding.  The next token is the trace, or drawn from p itself."""
    g = torch.Generator().manual_seed(V)
    n, R = 60, 24
    d = make_draft(n, R, V, torch.float32, 21, "star", drawn=False)
    d["p_last"][:] = 0
    d["u"][:] = 1.0
    d["u_next"][::3] = 0
    for s in range(n):
        where = torch.randperm(V, generator=g)[:R + 1]
        d["tokens"][s] = where[:R]
        values = torch.rand(R, generator=g) * 2.0 ** -torch.arange(2, R + 2) * 2.0 ** -torch.randint(0, 20, (R,), generator=g)
        d["p_last"][s, where[:R]] = values[torch.randperm(R, generator=g)]
        if s % 2:
            d["p_last"][s, where[R]] = 1e-25
    wp, wn = check(d)
    assert all(p == [] for p in wp)
    assert all(d["p_last"][s, wn[s]] == torch.tensor(1e-25) for s in range(1, n, 2))


@pytest.mark.parametrize("io,V,n", [("bf16", 131072, 3), ("f32", 131071, 2), ("f32", 40001, 90), ("bf16", 32768, 160), ("bf16", 30011, 330)])
@pytest.mark.parametrize("drawn", [True, False])
def test_long_rows(io, V, n, drawn):
    """Several steps of copies a warp, pieces long enough to keep their parts' sums, in one CTA to 16; a
    few entries that count as zero among them."""
    d = make_draft(n, 3, V, IO[io], 22, "star" if drawn else "chain", drawn)
    d["u"] = 0.5 + 0.5 * d["u"]
    for t in ("p", "p_last", "q", "q_last"):
        if d[t] is not None:
            d[t][1, ..., 1000] = float("nan")
            d[t][1, ..., V - 2] = -1.0
    d["p_last"][0, 5] = float("inf")
    check(d)
