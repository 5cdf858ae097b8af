"""Tree verification and the commit of the accepted path, against the oracle.

Greedy results and moved columns are exact.  Sampled: p / q is a quotient of fp32 sums over V
scores, so its relative error is below 1e-5 at these sizes (a thread's pairwise sums, V / 512 terms
of 2^-24, and ex2's 2^-21); rows with a test or an edge of the draw nearer than 1e-4 are left out
of the comparison (there are few, which is asserted).
"""
import numpy as np
import pytest
import torch

import oracle.tree_oracle as TO
from tree_testlib import DEV, i32, numpy64, random_parents, status

pytestmark = pytest.mark.gpu


def outputs(B, D):
    return [torch.full(s, -7, dtype=torch.int32, device=DEV) for s in ((B,), (B,), (B, D), (B, D))]


def strided(x, stride, shift=0):
    B, T, V = x.shape
    buf = torch.zeros(B * T * stride + shift, dtype=x.dtype, device=DEV)
    y = buf[shift:].view(B, T, stride)[:, :, :V]
    y.copy_(x)
    return y


def greedy_inputs(rng, B, T, V, dtype, alpha=0.8, unused=0.1):
    par = random_parents(rng, B, T, unused)
    tok = rng.integers(0, V, (B, T))
    z = torch.as_tensor(rng.normal(size=(B, T, V)), dtype=torch.float32)
    for b in range(B):
        for t in range(T):
            kids = TO.children(par[b], t)
            if kids and rng.random() < alpha:
                z[b, t, tok[b, kids[int(rng.integers(len(kids)))]]] = 9.0
    return z.to(dtype), tok, par


def run_greedy(z, tok, par, D):
    import speculative_decoding_specdec_gb300.specdec as sd
    out, st = outputs(z.shape[0], D), status()
    sd.verify_tree_greedy(z, i32(tok), None if par is None else i32(par), *out, st)
    torch.cuda.synchronize()
    return [o.cpu().numpy() for o in out], int(st)


def same_walk(got, b, path, token, tok, D):
    a, y, p, d = (x[b] for x in got)
    assert a == len(path) and y == token, (a, y, path, token)
    assert p.tolist() == path + [-1] * (D - len(path))
    assert d.tolist() == [int(tok[i]) for i in path] + [0] * (D - len(path))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,V,D,stride,shift", [
    (2, 7, 1000, 3, 1000, 0), (8, 16, 32000, 5, 32000, 0), (3, 64, 5003, 8, 5003, 0),
    (4, 9, 777, 8, 779, 1), (2, 1, 50, 1, 50, 0), (5, 12, 1, 4, 1, 0), (3, 6, 7, 31, 16, 3),
    (40, 10, 4000, 6, 4008, 0), (2, 5, 151936, 4, 151936, 0)])
def test_greedy(dtype, B, T, V, D, stride, shift):
    rng = np.random.default_rng(V + T)
    z, tok, par = greedy_inputs(rng, B, T, V, dtype)
    got, st = run_greedy(strided(z, stride, shift), tok, par, D)
    assert st == 0
    zz = numpy64(z)
    for b in range(B):
        same_walk(got, b, *TO.verify_greedy(zz[b], tok[b], par[b], D), tok[b], D)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_greedy_chain_ties_and_strange_scores(dtype):
    import speculative_decoding_specdec_gb300.specdec as sd
    rng = np.random.default_rng(0)
    B, T, V = 6, 5, 3000
    z = torch.as_tensor(rng.integers(-3, 4, (B, T, V)), dtype=torch.float32)   # ties everywhere
    z[1, :, :2000] = float("nan")
    z[2] = -float("inf")                                                      # the first index wins
    z[3, 0, 70] = z[3, 0, 2900] = float("inf")
    z[4, 1] = float("nan")
    tok = np.zeros((B, T), np.int64)
    for b in range(B):
        for j in range(1, T):
            c = TO.greedy_choice(numpy64(z.to(dtype))[b, j - 1])
            tok[b, j] = 0 if c is None else c
    tok[5, 2], tok[0, 4] = V + 5, -1                                          # never a match
    got, st = run_greedy(z.to(dtype).to(DEV), tok, None, T - 1)
    assert st == sd.ERR_INPUT_RANGE                                           # row 4 has nothing but NaN
    for b in range(B):
        path, token = TO.verify_greedy(numpy64(z.to(dtype))[b], tok[b], TO.chain(T), T - 1)
        same_walk(got, b, path, -1 if token is None else token, tok[b], T - 1)


def test_first_matching_sibling_and_bad_trees():
    import speculative_decoding_specdec_gb300.specdec as sd
    z = torch.zeros(3, 5, 8)
    z[:, 0, 3] = z[:, 1, 5] = z[:, 2, 6] = 1
    tok = np.array([[0, 3, 3, 6, 5]] * 3)
    par = np.array([[-1, 0, 0, 2, 1], [-1, 0, 2, 0, 0], [-2] * 5])
    got, st = run_greedy(z.to(DEV), tok, par, 4)
    assert st == sd.ERR_INPUT_RANGE
    same_walk(got, 0, [1, 4], 0, tok[0], 4)
    assert all((g[1] == -7).all() for g in got)          # not written
    same_walk(got, 2, [], -1, tok[2], 4)


# ---------------------------------------------------------------------------------------- sampled

def sample_inputs(rng, B, T, V, temperature, replacement, dtype, unused=0.1):
    par = random_parents(rng, B, T, unused)
    z = rng.normal(size=(B, T, V)) * 1.5
    for b in range(B):
        for t in range(T):
            hot = rng.integers(0, V, 6)
            z[b, t, hot] = np.log(V) - 0.7 * np.arange(6)
    z = torch.as_tensor(z, dtype=torch.float32).to(dtype)
    w = (z.float() + 0.5 * torch.as_tensor(rng.normal(size=(B, T, V)), dtype=torch.float32)).to(dtype)
    tok = rng.integers(0, V, (B, T))
    wn = numpy64(w)
    for b in range(B):
        for t in range(T):
            kids = TO.children(par[b], t)
            if kids:
                q = TO.softmax(wn[b, t] / temperature)
                k = min(len(kids), V) if not replacement else len(kids)
                got = rng.choice(V, k, p=q, replace=replacement)
                tok[b, kids[:k]] = got
    return z, w, tok, par, rng.random((B, T)).astype(np.float32)


def run_sample(z, w, tok, par, u, temperature, D, replacement):
    import speculative_decoding_specdec_gb300.specdec as sd
    out, st = outputs(z.shape[0], D), status()
    sd.verify_tree_sample(z, w, i32(tok), None if par is None else i32(par),
                          torch.as_tensor(u, dtype=torch.float32).to(DEV), temperature, *out, st,
                          replacement=replacement)
    torch.cuda.synchronize()
    return [o.cpu().numpy() for o in out], int(st)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("replacement", [False, True])
@pytest.mark.parametrize("B,T,V,D,temperature,stride,shift", [
    (2, 7, 1000, 3, 1.0, 1000, 0), (6, 16, 32000, 5, 0.7, 32000, 0), (5, 12, 777, 31, 1.3, 779, 1),
    (24, 10, 501, 3, 0.5, 501, 0), (3, 1, 60, 1, 1.0, 60, 0), (6, 5, 3, 4, 1.0, 8, 0),
    (2, 40, 2000, 8, 0.9, 2000, 0), (2, 4, 151552, 3, 0.7, 151552, 0)])
def test_sampled(dtype, replacement, B, T, V, D, temperature, stride, shift):
    rng = np.random.default_rng(V + T + replacement)
    z, w, tok, par, u = sample_inputs(rng, B, T, V, temperature, replacement, dtype)
    got, st = run_sample(strided(z, stride, shift), strided(w, stride, shift), tok, par, u, temperature, D, replacement)
    assert st == 0
    near, zz, ww = 0, numpy64(z), numpy64(w)
    for b in range(B):
        path, token, p, margins = TO.verify_sample(zz[b], ww[b], tok[b], par[b], u[b].astype(np.float64), temperature, D, replacement)
        if margins and min(margins) < 1e-4:
            near += 1
            continue
        edges = np.cumsum(p)
        if np.abs(edges / edges[-1] - u[b, 0]).min() < 1e-4:   # an edge near: the walk alone, and a neighbour
            assert got[0][b] == len(path) and got[2][b].tolist()[:len(path)] == path
            y = int(got[1][b])
            lo, hi = sorted((y, token))
            assert p[y] > 0 and edges[hi] - edges[lo] - p[hi] < 2e-4
            continue
        same_walk(got, b, path, token, tok[b], D)
    assert near <= max(1, B // 8)


@pytest.mark.parametrize("replacement", [False, True])
def test_sampled_zero_probabilities(replacement):
    """-inf scores are tokens of probability zero: p(x) = 0 rejects, q(x) = 0 < p(x) accepts, and
    an empty residual leaves p."""
    V, inf = 40, float("inf")
    z = torch.zeros(4, 3, V)
    w = torch.zeros(4, 3, V)
    z[0, 0, 5] = -inf                        # the target cannot emit the first child
    w[1, 0, 5] = -inf                        # the draft model could not have drawn it
    z[2, 0, :39] = -inf                      # one token left
    tok = np.array([[0, 5, 6]] * 4)
    par = np.array([[-1, 0, 0]] * 4)
    u = np.full((4, 3), 0.999, np.float32)
    u[:, 0] = 0.5
    got, st = run_sample(z.to(DEV), w.to(DEV), tok, par, u, 1.0, 2, replacement)
    assert st == 0
    zz, ww = numpy64(z), numpy64(w)
    for b in (0, 1, 2):
        path, token, _, _ = TO.verify_sample(zz[b], ww[b], tok[b], par[b], u[b], 1.0, 2, replacement)
        same_walk(got, b, path, token, tok[b], 2)
    assert got[0][1] == 1 and got[1][2] == 39


def test_sampled_errors():
    import speculative_decoding_specdec_gb300.specdec as sd
    z = torch.randn(5, 2, 50)
    z[1, 0, 7] = float("nan")
    z[2, 0] = -float("inf")
    tok, par = np.array([[0, 3]] * 5), np.array([[-1, 0]] * 5)
    tok[3, 1] = 50                           # rejected without a test
    u = np.full((5, 2), 0.5, np.float32)
    u[4, 1] = 1.0
    got, st = run_sample(z.to(DEV), torch.randn(5, 2, 50).to(DEV), tok, par, u, 1.0, 1, False)
    assert st == sd.ERR_INPUT_RANGE
    assert got[1][1] == -1 and got[1][2] == -1 and (got[0][[1, 2, 3]] == 0).all()
    path, token, _, _ = TO.verify_sample(numpy64(z)[3], numpy64(z)[3], tok[3], par[3], u[3], 1.0, 0, False)
    assert got[1][3] == token
    assert all((g[4] == -7).all() for g in got)


def test_sampled_frequencies():
    """Many rows of one small tree whose tokens are drawn from q: the first committed token has the
    target's distribution (chi-square over 8 tokens; 30 is its 1 - 1e-4 quantile with 7 degrees)."""
    rng = np.random.default_rng(9)
    V, B = 8, 20000
    z, w = rng.normal(size=V), rng.normal(size=V)
    p, q = TO.softmax(z), TO.softmax(w)
    for replacement in (False, True):
        keys = rng.exponential(size=(B, V)) / q
        kids = rng.choice(V, (B, 2), p=q) if replacement else np.argsort(keys, 1)[:, :2]
        tok = np.concatenate([np.zeros((B, 1), int), kids], 1)
        zz = torch.as_tensor(z, dtype=torch.float32).expand(B, 3, V).contiguous().to(DEV)
        ww = torch.as_tensor(w, dtype=torch.float32).expand(B, 3, V).contiguous().to(DEV)
        got, st = run_sample(zz, ww, tok, np.array([[-1, 0, 0]] * B), rng.random((B, 3)).astype(np.float32), 1.0, 2, replacement)
        assert st == 0
        first = np.where(got[0] > 0, got[3][:, 0], got[1])
        seen = np.bincount(first, minlength=V)
        assert ((seen - B * p) ** 2 / (B * p)).sum() < 30


def test_verification_refusals():
    import speculative_decoding_specdec_gb300.specdec as sd
    z, tok, par, st = torch.zeros(1, 3, 10, device=DEV), i32([[0, 1, 2]]), i32([[-1, 0, 0]]), status()
    u = torch.zeros(1, 3, device=DEV)
    out = outputs(1, 2)
    bad = [dict(tok=i32([[0, 1]])), dict(par=i32([[0]])), dict(z=z[:, :, ::2]), dict(z=z.half()), dict(out=outputs(2, 2)),
           dict(out=outputs(1, 32)), dict(z=torch.zeros(1, 65, 4, device=DEV), tok=i32(np.zeros((1, 65))), par=None, u=torch.zeros(1, 65, device=DEV))]
    for kw in bad:
        a = dict(z=z, tok=tok, par=par, u=u, out=out) | kw
        with pytest.raises((sd.SpecdecError, ValueError)):
            sd.verify_tree_greedy(a["z"], a["tok"], a["par"], *a["out"], st)
        with pytest.raises((sd.SpecdecError, ValueError)):
            sd.verify_tree_sample(a["z"], a["z"], a["tok"], a["par"], a["u"], 1.0, *a["out"], st)
    for t in (0.0, -1.0, float("inf"), float("nan")):
        with pytest.raises(sd.SpecdecError):
            sd.verify_tree_sample(z, z, tok, par, u, t, *out, st)
    with pytest.raises(ValueError):
        sd.verify_tree_sample(z, z, tok, par, u[:, :2], 1.0, *out, st)
    with pytest.raises(ValueError):
        sd.verify_tree_sample(z, z.bfloat16(), tok, par, u, 1.0, *out, st)
    torch.cuda.synchronize()
    assert int(st) == 0


# ----------------------------------------------------------------------------------------- commit

def paths(rng, B, T, D, amax):
    a = rng.integers(0, min(amax, T - 1, D) + 1, B)
    p = np.full((B, D), -1)
    for b in range(B):
        p[b, :a[b]] = np.sort(rng.choice(np.arange(1, T), a[b], replace=False))
    return a, p


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("L,B,H,hd,T,D", [(1, 2, 2, 64, 7, 3), (3, 5, 3, 128, 64, 31), (2, 1, 1, 8, 2, 1), (2, 17, 2, 96, 20, 12)])
def test_commit(dtype, L, B, H, hd, T, D):
    import speculative_decoding_specdec_gb300.specdec as sd
    rng = np.random.default_rng(T + D)
    W = 11
    src = torch.randn(L, 2, B, H, W + T, hd, device=DEV).to(dtype)
    dst = torch.randn(L, 2, B, H, W + T + 5, hd, device=DEV).to(dtype)
    a, p = paths(rng, B, T, D, D)
    before, kept = numpy64(src), numpy64(dst)
    Wd, st = W + int(a.max()) + 1, status()
    sd.tree_commit(src, dst, i32([W]), i32(a), i32(p), st, width_dst=i32([Wd]), nodes=T)
    want = kept.copy()
    for b in range(B):
        for i in range(a[b]):
            want[:, :, b, :, Wd - 1 - a[b] + i] = before[:, :, b, :, W - 1 + p[b, i]]
    np.testing.assert_array_equal(numpy64(dst), want)
    np.testing.assert_array_equal(numpy64(src), before)
    sd.tree_commit(src, src, i32([W]), i32(a), i32(p), st, nodes=T)       # in place, overlapping
    want = before.copy()
    for b in range(B):
        for i in range(a[b]):
            want[:, :, b, :, W + i] = before[:, :, b, :, W - 1 + p[b, i]]
    np.testing.assert_array_equal(numpy64(src), want)
    assert int(st) == 0


def test_commit_in_an_arena():
    import speculative_decoding_specdec_gb300.specdec as sd
    rng = np.random.default_rng(1)
    S, T, D, H, hd = 5, 12, 6, 2, 64
    lens = rng.integers(1, 30, S)
    first = np.r_[0, np.cumsum(lens + T)][:S]
    arena = torch.randn(2, 2, 1, H, int(first[-1] + lens[-1] + T), hd, device=DEV)
    rows = np.array([3, 0, 4])
    a, p = paths(rng, 3, T, D, D)
    want, st = numpy64(arena), status()
    old = want.copy()
    sd.tree_commit(arena, arena, None, i32(a), i32(p), st, nodes=T, n_committed=i32(lens), rows=i32(rows), first_col=i32(first))
    for b, s in enumerate(rows):
        for i in range(a[b]):
            want[:, :, 0, :, first[s] + lens[s] + i] = old[:, :, 0, :, first[s] + lens[s] - 1 + p[b, i]]
    np.testing.assert_array_equal(numpy64(arena), want)
    assert int(st) == 0


@pytest.mark.parametrize("a,p,W,code", [
    (3, [1, 2], 5, "ERR_INPUT_RANGE"), (-1, [1, 2], 5, "ERR_INPUT_RANGE"), (2, [2, 2], 5, "ERR_INPUT_RANGE"),
    (2, [0, 2], 5, "ERR_INPUT_RANGE"), (2, [1, 6], 5, "ERR_INPUT_RANGE"), (1, [1, 0], 0, "ERR_INPUT_RANGE"),
    (2, [1, 5], 6, "ERR_CAPACITY")])
def test_commit_errors(a, p, W, code):
    import speculative_decoding_specdec_gb300.specdec as sd
    c = torch.randn(1, 2, 1, 1, 10, 8, device=DEV)
    before, st = c.clone(), status()
    sd.tree_commit(c, c, i32([W]), i32([a]), i32([p]), st, nodes=6)
    torch.cuda.synchronize()
    assert int(st) == getattr(sd, code) and (c == before).all()


def test_commit_refusals():
    import speculative_decoding_specdec_gb300.specdec as sd
    c, d, w, st = torch.zeros(1, 2, 1, 1, 10, 8, device=DEV), torch.zeros(1, 2, 1, 1, 10, 16, device=DEV), i32([3]), status()
    for args, kw in (((c, d, w), {}), ((c, c, None), {}), ((c, c, w), dict(width_dst=w)), ((c, c, w), dict(nodes=65)),
                     ((c, c, w), dict(nodes=0)), ((c, c, w), dict(rows=i32([0]))), ((c, c, w), dict(first_col=w)),
                     ((c, c[:, :, :, :, 1:], w), {})):
        with pytest.raises((sd.SpecdecError, ValueError, AttributeError)):
            sd.tree_commit(*args, i32([1]), i32([[2, 0]]), st, **kw)
    torch.cuda.synchronize()
    assert int(st) == 0
