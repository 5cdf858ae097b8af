"""The tree operators at the edges of what their callers may pass, against the oracle.

Comparisons are exact (copies, zeros, whole numbers, results that must not depend on what is hidden)
or take the bounds that are derived in the operator's own test file.
"""
import numpy as np
import pytest
import torch

import oracle.tree_oracle as TO
import test_gpu_rotary as R
import test_gpu_tree_attention as A
import test_gpu_tree_verify as V
from tree_testlib import DEV, i32, numpy64, random_parents, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("position", [-1, -2 ** 31, 40, 2 ** 31 - 1])   # (the table has 40)
@pytest.mark.parametrize("hd,rot,interleaved", [(64, 64, False), (80, 20, True)])
def test_a_padding_tokens_position_does_not_matter(dtype, in_place, position, hd, rot, interleaved):
    """A token with a negative column is padding whatever its position says: q_out is zero, nothing
    is written to the cache and no error recorded."""
    import speculative_decoding_specdec_gb300.specdec as sd
    gen = torch.Generator().manual_seed(1)
    B, T, H = 2, 6, 2
    q, k, v = (torch.randn(B, T, H, hd, generator=gen).to(dtype).to(DEV) for _ in range(3))
    cache = torch.randn(1, 2, B, H, 9, hd, generator=gen).to(dtype).to(DEV)
    pos = np.tile(np.arange(T), (B, 1))
    col = pos + 2
    for b, t, c in ((0, 0, -1), (0, 1, -5), (1, 5, -2 ** 31)):
        pos[b, t], col[b, t] = position, c
    q0, want, table, st = numpy64(q), numpy64(cache), R.make_table(40, rot), status()
    out = q if in_place else torch.full_like(q, 7.0)
    sd.rotary_append(q, k, v, cache, 0, table, out, st, positions=i32(pos), columns=i32(col), interleaved=interleaved)
    torch.cuda.synchronize()
    assert int(st) == 0
    got, cs = numpy64(cache), numpy64(table)
    for b in range(B):
        for t in range(T):
            if col[b, t] < 0:
                assert (out[b, t] == 0).all()
                continue
            c, s = cs[pos[b, t], :, 0], cs[pos[b, t], :, 1]
            R.close(numpy64(out[b, t]), TO.rotate(q0[b, t], c, s, interleaved), q0[b, t], dtype)
            R.close(got[0, 0, b, :, col[b, t]], TO.rotate(numpy64(k[b, t]), c, s, interleaved), numpy64(k[b, t]), dtype)
            want[0, 0, b, :, col[b, t]] = got[0, 0, b, :, col[b, t]]
            want[0, 1, b, :, col[b, t]] = numpy64(v[b, t])
    np.testing.assert_array_equal(got, want)


# Query rows per K/V head for every kernel and place a row's result is written from: (T, G, hd, the
# committed columns of a unit that share borders cut, or of one that they do not)
SHAPES = [(5, 2, 64), (12, 2, 128), (20, 5, 64), (16, 8, 128), (25, 8, 128), (50, 8, 64)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,G,hd", SHAPES + [(6, 2, 80), (10, 4, 256)])
@pytest.mark.parametrize("n", [[40, 9, 150], [5000]])
@pytest.mark.parametrize("where", ["q", "k", "v"])
def test_unused_nodes_give_zeros_whatever_there_is(dtype, T, G, hd, n, where):
    """Zeros (lse: -infinity) for unused nodes, also where their q is NaN or infinite or a committed
    column is, and no trace of that q in any other row."""
    rng = np.random.default_rng(T * G + hd)
    B, H, n = len(n), 2 if len(n) > 1 else 1, np.array(n)
    q, cache, W = A.inputs(rng, B, T, H * G, H, hd, n, dtype)
    par = random_parents(rng, B, T, unused=0.3)
    par[:, T - 1] = -2
    if B > 1:
        par[1] = -2
    A.hide(cache, n, W, T, par)
    unused, clean, held = par == -2, q.clone(), cache.clone()
    for b in range(B):
        for j, t in enumerate(np.flatnonzero(unused[b])):
            if where == "q":
                q[b, t] = (float("nan"), float("inf"), -float("inf"))[j % 3]
        if where != "q":
            cache[1, 0 if where == "k" else 1, b, :, W - 2, 3] = float("nan")
    out, lse, st = A.run(q, cache, 1, n, W, par)
    assert st == 0
    assert (out[unused] == 0).all() and np.isneginf(lse[unused]).all()
    if where == "q":
        A.check(out, lse, clean, held, 1, n, W, par)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,G,hd", SHAPES)
@pytest.mark.parametrize("n", [[40, 9, 150], [5000]])
@pytest.mark.parametrize("value", ["inf", "-inf", "nan"])
def test_a_value_that_is_not_finite_stays_in_its_dimension(dtype, T, G, hd, n, value):
    """V of a node is not finite in some of the head's values: nodes that see it are not finite in
    those, and everything else (lse, which V does not enter, too) is what it was."""
    rng = np.random.default_rng(T * G + hd + 1)
    B, H, n = len(n), 2 if len(n) > 1 else 1, np.array(n)
    q, cache, W = A.inputs(rng, B, T, H * G, H, hd, n, dtype)
    par = random_parents(rng, B, T, deep=0.5)
    clean, lse0, _ = A.run(q, cache, 1, n, W, par)
    nodes, dims = (T // 2, T - 1), (0, 3, hd - 1)
    for node in nodes:
        for d in dims:
            cache[1, 1, :, :, W - 1 + node, d] = float(value)
    out, lse, st = A.run(q, cache, 1, n, W, par)
    assert st == 0
    np.testing.assert_array_equal(lse, lse0)
    rest = [d for d in range(hd) if d not in dims]
    np.testing.assert_array_equal(out[..., rest], clean[..., rest])
    for b in range(B):
        for t in range(T):
            if set(nodes) & set(TO.line_of(par[b], t)):
                assert not np.isfinite(out[b, t][:, dims]).any()
            else:
                np.testing.assert_array_equal(out[b, t], clean[b, t])


def test_rotary_into_one_cache_row():
    """Rows of an arena (one cache row): columns that are given are taken, a verification pass, whose
    nodes would all go to the same columns, is refused."""
    import speculative_decoding_specdec_gb300.specdec as sd
    gen = torch.Generator().manual_seed(2)
    B, T, H, hd = 3, 4, 2, 64
    q, k, v = (torch.randn(B, T, H, hd, generator=gen).to(DEV) for _ in range(3))
    cache, table, st = torch.zeros(1, 2, 1, H, 30, hd, device=DEV), R.make_table(20, hd), status()
    pos, col = np.tile(np.arange(T), (B, 1)), np.array([[20, 21, 22, 23], [3, 4, 5, 6], [10, 11, 12, 13]])
    out = torch.empty_like(q)
    sd.rotary_append(q, k, v, cache, 0, table, out, st, positions=i32(pos), columns=i32(col))
    want, cs = np.zeros((H, 30, hd)), numpy64(table)
    for b in range(B):
        want[:, col[b]] = numpy64(v)[b].transpose(1, 0, 2)
        for t in range(T):
            R.close(numpy64(cache)[0, 0, 0, :, col[b, t]], TO.rotate(numpy64(k)[b, t], cs[t, :, 0], cs[t, :, 1], False), numpy64(k)[b, t], torch.float32)
    np.testing.assert_array_equal(numpy64(cache)[0, 1, 0], want)
    before = cache.clone()
    with pytest.raises(sd.SpecdecError):
        sd.rotary_append(q, k, v, cache, 0, table, out, st, n_committed=i32([2, 2, 2]), width=i32([2]))
    torch.cuda.synchronize()
    assert int(st) == 0 and torch.equal(cache, before)


def test_slots_columns_and_lengths_go_together():
    """Without ``rows`` there is a length and a first column per batch row, with it one of each per
    slot: tensors that are too short are refused, not read behind their end."""
    import speculative_decoding_specdec_gb300.specdec as sd
    q = torch.zeros(3, 2, 2, 64, device=DEV)
    arena = torch.zeros(1, 2, 1, 2, 40, 64, device=DEV)
    st, ws = status(), torch.zeros(sd.tree_attention_workspace_bytes(q, arena), dtype=torch.uint8, device=DEV)
    n3, c3, n5, c5, rows = i32([2, 2, 2]), i32([0, 10, 20]), i32([2] * 5), i32([0, 6, 12, 18, 24]), i32([4, 0, 2])
    def attend(n, first, rows=None):
        sd.tree_attention(q, arena, 0, torch.empty_like(q), n, None, None, st, ws, first_col=first, rows=rows)
    def commit(n, first, rows=None):
        sd.tree_commit(arena, arena, None, i32([1, 0, 1]), i32([[1], [-1], [1]]), st, nodes=2, n_committed=n, first_col=first, rows=rows)
    for call in (attend, commit):
        call(n3, c3)
        call(n5, c5, rows)
        call(n3, c5)
        for bad in ((n3, c3[:2]), (n3[:2], c3), (n3[:1], c3[:1]), (n5, c3, rows)):
            with pytest.raises(ValueError):
                call(*bad)
    torch.cuda.synchronize()
    assert int(st) == 0


@pytest.mark.parametrize("W", [2 ** 31 - 1, 2 ** 31 - 3, 12])
@pytest.mark.parametrize("tree", [False, True])
def test_rotary_at_a_width_beyond_the_cache(W, tree):
    """Columns W - 1 + t that the cache does not have, the largest integers among them: reported, and
    nothing is written for those nodes."""
    import speculative_decoding_specdec_gb300.specdec as sd
    gen = torch.Generator().manual_seed(6)
    B, T, H, hd, cap = 2, 5, 2, 64, 14
    q, k, v = (torch.randn(B, T, H, hd, generator=gen).to(DEV) for _ in range(3))
    cache = torch.randn(1, 2, B, H, cap, hd, generator=gen).to(DEV)
    want, table, st = cache.clone(), R.make_table(30, hd), status()
    out = torch.full_like(q, 7.0)
    par = None if not tree else i32([[-1, 0, 0, 1, 3]] * B)
    sd.rotary_append(q, k, v, cache, 0, table, out, st, n_committed=i32([3, 12]), width=i32([W]), parents=par)
    torch.cuda.synchronize()
    assert int(st) == sd.ERR_CAPACITY
    fit = max(0, min(T, cap + 1 - W))
    assert torch.equal(cache[..., :11, :], want[..., :11, :]) and (fit > 0 or torch.equal(cache, want))
    if fit:
        assert torch.equal(cache[0, 1, :, :, W - 1:W - 1 + fit], v[:, :fit].transpose(1, 2))
    assert (out[:, fit:] == 7).all() and (out[:, :fit] != 7).any() == (fit > 0)


def test_commit_of_nearly_two_to_the_31_vectors():
    """As many layers and heads as a call takes (repeated views of one head's columns): the count of
    vectors and the grid's step add up behind 2^31."""
    import speculative_decoding_specdec_gb300.specdec as sd
    src, dst = torch.randn(1, 2, 1, 1, 9, 4, device=DEV), torch.randn(1, 2, 1, 1, 12, 4, device=DEV)
    want, st = dst.clone(), status()
    want[..., 6:8, :] = src[..., [4, 7], :]
    def wide(t):
        return t.expand(32767, -1, -1, 32768, -1, -1)
    sd.tree_commit(wide(src), wide(dst), i32([4]), i32([2]), i32([[1, 4, -1]]), st, width_dst=i32([9]), nodes=6)
    torch.cuda.synchronize()
    assert int(st) == 0 and torch.equal(dst, want)
    with pytest.raises(sd.SpecdecError):
        sd.tree_commit(src.expand(32768, -1, -1, 32768, -1, -1), dst.expand(32768, -1, -1, 32768, -1, -1), i32([4]), i32([2]),
                       i32([[1, 4, -1]]), st, width_dst=i32([9]), nodes=6)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_scores_of_one_position_of_a_longer_pass(dtype):
    """One token per row whose scores are a slice [:, -1:] of a pass over several: evenly spaced rows."""
    import speculative_decoding_specdec_gb300.specdec as sd
    rng = np.random.default_rng(5)
    z = torch.as_tensor(rng.normal(size=(3, 4, 600)) * 3, dtype=torch.float32).to(dtype).to(DEV)
    tok, u = np.zeros((3, 1), int), np.array([[0.1], [0.5], [0.9]], np.float32)
    for s in (z[:, -1:], z[:1, 1:2], z[:, :1]):
        B = s.shape[0]
        got, st = V.run_greedy(s, tok[:B], None, 1)
        assert st == 0 and got[0].tolist() == [0] * B
        assert got[1].tolist() == [TO.greedy_choice(r) for r in numpy64(s)[:, 0]]
        got, st = V.run_sample(s, s, tok[:B], None, u[:B], 1.0, 1, False)
        assert st == 0 and got[0].tolist() == [0] * B
        for b in range(B):
            edges = np.cumsum(TO.softmax(numpy64(s)[b, 0]))
            y = int(got[1][b])
            assert (edges[y - 1] if y else 0) - 1e-5 <= u[b, 0] <= edges[y] + 1e-5
    with pytest.raises(ValueError):
        sd.verify_tree_greedy(z[:, :2], i32(np.zeros((3, 2))), None, *V.outputs(3, 1), status())


@pytest.mark.parametrize("replacement", [False, True])
def test_a_residual_too_small_to_be_inverted_leaves_p(replacement):
    """p and q agree but for tokens of about 2^-126: what a rejection leaves is a sum whose inverse is
    infinite in fp32."""
    z, w = torch.full((1, 2, 40), -float("inf")), torch.full((1, 2, 40), -float("inf"))
    z[0, 0, [7, 20, 31]] = torch.tensor([0.0, -87.0, -87.0])
    w[0, 0, [7, 20, 31]] = torch.tensor([0.0, -86.5, -87.1])
    u = np.array([[0.5, 0.9]], np.float32)               # p / q of token 20 is 0.61
    got, st = V.run_sample(z.to(DEV), w.to(DEV), np.array([[0, 20]]), np.array([[-1, 0]]), u, 1.0, 1, replacement)
    assert st == 0
    V.same_walk(got, 0, [], 7, [0, 20], 1)


def test_a_draw_of_zero_beside_probabilities_that_round_to_zero():
    """u = 0 takes the first token of any probability.  A slice of the vocabulary holds one score where
    2^x is just not zero or just zero, as the roundings have it: the token is one that has a
    probability, whichever that is."""
    c2 = np.float32(1.4426950408889634)
    top = np.linspace(1, 20, 4001).astype(np.float32)[:, None]
    mt = top * c2
    x = ((np.float64(mt) - 126) / np.float64(c2)).astype(np.float32)
    x = (x + np.arange(-4, 5) * np.spacing(x)).astype(np.float32)
    twice = x * c2 - mt                                                         # rounded, and again
    once = (x.astype(np.float64) * np.float64(c2) - np.float64(mt)).astype(np.float32)
    at = (twice >= -126) & (once < -126)
    pick, top = torch.as_tensor(x[at])[:32], torch.as_tensor(np.broadcast_to(top, x.shape)[at])[:32]
    assert len(pick) > 8
    for V_ in (4096, 32768):
        z = torch.full((len(pick), 1, V_), -float("inf"))
        z[:, 0, 3], z[:, 0, V_ - 6] = pick, top
        u = np.zeros((len(pick), 1), np.float32)
        got, st = V.run_sample(z.to(DEV), z.to(DEV), np.zeros((len(pick), 1), int), None, u, 1.0, 1, False)
        assert st == 0 and set(got[1].tolist()) <= {3, V_ - 6}


@pytest.mark.parametrize("dtype,V_", [(torch.float32, 262147), (torch.bfloat16, 400009)])
@pytest.mark.parametrize("replacement", [False, True])
def test_sampled_vocabularies_that_no_cluster_holds(dtype, V_, replacement):
    """Slices too large for shared memory are read again in every pass, and the draw goes over them
    in several windows: the token is one near the start, in the middle and at the end."""
    rng = np.random.default_rng(V_)
    par, tok = np.array([[-1, 0, 0, 1, -2]] * 6), np.zeros((6, 5), int)
    z = rng.normal(size=(6, 5, V_))
    heavy = np.r_[2, rng.integers(0, V_, 9), V_ - 2]
    z[:, :, heavy] = np.log(V_) - 0.2 * np.arange(len(heavy))
    z = torch.as_tensor(z, dtype=torch.float32).to(dtype)
    w = (z.float() + 0.5 * torch.as_tensor(rng.normal(size=z.shape), dtype=torch.float32)).to(dtype)
    for b in range(6):
        for node in (0, 1):
            kids = TO.children(par[b], node)
            tok[b, kids] = rng.choice(heavy, len(kids), replace=False)
    u = rng.random((6, 5)).astype(np.float32)
    u[2:4, 1:] = 0.9999                       # children are rejected: the draw is from the residual
    zz, ww, want = numpy64(z), numpy64(w), []
    for b in range(6):                        # u[0] in the middle of a heavy token's share
        path, _, p, margins = TO.verify_sample(zz[b], ww[b], tok[b], par[b], u[b].astype(np.float64), 0.9, 3, replacement)
        edges = np.cumsum(p)
        likely = np.flatnonzero(p > 2e-3)
        y = int(likely[(0, -1, len(likely) // 2)[b % 3]])
        u[b, 0] = (edges[y] - p[y] / 2) / edges[-1]
        want.append((path, y, min(margins)))
    got, st = V.run_sample(z.to(DEV), w.to(DEV), tok, par, u, 0.9, 3, replacement)
    assert st == 0
    assert sum(m < 1e-4 for _, _, m in want) <= 1
    for b, (path, y, margin) in enumerate(want):
        if margin >= 1e-4:
            V.same_walk(got, b, path, y, tok[b], 3)


@pytest.mark.parametrize("T,G", [(40, 2), (40, 4)])
def test_a_unit_of_very_many_parts(T, G):
    """One K/V head over so many columns that more shares hold parts of it than the merge takes in
    at a time."""
    rng = np.random.default_rng(T * G)
    n = np.array([20011])
    q, cache, W = A.inputs(rng, 1, T, G, 1, 128, n, torch.bfloat16, layers=2)
    par = random_parents(rng, 1, T, unused=0.1)
    A.hide(cache, n, W, T, par)
    out, lse, st = A.run(q, cache, 1, n, W, par)
    assert st == 0
    A.check(out, lse, q, cache, 1, n, W, par)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_trees_path_is_appended_to_its_pool_slots(dtype):
    """Rounds of a pool with trees: gathered into the padded buffer or verified in their slots, the
    committed paths appended as a chain's drafts are; every slot then holds its sequence's columns."""
    import speculative_decoding_specdec_gb300.specdec as sd
    rng = np.random.default_rng(3)
    S, cap, L, H, hd, T, D, vocab = 7, 90, 2, 2, 64, 10, 4, 200
    lens = [5, 17, 30, 17, 2, 17, 11]
    rows = [list(rng.integers(0, vocab, n)) for n in lens]
    tag = torch.randn(cap, vocab, L, 2, H, hd, generator=torch.Generator().manual_seed(0)).to(dtype).to(DEV)
    arena = torch.full((L, 2, 1, H, S * cap, hd), float("nan"), dtype=dtype, device=DEV)
    ids = np.zeros((S, cap), int)
    for s, r in enumerate(rows):
        ids[s, :len(r)] = r
        for i, x in enumerate(r[:-1]):
            arena[:, :, 0, :, s * cap + i] = tag[i, x]
    col, caps, length, pool_ids = i32(np.arange(S) * cap), i32([cap] * S), i32(lens), i32(ids)
    scratch = torch.full((L, 2, 4, H, 80, hd), float("nan"), dtype=dtype, device=DEV)
    sids, smask, spos = (torch.zeros(4, 80, dtype=d, device=DEV) for d in (torch.int32, torch.uint8, torch.int32))
    blen, width, st = i32(np.zeros(4)), i32([0]), status()
    for batch, in_place in (([0, 2, 4], False), ([1, 3, 5], True), ([6, 0, 3, 1], False), ([5, 2], False)):
        B = len(batch)
        slots = i32(batch)
        sd.pool_gather(arena, scratch, slots, D, col, caps, length, pool_ids, blen[:B], width, st, sids, smask, spos, in_place=in_place)
        par = random_parents(rng, B, T, unused=0.1)
        z, tok = np.full((B, T, vocab), -1.0), rng.integers(0, vocab, (B, T))
        for b, s in enumerate(batch):
            tok[b, 0] = rows[s][-1]
            for t in range(T):
                line = TO.line_of(par[b], t)
                if line:
                    where = (s * cap + len(rows[s]) - 1) if in_place else int(width) - 1
                    (arena[:, :, 0] if in_place else scratch[:, :, b])[:, :, :, where + t] = tag[len(rows[s]) - 2 + len(line), tok[b, t]]
                kids = TO.children(par[b], t)
                z[b, t, tok[b, kids[-1]] if kids and rng.random() < 0.8 else rng.integers(vocab)] = 1
        a, y, path, draft = V.outputs(B, D)
        sd.verify_tree_greedy(torch.as_tensor(z, dtype=torch.float32).to(DEV), i32(tok), i32(par), a, y, path, draft, st)
        if in_place:
            sd.tree_commit(arena, arena, None, a, path, st, nodes=T, n_committed=length, rows=slots, first_col=col)
        else:
            sd.tree_commit(scratch, scratch, width, a, path, st, nodes=T)
        sd.pool_append(arena, scratch, slots, D, col, caps, length, pool_ids, blen[:B], width, a, y, draft, st, in_place=in_place)
        torch.cuda.synchronize()
        assert int(st) == 0
        for b, s in enumerate(batch):
            nodes, token = TO.verify_greedy(z[b], tok[b], par[b], D)
            V.same_walk([x.cpu().numpy() for x in (a, y, path, draft)], b, nodes, token, tok[b], D)
            rows[s] += [int(tok[b, i]) for i in nodes] + [token]
        assert length.tolist() == [len(r) for r in rows]
    for s, r in enumerate(rows):
        assert pool_ids[s, :len(r)].tolist() == r
        for i, x in enumerate(r[:-1]):
            assert torch.equal(arena[:, :, 0, :, s * cap + i], tag[i, x])


@pytest.mark.parametrize("dtype,hd", [(torch.float32, 4), (torch.float32, 12), (torch.bfloat16, 8), (torch.bfloat16, 40), (torch.float32, 252), (torch.bfloat16, 248)])
@pytest.mark.parametrize("T,G", [(1, 1), (3, 4), (16, 3)])
def test_the_smallest_and_oddest_heads(dtype, hd, T, G):
    """Heads of one 16-byte vector and of numbers of vectors that divide nothing."""
    rng = np.random.default_rng(hd + T)
    n = np.array([70, 3])
    q, cache, W = A.inputs(rng, 2, T, G, 1, hd, n, dtype)
    par = random_parents(rng, 2, T, unused=0.1)
    A.hide(cache, n, W, T, par)
    out, lse, st = A.run(q, cache, 1, n, W, par)
    assert st == 0
    A.check(out, lse, q, cache, 1, n, W, par)
