"""Attention of a draft tree over the cache, against the float64 oracle.

Tolerance, derived: a score is a sum of hd products in fp32 (in any order), so its error is at most
dz = (hd + 4) * 2^-24 * max sum|q k| * scale, and a weight's relative error 2 * dz + 2^-20 (two
exponentials and the normalisation); sums over n columns add n * 2^-24.  That holds for the
weighted sum of |v|.  With bf16 tensors every weight is also rounded (2^-8 relative, independent):
by Hoeffding's inequality the sum of those errors stays below 7 * 2^-8 * sqrt(sum (p v)^2) but for
one value in 10^10; and the result is rounded once, 2^-8 of it.
"""
import numpy as np
import pytest
import torch

import oracle.tree_oracle as TO
from tree_testlib import DEV, i32, numpy64, random_parents, status

pytestmark = pytest.mark.gpu


def run(q, cache, layer, n, W, parents, scale=None, lse=True, ws=None, rows=None, first_col=None):
    import speculative_decoding_specdec_gb300.specdec as sd
    B, T, Hq, hd = q.shape
    out = torch.full((B, T, Hq, hd), 7.0, dtype=q.dtype, device=DEV)
    ls = torch.full((B, T, Hq), 7.0, device=DEV) if lse else None
    st = status()
    if ws is None:
        ws = torch.zeros(sd.tree_attention_workspace_bytes(q, cache), dtype=torch.uint8, device=DEV)
    sd.tree_attention(q, cache, layer, out, i32(n), None if W is None else i32([W]),
                      None if parents is None else i32(parents), st, ws, scale=scale, lse=ls,
                      rows=None if rows is None else i32(rows),
                      first_col=None if first_col is None else i32(first_col))
    torch.cuda.synchronize()
    return numpy64(out), numpy64(ls) if lse else None, int(st)


def check(got, lse, q, cache, layer, n, W, parents, scale=None, first=None, crow=None, only=None):
    B, T, Hq, hd = q.shape
    scale = hd ** -0.5 if scale is None else scale
    bf16 = q.dtype == torch.bfloat16
    q, kv = numpy64(q), cache[layer]
    for b in range(B):
        if only is not None and b not in only:
            continue
        lo = (W - n[b]) if first is None else first[b]
        r = b if crow is None else crow
        k, v = (numpy64(kv[j, r, :, lo:lo + n[b] - 1 + T]) for j in (0, 1))
        out, ls, sums, squares = TO.attention(q[b], k, v, n[b] - 1, TO.chain(T) if parents is None else parents[b], scale)
        big = np.abs(np.nan_to_num(k)).sum(-1).max() * np.abs(q[b]).max() * abs(scale)
        eps = 2 * (hd + 4) * 2.0 ** -24 * big + 2.0 ** -20 + (n[b] + T) * 2.0 ** -24
        tol = eps * sums + 1e-30
        if bf16:
            tol = tol + 7 * 2.0 ** -8 * np.sqrt(squares) + 2.0 ** -8 * np.abs(out)
        bad = ~(np.abs(got[b] - out) <= tol)
        assert not bad.any(), (b, np.argwhere(bad)[:5], np.abs(got[b] - out).max(), bad.mean())
        if lse is not None:
            fine = np.isfinite(ls)
            assert (np.isneginf(lse[b]) == ~fine).all()
            assert (np.abs(lse[b] - ls)[fine] <= eps * 2 + 2.0 ** -20 * (1 + np.abs(ls[fine]))).all()


def inputs(rng, B, T, Hq, H, hd, n, dtype, slack=5, layers=2, scale_q=1.0):
    W = int(max(n)) + 2
    gen = torch.Generator(device=DEV).manual_seed(int(rng.integers(1 << 30)))
    q = (torch.randn(B, T, Hq, hd, generator=gen, device=DEV) * scale_q).to(dtype)
    cache = torch.randn(layers, 2, B, H, W + T + slack, hd, generator=gen, device=DEV).to(dtype)
    return q, cache, W


def hide(cache, n, W, T, parents):
    """NaN wherever nothing may be read: left of the committed columns, behind the nodes', and the
    columns of unused nodes; the other layers too."""
    for b in range(cache.shape[2]):
        cache[:, :, b, :, :W - n[b]] = float("nan")
        cache[:, :, b, :, W - 1 + T:] = float("nan")
        if parents is not None:
            for t in np.flatnonzero(parents[b] == -2):
                cache[:, :, b, :, W - 1 + t] = float("nan")
    cache[0] = float("nan")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,Hq,H,hd,lo,hi,tree", [
    (2, 1, 4, 2, 64, 1, 20, False),        # single tokens, a row with nothing before its token
    (2, 5, 4, 2, 64, 5, 20, False),        # tiny chain
    (3, 6, 8, 8, 128, 100, 300, False),    # one query head per K/V head
    (4, 16, 8, 2, 128, 30, 700, True),     # 64 query rows a K/V head
    (2, 32, 32, 2, 128, 200, 900, True),   # 512 query rows a K/V head
    (1, 64, 8, 2, 64, 129, 129, True),     # the largest tree
    (1, 3, 4, 1, 128, 5000, 5000, True),   # one long row: the columns are split
    (5, 7, 6, 2, 64, 1, 260, True),        # a group that is no power of two
    (2, 9, 12, 4, 80, 1, 70, True),        # other head sizes
    (2, 4, 4, 2, 256, 40, 90, True),
    (1, 2, 2, 2, 16, 33, 33, True),
    (33, 2, 4, 4, 64, 1, 50, False),       # more rows than a warp plans at once
])
def test_against_oracle(dtype, B, T, Hq, H, hd, lo, hi, tree):
    rng = np.random.default_rng(B * T + hd)
    n = np.r_[hi, rng.integers(lo, hi + 1, B - 1)] if B > 1 else np.array([hi])
    n[-1] = lo
    q, cache, W = inputs(rng, B, T, Hq, H, hd, n, dtype)
    par = random_parents(rng, B, T, unused=0.15) if tree else None
    hide(cache, n, W, T, par)
    out, lse, st = run(q, cache, 1, n, W, par)
    assert st == 0
    check(out, lse, q, cache, 1, n, W, par)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,G", [(1, 1), (4, 1), (8, 2), (16, 4), (40, 3), (64, 16)])
@pytest.mark.parametrize("cols", [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257])
def test_tile_borders(dtype, T, G, cols):
    """Committed columns around tile borders, so that a tile ends inside, before and behind them."""
    rng = np.random.default_rng(cols + T)
    n = np.array([cols, max(1, cols - 1)])
    hd = 128 if T > 8 else 64
    q, cache, W = inputs(rng, 2, T, G, 1, hd, n, dtype)
    par = random_parents(rng, 2, T)
    hide(cache, n, W, T, par)
    out, lse, st = run(q, cache, 1, n, W, par)
    assert st == 0
    check(out, lse, q, cache, 1, n, W, par)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,G,hd", [(3, 1, 64), (12, 4, 128), (32, 8, 128)])
def test_values_of_unseen_nodes_do_not_leak(dtype, T, G, hd):
    """K and V of some nodes are NaN or infinite: nodes that do not see them give what they gave."""
    rng = np.random.default_rng(T)
    n = np.array([37, 200])
    q, cache, W = inputs(rng, 2, T, 2 * G, 2, hd, n, dtype)
    par = random_parents(rng, 2, T, deep=0.2)
    clean, _, _ = run(q, cache, 1, n, W, par)
    poison = T // 2
    for kv, value in ((1, float("nan")), (1, float("inf")), (0, float("nan"))):
        dirty = cache.clone()
        dirty[1, kv, :, :, W - 1 + poison] = value
        out, _, st = run(q, dirty, 1, n, W, par)
        assert st == 0
        for b in range(2):
            for t in range(T):
                if poison in TO.line_of(par[b], t):
                    assert not np.isfinite(out[b, t]).all()
                else:
                    np.testing.assert_array_equal(out[b, t], clean[b, t])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_large_scores_and_flat_scores(dtype):
    rng = np.random.default_rng(0)
    n = np.array([150, 40])
    q, cache, W = inputs(rng, 2, 5, 4, 2, 64, n, dtype, scale_q=1.0)
    for scale in (30.0, 0.0, -1.0):       # one column takes all; all equal; reversed
        out, lse, st = run(q, cache, 1, n, W, None, scale=scale)
        assert st == 0
        check(out, lse, q, cache, 1, n, W, None, scale=scale)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_without_nodes(dtype):
    rng = np.random.default_rng(1)
    n = np.array([10, 20, 30])
    q, cache, W = inputs(rng, 3, 4, 4, 2, 64, n, dtype)
    par = np.array([[-2] * 4, [-1, -2, 0, -2], [-2] * 4])
    hide(cache, n, W, 4, par)
    out, lse, st = run(q, cache, 1, n, W, par)
    assert st == 0 and (out[[0, 2]] == 0).all() and np.isneginf(lse[[0, 2]]).all()
    check(out, lse, q, cache, 1, n, W, par)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,G", [(2, 1), (24, 8)])
def test_pool_arena_rows(dtype, T, G):
    """Slots of one arena row, taken in any order through rows / first_col."""
    rng = np.random.default_rng(2)
    S, H, hd = 6, 2, 128
    lens = rng.integers(1, 200, S)
    cols = np.r_[0, np.cumsum(lens + T + 3)][:S]
    cache = torch.randn(1, 2, 1, H, int(cols[-1] + lens[-1] + T), hd, device=DEV).to(dtype)
    rows = np.array([4, 0, 5])
    q = torch.randn(3, T, H * G, hd, device=DEV).to(dtype)
    par = random_parents(rng, 3, T)
    out, lse, st = run(q, cache, 0, lens, None, par, rows=rows, first_col=cols)
    assert st == 0
    check(out, lse, q, cache, 0, lens[rows], None, par, first=cols[rows], crow=0)


def test_workspace_is_reused_and_results_repeat():
    """The same call gives the same bits, also behind calls of other shapes in one workspace."""
    import speculative_decoding_specdec_gb300.specdec as sd
    rng = np.random.default_rng(3)
    shapes = [(1, 3, 4, 1, 128, 4000), (4, 16, 8, 2, 128, 500), (2, 32, 16, 1, 64, 900)]
    made = [inputs(rng, B, T, Hq, H, hd, np.full(B, n), torch.bfloat16) + (np.full(B, n),)
            for B, T, Hq, H, hd, n in shapes]
    need = max(sd.tree_attention_workspace_bytes(q, c) for q, c, _, _ in made)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    first = [run(q, c, 1, n, W, None, ws=ws)[0] for q, c, W, n in made]
    for _ in range(5):
        for (q, c, W, n), want in zip(made, first):
            got, _, st = run(q, c, 1, n, W, None, ws=ws)
            assert st == 0
            np.testing.assert_array_equal(got, want)


def test_one_workspace_for_shapes_of_any_size():
    """What one shape leaves in the workspace (cut units' parts of long rows) disturbs no other, with
    many or few units, rows and splits, in either direction."""
    import speculative_decoding_specdec_gb300.specdec as sd
    rng = np.random.default_rng(4)
    shapes = [(1, 64, 16, 1, 128, 6000, torch.bfloat16), (24, 1, 16, 16, 128, 700, torch.bfloat16), (1, 2, 4, 1, 64, 3000, torch.float32),
              (16, 2, 32, 8, 64, 900, torch.bfloat16), (2, 20, 4, 4, 128, 1200, torch.bfloat16), (8, 1, 8, 8, 128, 500, torch.float32)]
    made = [inputs(rng, B, T, Hq, H, hd, np.full(B, n), dt) + (np.full(B, n),) for B, T, Hq, H, hd, n, dt in shapes]
    ws = torch.zeros(max(sd.tree_attention_workspace_bytes(q, c) for q, c, _, _ in made), dtype=torch.uint8, device=DEV)
    want = [run(q, c, 1, n, W, None)[0] for q, c, W, n in made]
    for order in (range(6), reversed(range(6)), (0, 1, 0, 3, 2, 5, 4, 1)):
        for i in order:
            q, c, W, n = made[i]
            got, _, st = run(q, c, 1, n, W, None, ws=ws)
            assert st == 0
            np.testing.assert_array_equal(got, want[i])


def test_strides_layers_and_another_stream():
    import speculative_decoding_specdec_gb300.specdec as sd
    rng = np.random.default_rng(5)
    n = np.array([60, 90])
    B, T, Hq, H, hd = 2, 6, 8, 2, 64
    q0, cache, W = inputs(rng, B, T, Hq, H, hd, n, torch.bfloat16, layers=3)
    buf = torch.zeros(B, T, Hq * hd + 32, dtype=torch.bfloat16, device=DEV)
    q = buf[:, :, :Hq * hd].unflatten(2, (Hq, hd))
    q.copy_(q0)
    obuf = torch.zeros(T, B, Hq, hd, dtype=torch.bfloat16, device=DEV)
    out, st = obuf.transpose(0, 1), status()
    ws = torch.zeros(sd.tree_attention_workspace_bytes(q, cache), dtype=torch.uint8, device=DEV)
    nn, ww = i32(n), i32([W])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sd.tree_attention(q, cache, 2, out, nn, ww, None, st, ws, stream=s)
    s.synchronize()
    assert int(st) == 0
    check(numpy64(out), None, q, cache, 2, n, W, None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_bad_rows_are_reported_and_not_written(dtype):
    import speculative_decoding_specdec_gb300.specdec as sd
    rng = np.random.default_rng(6)
    n = np.array([30, 50, 8])
    q, cache, W = inputs(rng, 3, 3, 4, 2, 64, n, dtype, slack=0)
    tree = np.array([[-1, 0, 1]] * 3)
    def go(n, W, par, code, only):
        out, lse, st = run(q, cache, 1, n, W, par)
        assert st == code
        bad = [b for b in range(3) if b not in only]
        assert (out[bad] == 7).all() and (lse[bad] == 7).all()
        check(out, lse, q, cache, 1, n, W, par, only=only)
    go(np.array([30, 0, 8]), W, tree, sd.ERR_INPUT_RANGE, [0, 2])
    go(np.array([30, W + 1, 8]), W, tree, sd.ERR_INPUT_RANGE, [0, 2])
    go(n, cache.shape[4] - 1, tree, sd.ERR_CAPACITY, [])
    for row in ([-1, 1, 0], [-1, -2, 1], [0, 0, 0]):
        par = tree.copy()
        par[1] = row
        go(n, W, par, sd.ERR_INPUT_RANGE, [0, 2])


def test_refusals():
    import speculative_decoding_specdec_gb300.specdec as sd
    q = torch.zeros(1, 2, 4, 64, device=DEV)
    cache = torch.zeros(1, 2, 1, 2, 8, 64, device=DEV)
    st, one = status(), i32([2])
    ws = torch.zeros(sd.tree_attention_workspace_bytes(q, cache), dtype=torch.uint8, device=DEV)
    def call(q=q, cache=cache, layer=0, out=None, n=one, w=one, ws=ws, **kw):
        sd.tree_attention(q, cache, layer, torch.empty_like(q) if out is None else out, n, w, None, st, ws, **kw)
    call()
    for bad in (dict(layer=1), dict(cache=cache.bfloat16()), dict(q=q[:, :, :3].contiguous()), dict(w=None),
                dict(ws=ws[:256]), dict(ws=ws[1:]), dict(scale=float("inf")), dict(rows=i32([0])),
                dict(n=i32([1, 2])), dict(q=torch.zeros(1, 65, 4, 64, device=DEV)),
                dict(q=torch.zeros(1, 2, 4, 2, device=DEV), cache=torch.zeros(1, 2, 1, 2, 8, 2, device=DEV)),
                dict(lse=torch.zeros(1, 2, 3, device=DEV))):
        with pytest.raises((sd.SpecdecError, ValueError, AttributeError)):
            call(**bad)
    torch.cuda.synchronize()
    assert int(st) == 0
    assert sd.lib.specdec_tree_attention_workspace(sd.BF16, 1, 65, 4, 2, 64) == 0
    assert sd.lib.specdec_tree_attention_workspace(sd.BF16, 1, 2, 5, 2, 64) == 0
