"""Attention over shared prefixes at its limits and beside what is refused or not used.

Tolerances are those of test_gpu_prefix_attention.
"""
import numpy as np
import pytest
import torch

import oracle.tree_oracle as TO
import test_gpu_prefix_attention as PA
from tree_testlib import DEV, i32, random_parents, status

DT = [torch.float32, torch.bfloat16]
# few rows of query rows; more, behind a pass of their group; rows that fill tiles; other heads
SHAPES = [(4, 3, 4, 2, 64), (4, 9, 8, 2, 128), (4, 40, 4, 2, 64), (4, 50, 8, 2, 128), (4, 64, 8, 1, 64), (4, 5, 4, 2, 96)]


@pytest.mark.gpu
def test_a_refused_call_launches_nothing():
    """1024 rows of 32 heads over an arena of a million columns are more tiles than 32 bits number, which
    the rows' own pass refuses: the pass over the prefix must not have run then, nor told of its bounds."""
    import speculative_decoding_specdec_gb300.specdec as sd
    B, H, hd, cap = 1024, 32, 8, (1 << 20) + 64
    dtype = torch.bfloat16
    arena = torch.zeros(1, 2, 1, 1, cap, hd, dtype=dtype, device=DEV).expand(-1, -1, -1, H, -1, -1)
    prefix = torch.zeros(1, 2, 1, H, 64, hd, dtype=dtype, device=DEV)
    q = torch.zeros(B, 1, H, hd, dtype=dtype, device=DEV)
    ws, st = torch.zeros(sd.prefix_attention_workspace_bytes(q, arena, 1), dtype=torch.uint8, device=DEV), status()
    out = torch.full_like(q, 7.0)
    for groups in ([0, 5], [3, 2]):
        with pytest.raises(sd.SpecdecError):
            sd.prefix_attention(q, arena, 0, out, i32(np.full(B, 3)), None, None, st, ws, prefix, i32([40]), i32(groups),
                                first_col=i32(np.arange(B)))
        torch.cuda.synchronize()
        assert int(st) == 0 and not ws.any() and (out == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,T,Hq,H,hd", SHAPES)
@pytest.mark.parametrize("bad", ["none", "wide", "tree"])
def test_a_bad_row_of_a_group_is_left_and_the_others_are_right(dtype, B, T, Hq, H, hd, bad):
    rng = np.random.default_rng(T)
    lens, groups, n = [140], [0, B], np.array([5, 9, 9, 6])
    par = random_parents(rng, B, T)
    q, cache, W, prefix = PA.inputs(6, B, T, Hq, H, hd, n, dtype, 1, lens)
    told, broken = n.copy(), par.copy()
    if bad == "tree":
        broken[1, T - 1] = T - 1                # its own parent
    else:
        told[1] = 0 if bad == "none" else W + 1
    out, lse, st = PA.run(q, cache, 1, told, W, broken, prefix, lens, groups)
    assert st == 5 and (out[1] == 7).all() and (lse[1] == 7).all()
    PA.check(out, lse, q, cache, 1, n, W, par, prefix, lens, groups, only=[0, 2, 3])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,T,Hq,H,hd", SHAPES)
@pytest.mark.parametrize("lens,groups,written", [([50, -1], [0, 2, 4], [0, 1]), ([91, 50], [0, 1, 3], [1, 2, 3]),
                                                 ([50, 70], [0, 3, 2], [])])
def test_rows_of_bad_groups_keep_their_sums_too(dtype, B, T, Hq, H, hd, lens, groups, written):
    n = np.full(B, 10)
    q, cache, W, prefix = PA.inputs(5, B, T, Hq, H, hd, n, dtype, 2, [90, 90], slack=0)
    out, lse, st = PA.run(q, cache, 1, n, W, None, prefix, lens, groups)
    assert st in (4, 5)
    left = [b for b in range(B) if b not in written]
    assert (out[left] == 7).all() and (lse[left] == 7).all()
    PA.check(out, lse, q, cache, 1, n, W, None, prefix, lens, groups, only=written)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,T,Hq,H,hd", SHAPES)
def test_what_unused_nodes_hold_is_not_felt(dtype, B, T, Hq, H, hd):
    """Queries of nodes that a row does not use, and their columns: NaN."""
    rng = np.random.default_rng(B * T)
    n, lens, groups = np.array([5, 1, 30, 12]), [300, 33], [0, 3, 4]
    par = random_parents(rng, B, T, unused=0.4)
    q, cache, W, prefix = PA.inputs(2, B, T, Hq, H, hd, n, dtype, 2, lens)
    for b, t in zip(*np.nonzero(par == -2)):
        q[b, t] = float("nan")
        cache[:, :, b, :, W - 1 + t] = float("nan")
    out, lse, st = PA.run(q, cache, 1, n, W, par, prefix, lens, groups)
    assert st == 0
    q = q.nan_to_num(0.0)                       # (the plain form multiplies them by zero)
    PA.check(out, lse, q, cache, 1, n, W, par, prefix, lens, groups)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,Hq,hd,B,P", [(1, 2, 64, 1024, 512), (3, 4, 128, 1024, 512), (24, 4, 64, 1024, 512), (1, 2, 96, 1024, 512),
                                         (2, 2, 64, 5, 512)])
def test_the_most_rows_and_prefixes(dtype, T, Hq, hd, B, P):
    rng = np.random.default_rng(T)
    lens = rng.integers(0, 60, P)
    groups = np.sort(rng.integers(0, B + 1, P + 1))
    groups[[0, 1]], groups[-1] = [0, min(3, groups[2])], B
    n = rng.integers(1, 20, B)
    q, cache, W, prefix = PA.inputs(3, B, T, Hq, 1, hd, n, dtype, P, lens)
    out, lse, st = PA.run(q, cache, 1, n, W, None, prefix, lens, groups)
    assert st == 0
    only = set(range(min(B, 6))) | set(range(max(0, B - 6), B)) | set(rng.integers(0, B, 40).tolist())
    PA.check(out, lse, q, cache, 1, n, W, None, prefix, lens, groups, only=only)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,Hq,H,hd", [(1, 8, 2, 128), (6, 8, 2, 128), (2, 4, 1, 64), (3, 6, 2, 96)])
def test_groups_of_very_unlike_sizes(dtype, T, Hq, H, hd):
    """Units that are full beside units of a few rows, long prefixes beside short ones."""
    rng = np.random.default_rng(T + hd)
    lens, rows = [3000, 17, 2100, 1, 700, 40], [66, 1, 3, 1, 12, 1]
    groups = np.concatenate(([0], np.cumsum(rows)))
    B = int(groups[-1])
    n = rng.integers(1, 90, B)
    q, cache, W, prefix = PA.inputs(T, B, T, Hq, H, hd, n, dtype, len(lens), lens)
    out, lse, st = PA.run(q, cache, 1, n, W, None, prefix, lens, groups)
    assert st == 0
    PA.check(out, lse, q, cache, 1, n, W, None, prefix, lens, groups)
    again = PA.run(q, cache, 1, n, W, None, prefix, lens, groups)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,T,Hq,H,hd", SHAPES)
@pytest.mark.parametrize("shared", [40, 2500])
def test_own_values_that_are_not_finite_stay_in_their_place(dtype, B, T, Hq, H, hd, shared):
    """Of a committed column: that value of all the row's nodes; of a node's: of those below it alone."""
    rng = np.random.default_rng(T)
    n, lens, groups = np.array([40, 9, 30, 12]), [shared, 33], [0, 3, 4]
    par = random_parents(rng, B, T)
    q, cache, W, prefix = PA.inputs(2, B, T, Hq, H, hd, n, dtype, 2, lens)
    clean = PA.run(q, cache, 1, n, W, par, prefix, lens, groups)
    node, G = T // 2, Hq // H
    cache[1, 1, 0, 0, W - 3, 5] = float("inf")               # committed, row 0
    cache[1, 1, 2, H - 1, W - 1 + node, hd - 1] = float("nan")    # a node's, row 2
    cache[1, 1, 3, 0, W - 1, 0] = float("-inf")              # the pending token's, row 3
    out, lse, st = PA.run(q, cache, 1, n, W, par, prefix, lens, groups)
    assert st == 0 and torch.equal(lse, clean[1])
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[0, :, :G, 5] = True
    for t in range(T):
        if node in TO.line_of(par[2], t):
            hit[2, t, -G:, hd - 1] = True
    hit[3, :, :G, 0] = True
    assert not torch.isfinite(out[hit]).any() and torch.equal(out[~hit], clean[0][~hit])
