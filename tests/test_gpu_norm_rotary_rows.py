"""Normed heads, rotary positions and append: more tokens than the GPU holds warps, so that a warp takes
several of several rows, and what is refused token by token and row by row.

Values are checked as in test_gpu_norm_rotary; beside something refused, everything else has to be what the
call without it writes, bit for bit.
"""
import numpy as np
import pytest
import torch

import test_gpu_norm_rotary as NR
from tree_testlib import DEV, i32, random_parents, status

DT = [torch.float32, torch.bfloat16]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("Hq,H,hd,rot,case", [
    (2, 1, 64, 64, {}), (3, 2, 32, 16, dict(interleaved=True, wdtype=torch.float32)), (2, 1, 40, 20, dict(extra=1)),
    (1, 1, 512, 512, {}),
])
def test_more_tokens_than_warps(dtype, Hq, H, hd, rot, case):
    """Given positions and columns, padding among them."""
    NR.run(3, 2000, Hq, H, hd, rot, dtype, explicit=True, seed=hd, start=[0, 40, 7], **case)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,T,Hq,H,hd,rot,case", [
    (80, 64, 2, 1, 64, 64, {}), (300, 17, 2, 1, 64, 32, dict(interleaved=True, offset=1.0)), (60, 50, 1, 1, 504, 8, {}),
])
def test_a_warp_takes_rows_of_unlike_trees(dtype, B, T, Hq, H, hd, rot, case):
    par = random_parents(np.random.default_rng(B), B, T, unused=0.3)
    NR.run(B, T, Hq, H, hd, rot, dtype, parents=par, seed=T, start=(np.arange(B) * 3 % 50).tolist(), **case)


def call(dtype, where, B, T, W, cap, P, start=None, hd=64, rot=64):
    import speculative_decoding_specdec_gb300.specdec as sd
    gen = torch.Generator().manual_seed(B * T)
    q, k, v = (torch.randn(B, T, h, hd, generator=gen).to(dtype).to(DEV) for h in (4, 2, 2))
    cache = torch.randn(1, 2, B, 2, cap, hd, generator=gen).to(dtype).to(DEV)
    table = torch.randn(P, rot // 2, 2, generator=gen).to(DEV)
    w = torch.randn(hd, generator=gen).to(dtype).to(DEV)
    out, st = torch.full_like(q, 7.0), status()
    sd.norm_rotary_append(q, k, v, cache, 0, table, out, st, w, w, start=None if start is None else i32(start), **where)
    torch.cuda.synchronize()
    return out, cache[0], int(st)


def cache_before(B, T, cap, hd, dtype):
    """What `call`'s cache holds before."""
    gen = torch.Generator().manual_seed(B * T)
    for h in (4, 2, 2):
        torch.randn(B, T, h, hd, generator=gen)
    return torch.randn(1, 2, B, 2, cap, hd, generator=gen).to(dtype).to(DEV)[0]


def same_but(good, bad, before, refused, columns):
    """refused [B, T]: tokens that the bad call must not have written; columns [B, T]: where the good one did."""
    out, cache = good[0].clone(), good[1].clone()
    for b, t in zip(*np.nonzero(refused)):
        out[b, t] = 7.0
        if columns[b, t] >= 0:
            cache[:, b, :, columns[b, t]] = before[:, b, :, columns[b, t]]
    return torch.equal(out, bad[0]) and torch.equal(cache, bad[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,T", [(3, 5), (90, 64)])
@pytest.mark.parametrize("what", ["own parent", "unused parent", "root's parent", "later parent", "no tokens", "more than the width",
                                  "lowest", "highest"])
def test_bad_rows_are_told_and_not_written(dtype, B, T, what):
    rng = np.random.default_rng(T)
    par = random_parents(rng, B, T)
    n, W = rng.integers(1, 20, B), 25
    cap, b = W + T, B - 2
    good = call(dtype, dict(n_committed=i32(n), width=i32([W]), parents=i32(par)), B, T, W, cap, 200)
    assert good[2] == 0
    told, broken = n.copy(), par.copy()
    if what == "own parent":
        broken[b, T - 1] = T - 1
    elif what == "unused parent":
        broken[b, 2], broken[b, 3:] = -2, 2
    elif what == "root's parent":
        broken[b, 0] = 0
    elif what == "later parent":
        broken[b, 2] = 3
    else:
        told[b] = {"no tokens": 0, "more than the width": W + 1, "lowest": -2 ** 31, "highest": 2 ** 31 - 1}[what]
    bad = call(dtype, dict(n_committed=i32(told), width=i32([W]), parents=i32(broken)), B, T, W, cap, 200)
    refused = np.zeros((B, T), bool)
    refused[b] = True                            # (unused nodes too)
    assert bad[2] == 5
    columns = np.broadcast_to(W - 1 + np.arange(T), (B, T))
    assert same_but(good, bad, cache_before(B, T, cap, 64, dtype), refused, columns)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,T", [(3, 5), (90, 64)])
def test_columns_beyond_the_cache(dtype, B, T):
    """A width that leaves no room for the last nodes, and one near the integers' end."""
    n, cap = np.full(B, 3), 100
    good = call(dtype, dict(n_committed=i32(n), width=i32([cap - T + 1])), B, T, 0, cap, 200)
    assert good[2] == 0
    before = cache_before(B, T, cap, 64, dtype)
    W = cap - T + 3                              # the last two do not fit
    bad = call(dtype, dict(n_committed=i32(n), width=i32([W])), B, T, 0, cap, 200)
    assert bad[2] == 4
    assert torch.equal(bad[0][:, :T - 2], good[0][:, :T - 2]) and (bad[0][:, T - 2:] == 7).all()
    first = W - 1
    assert torch.equal(bad[1][..., :first, :], before[..., :first, :])
    assert torch.equal(bad[1][..., first:, :], good[1][..., cap - T:cap - 2, :])
    for W in (2 ** 31 - 1, 2 ** 31 - T):
        out, cache, st = call(dtype, dict(n_committed=i32(n), width=i32([W])), B, T, 0, cap, 200)
        assert st == 4 and (out == 7).all() and torch.equal(cache, before)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,T", [(3, 5), (3, 1500)])
@pytest.mark.parametrize("pos,col,start,code", [(200, None, 0, 5), (-1, None, 0, 5), (-2 ** 31, None, 9, 5), (None, "cap", 0, 4),
                                                (None, 2 ** 31 - 1, 0, 4), (199, None, 1, 5), (2 ** 31 - 1, None, 2 ** 31 - 1, 5),
                                                (2 ** 31 - 1, -1, 0, 0), (-5, -2 ** 31, 0, 0)])
def test_given_places_out_of_range(dtype, B, T, pos, col, start, code):
    """One token of a call; as padding it is zero, whatever its position says."""
    rng = np.random.default_rng(T)
    P, cap = 200, T + 9
    positions, columns = rng.integers(0, P - 60, (B, T)), np.stack([rng.permutation(cap)[:T] for _ in range(B)])
    columns[rng.random((B, T)) < 0.2] = -1
    b, t = 1, T - 2
    columns[b, t] = next(c for c in range(cap) if c not in columns[b])
    starts = np.full(B, 3)
    if start:
        positions[b] = -1                        # the row's other tokens are padding
        keep = columns[b, t]
        columns[b] = -1
        columns[b, t], positions[b, t] = keep, 4
    place = lambda: dict(positions=i32(positions), columns=i32(columns))
    good = call(dtype, place(), B, T, 0, cap, P, starts)
    assert good[2] == 0
    was = columns.copy()
    if pos is not None:
        positions[b, t] = pos if start or pos < 0 or pos > P else pos - 3
    if col is not None:
        columns[b, t] = cap if col == "cap" else col
    if start:
        starts[b] = start
    bad = call(dtype, place(), B, T, 0, cap, P, starts)
    assert bad[2] == code
    refused = np.zeros((B, T), bool)
    refused[b, t] = True
    if code == 0:                                # padding now
        bad[0][b, t] = 7.0
    assert same_but(good, bad, cache_before(B, T, cap, 64, dtype), refused, was)
