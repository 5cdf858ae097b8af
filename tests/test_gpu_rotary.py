"""Rotary positions with the append to the cache, against the float64 oracle.

Tolerance: three fp32 roundings of a product sum, 3 * 2^-24 * (|x1| + |x2|), and for bf16 one
rounding more, 2^-8 of the result (bf16 has 8 significant bits).  Copies are exact.
"""
import numpy as np
import pytest
import torch

import oracle.tree_oracle as TO
from tree_testlib import DEV, i32, numpy64, random_parents, status

pytestmark = pytest.mark.gpu


def make_table(P, rot, base=10000.0, factor=1.0):
    f = base ** (-np.arange(rot // 2) / (rot // 2)) / factor
    a = np.arange(P)[:, None] * f
    return torch.as_tensor(np.stack((np.cos(a), np.sin(a)), -1), dtype=torch.float32).to(DEV)


def close(got, want, x, dtype):
    """|got - want| within the derived bound; x: the unrotated values (same norm per pair)."""
    tol = 3 * 2.0 ** -24 * 2 * np.abs(x).max(-1, keepdims=True)
    if dtype == torch.bfloat16:
        tol = tol * 1.01 + 2.0 ** -8 * np.abs(want) + 2.0 ** -133
    assert (np.abs(got - want) <= tol).all()


def run_pass(B, T, Hq, H, hd, rot, dtype, interleaved, parents, n, W, extra=0, fused=True, seed=0,
             in_place=False, one_row=False, layers=2):
    import speculative_decoding_specdec_gb300.specdec as sd
    gen = torch.Generator().manual_seed(seed)
    width = (Hq + 2 * H) * hd + extra
    if fused:     # q, k and v are slices of one projection, `extra` elements between tokens
        buf = torch.randn(B, T, width, generator=gen).to(dtype).to(DEV)
        q = buf[:, :, :Hq * hd].unflatten(2, (Hq, hd))
        k = buf[:, :, Hq * hd:(Hq + H) * hd].unflatten(2, (H, hd))
        v = buf[:, :, (Hq + H) * hd:(Hq + 2 * H) * hd].unflatten(2, (H, hd))
    else:
        q, k, v = (torch.randn(B, T, h, hd, generator=gen).to(dtype).to(DEV) for h in (Hq, H, H))
    cap = W + T
    cache = torch.randn(layers, 2, 1 if one_row else B, H, cap, hd, generator=gen).to(dtype).to(DEV)
    before = numpy64(cache)
    table = make_table(W + T, rot, factor=4.0)
    q0 = numpy64(q)
    out = q if in_place else torch.full((B, T, Hq, hd), 7.0, dtype=dtype, device=DEV)
    st = status()
    sd.rotary_append(q, k, v, cache, layers - 1, table, out, st, n_committed=i32(n), width=i32([W]),
                     parents=None if parents is None else i32(parents), interleaved=interleaved)
    torch.cuda.synchronize()
    return dict(q=q0, k=numpy64(k), v=numpy64(v), before=before, cache=numpy64(cache),
                table=numpy64(table), out=numpy64(out), status=int(st))


def check_pass(r, parents, n, W, dtype, interleaved, rows=None):
    B, T = r["q"].shape[:2]
    want = r["before"].copy()
    layer, L = want[-1], want.shape[0]
    for b in range(B) if rows is None else rows:
        for t in range(T):
            line = TO.line_of(TO.chain(T) if parents is None else parents[b], t)
            if not line:
                assert (r["out"][b, t] == 0).all()
                continue
            cs = r["table"][n[b] - 2 + len(line)]
            close(r["out"][b, t], TO.rotate(r["q"][b, t], cs[:, 0], cs[:, 1], interleaved), r["q"][b, t], dtype)
            kk = TO.rotate(r["k"][b, t], cs[:, 0], cs[:, 1], interleaved)
            close(r["cache"][L - 1, 0, b, :, W - 1 + t], kk, r["k"][b, t], dtype)
            layer[0, b, :, W - 1 + t] = r["cache"][L - 1, 0, b, :, W - 1 + t]
            layer[1, b, :, W - 1 + t] = r["v"][b, t]
    np.testing.assert_array_equal(r["cache"], want)      # nothing else was written


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,Hq,H,hd,rot,interleaved,tree", [
    (2, 5, 4, 2, 64, 64, False, False),     # tiny chain
    (1, 1, 1, 1, 16, 2, True, False),       # one token, one pair
    (3, 7, 6, 3, 64, 32, True, True),       # part of the head, interleaved pairs
    (3, 64, 8, 2, 128, 64, False, True),    # the largest tree
    (2, 9, 5, 1, 80, 20, False, True),      # pairs that no 16-byte vector divides
    (2, 3, 4, 4, 96, 96, True, False),
])
def test_verification_pass(dtype, B, T, Hq, H, hd, rot, interleaved, tree):
    rng = np.random.default_rng(T)
    n = rng.integers(1, 40, B)
    W = int(n.max()) + 3
    par = random_parents(rng, B, T, unused=0.2) if tree else None
    r = run_pass(B, T, Hq, H, hd, rot, dtype, interleaved, par, n, W)
    assert r["status"] == 0
    check_pass(r, par, n, W, dtype, interleaved)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("extra", [1, 8])
def test_strides_and_in_place(dtype, extra):
    n, W, T = np.array([4, 9]), 9, 6
    for in_place in (False, True):
        r = run_pass(2, T, 4, 2, 64, 64, dtype, False, None, n, W, extra=extra, in_place=in_place)
        assert r["status"] == 0
        check_pass(r, None, n, W, dtype, False)
    r = run_pass(2, T, 4, 2, 64, 64, dtype, True, None, n, W, fused=False, in_place=True)
    check_pass(r, None, n, W, dtype, True)


def test_an_unused_row_and_unused_nodes():
    par = np.array([[-2, -2, -2], [-1, 0, -2]])
    r = run_pass(2, 3, 2, 2, 16, 16, torch.float32, False, par, np.array([3, 2]), 5)
    assert r["status"] == 0
    check_pass(r, par, [3, 2], 5, torch.float32, False)


@pytest.mark.parametrize("par,n,W", [
    ([[-1, 0, 0], [-1, 1, 0]], [3, 3], 3),    # a parent that is the node itself
    ([[-1, 0, 0], [-1, -2, 1]], [3, 3], 3),   # an unused parent
    ([[-1, 0, 0], [0, 0, 0]], [3, 3], 3),     # the root's parent
    ([[-1, 0, 0], [-1, 0, 0]], [3, 4], 3),    # more tokens than the width
    ([[-1, 0, 0], [-1, 0, 0]], [3, 0], 3),
])
def test_bad_rows_are_reported_and_not_written(par, n, W):
    import speculative_decoding_specdec_gb300.specdec as sd
    r = run_pass(2, 3, 2, 2, 16, 16, torch.float32, False, np.array(par), np.array(n), W)
    assert r["status"] == sd.ERR_INPUT_RANGE
    assert (r["out"][1] == 7).all()
    check_pass(r, np.array(par), n, W, torch.float32, False, rows=[0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_explicit_positions_and_columns(dtype):
    import speculative_decoding_specdec_gb300.specdec as sd
    gen = torch.Generator().manual_seed(4)
    B, T, H, hd, cap, P = 3, 130, 2, 64, 150, 200
    x = [torch.randn(B, T, H, hd, generator=gen).to(dtype).to(DEV) for _ in range(3)]
    cache = torch.randn(1, 2, B, H, cap, hd, generator=gen).to(dtype).to(DEV)
    want, table, out, st = numpy64(cache), make_table(P, hd), torch.empty_like(x[0]), status()
    rng = np.random.default_rng(0)
    pos = rng.integers(0, P, (B, T))
    col = np.stack([rng.permutation(cap)[:T] for _ in range(B)])
    col[rng.random((B, T)) < 0.2] = -1
    sd.rotary_append(*x, cache, 0, table, out, st, positions=i32(pos), columns=i32(col))
    torch.cuda.synchronize()
    assert int(st) == 0
    q, k, v = (numpy64(t) for t in x)
    got, cs = numpy64(cache), numpy64(table)
    for b in range(B):
        for t in range(T):
            if col[b, t] < 0:
                assert (out[b, t] == 0).all()
                continue
            c, s = cs[pos[b, t], :, 0], cs[pos[b, t], :, 1]
            close(numpy64(out[b, t]), TO.rotate(q[b, t], c, s, False), q[b, t], dtype)
            close(got[0, 0, b, :, col[b, t]], TO.rotate(k[b, t], c, s, False), k[b, t], dtype)
            want[0, 0, b, :, col[b, t]] = got[0, 0, b, :, col[b, t]]
            want[0, 1, b, :, col[b, t]] = v[b, t]
    np.testing.assert_array_equal(got, want)
    for bad_pos, bad_col, code in ((P, 0, sd.ERR_INPUT_RANGE), (-1, 0, sd.ERR_INPUT_RANGE), (0, cap, sd.ERR_CAPACITY)):
        st = status()
        pos[1, 3], col[1, 3] = bad_pos, bad_col
        sd.rotary_append(*x, cache, 0, table, out, st, positions=i32(pos), columns=i32(col))
        torch.cuda.synchronize()
        assert int(st) == code


def test_refusals():
    import speculative_decoding_specdec_gb300.specdec as sd
    q = torch.zeros(1, 2, 2, 16, device=DEV)
    cache = torch.zeros(1, 2, 1, 2, 8, 16, device=DEV)
    tab, st, one = make_table(8, 16), status(), i32([2])
    ok = dict(n_committed=one, width=one)
    sd.rotary_append(q, q, q, cache, 0, tab, torch.empty_like(q), st, **ok)
    for bad in (dict(cache=cache.bfloat16()), dict(tab=make_table(8, 18)), dict(layer=1), dict(layer=-1),
                dict(k=q[:, :1]), dict(kw=dict(n_committed=one)), dict(kw=dict(positions=i32([[0, 0]]))),
                dict(kw={}), dict(q=q.transpose(1, 2))):
        a = dict(q=q, k=q, cache=cache, layer=0, tab=tab, kw=ok) | bad
        with pytest.raises((sd.SpecdecError, ValueError, AttributeError)):
            sd.rotary_append(a["q"], a["k"], q, a["cache"], a["layer"], a["tab"], torch.empty_like(q), st, **a["kw"])
    torch.cuda.synchronize()
    assert int(st) == 0
