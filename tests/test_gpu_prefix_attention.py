"""Attention over a shared prefix and the rows' own columns, against a float64 form of both together.

Tolerance: as for the attention of a tree (a score is a sum of hd products in fp32, off by at most
dz = (hd + 4) * 2^-24 * max sum |q k| * scale; a weight 2 dz + 2^-20; sums over n columns n * 2^-24), and
2^-20 more for the merging of the two passes' parts (two exponentials, five roundings).  With bf16 tensors
every weight is also rounded, 2^-8 of it and independent, so that by Hoeffding's inequality the sum of
those errors stays below 7 * 2^-8 * sqrt(sum (p v)^2) but for one value in 10^10, and the result is
rounded once, 2^-8 of it.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle.tree_oracle as TO
from tree_testlib import DEV, i32, random_parents, status

DT = [torch.float32, torch.bfloat16]


def run(q, cache, layer, n, W, parents, prefix, lens, groups, first=None, scale=None, ws=None, rows=None, first_col=None,
        out=None):
    import speculative_decoding_specdec_gb300.specdec as sd
    B, T, Hq, hd = q.shape
    if out is None:
        out = torch.full((B, T, Hq, hd), 7.0, dtype=q.dtype, device=DEV)
    lse, st = torch.full((B, T, Hq), 7.0, device=DEV), status()
    if ws is None:
        ws = torch.zeros(sd.prefix_attention_workspace_bytes(q, cache, len(lens)), dtype=torch.uint8, device=DEV)
    opt = lambda x: None if x is None else i32(x)
    sd.prefix_attention(q, cache, layer, out, i32(n), None if W is None else i32([W]), opt(parents), st, ws, prefix,
                        i32(lens), i32(groups), prefix_first=opt(first), scale=scale, lse=lse, rows=opt(rows),
                        first_col=opt(first_col))
    torch.cuda.synchronize()
    return out, lse, int(st)


def whole(q, k, v, see, scale):
    """q [T, Hq, hd], k and v [H, cols, hd], see [T, cols]: out, lse, sum p |v|, sum (p v)^2."""
    T, Hq, hd = q.shape
    H = k.shape[0]
    x = q.view(T, H, Hq // H, hd).permute(1, 2, 0, 3)
    z = scale * (x @ k[:, None].transpose(-1, -2))
    z = z.masked_fill(~see, float("-inf"))
    lse = torch.logsumexp(z, -1)
    w = torch.exp(z - lse.nan_to_num(0.0, neginf=0.0)[..., None]).masked_fill(~see, 0.0)
    back = lambda y: y.permute(2, 0, 1, 3).reshape(T, Hq, hd)
    return (back(w @ v[:, None]), lse.permute(2, 0, 1).reshape(T, Hq), back(w @ v.abs()[:, None]),
            back((w ** 2) @ (v ** 2)[:, None]))


def check(got, lse, q, cache, layer, n, W, parents, prefix, lens, groups, first=None, scale=None, only=None, start=None,
          crow=None):
    B, T, Hq, hd = q.shape
    scale = hd ** -0.5 if scale is None else scale
    for b in range(B):
        if only is not None and b not in only:
            continue
        p = next((i for i in range(len(lens)) if groups[i] <= b < groups[i + 1]), None)
        m = 0 if p is None else int(lens[p])
        f = 0 if p is None or first is None else int(first[p])
        pr = 0 if p is None or prefix.shape[2] == 1 else p
        lo = W - n[b] if start is None else start[b]
        r = b if crow is None else crow
        par = TO.chain(T) if parents is None else parents[b]
        see = torch.zeros(T, m + n[b] - 1 + T, dtype=torch.bool)
        for t in range(T):
            line = TO.line_of(par, t)
            if line:
                see[t, :m + n[b] - 1] = True
                see[t, [m + n[b] - 1 + j for j in line]] = True
        see = see.to(DEV)
        k, v = (torch.cat((prefix[layer, j, pr, :, f:f + m], cache[layer, j, r, :, lo:lo + n[b] - 1 + T]), 1).double()
                for j in (0, 1))
        hidden = ~see.any(0)
        k[:, hidden] = 0
        v[:, hidden] = 0
        out, ls, sums, squares = whole(q[b].double(), k, v, see, scale)
        big = float(k.abs().sum(-1).max() * q[b].double().abs().max()) * abs(scale)
        eps = 2 * (hd + 4) * 2.0 ** -24 * big + 2 * 2.0 ** -20 + (m + n[b] + T) * 2.0 ** -24
        tol = eps * sums + 1e-30
        if q.dtype == torch.bfloat16:
            tol = tol + 7 * 2.0 ** -8 * squares.sqrt() + 2.0 ** -8 * out.abs()
        used = see.any(-1)
        assert (got[b][~used] == 0).all() and torch.isneginf(lse[b][~used]).all()
        bad = ~((got[b].double() - out).abs() <= tol)[used]
        assert not bad.any(), (b, float((got[b].double() - out)[used].abs().max()), float(bad.double().mean()))
        near = (lse[b].double() - ls)[used].abs() <= 2 * eps + 2.0 ** -20 * (1 + ls[used].abs())
        assert near.all()


def inputs(seed, B, T, Hq, H, hd, n, dtype, P, lens, first=None, arena=None, slack=5):
    W = int(max(n)) + 2
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randn(B, T, Hq, hd, generator=g, device=DEV).to(dtype)
    cache = torch.randn(2, 2, B, H, W + T + slack, hd, generator=g, device=DEV).to(dtype)
    cols = arena or max(list(lens) + [1]) + slack
    prefix = torch.randn(2, 2, 1 if arena else P, H, cols, hd, generator=g, device=DEV).to(dtype)
    # NaN wherever nothing may be read
    used = torch.zeros(prefix.shape[2], cols, dtype=torch.bool, device=DEV)
    for p in range(P):
        f = 0 if first is None else first[p]
        used[0 if arena else p, f:f + lens[p]] = True
    prefix.permute(2, 4, 0, 1, 3, 5)[~used] = float("nan")
    prefix[0] = float("nan")
    for b in range(B):
        cache[:, :, b, :, :W - n[b]] = float("nan")
        cache[:, :, b, :, W - 1 + T:] = float("nan")
    cache[0] = float("nan")
    return q, cache, W, prefix


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,T,Hq,H,hd,lens,groups,tree", [
    (2, 1, 4, 2, 64, [100], [0, 2], False),                   # single tokens
    (1, 1, 2, 2, 16, [33], [0, 1], False),                    # one row, the smallest head
    (3, 1, 8, 8, 128, [700], [0, 3], False),                  # one query head per K/V head
    (8, 2, 8, 4, 64, [1500], [0, 8], False),                  # 32 query rows
    (6, 3, 8, 2, 128, [257, 64], [0, 2, 6], True),            # 72 query rows, two prefixes
    (9, 16, 8, 2, 128, [300, 1, 129], [0, 5, 6, 9], True),    # several units of a prefix, the last ragged
    (4, 32, 16, 1, 64, [900], [0, 4], True),                  # 2048 query rows
    (5, 7, 6, 2, 64, [150, 80], [1, 3, 4], True),             # rows before and behind the groups; 3 heads a K/V head
    (4, 4, 4, 4, 80, [50], [0, 4], True),                     # other head sizes
    (3, 5, 4, 2, 256, [65, 40], [0, 1, 3], True),
    (40, 1, 4, 2, 96, [77, 0, 31], [0, 13, 20, 40], False),   # a prefix without columns
    (7, 2, 4, 2, 128, [40, 50, 60], [0, 3, 3, 7], False),     # a group without rows
    (64, 1, 32, 8, 128, [2000], [0, 64], False),
    (5, 32, 32, 8, 128, [700, 129], [1, 3, 4], True),         # rows whose own queries fill tiles, of no group too
    (6, 64, 8, 2, 64, [0, 257], [0, 2, 6], True),
])
def test_against_the_definition(dtype, B, T, Hq, H, hd, lens, groups, tree):
    rng = np.random.default_rng(B * T + hd)
    n = rng.integers(1, 200, B)
    n[0] = 1
    par = random_parents(rng, B, T, unused=0.15) if tree else None
    q, cache, W, prefix = inputs(B + hd, B, T, Hq, H, hd, n, dtype, len(lens), lens)
    out, lse, st = run(q, cache, 1, n, W, par, prefix, lens, groups)
    assert st == 0
    check(out, lse, q, cache, 1, n, W, par, prefix, lens, groups)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,T,G,hd", [(2, 1, 1, 64), (5, 1, 1, 128), (7, 2, 2, 64), (9, 8, 2, 128), (5, 16, 4, 64), (3, 32, 4, 128), (3, 25, 8, 64), (2, 64, 9, 64)])
@pytest.mark.parametrize("cols", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 511])
def test_tile_borders(dtype, B, T, G, hd, cols):
    lens, n = [cols, max(1, cols - 1)], np.arange(1, B + 1)
    groups = [0, (B + 1) // 2, B]
    q, cache, W, prefix = inputs(cols, B, T, G, 1, hd, n, dtype, 2, lens)
    out, lse, st = run(q, cache, 1, n, W, None, prefix, lens, groups)
    assert st == 0
    check(out, lse, q, cache, 1, n, W, None, prefix, lens, groups)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,T,Hq,H,hd,cols", [(2, 1, 4, 2, 128, 40000), (16, 1, 8, 2, 128, 20000), (33, 5, 8, 1, 64, 9000)])
def test_long_prefixes_are_split(dtype, B, T, Hq, H, hd, cols):
    n = np.random.default_rng(B).integers(1, 60, B)
    q, cache, W, prefix = inputs(B, B, T, Hq, H, hd, n, dtype, 1, [cols])
    one = run(q, cache, 1, n, W, None, prefix, [cols], [0, B])
    assert one[2] == 0
    check(one[0], one[1], q, cache, 1, n, W, None, prefix, [cols], [0, B])
    two = run(q, cache, 1, n, W, None, prefix, [cols], [0, B])
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])      # bit for bit


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,Hq,H,hd", [(1, 4, 2, 64), (6, 8, 2, 128), (20, 16, 1, 64), (16, 16, 1, 128), (3, 2, 2, 48)])
def test_a_pool_and_prefixes_in_an_arena(dtype, T, Hq, H, hd):
    """Prefixes and rows anywhere in one cache row each."""
    rng = np.random.default_rng(T)
    B, lens, first = 5, [130, 60, 7], [11, 300, 150]
    n, cols = rng.integers(1, 40, B), np.arange(B) * (40 + T) + 3
    q, _, _, prefix = inputs(T, B, T, Hq, H, hd, n, dtype, 3, lens, first=first, arena=400)
    arena = torch.randn(2, 2, 1, H, B * (40 + T) + 10, hd, generator=torch.Generator().manual_seed(3)).to(dtype).to(DEV)
    order = rng.permutation(B)
    groups = [0, 2, 4, 5]
    out, lse, st = run(q, arena, 1, n, None, None, prefix, lens, groups, first=first, rows=order, first_col=cols)
    assert st == 0
    check(out, lse, q, arena, 1, n[order], None, None, prefix, lens, groups, first=first, start=cols[order], crow=0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
@pytest.mark.parametrize("B,T", [(2, 1), (6, 9), (9, 32), (3, 64)])
def test_scales(dtype, scale, B, T):
    n, lens = np.full(B, 30), [200]
    q, cache, W, prefix = inputs(7, B, T, 4, 2, 64, n, dtype, 1, lens)
    out, lse, st = run(q, cache, 1, n, W, None, prefix, lens, [0, B], scale=scale)
    assert st == 0
    check(out, lse, q, cache, 1, n, W, None, prefix, lens, [0, B], scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("far", [0, 1])
@pytest.mark.parametrize("B,T", [(2, 1), (6, 9), (9, 32), (3, 64)])
def test_one_part_far_above_the_other(dtype, far, B, T):
    """Scores of one part a hundred above the other's: the other's weights vanish, and nothing overflows."""
    n, lens = np.full(B, 20), [150]
    q, cache, W, prefix = inputs(8, B, T, 4, 2, 64, n, dtype, 1, lens)
    direction = torch.sign(q.float().mean((0, 1, 2)))
    q.copy_((q.float().abs() * direction).to(dtype))
    t = (prefix, cache)[far]
    t[1, 0] = (t[1, 0].float().nan_to_num(0.0).abs() * direction * 16).to(dtype)
    out, lse, st = run(q, cache, 1, n, W, None, prefix, lens, [0, B], scale=0.5)
    assert st == 0 and torch.isfinite(out).all()
    check(out, lse, q, cache, 1, n, W, None, prefix, lens, [0, B], scale=0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,T,hd", [(2, 1, 64), (6, 9, 128), (9, 32, 64), (4, 64, 128), (3, 4, 96)])
def test_values_that_are_not_finite_stay_in_their_place(dtype, B, T, hd):
    n, lens = np.full(B, 10), [70, 90]
    groups = [0, B // 2, B]
    q, cache, W, prefix = inputs(9, B, T, 4, 2, hd, n, dtype, 2, lens)
    clean = run(q, cache, 1, n, W, None, prefix, lens, groups)
    prefix[1, 1, 1, 0, 33, 5] = float("inf")
    prefix[1, 1, 1, 1, 89, 7] = float("nan")
    out, lse, st = run(q, cache, 1, n, W, None, prefix, lens, groups)
    assert st == 0 and torch.equal(lse, clean[1])
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[B // 2:, :, :2, 5] = True
    hit[B // 2:, :, 2:, 7] = True
    assert not torch.isfinite(out[hit]).any() and torch.equal(out[~hit], clean[0][~hit])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
def test_strides_other_streams_and_a_captured_graph(dtype):
    import speculative_decoding_specdec_gb300.specdec as sd
    B, T, Hq, H, hd = 6, 5, 8, 2, 64
    n, lens, groups = np.arange(3, 3 + B), [300, 20], [0, 4, 6]
    q0, cache, W, prefix = inputs(4, B, T, Hq, H, hd, n, dtype, 2, lens)
    buf = torch.zeros(B, T, 3 * Hq * hd, dtype=dtype, device=DEV)
    q, out = buf[:, :, :Hq * hd].unflatten(2, (Hq, hd)), buf[:, :, Hq * hd:2 * Hq * hd].unflatten(2, (Hq, hd))
    lse, st = torch.zeros(B, T, Hq, device=DEV), status()
    ws = torch.zeros(sd.prefix_attention_workspace_bytes(q, cache, 2), dtype=torch.uint8, device=DEV)
    args = (i32(n), i32([W]), None, st, ws, prefix, i32(lens), i32(groups))
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        sd.prefix_attention(q, cache, 1, out, *args, lse=lse)
    for k in range(3):
        q.copy_(q0 * (1 + k))
        graph.replay()
        torch.cuda.synchronize()
        check(out, lse, q, cache, 1, n, W, None, prefix, lens, groups)
    assert int(st) == 0 and (buf[:, :, 2 * Hq * hd:] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
def test_one_workspace_serves_every_shape(dtype):
    """The largest shape's workspace, used for others and for the attention without a prefix in between."""
    import speculative_decoding_specdec_gb300.specdec as sd
    shapes = [(9, 32, 16, 1, 64), (2, 1, 4, 2, 64), (33, 1, 8, 2, 128), (3, 4, 4, 4, 80), (7, 5, 8, 2, 128)]
    ws = torch.zeros(max(sd.prefix_attention_workspace_bytes(torch.empty(B, T, Hq, hd, dtype=dtype),
                                                             torch.empty(1, 2, B, H, 1, hd), 2)
                         for B, T, Hq, H, hd in shapes), dtype=torch.uint8, device=DEV)
    for B, T, Hq, H, hd in shapes + shapes[::-1]:
        n, lens, groups = np.full(B, 50), [1000, 30], [0, B // 2 + 1, B]
        q, cache, W, prefix = inputs(B, B, T, Hq, H, hd, n, dtype, 2, lens)
        out, lse, st = run(q, cache, 1, n, W, None, prefix, lens, groups, ws=ws)
        assert st == 0
        check(out, lse, q, cache, 1, n, W, None, prefix, lens, groups)
        a, b, s = torch.zeros_like(q), torch.zeros_like(q), status()
        sd.tree_attention(q, cache, 1, a, i32(n), i32([W]), None, s, ws)
        fresh = torch.zeros(sd.tree_attention_workspace_bytes(q, cache), dtype=torch.uint8, device=DEV)
        sd.tree_attention(q, cache, 1, b, i32(n), i32([W]), None, s, fresh)
        torch.cuda.synchronize()
        assert int(s) == 0 and torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
def test_without_prefixes_it_is_the_attention_of_a_tree(dtype):
    import speculative_decoding_specdec_gb300.specdec as sd
    for B, T, Hq, H, hd in ((2, 1, 4, 2, 64), (5, 9, 8, 2, 128), (3, 32, 16, 1, 64)):
        n = np.full(B, 77)
        q, cache, W, prefix = inputs(1, B, T, Hq, H, hd, n, dtype, 1, [4])
        a, st = torch.zeros_like(q), status()
        ws = torch.zeros(sd.prefix_attention_workspace_bytes(q, cache, 1), dtype=torch.uint8, device=DEV)
        sd.tree_attention(q, cache, 1, a, i32(n), i32([W]), None, st, ws)
        for lens, groups in (([], [0]), ([0], [0, B]), ([4], [0, 0]), ([4], [B, B])):
            out, _, code = run(q, cache, 1, n, W, None, prefix, lens, groups, ws=ws)
            assert code == 0 and torch.equal(out, a)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,T,hd", [(4, 1, 64), (6, 9, 128), (9, 32, 64), (5, 50, 64), (4, 3, 96)])
@pytest.mark.parametrize("lens,first,groups,code,written", [
    ([50, -1], None, [0, 2, 4], 5, [0, 1]),             # a negative length
    ([50, 70], [0, -3], [0, 2, 4], 5, [0, 1]),          # a negative first column
    ([50, 91], None, [0, 2, 4], 4, [0, 1]),             # beyond the cache
    ([50, 40], [0, 60], [0, 2, 4], 4, [0, 1]),
    ([50, 2 ** 31 - 1], [0, 2 ** 31 - 1], [0, 2, 4], 4, [0, 1]),
    ([91, 50], None, [0, 0, 4], 4, [0, 1, 2, 3]),       # of a group without rows: reported alone
    ([50, 70], None, [0, 3, 2], 5, []),                 # bounds that descend
    ([50, 70], None, [-1, 2, 4], 5, []),
    ([50, 70], None, [0, 2, 2000], 5, []),
])
def test_bad_groups_are_told_and_not_written(dtype, B, T, hd, lens, first, groups, code, written):
    n, ok = np.full(B, 10), [90, 90]
    groups = [B if x == 4 else x for x in groups]
    q, cache, W, prefix = inputs(5, B, T, 4, 2, hd, n, dtype, 2, ok, slack=0)
    out, lse, st = run(q, cache, 1, n, W, None, prefix, lens, groups, first=first)
    assert st == code
    written = [b for b in range(B) if b in written or (len(written) == 4 and b < B)]
    left = [b for b in range(B) if b not in written]
    assert (out[left] == 7).all()
    check(out, lse, q, cache, 1, n, W, None, prefix, lens, groups, first=first, only=written)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
def test_a_bad_row_leaves_the_others(dtype):
    n, W, lens = np.array([5, 0, 9, 6]), 9, [40]
    q, cache, _, prefix = inputs(6, 4, 3, 4, 2, 64, np.array([5, 9, 9, 6]), dtype, 1, lens)
    out, lse, st = run(q, cache, 1, n, 9, None, prefix, lens, [0, 4])
    assert st == 5 and (out[1] == 7).all()
    assert (out[[0, 2, 3]] != 7).any()


def fake(sd, **kw):
    F, s = 1 << 20, 16 * 32 * 2
    view = lambda rows, **k: sd.KvView(F, 2 * s * rows, s * rows, s, 16 * 32, k.get("dtype", sd.F32), k.get("layers", 1), rows,
                                       k.get("heads", 2), k.get("hd", 16), 32)
    a = sd.PrefixAttentionArgs(P=1, prefix=view(1), prefix_len=F, group_start=F)
    o = a.own
    o.cache, o.B, o.T, o.heads_q, o.scale, o.workspace_bytes = view(2), 2, 1, 2, 1.0, 0
    for f in ("q", "out", "n_committed", "width", "workspace", "dev_status"):
        setattr(o, f, F)
    for f, v in kw.items():
        if f == "view":
            a.prefix = view(**v)
        elif hasattr(o, f) and f not in ("prefix",):
            setattr(o, f, v)
        else:
            setattr(a, f, v)
    return a


def test_host_checks():
    """Refused before anything is launched, so no GPU is needed (a workspace of no bytes refuses the rest)."""
    import speculative_decoding_specdec_gb300.specdec as sd
    f = sd.lib.specdec_prefix_attention
    assert f(None, None) == sd.ERR_INVALID_ARG
    for kw in (dict(P=-1), dict(prefix_len=None), dict(group_start=None), dict(prefix_len=(1 << 20) + 2),
               dict(prefix_first=(1 << 20) + 1), dict(view=dict(rows=1, heads=1)), dict(view=dict(rows=1, hd=32)),
               dict(view=dict(rows=1, dtype=sd.BF16)), dict(view=dict(rows=1, dtype=7)), dict(P=2), dict(q=None),
               dict(layer=1), dict(scale=float("nan")), dict(dev_status=None)):
        assert f(ctypes.byref(fake(sd, **kw)), None) == sd.ERR_INVALID_ARG, kw
    for kw in (dict(P=513), dict(T=65), dict(B=1025), dict(view=dict(rows=1, hd=6))):
        assert f(ctypes.byref(fake(sd, **kw)), None) == sd.ERR_UNSUPPORTED, kw
    assert f(ctypes.byref(fake(sd, B=0)), None) == sd.OK
    size = sd.lib.specdec_prefix_attention_workspace
    for bad in ((9, 2, 1, 2, 2, 16, 1), (sd.F32, 0, 1, 2, 2, 16, 1), (sd.F32, 2, 1, 3, 2, 16, 1), (sd.F32, 2, 1, 2, 2, 16, -1),
                (sd.F32, 2, 1, 2, 2, 16, 513)):
        assert size(*bad) == 0
    assert size(sd.F32, 2, 1, 2, 2, 16, 1) >= sd.lib.specdec_tree_attention_workspace(sd.F32, 2, 1, 2, 2, 16)


def test_struct_layout_and_packing(tmp_path):
    import os
    import subprocess
    import speculative_decoding_specdec_gb300.specdec as sd
    names = {"specdec_prefix_attention_args": sd.PrefixAttentionArgs, "specdec_norm_rotary_args": sd.NormRotaryArgs,
             "specdec_sample_args": sd.SampleArgs}
    lines = [f'printf("{c} %zu\\n", sizeof({c}));' for c in names]
    lines += [f'printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for c, py in names.items() for f, _ in py._fields_]
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "specdec.h"\nint main(void) {' + "\n".join(lines) + "return 0; }")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(x.rsplit(" ", 1) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n") if x)
    for c, py in names.items():
        assert int(got[c]) == ctypes.sizeof(py)
        for f, _ in py._fields_:
            assert int(got[f"{c}.{f}"]) == getattr(py, f).offset, (c, f)
    flat = lambda s: [x for f, t in s._fields_ for x in (flat(getattr(s, f)) if hasattr(t, "_fields_") else [getattr(s, f)])]
    for py, fmt in ((sd.PrefixAttentionArgs, sd._PACK_PREFIX), (sd.NormRotaryArgs, sd._PACK_NORM_ROTARY), (sd.SampleArgs, sd._PACK_SAMPLE)):
        values = list(range(1, len(fmt.unpack(bytes(fmt.size))) + 1))
        assert flat(py.from_buffer_copy(fmt.pack(*values).ljust(ctypes.sizeof(py), b"\0"))) == values
