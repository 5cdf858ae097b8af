"""Norms of q's and k's heads with rotary positions and the append, against a float64 form.

Tolerance, relative to |x1| + |x2| of the normed pair: the sum of squares takes at most 16 products
and sums in a lane and 5 sums across lanes, so it is off by at most 21 * 2^-24, half of which enters
its inverse root, whose own error is at most 2 ulp (4 * 2^-24); the factor 1 / head_dim and eps are
one rounding each (half again); x * inv, offset + w and their product three more, and the rotation
three: under 24 * 2^-24 in all.  bf16 results are rounded once more, 2^-8 of the value.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle.tree_oracle as TO
from tree_testlib import DEV, i32, numpy64, random_parents, status


def normed(x, w, eps, offset):
    """x [.., hd] float64; w [hd] or None."""
    if w is None:
        return np.array(x)
    return x / np.sqrt((x ** 2).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * (offset + w)


def close(got, y, cos, sin, interleaved, dtype):
    want = TO.rotate(y, cos, sin, interleaved)
    half = len(cos)
    pair = np.abs(y).copy()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    both = pair[..., a] + pair[..., b]
    pair[..., a] = both
    pair[..., b] = both
    tol = 24 * 2.0 ** -24 * pair
    if dtype == torch.bfloat16:
        tol = tol * 1.01 + 2.0 ** -8 * np.abs(want) + 2.0 ** -133
    assert (np.abs(got - want) <= tol).all()


def run(B, T, Hq, H, hd, rot, dtype, interleaved=False, parents=None, offset=0.0, eps=1e-6, start=None,
        q_norm=True, k_norm=True, wdtype=None, explicit=None, extra=0, in_place=False, seed=0, unaligned_w=False):
    import speculative_decoding_specdec_gb300.specdec as sd
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    buf = (2.5 * torch.randn(B, T, (Hq + 2 * H) * hd + extra, generator=gen)).to(dtype).to(DEV)
    q = buf[:, :, :Hq * hd].unflatten(2, (Hq, hd))
    k = buf[:, :, Hq * hd:(Hq + H) * hd].unflatten(2, (H, hd))
    v = buf[:, :, (Hq + H) * hd:(Hq + 2 * H) * hd].unflatten(2, (H, hd))
    n = rng.integers(1, 30, B)
    W = int(n.max()) + 2
    cap = W + T
    cache = torch.randn(2, 2, B, H, cap, hd, generator=gen).to(dtype).to(DEV)
    before = numpy64(cache)
    P = cap + (0 if start is None else max(start))
    angle = np.arange(P)[:, None] * 1e4 ** (-np.arange(rot // 2) / (rot // 2))
    table = torch.as_tensor(np.stack((np.cos(angle), np.sin(angle)), -1), dtype=torch.float32).to(DEV)
    w = []
    for on in (q_norm, k_norm):
        x = torch.randn(hd + 1, generator=gen).to(wdtype or dtype).to(DEV)
        w.append((x[1:] if unaligned_w else x[:-1].clone()) if on else None)
    q0, k0, v0 = numpy64(q), numpy64(k), numpy64(v)
    out = q if in_place else torch.full((B, T, Hq, hd), 7.0, dtype=dtype, device=DEV)
    st = status()
    if explicit:
        pos = rng.integers(0, cap, (B, T))
        col = np.stack([rng.permutation(cap)[:T] for _ in range(B)])
        col[rng.random((B, T)) < 0.3] = -1
        where = dict(positions=i32(pos), columns=i32(col))
    else:
        par = [TO.chain(T)] * B if parents is None else parents
        lines = [[TO.line_of(par[b], t) for t in range(T)] for b in range(B)]
        pos = np.array([[n[b] - 2 + len(x) for x in lines[b]] for b in range(B)])
        col = np.array([[W - 1 + t if lines[b][t] else -1 for t in range(T)] for b in range(B)])
        where = dict(n_committed=i32(n), width=i32([W]), parents=None if parents is None else i32(parents))
    sd.norm_rotary_append(q, k, v, cache, 1, table, out, st, w[0], w[1], eps=eps, weight_offset=offset,
                          start=None if start is None else i32(start), interleaved=interleaved, **where)
    torch.cuda.synchronize()
    assert int(st) == 0
    if start is not None:
        pos = pos + np.array(start)[:, None]
    tab, got, after = numpy64(table), numpy64(out), numpy64(cache)
    want = before.copy()
    wq, wk = (None if x is None else numpy64(x) for x in w)
    for b in range(B):
        for t in range(T):
            if col[b, t] < 0:
                assert (got[b, t] == 0).all()
                continue
            cs = tab[pos[b, t]]
            close(got[b, t], normed(q0[b, t], wq, eps, offset), cs[:, 0], cs[:, 1], interleaved, dtype)
            close(after[1, 0, b, :, col[b, t]], normed(k0[b, t], wk, eps, offset), cs[:, 0], cs[:, 1], interleaved, dtype)
            want[1, 0, b, :, col[b, t]] = after[1, 0, b, :, col[b, t]]
            want[1, 1, b, :, col[b, t]] = v0[b, t]
    np.testing.assert_array_equal(after, want)      # nothing else was written


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,Hq,H,hd,rot,interleaved,tree", [
    (2, 1, 4, 2, 64, 64, False, False),
    (1, 1, 1, 1, 16, 2, True, False),       # one token, one pair
    (3, 7, 6, 3, 64, 32, True, True),       # part of the head, interleaved pairs
    (2, 64, 8, 2, 128, 128, False, True),   # the largest tree
    (2, 9, 5, 1, 80, 20, False, True),      # pairs that no 16-byte vector divides
    (2, 3, 3, 3, 96, 96, False, True),      # lanes of a head that stay without values
    (1, 5, 33, 7, 256, 64, True, False),    # heads that fill no CTA
    (2, 2, 3, 1, 512, 512, False, False),   # the largest head
    (1, 2, 2, 1, 504, 8, False, False),     # the most scalars
])
def test_verification_pass(dtype, B, T, Hq, H, hd, rot, interleaved, tree):
    par = random_parents(np.random.default_rng(T), B, T, unused=0.2) if tree else None
    run(B, T, Hq, H, hd, rot, dtype, interleaved, par)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", [
    dict(offset=1.0), dict(q_norm=False), dict(k_norm=False), dict(q_norm=False, k_norm=False),
    dict(wdtype=torch.float32), dict(wdtype=torch.bfloat16), dict(unaligned_w=True), dict(start=[0, 17, 5]),
    dict(explicit=True), dict(explicit=True, start=[3, 0, 900]), dict(extra=1), dict(extra=8, in_place=True),
    dict(extra=1, in_place=True), dict(eps=0.0), dict(eps=1.0)])
def test_variants(dtype, interleaved, case):
    run(3, 11, 4, 2, 64, 64, dtype, interleaved, seed=5, **case)


@pytest.mark.gpu
def test_a_long_prompt():
    run(2, 700, 32, 8, 128, 128, torch.bfloat16, explicit=True, seed=2)


@pytest.mark.gpu
def test_values_that_are_not_finite_stay_in_their_heads():
    import speculative_decoding_specdec_gb300.specdec as sd
    q = torch.randn(1, 1, 4, 64, device=DEV)
    k, v = torch.randn(1, 1, 2, 64, device=DEV), torch.randn(1, 1, 2, 64, device=DEV)
    q[0, 0, 1, 3] = float("nan")
    k[0, 0, 0, 5] = float("inf")
    v[0, 0, 1, 2] = float("nan")
    cache, out, st = torch.zeros(1, 2, 1, 2, 4, 64, device=DEV), torch.zeros_like(q), status()
    table = torch.zeros(4, 32, 2, device=DEV)
    table[..., 0] = 1
    w = torch.ones(64, device=DEV)
    sd.norm_rotary_append(q, k, v, cache, 0, table, out, st, w, w, n_committed=i32([2]), width=i32([2]))
    torch.cuda.synchronize()
    assert int(st) == 0
    good = torch.isfinite(out[0, 0]).all(-1).tolist()
    assert good == [True, False, True, True]
    assert torch.isfinite(cache[0, 0, 0, 1, 1]).all() and not torch.isfinite(cache[0, 0, 0, 0, 1]).all()
    assert torch.equal(cache[0, 1, 0, :, 1].isnan(), v[0, 0].isnan())


@pytest.mark.gpu
@pytest.mark.parametrize("start,code", [([-1, 0], 5), ([0, 6], 5), ([0, 2 ** 31 - 1], 5), ([0, 5], 0)])
def test_starts_out_of_range(start, code):
    import speculative_decoding_specdec_gb300.specdec as sd
    q, k = torch.randn(2, 1, 2, 16, device=DEV), torch.randn(2, 1, 1, 16, device=DEV)
    cache, out, st = torch.zeros(1, 2, 2, 1, 4, 16, device=DEV), torch.full_like(q, 7.0), status()
    table, w = torch.ones(8, 8, 2, device=DEV), torch.ones(16, device=DEV)
    sd.norm_rotary_append(q, k, k, cache, 0, table, out, st, w, w, n_committed=i32([3, 3]), width=i32([3]),
                          start=i32(start))
    torch.cuda.synchronize()
    assert int(st) == code
    for b, s in enumerate(start):
        bad = not 0 <= s <= 5
        assert bool((out[b] == 7).all()) == bad and bool((cache[:, :, b] == 0).all()) == bad


def test_host_checks():
    """Refused before anything is launched, so no GPU is needed."""
    import speculative_decoding_specdec_gb300.specdec as sd
    fake = 1 << 20
    f = sd.lib.specdec_norm_rotary_append
    assert f(None, None) == sd.ERR_INVALID_ARG

    def call(base=(), B=1, **kw):
        s = 16 * 16 * 2
        a = sd.NormRotaryArgs(q_weight=fake, k_weight=fake, weight_dtype=sd.F32, eps=1e-6)
        r = a.rotary
        r.cache = sd.KvView(fake, 2 * s, s, s, 256, sd.F32, 1, 1, 2, 16, 16)
        r.B, r.T, r.heads_q, r.rot_dim, r.table_len = B, 1, 2, 16, 8
        for name in ("q", "k", "v", "q_out", "table", "dev_status", "n_committed", "width"):
            setattr(r, name, fake)
        for name, x in base:
            setattr(r, name, x)
        for name, x in kw.items():
            setattr(a, name, x)
        return f(ctypes.byref(a), None)

    assert call(B=0) == sd.OK
    for kw in (dict(weight_dtype=2), dict(q_weight=fake + 2), dict(k_weight=fake + 1), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(weight_offset=float("inf")), dict(start=fake + 2),
               dict(base=[("q", None)]), dict(base=[("rot_dim", 17)]), dict(base=[("T", 0)]), dict(B=-1)):
        assert call(**kw) == sd.ERR_INVALID_ARG, kw
    assert call(base=[("T", 65)]) == sd.ERR_UNSUPPORTED


def test_binding_wants_cuda_tensors_of_one_type():
    import speculative_decoding_specdec_gb300.specdec as sd
    cache, q = torch.zeros(1, 2, 1, 2, 4, 8), torch.zeros(1, 1, 2, 8)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        sd.norm_rotary_append(q, q, q, cache, 0, torch.zeros(4, 4, 2), q, i, q[0, 0, 0], q[0, 0, 0],
                              n_committed=i, width=i)
