"""Rows of scores that draw the same wherever they lie, what is too light to be drawn, and top-p beside
min-p.

A row's sums are those of its tokens in groups of 16 bytes counted from its first token, so nothing that
the row writes depends on its address or its neighbours: equal bit for bit.  DELTA is derived in
test_gpu_sample.
"""
import numpy as np
import pytest
import torch

import oracle.sample_oracle as SO
import test_gpu_sample as SA
from tree_testlib import DEV, i32, status

DT = [torch.float32, torch.bfloat16]


def draw(x, u, **kw):
    """(token, logprob, bounds) of x [R, V] on the device, settings given once for all rows."""
    import speculative_decoding_specdec_gb300.specdec as sd
    R = x.shape[0]
    token, lp, kb, st = i32(np.full(R, -7)), SA.f32(7.0, R), i32(np.full((R, 2), -7)), status()
    given = {k: i32(np.full(R, v)) if k == "top_k" else SA.f32(v, R) for k, v in kw.items()}
    sd.sample(x, u, token, st, logprob=lp, keep_bounds=kb, **given)
    torch.cuda.synchronize()
    assert int(st) == 0
    return token, lp.view(torch.int32), kb


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("V", [3, 9, 37, 1001, 20011, 151553])
@pytest.mark.parametrize("kw", [dict(), dict(temperature=0.7, top_p=0.9), dict(top_k=40), dict(min_p=1e-4),
                                dict(temperature=0.0)])
def test_a_row_draws_the_same_at_any_address(dtype, V, kw):
    R = 4
    x = SA.scores(R, V, V, spread=2.5, dtype=dtype).to(DEV)
    u = SA.f32([0.02, 0.4, 0.75, 0.999], R)
    want = draw(x, u, **kw)
    for lead in range(9):
        for gap in (0, 1, 5):
            buf = torch.full((R * (V + gap) + lead + 16,), float("nan"), dtype=dtype, device=DEV)
            z = buf[lead:lead + R * (V + gap)].view(R, V + gap)[:, :V]
            z.copy_(x)
            got = draw(z, u, **kw)
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (lead, gap)
    for r in range(R):                           # alone, and as the last of many
        many = torch.cat((x.roll(1, 0).repeat(40, 1), x[r:r + 1]))
        for z in (x[r:r + 1].clone(), many):
            got = draw(z, u[r].expand(len(z)).contiguous(), **kw)
            assert all(torch.equal(a[-1], b[r]) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("lead", [0, 1])
def test_what_is_too_light_to_be_drawn(dtype, lead):
    """Groups of 16 bytes, in all below 2^-42 of the highest, have no share; those above have theirs in
    whole 2^-42."""
    N = 16 // dtype.itemsize
    x = torch.full((3, 6 * N + 1), float("-inf"), dtype=torch.float64)
    x[:, 5 * N] = 0.0
    x[0, :N] = -60 * np.log(2)                   # N of 2^-60
    x[1, :N] = -60 * np.log(2)
    x[1, 2 * N + 1] = -30 * np.log(2)            # 2^-30, alone
    x[2, :N] = -41 * np.log(2)                   # N of 2^-41
    buf = torch.zeros(3 * x.shape[1] + lead, dtype=dtype, device=DEV)
    z = buf[lead:].view(x.shape)
    z.copy_(x.to(dtype))
    token, _, _ = draw(z, SA.f32(0.0, 3))
    assert token.tolist() == [5 * N, 2 * N + 1, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("V", [50, 5003, 151936])
def test_top_p_cuts_beside_min_p(dtype, V):
    """A cut by top-p that lies above min-p's: before the last kept token there is less than top_p of the
    mass of what top-k kept, and up to it at least that."""
    import speculative_decoding_specdec_gb300.specdec as sd
    R, d = 12, SA.delta(V)
    x = SA.scores(R, V, 3 * V, spread=0.5, likely=20, dtype=dtype)
    top_p = np.tile([0.3, 0.6, 0.8], 4).astype(np.float32)
    top_k = np.repeat([0, max(2, V // 2), 15, V], 3)
    min_p = np.float32(1e-3)
    token, kb, st = i32(np.zeros(R)), i32(np.zeros((R, 2))), status()
    sd.sample(x.to(DEV), SA.f32(0.5, R), token, st, top_p=SA.f32(top_p, R), min_p=SA.f32(min_p, R), top_k=i32(top_k),
              keep_bounds=kb)
    torch.cuda.synchronize()
    assert int(st) == 0
    bounds, tighter = kb.cpu().numpy(), 0
    for r in range(R):
        row = x[r].double().numpy()
        keep = set(SO.keep_from_bound(row, np.uint32(bounds[r, 0].astype(np.int64) & 0xFFFFFFFF), bounds[r, 1]))
        of_k = SO.kept(row, 1.0, int(top_k[r]))
        other = SO.kept(row, 1.0, int(top_k[r]), 1.0, float(min_p))
        n = len(keep)
        assert 0 < n and keep == set(of_k[:n]) and n <= len(other)
        e = SO.masses(row, 1.0)[of_k]
        assert e[:n - 1].sum() / e.sum() < top_p[r] + d
        if n < len(other):
            assert e[:n].sum() / e.sum() >= top_p[r] - d
            tighter += 1
    assert tighter >= 6


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,V", [(torch.float32, 358399), (torch.bfloat16, 716799)])
def test_the_longest_rows_at_any_address(dtype, V):
    """Sixteen CTAs to a row, whose parts end anywhere in memory's 16 bytes."""
    x = SA.scores(2, V, 1, dtype=dtype)
    for lead in (0, 1, 3):
        for kw in (dict(), dict(top_p=0.9), dict(top_k=[50, V - 1], min_p=0.01)):
            SA.run(x, [0.3, 0.999], lead=lead, **kw)
