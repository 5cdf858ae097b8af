"""Tokens drawn with sampling settings, against the float64 oracle.

Tolerances.  A mass 2^-z is off by ex2's 2^-22 of itself (2 ulp) and by z's error times ln 2: the
difference of scores, its product with log2(e) / T and that factor's second float are three roundings,
3 * 2^-24 of z.  Summed over the row, with sum p z <= log2 V (the entropy of the probabilities p is
log2(sum of masses) + sum p z, the highest mass being 1, and at most log2 V), that is 3 ln 2 log2(V)
2^-24 of the sum.  A vector's sum takes 7 additions, and whole numbers drop 2^-42 each.  So a running mass
over the kept mass is off by at most DELTA(V), twice all that: a token is right if u lies within DELTA of
its interval, and a top-p cut if top_p does.  A log probability is -(z ln 2 + log1p(sum - 1)), both terms
of one sign and in fp32: z takes the three roundings, ln 2 and the fused product and sum two more, sum - 1
one and log1p one ulp (two): under 6 * 2^-24 of itself, besides DELTA in the sum.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle.sample_oracle as SO
from tree_testlib import DEV, i32, status


def delta(V):
    return 2 * (2.0 ** -22 + 3 * np.log(2) * np.log2(max(V, 2)) * 2.0 ** -24 + 7 * 2.0 ** -24 + V * 2.0 ** -42)


def f32(x, R):
    return torch.as_tensor(np.broadcast_to(np.asarray(x, np.float32), (R,)).copy()).to(DEV)


def run(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, lead=0, gap=0, exact_set=False):
    """x [R, V] tensor on the host; checks every row."""
    import speculative_decoding_specdec_gb300.specdec as sd
    R, V = x.shape
    buf = torch.full((R * (V + gap) + lead,), 1e30, dtype=x.dtype, device=DEV)
    z = buf[lead:].view(R, V + gap)[:, :V]
    z.copy_(x)
    bounds = torch.full((R, 3, 2), -7, dtype=torch.int32, device=DEV)
    token, logprob, st = i32(np.full(R, -7)), f32(7.0, R), status()
    k = np.broadcast_to(np.asarray(top_k, np.int32), (R,))
    args = dict(temperature=np.broadcast_to(np.float32(temperature), (R,)), top_p=np.broadcast_to(np.float32(top_p), (R,)),
                min_p=np.broadcast_to(np.float32(min_p), (R,)))
    off = dict(temperature=1.0, top_p=1.0, min_p=0.0)
    given = {n: None if (v == off[n]).all() else f32(v, R) for n, v in args.items()}
    uu = np.broadcast_to(np.asarray(u, np.float32), (R,))
    sd.sample(z, f32(uu, R), token, st, top_k=None if (k == 0).all() else i32(k), logprob=logprob,
              keep_bounds=bounds[:, 1], **given)
    torch.cuda.synchronize()
    assert int(st) == 0
    host, got, lp, kb = x.double().numpy(), token.cpu().numpy(), logprob.cpu().numpy(), bounds.cpu().numpy()
    assert (kb[:, [0, 2]] == -7).all()
    for r in range(R):
        t, p = float(args["temperature"][r]), float(args["top_p"][r])
        row = host[r]
        keep = SO.keep_from_bound(row, np.uint32(kb[r, 1, 0].astype(np.int64) & 0xFFFFFFFF), kb[r, 1, 1])
        sure = SO.kept(row, t, int(k[r]), 1.0, float(args["min_p"][r]))       # without top-p
        if t == 0:
            assert got[r] == sure[0] and lp[r] == 0 and list(keep) == [got[r]]
            continue
        if p >= 1:
            assert set(keep) == set(sure)
        else:
            before_p = SO.kept(row, t, int(k[r]))
            e = SO.masses(row, t)[before_p]
            rank = np.empty(V, np.int64)
            rank[before_p] = np.arange(len(before_p))
            in_order = keep[np.isin(keep, before_p)]
            assert len(in_order) == len(keep) > 0
            at = np.sort(rank[keep])
            assert (at == np.arange(len(at))).all()                            # a beginning of the order
            if args["min_p"][r] > 0 and len(keep) == len(sure):
                pass                                                           # min-p cut it
            else:
                m = e.sum()
                d = delta(V)
                assert e[:len(at) - 1].sum() / m < p + d
                assert e[:len(at)].sum() / m >= p - d
            if args["min_p"][r] > 0:
                assert set(keep) <= set(sure)
        if exact_set:
            assert set(keep) == set(SO.kept(row, t, int(k[r]), p, float(args["min_p"][r])))
        want, _, edges, ids = SO.draw(row, t, keep, uu[r])
        at = int(np.searchsorted(ids, got[r]))
        assert at < len(ids) and ids[at] == got[r], "a token outside the kept set"
        lo, hi = (edges[at - 1] if at else 0.0), edges[at]
        assert lo - delta(V) <= float(uu[r]) <= hi + delta(V), (r, got[r], want)
        e = SO.masses(row, t)
        exact = (row[got[r]] - row.max()) / float(np.float32(t)) - np.log(e[ids].sum())
        assert abs(lp[r] - exact) <= delta(V) + 6 * 2.0 ** -24 * abs(exact) + 2.0 ** -149
    return got, kb


def scores(R, V, seed, spread=1.5, likely=8, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, V, generator=g) * spread
    for _ in range(min(likely, V)):
        x[torch.arange(R), torch.randint(0, V, (R,), generator=g)] = np.log(V) + 2 * torch.randn(R, generator=g)
    return x.to(dtype)


DT = [torch.float32, torch.bfloat16]
SETTINGS = [dict(), dict(top_k=20), dict(top_p=0.9), dict(min_p=0.05), dict(top_k=50, top_p=0.95, min_p=0.02),
            dict(top_k=1000, top_p=0.99), dict(temperature=0.0)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("V", [1, 2, 7, 100, 1000, 4095, 4097, 32000, 151936])
@pytest.mark.parametrize("which", range(len(SETTINGS)))
def test_settings(dtype, V, which):
    R = 5 if V < 100000 else 3
    rng = np.random.default_rng(V + which)
    run(scores(R, V, V + which, dtype=dtype), rng.random(R), **({"temperature": 0.8} | SETTINGS[which]))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("lead,gap", [(1, 0), (0, 1), (3, 5), (8, 16)])
def test_rows_that_begin_anywhere(dtype, lead, gap):
    for V in (1, 5, 999, 20011):
        run(scores(4, V, V, dtype=dtype), [0.0, 0.3, 0.7, 1 - 2.0 ** -24], top_k=30, top_p=0.9, lead=lead, gap=gap)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("R,V", [(300, 1000), (97, 32000), (256, 151552)])
def test_many_rows_with_settings_of_their_own(dtype, R, V):
    rng = np.random.default_rng(R)
    run(scores(R, V, R, dtype=dtype), rng.random(R), temperature=rng.choice([0.0, 0.3, 0.7, 1.0, 2.0], R),
        top_k=rng.choice([0, 1, 40, V // 2, V, V + 5], R), top_p=rng.choice([1.0, 0.5, 0.9, 0.999], R),
        min_p=rng.choice([0.0, 0.1, 1.0], R))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("kind", ["equal", "two", "few", "flat", "steps", "zeros", "near"])
@pytest.mark.parametrize("V", [3000, 50001])
def test_cuts_among_very_many_tokens(dtype, kind, V):
    """A bin of more tokens than the list holds, equal scores among them."""
    g = torch.Generator().manual_seed(V)
    x = {"equal": lambda: torch.full((6, V), 0.37),
         "two": lambda: torch.randint(0, 2, (6, V), generator=g).float(),
         "few": lambda: torch.randint(-3, 3, (6, V), generator=g) * 1e-3,
         "flat": lambda: torch.rand(6, V, generator=g) * 1e-2 + 5,
         "steps": lambda: (torch.arange(V) // 1500).float().expand(6, V) * 1e-4,
         "zeros": lambda: torch.where(torch.rand(6, V, generator=g) < 0.5, 0.0, -0.0),
         "near": lambda: 1e-30 * torch.randn(6, V, generator=g)}[kind]().to(dtype)
    u = [0.0, 0.1, 0.5, 0.9, 0.99999, 1 - 2.0 ** -24]
    run(x, u, top_k=[1, 2, V // 3, V // 2, V - 1, 1025])
    run(x, u, top_p=[1e-6, 0.1, 0.5, 0.9, 0.999, 1 - 2.0 ** -24])
    run(x, u, top_k=[V - 1, V // 2, 1024, 1500, 1501, 1499], top_p=[0.5, 0.9, 0.3, 0.999, 0.7, 0.2])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("temperature", [1e-38, 1e-4, 0.05, 4.0, 1e4, 3e38])
def test_temperatures(dtype, temperature):
    x = scores(4, 5000, 3, dtype=dtype)
    u = [0.0, 0.25, 0.75, 1 - 2.0 ** -24]
    run(x, u, temperature=temperature)
    run(x, u, temperature=temperature, top_k=[3, 0, 2000, 4999])
    run(x, u, temperature=temperature, top_p=0.9, top_k=[0, 5, 0, 3000])
    run(x, u, temperature=temperature, min_p=0.3)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("hidden", [float("-inf"), "lowest"])
def test_masked_tokens(dtype, hidden):
    """Scores of -infinity or the type's lowest value: never drawn, whatever the settings."""
    x = scores(6, 20000, 9, dtype=dtype)
    g = torch.Generator().manual_seed(1)
    hide = torch.rand(6, 20000, generator=g) < 0.999
    hide[:, 77] = False
    x[hide] = torch.finfo(dtype).min if hidden == "lowest" else hidden
    hide[5] = True
    hide[5, 77] = False                       # one token is left
    x[5][hide[5]] = x[0][hide[0]][0]
    for kw in SETTINGS[:-1] + [dict(top_k=19999), dict(top_p=0.99999)]:
        got, _ = run(x, [0.0, 0.2, 0.5, 0.8, 1 - 2.0 ** -24, 1 - 2.0 ** -24], **kw)
        assert not hide[torch.arange(6), torch.as_tensor(got).long()].any()
        assert got[5] == 77


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("lead", [0, 1, 5])
def test_a_cut_among_hidden_tokens(dtype, lead):
    """More tokens are to be kept than have a score: the cut lies among those of -infinity, by index."""
    for V in (40, 5003, 30007):
        x = torch.full((3, V), float("-inf"))
        x[:, 3::V // 7] = torch.randn(3, len(range(3, V, V // 7)))
        run(x.to(dtype), [0.0, 0.5, 1 - 2.0 ** -24], top_k=[20, V - 1, V // 2], lead=lead, exact_set=True)


@pytest.mark.gpu
def test_large_scores_and_the_largest_rows():
    x = scores(2, 4000, 4) * 1e37
    run(x, [0.3, 0.9], top_k=10)
    run(scores(3, 9000, 4) * 60, [0.3, 0.9, 0.5], top_k=[10, 4000, 0], top_p=[1.0, 0.9, 0.99])
    run((scores(3, 9000, 4) * 60).bfloat16(), [0.3, 0.9, 0.5], temperature=40.0, top_k=[10, 4000, 0], top_p=[1.0, 0.9, 0.99])
    run((scores(3, 9000, 4) - 500).bfloat16(), [0.3, 0.9, 0.5], top_k=[10, 4000, 0], top_p=[1.0, 0.9, 0.99])
    run((scores(3, 9000, 4) * 1e-4).bfloat16(), [0.3, 0.9, 0.5], top_k=[10, 4000, 0], top_p=[1.0, 0.9, 0.99])
    run(scores(1, 350000, 5), [0.7], top_p=0.9)
    run(scores(1, 700000, 6, dtype=torch.bfloat16), [0.7], top_k=50, min_p=0.01)


@pytest.mark.gpu
def test_a_row_repeats_whatever_is_beside_it():
    import speculative_decoding_specdec_gb300.specdec as sd
    x = scores(64, 32000, 8).to(DEV)
    u = torch.rand(64, generator=torch.Generator().manual_seed(0)).to(DEV)
    out = []
    for rows in (64, 64, 3):
        token, lp, kb, st = i32(np.zeros(rows)), f32(0, rows), i32(np.zeros((rows, 2))), status()
        sd.sample(x[:rows], u[:rows], token, st, top_p=f32(0.9, rows), logprob=lp, keep_bounds=kb)
        torch.cuda.synchronize()
        out.append((token[:3].tolist(), lp[:3].tolist(), kb[:3].tolist()))
    assert out[0] == out[1] == out[2]


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [dict(temperature=-1.0), dict(temperature=float("nan")), dict(temperature=float("inf")),
                                 dict(top_k=-1), dict(top_p=0.0), dict(top_p=1.5), dict(top_p=float("nan")),
                                 dict(min_p=-0.1), dict(min_p=1.1), dict(min_p=float("nan")), dict(u=1.0), dict(u=-0.1),
                                 dict(u=float("nan")), dict(x=float("nan")), dict(x=float("inf")), dict(x="hidden")])
@pytest.mark.parametrize("V", [50, 40000])
def test_bad_rows_are_told_and_not_written(bad, V):
    import speculative_decoding_specdec_gb300.specdec as sd
    x = scores(3, V, 1)
    if "x" in bad:
        if bad["x"] == "hidden":
            x[1] = float("-inf")
        else:
            x[1, V - 3] = bad["x"]
    val = dict(temperature=[1.0] * 3, top_p=[0.9] * 3, min_p=[0.0] * 3, u=[0.5] * 3, top_k=[0] * 3)
    for n, v in bad.items():
        if n != "x":
            val[n][1] = v
    token, lp, kb, st = i32(np.full(3, -7)), f32(7.0, 3), i32(np.full((3, 2), -7)), status()
    sd.sample(x.to(DEV), f32(val["u"], 3), token, st, temperature=f32(val["temperature"], 3), top_k=i32(val["top_k"]),
              top_p=f32(val["top_p"], 3), min_p=f32(val["min_p"], 3), logprob=lp, keep_bounds=kb)
    torch.cuda.synchronize()
    assert int(st) == sd.ERR_INPUT_RANGE
    assert token[1] == -7 and lp[1] == 7 and (kb[1] == -7).all()
    for r in (0, 2):
        keep = SO.kept(x[r].double().numpy(), 1.0, 0, 0.9)
        assert token[r] == SO.draw(x[r].double().numpy(), 1.0, keep, 0.5)[0]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
def test_bounds_serve_a_verification(dtype):
    """Bounds written as the drafts are drawn (and for the target's rows) give what the sampling
    filter's give."""
    import speculative_decoding_specdec_gb300.specdec as sd
    B, D, V = 6, 4, 9000
    g = torch.Generator().manual_seed(2)
    target = scores(B * (D + 1), V, 1, dtype=dtype).view(B, D + 1, V).to(DEV)
    near = target[:, :D].float() + 0.3 * torch.randn(B, D, V, generator=g).to(DEV)
    draft_logits = near.to(dtype).contiguous()
    st, temperature = status(), 0.8
    bounds = torch.zeros(B, 2 * D + 1, 2, dtype=torch.int32, device=DEV)
    draft = torch.zeros(B, D, dtype=torch.int32, device=DEV)
    kw = dict(temperature=f32(temperature, B), top_k=i32([50] * B), top_p=f32(0.9, B))
    for j in range(D):
        token = torch.zeros(B, dtype=torch.int32, device=DEV)
        sd.sample(draft_logits[:, j], torch.rand(B, generator=g).to(DEV), token, st, keep_bounds=bounds[:, D + 1 + j], **kw)
        draft[:, j] = token
    for j in range(D + 1):
        sd.sample(target[:, j], f32(0.0, B), torch.zeros_like(token), st, keep_bounds=bounds[:, j], **kw)
    u = torch.rand(B, D + 1, generator=g).to(DEV)
    other = torch.zeros_like(bounds)
    sd.sampling_filter(target, draft_logits, temperature, 50, 0.9, other, st)
    res = []
    for kb in (bounds, other):
        a, y = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
        sd.verify_sample(target, draft_logits, draft, u, temperature, a, y, st, keep_bounds=kb)
        torch.cuda.synchronize()
        res.append((a.tolist(), y.tolist()))
    assert int(st) == 0 and res[0] == res[1]
    assert max(res[0][0]) > 0


@pytest.mark.gpu
def test_in_a_graph_on_another_stream():
    import speculative_decoding_specdec_gb300.specdec as sd
    x, u = scores(4, 32000, 3).to(DEV), f32([0.1, 0.4, 0.6, 0.9], 4)
    token, st, p = i32(np.zeros(4)), status(), f32(0.9, 4)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        sd.sample(x, u, token, st, top_p=p)
    for _ in range(2):
        x.copy_(torch.roll(x, 1, 0))
        graph.replay()
        torch.cuda.synchronize()
        for r in range(4):
            row = x[r].double().cpu().numpy()
            assert token[r] == SO.draw(row, 1.0, SO.kept(row, 1.0, 0, 0.9), float(u[r]))[0]
    assert int(st) == 0


def test_host_checks():
    """Refused before anything is launched, so no GPU is needed."""
    import speculative_decoding_specdec_gb300.specdec as sd
    fake = 1 << 20

    def call(**kw):
        a = sd.SampleArgs(logits=fake, dtype=sd.BF16, R=1, V=10, row_stride=10, uniforms=fake, token=fake, dev_status=fake)
        for n, v in kw.items():
            setattr(a, n, v)
        return sd.lib.specdec_sample(ctypes.byref(a), None)

    assert sd.lib.specdec_sample(None, None) == sd.ERR_INVALID_ARG
    assert call(R=0) == sd.OK
    for kw in (dict(logits=None), dict(logits=fake + 1), dict(dtype=9), dict(R=-1), dict(V=0), dict(row_stride=9),
               dict(uniforms=None), dict(uniforms=fake + 2), dict(token=None), dict(dev_status=None), dict(temperature=fake + 1),
               dict(top_k=fake + 2), dict(top_p=fake + 2), dict(min_p=fake + 2), dict(logprob=fake + 2),
               dict(keep_bounds=fake + 2), dict(R=2, keep_bounds=fake, bounds_stride=0), dict(bounds_stride=-1)):
        assert call(**kw) == sd.ERR_INVALID_ARG, kw
    for kw in (dict(V=900000, row_stride=900000), dict(dtype=sd.F32, V=450000, row_stride=450000), dict(R=1 << 24)):
        assert call(**kw) == sd.ERR_UNSUPPORTED, kw


def test_binding_checks():
    import speculative_decoding_specdec_gb300.specdec as sd
    x, f, i = torch.zeros(2, 8), torch.zeros(2), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        sd.sample(x, f, i, i[:1])


def test_oracle_pins():
    """The oracle on rows that can be done by hand."""
    x = np.log([4.0, 2.0, 1.0, 1.0])
    assert list(SO.kept(x, 1.0)) == [0, 1, 2, 3]
    assert list(SO.kept(x, 1.0, top_k=3)) == [0, 1, 2]
    assert list(SO.kept(x, 1.0, top_p=0.5)) == [0] and list(SO.kept(x, 1.0, top_p=0.51)) == [0, 1]
    assert list(SO.kept(x, 1.0, top_k=2, top_p=0.66)) == [0] and list(SO.kept(x, 1.0, top_k=2, top_p=0.67)) == [0, 1]
    assert list(SO.kept(x, 1.0, min_p=0.4)) == [0, 1] and list(SO.kept(x, 0.5, min_p=0.4)) == [0]
    assert list(SO.kept(x[::-1], 0.0)) == [3] and list(SO.kept([1.0, 5.0, 5.0], 0.0)) == [1]
    for u, want in ((0.0, 0), (0.49, 0), (0.5, 1), (0.74, 1), (0.76, 2), (0.99, 3)):
        assert SO.draw(x, 1.0, SO.kept(x, 1.0), u)[0] == want
    assert abs(SO.draw(x, 1.0, SO.kept(x, 1.0, top_k=2), 0.9)[1] - np.log(1 / 3)) < 1e-12
