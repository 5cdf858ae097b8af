"""Operators of shared prompts at offsets beyond 32 bits, captured twice over one workspace, and at once.

Tolerances are those of test_gpu_prefix_attention, test_gpu_norm_rotary and test_gpu_sample.
"""
import numpy as np
import pytest
import torch

import oracle.sample_oracle as SO
import test_gpu_norm_rotary as NR
import test_gpu_prefix_attention as PA
import test_gpu_sample as SA
from tree_testlib import DEV, i32, numpy64, random_parents, status

DT = [torch.float32, torch.bfloat16]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
def test_prefixes_and_columns_beyond_four_gigabytes(dtype):
    import speculative_decoding_specdec_gb300.specdec as sd
    hd, H = 64, 1
    cap = (1 << 32) // (hd * (4 if dtype == torch.float32 else 2)) + 1024
    arena = torch.empty(1, 2, 1, H, cap, hd, dtype=dtype, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(3)
    first, lens, groups = [cap - 700, 5, cap - 130], [700, 100, 129], [0, 2, 3, 4]
    for f, m in zip(first, lens):
        arena[:, :, :, :, f:f + m] = torch.randn(1, 2, 1, H, m, hd, generator=gen, device=DEV).to(dtype)
    for T, Hq, tree in ((1, 4, False), (9, 4, True), (32, 8, True)):    # few rows, more, rows that fill tiles
        B = 4
        n = np.array([3, 20, 1, 64])
        q, cache, W, _ = PA.inputs(T, B, T, Hq, H, hd, n, dtype, 1, [1])
        par = random_parents(np.random.default_rng(T), B, T) if tree else None
        out, lse, st = PA.run(q, cache, 1, n, W, par, arena.expand(2, -1, -1, -1, -1, -1), lens, groups, first)
        assert st == 0
        PA.check(out, lse, q, cache, 1, n, W, par, arena.expand(2, -1, -1, -1, -1, -1), lens, groups, first)
    # heads normed and appended to its last columns
    B, T, Hq = 1, 2, 2
    q = torch.randn(B, T, Hq, hd, generator=gen, device=DEV).to(dtype)
    k, v = (torch.randn(B, T, H, hd, generator=gen, device=DEV).to(dtype) for _ in range(2))
    angle = np.arange(8)[:, None] * 1e4 ** (-np.arange(hd // 2) / (hd // 2))
    table = torch.as_tensor(np.stack((np.cos(angle), np.sin(angle)), -1), dtype=torch.float32).to(DEV)
    w = torch.randn(hd, generator=gen, device=DEV).to(dtype)
    out, st = torch.zeros_like(q), status()
    sd.norm_rotary_append(q, k, v, arena, 0, table, out, st, w, w, start=i32([3]), positions=i32([[0, 4]]),
                          columns=i32([[cap - 1, cap - 2]]))
    torch.cuda.synchronize()
    assert int(st) == 0
    tab, wn = numpy64(table), numpy64(w)
    for t, (pos, col) in enumerate(((3, cap - 1), (7, cap - 2))):
        cs = tab[pos]
        NR.close(numpy64(out)[0, t], NR.normed(numpy64(q)[0, t], wn, 1e-6, 0.0), cs[:, 0], cs[:, 1], False, dtype)
        NR.close(numpy64(arena[0, 0, 0, :, col]), NR.normed(numpy64(k)[0, t], wn, 1e-6, 0.0), cs[:, 0], cs[:, 1], False, dtype)
        assert torch.equal(arena[0, 1, 0, :, col], v[0, t])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
def test_score_rows_far_apart(dtype):
    import speculative_decoding_specdec_gb300.specdec as sd
    V, far = 5000, (1 << 31) + 8
    buf = torch.empty(far + V, dtype=dtype, device=DEV)
    x = buf.as_strided((2, V), (far, 1))
    x.copy_(SA.scores(2, V, 1, dtype=dtype))
    token, st = i32([-1, -1]), status()
    sd.sample(x, SA.f32([0.3, 0.7], 2), token, st, top_k=i32([20, 0]))
    torch.cuda.synchronize()
    assert int(st) == 0
    for r, (u, k) in enumerate(((0.3, 20), (0.7, 0))):
        row = x[r].double().cpu().numpy()
        want, _, edges, _ = SO.draw(row, 1.0, SO.kept(row, 1.0, k), float(np.float32(u)))
        assert np.abs(edges - np.float32(u)).min() > SA.delta(V) and token[r] == want


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
def test_two_captured_graphs_and_eager_calls_share_a_workspace(dtype):
    import speculative_decoding_specdec_gb300.specdec as sd
    shapes = [(4, 16, 8, 1, 64, [900, 33], [0, 3, 4]), (9, 1, 8, 2, 64, [4000], [1, 9])]
    calls, ws = [], None
    for B, T, Hq, H, hd, lens, groups in shapes:
        n = np.arange(2, 2 + B)
        q, cache, W, prefix = PA.inputs(B, B, T, Hq, H, hd, n, dtype, len(lens), lens)
        size = sd.prefix_attention_workspace_bytes(q, cache, len(lens))
        ws = size if ws is None else max(ws, size)
        calls.append([q, cache, n, W, prefix, lens, groups, torch.zeros_like(q), torch.zeros(q.shape[:3], device=DEV),
                      (i32(n), i32([W]), i32(lens), i32(groups)), status(), torch.cuda.CUDAGraph()])
    ws = torch.zeros(ws, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def one(c):
        q, cache, n, W, prefix, lens, groups, out, lse, dev, st, graph = c
        sd.prefix_attention(q, cache, 1, out, dev[0], dev[1], None, st, ws, prefix, dev[2], dev[3], lse=lse)
    for c in calls:
        with torch.cuda.graph(c[-1], stream=side):
            one(c)
    torch.cuda.synchronize()
    for turn in range(3):
        for c in calls:
            c[0].copy_(c[0].roll(1, 0))
        for c in calls:
            c[-1].replay()
        one(calls[turn % 2])                 # eager, behind the replays of the same stream
        for c in calls[::-1]:
            c[-1].replay()
        torch.cuda.synchronize()
        for q, cache, n, W, prefix, lens, groups, out, lse, _, st, _ in calls:
            assert int(st) == 0
            PA.check(out, lse, q, cache, 1, n, W, None, prefix, lens, groups)
    assert not ws[:32 << 10].any()           # the tickets are back at zero


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
def test_calls_on_two_streams_at_once(dtype):
    """Each stream its own workspace and outputs: the same results as one after the other, bit for bit."""
    import speculative_decoding_specdec_gb300.specdec as sd
    B, T, Hq, H, hd, lens, groups = 6, 4, 8, 2, 128, [3000, 700], [0, 4, 6]
    n = np.arange(3, 3 + B)
    q, cache, W, prefix = PA.inputs(1, B, T, Hq, H, hd, n, dtype, 2, lens)
    x, u, p = SA.scores(16, 32000, 2, dtype=dtype).to(DEV), SA.f32(np.linspace(0, 0.99, 16), 16), SA.f32(0.9, 16)
    dev, streams = (i32(n), i32([W]), i32(lens), i32(groups)), [torch.cuda.Stream() for _ in range(2)]
    made = [[torch.zeros(sd.prefix_attention_workspace_bytes(q, cache, 2), dtype=torch.uint8, device=DEV), torch.zeros_like(q),
             i32(np.zeros(16)), status()] for _ in range(3)]

    def work(ws, out, token, st, stream=None):
        for _ in range(4):
            sd.prefix_attention(q, cache, 1, out, dev[0], dev[1], None, st, ws, prefix, dev[2], dev[3], stream=stream)
            sd.sample(x, u, token, st, top_p=p, stream=stream)
    work(*made[2])
    torch.cuda.synchronize()
    for s, m in zip(streams, made):
        work(*m, stream=s)
    torch.cuda.synchronize()
    for m in made:
        assert int(m[3]) == 0 and torch.equal(m[1], made[2][1]) and torch.equal(m[2], made[2][2])


@pytest.mark.gpu
def test_one_pool_slot_twice_in_a_call():
    """Two batch rows may name the same slot of an arena (`rows` names lengths and first columns; the arena
    is the cache's one row), and uniforms and settings may be one tensor."""
    import speculative_decoding_specdec_gb300.specdec as sd
    T, Hq, H, hd = 3, 4, 2, 64
    n = np.array([9, 9])
    q, cache, W, prefix = PA.inputs(5, 2, T, Hq, H, hd, n, torch.bfloat16, 1, [200])
    q[1] = q[0]
    out, lse, st = PA.run(q, cache[:, :, 1:], 1, n, None, None, prefix, [200], [0, 2], rows=[1, 1], first_col=[0, W - 9])
    assert st == 0 and torch.equal(out[0], out[1]) and torch.equal(lse[0], lse[1])
    half, token, st = SA.f32(0.5, 3), i32(np.zeros(3)), status()
    x = SA.scores(3, 300, 1).to(DEV)
    sd.sample(x, half, token, st, temperature=half, top_p=half, min_p=half)
    torch.cuda.synchronize()
    for r in range(3):
        row = x[r].double().cpu().numpy()
        assert token[r] == SO.draw(row, 0.5, SO.kept(row, 0.5, 0, 0.5, 0.5), 0.5)[0]
    assert int(st) == 0
