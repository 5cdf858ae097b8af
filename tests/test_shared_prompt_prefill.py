"""The passes that prefill shared prompts: each has tensors of its own, which stay as they are for as
long as the batch lives, whatever stream the calls are on and in whatever order the passes are taken."""
import os
import sys
import weakref

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
DEV = "cuda"
CHUNK = 64


def batch_on_cpu(monkeypatch, lengths):
    """A batch whose operators only note what they are given: (name, tensors, values at the call)."""
    from speculative_decoding_specdec_gb300 import engine, specdec
    seen = []

    def rotary(q, k, v, cache, layer, table, q_out, status, *a, positions, columns, **kw):
        seen.append(("append", (positions, columns), (positions.tolist(), columns.tolist())))

    def attention(q, cache, layer, out, n_committed, width, parents, status, ws, first_col, **kw):
        t = (n_committed, parents, first_col)
        seen.append(("attend", t, tuple(x.tolist() for x in t)))
    monkeypatch.setattr(specdec, "norm_rotary_append", rotary)
    monkeypatch.setattr(specdec, "tree_attention", attention)
    monkeypatch.setattr(specdec, "tree_attention_workspace_bytes", lambda *a: 256)
    prompts = [[100 * p + i for i in range(n)] for p, n in enumerate(lengths)]
    b = engine.SharedPromptBatch(1, 2, 1, 16, torch.float32, prompts, [1] * len(prompts), 1, 1, 8, 1, device="cpu")
    return b, prompts, seen


def expected(prompts):
    """Per pass: tokens, positions, columns, lengths before the pass and one more, parents."""
    held = [len(p) - 1 for p in prompts]
    for t0 in range(0, max(held), CHUNK):
        T = min(CHUNK, max(held) - t0)
        at = [[t0 + t if t0 + t < n else -1 for t in range(T)] for n in held]
        yield ([[p[a] if a >= 0 else 0 for a in row] for p, row in zip(prompts, at)],
               [[max(a, 0) for a in row] for row in at], at,
               [t0 + 1 if row[0] >= 0 else 1 for row in at],
               [[t - 1 if a >= 0 else -2 for t, a in enumerate(row)] for row in at])


LENGTHS = [(201, 1, 70, 65), (1,), (2,), (64, 65), (66, 129)]


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("ahead", [False, True])
def test_each_pass_has_its_own_places(monkeypatch, lengths, ahead):
    """ahead: all passes are taken from the generator before the first is run."""
    b, prompts, seen = batch_on_cpu(monkeypatch, lengths)
    passes = b.prefill()
    n = 0
    for tokens, append, attend in (list(passes) if ahead else passes):
        append(0, None, None, None, None, None)
        attend(0, None, None)
        want = list(expected(prompts))[n]
        assert tokens.dtype is torch.int32 and tokens.tolist() == want[0]
        assert seen[2 * n][2] == (want[1], want[2])
        assert seen[2 * n + 1][2] == (want[3], want[4], [0] * len(prompts))
        n += 1
    assert n == len(list(expected(prompts)))


def test_a_passes_tensors_outlive_it(monkeypatch):
    """Kernels of a pass may still be queued on their stream when the generator goes on."""
    b, prompts, seen = batch_on_cpu(monkeypatch, (201, 30))
    alive, values = [], []
    for tokens, append, attend in b.prefill():
        append(0, None, None, None, None, None)
        attend(0, None, None)
        for t in seen[-2][1] + seen[-1][1] + (tokens,):
            alive.append((weakref.ref(t.untyped_storage()), t.data_ptr(), t.shape, t.tolist()))
            assert t.is_contiguous() and t.dtype is torch.int32
        seen[:] = [None, None]
        del tokens, append, attend, t
    assert len(alive) == 4 * 6
    spans = sorted({(p, p + 4 * s.numel()) for _, p, s, _ in alive})
    assert all(a[1] <= z[0] for a, z in zip(spans, spans[1:]))     # no two share memory
    again = list(b.prefill())                                       # a second time: the same tensors
    for (tokens, append, attend), k in zip(again, range(0, 24, 6)):
        append(0, None, None, None, None, None)
        attend(0, None, None)
        for t, (_, p, s, v) in zip(seen[-2][1] + seen[-1][1] + (tokens,), alive[k:k + 6]):
            assert (t.data_ptr(), t.shape, t.tolist()) == (p, s, v)


def filled(dtype, mode):
    """The prefix of four passes over two layers, from given q, k and v."""
    from speculative_decoding_specdec_gb300.engine import SharedPromptBatch, rotary_table
    L, Hq, H, hd = 2, 4, 2, 64
    gen = torch.Generator().manual_seed(5)
    prompts = [torch.randint(0, 99, (n,), generator=gen).tolist() for n in (230, 40, 129)]
    b = SharedPromptBatch(L, Hq, H, hd, dtype, prompts, [1, 2, 1], 1, 1, 8, 1)
    b.prefix.zero_()
    table, P = rotary_table(256, hd), len(prompts)
    w = torch.rand(hd, generator=gen).to(DEV)
    inputs = [[torch.randn(P, 64, n, hd, generator=gen).to(dtype).to(DEV) for n in (Hq, H, H)] for _ in range(4 * L)]
    outs = [torch.zeros(2, P, 64, Hq, hd, dtype=dtype, device=DEV) for _ in range(4 * L)]
    side = torch.cuda.Stream() if mode != "current" else None
    torch.cuda.synchronize()
    if side is not None:                         # a second or so of other work before the first pass
        with torch.cuda.stream(side):
            torch.cuda._sleep(1_000_000_000)
    passes = b.prefill()
    n = 0
    for tokens, append, attend in (list(passes) if mode == "ahead" else passes):
        T = tokens.shape[1]
        for layer in range(L):
            q, k, v = (x[:, :T] for x in inputs[n])
            turned, out = outs[n][:, :, :T]
            append(layer, q, k, v, table, turned, q_weight=w, k_weight=w, stream=side)
            attend(layer, turned, out, stream=side)
            n += 1
        for size in (2, 3):                      # what the current stream's allocator hands out is written
            torch.full((P, T), size, dtype=torch.int32, device=DEV)
            torch.full((P,), size, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    assert n == 4 * L and int(b.status) == 0
    return b.prefix, outs


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_prefill_on_a_busy_stream_of_its_own(dtype):
    """Bit for bit the current stream's, also with the passes taken from the generator ahead."""
    prefix, outs = filled(dtype, "current")
    assert prefix.isfinite().all() and (prefix[:, :, 0, :, :229] != 0).any(-1).all()
    assert all(o.isfinite().all() for o in outs)
    for mode in ("side", "ahead"):
        other, others = filled(dtype, mode)
        assert torch.equal(prefix, other)
        assert all(torch.equal(a, z) for a, z in zip(outs, others))
