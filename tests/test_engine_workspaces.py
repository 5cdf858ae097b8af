"""The engine's workspaces: made on the stream of the call that needs them, kept when outgrown."""
import contextlib

import pytest
import torch

from speculative_decoding_specdec_gb300 import engine, specdec


class FakeStreams:
    """Stands in for torch.cuda.stream and torch.zeros: on which stream each buffer is filled."""

    def __init__(self, monkeypatch):
        self.now, self.filled = "current", []
        zeros = torch.zeros

        @contextlib.contextmanager
        def stream(s):
            before, self.now = self.now, s or self.now
            yield
            self.now = before

        def recorded(*args, **kw):
            self.filled.append(self.now)
            return zeros(*args, **kw)

        monkeypatch.setattr(torch.cuda, "stream", stream)
        monkeypatch.setattr(torch, "zeros", recorded)


def test_the_zeros_are_written_on_the_calls_stream(monkeypatch):
    fake = FakeStreams(monkeypatch)
    ws = engine.Workspaces("cpu")
    draft = torch.empty(2, 3, dtype=torch.int32)
    first = ws.get("tree", 1000, "side")
    ws.bounds(draft, "side")
    ws.greedy(None, draft, "side")
    ws.get("tree", 4000)
    assert fake.filled == ["side", "side", "side", "current"]
    assert ws.get("tree", 500, "side").numel() == 4000 and len(fake.filled) == 4
    assert any(t is first for t in ws._outgrown)        # a call may still be using it


def test_every_call_hands_its_stream_on(monkeypatch):
    seen = []

    class Recorder:
        def get(self, kind, nbytes, stream=None):
            seen.append(stream)

        def greedy(self, logits, draft, stream=None):
            seen.append(stream)

        def bounds(self, draft, stream=None):
            seen.append(stream)

    for name in ("verify_greedy", "verify_sample", "sampling_filter", "tree_attention"):
        monkeypatch.setattr(specdec, name, lambda *a, **k: None)
    monkeypatch.setattr(specdec, "tree_attention_workspace_bytes", lambda q, cache: 256)
    draft, z = torch.empty(2, 3, dtype=torch.int32), torch.empty(2, 4, 10)
    for cls in (engine.TreeBatch, engine.ExspecPool, engine.SequencePool):
        b = object.__new__(cls)
        b.workspaces, b.max_rounds, b.round, b.B = Recorder(), 3, 0, 2
        b.status, b.accept_len, b.out_token = None, None, None
        if cls is engine.TreeBatch:
            b.kv, b.in_place, b.cur = [None, None], False, 0
            b.hist = torch.zeros(4, 7, dtype=torch.int32)
            b.n_hist, b.w_hist = b.hist[:, :2], b.hist[:, 2:3]
            b.attention(0, z, z, None, stream="side")
            b.verify_sample(z, z, draft, z, 1.0, stream="side", top_k=3)
        b.verify_greedy(z, draft, stream="side")
    assert seen == ["side"] * 5


@pytest.mark.gpu
def test_a_workspace_made_on_a_busy_stream_is_zero_for_a_call_on_another():
    """The current stream is held up while a batch's first attention runs on another one: its
    workspace has to be zero all the same, or units that several CTAs share are not merged."""
    B, T, H, hd, n = 1, 8, 1, 64, 3000
    gen = torch.Generator(device="cuda").manual_seed(0)
    batch = engine.TreeBatch(1, H, H, hd, torch.bfloat16, B, T, 3, n + T, 4)
    batch.start([list(range(n))])
    batch.cache.normal_(generator=gen)
    q = torch.randn(B, T, H, hd, generator=gen, device="cuda").bfloat16()
    want, got = torch.empty_like(q), torch.full_like(q, 7.0)
    batch.attention(0, q, want, None)
    # what the next allocation of that size finds is not zero
    need = specdec.tree_attention_workspace_bytes(q, batch.cache)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(s):
            torch.full((need,), 0x55, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    batch.workspaces = engine.Workspaces(batch.workspaces.device)
    torch.cuda._sleep(500_000_000)
    batch.attention(0, q, got, None, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    torch.cuda.synchronize()
    assert int(batch.status) == 0
