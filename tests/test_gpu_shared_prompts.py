"""The operators of shared prompts together (engine.SharedPromptBatch): prefill, rounds of sampled
tokens and rounds of greedy trees on a small decoder with normed heads, against the same decoder run
plainly on whole sequences in float64.

The decoder's sums have at most 256 terms, each good to 2^-24, through two layers: scores are off by far
less than 1e-3, and a token is checked where u is further than that from a border between two.
"""
import os
import sys

import numpy as np
import pytest
import torch

import oracle.sample_oracle as SO

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
DEV = "cuda"
PROMPTS, SAMPLES = (70, 1, 41), (3, 1, 2)


def prompts_of(seed):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randint(0, 256, (n,), generator=gen).tolist() for n in PROMPTS]


def decoder(seed=0):
    import tree_round
    model = tree_round.Decoder(seed=seed, device=DEV)
    gen = torch.Generator().manual_seed(seed + 9)
    for lay in model.layers:
        for w in ("qn", "kn"):
            lay[w] = (1 + 0.3 * torch.randn(model.hd, generator=gen)).to(DEV)
    return model


def plain64(model, tokens, table):
    """Scores [N, V] of a whole sequence in float64."""
    n, d = len(tokens), lambda t: t.double()
    x = d(model.embed)[torch.as_tensor(tokens, device=DEV)]
    cs = d(table)[:n, None]
    norm = lambda t, eps: t / torch.sqrt(t.square().mean(-1, keepdim=True) + eps)

    def turned(t):
        a, b = t.chunk(2, -1)
        return torch.cat((a * cs[..., 0] - b * cs[..., 1], a * cs[..., 1] + b * cs[..., 0]), -1)
    mask = torch.ones(n, n, dtype=torch.bool, device=DEV).tril()
    for lay in model.layers:
        q, k, v = model.split(norm(x, 1e-6) @ d(lay["qkv"]))
        q = turned(norm(q, 1e-5) * d(lay["qn"]))
        k = turned(norm(k, 1e-5) * d(lay["kn"]))
        g = model.heads_q // model.heads
        z = torch.einsum("qhd,khd->hqk", q, k.repeat_interleave(g, 1)) * model.hd ** -0.5
        w = torch.softmax(z.masked_fill(~mask, -torch.inf), -1)
        y = torch.einsum("hqk,khd->qhd", w, v.repeat_interleave(g, 1))
        x = x + y.flatten(1) @ d(lay["out"])
        x = x + torch.nn.functional.silu(norm(x, 1e-6) @ d(lay["up"])) @ d(lay["down"])
    return norm(x, 1e-6) @ d(model.head)


def begin(nodes, D, rounds, in_place):
    import tree_round
    from speculative_decoding_specdec_gb300.engine import SharedPromptBatch, rotary_table
    model = decoder()
    prompts = prompts_of(4)
    cap = 2 + rounds * (D + 1) + nodes
    table = rotary_table(max(PROMPTS) + cap, model.hd, device=DEV)
    batch = SharedPromptBatch(len(model.layers), model.heads_q, model.heads, model.hd, torch.float32, prompts, SAMPLES, nodes, D,
                              cap, rounds, in_place=in_place)
    for t in batch.kv + [batch.prefix]:
        t.fill_(float("nan"))                  # what was never written must never be read
    norms = lambda i: dict(q_weight=model.layers[i]["qn"], k_weight=model.layers[i]["kn"], eps=1e-5)
    for tokens, append, attend in batch.prefill():
        tree_round.pass_over(model, tokens, lambda i, q, k, v, out: append(i, q, k, v, table, out, **norms(i)), attend)

    def scores(tokens, parents):
        return tree_round.pass_over(model, tokens,
                                    lambda i, q, k, v, out: batch.rotary_append(i, q, k, v, table, out, parents, **norms(i)),
                                    lambda i, q, out: batch.attention(i, q, out, parents))
    rows = [list(prompts[p]) for p in batch.prompt_of]
    return model, table, batch, rows, scores


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
def test_sampled_tokens_are_those_of_plain_decoding(in_place):
    rounds = 6
    model, table, batch, rows, scores = begin(1, 1, rounds, in_place)
    B = batch.B
    gen = torch.Generator().manual_seed(1)
    settings = dict(temperature=[0.0, 0.7, 1.0, 1.3, 0.9, 1.0], top_k=[0, 0, 40, 0, 20, 0], top_p=[1.0, 0.9, 1.0, 0.8, 0.95, 1.0],
                    min_p=[0.0, 0.0, 0.0, 0.0, 0.02, 0.1])
    args = {k: torch.tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32, device=DEV) for k, v in settings.items()}
    logprob, draft = torch.zeros(B, device=DEV), torch.zeros(B, 1, dtype=torch.int32, device=DEV)
    checked = 0
    for _ in range(rounds):
        pending = torch.tensor([[r[-1]] for r in rows], dtype=torch.int32, device=DEV)
        z = scores(pending, None)[:, 0]
        u = torch.rand(B, generator=gen).to(DEV)
        batch.sample(z, u, logprob=logprob, **args)
        tokens, lp = batch.out_token.tolist(), logprob.tolist()
        batch.realign(draft)
        for b, r in enumerate(rows):
            want = plain64(model, r, table)[-1]
            assert (z[b].double() - want).abs().max() <= 1e-3
            x = want.cpu().numpy()
            s = {k: v[b] for k, v in settings.items()}
            keep = SO.kept(x, s["temperature"], s["top_k"], s["top_p"], s["min_p"])
            t, l, edges, ids = SO.draw(x, s["temperature"], keep, float(u[b]))
            if s["temperature"] == 0 or np.abs(edges - float(u[b])).min() > 1e-3:
                sharp = np.sort(x)[::-1]
                if s["temperature"] > 0 or sharp[0] - sharp[1] > 2e-3:
                    assert tokens[b] == t
                    assert abs(lp[b] - l) <= 5e-3
                    checked += 1
            r.append(tokens[b])
    assert int(batch.status) == 0 and checked > 25
    W = int(batch.width)
    assert W == 1 + rounds
    for b, r in enumerate(rows):
        assert batch.ids[batch.cur][b, :W].tolist() == r[-W:]


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
def test_greedy_trees_commit_plain_greedy_decoding(in_place):
    rounds, widths = 5, (2, 1, 1)
    nodes = 1 + 2 + 2 + 2
    model, table, batch, rows, scores = begin(nodes, len(widths), rounds, in_place)
    gen = torch.Generator().manual_seed(2)
    accepted = 0
    for _ in range(rounds):
        tokens, parents = torch.zeros(batch.B, nodes, dtype=torch.int32), torch.tensor([[-1, 0, 0, 1, 2, 3, 4]] * batch.B, dtype=torch.int32)
        for b, r in enumerate(rows):
            line = list(r)
            for node in (1, 3, 5):              # the right continuation now and then, beside a wrong one
                line.append(int(plain64(model, line, table)[-1].argmax()))
                right = torch.rand((), generator=gen) < 0.7
                tokens[b, node] = line[-1] if right else (line[-1] + 1) % 256
                tokens[b, node + 1] = (line[-1] + 7) % 256
            tokens[b, 0] = r[-1]
        tokens, parents = tokens.to(DEV), parents.to(DEV)
        batch.verify_tree_greedy(scores(tokens, parents), tokens, parents)
        batch.commit_realign()
        a, y, d = batch.accept_len.tolist(), batch.out_token.tolist(), batch.drafts.tolist()
        for b, r in enumerate(rows):
            r += d[b][:a[b]] + [y[b]]
            accepted += a[b]
    assert int(batch.status) == 0 and accepted > batch.B
    prompts = [batch.prompts[p] for p in batch.prompt_of]
    for p, r in zip(prompts, rows):
        plain = list(p)
        while len(plain) < len(r):
            plain.append(int(plain64(model, plain, table)[-1].argmax()))
        assert plain == r


def test_what_a_batch_of_shared_prompts_needs():
    from speculative_decoding_specdec_gb300.engine import SharedPromptBatch
    for prompts, samples in (([[1]], [1, 2]), ([[1], []], [1, 1]), ([[1]], [0]), ([], [])):
        with pytest.raises(ValueError):
            SharedPromptBatch(1, 2, 1, 16, torch.float32, prompts, samples, 1, 1, 8, 1, device="cpu")


def test_every_call_hands_its_stream_on(monkeypatch):
    import contextlib
    from speculative_decoding_specdec_gb300 import engine, specdec
    seen, on = [], []

    class Recorder:
        def get(self, kind, nbytes, stream=None):
            seen.append(stream)

    @contextlib.contextmanager
    def side(s):
        on.append(s)
        yield

    b = engine.SharedPromptBatch(1, 2, 1, 16, torch.float32, [[5] * 80], [2], 1, 1, 8, 1, device="cpu")
    b.workspaces = Recorder()
    monkeypatch.setattr(torch.cuda, "stream", side)
    for name in ("norm_rotary_append", "prefix_attention", "tree_attention", "sample"):
        monkeypatch.setattr(specdec, name, lambda *a, stream=None, **k: seen.append(stream))
    for name in ("prefix_attention_workspace_bytes", "tree_attention_workspace_bytes"):
        monkeypatch.setattr(specdec, name, lambda *a: 256)
    passes = 0
    for tokens, append, attend in b.prefill():
        assert tokens.shape == ((1, 64), (1, 15))[passes]
        append(0, None, None, None, None, None, stream="side")
        attend(0, None, None, stream="side")
        passes += 1
    b.rotary_append(0, None, None, None, None, None, None, stream="side")
    b.attention(0, None, None, None, stream="side")
    b.sample(torch.empty(2, 9), None, stream="side")
    assert passes == 2 and seen == ["side"] * (3 * passes + 4) and on == ["side"]
