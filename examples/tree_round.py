"""Tree speculation end to end on a small random model.

    python examples/tree_round.py [--sampled]

A decoder of a few layers keeps its K/V in a ``TreeBatch``.  The prompts are prefilled in chunks
(explicit positions and columns, attention over the tokens so far), then every round a draft model
(the same weights with noise) proposes a tree per row, the target scores all of it in one pass
(rotary append and tree attention per layer), the tree is verified, and the accepted paths are
committed and realigned.  With greedy verification the committed tokens are those of plain greedy
decoding, whatever the draft model proposes.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_decoding_specdec_gb300 import specdec  # noqa: E402
from speculative_decoding_specdec_gb300.engine import TreeBatch, rotary_table  # noqa: E402

CHUNK = 32   # prompt tokens per prefill pass


class Decoder:
    """Weights of a small decoder, and its forward pass on plain torch (a whole sequence at once)."""

    def __init__(self, vocab=256, width=128, layers=2, heads_q=4, heads=2, head_dim=64, seed=0,
                 device="cuda", dtype=torch.float32):
        gen = torch.Generator().manual_seed(seed)
        def weight(*shape):
            return (torch.randn(*shape, generator=gen) * shape[-2] ** -0.5).to(device=device, dtype=dtype)
        self.vocab, self.heads_q, self.heads, self.hd = vocab, heads_q, heads, head_dim
        self.embed = weight(vocab, width) * vocab ** 0.5
        self.layers = [{"qkv": weight(width, (heads_q + 2 * heads) * head_dim),
                        "out": weight(heads_q * head_dim, width), "up": weight(width, 2 * width),
                        "down": weight(2 * width, width)} for _ in range(layers)]
        self.head = weight(width, vocab) * 2

    def noisy(self, amount, seed):
        """The same decoder with noise on its weights: a draft model that mostly agrees."""
        other = object.__new__(Decoder)
        other.__dict__.update(self.__dict__)
        gen = torch.Generator().manual_seed(seed)
        def shaken(w):
            return w * (1 + amount * torch.randn(w.shape, generator=gen).to(w))
        other.layers = [{k: shaken(w) for k, w in lay.items()} for lay in self.layers]
        return other

    def split(self, x):
        """q [.., Hq, hd], k, v [.., H, hd] as slices of the fused projection's result."""
        q, k, v = x.split([n * self.hd for n in (self.heads_q, self.heads, self.heads)], -1)
        return (t.unflatten(-1, (-1, self.hd)) for t in (q, k, v))

    @staticmethod
    def norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    def mlp(self, lay, x):
        return x + torch.nn.functional.silu(self.norm(x) @ lay["up"]) @ lay["down"]

    def plain(self, tokens, table):
        """Scores [N, V] and the K/V of every layer [L, 2, H, N, hd] for one sequence."""
        n = len(tokens)
        x = self.embed[torch.as_tensor(tokens, device=self.embed.device)]
        cs = table[:n, None]
        def turned(t):
            a, b = t.chunk(2, -1)
            return torch.cat((a * cs[..., 0] - b * cs[..., 1], a * cs[..., 1] + b * cs[..., 0]), -1)
        mask = torch.ones(n, n, dtype=torch.bool, device=x.device).tril()
        kept = []
        for lay in self.layers:
            q, k, v = self.split(self.norm(x) @ lay["qkv"])
            q, k = turned(q), turned(k)
            kept.append(torch.stack((k.transpose(0, 1), v.transpose(0, 1))))
            g = self.heads_q // self.heads
            z = torch.einsum("qhd,khd->hqk", q, k.repeat_interleave(g, 1)) * self.hd ** -0.5
            w = torch.softmax(z.masked_fill(~mask, -torch.inf), -1)
            y = torch.einsum("hqk,khd->qhd", w, v.repeat_interleave(g, 1))
            x = self.mlp(lay, x + y.flatten(1) @ lay["out"])
        return self.norm(x) @ self.head, torch.stack(kept)


def pass_over(model, tokens, append, attend):
    """The target's pass over new tokens [B, T]: scores [B, T, V].  ``append(layer, q, k, v, q_out)``
    and ``attend(layer, q, out)`` do what needs the cache."""
    x = model.embed[tokens.long()]
    B, T = tokens.shape
    for i, lay in enumerate(model.layers):
        q, k, v = model.split(model.norm(x) @ lay["qkv"])
        turned, y = torch.empty((2, B, T, model.heads_q, model.hd), dtype=x.dtype, device=x.device)
        append(i, q, k, v, turned)
        attend(i, turned, y)
        x = model.mlp(lay, x + y.flatten(2) @ lay["out"])
    return model.norm(x) @ model.head


def prefill(model, batch, prompts, width, table):
    """K/V of every prompt token but the last (the pending one), CHUNK tokens of every row a pass."""
    dev = table.device
    n = torch.tensor([len(p) for p in prompts], dtype=torch.int32)
    most = int(n.max()) - 1
    for t0 in range(0, most, CHUNK):
        T = min(CHUNK, most - t0)
        at = t0 + torch.arange(T, dtype=torch.int32)[None]
        live = at < n[:, None] - 1
        tokens = torch.zeros(len(prompts), T, dtype=torch.int32)
        for b, p in enumerate(prompts):
            part = p[t0:min(t0 + T, len(p) - 1)]
            tokens[b, :len(part)] = torch.as_tensor(part, dtype=torch.int32)
        positions = torch.where(live, at, 0).int().to(dev)
        columns = torch.where(live, at + (width - n)[:, None], -1).int().to(dev)
        chain = torch.arange(-1, T - 1, dtype=torch.int32)[None]
        parents = torch.where(live, chain, -2).int().to(dev)
        any_live = live.any(1)          # (a row that is through has no nodes: any columns will do)
        done = torch.where(any_live, t0 + 1, 1).int().to(dev)
        first = torch.where(any_live, width - n, 0).int().to(dev)

        def append(i, q, k, v, out):
            specdec.rotary_append(q, k, v, batch.cache, i, table, out, batch.status,
                                  positions=positions, columns=columns)

        def attend(i, q, out):
            ws = batch.workspaces.get("prefill", specdec.tree_attention_workspace_bytes(q, batch.cache))
            specdec.tree_attention(q, batch.cache, i, out, done, None, parents, batch.status, ws,
                                   first_col=first)

        pass_over(model, tokens.to(dev), append, attend)


def draft_tree(draft, sequence, table, widths, gen, temperature):
    """Tokens, parents and the draft model's scores [T, V] of one row's tree: ``widths[d]`` children
    under every node of depth d, the likeliest or (with a temperature) drawn without replacement."""
    tokens, parents, scores, level = [sequence[-1]], [-1], [], [0]
    lines = {0: list(sequence)}
    for w in widths:
        below = []
        for node in level:
            z = draft.plain(lines[node], table)[0][-1]
            scores.append((node, z))
            if temperature:
                e = torch.empty_like(z).exponential_(generator=gen)
                kids = torch.topk(z / temperature - e.log(), w).indices.tolist()
            else:
                kids = torch.topk(z, w).indices.tolist()
            for t in kids:
                lines[len(tokens)] = lines[node] + [t]
                below.append(len(tokens))
                tokens.append(t)
                parents.append(node)
        level = below
    out = torch.zeros(len(tokens), draft.vocab, device=table.device)
    for node, z in scores:
        out[node] = z
    return tokens, parents, out


def generate(prompts, rounds=6, widths=(3, 2, 1), temperature=0.0, in_place=False, seed=0,
             noise=0.1, dtype=torch.float32, device="cuda"):
    """Runs ``rounds`` rounds; returns the committed tokens, accept lengths, batch, model, table."""
    model = Decoder(seed=seed, dtype=dtype, device=device)
    draft = model.noisy(noise, seed + 1)
    nodes, level = 1, 1
    for w in widths:
        level *= w
        nodes += level
    longest = max(len(p) for p in prompts)
    cap = longest + max(rounds * (len(widths) + 1) + nodes, CHUNK)   # a pass's columns all fit
    table = rotary_table(cap + nodes, model.hd, device=device)
    batch = TreeBatch(len(model.layers), model.heads_q, model.heads, model.hd, dtype, len(prompts),
                      nodes, len(widths), cap, rounds, device=device, in_place=in_place)
    width = batch.start(prompts)
    for cache in batch.kv:
        cache.fill_(float("nan"))      # what was never written must never be read
    prefill(model, batch, prompts, width, table)
    gen = torch.Generator(device=device).manual_seed(seed)
    rows, accepted = [list(p) for p in prompts], []
    for _ in range(rounds):
        trees = [draft_tree(draft, r, table.to(dtype), widths, gen, temperature) for r in rows]
        tokens = torch.tensor([t for t, _, _ in trees], dtype=torch.int32, device=device)
        parents = torch.tensor([p for _, p, _ in trees], dtype=torch.int32, device=device)
        scores = pass_over(model, tokens,
                           lambda i, q, k, v, out: batch.rotary_append(i, q, k, v, table, out, parents),
                           lambda i, q, out: batch.attention(i, q, out, parents))
        if temperature:
            u = torch.rand(len(rows), nodes, generator=gen, device=device)
            batch.verify_tree_sample(scores, torch.stack([z for _, _, z in trees]).to(dtype), tokens,
                                     parents, u, temperature)
        else:
            batch.verify_tree_greedy(scores, tokens, parents)
        batch.commit_realign()
        a, y, d = batch.accept_len.tolist(), batch.out_token.tolist(), batch.drafts.tolist()
        for b, r in enumerate(rows):
            r += d[b][:a[b]] + [y[b]]
        accepted.append(a)
    if int(batch.status) != 0:
        raise RuntimeError(specdec.status_string(int(batch.status)))
    return rows, accepted, batch, model, table


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--sampled", action="store_true")
    args = ap.parse_args()
    gen = torch.Generator().manual_seed(7)
    prompts = [torch.randint(0, 256, (n,), generator=gen).tolist() for n in (5, 41, 18)]
    rows, accepted, _, model, table = generate(prompts, temperature=0.8 if args.sampled else 0.0)
    for b, (row, p) in enumerate(zip(rows, prompts)):
        new = row[len(p):]
        print(f"row {b}: {len(new)} tokens, accepted per round {[a[b] for a in accepted]}: {new}")
        if not args.sampled:
            plain = list(p)
            while len(plain) < len(row):
                plain.append(int(model.plain(plain, table)[0][-1].argmax()))
            print("       the same as plain greedy decoding:", plain == row)


if __name__ == "__main__":
    main()
