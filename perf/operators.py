"""Measured cases of the tree-speculation operators: rotary positions with the append to the
K/V cache, attention of a tree of drafted tokens over the cache, tree verification (greedy and
sampled), and the commit of the accepted path's K/V columns.

A tree of T nodes per row is ``parents`` [B, T] int32: node 0 is the pending token (parent -1),
node i has a parent below i, and -2 marks a node that the row does not use.  The left-padded
cache is [L, 2, B, H, cap, hd]; row b holds N_b committed tokens that end at column W - 1, and
node i of its tree sits at column W - 1 + i with position N_b - 1 + depth(i).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
NO_PARENT, UNUSED = -1, -2


# ------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # A verification pass of 32-node trees at the GLM-4-9B head layout: rotary on the first
        # half of each head, interleaved pairs, frequencies scaled for a long context.
        dict(name="rotary_tree_glm4_9b", kind="rotary", B=32, T=32, D=8, Hq=32, Hkv=2, hd=128,
             rot=64, interleaved=True, factor=4.0, dtype="bf16", lo=1024, hi=8192, tree=True,
             prefill=False),
        # Prompt prefill of a ragged left-padded batch at the Vicuna-7B head layout (the whole
        # head rotated, half layout): the bandwidth end of the operator.
        dict(name="rotary_prefill_vicuna7b", kind="rotary", B=8, T=1024, D=1, Hq=32, Hkv=32,
             hd=128, rot=128, interleaved=False, factor=1.0, dtype="bf16", lo=128, hi=1024,
             tree=False, prefill=True),
        # The smallest call: one new token per row of a tiny fp32 cache; latency counts.
        dict(name="attention_single_tiny", kind="attention", B=2, T=1, D=1, Hq=4, Hkv=2, hd=64,
             dtype="fp32", lo=5, hi=20, tree=False),
        # A chain of five drafts and the pending token at the Vicuna-7B head layout (one query
        # head per K/V head): the K/V read bounds it.
        dict(name="attention_chain_vicuna7b", kind="attention", B=8, T=6, D=5, Hq=32, Hkv=32,
             hd=128, dtype="bf16", lo=128, hi=1024, tree=False),
        # 32-node trees at the GLM-4-9B head layout (16 query heads share a K/V head): 512 query
        # rows per K/V head and row, so the matrix products bound it.
        dict(name="attention_tree_glm4_9b", kind="attention", B=32, T=32, D=8, Hq=32, Hkv=2,
             hd=128, dtype="bf16", lo=1024, hi=8192, tree=True),
        # One long context with a 64-node tree at the Qwen3-8B head layout: few rows, so the work
        # has to be split over the columns.
        dict(name="attention_long_qwen3_8b", kind="attention", B=1, T=64, D=10, Hq=32, Hkv=8,
             hd=128, dtype="bf16", lo=131071, hi=131071, tree=True),
        # Greedy verification of small trees at the Vicuna-7B vocabulary: latency counts.
        dict(name="greedy_tree_vicuna7b", kind="greedy", B=8, T=16, D=5, V=32000, dtype="bf16",
             alpha=0.7),
        # Greedy verification of 64-node trees at the Qwen3-8B vocabulary.
        dict(name="greedy_tree_qwen3_8b", kind="greedy", B=16, T=64, D=8, V=151936, dtype="bf16",
             alpha=0.7),
        # Sampled verification of a tiny batch, siblings drawn independently: the smallest call.
        dict(name="sample_tree_tiny", kind="sample", B=2, T=7, D=3, V=1000, dtype="fp32",
             temperature=1.0, replacement=True),
        # Sampled verification of 16-node trees at the GLM-4-9B vocabulary, siblings drawn
        # without replacement.
        dict(name="sample_tree_glm4_9b", kind="sample", B=32, T=16, D=5, V=151552, dtype="bf16",
             temperature=0.7, replacement=False),
        # The accepted path's columns of every layer after a realignment, many heads.
        dict(name="commit_vicuna7b", kind="commit", L=32, B=8, H=32, hd=128, T=16, D=5,
             dtype="bf16", width=512, alpha=0.7),
        # The same with few heads and a larger batch.
        dict(name="commit_glm4_9b", kind="commit", L=40, B=32, H=2, hd=128, T=32, D=8,
             dtype="bf16", width=768, alpha=0.7),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rotary", "attention", "attention", "greedy", "sample", "commit"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    Hq, Hkv = rng.choice([(32, 32), (32, 8), (32, 2), (8, 2), (4, 4)])
    hd = rng.choice([64, 128, 128])
    T = _log(rng, 1, 64)
    D = min(max(1, T - 1), rng.randint(1, 12))
    if kind == "rotary":
        prefill = rng.random() < 0.4
        T = _log(rng, 16, 1024) if prefill else T
        lo = _log(rng, 1, T) if prefill else _log(rng, 1, 4096)
        hi = T if prefill else _log(rng, lo, 8192)
        rot = rng.choice([hd, hd // 2])
        return dict(kind=kind, B=_log(rng, 1, 8 if prefill else 32), T=T, D=1 if prefill else D,
                    Hq=Hq, Hkv=Hkv, hd=hd, rot=rot, interleaved=rng.random() < 0.5,
                    factor=rng.choice([1.0, 4.0, 8.0]), dtype=dtype, lo=lo, hi=hi,
                    tree=not prefill and T > 1, prefill=prefill)
    if kind == "attention":
        tree = T > 1 and rng.random() < 0.7
        hi = _log(rng, 5, 131072)
        lo = _log(rng, max(1, hi // 8), hi)
        B = _log(rng, 1, 32)
        c = dict(kind=kind, B=B, T=T, D=D, Hq=Hq, Hkv=Hkv, hd=hd, dtype=dtype, lo=lo, hi=hi,
                 tree=tree)
        most = work(listed()[4])
        # fp32 has no tensor cores: its cases are kept to a sixteenth of the products
        flops = most["flops"] / (16 if dtype == "fp32" else 1)
        while c["hi"] > 5 and (work(c)["flops"] > flops or work(c)["bytes"] > most["bytes"]
                               or c["B"] * c["hi"] > 262144):
            if c["B"] > 1:
                c["B"] -= max(1, c["B"] // 4)
            else:
                c["hi"] = max(5, c["hi"] * 3 // 4)
                c["lo"] = min(c["lo"], c["hi"])
        return c
    if kind == "commit":
        L = rng.choice([1, 32, 36, 40])
        T = max(T, 2)
        D = min(T - 1, D)
        return dict(kind=kind, L=L, B=_log(rng, 1, 32 if Hkv <= 8 else 8), H=Hkv, hd=hd, T=T, D=D,
                    dtype="bf16" if Hkv > 8 else dtype, width=_log(rng, 8, 512),
                    alpha=rng.uniform(0.3, 0.9))
    V = rng.choice([_log(rng, 100, 152000), 32000, 151936, 151552])
    T = max(T, 2)
    D = min(T - 1, D)
    if kind == "greedy":
        T, D = min(T, 64 if dtype == "bf16" else 24), D
        return dict(kind=kind, B=_log(rng, 1, 16), T=T, D=min(D, T - 1), V=V, dtype=dtype,
                    alpha=rng.uniform(0.3, 0.9))
    T = min(T, 16 if dtype == "bf16" else 8)
    return dict(kind=kind, B=_log(rng, 1, 32), T=T, D=min(D, T - 1), V=V, dtype=dtype,
                temperature=rng.choice([0.5, 0.7, 1.0, 1.3]), replacement=rng.random() < 0.5)


# -------------------------------------------------------------------- what a case fixes by itself

def _lengths(case):
    """N_b, spread evenly over [lo, hi]; the seed permutes them."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi if B == 1 else lo + (hi - lo) * b // (B - 1) for b in range(B)]


def _levels(T, D):
    """Nodes at each depth 1..D: one each, the rest mostly near the root as draft trees have it."""
    w = [0] * D
    for i in range(min(D, T - 1)):
        w[i] = 1
    left, k = T - 1 - sum(w), 0
    while left > 0:
        add = min(left, max(1, 3 - k % D // 2))
        w[k % D] += add
        left -= add
        k += 1
    return w


def _used(case):
    """Nodes each row uses: rows of one batch drop up to a quarter of them from the end."""
    T = case["T"]
    return [T - (5 * b) % (T // 4 + 1) for b in range(case["B"])]


def _depth_of(case, used):
    """Depth of the deepest of a row's first `used` nodes (nodes are numbered level by level)."""
    n, d = 1, 0
    for w in _levels(case["T"], case["D"]):
        if n >= used or w == 0:
            break
        n, d = n + w, d + 1
    return d


def _accepts(case):
    """Accepted nodes of each row: quantiles of the geometric distribution of `alpha`."""
    B, a = case["B"], case["alpha"]
    got = [int(math.log(1.0 - (b + 0.5) / B) / math.log(a)) for b in range(B)]
    return [min(x, _depth_of(case, u)) for x, u in zip(got, _used(case))]


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    kind = case["kind"]
    if kind == "rotary":
        n = sum(_lengths(case)) if case["prefill"] else sum(_used(case)) if case["tree"] else case["B"] * case["T"]
        skipped = case["B"] * case["T"] - n            # their q rows are written as zeros
        values = n * case["hd"] * (2 * case["Hq"] + 4 * case["Hkv"]) + skipped * case["hd"] * case["Hq"]
        return {"bytes": values * es + n * case["rot"] * 4 + n * 8,
                "flops": 3.0 * n * (case["Hq"] + case["Hkv"]) * case["rot"]}
    if kind == "attention":
        new = _used(case) if case["tree"] else [case["T"]] * case["B"]
        cols = sum(n - 1 + t for n, t in zip(_lengths(case), new))
        pairs = sum(t * (n - 1) + t for n, t in zip(_lengths(case), new))   # and the tree's few
        return {"bytes": (cols * case["Hkv"] * 2 + sum(new) * case["Hq"]
                          + case["B"] * case["T"] * case["Hq"]) * case["hd"] * es,
                "flops": 4.0 * pairs * case["Hq"] * case["hd"]}
    if kind == "greedy":
        rows = sum(a + 1 for a in _accepts(case))      # the score rows on the walk
        return {"bytes": rows * case["V"] * es, "flops": rows * case["V"]}
    if kind == "sample":
        # the walk's rows, target and draft, which the random numbers decide: the root's always,
        # and an estimate of one and a half more where the tree has them
        rows = case["B"] * (1 + min(1.5, 0.75 * case["D"]))
        return {"bytes": 2 * rows * case["V"] * es, "flops": 8 * rows * case["V"]}
    moved = sum(_accepts(case))
    return {"bytes": max(1, 2 * moved * case["L"] * 2 * case["H"] * case["hd"] * es), "flops": 0}


# --------------------------------------------------------------------------------------- inputs

def _tree(case, rs):
    """parents [B, T]: level by level, each node under a random node of the level above."""
    B, T = case["B"], case["T"]
    p = np.full((B, T), UNUSED, np.int32)
    levels = _levels(T, case["D"])
    for b, used in enumerate(_used(case)):
        p[b, 0] = NO_PARENT
        first, at = 0, 1
        for w in levels:
            end = min(at + w, used)
            if end <= at:
                break
            # low-numbered nodes of a level have the likelier tokens and get more children
            pick = np.sort((rs.random_sample(end - at) ** 2 * (at - first)).astype(np.int32))
            p[b, at:end] = first + pick
            first, at = at, end
    return p


def _path(parents, node):
    path = []
    while node > 0:
        path.append(int(node))
        node = parents[node]
    return path[::-1]


def _depths(parents):
    d = np.zeros_like(parents)
    for i in range(1, parents.shape[1]):
        up = parents[:, i]
        d[:, i] = np.where(up >= 0, d[np.arange(len(d)), np.maximum(up, 0)] + 1, 0)
    return d


def _randn(gen, shape, dtype):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    return out.normal_(generator=gen)


def _int(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def prepare(case, seed):
    rs = np.random.RandomState(seed % (2 ** 32))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    B, T = case["B"], case["T"]
    kind = case["kind"]
    if kind in ("rotary", "attention"):
        n = np.asarray(_lengths(case), np.int32)
        rs.shuffle(n)
        W = int(n.max())
        cap = W + T + 1
        s["n"], s["width"] = _int(n), _int([W])
        s["parents"] = _int(_tree(case, rs)) if case["tree"] else None
        s["q"] = _randn(gen, (B, T, case["Hq"], case["hd"]), dt)
        # two layers, so that a layer's caches are read where a model's would lie
        s["cache"] = _randn(gen, (2, 2, B, case["Hkv"], cap, case["hd"]), dt)
        s["layer"] = 1
        s["out"] = torch.empty_like(s["q"])
        if kind == "attention":
            return s
        s["k"] = _randn(gen, (B, T, case["Hkv"], case["hd"]), dt)
        s["v"] = _randn(gen, (B, T, case["Hkv"], case["hd"]), dt)
        # positions' cosines and sines, made once per model in 64 bits; frequencies divided by
        # `factor` where the context is stretched
        half = case["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half) / case["factor"]
        angle = torch.arange(cap, dtype=torch.float64)[:, None] * freq
        s["table"] = torch.stack((angle.cos(), angle.sin()), -1).float().cuda()
        if case["prefill"]:
            t = np.arange(T)[None]
            held = t < n[:, None]                   # row b's prompt has n_b tokens
            s["positions"] = _int(np.where(held, t, 0))
            s["columns"] = _int(np.where(held, W - n[:, None] + t, -1))
        return s
    if kind == "commit":
        parents = _tree(case, rs)
        depths = _depths(parents)
        a = np.asarray(_accepts(case), np.int32)
        path = np.full((B, case["D"]), -1, np.int32)
        for b in range(B):
            at = np.flatnonzero((depths[b] == a[b]) & (parents[b] != UNUSED))
            path[b, :a[b]] = _path(parents[b], int(rs.choice(at)))
        W = case["width"]
        n = rs.randint(max(1, W // 4), W + 1, B).astype(np.int32)
        n[rs.randint(B)] = W
        shape = (case["L"], 2, B, case["H"], W + T + case["D"] + 1, case["hd"])
        s["src"], s["dst"] = _randn(gen, shape, dt), _randn(gen, shape, dt)
        s["width"], s["width_dst"] = _int([W]), _int([int((n + a + 1).max())])
        s["accept_len"], s["path"] = _int(a), _int(path)
        return s
    parents = _tree(case, rs)
    s["parents"] = _int(parents)
    D, V = case["D"], case["V"]
    s.update(accept_len=torch.zeros(B, dtype=torch.int32, device="cuda"),
             out_token=torch.zeros(B, dtype=torch.int32, device="cuda"),
             path=torch.zeros((B, D), dtype=torch.int32, device="cuda"),
             draft=torch.zeros((B, D), dtype=torch.int32, device="cuda"))
    if kind == "greedy":
        tokens = rs.randint(0, V, (B, T)).astype(np.int32)
        z = _randn(gen, (B, T, V), dt)
        accepts = np.asarray(_accepts(case))
        depths = _depths(parents)
        for b in range(B):
            at = np.flatnonzero((depths[b] == accepts[b]) & (parents[b] != UNUSED))
            walk = _path(parents[b], int(rs.choice(at)))
            for up, node in zip([0] + walk[:-1], walk):
                z[b, up, int(tokens[b, node])] = 8.0          # above every normal score
            last = walk[-1] if walk else 0
            other = (int(tokens[b].max()) + 1 + int(rs.randint(V))) % V
            while V > T and other in tokens[b]:
                other = (other + 1) % V
            z[b, last, other] = 8.0
        s["tokens"], s["logits"] = _int(tokens), z
        return s
    # Sampled: scores with a few likely tokens over a long tail, the draft's a noisy copy; each
    # node's children drawn from the draft's distribution, with or without replacement.
    temp = case["temperature"]
    z = _randn(gen, (B, T, V), torch.float32).mul_(1.5)
    likely = torch.randint(0, V, (B, T, 8), generator=gen, device="cuda")
    lift = torch.arange(8, device="cuda") * -0.7 + math.log(V) - 1.0
    z.scatter_(2, likely, lift + 0.5 * torch.randn(B, T, 8, generator=gen, device="cuda"))
    noise = _randn(gen, (B, T, V), torch.float32).mul_(0.5)
    s["target_logits"], s["draft_logits"] = z.to(dt), noise.add_(z).to(dt)
    del z, noise
    tokens = torch.randint(0, V, (B, T), generator=gen, device="cuda")
    for i in range(T):
        under = np.where(parents == i, np.cumsum(parents == i, 1), 0)   # 1 for the first child, ..
        most = int(under.max())
        if most == 0:
            continue
        x = s["draft_logits"][:, i].float() / temp
        if case["replacement"]:
            got = torch.multinomial(torch.softmax(x, -1), most, replacement=True, generator=gen)
        else:
            e = torch.empty_like(x).exponential_(generator=gen)
            got = torch.topk(x - e.clamp_min(1e-30).log(), most, -1).indices
        r, c = np.nonzero(under)
        tokens[torch.as_tensor(r).cuda(), torch.as_tensor(c).cuda()] = \
            got[torch.as_tensor(r).cuda(), torch.as_tensor(under[r, c] - 1).cuda()]
    s["tokens"] = tokens.to(torch.int32)
    s["uniforms"] = _settled(s, gen)
    return s


def _settled(s, gen):
    """Uniforms [B, T] (column 0 for the draw, column i for node i), none of which lies so near
    the edge of its decision that 32-bit rounding could turn it: such ones are drawn again."""
    case, near = s["case"], 2e-5
    B, T = case["B"], case["T"]
    u = torch.rand(B, T, generator=gen, device="cuda")
    more = torch.rand(B, T, 16, generator=gen, device="cuda")
    rows, tok, par = torch.arange(B, device="cuda"), s["tokens"].long(), s["parents"]
    p = torch.softmax(s["target_logits"][:, 0].double() / case["temperature"], -1)
    q = torch.softmax(s["draft_logits"][:, 0].double() / case["temperature"], -1)
    cur = torch.zeros(B, dtype=torch.int32, device="cuda")
    deep = torch.zeros_like(cur)
    for i in range(1, T):
        on = (par[:, i] == cur) & (deep < case["D"])
        c = tok[:, i]
        ratio = p[rows, c] / q[rows, c].clamp_min(1e-300)
        tries = torch.cat((u[:, i:i + 1], more[:, i]), 1)
        safe = (tries.double() - ratio[:, None]).abs() > near
        u[:, i] = tries[rows, safe.float().argmax(1)]
        yes = on & (u[:, i].double() < ratio)
        no = on & ~yes
        r = (p - q).clamp_min(0)
        left = r.sum(-1, keepdim=True)
        r = torch.where(left > 0, r / left.clamp_min(1e-300), p)
        p = torch.where(no[:, None], r, p)
        if not case["replacement"]:
            gone = q.clone()
            gone[rows, c] = 0
            gone /= gone.sum(-1, keepdim=True).clamp_min(1e-300)
            q = torch.where(no[:, None], gone, q)
        p = torch.where(yes[:, None], torch.softmax(s["target_logits"][:, i].double() / case["temperature"], -1), p)
        q = torch.where(yes[:, None], torch.softmax(s["draft_logits"][:, i].double() / case["temperature"], -1), q)
        cur = torch.where(yes, torch.full_like(cur, i), cur)
        deep = deep + yes.int()
    edges = p.cumsum(-1)
    edges /= edges[:, -1:].clone()
    tries = torch.cat((u[:, :1], more[:, 0]), 1).double()
    k = torch.searchsorted(edges, tries, right=True).clamp_max(edges.shape[1] - 1)
    hi = edges.gather(1, k)
    lo = torch.where(k > 0, edges.gather(1, (k - 1).clamp_min(0)), torch.full_like(hi, -1.0))
    room = torch.minimum(hi - tries, tries - lo)
    best = torch.where((room > near).any(1), (room > near).float().argmax(1), room.argmax(1))
    u[:, 0] = tries[rows, best].float()
    return u


# ----------------------------------------------------------------------------------- one pass

def run(s):
    kind = s["case"]["kind"]
    if own:
        return {"rotary": _own_rotary, "attention": _own_attention, "greedy": _own_greedy,
                "sample": _own_sample, "commit": _own_commit}[kind](s)
    return {"rotary": _plain_rotary, "attention": _plain_attention, "greedy": _plain_greedy,
            "sample": _plain_sample, "commit": _plain_commit}[kind](s)


def _own_rotary(s):
    from speculative_decoding_specdec_gb300 import specdec
    case = s["case"]
    if case["prefill"]:
        specdec.rotary_append(s["q"], s["k"], s["v"], s["cache"], s["layer"], s["table"], s["out"],
                              s["status"], positions=s["positions"], columns=s["columns"],
                              interleaved=case["interleaved"])
    else:
        specdec.rotary_append(s["q"], s["k"], s["v"], s["cache"], s["layer"], s["table"], s["out"],
                              s["status"], n_committed=s["n"], width=s["width"],
                              parents=s["parents"], interleaved=case["interleaved"])
    return {"q": s["out"], "cache": s["cache"][s["layer"]]}


def _own_attention(s):
    from speculative_decoding_specdec_gb300 import specdec
    if "workspace" not in s:                    # kept by the program, made for the first pass
        need = specdec.tree_attention_workspace_bytes(s["q"], s["cache"])
        s["workspace"] = torch.zeros(max(need, 256), dtype=torch.uint8, device="cuda")
    specdec.tree_attention(s["q"], s["cache"], s["layer"], s["out"], s["n"], s["width"],
                           s["parents"], s["status"], s["workspace"])
    return s["out"]


def _own_greedy(s):
    from speculative_decoding_specdec_gb300 import specdec
    specdec.verify_tree_greedy(s["logits"], s["tokens"], s["parents"], s["accept_len"],
                               s["out_token"], s["path"], s["draft"], s["status"])
    return {"accept_len": s["accept_len"], "out_token": s["out_token"], "path": s["path"],
            "draft": s["draft"]}


def _own_sample(s):
    from speculative_decoding_specdec_gb300 import specdec
    specdec.verify_tree_sample(s["target_logits"], s["draft_logits"], s["tokens"], s["parents"],
                               s["uniforms"], s["case"]["temperature"], s["accept_len"],
                               s["out_token"], s["path"], s["draft"], s["status"],
                               replacement=s["case"]["replacement"])
    return {"accept_len": s["accept_len"], "out_token": s["out_token"], "path": s["path"],
            "draft": s["draft"]}


def _own_commit(s):
    from speculative_decoding_specdec_gb300 import specdec
    specdec.tree_commit(s["src"], s["dst"], s["width"], s["accept_len"], s["path"], s["status"],
                        width_dst=s["width_dst"])
    return s["dst"]


def _ancestors(parents, B, T):
    """[B, T, T] truth values: node j is node i or above it (a chain where parents is None)."""
    if parents is None:
        i = torch.arange(T, device="cuda")
        return (i[:, None] >= i[None]).expand(B, T, T), torch.arange(T, device="cuda").expand(B, T)
    step = (parents[:, :, None] == torch.arange(T, device="cuda")).float()
    above = step + torch.eye(T, device="cuda")
    for _ in range(5):                          # paths of up to 32 steps
        above = (above @ above).clamp_max(1.0)
    above = (above > 0) & (parents != UNUSED)[:, :, None]
    return above, above.sum(-1) - 1


def _rotated(x, cs, interleaved):
    """x [B, T, H, hd] float, cs [B, T, rot/2, 2]: the first rot values of each head rotated."""
    half = cs.shape[2]
    c, s = cs[:, :, None, :, 0], cs[:, :, None, :, 1]
    y = x.clone()
    one, two = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., one] * s + x[..., two] * c
    return y


def _plain_rotary(s):
    case, q = s["case"], s["q"]
    B, T = case["B"], case["T"]
    if case["prefill"]:
        pos, col, use = s["positions"].long(), s["columns"].long(), s["columns"] >= 0
    else:
        above, depth = _ancestors(s["parents"], B, T)
        use = above.any(-1)
        pos = (s["n"].long()[:, None] - 1 + depth).clamp_min(0)
        col = (s["width"].long() - 1 + torch.arange(T, device="cuda")).expand(B, T)
    cs = s["table"][pos]
    out = _rotated(q.float(), cs, case["interleaved"]) * use[:, :, None, None]
    k = _rotated(s["k"].float(), cs, case["interleaved"]).to(q.dtype)
    rows = torch.arange(B, device="cuda")[:, None].expand(B, T)
    b, c = rows[use], col[use]
    layer = s["cache"][s["layer"]]
    layer[0, b, :, c] = k[use]
    layer[1, b, :, c] = s["v"][use]
    return {"q": out.to(q.dtype), "cache": layer}


def _plain_attention(s):
    case, q = s["case"], s["q"]
    B, T, Hq, hd = q.shape
    k, v = s["cache"][s["layer"]].float()
    H, cap = k.shape[1], k.shape[2]
    above, _ = _ancestors(s["parents"], B, T)
    W = s["width"].long()
    col = torch.arange(cap, device="cuda")
    old = (col >= W - s["n"].long()[:, None]) & (col < W - 1)             # [B, cap]
    use = above.any(-1)                                                   # [B, T]
    see = old[:, None] & use[:, :, None]
    node = (col - (W - 1)).clamp(0, T - 1)
    new = above[:, :, node] & ((col >= W - 1) & (col < W - 1 + T))
    see = (see | new)[:, None, None]                                      # [B, 1, 1, T, cap]
    x = q.float().view(B, T, H, Hq // H, hd).permute(0, 2, 3, 1, 4)       # [B, H, G, T, hd]
    z = (x @ k[:, :, None].transpose(-1, -2)) / math.sqrt(hd)
    z = torch.where(see, z, float("-inf"))
    top = z.amax(-1, keepdim=True)
    e = torch.where(see, torch.exp(z - torch.where(top.isinf(), 0.0, top)), 0.0)
    out = (e @ v[:, :, None]) / e.sum(-1, keepdim=True).clamp_min(1e-30)
    return out.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, hd).to(q.dtype)


def _walked(s, cur, deep, path):
    """The verification's outputs from the last node, the depth and the nodes of each walk."""
    T = s["case"]["T"]
    draft = torch.where(path >= 0, s["tokens"].gather(1, path.clamp(0, T - 1).long()), 0)
    return deep, path, draft


def _plain_greedy(s):
    case, z = s["case"], s["logits"].float()
    B, T, D = case["B"], case["T"], case["D"]
    top = z.amax(-1, keepdim=True)
    index = torch.arange(case["V"], device="cuda", dtype=torch.int32)
    choice = torch.where(z == top, index, case["V"]).amin(-1)             # lowest index on ties
    rows = torch.arange(B, device="cuda")
    cur = torch.zeros(B, dtype=torch.int32, device="cuda")
    deep = torch.zeros_like(cur)
    path = torch.full((B, D), -1, dtype=torch.int32, device="cuda")
    slots = torch.arange(D, device="cuda", dtype=torch.int32)
    for i in range(1, T):                       # children come after their parents
        yes = (s["parents"][:, i] == cur) & (deep < D) & (s["tokens"][:, i] == choice[rows, cur.long()])
        path = torch.where(yes[:, None] & (slots == deep[:, None]), i, path)
        deep = deep + yes.int()
        cur = torch.where(yes, i, cur)
    deep, path, draft = _walked(s, cur, deep, path)
    return {"accept_len": deep, "out_token": choice[rows, cur.long()].int(), "path": path, "draft": draft}


def _softmax(x):
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_sample(s):
    case = s["case"]
    B, T, D = case["B"], case["T"], case["D"]
    rows, tok, par = torch.arange(B, device="cuda"), s["tokens"].long(), s["parents"]
    p = _softmax(s["target_logits"][:, 0].float() / case["temperature"])
    q = _softmax(s["draft_logits"][:, 0].float() / case["temperature"])
    cur = torch.zeros(B, dtype=torch.int32, device="cuda")
    deep = torch.zeros_like(cur)
    path = torch.full((B, D), -1, dtype=torch.int32, device="cuda")
    slots = torch.arange(D, device="cuda", dtype=torch.int32)
    index = torch.arange(case["V"], device="cuda")
    for i in range(1, T):                       # children come after their parents
        on = (par[:, i] == cur) & (deep < D)
        c = tok[:, i]
        pc, qc = p[rows, c], q[rows, c]
        yes = on & (s["uniforms"][:, i] * qc < pc)
        no = (on & ~yes)[:, None]
        r = (p - q).clamp_min(0.0)
        left = r.sum(-1, keepdim=True)
        p = torch.where(no & (left > 0), r / left, p)
        if not case["replacement"]:
            gone = torch.where(index == c[:, None], 0.0, q)
            q = torch.where(no, gone / gone.sum(-1, keepdim=True).clamp_min(1e-30), q)
        p = torch.where(yes[:, None], _softmax(s["target_logits"][:, i].float() / case["temperature"]), p)
        q = torch.where(yes[:, None], _softmax(s["draft_logits"][:, i].float() / case["temperature"]), q)
        path = torch.where(yes[:, None] & (slots == deep[:, None]), i, path)
        deep = deep + yes.int()
        cur = torch.where(yes, i, cur)
    below = torch.cumsum(p, -1)
    over = below > s["uniforms"][:, :1] * below[:, -1:]
    token = torch.where(over, index, case["V"] - 1).amin(-1).int()
    deep, path, draft = _walked(s, cur, deep, path)
    return {"accept_len": deep, "out_token": token, "path": path, "draft": draft}


def _plain_commit(s):
    B, D = s["path"].shape
    slot = torch.arange(D, device="cuda")
    b, i = torch.nonzero(slot < s["accept_len"][:, None], as_tuple=True)
    to = s["width_dst"].long() - 1 - s["accept_len"].long()[b] + i
    s["dst"][:, :, b, :, to] = s["src"][:, :, b, :, s["width"].long() - 1 + s["path"].long()[b, i]]
    return s["dst"]


# ------------------------------------------------------------------------- the same in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "rotary":
        return _exact_rotary(s)
    if case["kind"] == "attention":
        return _exact_attention(s)
    if case["kind"] == "commit":
        return _exact_commit(s)
    return None                                 # whole numbers


def _host_tree(s):
    """Per row and node, the node's ancestors and itself in order (an empty list if unused)."""
    B, T = s["case"]["B"], s["case"]["T"]
    if s["parents"] is None:
        return [[list(range(i + 1)) for i in range(T)] for _ in range(B)]
    par = s["parents"].cpu().numpy()
    return [[[0] + _path(par[b], i) if par[b, i] != UNUSED else [] for i in range(T)] for b in range(B)]


def _exact_rotary(s):
    case = s["case"]
    B, T, rot = case["B"], case["T"], case["rot"]
    n, W = s["n"].cpu().numpy(), int(s["width"])
    if case["prefill"]:
        pos, col = s["positions"].cpu().numpy(), s["columns"].cpu().numpy()
    else:
        lines = _host_tree(s)
        pos = np.array([[n[b] - 2 + len(lines[b][i]) for i in range(T)] for b in range(B)])
        col = np.array([[W - 1 + i if lines[b][i] else -1 for i in range(T)] for b in range(B)])
    table = s["table"].double()
    q, k = s["q"].double(), s["k"].double()
    layer = s["cache"][s["layer"]].double()
    out = torch.zeros_like(q)
    dims = torch.arange(rot, device="cuda")
    if case["interleaved"]:
        pair, mate, low = dims // 2, dims ^ 1, dims % 2 == 0
    else:
        pair, low = dims % (rot // 2), dims < rot // 2
        mate = torch.where(low, dims + rot // 2, dims - rot // 2)
    for b in range(B):
        t = np.flatnonzero(col[b] >= 0)
        if not len(t):
            continue
        at = torch.as_tensor(t).cuda()
        cs = table[torch.as_tensor(pos[b, t].astype(np.int64)).cuda()]
        c, sn = cs[:, pair, 0][:, None], cs[:, pair, 1][:, None]
        sn = torch.where(low, -sn, sn)
        for x, is_q in ((q[b, at], True), (k[b, at], False)):
            y = x.clone()
            y[..., :rot] = x[..., :rot] * c + x[..., mate] * sn
            if is_q:
                out[b, at] = y
            else:
                to = torch.as_tensor(col[b, t].astype(np.int64)).cuda()
                layer[0, b, :, to] = y.transpose(0, 1)
                layer[1, b, :, to] = s["v"][b, at].double().transpose(0, 1)
    return {"q": out, "cache": layer}


def _exact_commit(s):
    W, Wd, dst = int(s["width"]), int(s["width_dst"]), s["dst"].double()
    for b, (a, path) in enumerate(zip(s["accept_len"].tolist(), s["path"].tolist())):
        for i in range(a):                      # the last one ends just before the pending token
            dst[:, :, b, :, Wd - 1 - a + i] = s["src"][:, :, b, :, W - 1 + path[i]].double()
    return dst


def _exact_attention(s):
    case, q = s["case"], s["q"]
    B, T, Hq, hd = q.shape
    n, W, lines = s["n"].cpu().numpy(), int(s["width"]), _host_tree(s)
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    H = s["cache"].shape[3]
    for b in range(B):
        lo = W - int(n[b])
        see = torch.zeros(T, W - 1 - lo + T, dtype=torch.bool)
        for i in range(T):
            if lines[b][i]:
                see[i, :W - 1 - lo] = True
                see[i, [W - 1 - lo + j for j in lines[b][i]]] = True
        see = see.cuda()
        used = see.any(-1)
        for h in range(H):
            k, v = s["cache"][s["layer"], :, b, h, lo:W - 1 + T].double()
            x = q[b, :, h * (Hq // H):(h + 1) * (Hq // H)].double()
            z = torch.einsum("tgd,cd->gtc", x, k) * hd ** -0.5
            w = torch.softmax(z.masked_fill(~see, float("-inf")), -1).nan_to_num(0.0)
            y = torch.einsum("gtc,cd->tgd", w, v) * used[:, None, None]
            out[b, :, h * (Hq // H):(h + 1) * (Hq // H)] = y
    return out
