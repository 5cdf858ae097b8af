"""Measured cases of the operators of a pass over a batch that shares its prompts: norms of queries
and keys with rotary positions and the append to the K/V cache, attention over a shared prefix and
the rows' own columns, and the drawing of tokens with sampling settings.

Rows of one group were begun with the same prompt, whose K/V is held once: prefix p has
``prefix_len[p]`` columns at the start of row p of ``prefix`` [L, 2, P, H, cap, hd], and rows
``group_start[p]`` .. ``group_start[p + 1]`` of the batch belong to it.  What a row has of its own is
a left-padded batch as elsewhere: N_b committed tokens that end at column W - 1 of ``cache``
[L, 2, B, H, cap, hd], and T new nodes (``parents`` [B, T], -2 for one that the row does not use, None
for a chain) from column W - 1 on, at positions prefix + N_b - 1 + depth.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
UNUSED = -2


# ------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # The smallest call: one new token of two rows of a tiny fp32 model; latency counts.
        dict(name="norm_rotary_tiny", kind="norm_rotary", B=2, T=1, Hq=4, Hkv=2, hd=64, rot=64,
             interleaved=False, dtype="fp32", lo=5, hi=20, tree=False, prefill=False, shared=16,
             offset=0.0),
        # A verification pass of 32-node trees at the Qwen3-8B head layout (which norms its heads),
        # behind a shared prompt.
        dict(name="norm_rotary_tree_qwen3_8b", kind="norm_rotary", B=16, T=32, Hq=32, Hkv=8, hd=128,
             rot=128, interleaved=False, dtype="bf16", lo=64, hi=1024, tree=True, prefill=False,
             shared=4096, offset=0.0),
        # Prefill of a ragged batch of prompts at the same layout: the bandwidth end.
        dict(name="norm_rotary_prefill_qwen3_8b", kind="norm_rotary", B=8, T=1024, Hq=32, Hkv=8,
             hd=128, rot=128, interleaved=False, dtype="bf16", lo=128, hi=1024, tree=False,
             prefill=True, shared=0, offset=0.0),
        # The smallest attention: two samples of one short prompt, one new token each.
        dict(name="prefix_tiny", kind="prefix", B=2, T=1, Hq=4, Hkv=2, hd=64, dtype="fp32", P=1,
             shared=100, lo=2, hi=20, tree=False),
        # Single-token decoding of eight samples of one prompt at the Vicuna-7B head layout: few
        # query rows per K/V head, so the reading of K/V bounds it.
        dict(name="prefix_decode_vicuna7b", kind="prefix", B=8, T=1, Hq=32, Hkv=32, hd=128,
             dtype="bf16", P=1, shared=2048, lo=16, hi=256, tree=False),
        # Single-token decoding of 64 samples of one long document at the Qwen3-8B head layout.
        dict(name="prefix_decode_qwen3_8b", kind="prefix", B=64, T=1, Hq=32, Hkv=8, hd=128,
             dtype="bf16", P=1, shared=65537, lo=16, hi=512, tree=False),
        # Chains of five drafts and the pending token, four prompts of unequal length with unequal
        # numbers of samples, at the Qwen3-8B head layout.
        dict(name="prefix_chain_qwen3_8b", kind="prefix", B=32, T=6, Hq=32, Hkv=8, hd=128,
             dtype="bf16", P=4, shared=6000, lo=16, hi=512, tree=False),
        # 32-node trees of 32 samples of one prompt at the GLM-4-9B head layout: 16384 query rows
        # per K/V head over the prompt, so the matrix products bound it.
        dict(name="prefix_tree_glm4_9b", kind="prefix", B=32, T=32, Hq=32, Hkv=2, hd=128,
             dtype="bf16", P=1, shared=8192, lo=64, hi=1024, tree=True),
        # Tokens of a tiny batch: the smallest draw.
        dict(name="sample_tiny", kind="sample", R=2, V=1000, dtype="fp32", settings="top_p"),
        # The next tokens of eight rows at the Vicuna-7B vocabulary, top-p alone.
        dict(name="sample_vicuna7b", kind="sample", R=8, V=32000, dtype="bf16", settings="top_p"),
        # Requests with settings of their own (greedy ones among them) at the Qwen3-8B vocabulary.
        dict(name="sample_qwen3_8b", kind="sample", R=64, V=151936, dtype="bf16", settings="mixed"),
        # A large batch with the temperature alone at the GLM-4-9B vocabulary, fp32 scores.
        dict(name="sample_glm4_9b", kind="sample", R=256, V=151552, dtype="fp32", settings="none"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["norm_rotary", "prefix", "prefix", "sample"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    Hq, Hkv = rng.choice([(32, 32), (32, 8), (32, 2), (8, 2), (4, 4)])
    hd = rng.choice([64, 128, 128])
    T = _log(rng, 1, 64)
    if kind == "norm_rotary":
        prefill = rng.random() < 0.4
        T = _log(rng, 16, 1024) if prefill else T
        lo = _log(rng, 1, T) if prefill else _log(rng, 1, 2048)
        return dict(kind=kind, B=_log(rng, 1, 8 if prefill else 32), T=T, Hq=Hq,
                    Hkv=min(Hkv, 8) if prefill else Hkv, hd=hd, rot=rng.choice([hd, hd // 2]),
                    interleaved=rng.random() < 0.5, dtype="bf16" if prefill else dtype, lo=lo,
                    hi=T if prefill else _log(rng, lo, 2048),
                    tree=not prefill and T > 1 and rng.random() < 0.7, prefill=prefill,
                    shared=rng.choice([0, _log(rng, 1, 8192)]), offset=rng.choice([0.0, 1.0]))
    if kind == "prefix":
        hi = _log(rng, 2, 1024)
        B = _log(rng, 1, 64)
        c = dict(kind=kind, B=B, T=T, Hq=Hq, Hkv=Hkv, hd=hd, dtype=dtype,
                 P=rng.choice([1, 1, min(B, rng.randint(1, 5))]), shared=_log(rng, 1, 65537),
                 lo=_log(rng, 1, hi), hi=hi, tree=T > 1 and rng.random() < 0.5)
        tree, long = (work(listed()[i]) for i in (7, 5))
        # fp32 has no tensor cores: its cases are kept to a sixteenth of the products
        flops = tree["flops"] / (16 if dtype == "fp32" else 1)
        while c["shared"] > 1 and (work(c)["flops"] > flops or work(c)["bytes"] > long["bytes"]
                                   or c["B"] * c["T"] * c["Hq"] * c["shared"] > 2 ** 28):
            if c["B"] > c["P"]:
                c["B"] = max(c["P"], c["B"] * 3 // 4)
            else:
                c["shared"] = max(1, c["shared"] * 3 // 4)
        return c
    V = rng.choice([_log(rng, 100, 152000), 32000, 151936, 151552])
    return dict(kind=kind, R=_log(rng, 1, 256), V=V, dtype=dtype,
                settings=rng.choice(["none", "top_k", "top_p", "min_p", "mixed", "mixed"]))


# -------------------------------------------------------------------- what a case fixes by itself

def _lengths(case):
    """N_b, spread evenly over [lo, hi]; the seed permutes them."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi if B == 1 else lo + (hi - lo) * b // (B - 1) for b in range(B)]


def _used(case):
    """Nodes each row uses: trees of one batch drop up to a quarter of them from the end."""
    T = case["T"]
    return [T - (5 * b) % (T // 4 + 1) if case["tree"] else T for b in range(case["B"])]


def _groups(case):
    """Bounds of the groups: the first ones have more rows than the last."""
    B, P = case["B"], case["P"]
    weight = [P - p + 1 for p in range(P)]
    at, total = [0], sum(weight)
    for p in range(P):
        at.append(max(at[-1] + 1, B * sum(weight[:p + 1]) // total))
    at = [min(x, B - (P - i)) for i, x in enumerate(at)]
    at[P] = B
    return at


def _prefix_lengths(case):
    """The first prefix has `shared` columns, the others less and less."""
    return [max(1, case["shared"] - p * case["shared"] // (case["P"] + 1)) for p in range(case["P"])]


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    kind = case["kind"]
    if kind == "sample":
        n = case["R"] * case["V"]
        # one exponential and two sums per score
        return {"bytes": n * es + case["R"] * 28, "flops": 4 * n}
    if kind == "norm_rotary":
        n = sum(_lengths(case)) if case["prefill"] else sum(_used(case))
        skipped = case["B"] * case["T"] - n            # their q rows are written as zeros
        values = n * case["hd"] * (2 * case["Hq"] + 4 * case["Hkv"]) + skipped * case["hd"] * case["Hq"]
        return {"bytes": values * es + n * case["rot"] * 4 + n * 8,
                "flops": n * (case["Hq"] + case["Hkv"]) * (3.0 * case["rot"] + 4.0 * case["hd"])}
    used, n, at = _used(case), _lengths(case), _groups(case)
    own_cols = sum(n) - case["B"] + sum(used)
    shared = _prefix_lengths(case)
    pairs = sum(t * x for t, x in zip(used, n))          # and the tree's few
    pairs += sum(s * sum(used[at[p]:at[p + 1]]) for p, s in enumerate(shared))
    return {"bytes": ((own_cols + sum(shared)) * case["Hkv"] * 2 + sum(used) * case["Hq"]
                      + case["B"] * case["T"] * case["Hq"]) * case["hd"] * es,
            "flops": 4.0 * pairs * case["Hq"] * case["hd"]}


# --------------------------------------------------------------------------------------- inputs

def _tree(case, rs):
    """parents [B, T]: each node under one of the eight before it."""
    B, T = case["B"], case["T"]
    p = np.full((B, T), UNUSED, np.int32)
    for b, used in enumerate(_used(case)):
        p[b, 0] = -1
        for i in range(1, used):
            p[b, i] = max(0, i - 1 - int(rs.random_sample() ** 2 * 8))
    return p


def _randn(gen, shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen)


def _int(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def _float(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.float32).cuda()


def prepare(case, seed):
    rs = np.random.RandomState(seed % (2 ** 32))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if case["kind"] == "sample":
        return _prepare_sample(s, rs, gen, dt)
    B, T, Hkv, hd = case["B"], case["T"], case["Hkv"], case["hd"]
    n = np.asarray(_lengths(case), np.int32)
    rs.shuffle(n)
    W = int(n.max())
    cap = W + T + 1
    s["n"], s["width"] = _int(n), _int([W])
    s["parents"] = _int(_tree(case, rs)) if case["tree"] else None
    s["q"] = _randn(gen, (B, T, case["Hq"], hd), dt)
    # two layers, so that a layer's caches are read where a model's would lie
    s["cache"] = _randn(gen, (2, 2, B, Hkv, cap, hd), dt)
    s["layer"] = 1
    s["out"] = torch.empty_like(s["q"])
    if case["kind"] == "prefix":
        lengths = _prefix_lengths(case)
        s["prefix"] = _randn(gen, (2, 2, case["P"], Hkv, max(lengths) + 3, hd), dt)
        s["prefix_len"], s["group_start"] = _int(lengths), _int(_groups(case))
        return s
    s["q"].mul_(3.0)                            # what a projection gives before its norm
    s["k"] = _randn(gen, (B, T, Hkv, hd), dt).mul_(2.0)
    s["v"] = _randn(gen, (B, T, Hkv, hd), dt)
    mean = 1.0 - case["offset"]                 # some models hold their weights less one
    s["q_weight"] = (_randn(gen, (hd,), torch.float32) * 0.3 + mean).to(dt)
    s["k_weight"] = (_randn(gen, (hd,), torch.float32) * 0.3 + mean).to(dt)
    s["eps"] = 1e-6
    # positions' cosines and sines, made once per model in 64 bits
    half = case["rot"] // 2
    freq = 1e6 ** (-torch.arange(half, dtype=torch.float64) / half)
    angle = torch.arange(case["shared"] + cap, dtype=torch.float64)[:, None] * freq
    s["table"] = torch.stack((angle.cos(), angle.sin()), -1).float().cuda()
    if case["prefill"]:
        t = np.arange(T)[None]
        held = t < n[:, None]                   # row b's prompt has n_b tokens
        s["positions"] = _int(np.where(held, t, 0))
        s["columns"] = _int(np.where(held, W - n[:, None] + t, -1))
    s["start"] = _int(np.full(B, case["shared"])) if case["shared"] else None
    return s


def _prepare_sample(s, rs, gen, dt):
    """Scores with a few likely tokens and some dozens of possible ones over a long tail."""
    case = s["case"]
    R, V = case["R"], case["V"]
    z = _randn(gen, (R, V), torch.float32).mul_(1.5)
    count = min(56, V // 4)                     # in as many stretches of the vocabulary, one in each
    at = torch.randint(0, V // count, (R, count), generator=gen, device="cuda")
    at += torch.arange(count, device="cuda") * (V // count)
    rank = torch.rand(R, count, generator=gen, device="cuda").argsort(-1)
    lift = math.log(V) + torch.where(rank < 8, 1.5 - 0.7 * rank, -3.0 - 0.05 * rank)
    z.scatter_(1, at, lift + 0.5 * torch.randn(R, count, generator=gen, device="cuda"))
    s["logits"] = z.to(dt)
    kind = case["settings"]
    mixed = kind == "mixed"
    s["temperature"] = _float(rs.choice([0.0, 0.6, 0.7, 1.0, 1.3] if mixed else [0.7, 1.0], R))
    for name, to, alone, off in (("top_k", _int, [20, 50, 1000], 0),
                                 ("top_p", _float, [0.8, 0.9, 0.95, 0.99], 1.0),
                                 ("min_p", _float, [0.02, 0.05, 0.1], 0.0)):
        s[name] = to(rs.choice(alone + [off] if mixed else alone, R)) if kind in (name, "mixed") else None
    s["token"] = torch.zeros(R, dtype=torch.int32, device="cuda")
    s["logprob"] = torch.zeros(R, dtype=torch.float32, device="cuda")
    # Random numbers that a hair's breadth does not turn: where one lies within 1e-7 of the border
    # between two tokens, the last bits of the exponentials decide, and another is drawn.
    tries = torch.rand(R, 8, generator=gen, device="cuda")
    edges = _kept_mass(s).cumsum(-1)
    edges /= edges[:, -1:].clone()
    k = torch.searchsorted(edges, tries.double(), right=True).clamp_max(V - 1)
    hi = edges.gather(1, k)
    lo = torch.where(k > 0, edges.gather(1, (k - 1).clamp_min(0)), torch.full_like(hi, -1.0))
    room = torch.minimum(hi - tries, tries - lo)
    best = torch.where((room > 1e-7).any(1), (room > 1e-7).float().argmax(1), room.argmax(1))
    s["uniforms"] = tries.gather(1, best[:, None])[:, 0].contiguous()
    return s


# ----------------------------------------------------------------------------------- one pass

def run(s):
    kind = s["case"]["kind"]
    if own:
        return {"norm_rotary": _own_norm_rotary, "prefix": _own_prefix, "sample": _own_sample}[kind](s)
    return {"norm_rotary": _plain_norm_rotary, "prefix": _plain_prefix, "sample": _plain_sample}[kind](s)


def _own_norm_rotary(s):
    from speculative_decoding_specdec_gb300 import specdec
    where = (dict(positions=s["positions"], columns=s["columns"]) if s["case"]["prefill"]
             else dict(n_committed=s["n"], width=s["width"], parents=s["parents"]))
    specdec.norm_rotary_append(s["q"], s["k"], s["v"], s["cache"], s["layer"], s["table"], s["out"],
                               s["status"], s["q_weight"], s["k_weight"], eps=s["eps"],
                               weight_offset=s["case"]["offset"], start=s["start"],
                               interleaved=s["case"]["interleaved"], **where)
    return {"q": s["out"], "cache": s["cache"][s["layer"]]}


def _own_prefix(s):
    from speculative_decoding_specdec_gb300 import specdec
    if "workspace" not in s:                    # kept by the program, made for the first pass
        need = specdec.prefix_attention_workspace_bytes(s["q"], s["cache"], s["case"]["P"])
        s["workspace"] = torch.zeros(max(need, 256), dtype=torch.uint8, device="cuda")
    specdec.prefix_attention(s["q"], s["cache"], s["layer"], s["out"], s["n"], s["width"],
                             s["parents"], s["status"], s["workspace"], s["prefix"],
                             s["prefix_len"], s["group_start"])
    return s["out"]


def _own_sample(s):
    from speculative_decoding_specdec_gb300 import specdec
    specdec.sample(s["logits"], s["uniforms"], s["token"], s["status"],
                   temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                   min_p=s["min_p"], logprob=s["logprob"])
    return {"token": s["token"], "logprob": s["logprob"]}


def _ancestors(parents, B, T):
    """[B, T, T] truth values: node j is node i or above it (a chain where parents is None)."""
    if parents is None:
        i = torch.arange(T, device="cuda")
        return (i[:, None] >= i[None]).expand(B, T, T)
    step = (parents[:, :, None] == torch.arange(T, device="cuda")).float()
    above = step + torch.eye(T, device="cuda")
    for _ in range(6):                          # paths of up to 64 steps
        above = (above @ above).clamp_max(1.0)
    return (above > 0) & (parents != UNUSED)[:, :, None]


def _normed(x, weight, case, eps):
    y = x.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + eps)
    return y * (weight.float() + case["offset"])


def _rotated(x, cs, interleaved):
    """x [B, T, H, hd] float, cs [B, T, rot/2, 2]: the first rot values of each head rotated."""
    half = cs.shape[2]
    c, s = cs[:, :, None, :, 0], cs[:, :, None, :, 1]
    y = x.clone()
    one, two = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., one] * s + x[..., two] * c
    return y


def _plain_norm_rotary(s):
    case, q = s["case"], s["q"]
    B, T = case["B"], case["T"]
    if case["prefill"]:
        pos, col, use = s["positions"].long(), s["columns"].long(), s["columns"] >= 0
    else:
        above = _ancestors(s["parents"], B, T)
        use = above.any(-1)
        pos = (s["n"].long()[:, None] - 2 + above.sum(-1)).clamp_min(0)
        col = (s["width"].long() - 1 + torch.arange(T, device="cuda")).expand(B, T)
    if s["start"] is not None:
        pos = pos + s["start"].long()[:, None]
    cs = s["table"][pos]
    out = _rotated(_normed(q, s["q_weight"], case, s["eps"]), cs, case["interleaved"])
    k = _rotated(_normed(s["k"], s["k_weight"], case, s["eps"]), cs, case["interleaved"]).to(q.dtype)
    out = torch.where(use[:, :, None, None], out, 0.0)
    rows = torch.arange(B, device="cuda")[:, None].expand(B, T)
    b, c = rows[use], col[use]
    layer = s["cache"][s["layer"]]
    layer[0, b, :, c] = k[use]
    layer[1, b, :, c] = s["v"][use]
    return {"q": out.to(q.dtype), "cache": layer}


def _plain_prefix(s):
    case, q = s["case"], s["q"]
    B, T, Hq, hd = q.shape
    k, v = s["cache"][s["layer"]].float()
    H, cap = k.shape[1], k.shape[2]
    above = _ancestors(s["parents"], B, T)
    W = s["width"].long()
    col = torch.arange(cap, device="cuda")
    old = (col >= W - s["n"].long()[:, None]) & (col < W - 1)             # [B, cap]
    use = above.any(-1)                                                   # [B, T]
    node = (col - (W - 1)).clamp(0, T - 1)
    new = above[:, :, node] & ((col >= W - 1) & (col < W - 1 + T))
    see = ((old[:, None] & use[:, :, None]) | new)[:, None, None]         # [B, 1, 1, T, cap]
    x = q.float().view(B, T, H, Hq // H, hd).permute(0, 2, 3, 1, 4)       # [B, H, G, T, hd]
    x = x / math.sqrt(hd)
    z = torch.where(see, x @ k[:, :, None].transpose(-1, -2), float("-inf"))
    out = torch.zeros(B, H, Hq // H, T, hd, device="cuda")
    pk, pv = s["prefix"][s["layer"]].float()
    for p, (n, b0, b1) in enumerate(zip(_prefix_lengths(case), _groups(case), _groups(case)[1:])):
        # every row's queries against the one copy of the prefix
        rows = x[b0:b1].permute(1, 0, 2, 3, 4).reshape(H, -1, hd)
        zp = (rows @ pk[p, :, :n].transpose(-1, -2)).view(H, b1 - b0, Hq // H, T, n).transpose(0, 1)
        top = torch.maximum(z[b0:b1].amax(-1, keepdim=True), zp.amax(-1, keepdim=True))
        e, ep = torch.exp(z[b0:b1] - top), torch.exp(zp - top)
        del zp
        total = e.sum(-1, keepdim=True) + ep.sum(-1, keepdim=True)
        got = (ep.transpose(0, 1).reshape(H, -1, n) @ pv[p, :, :n]).view(H, b1 - b0, Hq // H, T, hd)
        out[b0:b1] = (got.transpose(0, 1) + e @ v[b0:b1, :, None]) / total
    out = torch.where(use[:, None, None, :, None], out, 0.0)
    return out.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, hd).to(q.dtype)


def _kept_mass(s):
    """[R, V] in 64 bits: exp((x - max) / T) of the tokens that the settings keep, else zero.  In
    order of score (lowest index first among equals) top-k keeps the first k, then top-p those with
    less than top_p of the mass of these before them; min-p keeps what has min_p of the highest
    probability.  A temperature of zero keeps the first token of that order alone."""
    x = s["logits"].double()
    R, V = x.shape
    t = s["temperature"].double()[:, None]
    top = x.amax(-1, keepdim=True)
    e = torch.exp((x - top) / torch.where(t > 0, t, 1.0))
    keep = torch.ones(R, V, dtype=torch.bool, device="cuda")
    if s["top_k"] is not None or s["top_p"] is not None:
        order = torch.sort(x, dim=-1, descending=True, stable=True).indices
        e_in = e.gather(1, order)
        first = torch.ones_like(keep)
        if s["top_k"] is not None:
            k = torch.where(s["top_k"] > 0, s["top_k"], V).long()[:, None]
            first = torch.arange(V, device="cuda") < k
        if s["top_p"] is not None:
            e_in = torch.where(first, e_in, 0.0)
            before = e_in.cumsum(-1) - e_in
            p = s["top_p"].double()[:, None]
            first = first & ((before < p * e_in.sum(-1, keepdim=True)) | (p >= 1))
        keep.scatter_(1, order, first)
    if s["min_p"] is not None:
        m = s["min_p"].double()[:, None]
        keep = keep & (x >= top + torch.where(t > 0, t, 1.0) * torch.log(m))
    index = torch.arange(V, device="cuda")
    best = torch.where(x == top, index, V).amin(-1, keepdim=True)
    keep = torch.where(t > 0, keep, index == best)
    return torch.where(keep, e, 0.0)


def _plain_sample(s):
    e = _kept_mass(s)
    below = e.cumsum(-1)
    index = torch.arange(e.shape[1], device="cuda")
    u = s["uniforms"].double()[:, None]
    token = torch.where((below > u * below[:, -1:]) & (e > 0), index, e.shape[1] - 1).amin(-1)
    logprob = torch.log(e.gather(1, token[:, None])[:, 0] / below[:, -1])
    return {"token": token.int(), "logprob": logprob.float()}


# ------------------------------------------------------------------------- the same in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rotary": _exact_norm_rotary, "prefix": _exact_prefix, "sample": _exact_sample}[case["kind"]](s)


def _lines(s):
    """Per row and node, the node's ancestors and itself in order (an empty list if unused)."""
    B, T = s["case"]["B"], s["case"]["T"]
    if s["parents"] is None:
        return [[list(range(i + 1)) for i in range(T)] for _ in range(B)]
    got = []
    for par in s["parents"].cpu().tolist():
        row = []
        for i in range(T):
            line, j = [], i if par[i] != UNUSED else -1
            while j >= 0:
                line.append(j)
                j = par[j]
            row.append(line[::-1])
        got.append(row)
    return got


def _exact_norm_rotary(s):
    case = s["case"]
    B, T, rot = case["B"], case["T"], case["rot"]
    n, W = s["n"].tolist(), int(s["width"])
    if case["prefill"]:
        pos, col = s["positions"].cpu().numpy().astype(np.int64), s["columns"].cpu().numpy()
    else:
        lines = _lines(s)
        pos = np.array([[n[b] - 2 + len(lines[b][i]) for i in range(T)] for b in range(B)])
        col = np.array([[W - 1 + i if lines[b][i] else -1 for i in range(T)] for b in range(B)])
    if s["start"] is not None:
        pos = pos + s["start"].cpu().numpy()[:, None]
    table = s["table"].double()
    layer = s["cache"][s["layer"]].double()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(B):
        t = np.flatnonzero(col[b] >= 0)
        if not len(t):
            continue
        at = torch.as_tensor(t).cuda()
        angle = torch.view_as_complex(table[torch.as_tensor(pos[b, t]).cuda()])[:, None]
        for name in "qk":
            x = s[name][b, at].double()
            x /= torch.sqrt((x ** 2).sum(-1, keepdim=True) / case["hd"] + s["eps"])
            x *= s[name + "_weight"].double() + case["offset"]
            y = x[..., :rot]
            pairs = y.unflatten(-1, (-1, 2)) if case["interleaved"] else y.unflatten(-1, (2, -1)).transpose(-1, -2)
            turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * angle)
            x[..., :rot] = (turned if case["interleaved"] else turned.transpose(-1, -2)).flatten(-2)
            if name == "q":
                out[b, at] = x
            else:
                to = torch.as_tensor(col[b, t].astype(np.int64)).cuda()
                layer[0, b, :, to] = x.transpose(0, 1)
                layer[1, b, :, to] = s["v"][b, at].double().transpose(0, 1)
    return {"q": out, "cache": layer}


def _exact_prefix(s):
    case, q = s["case"], s["q"]
    B, T, Hq, hd = q.shape
    if case["B"] * case["T"] * Hq * case["shared"] > 2 ** 29:
        return None                             # (minutes in 64 bits)
    n, W, lines = s["n"].tolist(), int(s["width"]), _lines(s)
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    H = s["cache"].shape[3]
    at = _groups(case)
    for p, shared in enumerate(_prefix_lengths(case)):
        for b in range(at[p], at[p + 1]):
            lo = W - n[b]
            see = torch.zeros(T, shared + n[b] - 1 + T, dtype=torch.bool)
            for i, line in enumerate(lines[b]):
                if line:
                    see[i, :shared + n[b] - 1] = True
                    see[i, [shared + n[b] - 1 + j for j in line]] = True
            see = see.cuda()
            used = see.any(-1)
            for h in range(H):
                k, v = (torch.cat((s["prefix"][s["layer"], j, p, h, :shared],
                                   s["cache"][s["layer"], j, b, h, lo:W - 1 + T])).double() for j in (0, 1))
                heads = slice(h * (Hq // H), (h + 1) * (Hq // H))
                z = torch.einsum("tgd,cd->gtc", q[b, :, heads].double(), k) * hd ** -0.5
                w = torch.softmax(z.masked_fill(~see, float("-inf")), -1).nan_to_num(0.0)
                out[b, :, heads] = torch.einsum("gtc,cd->tgd", w, v) * used[:, None, None]
    return out


def _exact_sample(s):
    """Row by row, the kept tokens as a list in order of score."""
    case = s["case"]
    x = s["logits"].double().cpu().numpy()
    settings = {name: None if s[name] is None else s[name].cpu().numpy().astype(np.float64)
                for name in ("temperature", "top_k", "top_p", "min_p", "uniforms")}
    token, logprob = np.zeros(case["R"], np.int32), np.zeros(case["R"])
    for r in range(case["R"]):
        t = settings["temperature"][r]
        order = np.argsort(-x[r], kind="stable")
        if t == 0:
            token[r] = order[0]
            continue
        k = 0 if settings["top_k"] is None else int(settings["top_k"][r])
        order = order[:k] if k > 0 else order
        p = np.exp((x[r][order] - x[r][order[0]]) / t)
        if settings["top_p"] is not None and settings["top_p"][r] < 1:
            before = np.concatenate(([0.0], np.cumsum(p)[:-1]))
            order = order[before < settings["top_p"][r] * p.sum()]
        if settings["min_p"] is not None and settings["min_p"][r] > 0:
            order = order[x[r][order] >= x[r][order[0]] + t * np.log(settings["min_p"][r])]
        order = np.sort(order)
        p = np.exp((x[r][order] - x[r][order].max()) / t)
        below = np.cumsum(p)
        at = int(np.argmax(below > settings["uniforms"][r] * below[-1]))
        token[r] = order[at]
        logprob[r] = np.log(p[at] / below[-1])
    return {"token": torch.as_tensor(token).cuda(), "logprob": torch.as_tensor(logprob).cuda()}
