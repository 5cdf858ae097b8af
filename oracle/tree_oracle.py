"""CPU oracle of the tree-speculation operators (test infrastructure only; float64 numpy).

Written from the definitions, row by row and node by node, without any code of the product path:
a tree is ``parents`` (-1 for the root, -2 for a node the row does not use), siblings are ordered by
index.  The acceptance rules are those of "Inference Engineering: Part 5/8", "Exactness Means
Different Things For Greedy And Sampled Output", applied among the children of a node:
min(1, p/q), then normalize(max(0, p - q)); a sibling drawn without replacement leaves q without
the tokens drawn before it.
"""
import numpy as np


class TreeError(ValueError):
    pass


def line_of(parents, i):
    """Nodes from the root to node i ([] for an unused node)."""
    if parents[i] == -2:
        return []
    line = [int(i)]
    while line[-1] != 0:
        up = int(parents[line[-1]])
        if not 0 <= up < line[-1]:
            raise TreeError(f"parent {up} of node {line[-1]}")
        line.append(up)
    if parents[0] != -1:
        raise TreeError("the root's parent")
    return line[::-1]


def chain(T):
    return np.arange(T) - 1


def children(parents, node):
    return [i for i in range(1, len(parents)) if parents[i] == node]


def rotate(x, cos, sin, interleaved):
    """x [.., hd]; cos, sin [rot / 2]: the first rot values turned pair by pair."""
    y = np.array(x, np.float64)
    for i, (c, s) in enumerate(zip(cos, sin)):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + len(cos))
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def attention(q, k, v, old, parents, scale):
    """One batch row: q [T, Hq, hd]; k, v [H, old + T, hd] (committed columns, then the nodes').
    Returns out, lse [T, Hq], and the sums over the columns of p |v| and of (p v)^2."""
    T, Hq, hd = q.shape
    H = k.shape[0]
    out, sums, squares = (np.zeros((T, Hq, hd)) for _ in range(3))
    lse = np.full((T, Hq), -np.inf)
    for t in range(T):
        line = line_of(parents, t)
        if not line:
            continue
        cols = np.r_[np.arange(old), old + np.array(line)].astype(int)
        for h in range(Hq):
            kk, vv = k[h // (Hq // H)][cols], v[h // (Hq // H)][cols]
            z = scale * (kk @ q[t, h])
            m = z.max()
            w = np.exp(z - m)
            lse[t, h] = m + np.log(w.sum())
            p = w / w.sum()
            out[t, h] = p @ vv
            sums[t, h] = p @ np.abs(vv)
            squares[t, h] = (p ** 2) @ (vv ** 2)
    return out, lse, sums, squares


def greedy_choice(row):
    """Highest score, lowest index on ties; NaN never (None if there is nothing else)."""
    ok = ~np.isnan(row)
    if not ok.any():
        return None
    return int(np.flatnonzero(ok & (row == row[ok].max()))[0])


def verify_greedy(logits, tokens, parents, depth):
    """One batch row: (accepted nodes, token or None)."""
    if parents[0] == -2:
        return [], -1
    node, path = 0, []
    while True:
        choice = greedy_choice(logits[node])
        if choice is None:
            return path, None
        nxt = [c for c in children(parents, node) if tokens[c] == choice]
        if len(path) == depth or not nxt:
            return path, choice
        node = nxt[0]
        path.append(node)


def softmax(x):
    e = np.exp(x - x.max())
    return e / e.sum()


def verify_sample(target, draft, tokens, parents, u, temperature, depth, replacement):
    """One batch row: (accepted nodes, token, distribution of the draw, margins).  A margin is how
    far a decision was from turning (|u - p/q| of every test made)."""
    if parents[0] == -2:
        return [], -1, None, []
    node, path, margins = 0, [], []
    while True:
        p = softmax(target[node] / temperature)
        kids = children(parents, node) if len(path) < depth else []
        q = softmax(draft[node] / temperature) if kids else None
        accepted = None
        for c in kids:
            x = tokens[c]
            if not 0 <= x < len(p):
                continue
            ratio = p[x] / q[x] if q[x] > 0 else (np.inf if p[x] > 0 else 0.0)
            margins.append(abs(u[c] - ratio))
            if u[c] < ratio:
                accepted = c
                break
            r = np.maximum(p - q, 0)
            if r.sum() > 0:
                p = r / r.sum()
            if not replacement:
                q = q.copy()
                q[x] = 0
                if q.sum() > 0:
                    q = q / q.sum()
        if accepted is None:
            edges = np.cumsum(p)
            over = np.flatnonzero(edges > u[0] * edges[-1])
            return path, int(over[0]), p, margins
        node = accepted
        path.append(node)


def one_step_distribution(p, q, tokens, replacement):
    """Probability of each next token when a node's children carry ``tokens`` in order (given those
    tokens): mass accepted at each child, and the draw's."""
    out, left = np.zeros_like(p), 1.0
    p, q = p.copy(), q.copy()
    for x in tokens:
        acc = min(1.0, p[x] / q[x]) if q[x] > 0 else float(p[x] > 0)
        out[x] += left * acc
        left *= 1 - acc
        r = np.maximum(p - q, 0)
        if r.sum() > 0:
            p = r / r.sum()
        if not replacement:
            q[x] = 0
            if q.sum() > 0:
                q /= q.sum()
    return out + left * p
