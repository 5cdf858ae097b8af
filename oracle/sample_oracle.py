"""CPU oracle of drawing tokens with sampling settings (test infrastructure only; float64 numpy).

Written from the definitions, without any code of the product path: tokens in order of score (highest
first, ties by lower index); top-k keeps the first k of them, top-p those before which less than
top_p of their mass lies, min-p those with at least min_p times the highest probability; the draw is
the first kept token by index whose running probability exceeds u.  ("Inference Engineering: Part
5/8", "Draft Possible Tokens, Then Verify Them Together": sampling settings such as temperature and
top-p.)
"""
import numpy as np


def masses(x, temperature):
    """exp((x - max) / T) of a row."""
    x = np.asarray(x, np.float64)
    return np.exp((x - x.max()) / np.float64(np.float32(temperature)))


def order_of(x):
    return np.lexsort((np.arange(len(x)), -np.asarray(x, np.float64)))


def kept(x, temperature, top_k=0, top_p=1.0, min_p=0.0):
    """Kept tokens of a row, in order of score."""
    x = np.asarray(x, np.float64)
    order = order_of(x)
    if temperature == 0:
        return order[:1]
    if 0 < top_k < len(x):
        order = order[:top_k]
    e = masses(x, temperature)
    if top_p < 1:
        m = e[order]
        before = np.concatenate(([0.0], np.cumsum(m)[:-1]))
        order = order[before < np.float64(np.float32(top_p)) * m.sum()]
    if min_p > 0:
        cut = x.max() + np.float64(np.float32(temperature)) * np.log(np.float64(np.float32(min_p)))
        order = order[x[order] >= cut]
    return order


def draw(x, temperature, keep, u):
    """(token, logprob, edges, ids): the running probabilities of the kept tokens by index."""
    ids = np.sort(keep)
    if temperature == 0:
        return int(ids[0]), 0.0, np.ones(1), ids
    e = masses(x, temperature)[ids]
    edges = np.cumsum(e) / e.sum()
    at = min(int(np.searchsorted(edges, np.float64(np.float32(u)), side="right")), len(ids) - 1)
    with np.errstate(divide="ignore"):
        return int(ids[at]), float(np.log(e[at] / e.sum())), edges, ids


def keep_from_bound(x, key, index):
    """Tokens that a keep bound keeps."""
    f = np.asarray(x, np.float32)
    bits = np.where(f == 0, np.float32(0), f).view(np.uint32)
    code = np.where(bits >> 31, ~bits, bits | np.uint32(1 << 31))
    return np.flatnonzero((code > key) | ((code == key) & (np.arange(len(f)) <= index)))
