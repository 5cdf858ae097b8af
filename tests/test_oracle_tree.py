"""The tree oracle against what the method fixes: the tests among siblings leave the target's own
distribution, chains are trees, rotations keep lengths and depend on position differences."""
import itertools

import numpy as np
import pytest

import oracle.specdec_oracle as O
import oracle.tree_oracle as TO


@pytest.mark.parametrize("replacement", [True, False])
@pytest.mark.parametrize("kids", [1, 2, 3])
def test_next_token_has_the_targets_distribution(replacement, kids):
    rng = np.random.default_rng(kids)
    V = 5
    p, q = TO.softmax(rng.normal(size=V)), TO.softmax(rng.normal(size=V))
    total = np.zeros(V)
    for toks in itertools.product(range(V), repeat=kids):
        w, left = 1.0, q.copy()
        for x in toks:                       # probability of drawing these siblings in order
            w *= left[x]
            if not replacement:
                left[x] = 0
                left = left / left.sum() if left.sum() > 0 else left
        if w > 0:
            total += w * TO.one_step_distribution(p, q, toks, replacement)
    np.testing.assert_allclose(total, p, atol=1e-12)


def test_a_chain_is_a_tree():
    rng = np.random.default_rng(0)
    D, V = 4, 9
    for _ in range(30):
        logits, tok = rng.normal(size=(D + 1, V)), rng.integers(0, V, D)
        for j in range(D):
            if rng.random() < 0.7:
                logits[j, tok[j]] = 9
        a, y = O.verify_greedy(logits[None], tok[None])
        path, t = TO.verify_greedy(logits, np.r_[0, tok], TO.chain(D + 1), D)
        assert (len(path), t) == (a[0], y[0]) and path == list(range(1, a[0] + 1))
        dl, u = logits[:D] + rng.normal(size=(D, V)) * 0.5, rng.random(D + 1)
        a, y = O.verify_sample(logits[None], dl[None], tok[None], u[None], 0.8)[:2]
        path, t, _, _ = TO.verify_sample(logits, np.r_[dl, dl[:1]], np.r_[0, tok], TO.chain(D + 1),
                                         np.r_[u[D], u[:D]], 0.8, D, False)
        assert (len(path), t) == (a[0], y[0])


def test_lines_and_bad_trees():
    par = np.array([-1, 0, 0, 1, 3, -2])
    assert TO.line_of(par, 4) == [0, 1, 3, 4] and TO.line_of(par, 5) == []
    assert TO.children(par, 0) == [1, 2]
    for bad in ([-1, 1], [-1, 2, 0], [-1, -2, 1], [-2, 0]):
        with pytest.raises(TO.TreeError):
            for i in range(len(bad)):
                TO.line_of(np.array(bad), i)


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotations_depend_on_the_difference(interleaved):
    rng = np.random.default_rng(1)
    q, k, f = rng.normal(size=10), rng.normal(size=10), 100.0 ** -np.arange(4)
    def turned(x, pos):
        return TO.rotate(x, np.cos(pos * f), np.sin(pos * f), interleaved)
    np.testing.assert_allclose(turned(q, 7) @ turned(k, 3), turned(q, 104) @ turned(k, 100), atol=1e-12)
    np.testing.assert_allclose(np.linalg.norm(turned(q, 9)), np.linalg.norm(q), atol=1e-12)
