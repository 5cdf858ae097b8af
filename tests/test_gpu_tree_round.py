"""The tree operators together (examples/tree_round.py): prefill, tree passes, verification, commit
and realignment of a small decoder, against the same decoder run plainly in float64.

Greedy tree speculation commits exactly what plain greedy decoding commits.  The cache holds the
K/V of every committed token but the pending one: fp32 through two layers of sums of at most 256
terms, each good to 2^-24 relative; 1e-4 of the largest value is far above what that leaves.
"""
import os
import sys

import numpy as np
import pytest
import torch

import oracle.specdec_oracle as O

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def prompts_of(lengths, seed=3):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randint(0, 256, (n,), generator=gen).tolist() for n in lengths]


def as64(model):
    other = object.__new__(type(model))
    other.__dict__.update(model.__dict__)
    other.embed, other.head = model.embed.double(), model.head.double()
    other.layers = [{k: w.double() for k, w in lay.items()} for lay in model.layers]
    return other


def check_cache(rows, batch, model, table):
    n, W = batch.n_committed.cpu().numpy(), int(batch.width)
    assert n.tolist() == [len(r) for r in rows] and W == max(n)
    assert O.check_invariants(batch.mask[batch.cur].cpu().numpy(), batch.pos[batch.cur].cpu().numpy(), n, W) == []
    for b, r in enumerate(rows):
        assert batch.ids[batch.cur][b, W - len(r):W].tolist() == r
        want = as64(model).plain(r[:-1], table.double())[1]
        got = batch.cache[:, :, b, :, W - len(r):W - 1].double()
        assert (got - want).abs().max() <= 1e-4 * want.abs().max()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lengths,widths", [((5, 41, 18), (3, 2, 1)), ((2, 70), (3, 3, 2, 1)), ((9,), (1, 1, 1))])
def test_greedy_rounds_commit_plain_greedy_decoding(in_place, lengths, widths):
    import tree_round
    prompts = prompts_of(lengths)
    rows, accepted, batch, model, table = tree_round.generate(prompts, rounds=5, widths=widths, in_place=in_place)
    check_cache(rows, batch, model, table)
    ref = as64(model)
    for p, r in zip(prompts, rows):
        plain = list(p)
        while len(plain) < len(r):
            plain.append(int(ref.plain(plain, table.double())[0][-1].argmax()))
        assert plain == r
    assert np.sum(accepted) > 0            # the trees were of use


@pytest.mark.parametrize("in_place", [False, True])
def test_sampled_rounds_keep_the_invariants(in_place):
    import tree_round
    rows, accepted, batch, model, table = tree_round.generate(prompts_of((3, 33, 12, 50)), rounds=6, temperature=0.8, in_place=in_place)
    check_cache(rows, batch, model, table)
    assert np.sum(accepted) > 0


def test_rotary_tables():
    from speculative_decoding_specdec_gb300.engine import rotary_table
    plain = rotary_table(50, 16)
    i = np.arange(8)
    want = np.arange(50)[:, None] * 10000.0 ** (-i / 8)
    np.testing.assert_allclose(plain[..., 0].cpu(), np.cos(want), atol=1e-7)
    np.testing.assert_allclose(plain[..., 1].cpu(), np.sin(want), atol=1e-7)
    linear = rotary_table(50, 16, scaling="linear", factor=4.0)
    torch.testing.assert_close(linear[4 * np.arange(12)], plain[:12], atol=1e-6, rtol=0)
    low = rotary_table(50, 16, scaling="base", factor=4.0)
    torch.testing.assert_close(low[:, 0], plain[:, 0])                       # the highest frequency stays
    torch.testing.assert_close(low[4 * np.arange(12), -1], plain[:12, -1], atol=1e-6, rtol=0)
    bands = rotary_table(50, 16, scaling="bands", factor=4.0, original=4096)
    amp = 0.1 * np.log(4.0) + 1
    torch.testing.assert_close(bands[:, 0], plain[:, 0] * amp)
    torch.testing.assert_close(bands[:, -1], linear[:, -1] * amp)
    for bad in (dict(rot_dim=3), dict(rot_dim=0), dict(factor=0.0), dict(scaling="other"), dict(scaling="bands")):
        with pytest.raises(ValueError):
            rotary_table(**({"positions": 4, "rot_dim": 8} | bad))
