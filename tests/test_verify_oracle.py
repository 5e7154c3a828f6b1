"""CPU: what verification emits, over all drafts and random numbers, with several
children to a node. The probabilities are such that every acceptance threshold
is a multiple of 1 / 12, so that a midpoint grid of 12 integrates exactly."""

import itertools

import numpy as np

import oracle

P = np.array([9, 5, 1, 1]) / 16
Q = np.full(4, 1 / 4)
GRID = (np.arange(12) + 0.5) / 12


def emitted(children, weight, draft, target=P):
    """The distribution of the first token, over weight[x] for each tuple x of the children's tokens."""
    n = children + 1
    p = np.broadcast_to(target, (1, n, 4))
    q = None if draft is None else np.broadcast_to(draft, (1, n, 4))
    first = np.zeros(4)
    for x, w in weight.items():
        for u in itertools.product(GRID, repeat=children):
            for un in GRID if draft is None else GRID[:1]:  # (with draft: one token is left at the end)
                kept, path, nxt, _ = oracle.verify_tree(p, q, [[0, *x]], [[-1] + [0] * children], [n], [[0, *u]], [un])
                first[x[path[0, 1] - 1] if kept[0] == 2 else nxt[0]] += w / 12 ** children / (12 if draft is None else 1)
    return first


def test_independent_children_follow_the_target():
    """P / Q = 9/4, 5/4, 1/4, 1/4; then P - Q = (5, 1, 0, 0) / 16, against 3/8 Q: 10/3,
    2/3, 0, 0; then only token 0 is left."""
    weight = {x: Q[x[0]] * Q[x[1]] for x in itertools.product(range(4), repeat=2)}
    assert np.allclose(emitted(2, weight, Q), P, atol=1e-12)


def test_children_without_replacement_do_not():
    """Pairs of distinct tokens, as two draws without replacement give them: token
    0, the most often drafted and accepted, is not emitted as often as it should be."""
    weight = {x: 1 / 12 for x in itertools.permutations(range(4), 2)}
    assert abs(emitted(2, weight, Q) - P).max() > 0.01


def test_any_children_without_draft_probabilities():
    """Fixed distinct tokens, their probabilities struck out one by one: every
    threshold is 1/4, 1/3, 1/2 or 2/3, and then one token is left."""
    target = np.array([1, 1, 2, 0]) / 4
    for x in itertools.permutations(range(3), 2):
        assert np.allclose(emitted(2, {x: 1.0}, None, target), target, atol=1e-12)
