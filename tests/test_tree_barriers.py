"""The barrier that opens an item of the tree attention's kernel, in every order of its agents.

A waiting thread names a phase of an mbarrier by its parity, so a phase must not complete
before everyone that waits for the one before has seen it.  The model: the softmax warps put
an item's q in place and arrive, then work on the item's tiles, which needs the issuers that
have one (an issuer takes every second tile; of one tile only the first).  An issuer waits for
every item's q.  How many arrivals a phase takes, and so whether the issuers' are among them,
is read from the source.
"""
import itertools
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "fp8_quantised_paged_gb300", "csrc", "tree.cuh")
SOFTMAX = 8  # warps, which stay together: they join at the end of an item


def arrivals():
    text = open(SOURCE).read()
    count = re.search(r"int tree_bar_count\(int i\) \{\s*return i < kTP\s*\?\s*([0-9]+)", text)
    return int(count.group(1)), text.count("mbar_arrive(bars + kTQ)")


def lapped(items, count):
    """Over every order of the agents through these items (tiles of each): the states in which
    an issuer waits for a phase that is over and another behind it too, and the ones in which
    someone waits for ever."""
    joins = count > SOFTMAX
    # softmax: (item, arrived); each issuer: the same; phases that are over; arrivals
    first = ((0, False), ((0, False), (0, False)), 0, 0)
    seen, todo, bad, stuck = {first}, [first], [], []

    def arrive(done, held, n):
        held += n
        return (done + 1, 0) if held == count else (done, held)

    while todo:
        state = todo.pop()
        (si, sa), issuers, done, held = state
        nexts = []
        if si < len(items) and not sa:
            nexts.append(((si, True), issuers, *arrive(done, held, SOFTMAX)))
        elif si < len(items):
            # an item is over once the issuers that have a tile of it have been through it
            if all(issuers[t][0] > si for t in range(min(items[si], 2))):
                nexts.append(((si + 1, False), issuers, done, held))
        for t, (it, arrived) in enumerate(issuers):
            if it == len(items):
                continue

            def moved(x):
                return tuple(x if k == t else issuers[k] for k in range(2))

            if joins and not arrived:
                nexts.append(((si, sa), moved((it, True)), *arrive(done, held, 1)))
                continue
            if done > it + 1:
                bad.append((items, state))
            if done % 2 != it % 2:  # the last phase that is over has the item's parity
                nexts.append(((si, sa), moved((it + 1, False)), done, held))
        if not nexts and (si, issuers[0][0], issuers[1][0]) != (len(items),) * 3:
            stuck.append((items, state))
        for n in nexts:
            if n not in seen:
                seen.add(n)
                todo.append(n)
    return bad, stuck


ITEMS = [x for n in (1, 2, 3, 4) for x in itertools.product((1, 2, 3), repeat=n)]


def test_no_issuer_is_lapped():
    count, places = arrivals()
    assert count in (SOFTMAX, SOFTMAX + 2)
    assert places == (2 if count > SOFTMAX else 1)
    for items in ITEMS:
        bad, stuck = lapped(items, count)
        assert not bad, bad[0]
        assert not stuck, stuck[0]


@pytest.mark.parametrize("items", [(1, 1), (1, 2), (3, 1, 1)])
def test_the_model_sees_an_issuer_without_a_tile_lapped(items):
    """Without the issuers' arrivals nothing holds the next item's phase back."""
    assert lapped(items, SOFTMAX)[0]
