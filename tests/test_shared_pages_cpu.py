"""How requests that share a prefix's pages end, by the page map's definition on the host.  No GPU."""
from __future__ import annotations

import numpy as np

import hybrid_ref

P, W = 16, 2  # page size, whole pages of the prefix


def step(ctx, held, ring, free, table):
    x = hybrid_ref.page_map(np.array(ctx), np.zeros(len(ctx), int), np.array(held), ring, free, table, P, 1, len(ctx))
    return x, x["ring"], x["free_out"], x["held_out"].tolist()


def in_ring(ring, free):
    return sorted(ring[(free[0] + np.arange(free[1])) % len(ring)].tolist())


def start():
    """Two requests of one prefix in pages 0 and 1, with a page each of their own; pages 4 to 7 are free."""
    return np.array([[0, 1, 2, 9], [0, 1, 3, 9]]), np.array([4, 5, 6, 7, 0, 0, 0, 0]), np.array([0, 4])


def test_a_page_is_given_back_by_every_request_that_holds_it():
    """Why: both requests end as ones that share nothing do, and the prefix's pages come back twice."""
    table, ring, free = start()
    _, ring, free, _ = step([0, 0], [3, 3], ring, free, table)
    assert free.tolist() == [0, 10]  # of eight pages
    assert ring.tolist() == [1, 3, 6, 7, 0, 1, 2, 0]  # 0, 1, 2 of the one and 0, 1, 3 of the other, over 4 and 5


def test_the_last_request_of_a_prefix_gives_its_pages_back():
    table, ring, free = start()
    x, ring, free, held = step([W * P, W * P + 5], [3, 3], ring, free, table)
    assert held == [W, 3] and in_ring(ring, free) == [2, 4, 5, 6, 7]
    held[0] = 0
    _, ring, free, held = step([0, W * P + 5], held, ring, free, table)  # a step in between changes nothing
    assert held == [0, 3] and in_ring(ring, free) == [2, 4, 5, 6, 7]
    _, ring, free, held = step([0, 0], held, ring, free, x["table"])
    assert held == [0, 0] and in_ring(ring, free) == list(range(8))


def test_a_request_that_joins_takes_pages_behind_the_prefix_alone():
    table, ring, free = start()
    table[1, :] = 9
    table[1, :W] = table[0, :W]
    x, ring, free, held = step([40, 37], [3, W], ring, free, table)  # its prefix ends inside its third page
    assert held == [3, 3] and x["table"][1].tolist() == [0, 1, 4, 9] and in_ring(ring, free) == [5, 6, 7]


def test_a_request_that_finds_no_page_joins_later():
    table, ring, _ = start()
    table[1, :] = 9
    table[1, :W] = table[0, :W]
    x, ring, free, held = step([40, 37], [3, W], ring, np.array([0, 0]), table)
    assert x["status"] == 32 and held == [3, W] and x["table"][1].tolist() == [0, 1, 9, 9]  # no page of its own to fill
    x, ring, free, held = step([W * P, 37], held, ring, free, x["table"])  # the other ends: its page is free from the next call on
    assert x["status"] == 32 and held == [W, W] and in_ring(ring, free) == [2]
    x, ring, free, held = step([0, 37], [0, W], ring, free, x["table"])
    assert x["status"] == 0 and held == [0, 3] and x["table"][1].tolist() == [0, 1, 2, 9] and free[1] == 0
