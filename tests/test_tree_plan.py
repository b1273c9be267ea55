"""The tree kernel's plan as restated in _tree_plan: every tile is served once, and pieces of split segments meet
at counters that no other meeting of the launch uses."""
import random
from collections import Counter

import pytest

from _tree_plan import FLAT_PIECES, GROUP_PIECES, TILE_KEYS, deliver, form_of, meetings, plan, shared
from _tree import MEETING_BATCHES


def check(q8, group, hkv, lens, nodes, sms=152, **kw):
    pieces, dealt = plan(q8, group, hkv, lens, nodes, sms, **kw)
    form = form_of(q8, group, kw.get("bound") or max(nodes))
    tiles = Counter()
    for p in pieces:
        assert p.n > 0 and p.first <= p.cta <= p.last < form.ctas_per_sm * sms
        tiles.update((p.segment, j) for j in range(p.j0, p.j0 + p.n))
        assert (p.j0 == 0) == (p.cta == p.first)
    want = Counter((((s, g, t), j)) for s, (length, n) in enumerate(zip(lens, nodes)) for g in range(hkv)
                   for t in range(-(-n // form.tokens)) for j in range(-(-length // TILE_KEYS)))
    assert tiles == want
    # a record's place: the CTA, and whether the segment begins there
    split = [p for p in pieces if p.last > p.first]
    assert len({(p.cta, p.j0 == 0) for p in split}) == len(split)
    assert not shared(pieces)
    # as many arrivals as the kernel waits for: pieces, pieces of a group, groups
    spans = {p.segment: p.last - p.first + 1 for p in split}
    for counter, who in meetings(pieces).items():
        for (segment, first), n in who.items():
            if first != "all":
                begin = next(p.first for p in split if p.segment == segment)
                assert n == min(GROUP_PIECES, begin + spans[segment] - first)
            else:
                assert n == (spans[segment] if spans[segment] <= FLAT_PIECES else -(-spans[segment] // GROUP_PIECES))
    return pieces, dealt


def test_uneven_batches_share_no_counter():
    r = random.Random(1)
    seen = Counter()
    for _ in range(600):
        q8, group, hkv = r.random() < 0.5, r.choice([1, 2, 4]), r.choice([1, 2, 3, 4, 8])
        n = r.randint(1, 40)
        top = r.choice([2000, 20000, 60000])
        hist = [r.randint(0, top) if r.random() < 0.7 else r.randint(0, 600) for _ in range(n)]
        nodes = [r.randint(0, r.choice([4, 40, 130])) for _ in range(n)]
        if r.random() < 0.5:  # a few long contexts before many short ones
            hist = [r.randint(20000, 140000)] * r.randint(1, 3) + [r.randint(30, 1000)] * n
            nodes = [r.randint(1, 64)] * len(hist)
        if not any(nodes):
            continue
        lens = [h + k for h, k in zip(hist, nodes)]
        pieces, dealt = check(q8, group, hkv, lens, nodes, sms=r.choice([8, 31, 152]))
        seen["dealt" if dealt else "runs"] += 1
        seen["alone"] += bool(shared(pieces, place=lambda first, begins: first))
    assert seen["dealt"] > 50 and seen["runs"] > 50 and seen["alone"] > 0  # (told apart by the CTA alone some would)


@pytest.mark.parametrize("name", sorted(MEETING_BATCHES))
def test_batches_in_which_two_segments_meet_in_a_cta(name):
    """In these one segment's last group, of one piece, and the next one's first group begin in one CTA."""
    pool, hkv, hist, nodes = MEETING_BATCHES[name]
    pieces, dealt = check(pool == "q8", 4, hkv, [h + n for h, n in zip(hist, nodes)], nodes)
    assert not dealt and shared(pieces, place=lambda first, begins: first)
    # in any order of the CTAs every split segment is weighed once its pieces are there, and the counters end at
    # zero; with one counter for both groups some order loses rows
    split = {p.segment for p in pieces if p.last > p.first}
    lost = 0
    for order in range(40):
        weighed, early, left = deliver(pieces, random.Random(order))
        assert weighed == split and not early and not left
        weighed, early, left = deliver(pieces, random.Random(order), place=lambda first, begins: first)
        lost += weighed != split or bool(early) or bool(left)
    assert lost > 0
