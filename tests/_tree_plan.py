"""The tree kernel's plan, restated: which tiles every CTA of a launch serves, the pieces of split segments,
and the counters at which these meet.  (The kernel's own is in csrc/tree.cu; the numbers are its constants.)"""
from __future__ import annotations

from collections import defaultdict
from typing import NamedTuple

TILE_KEYS, TILE_ROWS, BLOCK = 128, 128, 16
MIN_PIECE, FLAT_PIECES, GROUP_PIECES, DEALT_SEQS = 6, 10, 8, 1024


class Form(NamedTuple):
    """One instance of the kernel: rows of a segment, CTAs per SM, and what a piece and a meeting cost in tiles."""
    tokens: int
    ctas_per_sm: int
    piece_tiles: int
    split_tiles: int


def form_of(q8, group, max_query_len):
    halves = 2 if max_query_len * group > (TILE_ROWS // 2 if q8 else TILE_ROWS) else 1
    return Form(halves * TILE_ROWS // group, 2 if halves == 1 else 1, 3 if q8 else 4, 3 if q8 else 8)


class Piece(NamedTuple):
    cta: int
    segment: tuple  # sequence, K/V head, query tile
    j0: int         # its first tile, and how many
    n: int
    first: int      # CTAs that the segment is split over
    last: int


def plan(q8, group, hkv, lens, nodes, sms=152, width=None, bound=None):
    """Pieces in the order in which each CTA serves them, and whether CTAs were dealt to segments."""
    bound = bound or max(nodes)
    form = form_of(q8, group, bound)
    cost = form.piece_tiles
    width = width or max(-(-l // BLOCK) for l in lens)
    most = form.ctas_per_sm * sms
    ctas = min(most, len(lens) * hkv * -(-bound // form.tokens) * -(-width * BLOCK // TILE_KEYS))
    segments = [((s, g, t), -(-l // TILE_KEYS)) for s, (l, n) in enumerate(zip(lens, nodes))
                for g in range(hkv) for t in range(-(-n // form.tokens))]
    total = sum(tiles + cost for _, tiles in segments)
    pieces = []
    if len(segments) <= ctas and len(lens) <= DEALT_SEQS and total:
        low = max(-(-(total - cost * len(segments)) // ctas), MIN_PIECE)
        for t in range(low, low + form.split_tiles + 1):
            if sum(-(-tiles // t) for _, tiles in segments) <= ctas:
                cta = 0
                for seg, tiles in segments:
                    k = -(-tiles // t)
                    for i in range(k):
                        j0, j1 = tiles * i // k, tiles * (i + 1) // k
                        pieces.append(Piece(cta + i, seg, j0, j1 - j0, cta, cta + k - 1))
                    cta += k
                return pieces, True
    runs = min(ctas, max(total, 1))
    edge = [total * r // runs for r in range(runs + 1)]
    run_of = lambda at: ((at + 1) * runs + total - 1) // total - 1
    at = 0
    for seg, tiles in segments:
        first, last = run_of(at + cost), run_of(at + cost + tiles - 1)
        for cta in range(first, last + 1):
            j0 = max(edge[cta] - at - cost, 0)
            pieces.append(Piece(cta, seg, j0, min(edge[cta + 1] - at - cost, tiles) - j0, first, last))
        at += tiles + cost
    return pieces, False


def meetings(pieces, place=lambda first, begins: (first, begins)):
    """Every counter's users: {counter: {(segment, what meets there): arrivals}}.  Groups of a segment are
    counted by the CTA of their first piece and by whether the segment begins there."""
    users = defaultdict(lambda: defaultdict(int))
    for p in pieces:
        n = p.last - p.first + 1
        if n == 1:
            continue
        if n <= FLAT_PIECES:
            users["segments", p.first][p.segment, "all"] += 1
            continue
        first = p.first + (p.cta - p.first) // GROUP_PIECES * GROUP_PIECES
        users["groups", place(first, first == p.first)][p.segment, first] += 1
        if p.cta == first:
            users["segments", p.first][p.segment, "all"] += 1
    return users


def shared(pieces, **kw):
    """Counters that more than one meeting would use."""
    return [c for c, who in meetings(pieces, **kw).items() if len(who) > 1]


def deliver(pieces, rng, place=lambda first, begins: (first, begins)):
    """The meetings of a launch whose CTAs advance in an order of rng's: segments that were weighed with every piece
    delivered, ones weighed too early, and the counters that did not come back to zero."""
    queues = defaultdict(list)
    for p in pieces:
        if p.last > p.first:
            queues[p.cta].append(p)
    spans = defaultdict(set)
    for p in pieces:
        spans[p.segment].add(p.cta)
    counters, there, weighed, early = defaultdict(int), defaultdict(set), set(), set()

    def arrive(counter, count):
        counters[counter] += 1
        if counters[counter] != count:
            return False
        counters[counter] = 0
        return True

    waiting = [c for c in queues]
    while waiting:
        cta = rng.choice(waiting)
        p = queues[cta].pop(0)
        if not queues[cta]:
            waiting.remove(cta)
        there[p.segment].add(cta)
        n = p.last - p.first + 1
        done = False
        if n <= FLAT_PIECES:
            done = arrive(("segments", p.first), n)
        else:
            first = p.first + (cta - p.first) // GROUP_PIECES * GROUP_PIECES
            members = set(range(first, min(first + GROUP_PIECES, p.last + 1)))
            if arrive(("groups", place(first, first == p.first)), len(members)):
                if not members <= there[p.segment]:
                    early.add(p.segment)
                done = arrive(("segments", p.first), -(-n // GROUP_PIECES))
        if done:
            (weighed if there[p.segment] == spans[p.segment] else early).add(p.segment)
    return weighed, early, [c for c, n in counters.items() if n]
