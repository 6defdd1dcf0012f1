"""The turn of a serving loop around the layers, in plain Python and float64 numpy: the plan
of a batch on the paged cache, and the choice of a token from a row of logits.

Plain readings of the rules, one sequence, page and token at a time.
"""

from __future__ import annotations

import math

import numpy as np


def plan(lens, new, table, page: int, tokens: int, pages: int, free=None, count: int = 0, starts=None, reset=None):
    """(q_offsets, positions, slots, lens, table, free, count, lacking) after a step. free None:
    the table holds all pages. The arguments are left as they were."""
    blocks = table.shape[1]
    lens = [min(max(int(n), 0), blocks * page) for n in lens]
    new = [1] * len(lens) if new is None else [max(int(n), 0) for n in new]
    table = table.copy()
    stack = None if free is None else [int(p) for p in free[:min(max(count, 0), pages)]]
    memory = None if free is None else free.copy()
    for s in range(len(lens)):
        if reset is not None and reset[s]:
            for b in range(-(-lens[s] // page)):
                if stack is not None and len(stack) < pages:
                    memory[len(stack)] = table[s, b]
                    stack.append(int(table[s, b]))
            lens[s] = 0
    offsets, positions, slots, lacking = [0], [], [], 0
    for s in range(len(lens)):
        rows = min(new[s], tokens - offsets[-1])
        offsets.append(offsets[-1] + rows)
        start, stored = 0 if starts is None else int(starts[s]), lens[s]
        ended = False  # a page was not there: the tokens behind are not stored
        for t in range(lens[s], lens[s] + rows):
            b = t // page
            if t % page == 0 and b >= -(-lens[s] // page):
                if b >= blocks or (stack is not None and not stack):
                    lacking += 1
                    ended = True
                elif stack is not None:
                    table[s, b] = stack.pop()
            number = -1 if ended else int(table[s, b])
            positions.append(start + t)
            slots.append(number * page + t % page if 0 <= number < pages else -1)
            stored += not ended
        lens[s] = stored
    behind = tokens - offsets[-1]
    return (np.array(offsets), np.array(positions + [0] * behind), np.array(slots + [-1] * behind), np.array(lens), table,
            memory, None if stack is None else len(stack), lacking)


def sample(logits, u: float, temperature: float = 1.0, top_k: int = 0, top_p: float = 1.0, min_p: float = 0.0):
    """(token, its share of what the cuts left) of one row of logits (float64)."""
    x = np.where(np.isnan(logits), -np.inf, np.asarray(logits, dtype=np.float64))
    m = x.max()
    if m == -np.inf:
        return -1, 0.0
    greedy = not temperature > 0
    w = np.zeros(len(x))
    for i in np.flatnonzero(x > -np.inf):
        d = 0.0 if x[i] == m else x[i] - m
        w[i] = 1.0 if d == 0.0 else 0.0 if greedy or d == -np.inf else math.exp(d / temperature)
    rank = np.argsort(-x, kind="stable")                  # by logit, equal ones by index
    if greedy:
        rank = rank[:1]
    elif 0 < top_k < len(x):
        rank = rank[:top_k]
    if top_p < 1:
        sums = np.cumsum(w[rank])
        target = top_p * sums[-1]
        rank = rank[:1 + next((i for i, t in enumerate(sums) if t >= target), len(rank) - 1)]
    if min_p > 0:
        rank = [i for i in rank if w[i] >= min(min_p, 1.0)]
    kept = np.sort(np.asarray(rank))
    kept = kept[w[kept] > 0]
    sums = np.cumsum(w[kept])
    draw = u * sums[-1] if u > 0 else 0.0
    at = next((i for i, t in enumerate(sums) if t > draw), len(kept) - 1)
    return int(kept[at]), float(w[kept[at]] / sums[-1])
