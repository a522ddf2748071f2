"""Page tables whose requests' lengths go down between steps, and pages that requests hold ahead."""
from __future__ import annotations

import random

import pytest
import torch

import exact_bf16_top_gb300 as tk
import page_ref
from test_page_step_gpu import case, device, i32  # noqa: F401

pytestmark = pytest.mark.gpu


def step(table, lengths, new, free, count, held, q, page):
    """One step with held pages, request by request; lists in, and out: (positions, slots, valid, granted, table, free,
    lengths, count, held)."""
    table, free, held = [list(r) for r in table], list(free), list(held)
    pages, size, count = len(table[0]), len(free), min(max(count, 0), len(free))
    asked = taken = 0
    positions, slots, valid, granted, after, gone = [], [], [], [], [], []
    for r, ask in enumerate(new):
        n = min(max(lengths[r], 0), pages * page)
        own = max(-(-n // page), min(held[r], pages))
        add = min(max(ask, 0), q)
        if n + add > pages * page:
            add = 0
        need = max(0, -(-(n + add) // page) - own)
        asked += need
        if need and asked > count:
            add = need = 0
        for i in range(need):
            table[r][own + i] = free[count - 1 - taken]
            taken += 1
        if ask < 0:
            gone += table[r][:own]
        held[r] = 0 if ask < 0 else own + need
        granted.append(add)
        after.append(0 if ask < 0 else n + add)
        for j in range(q):
            at = (n + j) // page
            positions.append(n + j if j < add else 0)
            slots.append(table[r][at] * page + (n + j) % page if j < add else -1)
            valid.append(n + j + 1 if j < add else 0)
    left = count - taken
    for i, v in enumerate(gone[:max(0, size - left)]):
        free[left + i] = v
    return positions, slots, valid, granted, table, free, after, min(left + len(gone), size), held


NAMES = ("positions", "slots", "valid_len", "granted", "table", "free", "lengths", "count", "held")


def check(table, lengths, new, free, count, held, q, page, stream=None):
    tab, length, stack, top, mine = i32(table), i32(lengths), i32(free), i32([count]), i32(held)
    torch.cuda.synchronize()
    got = tk.page_step(tab, length, i32(new), stack, top, rows_per_request=q, page_size=page, held=mine, stream=stream)
    torch.cuda.synchronize()
    want = step(table, lengths, new, free, count, held, q, page)
    for name, g, w in zip(NAMES, (*got, tab, stack, length, top, mine), (*want[:7], [want[7]], want[8])):
        assert g.tolist() == w, name
    return want


@pytest.mark.parametrize("n,pages,q,page", [(1, 1, 1, 1), (1, 4, 1, 64), (2, 8, 3, 16), (7, 33, 5, 8), (33, 12, 4, 64),
                                            (512, 6, 4, 64), (513, 3, 2, 2), (3000, 3, 1, 64), (9, 20, 2048, 128),
                                            (700, 8, 30, 8)])
def test_steps_with_held_pages(n, pages, q, page):
    r = random.Random(n + q)
    for seed in range(3):
        table, lengths, new, free, count = case(n, pages, q, page, 100 * seed + n)
        full = [[p if p >= 0 else 10 ** 6 + i * pages + j for j, p in enumerate(row)] for i, row in enumerate(table)]
        own = [-(-v // page) for v in lengths]
        # What a request has by its length, some pages more, all and more than all; less than its length says counts
        # as that.
        held = [r.choice((0, -3, o, min(pages, o + 1), r.randint(o, pages), pages, pages + 5)) for o in own]
        check(full, lengths, new, free, count, held, q, page, torch.cuda.Stream() if seed == 2 else None)
        # With none held ahead it is the step without `held`.
        want = check(table, lengths, new, free, count, [0] * n, q, page)
        assert list(want[:8]) == list(page_ref.step(table, lengths, new, free, count, q, page, page))


def test_a_rejected_draft_keeps_its_page():
    # 63 tokens and four drafts take a second page; three are rejected (64 tokens, one page by length).
    table, lengths, free, count, held = i32([[5, -1, -1]]), i32([63]), i32([7, 8, 9, 0]), i32([3]), i32([0])
    got = tk.page_step(table, lengths, i32([4]), free, count, rows_per_request=4, held=held)
    assert table.tolist() == [[5, 9, -1]] and held.tolist() == [2] and got.slots.tolist() == [383, 576, 577, 578]
    lengths.fill_(64)
    got = tk.page_step(table, lengths, i32([1]), free, count, rows_per_request=4, held=held)
    assert table.tolist() == [[5, 9, -1]] and held.tolist() == [2] and count.item() == 2
    assert got.slots.tolist() == [576, -1, -1, -1] and lengths.tolist() == [65]
    # All rejected and the request finished: both pages go back.
    lengths.fill_(0)
    tk.page_step(table, lengths, i32([-1]), free, count, rows_per_request=4, held=held)
    assert held.tolist() == [0] and lengths.tolist() == [0] and count.item() == 4 and free.tolist() == [7, 8, 5, 9]


def test_many_steps_with_rejections_leave_every_page_owned_once():
    # A captured step; between replays the caller lowers lengths by what was rejected, across page borders too.
    n, pages, page, q, size = 40, 9, 16, 20, 200
    r = random.Random(5)
    table = torch.full((n, pages), -1, dtype=torch.int32, device="cuda")
    lengths, held, free, count = i32([0] * n), i32([0] * n), i32(list(range(size))), i32([size])
    new = i32([0] * n)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = tk.page_step(table, lengths, new, free, count, rows_per_request=q, page_size=page, held=held)
    state = [[[-1] * pages for _ in range(n)], [0] * n, list(range(size)), size, [0] * n]
    lowered = 0
    for _ in range(80):
        ask = [-1 if r.random() < 0.08 else r.randint(0, q) for _ in range(n)]
        new.copy_(i32(ask))
        graph.replay()
        want = step(state[0], state[1], ask, *state[2:], q, page)
        for name, g, w in zip(NAMES, (*got, table, free, lengths, count, held), (*want[:7], [want[7]], want[8])):
            assert g.tolist() == w, name
        keep = [v - r.randint(0, g) if g else v for v, g in zip(want[6], want[3])]
        lowered += sum(-(-k // page) < h for k, h in zip(keep, want[8]))
        lengths.copy_(i32(keep))
        state = [want[4], keep, want[5], want[7], want[8]]
        mine = [p for row, h in zip(state[0], state[4]) for p in row[:h]]
        assert sorted(mine + state[2][:state[3]]) == list(range(size))
    assert lowered > 100


def test_held_refusals():
    table, lengths, new, free, count = i32([[0, 1], [2, 3]]), i32([5, 6]), i32([1, 1]), i32([4, 5]), i32([2])
    for bad in (i32([1]), i32([1, 1]).long(), i32([1, 1]).cpu(), i32([1, 0, 1, 0])[::2], i32([[1, 1]]), 3):
        with pytest.raises(ValueError):
            tk.page_step(table, lengths, new, free, count, held=bad)
    assert lengths.tolist() == [5, 6] and count.item() == 2
