"""Page tables taken one step further on the GPU, against the definition."""
from __future__ import annotations

import random

import pytest
import torch

import exact_bf16_top_gb300 as tk
import page_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tk.load()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def case(n, pages, q, page, seed, spare=20, done=0.1, idle=0.1):
    """A batch whose requests own distinct pages, and a stack of the others."""
    r = random.Random(seed)
    width = pages * page
    lengths = [0 if r.random() < 0.1 else r.randint(0, width) for _ in range(n)]
    order = list(range(n * pages + spare))
    r.shuffle(order)
    table, at = [], 0
    for length in lengths:
        own = -(-length // page)
        table.append(order[at:at + own] + [-7] * (pages - own))
        at += own
    left = order[at:]
    count = min(len(left), max(0, r.randint(0, 2 * n * max(1, q // page))))
    free = left[:count] + [-9] * (len(order) - count)
    new = [-1 if r.random() < done else 0 if r.random() < idle else r.randint(1, q + 2) for _ in range(n)]
    return table, lengths, new, free, count


def check(table, lengths, new, free, count, q, page, block_rows=None, in_place=True, wide=0):
    n, pages = len(table), len(table[0]) if table else 4
    rows = block_rows or page
    tab = torch.full((n, pages + wide), 2 ** 30, dtype=torch.int32, device="cuda")[:, :pages]
    if n and pages:
        tab.copy_(i32(table))
    length, free_t, count_t = i32(lengths), i32(free), i32([count])
    kw = {} if in_place else dict(next_lengths=torch.full_like(length, -5), next_free_count=torch.full_like(count_t, -5))
    got = tk.page_step(tab, length, i32(new), free_t, count_t, rows_per_request=q, page_size=page,
                       block_rows=block_rows, **kw)
    want = page_ref.step(table, lengths, new, free, count, q, page, rows)
    after, left = (length, count_t) if in_place else (kw["next_lengths"], kw["next_free_count"])
    for name, g, w in zip(("positions", "slots", "valid_len", "granted", "table", "free", "lengths", "count"),
                          (*got, tab, free_t, after, left), (*want[:-1], [want[-1]])):
        assert g.tolist() == w, name
    if not in_place:
        assert length.tolist() == lengths and count_t.item() == count
    return got, tab, free_t, after, left


@pytest.mark.parametrize("n,pages,q,page", [
    (1, 1, 1, 1), (1, 4, 1, 64), (1, 40, 300, 64), (2, 8, 3, 16), (7, 33, 5, 8), (31, 5, 1, 64), (33, 12, 4, 64),
    (512, 6, 4, 64), (513, 3, 2, 2), (1025, 4, 3, 4), (3000, 3, 1, 64), (5, 64, 1000, 16), (2, 300, 4097, 64),
    (9, 20, 2048, 128), (700, 8, 30, 8)])
@pytest.mark.parametrize("in_place", [True, False])
def test_steps(n, pages, q, page, in_place):
    for seed in range(3):
        check(*case(n, pages, q, page, 100 * seed + n + q), q, page, in_place=in_place, wide=seed)


def test_the_most_requests():
    check(*case(32768, 2, 1, 4, 5), 1, 4)


def test_lengths_at_pages_borders():
    page, pages = 64, 4
    lengths = [0, 1, 63, 64, 65, 127, 128, 191, 192, 255, 256]
    n = len(lengths)
    for q in (1, 2, 64, 65, 129, 256):
        order = list(range(n * pages + 50))
        table = [order[r * pages:(r + 1) * pages] for r in range(n)]
        free = order[n * pages:]
        for new in ([q] * n, [1] * n, [0] * n, [-1] * n):
            check(table, lengths, new, free, len(free), q, page)


def test_too_few_pages_are_given_in_order_of_the_requests():
    # Request 1 asks for more than is left; 2 needs none and is served; 3 could be, but comes after what was asked for.
    table = [[0, -1, -1, -1], [1, -1, -1, -1], [2, -1, -1, -1], [3, -1, -1, -1]]
    got, *_ = check(table, [64, 64, 10, 64], [1, 150, 5, 1], [9, 8, 7], 3, 150, 64)
    assert got.granted.tolist() == [1, 0, 5, 0]
    # None at all, an empty pool, a count past the pool or below zero.
    check(table, [64, 64, 10, 64], [1, 1, 5, 1], [9, 8, 7], 0, 5, 64)
    check(table, [64, 64, 10, 64], [1, 1, 5, 1], [], 0, 5, 64)
    check(table, [64, 64, 10, 64], [1, 1, 5, 1], [9, 8, 7], 77, 5, 64)
    check(table, [64, 64, 10, 64], [1, 1, 5, 1], [9, 8, 7], -4, 5, 64)


def test_what_does_not_fit_the_table_is_refused():
    got, *_ = check([[0, 1], [2, 3], [4, 5]], [127, 127, 128], [1, 2, 1], [9, 8, 7], 3, 4, 64)
    assert got.granted.tolist() == [1, 0, 0]


def test_lengths_and_pages_out_of_range():
    check([[0, 1], [2, 3], [4, 5]], [-5, 10 ** 9, 2 ** 31 - 1], [1, 1, -1], [9, 8, 7, 6], 2, 4, 64)
    # Slots past 31 bits, and of a negative page, are none; the table keeps what the stack holds.
    got, *_ = check([[0, -1], [2 ** 26, -1], [-3, -1]], [64, 3, 3], [1, 1, 1], [2 ** 31 - 1, -8], 2, 1, 64)
    assert got.slots.tolist() == [-1, -1, -1]
    check([[5, -1], [2 ** 20 - 1, -1]], [3, 3], [1, 2], [1, 2], 2, 2, 64, block_rows=2048)


def test_pages_that_come_back_past_the_pool_are_dropped():
    got, _, free, _, count = check([[0, 1], [2, 3]], [128, 128], [-1, -1], [9, 8, 7], 2, 1, 64)
    assert free.tolist() == [9, 8, 0] and count.item() == 3


def test_no_requests_and_no_pages():
    empty = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    none = i32([])
    count = i32([3])
    got = tk.page_step(empty, none, none, i32([1, 2, 3]), count)
    assert all(t.numel() == 0 for t in got) and count.item() == 3
    table = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    got = tk.page_step(table, i32([0, 0]), i32([1, -1]), none, i32([0]))
    assert got.granted.tolist() == [0, 0] and got.slots.tolist() == [-1, -1]


def test_many_steps_leave_every_page_owned_once():
    n, pages, page, q = 40, 9, 16, 7
    r = random.Random(3)
    size = 200
    table = torch.full((n, pages), -1, dtype=torch.int32, device="cuda")
    lengths, free, count = i32([0] * n), i32(list(range(size))), i32([size])
    graph_new = i32([0] * n)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = tk.page_step(table, lengths, graph_new, free, count, rows_per_request=q, page_size=page)
    mine = ([[-1] * pages for _ in range(n)], [0] * n, list(range(size)), size)
    for _ in range(60):
        new = [-1 if r.random() < 0.08 else r.randint(0, q) for _ in range(n)]
        graph_new.copy_(i32(new))
        graph.replay()
        want = page_ref.step(mine[0], mine[1], new, mine[2], mine[3], q, page, page)
        for g, w in zip((*got, table, free, lengths, count), (*want[:-1], [want[-1]])):
            assert g.tolist() == w
        mine = (want[4], want[6], want[5], want[7])
        held = [p for row, n_ in zip(mine[0], mine[1]) for p in row[:-(-n_ // page)]]
        assert sorted(held + mine[2][:mine[3]]) == list(range(size))


def test_about_as_many_rows_as_31_bits_count():
    q = (2 ** 31 - 1) // 3
    table, lengths, free, count = i32([[7, -1]] * 3), i32([1, 0, 64]), i32([5, 6]), i32([2])
    got = tk.page_step(table, lengths, i32([2, 0, 1]), free, count, rows_per_request=q)
    assert got.positions.numel() == 3 * q and got.granted.tolist() == [2, 0, 1]
    for rows, want, pad in zip(got[:3], ((1, 2, 64), (449, 450, 6 * 64), (2, 3, 65)), (0, -1, 0)):
        assert (*rows[:2].tolist(), rows[2 * q].item()) == want
        assert rows[2:2 * q].min().item() == rows[2:2 * q].max().item() == pad
        assert rows[2 * q + 1:].min().item() == rows[2 * q + 1:].max().item() == pad
    assert table.tolist() == [[7, -1], [7, -1], [7, 6]] and lengths.tolist() == [3, 0, 65] and count.item() == 1


def test_on_another_stream():
    a = case(64, 8, 4, 16, 9)
    table, lengths, new, free, count = a
    side = torch.cuda.Stream()
    args = i32(table), i32(lengths), i32(new), i32(free), i32([count])
    side.wait_stream(torch.cuda.current_stream())
    got = tk.page_step(*args, rows_per_request=4, page_size=16, stream=side)
    torch.cuda.synchronize()
    want = page_ref.step(table, lengths, new, free, count, 4, 16, 16)
    assert [t.tolist() for t in got] == list(want[:4])


def test_refusals():
    table, lengths, new, free, count = i32([[0, 1], [2, 3]]), i32([5, 6]), i32([1, 1]), i32([4, 5]), i32([2])

    def call(t=table, l=lengths, w=new, f=free, c=count, **kw):
        return tk.page_step(t, l, w, f, c, **kw)

    for bad in (lambda: call(table.long()), lambda: call(table.cpu()), lambda: call(l=lengths.float()),
                lambda: call(f=free.cpu()), lambda: call(c=3), lambda: call(w=None)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: call(table.T.contiguous().T), lambda: call(l=lengths[:1]), lambda: call(w=new[:1]),
                lambda: call(c=i32([1, 2])), lambda: call(c=count[0]), lambda: call(page_size=48),
                lambda: call(page_size=0), lambda: call(rows_per_request=0), lambda: call(page_size=2 ** 30),
                lambda: call(rows_per_request=2 ** 31), lambda: call(block_rows=2 ** 31),
                lambda: call(next_lengths=i32([1])), lambda: call(next_free_count=i32([1, 2])),
                lambda: call(next_lengths=lengths.long()), lambda: call(table[:1].expand(2, 2)),
                lambda: call(l=i32([5, 0, 6, 0])[::2])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(tk.TopkError):
        call(block_rows=32)
    assert table.tolist() == [[0, 1], [2, 3]] and lengths.tolist() == [5, 6] and count.item() == 2
