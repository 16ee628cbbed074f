"""The indices of a step (nf4_plan_step) against a host program that handles one sequence after the other (GPU).
Everything is whole numbers: results are equal or wrong."""
from collections import deque

import numpy as np
import pytest
import torch

import nf4_weight_only_gb300 as nf4

from gpu_util import DEV, Guarded

pytestmark = pytest.mark.gpu


def host_plan(lengths, new, page, table, ring, first, count, t):
    """(table, ring, lengths, starts, slots, positions, sequences, first, count) as lists."""
    table, ring, pages, wide = [list(r) for r in table], list(ring), len(ring), len(table[0]) if len(table) else 0
    stock = deque(ring[(first + i) % pages] for i in range(count))
    end, back = first + count, 0
    lengths = [max(0, n) for n in lengths]
    for b, n in enumerate(new):
        if n < 0:
            for p in range(-(-lengths[b] // page)):
                stock.append(table[b][p])
                ring[(end + back) % pages] = table[b][p]
                back += 1
    out, starts, slots, positions, sequences = [], [0], [-1] * t, [0] * t, [-1] * t
    taken, empty = 0, False
    for b, n in enumerate(new):
        if n < 0:
            out.append(0)
            starts.append(starts[-1])
            continue
        held, want = -(-lengths[b] // page), -(-(lengths[b] + n) // page)
        ok = want <= wide and starts[-1] + n <= t
        if ok and want > held:
            empty = empty or want - held > len(stock)
            ok = not empty
            for p in range(held, want if ok else held):
                table[b][p] = stock.popleft()
                taken += 1
        for i in range(min(n, t - starts[-1])):
            row, pos = starts[-1] + i, lengths[b] + i
            sequences[row], positions[row] = b, pos
            if ok:
                slots[row] = table[b][pos // page] * page + pos % page
        out.append(lengths[b] + n if ok else lengths[b])
        starts.append(starts[-1] + n)
    return table, ring, out, starts, slots, positions, sequences, (first + taken) % max(1, pages), count + back - taken


class State:
    """Tensors of a call; every output in a guarded buffer."""

    def __init__(self, lengths, new, page, table, ring, first, count, t, in_place=False):
        b = len(lengths)
        self.page, self.t = page, t

        def filled(values, shape, dtype):
            g = Guarded(shape, dtype)
            if len(values):
                g.t.copy_(torch.tensor(np.asarray(values).reshape(shape), dtype=dtype))
            return g

        i32, i64 = torch.int32, torch.int64
        self.lengths, self.new = filled(lengths, (b,), i32), filled(new, (b,), i32)
        self.table = filled(table, (b, len(table[0]) if b else 3), i32)
        self.ring, self.state = filled(ring, (len(ring),), i32), filled([first, count], (2,), i64)
        self.lengths_out = self.lengths if in_place else Guarded((b,), i32)
        self.state_out = self.state if in_place else Guarded((2,), i64)
        self.starts, self.slots = Guarded((b + 1,), i32), Guarded((t,), i64)
        self.positions, self.sequences = Guarded((t,), i32), Guarded((t,), i32)
        self.want = host_plan(lengths, new, page, table, ring, first, count, t)

    def run(self, stream=None):
        nf4.nf4_plan_step(self.lengths.t, self.new.t, self.page, self.table.t, self.ring.t, self.state.t, self.state_out.t,
                          self.lengths_out.t, self.starts.t, self.slots.t, self.positions.t, self.sequences.t, stream=stream)

    def check(self):
        table, ring, lengths, starts, slots, positions, sequences, first, count = self.want
        for name, got, want in (("table", self.table, table), ("ring", self.ring, ring), ("lengths", self.lengths_out, lengths),
                                ("starts", self.starts, starts), ("slots", self.slots, slots),
                                ("positions", self.positions, positions), ("sequences", self.sequences, sequences),
                                ("state", self.state_out, [first, count])):
            assert got.t.flatten().tolist() == list(np.asarray(want, dtype=np.int64).flatten()), name
            assert got.canaries_intact(), name


def make(rng, b, page, wide, t, finished=0.0, idle=0.0, long=0.0, count=None, spare=50, in_place=False):
    lengths = rng.integers(0, wide * page + 1, b)
    lengths[rng.random(b) < 0.3] = page * rng.integers(0, wide + 1)
    new = np.where(rng.random(b) < long, rng.integers(1, 3 * page, b), 1)
    new[rng.random(b) < idle] = 0
    new[rng.random(b) < finished] = -rng.integers(1, 9)
    held = -(-lengths // page)
    pages = int(held.sum()) + spare
    order = rng.permutation(pages)
    table = np.full((b, wide), -7)
    table[np.arange(wide)[None] < held[:, None]] = order[:held.sum()]
    count, first = spare if count is None else count, int(rng.integers(0, max(1, pages)))
    ring = np.full(pages, -9)
    ring[(first + np.arange(count)) % max(1, pages)] = order[held.sum():held.sum() + count]
    return State(lengths.tolist(), new.tolist(), page, table.tolist(), ring.tolist(), first, count, t, in_place)


@pytest.mark.parametrize("b,page,wide,t", [
    (1, 16, 4, 1), (1, 16, 4, 0), (2, 48, 1, 5), (7, 16, 9, 7), (8, 64, 33, 40), (255, 16, 5, 300), (256, 32, 4, 256),
    (257, 16, 3, 513), (600, 80, 3, 2049), (1024, 16, 2, 1024), (1025, 16, 2, 4100), (3000, 16, 2, 9000),
    (8192, 16, 2, 8192), (31, 65536, 2, 31), (5, 16, 700, 17000),
])
@pytest.mark.parametrize("kind", ["decode", "mixed", "short", "in place"])
def test_against_one_sequence_after_the_other(b, page, wide, t, kind):
    rng = np.random.default_rng(b * 7 + t + len(kind))
    more = {} if kind == "decode" else dict(finished=0.2, idle=0.2, long=0.3)
    s = make(rng, b, page, wide, t, spare=b + 3 * b, count=b // 3 if kind == "short" else None,
             in_place=kind == "in place", **more)
    s.run()
    s.check()
    assert nf4.nf4_check_device_error() == 0


def test_empty_batch_and_empty_pool():
    s = State([], [], 16, [], [4, 5], 1, 1, 6)
    s.run()
    s.check()
    s = State([0, 0], [1, 0], 16, [[9], [9]], [], 0, 0, 3)
    s.run()
    s.check()
    assert s.lengths_out.t.tolist() == [0, 0] and s.slots.t.tolist() == [-1, -1, -1]


def test_what_is_given_back_serves_the_same_step():
    # two pages come back; the first sequence takes the ring's one page and one of them, the last takes the other
    s = State([32, 20, 0, 16], [17, -1, -3, 1], 16, [[5, 6, -1, -1], [7, 8, -1, -1], [-1] * 4, [2, -1, -1, -1]],
              [0, 0, 0, 4, 0, 0, 0, 0, 0], 3, 1, 18)
    s.run()
    s.check()
    assert s.table.t.tolist() == [[5, 6, 4, 7], [7, 8, -1, -1], [-1] * 4, [2, 8, -1, -1]]
    assert s.state_out.t.tolist() == [6, 0] and s.lengths_out.t.tolist() == [49, 0, 0, 17]


def test_refusals_keep_their_lengths():
    # no room in the table, no rows left, no pages left; those that need no page go on
    s = State([32, 3, 16, 15, 15, 5], [1, 2, 1, 1, 1, 40], 16,
              [[0, 1], [2, -1], [3, -1], [4, -1], [5, -1], [6, -1]], list(range(7)), 0, 0, 8)
    s.run()
    s.check()
    assert s.lengths_out.t.tolist() == [32, 5, 16, 16, 16, 5]
    assert s.slots.t.tolist() == [-1, 35, 36, -1, 79, 95, -1, -1]


def test_negative_lengths_count_as_none():
    s = State([-5, 7], [3, 1], 16, [[-1, -1], [1, -1]], [0, 9, 9], 0, 1, 4)
    s.run()
    s.check()
    assert s.lengths_out.t.tolist() == [3, 8]


@pytest.mark.parametrize("what", ["page", "first", "count", "overfull"])
def test_states_outside_the_pool_are_reported(what):
    assert nf4.nf4_check_device_error() == 0
    s = State([5, 20], [1, -1], 16, [[3, -1], [1, 2]], [0, 0, 0, 0, 0], 0, 0, 2)
    if what == "page":
        s.table.t[0, 0] = 77
    elif what == "first":
        s.state.t[0] = 1 << 40
    elif what == "count":
        s.state.t[1] = -3
    else:
        s.state.t[1] = 4  # two pages come back, room for one
    s.run()
    assert nf4.nf4_check_device_error() == 45
    if what == "page":
        assert s.slots.t.tolist() == [-1, -1]
    else:
        assert s.slots.t.tolist() == [53, -1] and s.lengths_out.t.tolist() == [6, 0]
    assert 0 <= int(s.state_out.t[0]) < 5 and 0 <= int(s.state_out.t[1]) <= 5
    assert s.table.canaries_intact() and s.ring.canaries_intact() and nf4.nf4_check_device_error() == 0


def test_totals_past_32_bits_refuse_what_does_not_fit():
    """Three sequences of 2^30 new tokens and one of two: the first three pass the rows, and so does the last."""
    big = 1 << 30
    for ring, slots, code in (([3, 4], [-1, -1], 45),  # pages that a pool of two does not have
                              ([1, 0], [65536, 65537], 0)):
        s = State([0, 0, 0, 0], [2, big, big, big], 65536, [[0, -1]] * 4, ring, 0, 2, 10)
        s.run()
        assert s.starts.t.tolist() == [0, 2, big + 2, (1 << 31) - 1, (1 << 31) - 1]
        assert s.lengths_out.t.tolist() == [2, 0, 0, 0] and s.sequences.t.tolist() == [0, 0] + [1] * 8
        assert s.slots.t.tolist() == slots + [-1] * 8 and nf4.nf4_check_device_error() == code


def test_replayed_steps_of_a_server():
    """Sixty replays of one captured call in place, requests coming and going between them."""
    rng = np.random.default_rng(8)
    b, page, wide, pages, t = 24, 16, 6, 60, 96
    ring, state = nf4.free_ring(pages)
    lengths = torch.zeros(b, dtype=torch.int32, device=DEV)
    new, table = torch.zeros_like(lengths), torch.zeros((b, wide), dtype=torch.int32, device=DEV)
    starts = torch.zeros(b + 1, dtype=torch.int32, device=DEV)
    slots = torch.zeros(t, dtype=torch.int64, device=DEV)
    positions, sequences = (torch.zeros(t, dtype=torch.int32, device=DEV) for _ in range(2))
    args = (lengths, new, page, table, ring, state, state, lengths, starts, slots, positions, sequences)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nf4.nf4_plan_step(*args)
    before = ([0] * b, table.tolist(), ring.tolist(), state.tolist())
    held = {}
    for step in range(60):
        n = np.ones(b, dtype=int)
        for i in range(b):
            if before[0][i] == 0:
                n[i] = rng.choice([0, int(rng.integers(1, 20))])
            elif rng.random() < 0.1:
                n[i] = -1
        new.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        want = host_plan(before[0], n.tolist(), page, before[1], before[2], *before[3], t)
        got = (table, ring, lengths, starts, slots, positions, sequences, state[0], state[1])
        for g, w in zip(got, want):
            assert np.array_equal(np.asarray(g.cpu()).flatten(), np.asarray(w).flatten()), step
        before = (lengths.tolist(), table.tolist(), ring.tolist(), state.tolist())
        # no page has two owners, none is lost
        owned = [p for i in range(b) for p in before[1][i][:-(-before[0][i] // page)]]
        free = [before[2][(before[3][0] + i) % pages] for i in range(before[3][1])]
        assert sorted(owned + free) == list(range(pages)), step
        held[step] = len(owned)
    assert max(held.values()) > pages // 2 and nf4.nf4_check_device_error() == 0


def test_two_streams_and_repeats_give_the_same():
    rng = np.random.default_rng(3)
    states = [make(rng, 500, 16, 20, 3000, finished=0.1, long=0.3, spare=900) for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, stream in zip(states, streams):
            s.run(stream)
    torch.cuda.synchronize()
    for s in states:
        s.check()
