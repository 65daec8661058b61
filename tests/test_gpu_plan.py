"""pa_plan_append against the oracle, which is pinned to the host allocator:
whole numbers, compared for equality.  Both layouts, ended requests, requests
that hold more than they need, refusals that change nothing, state updated in
place and apart, and steps replayed from a graph."""

import numpy as np
import pytest
import torch

import paged_kv_cache_354_b200 as pk
from oracle import tree_speculation as ots

pytestmark = pytest.mark.gpu


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=dtype).cuda()


class State:
    def __init__(self, rng, batch, bs, width, longest, spare, extra=True):
        self.bs, self.width = bs, width
        self.lens = [int(x) for x in rng.integers(0, longest, batch, endpoint=True)]
        self.held = [min(width, -(-n // bs) + (int(rng.integers(0, 2)) if extra else 0)) for n in self.lens]
        order = rng.permutation(sum(self.held) + spare)
        self.blocks = len(order)
        self.tables, at = [], 0
        for h in self.held:
            self.tables.append([int(x) for x in order[at:at + h]] + [0] * (width - h))
            at += h
        self.free = [int(x) for x in order[at:]]
        self.g_tables, self.g_held, self.g_lens = dev(self.tables), dev(self.held), dev(self.lens)
        self.g_free = dev(self.free + [-7] * (self.blocks - len(self.free)))
        self.g_num = dev([len(self.free)])

    def want(self, new):
        return ots.plan_append(self.tables, self.held, self.free, self.lens, new, self.bs, self.width)

    def same(self, got=None):
        """The device state equals `got` (or the state before)."""
        tables, held, free, lens = got[:4] if got else (self.tables, self.held, self.free, self.lens)
        assert self.g_tables.tolist() == tables and self.g_held.tolist() == held
        assert self.g_num.item() == len(free) and self.g_free.tolist()[: len(free)] == free
        assert self.g_lens.tolist() == lens


def call(s, new, most=None, num_slots=None, depths=None, out=None, appended=None, status=None):
    b = len(new)
    shape = (b, most) if most else (num_slots,)
    slots = torch.full(shape, 99, dtype=torch.int64, device="cuda")
    positions = torch.full(shape, 99, dtype=torch.int32, device="cuda")
    starts = torch.full((b + 1,), 99, dtype=torch.int32, device="cuda")
    more = {} if out is None else dict(zip(("seq_lens_out", "blocks_held_out", "num_free_out"), out))
    pk.pa_plan_append(s.g_tables, s.g_held, s.g_free, s.g_num, s.g_lens, dev(new), slots, positions, s.bs,
                      depths=depths, token_starts=starts, appended_out=appended, status_out=status, **more)
    return slots, positions, starts


def check_tokens(got, want, most, new):
    slots, positions, starts = (t.tolist() for t in got)
    counts = [max(c, 0) for c in new]
    assert starts == [sum(counts[:i]) for i in range(len(counts) + 1)]
    if most:
        assert slots == [s + [-1] * (most - len(s)) for s in want[4]]
        assert positions == [p + [-1] * (most - len(p)) for p in want[5]]
    else:
        flat = [x for s in want[4] for x in s], [x for p in want[5] for x in p]
        assert slots == flat[0] + [-1] * (len(slots) - len(flat[0]))
        assert positions == flat[1] + [-1] * (len(slots) - len(flat[0]))


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("batch,bs,most", [(1, 16, 1), (1, 16, 300), (3, 32, 5), (37, 16, 33), (129, 1, 7), (1500, 16, 9),
                                           (5000, 32, 2)])
def test_steps_match_the_oracle(packed, batch, bs, most):
    rng = np.random.default_rng(batch + most)
    width = 6 + (most + bs - 1) // bs
    s = State(rng, batch, bs, width, 4 * bs, batch * width)
    for step in range(3):
        new = [int(x) for x in rng.integers(0, most, batch, endpoint=True)]
        for b in range(batch):
            if rng.random() < 0.2 or s.lens[b] + new[b] > s.width * bs:
                new[b] = -1 - int(rng.integers(0, 3))
        appended, status = dev([99] * batch), dev([99])
        got = call(s, new, None if packed else most, sum(max(c, 0) for c in new) + 3, appended=appended, status=status)
        assert appended.tolist() == [max(c, 0) for c in new] and status.item() == 0
        want = s.want(new)
        check_tokens(got, want, None if packed else most, new)
        s.same(want)
        s.tables, s.held, s.free, s.lens = want[:4]
    assert pk.pa_device_error() == 0


def test_outputs_apart_from_inputs_and_again():
    rng = np.random.default_rng(3)
    s = State(rng, 20, 16, 8, 60, 100)
    new = [int(x) for x in rng.integers(-1, 20, 20)]
    want = s.want(new)
    lens, held, num = s.g_lens.clone(), s.g_held.clone(), s.g_num.clone()
    out = [torch.full_like(t, -5) for t in (s.g_lens, s.g_held, s.g_num)]
    for _ in range(2):  # the inputs are left as they were, so a second call gives the same
        got = call(s, new, 20, out=out)
        check_tokens(got, want, 20, new)
        assert torch.equal(s.g_lens, lens) and torch.equal(s.g_held, held) and torch.equal(s.g_num, num)
        assert out[0].tolist() == want[3] and out[1].tolist() == want[1] and out[2].item() == len(want[2])
        assert s.g_tables.tolist() == want[0] and s.g_free.tolist()[: len(want[2])] == want[2]


def test_depths_give_tree_positions():
    rng = np.random.default_rng(4)
    s = State(rng, 5, 16, 8, 60, 40)
    new = [4, 0, 3, 4, 1]
    depth = [[0, 1, 1, 2], [0, 0, 0, 0], [0, 0, 1, 5], [0, 1, 2, 3], [0, 9, 9, 9]]
    lens = list(s.lens)
    want = s.want(new)
    slots, positions, _ = call(s, new, 4, depths=dev(depth))
    assert slots.tolist() == [x + [-1] * (4 - len(x)) for x in want[4]]
    assert positions.tolist() == [[lens[b] + depth[b][t] if t < new[b] else -1 for t in range(4)] for b in range(5)]
    s.tables, s.held, s.free, s.lens = want[:4]
    lens = list(s.lens)
    _, positions, _ = call(s, [2, 2, 2, 2, 2], 2, depths=dev([0, 0]))
    assert positions.tolist() == [[n, n] for n in lens]


# one request's tokens are bounded in the padded layout, all together in the packed one
@pytest.mark.parametrize("what,packed", [(w, p) for w in ("blocks", "row", "length", "held", "free", "stack")
                                         for p in (False, True)] + [("count", False), ("capacity", True)])
def test_refused_calls_change_nothing(what, packed):
    rng = np.random.default_rng(5)
    s = State(rng, 6, 16, 8, 50, 4, extra=False)
    new, code, num_slots = [3, 2, 1, 0, 4, 2], pk.PA_DEVERR_PLAN, 20
    if what == "blocks":
        new, code = [4, 4, 4, -1, 4, 4], pk.PA_DEVERR_NO_BLOCKS
        s.g_lens = dev([32, 16, 48, 0, 16, 32])
        s.g_held = dev([2, 1, 3, 0, 1, 2])
    elif what == "row":
        s.g_lens[2] = 8 * 16
    elif what == "count":
        new[1] = 5
    elif what == "length":
        s.g_lens[0] = -1
    elif what == "held":
        s.g_held[4] = 9
    elif what == "free":
        s.g_num[0] = -1
    elif what == "capacity":
        num_slots = 11
    else:  # returned blocks beyond the stack
        s.g_num[0] = s.blocks
        s.g_held[3], new[3] = 1, -1
    before = [t.clone() for t in (s.g_tables, s.g_held, s.g_free, s.g_num, s.g_lens)]
    status, appended = dev([99]), dev([99] * 6)
    pk.pa_device_error(clear=True)
    slots, positions, starts = call(s, new, None if packed else 4, num_slots, appended=appended, status=status)
    assert pk.pa_device_error() == code and status.item() == code
    assert not appended.any()
    for t, was in zip((s.g_tables, s.g_held, s.g_free, s.g_num, s.g_lens), before):
        assert torch.equal(t, was)
    assert (slots == -1).all() and (positions == -1).all() and (starts == 0).all()


def test_a_bad_block_gives_no_slot():
    s = State(np.random.default_rng(6), 2, 16, 4, 30, 4, extra=False)
    s.g_lens = dev([4, 4])
    s.g_held = dev([1, 1])
    s.g_tables = dev([[s.blocks, 0, 0, 0], [-1, 0, 0, 0]])
    pk.pa_device_error(clear=True)
    slots, positions, _ = call(s, [1, 2], 2)
    assert pk.pa_device_error() == pk.PA_DEVERR_BLOCK_ID
    assert (slots == -1).all() and positions.tolist() == [[4, -1], [4, 5]]


def test_captured_steps():
    """An in-place step captured once and replayed advances the state as
    eager calls do."""
    rng = np.random.default_rng(8)
    s = State(rng, 9, 16, 30, 40, 200)
    new = dev([3, 0, 1, 4, 4, 2, 1, 1, 3])
    slots = torch.empty((9, 4), dtype=torch.int64, device="cuda")
    positions = torch.empty((9, 4), dtype=torch.int32, device="cuda")

    def step():
        pk.pa_plan_append(s.g_tables, s.g_held, s.g_free, s.g_num, s.g_lens, new, slots, positions, 16)

    step()
    want = s.want(new.tolist())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(5):
        s.tables, s.held, s.free, s.lens = want[:4]
        want = s.want(new.tolist())
        g.replay()
        assert slots.tolist() == [x + [-1] * (4 - len(x)) for x in want[4]]
        s.same(want)


@pytest.mark.parametrize("packed", [False, True])
def test_captured_large_steps(packed):
    """The launches of a large call, replayed: the in-place state advances."""
    rng = np.random.default_rng(9)
    batch, most = 700, 12
    s = State(rng, batch, 16, 30, 40, batch * 20)
    counts = [int(x) for x in rng.integers(0, most, batch, endpoint=True)]
    new = dev(counts)
    shape = (sum(counts) + 300,) if packed else (batch, most)
    slots = torch.empty(shape, dtype=torch.int64, device="cuda")
    positions = torch.empty(shape, dtype=torch.int32, device="cuda")
    starts = torch.empty(batch + 1, dtype=torch.int32, device="cuda")

    def step():
        pk.pa_plan_append(s.g_tables, s.g_held, s.g_free, s.g_num, s.g_lens, new, slots, positions, 16,
                          token_starts=starts)

    step()
    want = s.want(counts)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        s.tables, s.held, s.free, s.lens = want[:4]
        want = s.want(counts)
        g.replay()
        check_tokens((slots, positions, starts), want, None if packed else most, counts)
        s.same(want)


def test_one_long_prompt_among_empty_requests():
    """Packed slots whose requests are hundreds of entries apart."""
    batch = 1500
    s = State(np.random.default_rng(10), batch, 16, 700, 0, 4000, extra=False)
    new = [0] * batch
    new[0], new[700], new[701], new[1499] = 5000, 1, 4100, 3
    got = call(s, new, None, sum(new) + 1000)
    want = s.want(new)
    check_tokens(got, want, None, new)
    s.same(want)


@pytest.mark.parametrize("what", ["blocks", "row"])
@pytest.mark.parametrize("packed", [False, True])
def test_refused_large_calls_change_nothing(what, packed):
    batch, most = 2500, 3
    s = State(np.random.default_rng(11), batch, 16, 8, 50, 10 if what == "blocks" else batch, extra=False)
    new = [most] * batch
    if what == "blocks":
        s.g_held.zero_()
        s.g_lens.fill_(15)
    else:
        s.g_lens[2400] = 8 * 16
    before = [t.clone() for t in (s.g_tables, s.g_held, s.g_free, s.g_num, s.g_lens)]
    pk.pa_device_error(clear=True)
    slots, positions, starts = call(s, new, None if packed else most, most * batch + 9)
    assert pk.pa_device_error() == (pk.PA_DEVERR_NO_BLOCKS if what == "blocks" else pk.PA_DEVERR_PLAN)
    for t, was in zip((s.g_tables, s.g_held, s.g_free, s.g_num, s.g_lens), before):
        assert torch.equal(t, was)
    assert (slots == -1).all() and (positions == -1).all() and (starts == 0).all()


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("batch,most", [(700, 12), (2500, 3)])
def test_depths_in_large_plans(batch, most, shared):
    """Tree positions where several CTAs share the requests, some of which end,
    the state in place and then apart."""
    rng = np.random.default_rng(batch)
    s = State(rng, batch, 16, 8, 60, batch * 3)
    for apart in (False, True):
        new = [int(x) if rng.random() > 0.1 else -1 for x in rng.integers(0, most, batch, endpoint=True)]
        depth = rng.integers(0, 40, (most,) if shared else (batch, most))
        at = np.broadcast_to(depth, (batch, most))
        lens, want = list(s.lens), s.want(new)
        out = [torch.full_like(t, -5) for t in (s.g_lens, s.g_held, s.g_num)] if apart else None
        slots, positions, _ = call(s, new, most, depths=dev(depth), out=out)
        assert slots.tolist() == [x + [-1] * (most - len(x)) for x in want[4]]
        assert positions.tolist() == [[lens[b] + int(at[b, t]) if t < new[b] else -1 for t in range(most)]
                                      for b in range(batch)]
        if apart:
            s.g_lens, s.g_held, s.g_num = out
        s.same(want)
        s.tables, s.held, s.free, s.lens = want[:4]
    assert pk.pa_device_error() == 0
