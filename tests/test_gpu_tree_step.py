"""The four tree-speculation calls together, as a serving loop uses them
(engine.PagedTreeCache): prompts in, steps of drafted trees, accepted paths,
ended requests, a step without enough blocks, eager and replayed from a
graph.  After every call the device state is compared with the oracle's: block
tables, lengths and slots for equality, cached rows, queries and attention
within their tolerances."""

import numpy as np
import pytest
import torch

from oracle import tree_speculation as ots
from paged_kv_cache_354_b200.engine import PagedTreeCache
import paged_kv_cache_354_b200 as pk
import workloads
from tests.gpu_helpers import bf16_to_f64
from tests.test_gpu_decode_tree import pack, random_trees
from tests.test_gpu_norm_rope import EPS, close, table

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS, B, T, WIDTH = 8, 2, 128, 16, 5, 12, 20


class Loop:
    def __init__(self, num_blocks, seed):
        self.rng = np.random.default_rng(seed)
        order = self.rng.permutation(num_blocks)
        self.cs = table(WIDTH * BS + T, D).cuda()
        self.weights = [(1 + 0.2 * workloads.bf16_normal((D,), seed=seed + i)).bfloat16().cuda() for i in range(2)]
        self.c = PagedTreeCache(num_blocks, HQ, HKV, D, BS, B, WIDTH * BS, T, self.cs, *self.weights, eps=EPS,
                                initial_order=order)
        self.c.pool.fill_(float("nan"))
        self.state = [[0] * WIDTH for _ in range(B)], [0] * B, list(order[::-1]), [0] * B

    def same_state(self):
        tables, held, free, lens = self.state
        assert self.c.held.tolist() == held and self.c.lens.tolist() == lens
        assert self.c.tables.tolist() == tables
        assert self.c.num_free.item() == len(free) and self.c.free.tolist()[: len(free)] == [int(x) for x in free]

    def normed(self, x, weight, positions):
        return ots.norm_rope(bf16_to_f64(x), bf16_to_f64(weight), EPS, self.cs.double().cpu().numpy(), positions, False)

    def rows_are_cached(self, k, v, positions, slots, before):
        """The tokens' rows hold their keys and values; all others are as they were."""
        want, bound = self.normed(k, self.weights[1], positions)
        live = torch.as_tensor(slots >= 0).cuda()
        block, off = torch.as_tensor(slots // BS).cuda()[live], torch.as_tensor(slots % BS).cuda()[live]
        close(self.c.pool[block, 0, :, off], want[slots >= 0], bound[slots >= 0])
        assert torch.equal(self.c.pool[block, 1, :, off], v[live])
        now = self.c.pool.clone()
        now[block, :, :, off] = before[block, :, :, off]
        assert torch.equal(now.view(torch.int16), before.view(torch.int16))

    def slab(self, n):
        x = torch.as_tensor(self.rng.standard_normal((n, (HQ + 2 * HKV) * D))).bfloat16().cuda()
        return [x[:, a * D:(a + h) * D].unflatten(1, (h, D)) for a, h in ((0, HQ), (HQ, HKV), (HQ + HKV, HKV))]

    def prefill(self, counts):
        n = sum(counts) + 3
        q, k, v = self.slab(n)
        q_out = torch.empty((n, HQ, D), dtype=torch.bfloat16, device="cuda")
        before = self.c.pool.clone()
        slots, positions = self.c.prefill(torch.tensor(counts, dtype=torch.int32).cuda(), q, k, v, q_out)
        *self.state, want_slots, want_pos = ots.plan_append(*self.state, counts, BS, WIDTH)
        want_slots = np.array([x for r in want_slots for x in r] + [-1] * 3)
        want_pos = np.array([x for r in want_pos for x in r] + [-1] * 3)
        assert slots.tolist() == want_slots.tolist() and positions.tolist() == want_pos.tolist()
        self.same_state()
        self.rows_are_cached(k, v, want_pos, want_slots, before)
        close(q_out, *self.normed(q, self.weights[0], want_pos))

    def draft(self):
        counts = [int(x) if n else 0 for x, n in zip(self.rng.integers(0, T, B, endpoint=True), self.state[3])]
        sees = random_trees(self.rng, B, T)
        return counts, sees, sees.sum(-1) - 1, self.slab(B * T)

    def check_step(self, counts, sees, depths, qkv, out, before):
        base = list(self.state[3])
        *self.state, slots, _ = ots.plan_append(*self.state, counts, BS, WIDTH)
        self.same_state()
        flat = np.array([r + [-1] * (T - len(r)) for r in slots]).reshape(-1)
        positions = np.array([[base[b] + depths[b, t] if t < counts[b] else -1 for t in range(T)] for b in range(B)])
        self.rows_are_cached(qkv[1], qkv[2], positions.reshape(-1), flat, before)
        close(self.c.q.view(-1, HQ, D), *self.normed(qkv[0], self.weights[0], positions.reshape(-1)))
        # the attention, from the queries and rows as they were rounded
        want, spread, size, logit = ots.decode_tree(bf16_to_f64(self.c.q), bf16_to_f64(self.c.pool), sees,
                                                    self.state[0], self.state[3], counts, self.c.scale)
        length = np.array(self.state[3], dtype=np.float64)[:, None, None, None]
        fp32 = 2.0 ** -23 * (2 * (D + 4) * logit[..., None] + length + 1000)
        bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -8 * (1 + 2.0 ** -7) * spread + fp32 * size
        assert (np.abs(bf16_to_f64(out) - want) <= bound).all()

    def pick(self, counts, sees):
        """A random node per request, with all its ancestors."""
        path, accepted = np.zeros((B, T), dtype=np.int32), []
        for b, n in enumerate(counts):
            chain = np.flatnonzero(sees[b, int(self.rng.integers(0, n))]) if n else []
            path[b, : len(chain)] = chain
            accepted.append(len(chain))
        return path, accepted

    def check_accept(self, path, accepted, counts, before):
        pool = before.view(torch.int16).cpu().numpy()
        want, lens = ots.tree_accept(pool.copy(), path, accepted, counts, self.state[0], self.state[3])
        assert np.array_equal(self.c.pool.view(torch.int16).cpu().numpy(), want)
        self.state[3] = [int(n) for n in lens]
        self.same_state()


@pytest.mark.parametrize("captured", [False, True])
def test_serving_loop(captured):
    loop = Loop(60, seed=1)
    c = loop.c
    loop.prefill([40, 3, 0, 100, 17])
    loop.prefill([0, 5, 30, 1, 0])
    counts_d = torch.zeros(B, dtype=torch.int32, device="cuda")
    mask_d = torch.zeros((B, T, 1), dtype=torch.int32, device="cuda")
    depths_d = torch.zeros((B, T), dtype=torch.int32, device="cuda")
    path_d = torch.zeros((B, T), dtype=torch.int32, device="cuda")
    accepted_d = torch.zeros(B, dtype=torch.int32, device="cuda")
    slab_d = torch.zeros((B * T, (HQ + 2 * HKV) * D), dtype=torch.bfloat16, device="cuda")
    qkv_d = [slab_d[:, a * D:(a + h) * D].unflatten(1, (h, D)) for a, h in ((0, HQ), (HQ, HKV), (HQ + HKV, HKV))]
    out = torch.empty((B, T, HQ, D), dtype=torch.bfloat16, device="cuda")
    graphs = None
    for i in range(8):
        counts, sees, depths, qkv = loop.draft()
        for dst, src in zip(qkv_d, qkv):
            dst.copy_(src)
        counts_d.copy_(torch.tensor(counts, dtype=torch.int32))
        mask_d.copy_(pack(sees))
        depths_d.copy_(torch.as_tensor(depths))
        before = c.pool.clone()
        out.fill_(float("nan"))
        path, accepted = loop.pick(counts, sees)
        path_d.copy_(torch.as_tensor(path))
        accepted_d.copy_(torch.tensor(accepted, dtype=torch.int32))
        if captured and i == 1:  # the first step ran eagerly
            graphs = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
            with torch.cuda.graph(graphs[0]):
                c.step(*qkv_d, counts_d, mask_d, depths_d, out)
            with torch.cuda.graph(graphs[1]):
                c.accept(path_d, accepted_d)
        if graphs:
            graphs[0].replay()
        else:
            c.step(*qkv_d, counts_d, mask_d, depths_d, out)
        loop.check_step(counts, sees, depths, qkv_d, out, before)
        before = c.pool.clone()
        if graphs:
            graphs[1].replay()
        else:
            c.accept(path_d, accepted_d)
        loop.check_accept(path, accepted, counts, before)
        if i == 4:
            c.release(torch.tensor([False, True, False, True, False]).cuda())
            loop.state = list(ots.plan_append(*loop.state, [0, -1, 0, -1, 0], BS, WIDTH)[:4])
            loop.same_state()
            loop.prefill([0, 20, 0, 0, 2])
    assert pk.pa_device_error() == 0


def test_a_step_without_blocks_changes_nothing():
    loop = Loop(6, seed=2)
    c = loop.c
    loop.prefill([30, 16, 16, 16, 0])  # 5 of 6 blocks
    counts, sees, depths = [12, 1, 1, 0, 0], random_trees(loop.rng, B, T), np.zeros((B, T), dtype=np.int32)
    qkv = loop.slab(B * T)
    before = c.pool.clone()
    out = torch.full((B, T, HQ, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    pk.pa_device_error(clear=True)
    c.step(*qkv, torch.tensor(counts, dtype=torch.int32).cuda(), pack(sees).cuda(), torch.as_tensor(depths).cuda(), out)
    assert pk.pa_device_error() == pk.PA_DEVERR_NO_BLOCKS and c.status.item() == pk.PA_DEVERR_NO_BLOCKS
    loop.same_state()
    assert not out.any() and torch.equal(c.pool.view(torch.int16), before.view(torch.int16))
    c.accept(torch.arange(T, dtype=torch.int32).repeat(B, 1).cuda(), torch.tensor([3, 1, 1, 0, 0], dtype=torch.int32).cuda())
    assert pk.pa_device_error() == pk.PA_DEVERR_TREE
    loop.same_state()
    assert torch.equal(c.pool.view(torch.int16), before.view(torch.int16))


def test_step_on_another_stream():
    """Every call of a step goes to the current stream: behind a long fill on a
    stream of its own, nothing else may run ahead of its inputs."""
    loop = Loop(60, seed=3)
    c = loop.c
    loop.prefill([40, 3, 0, 100, 17])
    counts, sees, depths, qkv = loop.draft()
    path, accepted = loop.pick(counts, sees)
    host = [torch.tensor(counts, dtype=torch.int32), pack(sees), torch.as_tensor(depths, dtype=torch.int32),
            torch.as_tensor(path), torch.tensor(accepted, dtype=torch.int32)]
    given = [t.cuda() for t in host]
    late = [torch.zeros_like(t) for t in given]
    out = torch.full((B, T, HQ, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    filler = torch.empty(1 << 29, dtype=torch.uint8, device="cuda")
    before = c.pool.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(5):
            filler.fill_(1)
        for dst, src in zip(late, given):
            dst.copy_(src)
        c.step(*qkv, *late[:3], out)
        between = c.pool.clone()
        c.accept(*late[3:])
    side.synchronize()
    base = list(loop.state[3])
    *loop.state, slots, _ = ots.plan_append(*loop.state, counts, BS, WIDTH)
    flat = np.array([r + [-1] * (T - len(r)) for r in slots]).reshape(-1)
    positions = np.array([[base[b] + depths[b, t] if t < counts[b] else -1 for t in range(T)] for b in range(B)])
    after, c.pool = c.pool, between
    loop.rows_are_cached(qkv[1], qkv[2], positions.reshape(-1), flat, before)
    c.pool = after
    loop.check_accept(path, accepted, counts, between)
    assert torch.isfinite(out).all() and out.any() and pk.pa_device_error() == 0
