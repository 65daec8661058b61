"""Calls whose inputs the call before them wrote on the same stream: tables,
lengths and slots from pa_plan_append, rotated queries and keys from
pa_norm_rope_and_cache, lengths from pa_tree_accept, read by the cache write
and the single-token decodes.  Captured once and replayed back to back, the
state advancing on the device; compared with the oracles every few steps."""

import numpy as np
import pytest
import torch

import paged_kv_cache_354_b200 as pk
import workloads
from oracle import paged_attention as opa
from oracle import tree_speculation as ots
from tests.gpu_helpers import bf16_to_f64, compare, default_scale, workspace_for
from tests.test_gpu_norm_rope import EPS, close, table

pytestmark = pytest.mark.gpu

B, BS, D, WIDTH = 7, 16, 128, 30


class Chain:
    def __init__(self, hq, hkv, seed, partition_tokens=0):
        rng = np.random.default_rng(seed)
        self.hq, self.hkv = hq, hkv
        self.order = rng.permutation(B * WIDTH)
        self.cs = table(WIDTH * BS, D).cuda()
        self.pool = torch.zeros((B * WIDTH, 2, hkv, BS, D), dtype=torch.bfloat16, device="cuda")
        self.tables = torch.zeros((B, WIDTH), dtype=torch.int32, device="cuda")
        self.held, self.lens = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
        self.free = torch.as_tensor(self.order[::-1].astype(np.int32)).cuda()
        self.num_free = torch.full((1,), B * WIDTH, dtype=torch.int32, device="cuda")
        self.new = torch.ones(B, dtype=torch.int32, device="cuda")
        self.slots = torch.empty((B, 1), dtype=torch.int64, device="cuda")
        self.positions = torch.empty((B, 1), dtype=torch.int32, device="cuda")
        self.q, self.k, self.v = (workloads.bf16_normal((B, h, D), seed=seed + i).cuda()
                                  for i, h in enumerate((hq, hkv, hkv)))
        self.q_out, self.k_out, self.out = (torch.zeros_like(x) for x in (self.q, self.k, self.q))
        self.partition_tokens = partition_tokens
        self.ws, _ = workspace_for(B, hq, hkv, D, BS, WIDTH * BS, partition_tokens)
        self.state = [[0] * WIDTH for _ in range(B)], [0] * B, list(self.order[::-1]), [0] * B

    def plan(self, new=None):
        pk.pa_plan_append(self.tables, self.held, self.free, self.num_free, self.lens, self.new if new is None else new,
                          self.slots, self.positions, BS)

    def token(self, fused):
        """One token per request: planned, rotated, written and attended over."""
        self.plan()
        pk.pa_norm_rope_and_cache(self.q_out, self.q, self.k, self.v, None, None, self.positions.view(-1), self.cs,
                                  eps=EPS, k_out=self.k_out)
        if fused:
            pk.pa_decode_append(self.out, self.q_out, self.pool, self.k_out, self.v, self.slots.view(-1), self.tables,
                                self.lens, WIDTH * BS, default_scale(D), workspace=self.ws)
        else:
            pk.pa_reshape_and_cache(self.k_out, self.v, self.pool, self.slots.view(-1))
            pk.pa_decode(self.out, self.q_out, self.pool, self.tables, self.lens, WIDTH * BS, default_scale(D),
                         workspace=self.ws, partition_tokens=self.partition_tokens)

    def advance(self, new):
        *self.state, slots, positions = ots.plan_append(*self.state, new, BS, WIDTH)
        return slots, positions

    def check(self, slots, positions):
        tables, held, free, lens = self.state
        assert self.lens.tolist() == lens and self.held.tolist() == held and self.tables.tolist() == tables
        assert self.slots.tolist() == slots and self.positions.tolist() == positions
        at = np.array(positions).reshape(-1)
        for x, y in ((self.q, self.q_out), (self.k, self.k_out)):
            close(y, *ots.norm_rope(bf16_to_f64(x), None, EPS, self.cs.double().cpu().numpy(), at, False))
        slot = torch.as_tensor(np.array(slots).reshape(-1)).cuda()
        assert torch.equal(self.pool[slot // BS, 0, :, slot % BS], self.k_out)
        assert torch.equal(self.pool[slot // BS, 1, :, slot % BS], self.v)
        want = opa.decode(bf16_to_f64(self.q_out), bf16_to_f64(self.pool), np.array(tables), np.array(lens), default_scale(D))
        compare(bf16_to_f64(self.out), want)


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("hq,hkv,partition_tokens", [(8, 2, 0), (32, 2, 0), (8, 2, 64)])
def test_a_token_planned_rotated_written_and_attended(fused, hq, hkv, partition_tokens):
    c = Chain(hq, hkv, seed=hq, partition_tokens=0 if fused else partition_tokens)
    prompts = torch.tensor([0, 1, 15, 16, 17, 100, 250], dtype=torch.int32)  # rows of zeros before the first token
    slots = torch.empty(int(prompts.sum()), dtype=torch.int64, device="cuda")
    starts = torch.empty(B + 1, dtype=torch.int32, device="cuda")
    pk.pa_plan_append(c.tables, c.held, c.free, c.num_free, c.lens, prompts.cuda(), slots,
                      torch.empty_like(slots, dtype=torch.int32), BS, token_starts=starts)
    c.advance(prompts.tolist())
    c.token(fused)
    c.check(*c.advance([1] * B))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.token(fused)
    for replays in (1, 2, 30):
        for x in (c.q, c.k, c.v):
            x.copy_(torch.roll(x, 1, 0))
        for _ in range(replays):
            g.replay()
            want = c.advance([1] * B)
        c.check(*want)
    assert pk.pa_device_error() == 0


def test_lengths_after_accepted_paths_are_what_the_next_decode_sees():
    """Plan 4 nodes, accept some in place, decode over what is left; replayed."""
    c = Chain(8, 2, seed=3)
    c.pool.copy_(workloads.bf16_normal(tuple(c.pool.shape), seed=4))
    four = torch.full((B,), 4, dtype=torch.int32, device="cuda")
    slots, positions = (torch.empty((B, 4), dtype=t, device="cuda") for t in (torch.int64, torch.int32))
    path = torch.tensor([[1, 3]] * B, dtype=torch.int32, device="cuda")
    accepted = torch.tensor([2, 1, 0, 2, 2, 1, 1], dtype=torch.int32, device="cuda")

    def step():
        pk.pa_plan_append(c.tables, c.held, c.free, c.num_free, c.lens, four, slots, positions, BS)
        pk.pa_tree_accept(c.pool, path, accepted, c.tables, c.lens, four, seq_lens_out=c.lens)
        pk.pa_decode(c.out, c.q, c.pool, c.tables, c.lens, WIDTH * BS, default_scale(D), workspace=c.ws)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for steps in range(2, 40):
        g.replay()
        if steps % 6 and steps != 39:
            continue
        lens = [steps * int(a) for a in accepted]
        assert c.lens.tolist() == lens
        want = opa.decode(bf16_to_f64(c.q), bf16_to_f64(c.pool), c.tables.cpu().numpy(), np.array(lens), default_scale(D))
        compare(bf16_to_f64(c.out), want)
    assert pk.pa_device_error() == 0
