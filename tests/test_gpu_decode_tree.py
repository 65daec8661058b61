"""pa_decode_tree against the fp64 oracle.

Tolerance per element, from the roundings the call makes (p the softmax
weights, want = sum p v):
  * the output's rounding to bf16: 2^-8 |want|;
  * each probability's rounding to bf16, at most 2^-8 of it.  The sum that
    divides takes the rounded values, so the error is
    sum p d (v - want) / (1 + sum p d) with |d| <= 2^-8: at most
    2^-8 (1 + 2^-7) sum p |v - want|;
  * fp32: a logit of D products and its scaling is off by at most
    2^-23 (D + 4) S, S = max scale sum |q||k| over the row's positions (a
    truncating accumulator loses 2^-23 per addition), which moves every
    weight by twice that relatively; exp2's error and argument add below
    2^-20; a sum of L terms, rescaled at most once per 32 positions and
    merged over at most 512 pieces, is off by at most 2^-23 (L + 600):
    together 2^-23 (2 (D + 4) S + L + 1000) sum p |v|.
Unused pool rows are NaN."""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_354_b200 as pk
import workloads
from oracle import tree_speculation as ots
from tests.gpu_helpers import bf16_to_f64, build_tables, poison_unused

pytestmark = pytest.mark.gpu


def random_trees(rng, b, nodes, shared=False):
    sees = np.zeros((b, nodes, nodes), dtype=bool)
    for i in range(1 if shared else b):
        for t in range(nodes):
            parent = int(rng.integers(-1, t))
            if parent >= 0:
                sees[i, t] = sees[i, parent]
            sees[i, t, t] = True
    if shared:
        sees[:] = sees[0]
    return sees


def pack(sees):
    """bool [..., T, T] -> int32 bits [..., T, ceil(T / 32)]."""
    nodes = sees.shape[-1]
    words = -(-nodes // 32)
    bits = np.zeros(sees.shape[:-1] + (words * 32,), dtype=np.uint64)
    bits[..., :nodes] = sees
    packed = (bits.reshape(sees.shape[:-1] + (words, 32)) << np.arange(32, dtype=np.uint64)).sum(-1)
    return torch.as_tensor(packed.astype(np.uint32).view(np.int32))


class Case:
    def __init__(self, lens, counts, nodes, hq, hkv, d, bs, seed, sees=None, scale=None, shared=False):
        rng = np.random.default_rng(seed)
        lens = [int(n) for n in lens]
        nb = sum(-(-n // bs) for n in lens) + 3
        self.t_ref, self.l_ref, self.tables, self.lens, used = build_tables(lens, bs, nb, rng.permutation(nb))
        self.pool = poison_unused(workloads.bf16_normal((nb, 2, hkv, bs, d), seed=seed), used)
        self.q = workloads.bf16_normal((len(lens), nodes, hq, d), seed=seed + 1)
        self.counts = [nodes] * len(lens) if counts is None else [int(c) for c in counts]
        self.given = counts is not None
        self.sees = random_trees(rng, len(lens), nodes, shared) if sees is None else sees
        self.shared = shared
        self.scale = 1.0 / math.sqrt(d) if scale is None else scale
        self.bs = bs

    def slot(self, b, pos):
        return int(self.t_ref[b][pos // self.bs]), pos % self.bs

    def run(self, pool=None, out=None, max_len=None, stream=None, workspace=None):
        q = self.q.cuda()
        b, nodes, hq, d = q.shape
        pool = self.pool.cuda() if pool is None else pool
        max_len = max(1, int(np.max(self.lens))) if max_len is None else max_len
        if workspace is None:
            need = pk.pa_decode_tree_workspace_size(b, nodes, hq, pool.shape[2], d, self.bs, max_len)
            workspace = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
        out = torch.full_like(q, float("nan")) if out is None else out
        mask = pack(self.sees[0] if self.shared else self.sees).cuda()
        counts = torch.as_tensor(self.counts, dtype=torch.int32).cuda() if self.given else None
        pk.pa_decode_tree(out, q, pool, mask, torch.as_tensor(self.tables).cuda(), torch.as_tensor(self.lens).cuda(),
                          max_len, self.scale, workspace, tree_lens=counts, stream=stream)
        torch.cuda.synchronize()
        return out

    def want(self):
        return ots.decode_tree(bf16_to_f64(self.q), bf16_to_f64(self.pool), self.sees, self.t_ref, self.l_ref,
                               self.counts, self.scale)

    def tolerance(self, want, spread, size, logit):
        d = self.q.shape[3]
        length = self.l_ref[:, None, None, None].astype(np.float64)
        fp32 = 2.0 ** -23 * (2 * (d + 4) * logit[..., None] + length + 1000)
        return 2.0 ** -8 * np.abs(want) + 2.0 ** -8 * (1 + 2.0 ** -7) * spread + fp32 * size

    def check(self, out=None):
        out = bf16_to_f64(self.run() if out is None else out)
        want, spread, size, logit = self.want()
        assert np.isfinite(out).all()
        off = np.abs(out - want) - self.tolerance(want, spread, size, logit)
        assert (off <= 0).all(), (off.max(), np.argwhere(off > 0)[:5].tolist())
        for b, n in enumerate(self.counts):
            assert not out[b, n if self.l_ref[b] else 0:].any()
        assert pk.pa_device_error() == 0


@pytest.mark.parametrize("nodes,hq,hkv", [(1, 4, 4), (1, 8, 1), (2, 8, 2), (7, 3, 3), (16, 8, 2), (31, 4, 4), (33, 2, 2),
                                          (32, 8, 2), (17, 30, 2), (64, 8, 1), (65, 2, 1), (100, 6, 2), (130, 5, 1),
                                          (20, 64, 1)])
@pytest.mark.parametrize("d,bs", [(128, 16), (64, 32), (128, 32), (64, 16)])
def test_matches_the_oracle(nodes, hq, hkv, d, bs):
    lens = [nodes, nodes + 1, nodes + 15, nodes + 127, nodes + 128, nodes + 250, nodes + 777]
    Case(lens, None, nodes, hq, hkv, d, bs, seed=nodes + hq).check()


def test_ragged_batch_of_wide_trees():
    """Requests of one, several and no row-tile pairs in one batch; the
    requests of one count alone take the other order of work."""
    rng = np.random.default_rng(31)
    counts = np.array([70, 3, 0, 33, 64, 1, 70, 16, 48, 17])
    lens = counts + rng.integers(0, 700, 10)
    lens[2] = 0
    Case(lens, counts, 70, 16, 2, 128, 16, seed=32).check()
    counts = np.array([70, 0, 65, 70, 0, 66, 68, 70])
    lens = counts + rng.integers(0, 1500, 8)
    Case(lens, counts, 70, 16, 2, 128, 32, seed=33).check()
    Case(lens, counts, 70, 48, 2, 64, 16, seed=34).check()


@pytest.mark.parametrize("shared", [False, True])
def test_ragged_batch(shared):
    rng = np.random.default_rng(1)
    counts = rng.integers(0, 24, 40)
    lens = counts + rng.integers(0, 900, 40)
    counts[[3, 9]] = 0  # nothing drafted, with and without a prefix
    lens[[3, 17]] = 0
    counts[17] = 0
    lens[21] = counts[21] = 23  # the tree is all there is
    Case(lens, counts, 23, 8, 2, 128, 16, seed=2, shared=shared).check()


def test_long_contexts_are_split():
    Case([9000, 40, 20011, 128], [5, 5, 3, 5], 5, 8, 2, 128, 16, seed=3).check()


def test_many_small_requests():
    rng = np.random.default_rng(4)
    counts = rng.integers(0, 4, 1300)
    Case(counts + rng.integers(0, 40, 1300), counts, 3, 2, 1, 64, 16, seed=5).check()


def test_arbitrary_masks_and_rows_that_see_nothing():
    """Masks that are no trees: random sets (later nodes too), full, empty.
    Bits of nodes a request does not have are ignored."""
    rng = np.random.default_rng(6)
    nodes = 40
    sees = rng.random((6, nodes, nodes)) < 0.4
    sees[1] = True
    sees[2] = False
    sees[3, ::2] = False
    c = Case([40, 12, 30, 33, 500, 140], [40, 12, 30, 33, 37, 0], nodes, 4, 2, 128, 16, seed=7, sees=sees)
    out = c.run()
    c.check(out)
    assert not out[2].any() and not out[3, ::2].any()  # L = n: nothing but the mask


def test_unattended_nodes_may_hold_anything():
    """NaN and infinities at positions a node does not attend to leave it as
    it is, bit for bit; nodes that attend to them take part as usual."""
    for d, value in ((128, float("nan")), (64, float("inf")), (128, float("-inf"))):
        c = Case([300, 28, 1000], None, 28, 8, 2, d, 16, seed=8)
        clean = c.run()
        rows = [(0, 5), (1, 0), (2, 27), (2, 13)]
        for b, node in rows:
            block, off = c.slot(b, int(c.l_ref[b]) - 28 + node)
            c.pool[block, 0, :, off] = value
            c.pool[block, 1, :, off, ::3] = value
        got = c.run()
        touched = np.zeros((3, 28), dtype=bool)
        for b, node in rows:
            touched[b] |= c.sees[b, :, node]
        touched = torch.as_tensor(touched).cuda()
        assert torch.equal(got[~touched], clean[~touched])
        assert not torch.isfinite(got[touched].float()).all(-1).any()


def test_infinite_values_reach_the_nodes_that_attend():
    """A value of +-inf under an attended position gives that infinity (both
    signs NaN), elsewhere the finite result stays."""
    c = Case([200, 77], None, 12, 4, 2, 128, 16, seed=9)
    c.sees[:, :, 0] = True
    for node, value in ((0, float("inf")), (3, float("-inf"))):
        block, off = c.slot(0, 200 - 12 + node)
        c.pool[block, 1, :, off, 7 + node] = value
    block, off = c.slot(1, 10)  # in the prefix: every node attends
    c.pool[block, 1, 0, off, 100] = float("-inf")
    got = c.run().float().cpu()
    assert (got[0, :, :, 7] == math.inf).all()
    sees3 = torch.as_tensor(c.sees[0, :, 3])
    assert (got[0, sees3][..., 10] == -math.inf).all() and torch.isfinite(got[0, ~sees3][..., 10]).all()
    assert (got[1, :, :2, 100] == -math.inf).all() and torch.isfinite(got[1, :, 2:, 100]).all()
    finite = torch.isfinite(got)
    assert finite.sum() == got.numel() - 12 * 4 - int(sees3.sum()) * 4 - 12 * 2


def test_large_logits():
    """One-hot softmaxes: scale 4 puts logits up to ~200 apart."""
    Case([500, 33, 1500], None, 20, 8, 2, 128, 16, seed=10, scale=4.0).check()
    Case([500, 33, 1500], None, 20, 8, 2, 64, 16, seed=11, scale=-2.0).check()


def test_growing_logits():
    """Every tile raises the running maximum."""
    c = Case([1024, 700], None, 8, 4, 1, 128, 16, seed=12)
    c.q[:] = 1.0
    for b in range(2):
        for p in range(int(c.l_ref[b])):
            block, off = c.slot(b, p)
            c.pool[block, 0, :, off] = p / 64.0
    c.scale = 0.05
    c.check()


def test_chain_matches_decode_multi_and_single_token_pa_decode():
    lens = [5, 300, 1200, 64]
    nodes = 4
    sees = np.broadcast_to(np.tril(np.ones((nodes, nodes), dtype=bool)), (4, nodes, nodes)).copy()
    c = Case(lens, None, nodes, 16, 4, 128, 16, seed=13, sees=sees)
    got = c.run().float()
    ws = torch.empty(pk.pa_decode_multi_workspace_size(4, nodes, 16, 4, 128, 16, 1200), dtype=torch.uint8, device="cuda")
    multi = torch.empty_like(c.q.cuda())
    pk.pa_decode_multi(multi, c.q.cuda(), c.pool.cuda(), torch.as_tensor(c.tables).cuda(),
                       torch.as_tensor(c.lens).cuda(), 1200, c.scale, ws)
    want, spread, size, logit = c.want()
    both = torch.as_tensor(2 * c.tolerance(want, spread, size, logit)).cuda()
    assert ((got - multi.float()).abs() <= both).all()


def test_bad_lengths_counts_and_blocks_are_flagged():
    base = dict(nodes=6, hq=4, hkv=2, d=64, bs=16, seed=14)
    c = Case([100, 40, 60], [6, 6, 6], **base)
    clean = c.run()
    pk.pa_device_error(clear=True)
    for bad in (7, -1, 41):
        c.counts[1] = bad
        got = c.run(max_len=100)
        assert pk.pa_device_error() == pk.PA_DEVERR_TREE
        assert not got[1].any() and torch.equal(got[[0, 2]], clean[[0, 2]])
    c.counts[1] = 6
    c.lens[1] = -3
    got = c.run()
    assert pk.pa_device_error() == pk.PA_DEVERR_SEQ_LEN and not got[1].any()
    c.lens[1] = 10 ** 9  # beyond the table row: clamped, and its blocks beyond the request's own are block 0
    got = c.run(max_len=1 << 30)
    assert pk.pa_device_error() & pk.PA_DEVERR_SEQ_LEN
    assert torch.equal(got[[0, 2]], clean[[0, 2]])
    c.lens[1] = 40
    for bad in (c.pool.shape[0], -1, 2 ** 31 - 1):
        c.tables[1, 0] = bad
        got = c.run()
        assert pk.pa_device_error() == pk.PA_DEVERR_BLOCK_ID
        zeros = Case([100, 40, 60], [6, 6, 6], **base)
        block, _ = zeros.slot(1, 0)
        zeros.pool[block] = 0
        want, spread, size, logit = zeros.want()
        assert (np.abs(bf16_to_f64(got) - want) <= zeros.tolerance(want, spread, size, logit)).all()
        assert torch.equal(got[[0, 2]], clean[[0, 2]])


@pytest.mark.parametrize("nodes,hq,d", [(12, 4, 128), (40, 8, 128), (40, 8, 64)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_infinite_value_of_vanishing_weight_in_a_cut_request(nodes, hq, d, value):
    """A request long enough to be cut between CTAs whose prefix outweighs the
    tree by more than fp32 can hold: an infinite value under a node still
    reaches the nodes that attend to it, and only them."""
    length = 20000
    c = Case([length], None, nodes, hq, 1, d, 16, seed=50, scale=1.0)
    c.q.fill_(2.0)
    block, off = c.slot(0, 5)
    c.pool[block, 0, 0, off] = 4.0  # a logit of 8 d; the others are within a few times 2 sqrt(d)
    clean = c.run()
    block, off = c.slot(0, length - nodes + 3)
    c.pool[block, 1, 0, off, 7] = value
    got = c.run()
    sees = torch.as_tensor(c.sees[0, :, 3])
    assert sees.any() and not sees.all()
    hit = got.cpu()[0, sees][..., 7]
    assert torch.isnan(hit).all() if math.isnan(value) else (hit == math.inf).all()
    got[0, sees.cuda(), :, 7] = clean[0, sees.cuda(), :, 7]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("nodes,hq,hkv,d", [(1024, 2, 2, 64), (300, 48, 1, 128), (513, 3, 1, 128)])
def test_the_largest_trees(nodes, hq, hkv, d):
    Case([nodes, nodes + 300], [nodes, nodes - 7], nodes, hq, hkv, d, 32, seed=40).check()


@pytest.mark.parametrize("d", [64, 128])
def test_one_position_one_node_one_head(d):
    Case([1], None, 1, 1, 1, d, 16, seed=41).check()
    Case([1, 0, 2], [1, 0, 1], 1, 3, 3, d, 16, seed=42).check()


def test_scale_zero_gives_the_mean_of_the_attended_values():
    Case([300, 40], None, 12, 8, 2, 128, 16, seed=43, scale=0.0).check()


def test_output_on_a_16_byte_boundary():
    c = Case([100, 40, 600], None, 6, 8, 2, 128, 16, seed=44)
    clean = c.run()
    buffer = torch.full((clean.numel() + 16,), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = buffer[8:-8].view(clean.shape)
    assert out.data_ptr() % 32 == 16
    assert torch.equal(c.run(out=out), clean)
    assert torch.isnan(buffer[:8]).all() and torch.isnan(buffer[-8:]).all()


def test_output_over_the_queries_is_refused():
    c = Case([100], None, 6, 8, 2, 128, 16, seed=45)
    q, mask = c.q.cuda(), pack(c.sees).cuda()
    ws = torch.empty(pk.pa_decode_tree_workspace_size(1, 6, 8, 2, 128, 16, 100), dtype=torch.uint8, device="cuda")
    with pytest.raises(pk.PaError, match="overlaps"):
        pk.pa_decode_tree(q, q, c.pool.cuda(), mask, torch.as_tensor(c.tables).cuda(), torch.as_tensor(c.lens).cuda(),
                          100, c.scale, ws)


def test_two_calls_at_once():
    """Two streams, a workspace each, many calls in flight on both."""
    cases = [Case([3000, 40, 777], None, 9, 16, 2, 128, 16, seed=46), Case([70, 4000], None, 30, 16, 2, 128, 16, seed=47)]
    clean = [c.run() for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    args, outs = [], []
    for c in cases:
        b, nodes, hq, d = c.q.shape
        max_len = int(c.lens.max())
        need = pk.pa_decode_tree_workspace_size(b, nodes, hq, 2, d, 16, max_len)
        args.append((c.q.cuda(), c.pool.cuda(), pack(c.sees).cuda(), torch.as_tensor(c.tables).cuda(),
                     torch.as_tensor(c.lens).cuda(), max_len, c.scale,
                     torch.empty(need, dtype=torch.uint8, device="cuda")))
        outs.append([torch.empty_like(args[-1][0]) for _ in range(10)])
    torch.cuda.synchronize()
    for i in range(10):
        for j in range(2):
            pk.pa_decode_tree(outs[j][i], *args[j], stream=streams[j])
    torch.cuda.synchronize()
    for j in range(2):
        assert all(torch.equal(o, clean[j]) for o in outs[j])
    assert pk.pa_device_error() == 0


def test_pinned_output_and_refused_pageable_output():
    c = Case([100, 40, 60, 300], None, 6, 8, 2, 128, 16, seed=15)
    clean = c.run()
    pinned = torch.full(c.q.shape, float("nan"), dtype=torch.bfloat16).pin_memory()
    assert torch.equal(c.run(out=pinned).cuda(), clean)
    with pytest.raises(TypeError):
        c.run(out=torch.empty(c.q.shape, dtype=torch.bfloat16))


def test_results_do_not_depend_on_what_ran_before_or_the_stream():
    """Same bits again: with a used workspace, on another stream, after a
    call of other sizes in the same workspace, and replayed from two graphs
    that share it."""
    c = Case([2000, 40, 777, 0, 31], [9, 9, 9, 0, 9], 9, 16, 2, 128, 16, seed=16)
    other = Case([70, 4000], None, 30, 16, 2, 128, 16, seed=17)
    need = max(pk.pa_decode_tree_workspace_size(5, 9, 16, 2, 128, 16, 2000),
               pk.pa_decode_tree_workspace_size(2, 30, 16, 2, 128, 16, 4000))
    ws = torch.full((need,), 0x7f, dtype=torch.uint8, device="cuda")
    pools = c.pool.cuda(), other.pool.cuda()
    first, second = c.run(pools[0], workspace=ws), other.run(pools[1], workspace=ws)
    c.check(first)
    other.check(second)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(c.run(pools[0], workspace=ws), first)
    assert torch.equal(other.run(pools[1], workspace=ws, stream=side), second)
    graphs, outs = [], []
    for case, pool in ((c, pools[0]), (other, pools[1])):
        q, mask = case.q.cuda(), pack(case.sees).cuda()
        tables, lens = torch.as_tensor(case.tables).cuda(), torch.as_tensor(case.lens).cuda()
        counts = torch.as_tensor(case.counts, dtype=torch.int32).cuda()
        out = torch.empty_like(q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pk.pa_decode_tree(out, q, pool, mask, tables, lens, int(case.lens.max()), case.scale, ws, tree_lens=counts)
        graphs.append((g, q, mask, tables, lens, counts))
        outs.append(out)
    for _ in range(3):
        for g, *_ in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first) and torch.equal(outs[1], second)


def test_lengths_that_change_under_a_captured_call():
    """A captured call serves later lengths up to max_seq_len."""
    c = Case([700, 300], [8, 8], 8, 8, 2, 128, 16, seed=18)
    q, mask, pool = c.q.cuda(), pack(c.sees).cuda(), c.pool.cuda()
    tables, lens = torch.as_tensor(c.tables).cuda(), torch.as_tensor(c.lens).cuda()
    counts = torch.as_tensor(c.counts, dtype=torch.int32).cuda()
    ws = torch.empty(pk.pa_decode_tree_workspace_size(2, 8, 8, 2, 128, 16, 5000), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pk.pa_decode_tree(out, q, pool, mask, tables, lens, 5000, c.scale, ws, tree_lens=counts)
    for new_lens, new_counts in (([700, 300], [8, 8]), ([90, 8], [3, 8]), ([0, 299], [0, 1])):
        lens.copy_(torch.tensor(new_lens, dtype=torch.int32))
        counts.copy_(torch.tensor(new_counts, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        c.l_ref, c.counts = np.array(new_lens), new_counts
        c.check(out)


def test_offsets_beyond_two_to_the_31():
    """A pool of more than 2^31 elements whose last blocks are used."""
    hkv, bs, d, nodes = 8, 16, 128, 5
    nb = (1 << 31) // (2 * hkv * bs * d) + 40
    pool = torch.zeros((nb, 2, hkv, bs, d), dtype=torch.bfloat16, device="cuda")
    small = Case([200, 90], None, nodes, 16, hkv, d, bs, seed=19)
    n = small.pool.shape[0]
    pool[-n:] = small.pool.cuda()
    want = small.run()
    small.tables += nb - n
    assert torch.equal(small.run(pool), want)


@pytest.mark.parametrize("workload,nodes", [("llama8b", 16), ("beam", 64)])
def test_full_size_heads(workload, nodes):
    """The benchmark's shapes on a few requests, group 4 and 8."""
    s = workloads.SHAPES[workload]
    rng = np.random.default_rng(20)
    lens = rng.integers(512, 4096, 3)
    Case(lens, None, nodes, s.num_q_heads, s.num_kv_heads, s.head_dim, s.block_size, seed=21).check()


@pytest.mark.parametrize("nodes,hq,d,tiles", [(8, 8, 128, 2), (8, 8, 64, 2), (8, 8, 128, 3), (60, 8, 128, 2), (60, 8, 64, 3)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_a_value_that_is_not_finite_in_an_outweighed_prefix_position(nodes, hq, d, tiles, value):
    """Every node attends to the prefix, so a value there that is not finite
    shows in its column of every row, however little its weight: in each tile,
    with the dominating key in each other one.  As many equal items per CTA, of
    one row tile (8 nodes) or of two (60), so that none of them is cut."""
    hkv = 2
    batch = torch.cuda.get_device_properties(0).multi_processor_count
    length = 128 * tiles
    c = Case([length] * batch, None, nodes, hq, hkv, d, 16, seed=60, scale=1.0)
    c.q.fill_(2.0)
    last = length - nodes - 1
    where = [5, 131, 260][:tiles]
    pairs = [(i, j) for i in range(tiles) for j in range(tiles) if i != j]  # value's tile, key's tile
    for b in range(batch):
        block, off = c.slot(b, where[pairs[b % len(pairs)][1]])
        c.pool[block, 0, :, off] = 4.0  # a logit of 8 d; the others are within a few times 2 sqrt(d)
    clean = c.run()
    assert torch.isfinite(clean).all() and max(where) < last
    for b in range(batch):
        block, off = c.slot(b, where[pairs[b % len(pairs)][0]] + 1)
        c.pool[block, 1, :, off, 7] = value
    got = c.run()
    hit = got[..., 7]
    assert torch.isnan(hit).all() if math.isnan(value) else not torch.isfinite(hit).any()
    got[..., 7] = clean[..., 7]
    assert torch.equal(got, clean)
    assert pk.pa_device_error() == 0


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_such_a_value_in_a_request_that_is_cut(d, value):
    """The same in one long request, a few tiles per CTA: join and merge."""
    nodes, length = 8, 60000
    c = Case([length], None, nodes, 8, 1, d, 16, seed=61, scale=1.0)
    c.q.fill_(2.0)
    block, off = c.slot(0, 128 * 7 + 3)
    c.pool[block, 0, :, off] = 4.0
    clean = c.run()
    for tile in (0, 1, 4, 5, 6, 7, 8, 9, 300, 301):
        block, off = c.slot(0, 128 * tile + 50)
        was = c.pool[block, 1, 0, off, 9].clone()
        c.pool[block, 1, 0, off, 9] = value
        got = c.run()
        c.pool[block, 1, 0, off, 9] = was
        hit = got[..., 9]
        assert torch.isnan(hit).all() if math.isnan(value) else not torch.isfinite(hit).any(), tile
        got[..., 9] = clean[..., 9]
        assert torch.equal(got, clean)
    assert pk.pa_device_error() == 0


@pytest.mark.parametrize("lens,counts", [([0, 0, 0], None), ([0, 0], [0, 0]), ([50, 0, 700], [0, 0, 0])])
def test_no_request_has_a_node(lens, counts):
    """Nothing to do at sizes of several row-tile pairs: all rows are zeroed."""
    out = Case(lens, counts, 300, 4, 2, 128, 16, seed=62).run()
    assert not out.any() and pk.pa_device_error() == 0


@pytest.mark.parametrize("hq,hkv,d,bs", [(16, 4, 128, 16), (4, 4, 64, 32), (32, 2, 128, 16)])
def test_one_node_matches_single_token_pa_decode(hq, hkv, d, bs):
    """A tree of one node is the newest token: both answers lie within the
    roundings of the exact one that each call makes."""
    lens = [1, 5, 300, 1200, 64, 129]
    c = Case(lens, None, 1, hq, hkv, d, bs, seed=63)
    got = c.run().float()
    need, _ = pk.pa_decode_workspace_size(len(lens), hq, hkv, d, bs, 1200)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    single = torch.empty((len(lens), hq, d), dtype=torch.bfloat16, device="cuda")
    pk.pa_decode(single, c.q[:, 0].contiguous().cuda(), c.pool.cuda(), torch.as_tensor(c.tables).cuda(),
                 torch.as_tensor(c.lens).cuda(), 1200, c.scale, workspace=ws)
    want, spread, size, logit = c.want()
    both = torch.as_tensor(2 * c.tolerance(want, spread, size, logit)).cuda()
    assert ((got - single.float()[:, None]).abs() <= both).all()
    c.check(got.bfloat16())
