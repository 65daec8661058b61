"""The tree-speculation oracle against other statements of the same things:
the host allocator (plan), causal multi-token decode (tree), complex products
(rotation), and array indexing (accept).  No GPU needed."""

import numpy as np
import pytest

import paged_kv_cache_354_b200 as pk
from oracle import paged_attention as opa
from oracle import tree_speculation as ots


@pytest.mark.parametrize("seed,bs", [(0, 16), (1, 5), (2, 1)])
def test_plan_matches_the_host_allocator(seed, bs):
    """Ended requests first, then the appends: the calls of the C++ allocator
    in that order give the same blocks, slots and free list."""
    rng = np.random.default_rng(seed)
    nb, batch, width = 90, 7, 40
    order = rng.permutation(nb)
    alloc = pk.PaAlloc(nb, bs, order)
    for i in range(batch):
        alloc.add_seq(i)
    tables, held = [[0] * width for _ in range(batch)], [0] * batch
    free, lens = list(order[::-1]), [0] * batch
    for _ in range(40):
        new = [int(x) for x in rng.integers(0, 2 * bs + 2, batch)]
        for b in range(batch):
            if rng.random() < 0.15 or lens[b] + new[b] > width * bs:
                new[b] = -1
        got = ots.plan_append(tables, held, free, lens, new, bs, width)
        if got is None:  # out of blocks: end one request instead
            new = [-1 if b == 0 else 0 for b in range(batch)]
            got = ots.plan_append(tables, held, free, lens, new, bs, width)
        for b, c in enumerate(new):
            if c < 0:
                alloc.free_seq(b)
                alloc.add_seq(b)
        slots = [alloc.append(b, c)[0] if c > 0 else [] for b, c in enumerate(new)]
        tables, held, free, lens, mine, positions = got
        assert mine == slots
        assert [tables[b][: held[b]] for b in range(batch)] == [alloc.block_table(b) for b in range(batch)]
        assert free[::-1] == alloc.free_list()
        assert lens == [alloc.seq_len(b) for b in range(batch)]
        assert all(p == list(range(lens[b] - len(p), lens[b])) for b, p in enumerate(positions))


def test_plan_refuses_as_a_whole():
    tables, held, free, lens = [[3, 0], [1, 0]], [1, 1], [0, 2], [4, 3]
    assert ots.plan_append(tables, held, free, lens, [3, 4], 4, 2) is not None
    assert ots.plan_append(tables, held, [2], lens, [3, 4], 4, 2) is None
    assert ots.plan_append(tables, held, free, lens, [5, 0], 4, 2) is None  # beyond the table row


def test_chain_is_causal_decode():
    rng = np.random.default_rng(3)
    lens, nodes, bs = [9, 4, 33, 5], 4, 4
    tables = rng.permutation(40).reshape(4, 10)
    pool = rng.standard_normal((40, 2, 2, bs, 8))
    q = rng.standard_normal((4, nodes, 6, 8))
    chain = np.broadcast_to(np.tril(np.ones((nodes, nodes), dtype=bool)), (4, nodes, nodes))
    got, spread, size, logit = ots.decode_tree(q, pool, chain, tables, lens, [nodes] * 4, 0.3)
    assert np.allclose(got, opa.decode_multi(q, pool, tables, lens, 0.3), atol=1e-12)
    assert (np.abs(got) <= size + 1e-12).all() and (spread >= 0).all() and (logit > 0).all()


def test_unattended_positions_have_no_effect():
    rng = np.random.default_rng(4)
    tables = np.arange(8).reshape(1, 8)
    pool = rng.standard_normal((8, 2, 1, 4, 8))
    q = rng.standard_normal((1, 3, 2, 8))
    sees = np.array([[[1, 0, 0], [0, 1, 0], [1, 0, 1]]], dtype=bool)
    want = ots.decode_tree(q, pool, sees, tables, [13], [3], 0.4)[0]
    pool[2, :, :, 3] = np.nan  # node 1 sits at position 11
    got = ots.decode_tree(q, pool, sees, tables, [13], [3], 0.4)[0]
    assert np.array_equal(got[:, [0, 2]], want[:, [0, 2]]) and np.isnan(got[:, 1]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((4, 3, 8))
    angle = rng.uniform(0, 6, (10, 3))
    cos_sin = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    pos = np.array([3, 9, -1, 0])
    y, bound = ots.norm_rope(x, None, 0.0, cos_sin, pos, interleaved)
    a, b = (slice(0, 6, 2), slice(1, 6, 2)) if interleaved else (slice(0, 3), slice(3, 6))
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * angle[pos.clip(0)])[:, None]
    real = pos >= 0
    assert np.allclose(y[real][..., a], z.real[real]) and np.allclose(y[real][..., b], z.imag[real])
    assert np.array_equal(y[real][..., 6:], x[real][..., 6:]) and not y[2].any()
    assert (np.abs(y[real]) <= bound[real] + 1e-12).all()


def test_norm_gives_unit_mean_square():
    x = np.random.default_rng(6).standard_normal((5, 2, 16)) * 7
    y, _ = ots.norm_rope(x, np.full(16, 2.0), 0.0, None, None, False)
    assert np.allclose((y ** 2).mean(-1), 4.0)


def test_accept_is_a_gather():
    rng = np.random.default_rng(7)
    pool = rng.standard_normal((6, 2, 2, 4, 3))
    tables = np.array([[5, 1, 3], [0, 2, 4]])
    flat = lambda p, b: p[tables[b]].transpose(0, 3, 1, 2, 4).reshape(12, 2, 2, 3)  # noqa: E731
    before = pool.copy()
    got, lens = ots.tree_accept(pool, [[1, 2, 5], [0, 3, 9]], [3, 2], [6, 4], tables, [11, 9])
    assert lens == [8, 7]
    assert np.array_equal(flat(got, 0)[5:8], flat(before, 0)[[6, 7, 10]])
    assert np.array_equal(flat(got, 0)[8:], flat(before, 0)[8:])
    assert np.array_equal(flat(got, 1)[5:7], flat(before, 1)[[5, 8]])
