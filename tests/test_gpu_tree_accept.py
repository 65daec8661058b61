"""pa_tree_accept against the oracle, bit for bit over the whole pool."""

import numpy as np
import pytest
import torch

import paged_kv_cache_354_b200 as pk
import workloads
from oracle import tree_speculation as ots
from tests.gpu_helpers import build_tables

pytestmark = pytest.mark.gpu


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def make(lens, hkv, d, bs, seed):
    rng = np.random.default_rng(seed)
    nb = sum(-(-int(n) // bs) for n in lens) + 2
    t_ref, l_ref, tables, lens32, _ = build_tables(lens, bs, nb, rng.permutation(nb))
    pool = workloads.bf16_normal((nb, 2, hkv, bs, d), seed=seed)
    return pool, t_ref, torch.as_tensor(tables).cuda(), torch.as_tensor(lens32).cuda()


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


@pytest.mark.parametrize("batch,nodes,most,hkv,d,bs", [(1, 1, 1, 1, 64, 16), (1, 40, 40, 2, 128, 16), (7, 16, 5, 8, 128, 16),
                                                       (33, 9, 9, 4, 64, 32), (300, 64, 17, 2, 64, 16), (3, 20, 20, 3, 8, 5),
                                                       (2, 300, 290, 1, 128, 16)])
def test_matches_the_oracle(batch, nodes, most, hkv, d, bs):
    rng = np.random.default_rng(nodes)
    counts = rng.integers(0, nodes, batch, endpoint=True)
    counts[0] = nodes
    lens = counts + rng.integers(0, 70, batch)
    lens = np.maximum(lens, 1)
    accepted = np.array([rng.integers(0, min(c, most), endpoint=True) for c in counts])
    accepted[0] = min(nodes, most)
    path = np.full((batch, most), -9)
    for b in range(batch):
        path[b, : accepted[b]] = np.sort(rng.permutation(int(counts[b]))[: accepted[b]])
    pool, t_ref, tables, g_lens = make(lens, hkv, d, bs, nodes)
    want, want_lens = ots.tree_accept(bits(pool).copy(), path, accepted, counts, t_ref, lens)
    got, out = pool.cuda(), torch.full((batch,), -5, dtype=torch.int32, device="cuda")
    pk.pa_tree_accept(got, i32(path), i32(accepted), tables, g_lens, i32(counts), seq_lens_out=out)
    assert np.array_equal(bits(got), want) and out.tolist() == want_lens
    # without new lengths, then with the lengths in place
    again = pool.cuda()
    pk.pa_tree_accept(again, i32(path), i32(accepted), tables, g_lens, i32(counts))
    assert torch.equal(again.view(torch.int16), got.view(torch.int16)) and g_lens.tolist() == list(lens)
    again = pool.cuda()
    pk.pa_tree_accept(again, i32(path), i32(accepted), tables, g_lens, i32(counts), seq_lens_out=g_lens)
    assert torch.equal(again.view(torch.int16), got.view(torch.int16)) and g_lens.tolist() == want_lens
    assert pk.pa_device_error() == 0


def test_one_count_for_all_and_empty_requests():
    pool, t_ref, tables, lens = make([30, 0, 8], 2, 64, 16, 3)
    want, _ = ots.tree_accept(bits(pool).copy(), [[1, 3, 7], [0, 0, 0], [0, 1, 2]], [3, 0, 2], [8, 0, 8], t_ref, [30, 0, 8])
    got = pool.cuda()
    pk.pa_tree_accept(got, i32([[1, 3, 7], [0, 0, 0], [0, 1, 2]]), i32([3, 0, 2]), tables, lens, None, num_nodes=8,
                      seq_lens_out=lens)
    assert np.array_equal(bits(got), want) and lens.tolist() == [25, 0, 2]
    assert pk.pa_device_error() == 0
    with pytest.raises(ValueError):
        pk.pa_tree_accept(got, i32([[1]] * 3), i32([0] * 3), tables, lens, None)


@pytest.mark.parametrize("path,accepted,count,length", [
    ([3, 3], 2, 6, 40), ([4, 2], 2, 6, 40), ([-1, 2], 2, 6, 40), ([0, 6], 2, 6, 40), ([0, 1], 3, 6, 40),
    ([0, 1], -1, 6, 40), ([0, 1], 2, 1, 40), ([0, 1], 2, 41, 40), ([0, 1], 2, -1, 40), ([0, 1], 2, 6, -1),
    ([0, 1], 2, 6, 10 ** 9)])
def test_bad_paths_are_flagged_and_nothing_moves(path, accepted, count, length):
    pool, _, tables, lens = make([40, 40], 2, 64, 16, 4)
    lens[1] = length
    got = pool.cuda()
    out = torch.zeros(2, dtype=torch.int32, device="cuda")
    pk.pa_device_error(clear=True)
    pk.pa_tree_accept(got, i32([[2, 4], path]), i32([0, accepted]), tables, lens, i32([6, count]), seq_lens_out=out)
    assert pk.pa_device_error() == pk.PA_DEVERR_TREE
    assert torch.equal(got.cpu().view(torch.int16), pool.view(torch.int16)) and out.tolist() == [34, length]


@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_bad_blocks_are_flagged_and_nothing_moves(bad):
    pool, _, tables, lens = make([40, 40], 2, 64, 16, 5)
    tables[1, 2] = bad
    got = pool.cuda()
    pk.pa_device_error(clear=True)
    pk.pa_tree_accept(got, i32([[0], [3]]), i32([1, 1]), tables, lens, i32([6, 6]))
    assert pk.pa_device_error() == pk.PA_DEVERR_BLOCK_ID
    assert torch.equal(got.cpu().view(torch.int16), pool.view(torch.int16))


def test_offsets_beyond_two_to_the_31():
    """Requests in the last blocks of a pool of more than 2^31 elements."""
    pool, _, tables, lens = make([40, 90, 33], 8, 128, 16, 5)
    n = pool.shape[0]
    path, accepted, counts = i32([[1, 3, 8], [0, 2, 4], [5, 6, 7]]), i32([3, 3, 2]), i32([9, 9, 9])
    small = pool.cuda()
    pk.pa_tree_accept(small, path, accepted, tables, lens, counts)
    blocks = (1 << 31) // (2 * 8 * 16 * 128) + n + 1
    big = torch.zeros((blocks,) + tuple(pool.shape[1:]), dtype=torch.bfloat16, device="cuda")
    big[-n:] = pool.cuda()
    pk.pa_tree_accept(big, path, accepted, tables + (blocks - n), lens, counts)
    assert np.array_equal(bits(big[-n:]), bits(small)) and not np.array_equal(bits(small), bits(pool))
    assert not big[:-n].view(torch.int32).any()
    assert pk.pa_device_error() == 0
