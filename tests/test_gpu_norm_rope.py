"""pa_norm_rope_and_cache against the fp64 oracle.

Tolerance per element: the one rounding to bf16, 2^-8 |want|, plus 2^-16
(|y_a cos| + |y_b sin|) for the fp32 arithmetic -- a sum of up to 128 squares
(relative error up to 64 * 2^-23 in any order, halved by the square root), the
reciprocal root (2 ulp), two products and the rotation's two products and sum,
in all below 80 roundings of 2^-24 each way, under 2^-16 -- relative to the
summands of the rotation, which can cancel."""

import numpy as np
import pytest
import torch

import paged_kv_cache_354_b200 as pk
import workloads
from oracle import tree_speculation as ots
from tests.gpu_helpers import bf16_to_f64

pytestmark = pytest.mark.gpu

EPS = 1e-5


def table(most, rot, seed=0):
    angle = np.random.default_rng(seed).uniform(0, 1000, (most, rot // 2))
    return torch.as_tensor(np.concatenate([np.cos(angle), np.sin(angle)], 1)).float()


def make(n, hq, hkv, d, bs, seed, slab=False, most=500):
    rng = np.random.default_rng(seed)
    if slab:
        x = workloads.bf16_normal((n, (hq + 2 * hkv) * d + 24), seed=seed).cuda()
        q, k, v = (x[:, a * d:(a + h) * d].unflatten(1, (h, d))
                   for a, h in ((0, hq), (hq, hkv), (hq + hkv, hkv)))
    else:
        q, k, v = (workloads.bf16_normal((n, h, d), seed=seed + i).cuda() for i, h in enumerate((hq, hkv, hkv)))
    blocks = -(-n // bs) + 2
    slots = rng.permutation(blocks * bs)[:n]
    pos = rng.integers(0, most, n)
    if n > 2:
        slots[1] = -1  # computed, not cached
        pos[2] = -4  # padding
    pool = torch.full((blocks, 2, hkv, bs, d), 7.5, dtype=torch.bfloat16, device="cuda")
    weights = [(1 + 0.2 * workloads.bf16_normal((d,), seed=seed + 9 + i)).bfloat16().cuda() for i in range(2)]
    return q, k, v, pool, slots, pos, weights


def close(got, want, bound):
    got = bf16_to_f64(got)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -16 * bound).all()


def check(q_out, pool, k_out, q, k, v, slots, pos, weights, cs, interleaved):
    cs64 = None if cs is None else cs.double().cpu().numpy()
    w = [None if x is None else bf16_to_f64(x) for x in weights]
    want_q, bound_q = ots.norm_rope(bf16_to_f64(q), w[0], EPS, cs64, pos, interleaved)
    want_k, bound_k = ots.norm_rope(bf16_to_f64(k), w[1], EPS, cs64, pos, interleaved)
    close(q_out, want_q, bound_q)
    if k_out is not None:
        close(k_out, want_k, bound_k)
    if pool is None:
        return
    bs = pool.shape[3]
    live = (slots >= 0) & (pos >= 0)
    block, offset = torch.as_tensor(slots[live] // bs).cuda(), torch.as_tensor(slots[live] % bs).cuda()
    close(pool[block, 0, :, offset], want_k[live], bound_k[live])
    assert torch.equal(pool[block, 1, :, offset], v[torch.as_tensor(live).cuda()])
    rest = pool.clone()  # every other row is as it was
    rest[block, :, :, offset] = 7.5
    assert (rest == 7.5).all()


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("n,hq,hkv,d,rot,interleaved,slab", [
    (1, 4, 4, 64, 64, False, False), (1, 32, 8, 128, 128, False, True), (3, 5, 1, 128, 64, False, True),
    (17, 8, 2, 64, 32, True, True), (33, 3, 3, 128, 128, True, False), (131, 32, 8, 128, 128, False, True),
    (9, 2, 1, 128, 16, False, False), (9, 2, 2, 64, 16, True, False), (5, 6, 2, 128, 96, False, True),
    (5, 6, 2, 128, 112, True, True), (2, 7, 7, 64, 48, False, False), (1030, 4, 1, 64, 64, False, True)])
def test_matches_the_oracle(norm, n, hq, hkv, d, rot, interleaved, slab):
    q, k, v, pool, slots, pos, weights = make(n, hq, hkv, d, 16, n + d + rot, slab)
    if not norm:
        weights = [None, None]
    cs = table(500, rot).cuda()
    q_out = torch.full((n, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((n, hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    pk.pa_norm_rope_and_cache(q_out, q, k, v, pool, torch.as_tensor(slots).cuda(),
                              torch.as_tensor(pos).int().cuda(), cs, *weights, eps=EPS, interleaved=interleaved,
                              k_out=k_out)
    check(q_out, pool, k_out, q, k, v, slots, pos, weights, cs, interleaved)
    assert pk.pa_device_error() == 0


def test_norm_alone_and_no_cache():
    q, k, v, _, slots, pos, weights = make(19, 6, 2, 128, 32, 5, True)
    q_out, k_out = torch.empty_like(q.contiguous()), torch.empty_like(k.contiguous())
    pk.pa_norm_rope_and_cache(q_out, q, k, None, None, None, None, None, *weights, eps=EPS, k_out=k_out)
    check(q_out, None, k_out, q, k, v, slots, np.zeros(19, dtype=int), weights, None, False)


@pytest.mark.parametrize("which", [0, 1])
def test_only_queries_or_only_keys_have_a_weight(which):
    q, k, v, pool, slots, pos, weights = make(21, 4, 2, 64, 16, 6)
    weights[which] = None
    cs = table(500, 64).cuda()
    q_out = torch.empty_like(q)
    pk.pa_norm_rope_and_cache(q_out, q, k, v, pool, torch.as_tensor(slots).cuda(), torch.as_tensor(pos).int().cuda(),
                              cs, *weights, eps=EPS)
    check(q_out, pool, None, q, k, v, slots, pos, weights, cs, False)


def test_in_place():
    q, k, v, pool, slots, pos, weights = make(40, 8, 2, 128, 16, 7, slab=True)
    cs = table(500, 128).cuda()
    was_q, was_k = q.clone(), k.clone()
    pk.pa_norm_rope_and_cache(q, q, k, v, pool, torch.as_tensor(slots).cuda(), torch.as_tensor(pos).int().cuda(), cs,
                              *weights, eps=EPS, k_out=k)
    check(q, pool, k, was_q, was_k, v, slots, pos, weights, cs, False)


def test_bad_positions_and_slots_are_flagged_and_skipped():
    q, k, v, pool, slots, pos, weights = make(12, 4, 2, 64, 16, 8)
    cs = table(500, 64).cuda()
    pos[5], slots[7] = 500, pool.shape[0] * 16
    q_out = torch.empty_like(q)
    pk.pa_device_error(clear=True)
    pk.pa_norm_rope_and_cache(q_out, q, k, v, pool, torch.as_tensor(slots).cuda(), torch.as_tensor(pos).int().cuda(),
                              cs, *weights, eps=EPS)
    assert pk.pa_device_error() == pk.PA_DEVERR_POSITION | pk.PA_DEVERR_SLOT
    pos[5], slots[7] = -1, -1
    check(q_out, pool, None, q, k, v, slots, pos, weights, cs, False)


def test_large_and_tiny_rows():
    """Rows of 1e4 and 1e-4 norm alike, a row of zeros stays zero."""
    q, k, v, pool, slots, pos, weights = make(4, 2, 1, 128, 16, 9)
    slots[:], pos[:] = range(4), range(4)
    for i, f in enumerate((1e4, 1e-4, 0.0, 1.0)):
        q[i] *= f
        k[i] *= f
    cs = table(500, 128).cuda()
    q_out = torch.empty_like(q)
    pk.pa_norm_rope_and_cache(q_out, q, k, v, pool, torch.as_tensor(slots).cuda(), torch.as_tensor(pos).int().cuda(),
                              cs, *weights, eps=EPS)
    check(q_out, pool, None, q, k, v, slots, pos, weights, cs, False)
    assert not q_out[2].any()


def test_strides_that_do_not_fit_are_refused():
    x = torch.zeros((4, 64, 8), dtype=torch.bfloat16, device="cuda").transpose(1, 2)  # heads interleaved
    y = torch.zeros((4, 8, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="heads"):
        pk.pa_norm_rope_and_cache(y, x, y, y, None, None, None, None, k_out=y)
    odd = torch.zeros((4, 8 * 64 + 4), dtype=torch.bfloat16, device="cuda")[:, :512].unflatten(1, (8, 64))
    with pytest.raises(pk.PaError):
        pk.pa_norm_rope_and_cache(y, odd, y, y, None, None, None, None, k_out=y)


def test_queries_alone_and_keys_alone():
    """No KV heads, or no query heads: the other side is written as usual."""
    q, k, v, pool, slots, pos, weights = make(23, 6, 2, 64, 16, 10)
    cs = table(500, 64).cuda()
    none = torch.empty((23, 0, 64), dtype=torch.bfloat16, device="cuda")
    g_slots, g_pos = torch.as_tensor(slots).cuda(), torch.as_tensor(pos).int().cuda()
    q_out = torch.empty_like(q)
    pk.pa_norm_rope_and_cache(q_out, q, none, None, None, None, g_pos, cs, q_weight=weights[0], eps=EPS, k_out=none)
    pk.pa_norm_rope_and_cache(none, none, k, v, pool, g_slots, g_pos, cs, k_weight=weights[1], eps=EPS)
    check(q_out, pool, None, q, k, v, slots, pos, weights, cs, False)
    assert pk.pa_device_error() == 0


def test_many_heads_and_many_tokens():
    """More rows per token than one thread takes at once, more tokens than
    the resident blocks take in one round."""
    q, k, v, pool, slots, pos, weights = make(3000, 128, 16, 64, 32, 11, slab=True)
    cs = table(500, 64).cuda()
    q_out = torch.empty((3000, 128, 64), dtype=torch.bfloat16, device="cuda")
    pk.pa_norm_rope_and_cache(q_out, q, k, v, pool, torch.as_tensor(slots).cuda(), torch.as_tensor(pos).int().cuda(),
                              cs, *weights, eps=EPS)
    check(q_out, pool, None, q, k, v, slots, pos, weights, cs, False)


def test_offsets_beyond_two_to_the_31():
    """Slots in the last blocks of a pool of more than 2^31 elements."""
    q, k, v, pool, slots, pos, weights = make(40, 8, 8, 128, 16, 12)
    cs = table(500, 128).cuda()
    n = pool.shape[0]
    blocks = (1 << 31) // (2 * 8 * 16 * 128) + n + 1
    big = torch.zeros((blocks,) + pool.shape[1:], dtype=torch.bfloat16, device="cuda")
    big[-n:] = 7.5
    q_out, q_out2 = torch.empty_like(q), torch.empty_like(q)
    g_slots, g_pos = torch.as_tensor(slots).cuda(), torch.as_tensor(pos).int().cuda()
    pk.pa_norm_rope_and_cache(q_out, q, k, v, pool, g_slots, g_pos, cs, *weights, eps=EPS)
    far = torch.where(g_slots < 0, g_slots, g_slots + (blocks - n) * 16)
    pk.pa_norm_rope_and_cache(q_out2, q, k, v, big, far, g_pos, cs, *weights, eps=EPS)
    assert torch.equal(big[-n:], pool) and torch.equal(q_out, q_out2)
    assert not big[:-n].view(torch.int32).any()
    assert pk.pa_device_error() == 0


def test_two_streams_at_once():
    q, k, v, pool, slots, pos, weights = make(700, 8, 2, 128, 16, 13)
    cs = table(500, 128).cuda()
    g_slots, g_pos = torch.as_tensor(slots).cuda(), torch.as_tensor(pos).int().cuda()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    pools, outs = [pool.clone(), pool.clone()], [torch.empty_like(q), torch.empty_like(q)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            pk.pa_norm_rope_and_cache(outs[i], q, k, v, pools[i], g_slots, g_pos, cs, *weights, eps=EPS,
                                      stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        check(outs[i], pools[i], None, q, k, v, slots, pos, weights, cs, False)


def test_outputs_between_the_inputs_of_one_slab():
    """Results beside their inputs in one slab, in place, and one token
    directly behind the other: nothing is shared, so nothing is refused."""
    n, hq, hkv, d = 21, 4, 2, 64
    rng = np.random.default_rng(14)
    pool = torch.full((4, 2, hkv, 16, d), 7.5, dtype=torch.bfloat16, device="cuda")
    weights = [(1 + 0.2 * workloads.bf16_normal((d,), seed=i)).bfloat16().cuda() for i in range(2)]
    slots, pos = rng.permutation(64)[:n], rng.integers(0, 500, n)
    cs = table(500, d).cuda()
    heads = (hq, hkv, hkv, hq, hkv)  # q, k, v, q_out, k_out
    slab = workloads.bf16_normal((n, sum(heads) * d), seed=15).cuda()
    q, k, v, q_out, k_out = (x.unflatten(1, (-1, d)) for x in slab.split([h * d for h in heads], 1))
    was = q.clone(), k.clone(), v.clone()
    g_slots, g_pos = torch.as_tensor(slots).cuda(), torch.as_tensor(pos).int().cuda()
    pk.pa_norm_rope_and_cache(q_out, q, k, v, pool, g_slots, g_pos, cs, *weights, eps=EPS, k_out=k_out)
    check(q_out, pool, k_out, *was, slots, pos, weights, cs, False)
    assert all(torch.equal(x, w) for x, w in zip((q, k, v), was))
    pool.fill_(7.5)
    pk.pa_norm_rope_and_cache(q, q, k, v, pool, g_slots, g_pos, cs, *weights, eps=EPS, k_out=k)
    check(q, pool, k, *was, slots, pos, weights, cs, False)
    # contiguous tensors one behind the other in a single buffer
    sizes = [n * h * d for h in (hq, hkv, hkv, hq, hkv)] + [pool.numel()]
    flat = workloads.bf16_normal((sum(sizes),), seed=16).cuda()
    parts = flat.split(sizes)
    q, k, v, q_out, k_out = (x.view(n, -1, d) for x in parts[:5])
    pool = parts[5].view(pool.shape).fill_(7.5)
    was = q.clone(), k.clone(), v.clone()
    pk.pa_norm_rope_and_cache(q_out, q, k, v, pool, g_slots, g_pos, cs, *weights, eps=EPS, k_out=k_out)
    check(q_out, pool, k_out, *was, slots, pos, weights, cs, False)
    assert all(torch.equal(x, w) for x, w in zip((q, k, v), was))


def test_an_output_over_another_tokens_input_is_refused():
    q, k, v, pool, slots, pos, weights = make(12, 4, 2, 64, 16, 17)
    buffer = torch.zeros((13, 4, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pk.PaError, match="overlap"):
        pk.pa_norm_rope_and_cache(buffer[1:], buffer[:-1], k, v, pool, torch.as_tensor(slots).cuda(),
                                  torch.as_tensor(pos).int().cuda(), table(500, 64).cuda(), *weights, eps=EPS)
