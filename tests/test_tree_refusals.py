"""The tree-speculation calls report bad arguments before any launch (C ABI),
and the binding refuses tensors of the wrong type, shape or place.  No GPU
needed: every call below returns before it touches a device."""

import ctypes

import pytest
import torch

import paged_kv_cache_354_b200 as pk

lib = pk.lib
A = 1 << 20  # a well-aligned address that is never dereferenced


def message():
    return lib.pa_last_error_string().decode()


def plan(tables=A, held=A, free=A, num_free=A, lens=A, new=A, depths=None, stride=0, slots=A, positions=A, starts=A,
         lens_out=A, held_out=A, num_free_out=A, appended=None, status=None, batch=4, most=2, num_slots=8, blocks=10, bs=16,
         width=4):
    return lib.pa_plan_append(tables, held, free, num_free, lens, new, depths, stride, slots, positions, starts,
                              lens_out, held_out, num_free_out, appended, status, batch, most, num_slots, blocks, bs, width,
                              None)


def test_plan_refusals():
    assert plan(batch=0, num_slots=0) == pk.PA_OK
    for bad in ({"batch": -1}, {"blocks": 0}, {"bs": 0}, {"width": 0}, {"most": -1}, {"num_slots": -1}, {"stride": -1}):
        assert plan(**bad) == pk.PA_ERR_INVALID, bad
    assert plan(num_slots=9) == pk.PA_ERR_INVALID and "padded" in message()
    for name in ("tables", "held", "free", "num_free", "lens", "new", "slots", "positions", "lens_out", "held_out",
                 "num_free_out"):
        assert plan(**{name: None}) == pk.PA_ERR_INVALID and "NULL" in message()
        assert plan(**{name: A + 2}) == pk.PA_ERR_INVALID and "misaligned" in message()
    assert plan(slots=A + 4) == pk.PA_ERR_INVALID
    for name in ("depths", "appended", "status"):
        assert plan(**{name: A + 2}) == pk.PA_ERR_INVALID and "misaligned" in message()
    assert plan(starts=None, most=0) == pk.PA_ERR_INVALID  # packed needs the starts
    assert plan(depths=A, most=0) == pk.PA_ERR_INVALID and "padded" in message()
    assert plan(depths=A, stride=1) == pk.PA_ERR_INVALID
    assert plan(width=1 << 27, bs=16) == pk.PA_ERR_UNSUPPORTED
    assert plan(batch=(1 << 20) + 1, num_slots=2 * ((1 << 20) + 1)) == pk.PA_ERR_UNSUPPORTED


def rope(q_out=A, qos=256, k_out=None, kos=0, pool=A, q=A, qs=256, k=A, ks=128, v=A, vs=128, qw=None, kw=None,
         eps=1e-6, table=A, most=64, rot=64, inter=0, pos=A, slots=A, n=3, hq=4, hkv=2, d=64, blocks=4, bs=16):
    return lib.pa_norm_rope_and_cache(q_out, qos, k_out, kos, pool, q, qs, k, ks, v, vs, qw, kw, eps, table, most,
                                      rot, inter, pos, slots, n, hq, hkv, d, blocks, bs, None)


def test_norm_rope_refusals():
    assert rope(n=0) == pk.PA_OK
    for bad in ({"d": 96}, {"hq": 65537}, {"hkv": 65537}):
        assert rope(**bad) == pk.PA_ERR_UNSUPPORTED, bad
    for bad in ({"n": -1}, {"hq": -1}, {"hkv": -1}, {"hq": 0, "hkv": 0}, {"rot": 8}, {"rot": 72}, {"rot": 80},
                {"rot": -16}, {"eps": -1.0}, {"eps": float("nan")}, {"most": 0}, {"blocks": 0}, {"bs": 0}):
        assert rope(**bad) == pk.PA_ERR_INVALID, bad
    for name in ("q_out", "q", "k", "v", "table", "pos", "slots"):
        assert rope(**{name: None}) == pk.PA_ERR_INVALID and "NULL" in message(), name
    assert rope(pool=None, k_out=None) == pk.PA_ERR_INVALID  # the keys would go nowhere
    for name in ("q_out", "q", "k", "v", "pool", "qw", "kw", "table"):
        assert rope(**{name: A + 8}) == pk.PA_ERR_INVALID and "misaligned" in message(), name
    assert rope(pos=A + 2) == pk.PA_ERR_INVALID and rope(slots=A + 4) == pk.PA_ERR_INVALID
    for name in ("qs", "qos", "ks", "vs"):
        assert rope(**{name: 64}) == pk.PA_ERR_INVALID and "stride" in message(), name
        assert rope(**{name: 260}) == pk.PA_ERR_INVALID, name
    assert rope(q_out=A, q=A, qs=512) == pk.PA_ERR_INVALID and "in place" in message()


def tree(out=A, q=2 * A, pool=A, mask=A, per=1, tables=A, lens=A, counts=None, b=2, t=3, hq=8, hkv=2, d=128, bs=16,
         blocks=10, width=4, longest=64, ws=A, nbytes=1 << 40):
    return lib.pa_decode_tree(out, q, pool, mask, per, tables, lens, counts, b, t, hq, hkv, d, bs, blocks, width,
                              longest, 0.1, ws, nbytes, None)


def test_decode_tree_refusals():
    assert tree(b=0) == pk.PA_OK
    for bad in ({"b": -1}, {"t": 0}, {"hq": 0}, {"hkv": 0}, {"hq": 9}, {"blocks": 0}, {"width": 0}, {"longest": -1}):
        assert tree(**bad) == pk.PA_ERR_INVALID, bad
    for bad in ({"d": 96}, {"bs": 8}, {"hq": 130}, {"t": 1025}, {"b": 32769}):
        assert tree(**bad) == pk.PA_ERR_UNSUPPORTED, bad
    for name in ("out", "q", "pool", "mask", "tables", "lens", "ws"):
        assert tree(**{name: None}) == pk.PA_ERR_INVALID and "NULL" in message(), name
        assert tree(**{name: A + 2}) == pk.PA_ERR_INVALID and "misaligned" in message(), name
    assert tree(nbytes=0) == pk.PA_ERR_INVALID and "workspace" in message()
    size = 2 * 3 * 8 * 128 * 2  # bytes of q and of out
    for q in (A, A + 16, A + size - 16, A - size + 16):
        assert tree(q=q) == pk.PA_ERR_INVALID and "overlaps" in message()
    for q in (A + size, A - size):
        assert tree(q=q, nbytes=0) == pk.PA_ERR_INVALID and "workspace" in message()
    size = ctypes.c_size_t()
    assert lib.pa_decode_tree_workspace_size(2, 3, 8, 2, 128, 16, 64, None) == pk.PA_ERR_INVALID
    assert lib.pa_decode_tree_workspace_size(2, 3, 8, 2, 96, 16, 64, ctypes.byref(size)) == pk.PA_ERR_UNSUPPORTED


def accept(pool=A, path=A, counts=A, nodes_each=None, tables=A, lens=A, lens_out=None, b=2, nodes=4, most=3, blocks=10,
           hkv=2, bs=16, d=64, width=4):
    return lib.pa_tree_accept(pool, path, counts, nodes_each, tables, lens, lens_out, b, nodes, most, blocks, hkv, bs,
                              d, width, None)


def test_tree_accept_refusals():
    assert accept(b=0) == pk.PA_OK
    for bad in ({"b": -1}, {"nodes": -1}, {"most": -1}, {"blocks": 0}, {"hkv": 0}, {"bs": 0}, {"d": 12}, {"d": 0},
                {"width": 0}):
        assert accept(**bad) == pk.PA_ERR_INVALID, bad
    assert accept(most=1025) == pk.PA_ERR_UNSUPPORTED
    for name in ("pool", "path", "counts", "tables", "lens"):
        assert accept(**{name: None}) == pk.PA_ERR_INVALID and "NULL" in message(), name
        assert accept(**{name: A + 2}) == pk.PA_ERR_INVALID and "misaligned" in message(), name
    assert accept(nodes_each=A + 1) == pk.PA_ERR_INVALID and accept(lens_out=A + 1) == pk.PA_ERR_INVALID


def test_binding_refuses_host_tensors_and_wrong_types():
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        pk.pa_plan_append(torch.zeros((2, 4), dtype=torch.int64), i, i, i[:1], i, i, torch.zeros((2, 1)),
                          torch.zeros((2, 1)), 16)
    with pytest.raises(TypeError, match="CUDA"):
        pk.pa_plan_append(torch.zeros((2, 4), dtype=torch.int32), i, i, i[:1], i, i, torch.zeros((2, 1)),
                          torch.zeros((2, 1)), 16)
    x = torch.zeros((2, 4, 64), dtype=torch.float16)
    with pytest.raises(TypeError, match="bfloat16"):
        pk.pa_norm_rope_and_cache(x, x, x, x, None, None, None, None)
    with pytest.raises(TypeError, match="CUDA"):
        pk.pa_norm_rope_and_cache(*[x.bfloat16()] * 4, None, None, None, None)
    q = torch.zeros((2, 3, 8, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="CUDA"):
        pk.pa_decode_tree(q, q, q, i, i, i, 1, 1.0, i)
    with pytest.raises(TypeError, match="CUDA"):
        pk.pa_tree_accept(q, i, i, i, i, i)


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), float("-inf"), 3.4e38, -3.4e38])
def test_decode_tree_refuses_a_scale_that_is_not_finite(scale):
    """... or whose product with log2(e) is not."""
    assert lib.pa_decode_tree(A, 2 * A, A, A, 1, A, A, None, 2, 3, 8, 2, 128, 16, 10, 4, 64, scale, A, 1 << 40,
                              None) == pk.PA_ERR_INVALID
    assert "scale" in message()


def test_norm_rope_refuses_outputs_over_inputs_and_one_another():
    """Token rows that share memory, at any offset, are refused unless an
    output lies exactly over its own input.  Three tokens of 4 and 2 heads of
    64; every tensor is far from the others unless the case says so."""
    far = {name: A << i for i, name in enumerate(("q", "k", "v", "q_out", "pool"), 1)}
    q, k, v, pool = (far[n] for n in ("q", "k", "v", "pool"))
    q_bytes, k_bytes = 3 * 512, 3 * 256
    pool_bytes = 4 * 2 * 2 * 16 * 64 * 2
    bad = [
        {"q_out": q + 16}, {"q_out": q + q_bytes - 16}, {"q_out": q - 16}, {"q_out": q - q_bytes + 16},
        {"q_out": k}, {"q_out": k + k_bytes - 16}, {"q_out": k - q_bytes + 16}, {"q_out": v}, {"q_out": v + 16},
        {"k_out": q, "kos": 128}, {"k_out": q + 16, "kos": 128}, {"k_out": k + 16, "kos": 128},
        {"k_out": v, "kos": 128}, {"k_out": far["q_out"] + 32, "kos": 128}, {"k_out": pool, "kos": 128},
        {"q_out": pool + pool_bytes - 16}, {"q": pool}, {"k": pool + 64}, {"v": pool + pool_bytes - 16},
        {"k": q, "q_out": q},  # in place, and the keys read there too
        {"v": k, "k_out": k, "kos": 128},
        # slices of one slab of 8 heads a token: the queries' result over the last head of the queries
        {"q": q, "qs": 512, "q_out": q + 3 * 128, "qos": 512},
        {"q": q, "qs": 512, "k": q + 512, "ks": 512, "q_out": q + 3 * 128, "qos": 512},
        {"k": q + 512, "ks": 512, "q": q, "qs": 512, "k_out": q + 128, "kos": 512},
        {"q": q, "qs": 512, "q_out": q + 1024 - 16, "qos": 512},  # its end over the next token
        {"q": q, "qs": 512, "q_out": q + 512, "qos": 256},  # strides apart
    ]
    for more in bad:
        assert rope(**(far | more)) == pk.PA_ERR_INVALID and "overlap" in message(), more
