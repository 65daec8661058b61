"""fp64 oracle of the tree-speculation operators -- test infrastructure only.

Plain loops over requests, nodes and heads; layouts as in
``oracle/paged_attention.py``.  Block tables and free lists are Python lists.
"""

import numpy as np

from oracle.paged_attention import gather_kv


def plan_append(tables, held, free, seq_lens, new_tokens, block_size, max_blocks):
    """Append (or, with a negative count, end) every request, in order.

    tables : list of lists, the first ``held[b]`` entries of row b are the
    request's blocks; free : list, the top of the stack last.  Returns
    (tables, held, free, seq_lens, slots, positions) with per-request lists of
    slots and positions, or None when the call is refused.
    """
    tables = [list(t) for t in tables]
    held, free, lens = list(held), list(free), list(seq_lens)
    for b, c in enumerate(new_tokens):
        if lens[b] < 0 or lens[b] + max(c, 0) > max_blocks * block_size:
            return None
        if c < 0:
            free += tables[b][: held[b]]
            held[b] = lens[b] = 0
    slots, positions = [], []
    for b, c in enumerate(new_tokens):
        mine, at = [], []
        for p in range(lens[b], lens[b] + max(c, 0)):
            at.append(p)
        while held[b] * block_size < lens[b] + max(c, 0):
            if not free:
                return None
            block = free.pop()
            tables[b][held[b]:held[b] + 1] = [block]
            held[b] += 1
        for p in at:
            mine.append(tables[b][p // block_size] * block_size + p % block_size)
        lens[b] += max(c, 0)
        slots.append(mine)
        positions.append(at)
    return tables, held, free, lens, slots, positions


def norm_rope(x, weight, eps, cos_sin, positions, interleaved):
    """x float64 [n, heads, D] -> (y, bound): the normed and rotated rows and
    |y_a cos| + |y_b sin| of every element, the scale of its rounding error."""
    y = np.array(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * weight
    bound = np.abs(y)
    rot = 0 if cos_sin is None else cos_sin.shape[1]
    out = y.copy()
    for t in range(x.shape[0]):
        if positions is not None and positions[t] < 0:
            out[t] = 0
            continue
        for i in range(rot // 2):
            c, s = cos_sin[positions[t], i], cos_sin[positions[t], rot // 2 + i]
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            out[t, :, a] = y[t, :, a] * c - y[t, :, b] * s
            out[t, :, b] = y[t, :, b] * c + y[t, :, a] * s
            bound[t, :, a] = np.abs(y[t, :, a] * c) + np.abs(y[t, :, b] * s)
            bound[t, :, b] = np.abs(y[t, :, b] * c) + np.abs(y[t, :, a] * s)
    return out, bound


def decode_tree(q, kv_pool, sees, block_tables, seq_lens, tree_lens, scale):
    """Tree attention, one request, node and KV head at a time.

    q float64 [B, T, Hq, D]; sees bool [B, T, T]: node t attends to node i.
    Returns (out, spread, size, logit): per element sum p |v - out| and
    sum p |v|, and per row the largest scale * sum |q| |k| over its positions
    (the scales of the rounding errors).
    """
    batch, nodes, hq, d = q.shape
    hkv = kv_pool.shape[2]
    group = hq // hkv
    out, spread, size = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    logit = np.zeros(q.shape[:3])
    for b in range(batch):
        length, n = int(seq_lens[b]), int(tree_lens[b])
        if length == 0 or n == 0:
            continue
        keys, values = gather_kv(kv_pool, block_tables[b], length)
        for t in range(n):
            attended = np.concatenate([np.ones(length - n, dtype=bool), sees[b, t, :n]])
            if not attended.any():
                continue
            for h in range(hkv):
                k, v = keys[attended, h], values[attended, h]
                rows = q[b, t, h * group:(h + 1) * group]
                s = scale * rows @ k.T
                p = np.exp(s - s.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                o = p @ v
                at = (b, t, slice(h * group, (h + 1) * group))
                out[at] = o
                spread[at] = np.stack([p[j] @ np.abs(v - o[j]) for j in range(group)])
                size[at] = p @ np.abs(v)
                logit[at] = (abs(scale) * np.abs(rows) @ np.abs(k).T).max(-1)
    return out, spread, size, logit


def tree_accept(kv_pool, path, accept_lens, tree_lens, block_tables, seq_lens):
    """Rows of the accepted nodes move behind the prefix; returns (pool, lengths).
    Every source row is read before any row is written."""
    block_size = kv_pool.shape[3]
    lens = []
    moves = []
    for b in range(len(seq_lens)):
        base = int(seq_lens[b]) - int(tree_lens[b])
        for i in range(int(accept_lens[b])):
            src, dst = base + int(path[b][i]), base + i
            row = kv_pool[block_tables[b][src // block_size], :, :, src % block_size].copy()
            moves.append((block_tables[b][dst // block_size], dst % block_size, row))
        lens.append(base + int(accept_lens[b]))
    for block, offset, row in moves:
        kv_pool[block, :, :, offset] = row
    return kv_pool, lens
