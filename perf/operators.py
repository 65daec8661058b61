"""Measured cases of the tree-speculation operators of the paged KV cache.

A serving loop that verifies trees of drafted tokens runs four operators per
step: block tables and slots for the drafted tokens (``plan``), per-head norms
and rotation of their queries and keys with the cache write (``rope``), the
attention of every tree over its request's cache (``tree``), and the move of
the accepted path's rows behind the committed prefix (``accept``).  ``run``
makes one pass through one of them: through the package's entry points where
``own`` is true, otherwise in elementary torch operations.
"""

import math

import torch

own = False

MAX_POSITION = 32768  # rows of the rotation table
EPS = 1e-6


def listed():
    return [
        # one interactive request with a small draft tree: pure latency
        {"name": "tree_one_request", "op": "tree", "batch": 1, "heads": 32, "kv_heads": 8, "dim": 128, "block": 16,
         "nodes": 8, "low": 700, "high": 700, "ragged": False},
        # the 64-request batch of the decode benchmark, 16 drafted nodes each: bound by the cache's bytes
        {"name": "tree_batch64", "op": "tree", "batch": 64, "heads": 32, "kv_heads": 8, "dim": 128, "block": 16,
         "nodes": 16, "low": 512, "high": 4096, "ragged": False},
        # few long contexts: the work is one long axis, split over the whole GPU
        {"name": "tree_long4", "op": "tree", "batch": 4, "heads": 32, "kv_heads": 8, "dim": 128, "block": 16,
         "nodes": 32, "low": 32768, "high": 32768, "ragged": False},
        # large trees at group 8: 512 query rows per KV head, bound by the matrix products
        {"name": "tree_wide64", "op": "tree", "batch": 32, "heads": 64, "kv_heads": 8, "dim": 128, "block": 32,
         "nodes": 64, "low": 1500, "high": 3000, "ragged": False},
        # a padded batch: odd lengths, trees of 0 to 33 nodes, requests with nothing cached, head dim 64
        {"name": "tree_ragged_d64", "op": "tree", "batch": 37, "heads": 4, "kv_heads": 4, "dim": 64, "block": 16,
         "nodes": 33, "low": 0, "high": 1531, "ragged": True},
        # the drafted tokens of 64 requests, slices of a fused projection's output
        {"name": "rope_step", "op": "rope", "tokens": 1024, "heads": 32, "kv_heads": 8, "dim": 128, "block": 16,
         "rotary": 128, "interleaved": False, "norm": True, "slab": True},
        # a prompt chunk: streaming
        {"name": "rope_prompt", "op": "rope", "tokens": 16384, "heads": 32, "kv_heads": 8, "dim": 128, "block": 16,
         "rotary": 128, "interleaved": False, "norm": True, "slab": True},
        # partial interleaved rotation, no norm, head dim 64, an odd number of tokens
        {"name": "rope_partial_d64", "op": "rope", "tokens": 4099, "heads": 12, "kv_heads": 4, "dim": 64, "block": 16,
         "rotary": 32, "interleaved": True, "norm": False, "slab": False},
        # one step's drafted tokens of 64 requests
        {"name": "plan_step", "op": "plan", "batch": 64, "block": 16, "low": 512, "high": 4096, "most": 16,
         "packed": False, "release": False},
        # a large serving step: prompts and single tokens packed behind one another, finished requests released
        {"name": "plan_prompts", "op": "plan", "batch": 1000, "block": 16, "low": 0, "high": 4096, "most": 1024,
         "packed": True, "release": True},
        # accepted paths of 64 requests
        {"name": "accept_step", "op": "accept", "batch": 64, "kv_heads": 8, "dim": 128, "block": 16, "nodes": 16,
         "low": 100, "high": 300, "path": 6},
        # accepted paths of a large batch of large trees
        {"name": "accept_batch", "op": "accept", "batch": 600, "kv_heads": 8, "dim": 128, "block": 32, "nodes": 64,
         "low": 20, "high": 200, "path": 16},
    ]


def draw(rng):
    def spread(low, high):
        return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))

    op = rng.choice(["tree", "tree", "rope", "plan", "accept"])
    block = rng.choice([16, 32])
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    if op == "tree":
        group = rng.choice([1, 2, 3, 4, 7, 8, 16])
        nodes = spread(1, 100)
        batch = spread(1, 96)
        high = spread(16, 40000)
        # keep the cache and the score matrix below the largest listed case's
        high = min(high, 260000 * 8 // (batch * max(kv_heads, 4)), 250000000 // (batch * kv_heads * group * nodes))
        high = max(high, 8)
        return {"op": "tree", "batch": batch, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim,
                "block": block, "nodes": nodes, "low": rng.randint(0, high), "high": high,
                "ragged": rng.random() < 0.5}
    if op == "rope":
        group = rng.choice([1, 2, 3, 4, 8])
        return {"op": "rope", "tokens": spread(1, 16000), "heads": kv_heads * group, "kv_heads": kv_heads,
                "dim": dim, "block": block, "rotary": rng.choice([dim, dim, dim // 2, 16]),
                "interleaved": rng.random() < 0.3, "norm": rng.random() < 0.7, "slab": rng.random() < 0.5}
    if op == "plan":
        packed = rng.random() < 0.4
        return {"op": "plan", "batch": spread(1, 2000), "block": block, "low": 0, "high": spread(16, 4096),
                "most": spread(1, 600) if packed else spread(1, 64), "packed": packed,
                "release": rng.random() < 0.5}
    nodes = spread(1, 100)
    return {"op": "accept", "batch": spread(1, 500), "kv_heads": kv_heads, "dim": dim, "block": block,
            "nodes": nodes, "low": 0, "high": spread(4, 200), "path": rng.randint(1, min(nodes, 20))}


def _room(case):
    """Slots of a packed step: six deviations above the mean of the drawn token counts."""
    b, most = case["batch"], case["most"]
    mean = b * (0.6 + 0.4 * most / 2)
    return min(b * most, math.ceil(mean + 6 * math.sqrt(b * 0.4 / 3) * most) + 5)


def prepare(case, seed):
    gen = torch.Generator().manual_seed(seed)  # small integers: drawn on the host
    dev_gen = torch.Generator(device="cuda").manual_seed(seed)
    bs = case["block"]

    def integers(low, high, shape):  # low .. high, both included
        return torch.randint(low, high + 1, shape, generator=gen)

    def normal(shape):
        return torch.randn(shape, generator=dev_gen, device="cuda").bfloat16()

    def tables_for(lens, blocks, width=None):
        """Block tables over a shuffled pool of `blocks` blocks; unused entries 0."""
        held = (lens + bs - 1) // bs
        order = torch.randperm(blocks, generator=gen)
        at = torch.arange(width or max(1, int(held.max())))
        start = held.cumsum(0) - held
        inside = at[None] < held[:, None]
        table = torch.where(inside, order[(start[:, None] + at[None]).clamp(max=blocks - 1)], 0)
        return table.int(), held.int(), order

    def blocks_of(length):
        return (length + bs - 1) // bs

    state = dict(case)
    if case["op"] == "tree":
        b, nodes = case["batch"], case["nodes"]
        context = integers(case["low"], case["high"], (b,))
        counts = integers(0, nodes, (b,)) if case["ragged"] else torch.full((b,), nodes)
        lens = context + counts
        blocks = math.ceil(1.1 * int(blocks_of(lens).sum())) + 1
        tables, _, _ = tables_for(lens, blocks)
        # random trees: node t's parent is an earlier node (or the last committed token)
        parent = (torch.rand((b, nodes), generator=gen) * (torch.arange(nodes) + 1)).long() - 1
        sees = torch.zeros((b, nodes, nodes), dtype=torch.bool)
        rows = torch.arange(b)
        for t in range(nodes):
            p = parent[:, t]
            sees[:, t] = torch.where((p >= 0)[:, None], sees[rows, p.clamp(min=0)], False)
            sees[:, t, t] = True
        words = (nodes + 31) // 32
        bits = torch.zeros((b, nodes, words * 32), dtype=torch.int64)
        bits[:, :, :nodes] = sees
        packed = (bits.view(b, nodes, words, 32) << torch.arange(32)).sum(-1)
        packed = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).int()
        state |= {
            "q": normal((b, nodes, case["heads"], case["dim"])),
            "pool": normal((blocks, 2, case["kv_heads"], bs, case["dim"])),
            "mask": packed.cuda(), "tables": tables.cuda(), "lens": lens.int().cuda(), "counts": counts.int().cuda(),
            "longest": case["high"] + nodes, "scale": 1.0 / math.sqrt(case["dim"]),
        }
        state["out"] = torch.empty_like(state["q"])
    elif case["op"] == "rope":
        n, dim, rot = case["tokens"], case["dim"], case["rotary"]
        hq, hkv = case["heads"], case["kv_heads"]
        if case["slab"]:  # slices of one projection's output
            slab = normal((n, (hq + 2 * hkv) * dim))
            q, k, v = (s.view(n, -1, dim) for s in slab.split([hq * dim, hkv * dim, hkv * dim], 1))
        else:
            q, k, v = normal((n, hq, dim)), normal((n, hkv, dim)), normal((n, hkv, dim))
        blocks = n // bs + 3
        order = torch.randperm(blocks, generator=gen)
        token = torch.arange(n)
        slots = order[token // bs] * bs + token % bs
        positions = (token + int(integers(0, MAX_POSITION - 1, (1,)))) % MAX_POSITION
        padding = token % 97 == 96
        slots[padding], positions[padding] = -1, -1
        speed = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
        angle = torch.arange(MAX_POSITION, dtype=torch.float64).cuda()[:, None] * speed.cuda()
        state |= {
            "q": q, "k": k, "v": v, "q_out": torch.empty((n, hq, dim), dtype=torch.bfloat16, device="cuda"),
            "pool": normal((blocks, 2, hkv, bs, dim)), "slots": slots.cuda(), "positions": positions.int().cuda(),
            "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).float(),
            "q_weight": 1 + 0.1 * normal((dim,)) if case["norm"] else None,
            "k_weight": 1 + 0.1 * normal((dim,)) if case["norm"] else None,
        }
    elif case["op"] == "plan":
        b, most = case["batch"], case["most"]
        lens = integers(case["low"], case["high"], (b,))
        new = integers(0, most, (b,)) if case["packed"] or case["release"] else torch.full((b,), most)
        if case["packed"]:  # most requests decode one token, some bring a prompt
            new = torch.where(torch.rand((b,), generator=gen) < 0.6, 1, new)
        if case["release"]:
            new = torch.where(torch.rand((b,), generator=gen) < 0.1, -1, new)
        # some requests hold a block more than they need: rejected tokens leave them so
        extra = (torch.rand((b,), generator=gen) < 0.2).long()
        width = blocks_of(case["high"] + most) + 2
        blocks = b * width  # room for every request at its longest
        tables, held, order = tables_for(lens + extra * bs, blocks, width)
        free = torch.zeros(blocks, dtype=torch.int32)
        rest = order[int(held.sum()):]
        free[: len(rest)] = rest.int()
        shape = (_room(case),) if case["packed"] else (b, most)
        state |= {
            "tables": tables.cuda(), "held": held.cuda(), "free": free.cuda(),
            "num_free": torch.tensor([len(rest)], dtype=torch.int32).cuda(), "lens": lens.int().cuda(),
            "new": new.int().cuda(), "blocks": blocks,
            "slots": torch.empty(shape, dtype=torch.int64, device="cuda"),
            "positions": torch.empty(shape, dtype=torch.int32, device="cuda"),
            "starts": torch.empty(b + 1, dtype=torch.int32, device="cuda"),
            "lens_out": torch.empty(b, dtype=torch.int32, device="cuda"),
            "held_out": torch.empty(b, dtype=torch.int32, device="cuda"),
            "num_free_out": torch.empty(1, dtype=torch.int32, device="cuda"),
        }
    else:
        b, nodes, path = case["batch"], case["nodes"], case["path"]
        context = integers(case["low"], case["high"], (b,))
        counts = torch.full((b,), nodes)
        lens = context + counts
        blocks = b * blocks_of(case["high"] + nodes)
        tables, _, _ = tables_for(lens, blocks)
        chosen = torch.rand((b, nodes), generator=gen).argsort(1)[:, :path].sort(1).values
        state |= {
            "pool": normal((blocks, 2, case["kv_heads"], bs, case["dim"])), "tables": tables.cuda(),
            "lens": lens.int().cuda(), "counts": counts.int().cuda(), "chosen": chosen.int().cuda(),
            "accepted": integers(0, path, (b,)).int().cuda(),
            "lens_out": torch.empty(b, dtype=torch.int32, device="cuda"),
        }
    return state


def run(state):
    if own:
        return _run_own(state)
    return {"tree": _tree, "rope": _rope, "plan": _plan, "accept": _accept}[state["op"]](state)


def _run_own(s):
    import paged_kv_cache_354_b200 as pk

    if s["op"] == "tree":
        if "workspace" not in s:  # kept by the program, like the pool
            b, nodes, heads, dim = s["q"].shape
            need = pk.pa_decode_tree_workspace_size(b, nodes, heads, s["kv_heads"], dim, s["block"], s["longest"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        pk.pa_decode_tree(s["out"], s["q"], s["pool"], s["mask"], s["tables"], s["lens"], s["longest"], s["scale"],
                          s["workspace"], tree_lens=s["counts"])
        return s["out"]
    if s["op"] == "rope":
        pk.pa_norm_rope_and_cache(s["q_out"], s["q"], s["k"], s["v"], s["pool"], s["slots"], s["positions"],
                                  s["cos_sin"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                                  interleaved=s["interleaved"])
        return s["q_out"], s["pool"]
    if s["op"] == "plan":
        pk.pa_plan_append(s["tables"], s["held"], s["free"], s["num_free"], s["lens"], s["new"], s["slots"],
                          s["positions"], s["block"], token_starts=s["starts"], seq_lens_out=s["lens_out"],
                          blocks_held_out=s["held_out"], num_free_out=s["num_free_out"])
        return (s["slots"], s["positions"], s["starts"], s["tables"], s["free"], s["lens_out"], s["held_out"],
                s["num_free_out"])
    pk.pa_tree_accept(s["pool"], s["chosen"], s["accepted"], s["tables"], s["lens"], s["counts"],
                      seq_lens_out=s["lens_out"])
    return s["pool"], s["lens_out"]


# ---------------------------------------------------------------- plain forms
def _tree(s):
    """softmax(scale q K^T, masked) V over every request's gathered cache."""
    b, nodes, heads, dim = s["q"].shape
    hkv, bs = s["kv_heads"], s["block"]
    width = s["tables"].shape[1] * bs
    both = s["pool"][s["tables"].long()]  # [B, blocks, 2, Hkv, bs, D]
    keys, values = (both[:, :, i].permute(0, 2, 1, 3, 4).reshape(b, hkv, width, dim).float() for i in (0, 1))
    at = torch.arange(width, device="cuda")
    base = (s["lens"] - s["counts"]).long()
    node = at[None] - base[:, None]  # [B, width]: the tree node at a position
    word = (node.clamp(0, nodes - 1) >> 5)[:, None].expand(b, nodes, width)
    bit = (s["mask"].long().gather(2, word) >> (node & 31)[:, None]) & 1
    sees = torch.where(node[:, None] < 0, True, bit != 0) & (at[None] < s["lens"][:, None])[:, None]
    sees &= (torch.arange(nodes, device="cuda")[None] < s["counts"][:, None])[:, :, None]
    q = s["q"].float().view(b, nodes, hkv, heads // hkv, dim).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, dim)
    scores = (q @ keys.transpose(2, 3)).view(b, hkv, heads // hkv, nodes, width) * s["scale"]
    scores = scores.masked_fill(~sees[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    weight = (scores - top).exp()
    weight /= weight.sum(-1, keepdim=True).clamp(min=1e-30)
    values = values.masked_fill((at[None] >= s["lens"][:, None])[:, None, :, None], 0)
    out = weight.view(b, hkv, -1, width) @ values
    return out.view(b, hkv, heads // hkv, nodes, dim).permute(0, 3, 1, 2, 4).reshape(b, nodes, heads, dim).bfloat16()


def _normed(x, weight):
    if weight is None:
        return x
    return x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * weight.float()


def _rotated(x, cos, sin, interleaved):
    half = cos.shape[-1]
    turned, rest = x[..., : 2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = turned[..., :half], turned[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, rest], -1)


def _rope(s):
    real = s["positions"] >= 0
    turn = s["cos_sin"][s["positions"].clamp(min=0).long()]
    cos, sin = (t[:, None] for t in turn.chunk(2, -1))
    q = _rotated(_normed(s["q"].float(), s["q_weight"]), cos, sin, s["interleaved"])
    k = _rotated(_normed(s["k"].float(), s["k_weight"]), cos, sin, s["interleaved"])
    bs = s["block"]
    # a padding token writes the last token's rows again instead
    last = torch.where(s["slots"] >= 0, torch.arange(len(real), device="cuda"), -1).amax().clamp(min=0)
    take = torch.where(s["slots"] >= 0, torch.arange(len(real), device="cuda"), last)
    slot = s["slots"][take].clamp(min=0)
    s["pool"][slot // bs, 0, :, slot % bs] = k.bfloat16()[take]
    s["pool"][slot // bs, 1, :, slot % bs] = s["v"][take]
    return torch.where(real[:, None, None], q, 0).bfloat16(), s["pool"]


def _plan(s):
    b, width, bs = s["tables"].shape[0], s["tables"].shape[1], s["block"]
    lens, held, new = s["lens"].long(), s["held"].long(), s["new"].long()
    num_free = s["num_free"].long()
    gone, count = new < 0, new.clamp(min=0)
    # released blocks go on top of the stack, in (request, table) order
    back = torch.where(gone, held, 0)
    back_at = back.cumsum(0) - back
    col = torch.arange(width, device="cuda")
    stack = torch.cat([s["free"].long(), torch.zeros(1, dtype=torch.long, device="cuda")])
    where = torch.where(col[None] < back[:, None], num_free + back_at[:, None] + col[None], s["blocks"])
    stack[where.clamp(max=s["blocks"])] = s["tables"].long()
    free = num_free + back.sum()
    end = torch.where(gone, 0, lens + count)
    need = torch.where(gone, 0, ((end + bs - 1) // bs - held).clamp(min=0))
    need_at = need.cumsum(0) - need
    fresh = (col[None] >= held[:, None]) & (col[None] < (held + need)[:, None])
    popped = stack[(free - 1 - need_at[:, None] - (col[None] - held[:, None])).clamp(0, s["blocks"] - 1)]
    tables = torch.where(fresh, popped, s["tables"].long())
    starts = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), count.cumsum(0)])
    if s["packed"]:
        token = torch.arange(s["slots"].shape[0], device="cuda")
        row = torch.searchsorted(starts, token, right=True) - 1
        inside = token < starts[-1]
        row = row.clamp(max=b - 1)
        offset = token - starts[row]
    else:
        row = torch.arange(b, device="cuda")[:, None]
        offset = torch.arange(s["slots"].shape[1], device="cuda")[None]
        inside = offset < count[:, None]
    position = lens[row] + offset
    block = tables[row, (position // bs).clamp(max=width - 1)]
    slots = torch.where(inside, block * bs + position % bs, -1)
    return (slots, torch.where(inside, position, -1).int(), starts.int(), tables.int(), stack[:-1].int(), end.int(),
            torch.where(gone, 0, held + need).int(), (free - need.sum()).int())


def _accept(s):
    bs = s["block"]
    base = (s["lens"] - s["counts"]).long()
    step = torch.arange(s["chosen"].shape[1], device="cuda")
    to = base[:, None] + step[None]
    frm = base[:, None] + s["chosen"].long()
    # steps that are not accepted move a row onto itself
    to = torch.where(step[None] < s["accepted"][:, None], to, frm)
    keep = step[None] >= s["accepted"][:, None]
    # two writers of one row have to bring the same value: accepted steps go last
    rows = []
    for at in (frm, to):
        rows.append((s["tables"].long().gather(1, at // bs), at % bs))
    moved = s["pool"][rows[0][0], :, :, rows[0][1]]
    live = (~keep).flatten().nonzero().flatten()
    s["pool"][rows[1][0].flatten()[live], :, :, rows[1][1].flatten()[live]] = moved.flatten(0, 1)[live]
    return s["pool"], (base + s["accepted"].long()).int()


# ------------------------------------------------------------------ the floor
def work(case):
    bs = case["block"]
    if case["op"] == "tree":
        nodes = case["nodes"] * (0.5 if case["ragged"] else 1.0)
        length = (case["low"] + case["high"]) / 2 + nodes
        cache = case["batch"] * length * case["kv_heads"] * case["dim"] * 4
        ends = 4 * case["batch"] * case["nodes"] * case["heads"] * case["dim"]
        mask = case["batch"] * case["nodes"] * 4 * ((case["nodes"] + 31) // 32)
        tables = case["batch"] * (4 * length / bs + 8)
        return {"bytes": cache + ends + mask + tables,
                "flops": 4.0 * case["batch"] * length * nodes * case["heads"] * case["dim"]}
    if case["op"] == "rope":
        n = case["tokens"]
        rows = n * (case["heads"] + 2 * case["kv_heads"]) * case["dim"] * 2
        turned = n * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 2 * rows + min(n, MAX_POSITION) * case["rotary"] * 4 + 12 * n, "flops": 8.0 * turned}
    if case["op"] == "plan":
        b = case["batch"]
        tokens = _room(case) if case["packed"] else b * case["most"]
        length = (case["low"] + case["high"]) / 2
        # lengths, counts and holdings in and out, a table entry per block that a token falls in, slots and positions
        return {"bytes": 24 * b + 8 * (b + tokens / bs) + 12 * tokens
                + (0.1 * b * length / bs * 8 if case["release"] else 0), "flops": 4.0 * tokens}
    moved = case["batch"] * case["path"] / 2 * case["kv_heads"] * case["dim"] * 4
    return {"bytes": 2 * moved + case["batch"] * (12 + 6 * case["path"]), "flops": 0}


# ------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    bs = s["block"]
    if case["op"] == "tree":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        group = case["heads"] // case["kv_heads"]
        lens, counts = s["lens"].tolist(), s["counts"].tolist()
        for b in range(case["batch"]):
            length, n = lens[b], counts[b]
            if n == 0 or length == 0:
                continue
            blocks = s["tables"][b, : -(-length // bs)].long()
            kv = s["pool"][blocks].double().transpose(1, 3).reshape(-1, case["kv_heads"], 2, case["dim"])[:length]
            # [n, n] truth values of the tree, then [n, length]
            i = torch.arange(n, device="cuda")
            tree = (s["mask"][b, :n].long()[:, i // 32] >> (i % 32)) & 1
            sees = torch.cat([torch.ones((n, length - n), dtype=torch.long, device="cuda"), tree], 1).bool()
            for h in range(case["kv_heads"]):
                q = s["q"][b, :n, h * group:(h + 1) * group].double()
                score = torch.einsum("tgd,pd->tgp", q, kv[:, h, 0]) * s["scale"]
                score = torch.where(sees[:, None], score, -math.inf)
                out[b, :n, h * group:(h + 1) * group] = torch.einsum("tgp,pd->tgd", torch.softmax(score, -1),
                                                                     kv[:, h, 1])
        return out
    if case["op"] == "rope":
        pool = s["pool"].double()
        half = case["rotary"] // 2
        answers = []
        for x, weight in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
            y = x.double()
            if weight is not None:
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / case["dim"] + EPS) * weight.double()
            turn = s["cos_sin"].double()[s["positions"].clamp(min=0).long()]
            z = torch.complex(turn[:, :half], turn[:, half:])[:, None]
            first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"] else (
                slice(0, half), slice(half, 2 * half))
            c = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * z
            y = y.clone()
            y[..., first], y[..., second] = c.real, c.imag
            answers.append(y)
        answers[0][s["positions"] < 0] = 0
        live = s["slots"] >= 0
        slot = s["slots"][live]
        pool[slot // bs, 0, :, slot % bs] = answers[1][live]
        pool[slot // bs, 1, :, slot % bs] = s["v"][live].double()
        return answers[0], pool
    if case["op"] == "plan":
        return None  # whole numbers: compared for equality
    pool = s["pool"].double()
    lens, counts, accepted, chosen = (s[k].tolist() for k in ("lens", "counts", "accepted", "chosen"))
    tables = s["tables"].tolist()
    source, target = [], []
    for b in range(case["batch"]):
        base = lens[b] - counts[b]
        for i in range(accepted[b]):
            for rows, p in ((source, base + chosen[b][i]), (target, base + i)):
                rows.append((tables[b][p // bs], p % bs))
    if source:
        src, dst = (torch.tensor(r, device="cuda") for r in (source, target))
        pool[dst[:, 0], :, :, dst[:, 1]] = pool[src[:, 0], :, :, src[:, 1]].clone()
    return pool, None
