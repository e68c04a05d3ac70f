"""The operators of a serving step over a paged cache held in 8 bits, as they are measured.

A step appends each sequence's new tokens to the block pool on the device (block tables, slot map, copy-on-write
pairs), returns the blocks of finished sequences, writes the new K/V rows into an int8 cache that keeps one fp32
scale per (block, kv head), and decodes over that cache:

  append   pa_dpool_append   block tables, context lengths, q_start, slot map and copy pairs from the lengths
  release  pa_dpool_release  the blocks of finished sequences back to the free list
  write    pa_append_q8b     quantising write of the new tokens' K/V rows
  decode   pa_decode_q8b     attention of one query token per sequence over the cache

Where ``own`` is false, ``run`` computes them in plain torch operations. Lengths go by the case alone
(``shape_seed``); pool order, tables and values go by the seed.

The pool operators change their state, so a pass first puts the state back (one device copy in both forms). The
quantised codes are defined bit for bit (every step is one IEEE fp32 operation): they are whole numbers here, with
their scales beside them.
"""
import numpy as np
import torch

own = False

LIFO, FIFO = 0, 1
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token for each of a small batch's sequences, some of them forks that must copy their last block
        dict(name="append_decode_64", op="append", seqs=64, ctx_lo=256, ctx_hi=2048, new_lo=1, new_hi=1, long_every=0,
             fork_every=8, block_size=16, policy=LIFO, pad_tokens=0, shape_seed=1),
        # a continuous batch: most sequences append one token, every 16th a chunk of its prompt
        dict(name="append_mixed_1000", op="append", seqs=1000, ctx_lo=0, ctx_hi=4096, new_lo=0, new_hi=1, long_every=16,
             fork_every=5, block_size=16, policy=FIFO, pad_tokens=333, shape_seed=2),
        # whole prompts of a large batch, from empty
        dict(name="append_prompts_256", op="append", seqs=256, ctx_lo=0, ctx_hi=0, new_lo=1, new_hi=2048, long_every=0,
             fork_every=0, block_size=32, policy=FIFO, pad_tokens=0, shape_seed=3),
        # a few finished sequences of a small batch
        dict(name="release_few_of_64", op="release", seqs=64, ctx_lo=256, ctx_hi=2048, finish_pct=10, fork_every=8,
             block_size=16, policy=LIFO, shape_seed=4),
        # half of a large batch, with long contexts and shared blocks
        dict(name="release_half_of_1000", op="release", seqs=1000, ctx_lo=1, ctx_hi=4096, finish_pct=50, fork_every=5,
             block_size=16, policy=FIFO, shape_seed=5),
        # each sequence's newest token, into blocks that already hold older ones
        dict(name="write_decode_64_gqa", op="write", seqs=64, old_lo=1, old_hi=500, new_lo=1, new_hi=1, pad_tokens=0,
             kv_heads=8, head_dim=128, block_size=16, dtype="bf16", shape_seed=6),
        # eight prompts of 2048 tokens, 32 heads
        dict(name="write_prompts_mha", op="write", seqs=8, old_lo=0, old_hi=0, new_lo=2048, new_hi=2048, pad_tokens=0,
             kv_heads=32, head_dim=128, block_size=16, dtype="f16", shape_seed=7),
        # ragged chunks of a padded batch, 32-bit source, narrow heads
        dict(name="write_ragged_f32", op="write", seqs=100, old_lo=0, old_hi=300, new_lo=1, new_hi=512, pad_tokens=77,
             kv_heads=6, head_dim=64, block_size=32, dtype="f32", shape_seed=8),
        # four short sequences, one of a single token: the smallest call
        dict(name="decode_small_d64", op="decode", seqs=4, ctx_lo=1, ctx_hi=100, heads=8, kv_heads=4, head_dim=64,
             block_size=16, dtype="f16", out="f32", shape_seed=9),
        # 64 sequences of 256 to 2048 tokens, every query head with its own kv head
        dict(name="decode_mha_fp16", op="decode", seqs=64, ctx_lo=256, ctx_hi=2048, heads=32, kv_heads=32,
             head_dim=128, block_size=16, dtype="f16", out="f16", shape_seed=10),
        # 256 sequences of 128 to 4096 tokens, four query heads to a kv head
        dict(name="decode_gqa_bf16", op="decode", seqs=256, ctx_lo=128, ctx_hi=4096, heads=32, kv_heads=8,
             head_dim=128, block_size=16, dtype="bf16", out="bf16", shape_seed=11),
        # eight very long sequences
        dict(name="decode_long_bf16", op="decode", seqs=8, ctx_lo=32768, ctx_hi=131072, heads=32, kv_heads=8,
             head_dim=128, block_size=32, dtype="bf16", out="f32", shape_seed=12),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(float(np.exp(rng.uniform(np.log(max(lo, 1)), np.log(hi))))))))


def draw(rng):
    op = rng.choice(["append", "release", "write", "decode"])
    c = dict(op=op, block_size=rng.choice([16, 32]), shape_seed=rng.randrange(1 << 30))
    if op in ("append", "release"):
        c.update(seqs=_log_int(rng, 1, 1000), ctx_lo=0, ctx_hi=_log_int(rng, 16, 4096), fork_every=rng.choice([0, 2, 3, 7]),
                 policy=rng.choice([LIFO, FIFO]))
        if op == "append":
            hi = _log_int(rng, 1, 250000 // max(c["seqs"], 122))
            c.update(new_lo=rng.choice([0, 1]), new_hi=hi, long_every=0, pad_tokens=rng.choice([0, 5, 1000]))
        else:
            c.update(ctx_lo=1, finish_pct=rng.choice([5, 30, 100]))
        return c
    c.update(kv_heads=rng.choice([1, 2, 3, 5, 8, 16, 32]), head_dim=rng.choice([64, 128]))
    if op == "write":
        c.update(dtype=rng.choice(["f16", "bf16", "f32"]), seqs=_log_int(rng, 1, 300), old_lo=0,
                 old_hi=rng.choice([0, 40, 500]), pad_tokens=rng.choice([0, 1, 50]))
        most = (1 << 26) // (c["seqs"] * c["kv_heads"] * c["head_dim"] * (2 if c["dtype"] == "f32" else 1))
        c.update(new_lo=1, new_hi=_log_int(rng, 1, max(2, min(4096, most))))
        return c
    c.update(seqs=_log_int(rng, 1, 300), heads=c["kv_heads"] * rng.choice([1, 2, 3, 4, 6, 8]),
             dtype=rng.choice(["f16", "bf16"]))
    c["out"] = rng.choice([c["dtype"], "f32"])
    most = (1 << 29) // (c["seqs"] * c["kv_heads"] * c["head_dim"])
    c.update(ctx_lo=1, ctx_hi=_log_int(rng, 16, max(32, min(131072, most))))
    return c


# ------------------------------------------------------------------ lengths

def _cdiv(a, b):
    return -(-a // b)


def _pool_lengths(c):
    """(context lengths, new lengths or None, finished or None) of a pool case."""
    r = np.random.default_rng(c["shape_seed"])
    S = c["seqs"]
    ctx = r.integers(c["ctx_lo"], c["ctx_hi"] + 1, S)
    if c["fork_every"]:  # sequence i + 1 is a fork of sequence i, with the same tokens so far
        for i in range(0, S - 1, c["fork_every"]):
            ctx[i + 1] = ctx[i]
    if c["op"] == "release":
        fin = r.random(S) * 100 < c["finish_pct"]
        fin[r.integers(0, S)] = True
        return ctx, None, fin
    new = r.integers(c["new_lo"], c["new_hi"] + 1, S)
    if c["long_every"]:
        new[::c["long_every"]] = r.integers(1, 513, new[::c["long_every"]].size)
    return ctx, new, None


def _write_lengths(c):
    r = np.random.default_rng(c["shape_seed"])
    return r.integers(c["old_lo"], c["old_hi"] + 1, c["seqs"]), r.integers(c["new_lo"], c["new_hi"] + 1, c["seqs"])


def _decode_lengths(c):
    r = np.random.default_rng(c["shape_seed"])
    lo, hi = np.log(c["ctx_lo"]), np.log(c["ctx_hi"] + 1)
    return np.clip(np.exp(r.uniform(lo, hi, c["seqs"])).astype(np.int64), c["ctx_lo"], c["ctx_hi"])


def work(case):
    c, bs = case, case["block_size"]
    if c["op"] == "append":
        ctx, new, _ = _pool_lengths(c)
        takes = int((_cdiv(ctx + new, bs) - _cdiv(ctx, bs)).sum())
        tokens = int(new.sum()) + c["pad_tokens"]
        # lengths in and out, last block and its count, q_start; ring, table and count of each take; slots
        return dict(bytes=c["seqs"] * 24 + takes * 12 + tokens * 4, flops=0)
    if c["op"] == "release":
        ctx, _, fin = _pool_lengths(c)
        entries = int(_cdiv(ctx[fin], bs).sum())
        # lengths and mask; table entry in and out, count in and out, ring entry
        return dict(bytes=c["seqs"] * 8 + entries * 20, flops=0)
    H, D = c["kv_heads"], c["head_dim"]
    if c["op"] == "write":
        old, new = _write_lengths(c)
        rows = int(new.sum()) * H * 2
        blocks = int((_cdiv(old + new, bs) - old // bs).sum())
        elt = DTYPES[c["dtype"]].itemsize
        return dict(bytes=rows * D * (elt + 1) + blocks * (H * 8 + 4) + c["seqs"] * 8, flops=rows * D * 3)
    ctx = _decode_lengths(c)
    n, blocks = int(ctx.sum()), int(_cdiv(ctx, bs).sum())
    q = c["seqs"] * c["heads"] * D
    return dict(bytes=2 * n * H * D + blocks * (H * 8 + 4) + q * (2 + DTYPES[c["out"]].itemsize) + 4 * c["seqs"],
                flops=4 * n * c["heads"] * D)


# ------------------------------------------------------------------- inputs

class _HostPool:
    """A pool's counts and free list on the host, as a device pool is loaded from them."""

    def __init__(self, num_blocks, block_size, ref, free):
        self.num_blocks, self.block_size, self._ref, self._free = num_blocks, block_size, ref, free

    def export(self):
        return self._ref, self._free


def _pool_start(c, seed):
    """Host arrays of a pool case before the call: tables, context lengths, counts, free list."""
    ctx, new, fin = _pool_lengths(c)
    S, bs = c["seqs"], c["block_size"]
    have = _cdiv(ctx, bs)
    end = _cdiv(ctx + (new if new is not None else 0), bs)
    mb = int(max(1, end.max())) + 3
    nb = int(end.sum()) + S + 16
    order = np.random.default_rng(seed).permutation(nb).astype(np.int32)
    tables = np.full((S, mb), -1, np.int32)
    ref = np.zeros(nb, np.int32)
    at = 0
    for s in range(S):
        n = int(have[s])
        fork = c["fork_every"] and s and (s - 1) % c["fork_every"] == 0
        if fork:
            tables[s, :n] = tables[s - 1, :n]
        else:
            tables[s, :n] = order[at:at + n]
            at += n
        ref[tables[s, :n]] += 1
    return dict(tables=tables, ctx=ctx.astype(np.int32), new=new, fin=fin, ref=ref, free=order[at:].copy(), nb=nb, mb=mb)


def _prepare_pool(c, seed):
    h = _pool_start(c, seed)
    nb, S, mb = h["nb"], c["seqs"], h["mb"]
    ring = np.full(nb, -1, np.int32)
    ring[:h["free"].size] = h["free"]
    st = dict(case=c, nb=nb)
    if own:
        from paged_kv_cache_340_b200 import DevicePool
        pool = DevicePool(nb, c["block_size"], c["policy"], host_pool=_HostPool(nb, c["block_size"], h["ref"], h["free"]))
        words = pool.state.numel()
        lead = pool.state.cpu().numpy()
    else:
        words = 8 + 2 * nb
        lead = np.concatenate([np.array([nb, c["block_size"], c["policy"], 0, h["free"].size, 0, 0, 0], np.int32), h["ref"], ring])
    # the pool's state, the tables and the context lengths in one buffer, so that one copy puts them back
    pad = _cdiv(words, 4) * 4
    start = np.concatenate([lead, np.zeros(pad - words, np.int32), h["tables"].reshape(-1), h["ctx"]])
    st["start"] = torch.from_numpy(start).cuda()
    a = st["arena"] = st["start"].clone()
    st["header"], st["ref"], st["ring"] = a[:5], a[8:8 + nb], a[8 + nb:8 + 2 * nb]
    st["tables"] = a[pad:pad + S * mb].view(S, mb)
    st["ctx"] = a[pad + S * mb:]
    if own:
        pool.state = a[:words]
        st["pool"] = pool
    if c["op"] == "append":
        tokens = int(h["new"].sum()) + c["pad_tokens"]
        st["new"] = torch.from_numpy(h["new"].astype(np.int32)).cuda()
        st["q_start"] = torch.empty(S + 1, dtype=torch.int32, device="cuda")
        st["slots"] = torch.empty(tokens, dtype=torch.int32, device="cuda")
        st["pairs"] = torch.empty((S, 2), dtype=torch.int64, device="cuda")
        st["num_cow"] = torch.empty(1, dtype=torch.int32, device="cuda")
    else:
        st["finished"] = torch.from_numpy(h["fin"].astype(np.int32)).cuda()
    return st


def _tables_for(lens, bs, r, spare=3):
    """Tables [S, MB] over a random order of just enough blocks and a few more, and the number of blocks."""
    n = _cdiv(lens, bs)
    nb = int(n.sum()) + spare
    order = r.permutation(nb).astype(np.int32)
    tables = np.full((len(lens), int(max(1, n.max()))), -1, np.int32)
    at = 0
    for s, k in enumerate(n):
        tables[s, :k] = order[at:at + k]
        at += int(k)
    return tables, nb


def _codes(nb, H, bs, D, g):
    """Codes and scales of random rows, some heads and blocks larger than others."""
    x = torch.randn((nb, H, bs, D), generator=g, device="cuda")
    x *= torch.rand((nb, H, 1, 1), generator=g, device="cuda") + 0.5
    s = x.abs().amax(dim=(2, 3)) / 127
    return torch.round(x / s[:, :, None, None]).clamp(-127, 127).to(torch.int8), s


def prepare(case, seed):
    c = case
    if c["op"] in ("append", "release"):
        return _prepare_pool(c, seed)
    r = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    H, D, bs, S, dt = c["kv_heads"], c["head_dim"], c["block_size"], c["seqs"], DTYPES[c["dtype"]]
    if c["op"] == "write":
        old, new = _write_lengths(c)
        tables, nb = _tables_for(old + new, bs, r)
        kc, ks = _codes(nb, H, bs, D, g)
        vc, vs = _codes(nb, H, bs, D, g)
        T = int(new.sum()) + c["pad_tokens"]
        key, value = (torch.randn((T, H, D), generator=g, device="cuda").to(dt) for _ in range(2))
        q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        return dict(case=c, key=key, value=value, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs,
                    q_start=torch.from_numpy(q_start).cuda(), tables=torch.from_numpy(tables).cuda(),
                    ctx=torch.from_numpy((old + new).astype(np.int32)).cuda())
    ctx = _decode_lengths(c)
    tables, nb = _tables_for(ctx, bs, r)
    kc, ks = _codes(nb, H, bs, D, g)
    vc, vs = _codes(nb, H, bs, D, g)
    q = torch.randn((S, c["heads"], D), generator=g, device="cuda").to(dt)
    order = np.argsort(-ctx, kind="stable").astype(np.int32)  # longest first
    st = dict(case=c, q=q, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, tables=torch.from_numpy(tables).cuda(),
              ctx=torch.from_numpy(ctx.astype(np.int32)).cuda(), max_ctx=int(ctx.max()),
              order=torch.from_numpy(order).cuda(), scale=D ** -0.5,
              out=torch.empty((S, c["heads"], D), dtype=DTYPES[c["out"]], device="cuda"))
    if own:
        from paged_kv_cache_340_b200 import pa_decode_q8b_workspace_bytes
        n = pa_decode_q8b_workspace_bytes(S, c["heads"], H, D, st["max_ctx"])
        st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return st


# -------------------------------------------------------------- plain forms

def _plain_append(st):
    c, nb = st["case"], st["nb"]
    bs, S, mb = c["block_size"], c["seqs"], st["tables"].shape[1]
    ref, ring, hdr = st["ref"].long(), st["ring"].long(), st["header"].long()
    tables, ctx, new = st["tables"].long(), st["ctx"].long(), st["new"].long()
    dev = ctx.device
    s = torch.arange(S, device=dev)
    last = ctx // bs
    partial = (new > 0) & (ctx % bs > 0)
    b = torch.where(partial, tables.gather(1, last.clamp(max=mb - 1)[:, None])[:, 0], nb)  # nb: nowhere
    holders = torch.cat([ref, ref.new_zeros(1)])
    writers = torch.zeros(nb + 1, dtype=torch.long, device=dev).scatter_add(0, b, partial.long())
    latest = torch.full((nb + 1,), -1, device=dev).scatter_reduce(0, b, s, "amax")
    cow = partial & (holders[b] > 1) & ~((writers[b] == holders[b]) & (latest[b] == s))
    have = (ctx + bs - 1) // bs
    grow = torch.where(new > 0, (ctx + new + bs - 1) // bs - have, 0)
    takes = grow + cow
    before = takes.cumsum(0) - takes
    total = takes.sum()
    head, count = hdr[3], hdr[4]

    def block_of(k):
        return ring[((head + k) if c["policy"] == FIFO else (head + count - 1 - k)) % nb]

    j = torch.arange(mb, device=dev)[None, :]
    i = j - have[:, None]
    fresh = (i >= 0) & (i < grow[:, None])
    copied = cow[:, None] & (j == last[:, None])
    k = torch.where(copied, before[:, None], before[:, None] + cow[:, None] + i)
    tables = torch.where(fresh | copied, block_of(k.clamp(min=0)), tables)
    pairs_at = torch.where(cow, cow.cumsum(0) - 1, S)
    pairs = torch.full((S + 1, 2), -1, dtype=torch.long, device=dev)
    mine = tables.gather(1, last.clamp(max=mb - 1)[:, None])[:, 0]
    pairs = pairs.index_copy(0, pairs_at, torch.stack([b, mine], 1))[:S]
    taken = torch.where(fresh | copied, tables, nb)
    ref = holders.scatter_add(0, torch.where(cow, b, nb), torch.full_like(b, -1))
    ref = ref.scatter(0, taken.reshape(-1), 1)[:nb]
    q_start = torch.cat([new.new_zeros(1), new.cumsum(0)])
    t = torch.arange(st["slots"].shape[0], device=dev)
    of = torch.searchsorted(q_start[1:], t, right=True).clamp(max=S - 1)
    pos = ctx[of] + t - q_start[of]
    slot = tables[of, (pos // bs).clamp(max=mb - 1)] * bs + pos % bs
    slots = torch.where(t < q_start[S], slot, -1)
    head = (head + total) % nb if c["policy"] == FIFO else head
    hdr = torch.stack([hdr[0], hdr[1], hdr[2], head, count - total])
    n32 = torch.int32
    return dict(tables=tables.to(n32), ctx=(ctx + new).to(n32), q_start=q_start.to(n32), slots=slots.to(n32), pairs=pairs,
                num_cow=cow.sum().to(n32).reshape(1), header=hdr.to(n32), ref=ref.to(n32), ring=st["ring"])


def _plain_release(st):
    c, nb = st["case"], st["nb"]
    bs, S, mb = c["block_size"], c["seqs"], st["tables"].shape[1]
    ref, ring, hdr = st["ref"].long(), st["ring"].long(), st["header"].long()
    tables, ctx, fin = st["tables"].long(), st["ctx"].long(), st["finished"] != 0
    dev = ctx.device
    have = (ctx + bs - 1) // bs
    used = fin[:, None] & (torch.arange(mb, device=dev)[None, :] < have[:, None])
    ids = torch.where(used, tables, nb).reshape(-1)
    place = torch.arange(S * mb, device=dev)
    drops = torch.zeros(nb + 1, dtype=torch.long, device=dev).scatter_add(0, ids, used.reshape(-1).long())
    latest = torch.full((nb + 1,), -1, device=dev).scatter_reduce(0, ids, place, "amax")
    holders = torch.cat([ref, ref.new_zeros(1)])
    freed = used.reshape(-1) & (drops[ids] == holders[ids]) & (latest[ids] == place)
    rank = freed.long().cumsum(0) - 1
    at = torch.where(freed, (hdr[3] + hdr[4] + rank) % nb, nb)
    ring = torch.cat([ring, ring.new_zeros(1)]).scatter(0, at, ids)[:nb]
    hdr = torch.stack([hdr[0], hdr[1], hdr[2], hdr[3], hdr[4] + freed.sum()])
    n32 = torch.int32
    return dict(tables=torch.where(used, -1, tables).to(n32), ctx=torch.where(fin, 0, ctx).to(n32),
                header=hdr.to(n32), ref=(ref - drops[:nb]).to(n32), ring=ring.to(n32))


def _plain_write(st):
    c = st["case"]
    bs, S, H, D = c["block_size"], c["seqs"], c["kv_heads"], c["head_dim"]
    q_start, ctx, tables = st["q_start"].long(), st["ctx"].long(), st["tables"].long()
    nb, T = st["k_cache"].shape[0], st["key"].shape[0]
    dev = ctx.device
    t = torch.arange(T, device=dev)
    live = t < q_start[S]
    of = torch.searchsorted(q_start[1:], t, right=True).clamp(max=S - 1)
    old = ctx - (q_start[1:] - q_start[:-1])  # tokens held before
    pos = old[of] + t - q_start[of]
    block = torch.where(live, tables[of, (pos // bs).clamp(0, tables.shape[1] - 1)], nb)
    offset = pos % bs
    first = tables.gather(1, (old // bs)[:, None])[:, 0]  # each sequence's first block that is written
    kept = torch.arange(bs, device=dev)[None, :] < (old % bs)[:, None]  # its rows that stay
    out = []
    for x, cache, scale in ((st["key"], st["k_cache"], st["k_scale"]), (st["value"], st["v_cache"], st["v_scale"])):
        x = x.float()
        amax = torch.zeros((nb + 1, H), device=dev).scatter_reduce(0, block[:, None].expand(T, H), x.abs().amax(2), "amax")
        s = amax / torch.full((), 127.0, device=dev)  # a tensor: division by a number would multiply by its reciprocal
        s = torch.where(s < torch.finfo(torch.float32).tiny, 0.0, s)
        was = torch.where((old % bs > 0)[:, None], scale[first], 0.0)  # [S, H]
        now = torch.maximum(was, s[first])
        s[first] = now
        ratio = torch.where(now > 0, was / now, 0.0)
        held = cache[first]
        moved = torch.round(held.float() * ratio[:, :, None, None]).to(torch.int8)
        cache[first] = torch.where(kept[:, None, :, None], moved, held)
        inv = torch.where(s > 0, 1.0 / s, 0.0)
        code = torch.round(x * inv[block][:, :, None]).clamp(-127, 127).to(torch.int8)
        place = torch.where(live, block * bs + offset, nb * bs)
        rows = torch.cat([cache.permute(0, 2, 1, 3).reshape(nb * bs, H, D), cache.new_zeros((1, H, D))])
        rows = rows.index_copy(0, place, code)[:nb * bs]
        cache.copy_(rows.view(nb, bs, H, D).permute(0, 2, 1, 3))
        touched = torch.zeros(nb + 1, dtype=torch.bool, device=dev).index_fill(0, block, True)[:nb]
        scale.copy_(torch.where(touched[:, None], s[:nb], scale))
        out += [cache, scale]
    return out


def _plain_decode(st):
    c = st["case"]
    S, H, D, bs = c["seqs"], c["kv_heads"], c["head_dim"], c["block_size"]
    G = c["heads"] // H
    ids = st["tables"].long().clamp(min=0)
    L = ids.shape[1] * bs
    k = (st["k_cache"][ids] * st["k_scale"][ids][..., None, None]).transpose(1, 2).reshape(S, H, L, D)
    x = (st["q"].float().view(S, H, G, D) * st["scale"]) @ k.transpose(2, 3)
    del k
    past = torch.arange(L, device=x.device)[None, :] >= st["ctx"][:, None]
    x = x.masked_fill(past[:, None, None, :], float("-inf"))
    p = torch.exp(x - x.amax(3, keepdim=True))
    v = (st["v_cache"][ids] * st["v_scale"][ids][..., None, None]).transpose(1, 2).reshape(S, H, L, D)
    o = (p @ v) / p.sum(3, keepdim=True)
    return o.view(S, c["heads"], D).to(DTYPES[c["out"]])


# ---------------------------------------------------------------------- run

def run(state):
    st, op = state, state["case"]["op"]
    if op in ("append", "release"):
        st["arena"].copy_(st["start"])
    if own:
        import paged_kv_cache_340_b200 as pa
        if op == "append":
            pa.pa_dpool_append(st["pool"], st["tables"], st["ctx"], st["new"], st["q_start"], st["slots"], st["pairs"],
                               st["num_cow"])
            return {k: st[k] for k in ("tables", "ctx", "q_start", "slots", "pairs", "num_cow", "header", "ref", "ring")}
        if op == "release":
            pa.pa_dpool_release(st["pool"], st["tables"], st["ctx"], st["finished"])
            return {k: st[k] for k in ("tables", "ctx", "header", "ref", "ring")}
        if op == "write":
            pa.pa_append_q8b(st["key"], st["value"], st["q_start"], st["k_cache"], st["v_cache"], st["k_scale"],
                             st["v_scale"], st["tables"], st["ctx"])
            return [st["k_cache"], st["k_scale"], st["v_cache"], st["v_scale"]]
        pa.pa_decode_q8b(st["out"], st["q"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], st["tables"],
                         st["ctx"], st["scale"], st["max_ctx"], st["workspace"], seq_order=st["order"])
        return st["out"]
    return {"append": _plain_append, "release": _plain_release, "write": _plain_write, "decode": _plain_decode}[op](st)


# -------------------------------------------------------------------- exact

def _exact_append(c, seed):
    """Sequence by sequence and token by token, from the definition."""
    h = _pool_start(c, seed)
    bs, nb, tables, ctx, ref = c["block_size"], h["nb"], h["tables"], h["ctx"], h["ref"]
    free = h["free"].tolist()
    ring = np.full(nb, -1, np.int32)
    ring[:len(free)] = h["free"]
    n0, head, slots, pairs, q_start = len(free), 0, [], [], [0]

    def take():
        nonlocal head
        if c["policy"] == LIFO:
            return free.pop()
        head += 1
        return free[head - 1]

    for s in range(c["seqs"]):
        for _ in range(int(h["new"][s])):
            j, o = divmod(int(ctx[s]), bs)
            if o == 0:
                tables[s, j] = take()
                ref[tables[s, j]] = 1
            elif ref[tables[s, j]] > 1:
                was, got = int(tables[s, j]), take()
                ref[was] -= 1
                ref[got] = 1
                tables[s, j] = got
                pairs.append((was, got))
            slots.append(int(tables[s, j]) * bs + o)
            ctx[s] += 1
        q_start.append(len(slots))
    left = len(free) if c["policy"] == LIFO else n0 - head
    n = len(pairs)
    all_pairs = np.full((c["seqs"], 2), -1, np.int64)
    if n:
        all_pairs[:n] = pairs
    slots += [-1] * c["pad_tokens"]
    return dict(tables=tables, ctx=ctx, q_start=np.array(q_start, np.int32), slots=np.array(slots, np.int32), pairs=all_pairs,
                num_cow=np.array([n], np.int32), header=np.array([nb, bs, c["policy"], head % nb, left], np.int32), ref=ref,
                ring=ring)


def _exact_release(c, seed):
    h = _pool_start(c, seed)
    bs, nb, tables, ctx, ref = c["block_size"], h["nb"], h["tables"], h["ctx"], h["ref"]
    ring = np.full(nb, -1, np.int32)
    count = h["free"].size
    ring[:count] = h["free"]
    for s in range(c["seqs"]):
        if h["fin"][s]:
            for j in range(_cdiv(int(ctx[s]), bs)):
                b = tables[s, j]
                ref[b] -= 1
                if ref[b] == 0:
                    ring[count % nb] = b
                    count += 1
                tables[s, j] = -1
            ctx[s] = 0
    return dict(tables=tables, ctx=ctx, header=np.array([nb, bs, c["policy"], 0, count], np.int32), ref=ref, ring=ring)


def _exact_write(c, seed):
    """The scales, block by block in 64 bits; the codes, whole numbers, have no value in 64 bits of their own."""
    st = prepare(c, seed)
    q0, ctx, tables = (st[k].cpu().numpy().astype(np.int64) for k in ("q_start", "ctx", "tables"))
    bs, out = c["block_size"], []
    for x, scale in ((st["key"], st["k_scale"]), (st["value"], st["v_scale"])):
        row = x.double().abs().amax(2).cpu().numpy()
        res = scale.double().cpu().numpy()
        for s in range(c["seqs"]):
            n = int(q0[s + 1] - q0[s])
            p0 = int(ctx[s]) - n
            for j in range(p0 // bs, _cdiv(p0 + n, bs)):
                a, e = max(p0, j * bs), min(p0 + n, (j + 1) * bs)
                top = row[q0[s] + a - p0:q0[s] + e - p0].max(0) / 127
                b = tables[s, j]
                res[b] = np.maximum(top, res[b]) if a > j * bs else top
        out += [None, res]
    return out


def _exact_decode(c, seed):
    st = prepare(c, seed)
    H, D, bs = c["kv_heads"], c["head_dim"], c["block_size"]
    G = c["heads"] // H
    out = torch.zeros((c["seqs"], H, G, D), dtype=torch.float64, device="cuda")
    lens = st["ctx"].tolist()
    q = st["q"].double().view(c["seqs"], H, G, D)
    for s, n in enumerate(lens):
        ids = st["tables"][s, :_cdiv(n, bs)].long()

        def rows(codes, scale):
            x = codes[ids].double() * scale[ids].double()[:, :, None, None]
            return x.permute(1, 0, 2, 3).reshape(H, -1, D)[:, :n]

        w = torch.softmax(torch.einsum("hgd,htd->hgt", q[s], rows(st["k_cache"], st["k_scale"])) / D ** 0.5, -1)
        out[s] = torch.einsum("hgt,htd->hgd", w, rows(st["v_cache"], st["v_scale"]))
    return out.view(c["seqs"], c["heads"], D)


def exact(case, seed):
    return {"append": _exact_append, "release": _exact_release, "write": _exact_write, "decode": _exact_decode}[case["op"]](
        case, seed)
