"""pa_dpool_append and pa_dpool_release on the GPU: tables, lengths, slots,
query starts, copy pairs and the pool's whole state must equal, number for
number, those of the host pool's pa_pool_append / pa_pool_release called
sequence by sequence (the host pool itself is checked against the oracle's)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_340_b200 import _build
    _build.build()
    import paged_kv_cache_340_b200 as pa
    return pa


class Both:
    """The same pool and sequences on the host and on the device."""

    def __init__(self, pa, S, MB, NB, bs, policy, seed, forks=()):
        self.pa, self.S, self.MB, self.bs = pa, S, MB, bs
        rng = np.random.default_rng(seed)
        self.host = pa.BlockPool(NB, bs, policy, free_order=rng.permutation(NB))
        self.tables = np.full((S, MB), -1, np.int32)
        self.ctx = np.zeros(S, np.int32)
        for src, dst, n in forks:  # sequence dst starts as a fork of src, which holds n tokens
            if self.ctx[src] == 0:
                self.ctx[src], _, _ = self.host.append(self.tables[src], 0, n)
            self.host.fork(self.tables[src], n, self.tables[dst])
            self.ctx[dst] = n
        self.pool = pa.DevicePool(NB, bs, policy, host_pool=self.host)
        self.d_tables, self.d_ctx = torch.from_numpy(self.tables).cuda(), torch.from_numpy(self.ctx).cuda()

    def append(self, new, pad=0, stream=None):
        """The host's result, checked against the device's; returns the device's outputs."""
        S = self.S
        slots, pairs = [], []
        for s in range(S):
            n, sl, cow = self.host.append(self.tables[s], int(self.ctx[s]), int(new[s]))
            self.ctx[s] = n
            slots += sl.tolist()
            pairs += cow.tolist()
        T = len(slots)
        out = self.call(new, T + pad, stream)
        q_start, d_slots, d_pairs, num_cow = (t.cpu().numpy() for t in out)
        assert self.pa.pa_read_device_errors() == 0
        assert q_start.tolist() == [0] + np.cumsum(new).tolist()
        assert d_slots.tolist() == slots + [-1] * pad
        assert num_cow.tolist() == [len(pairs)]
        assert d_pairs.tolist() == pairs + [[-1, -1]] * (S - len(pairs))
        self.same()
        return out

    def call(self, new, max_tokens, stream=None, pool=None):
        i32 = dict(dtype=torch.int32, device="cuda")
        out = (torch.full((self.S + 1,), 7, **i32), torch.full((max_tokens,), 7, **i32),
               torch.full((self.S, 2), 7, dtype=torch.int64, device="cuda"), torch.full((1,), 7, **i32))
        self.pa.pa_dpool_append(pool or self.pool, self.d_tables, self.d_ctx, torch.tensor(new, **i32), *out, stream=stream)
        return out

    def release(self, finished):
        for s in range(self.S):
            if finished[s]:
                self.host.release(self.tables[s], int(self.ctx[s]))
                self.tables[s, :-(-int(self.ctx[s]) // self.bs)] = -1
                self.ctx[s] = 0
        self.pa.pa_dpool_release(self.pool, self.d_tables, self.d_ctx, torch.tensor(finished, dtype=torch.int32, device="cuda"))
        assert self.pa.pa_read_device_errors() == 0
        self.same()

    def same(self):
        assert np.array_equal(self.d_tables.cpu().numpy(), self.tables)
        assert np.array_equal(self.d_ctx.cpu().numpy(), self.ctx)
        ref, free = self.host.export()
        assert np.array_equal(self.pool.ref.cpu().numpy(), ref)
        assert self.pool.free_list() == free.tolist()
        self.scratch_clean()

    def scratch_clean(self):
        nb = self.pool.num_blocks
        scratch = self.pool.state[8 + 2 * nb:8 + 6 * nb].view(4, nb).cpu()
        assert (scratch[0] == 0).all() and (scratch[1] == -1).all()
        assert (scratch[2] == 0).all() and (scratch[3] == -1).all()


@pytest.mark.parametrize("policy", ["LIFO", "FIFO"])
@pytest.mark.parametrize("S,bs,MB", [(1, 16, 8), (5, 4, 40), (33, 16, 24), (130, 32, 9)])
def test_random_steps_equal_the_host_pool(pa, policy, S, bs, MB):
    rng = np.random.default_rng(S * 7 + bs)
    forks = [(0, i, 3 * bs + 5) for i in range(1, min(S, 4))] + [(i, i + 1, 2 * bs) for i in range(6, S - 1, 9)] + \
            [(i, i + 1, bs + 1) for i in range(10, S - 1, 9)]
    NB = S * MB // 2 + 8
    b = Both(pa, S, MB, NB, bs, getattr(pa, "PA_POOL_" + policy), 3, forks)
    for step in range(14):
        hi = [1, bs, 2 * bs + 3][step % 3]
        new = rng.integers(0, hi + 1, S)
        room = np.minimum(new, MB * bs - b.ctx)
        takes = sum(-(-int(c + n) // bs) - -(-int(c) // bs) + 1 for c, n in zip(b.ctx, room))
        if takes <= b.host.num_free():
            b.append(room, pad=step % 2 * 3)
        fin = rng.random(S) < (0.3 if b.host.num_free() > NB // 3 else 0.8)
        b.release(fin)
    b.release(np.ones(S, int))
    assert b.host.num_free() == NB


def test_many_sequences_and_tokens(pa):
    """More sequences than threads of a block (several to a thread), tables
    longer than an item of the release, more tokens than threads."""
    S, bs = 2500, 16
    rng = np.random.default_rng(9)
    b = Both(pa, S, 70, 60000, bs, pa.PA_POOL_FIFO, 4, [(i, i + 1, 37) for i in range(0, S - 1, 7)])
    new = rng.integers(0, 40, S)
    new[[3, 1000, 2499]] = [1000, 0, 1025]
    b.append(new, pad=11)
    b.release(rng.random(S) < 0.5)
    b.append(rng.integers(0, 3, S))
    b.release(np.ones(S, int))


def test_largest_batch(pa):
    S = pa.PA_DPOOL_MAX_SEQS
    b = Both(pa, S, 3, 2 * S, 16, pa.PA_POOL_LIFO, 5)
    b.append(np.arange(S) % 20)
    b.release(np.arange(S) % 3 == 0)


@pytest.mark.parametrize("extra", [0, 1])
def test_shared_last_block(pa, extra):
    """Four sequences share a partly filled block. All four append: three copy
    it, the last one in order keeps it. With a holder that does not append,
    all that append copy it."""
    b = Both(pa, 5 + extra, 6, 40, 16, pa.PA_POOL_FIFO, 6, [(1, j, 20) for j in (0, 2, 4, 5)[:3 + extra]])
    new = np.array([1, 2, 1, 0, 30, 0][:5 + extra])
    out = b.append(new)
    assert int(out[3]) == (4 if extra else 3)


def test_free_list_used_up_exactly_and_wrapped(pa):
    for policy in (pa.PA_POOL_FIFO, pa.PA_POOL_LIFO):
        b = Both(pa, 3, 8, 6, 4, policy, 7)
        for _ in range(5):
            b.append(np.array([8, 5, 7]))
            b.release(np.array([0, 1, 1]))
            b.append(np.array([0, 4, 8]))
            b.release(np.array([1, 1, 1]))


def test_empty_calls(pa):
    b = Both(pa, 4, 4, 10, 16, pa.PA_POOL_FIFO, 8)
    b.append(np.zeros(4, int), pad=3)
    b.append(np.zeros(4, int))
    b.release(np.zeros(4, int))
    e = Both(pa, 0, 4, 10, 16, pa.PA_POOL_FIFO, 8)
    e.append(np.zeros(0, int), pad=2)
    e.release(np.zeros(0, int))


@pytest.mark.parametrize("what,bit", [("blocks", 0x20), ("row", 0x20), ("tokens", 0x20), ("negative", 0x4),
                                      ("context", 0x4), ("block id", 0x1), ("state", 0x20), ("free block", 0x20)])
def test_append_errors_apply_nothing(pa, what, bit):
    b = Both(pa, 3, 4, 9, 16, pa.PA_POOL_FIFO, 9, [(0, 1, 20)])
    new, max_tokens, pool = [4, 4, 4], 40, None
    if what == "blocks":
        new, max_tokens = [40, 40, 64], 200
    elif what == "row":
        new, max_tokens = [4, 4, 65], 200
    elif what == "tokens":
        max_tokens = 11
    elif what == "negative":
        new = [4, -1, 4]
    elif what == "context":
        b.d_ctx[2] = 65
    elif what == "block id":
        b.d_tables[1, 1] = 9
    elif what == "state":  # a state of other sizes
        pool = pa.DevicePool(9, 32, pa.PA_POOL_FIFO)
    elif what == "free block":
        b.d_tables[0, 1] = b.pool.free_list()[0]
    before = [t.clone() for t in (b.pool.state, b.d_tables, b.d_ctx)]
    q_start, slots, pairs, num_cow = b.call(new, max_tokens, pool=pool)
    assert pa.pa_read_device_errors() == bit
    for t, w in zip((b.pool.state, b.d_tables, b.d_ctx), before):
        assert torch.equal(t, w)
    assert (q_start == 0).all() and (slots == -1).all() and (pairs == -1).all() and int(num_cow) == 0
    b.scratch_clean()


@pytest.mark.parametrize("what,bit", [("context", 0x4), ("block id", 0x1), ("state", 0x20), ("twice", 0x20)])
def test_release_errors_apply_nothing(pa, what, bit):
    b = Both(pa, 3, 4, 12, 16, pa.PA_POOL_FIFO, 10, [(0, 1, 40)])
    pool = b.pool
    if what == "context":
        b.d_ctx[1] = -1
    elif what == "block id":
        b.d_tables[1, 2] = -5
    elif what == "state":
        pool = pa.DevicePool(12, 32, pa.PA_POOL_FIFO)
    elif what == "twice":  # a third holder of blocks whose count is two
        b.d_tables[2] = b.d_tables[0]
        b.d_ctx[2] = 40
    before = [t.clone() for t in (b.pool.state, b.d_tables, b.d_ctx)]
    pa.pa_dpool_release(pool, b.d_tables, b.d_ctx, torch.ones(3, dtype=torch.int32, device="cuda"))
    assert pa.pa_read_device_errors() == bit
    for t, w in zip((b.pool.state, b.d_tables, b.d_ctx), before):
        assert torch.equal(t, w)
    b.scratch_clean()


def test_beam_step_after_append(pa):
    """The beam step and the new calls share a state: each leaves it as the other expects."""
    from paged_kv_cache_340_b200.batch import host_beam_step
    rng = np.random.default_rng(12)
    W, bs, MB = 6, 4, 30
    b = Both(pa, W, MB, 200, bs, pa.PA_POOL_FIFO, 11, [(0, j, 9) for j in range(1, W)])
    for _ in range(4):
        b.append(rng.integers(0, 6, W))
        parents = rng.integers(0, W, W).astype(np.int32)
        b.tables, b.ctx, _, _ = host_beam_step(b.host, b.tables, b.ctx, parents)
        nt, nc = torch.empty_like(b.d_tables), torch.empty_like(b.d_ctx)
        i32 = dict(dtype=torch.int32, device="cuda")
        pa.pa_beam_step(b.pool, b.d_tables, b.d_ctx, torch.from_numpy(parents).cuda(), nt, nc, torch.empty(W, **i32),
                        torch.empty((W, 2), dtype=torch.int64, device="cuda"), torch.empty(1, **i32))
        b.d_tables, b.d_ctx = nt, nc
        b.same()
    b.release(np.array([1, 0, 1, 0, 0, 1]))


def test_on_a_side_stream(pa):
    b = Both(pa, 9, 8, 60, 16, pa.PA_POOL_LIFO, 13, [(2, 5, 18)])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        b.append(np.arange(9), stream=st)
        b.release(np.arange(9) % 2)


def test_release_of_many_entries(pa):
    """More table entries than the warps hold at once (each pass reads them
    again), shared and single blocks mixed; then the same refused."""
    S, bs, MB = 40, 4, 3000
    b = Both(pa, S, MB, 130000, bs, pa.PA_POOL_FIFO, 14, [(0, j, 9001) for j in (1, 2, 5)] + [(7, 8, 11990)])
    rng = np.random.default_rng(15)
    new = rng.integers(8000, 12001, S)
    new = np.minimum(new, MB * bs - b.ctx)
    b.append(new, pad=1)
    for bad_at in ((30, 1500), (3, 7)):
        keep = int(b.d_tables[bad_at])
        for value, bit in ((130000, 0x1), (int(b.d_tables[0, 0]), 0x20), (int(b.d_tables[20, 5]), 0x20),
                           (int(b.pool.free_list()[3]), 0x20)):
            b.d_tables[bad_at] = value  # out of range; one drop too many of a shared block, of a single one; a free one
            before = [t.clone() for t in (b.pool.state, b.d_tables, b.d_ctx)]
            pa.pa_dpool_release(b.pool, b.d_tables, b.d_ctx, torch.ones(S, dtype=torch.int32, device="cuda"))
            assert pa.pa_read_device_errors() == bit
            for t, w in zip((b.pool.state, b.d_tables, b.d_ctx), before):
                assert torch.equal(t, w)
        b.d_tables[bad_at] = keep
    b.release(rng.random(S) < 0.5)
    b.release(np.ones(S, int))
    assert b.host.num_free() == 130000


@pytest.mark.parametrize("S,pad", [(1000, 0), (1000, 9000), (1024, 5), (1025, 5)])
def test_shared_blocks_of_many_writers(pa, S, pad):
    """Every sequence is a fork of some other, in groups of one to nine; all of
    a group write into its last block, or all but some. Few slots and many,
    and on both sides of where a thread holds one sequence."""
    rng = np.random.default_rng(S + pad)
    forks, at = [], 0
    while at < S:
        n = int(rng.integers(1, 10))
        forks += [(at, j, 5 + at % 40) for j in range(at + 1, min(S, at + n))]
        at += n
    b = Both(pa, S, 8, 9 * S, 16, pa.PA_POOL_FIFO, 16, forks)
    b.append((rng.random(S) < 0.9).astype(int), pad=pad)
    b.append(rng.integers(0, 4, S), pad=pad)
    b.release(rng.random(S) < 0.5)
    b.append(rng.integers(0, 20, S), pad=pad)


@pytest.mark.parametrize("S,MB", [(5, 6), (400, 6)])
def test_release_of_a_block_listed_twice_or_free_changes_nothing(pa, S, MB):
    """Blocks of one holder each, so that each is claimed at once: one that a
    second entry lists too, and one that is free already."""
    b = Both(pa, S, MB, 3 * S + 5, 16, pa.PA_POOL_LIFO, 17)
    b.append(np.full(S, 33))
    keep = int(b.d_tables[S - 2, 1])
    for value in (int(b.d_tables[0, 2]), b.pool.free_list()[1]):
        b.d_tables[S - 2, 1] = value
        before = [t.clone() for t in (b.pool.state, b.d_tables, b.d_ctx)]
        pa.pa_dpool_release(b.pool, b.d_tables, b.d_ctx, torch.ones(S, dtype=torch.int32, device="cuda"))
        assert pa.pa_read_device_errors() == 0x20
        for t, w in zip((b.pool.state, b.d_tables, b.d_ctx), before):
            assert torch.equal(t, w)
    b.d_tables[S - 2, 1] = keep
    b.release(np.ones(S, int))


def test_binding_refuses_wrong_types_and_shapes(pa):
    b = Both(pa, 3, 4, 20, 16, pa.PA_POOL_FIFO, 18)
    i32 = dict(dtype=torch.int32, device="cuda")
    good = [b.d_tables, b.d_ctx, torch.ones(3, **i32), torch.empty(4, **i32), torch.empty(9, **i32),
            torch.empty((3, 2), dtype=torch.int64, device="cuda"), torch.empty(1, **i32)]
    before = [t.clone() for t in (b.pool.state, b.d_tables, b.d_ctx)]
    for i, bad in ((0, b.d_tables.t()), (0, b.d_ctx), (1, b.d_ctx[:2]), (1, b.d_ctx.long()), (2, torch.ones(3, dtype=torch.int32)),
                   (3, torch.empty(3, **i32)), (4, torch.empty((3, 3), **i32)), (4, torch.empty(18, **i32)[::2]),
                   (5, torch.empty((3, 2), **i32)), (5, torch.empty((2, 2), dtype=torch.int64, device="cuda")),
                   (6, torch.empty(0, **i32))):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError):
            pa.pa_dpool_append(b.pool, *args)
    with pytest.raises(TypeError):
        pa.pa_dpool_append(b.pool, *good[:2], [1, 1, 1], *good[3:])
    with pytest.raises(ValueError):
        pa.pa_dpool_release(b.pool, b.d_tables, b.d_ctx, torch.ones(3, dtype=torch.bool, device="cuda"))
    with pytest.raises(AttributeError):
        pa.pa_dpool_append(b.pool, *good, stream="0")
    torch.cuda.synchronize()
    assert all(torch.equal(t, w) for t, w in zip((b.pool.state, b.d_tables, b.d_ctx), before))
    assert pa.pa_read_device_errors() == 0


@pytest.mark.parametrize("bs", [1, 3, 24, 48])
def test_block_sizes_of_every_kind(pa, bs):
    rng = np.random.default_rng(bs)
    b = Both(pa, 40, 60, 3000, bs, pa.PA_POOL_FIFO, 19, [(i, i + 1, bs + 1) for i in range(0, 40, 5)])
    for hi in (1, 2 * bs, 7):
        b.append(np.minimum(rng.integers(0, hi + 1, 40), 60 * bs - b.ctx), pad=2)
    b.release(rng.random(40) < 0.5)
    b.append(np.minimum(rng.integers(0, 20 * bs, 40), 60 * bs - b.ctx))
    b.release(np.ones(40, int))
