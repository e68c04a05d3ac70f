"""The serving step's calls together, as an engine makes them: pool release and
append, copy-on-write copies, quantizing write and decode on one stream, with
nothing read back between them. Checked against the host pool, the write's
definition in numpy and the oracle's attention in double precision."""
import numpy as np
import pytest
import torch

import oracle
from _helpers import f64
from test_gpu_q8b import Case, write_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_340_b200 import _build
    _build.build()
    import paged_kv_cache_340_b200 as pa
    return pa


class Reference:
    """The same steps on the host."""

    def __init__(self, pa, S, MB, NB, bs, Hq, Hkv, D):
        self.pool = pa.BlockPool(NB, bs, pa.PA_POOL_FIFO)
        self.tables, self.ctx = np.full((S, MB), -1, np.int32), np.zeros(S, np.int32)
        self.codes = [np.zeros((NB, Hkv, bs, D), np.int8) for _ in range(2)]
        self.scales = [np.zeros((NB, Hkv), np.float32) for _ in range(2)]
        self.bs, self.Hq, self.Hkv, self.D = bs, Hq, Hkv, D

    def step(self, new, fin, key, value):
        for s in np.nonzero(fin)[0]:
            self.pool.release(self.tables[s], int(self.ctx[s]))
            self.tables[s, :-(-int(self.ctx[s]) // self.bs)] = -1
            self.ctx[s] = 0
        for s, n in enumerate(new):
            self.ctx[s], _, cow = self.pool.append(self.tables[s], int(self.ctx[s]), int(n))
            for a, b in cow:
                for x in self.codes + self.scales:
                    x[b] = x[a]
        q_start = np.concatenate([[0], np.cumsum(new)])
        for codes, scale, x in zip(self.codes, self.scales, (key, value)):
            write_rows(codes, scale, x.float().numpy(), q_start, self.tables, self.ctx, self.bs)

    def check_out(self, out, q, scale):
        c = Case.__new__(Case)
        c.ctx, c.bs, c.D, c.Hq, c.Hkv, c.tables, c.scale = self.ctx, self.bs, self.D, self.Hq, self.Hkv, self.tables, scale
        (c.kq, c.vq), (c.ks, c.vs), c.q = self.codes, self.scales, q.float()
        c.check(out, q.dtype)


def drive(pa, sv, ref, S, T, rng, steps, run, reset=None):
    """Random steps: prompts into empty rows, single tokens into others, some rows finished."""
    Hq, Hkv, D = ref.Hq, ref.Hkv, ref.D
    gen = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
    for step in range(steps):
        fin = (rng.random(S) < 0.15) & (ref.ctx > 0)
        held = np.where(fin, 0, ref.ctx)
        new = np.where(held == 0, rng.integers(0, 40, S), rng.integers(0, 2, S))
        new = np.minimum(new, sv.max_context_len - held)
        while new.sum() > T:
            new[rng.integers(S)] = 0
        key, value = (torch.randn((T, Hkv, D), generator=gen).to(sv.out.dtype) for _ in range(2))
        q = torch.randn((S, Hq, D), generator=gen).to(sv.out.dtype)
        out = run(new, fin, key, value, q)
        ref.step(new, fin, key, value)
        torch.cuda.synchronize()
        assert pa.pa_read_device_errors() == 0
        assert np.array_equal(sv.block_tables.cpu().numpy(), ref.tables)
        assert np.array_equal(sv.context_lens.cpu().numpy(), ref.ctx)
        for got, want in zip(sv.cache(), ref.codes + ref.scales):
            assert np.array_equal(got.cpu().numpy(), want)
        ref.check_out(out, q, sv.scale)


def dev(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("bs,Hq,Hkv,D", [(16, 8, 2, 128), (32, 4, 4, 64)])
def test_steps_equal_the_host(pa, bs, Hq, Hkv, D):
    from paged_kv_cache_340_b200.batch import ServingStep
    S, MB, NB, T = 12, 6, 80, 300
    sv = ServingStep(S, MB, NB, bs, Hq, Hkv, D, T, dtype=torch.float16)
    ref = Reference(pa, S, MB, NB, bs, Hq, Hkv, D)
    drive(pa, sv, ref, S, T, np.random.default_rng(bs), 12,
          lambda new, fin, k, v, q: sv.step(dev(new), dev(fin), k.cuda(), v.cuda(), q.cuda()))


def test_captured_step_replayed(pa):
    """One captured step, replayed with new contents in its input buffers."""
    from paged_kv_cache_340_b200.batch import ServingStep
    S, MB, NB, T, bs, Hq, Hkv, D = 9, 8, 70, 200, 16, 8, 2, 128
    sv = ServingStep(S, MB, NB, bs, Hq, Hkv, D, T)
    ref = Reference(pa, S, MB, NB, bs, Hq, Hkv, D)
    new, fin = dev(np.zeros(S)), dev(np.zeros(S))
    key, value = (torch.zeros((T, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros((S, Hq, D), dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        sv.step(new, fin, key, value, q)   # an empty step first: everything is loaded
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = sv.step(new, fin, key, value, q)

    def run(n, f, k, v, qq):
        for a, b in ((new, dev(n)), (fin, dev(f)), (key, k), (value, v), (q, qq)):
            a.copy_(b)
        g.replay()
        return out

    drive(pa, sv, ref, S, T, np.random.default_rng(5), 8, run)


def test_two_engines_on_two_streams(pa):
    """Two engines' steps in flight at the same time, each with its own buffers."""
    from paged_kv_cache_340_b200.batch import ServingStep
    S, MB, NB, T, bs, Hq, Hkv, D = 5, 40, 150, 700, 16, 4, 2, 64
    rng = np.random.default_rng(6)
    sides = []
    for i in range(2):
        sv, ref = ServingStep(S, MB, NB, bs, Hq, Hkv, D, T, dtype=torch.float16), Reference(pa, S, MB, NB, bs, Hq, Hkv, D)
        sides.append((sv, ref, torch.cuda.Stream()))
    torch.cuda.synchronize()
    gen = torch.Generator().manual_seed(7)
    outs = []
    for step in range(4):
        todo = []
        for sv, ref, st in sides:
            new = rng.integers(0, 130, S) if step == 0 else rng.integers(0, 3, S)
            k, v = (torch.randn((T, Hkv, D), generator=gen).half() for _ in range(2))
            q = torch.randn((S, Hq, D), generator=gen).half()
            todo.append((sv, ref, st, new, k, v, q, [dev(new), dev(np.zeros(S)), k.cuda(), v.cuda(), q.cuda()]))
        torch.cuda.synchronize()
        for sv, ref, st, *_, args in todo:
            sv.step(*args, stream=st)
        torch.cuda.synchronize()
        for sv, ref, st, new, k, v, q, _ in todo:
            ref.step(new, np.zeros(S, bool), k, v)
            ref.check_out(sv.out, q, sv.scale)
            for got, want in zip(sv.cache(), ref.codes + ref.scales):
                assert np.array_equal(got.cpu().numpy(), want)
    assert pa.pa_read_device_errors() == 0


def test_step_without_room_changes_nothing(pa):
    from paged_kv_cache_340_b200.batch import ServingStep
    S, MB, NB, T, bs, Hq, Hkv, D = 3, 8, 6, 100, 16, 2, 1, 128
    sv = ServingStep(S, MB, NB, bs, Hq, Hkv, D, T, dtype=torch.float16)
    k, v = (torch.randn((T, Hkv, D)).half().cuda() for _ in range(2))
    q = torch.randn((S, Hq, D)).half().cuda()
    none = dev(np.zeros(S))
    a = sv.step(dev([20, 30, 5]), none, k, v, q).clone()
    before = [t.clone() for t in (sv.pool.state, sv.block_tables, sv.context_lens, *sv.cache())]
    out = sv.step(dev([20, 20, 20]), none, k, v, q)
    assert pa.pa_read_device_errors() == 0x20
    assert all(torch.equal(x, y) for x, y in zip(before, (sv.pool.state, sv.block_tables, sv.context_lens, *sv.cache())))
    assert torch.equal(a, out)


def test_copy_on_write_of_forked_sequences(pa):
    """Forks of one prompt (made on the host) append into their shared block."""
    from paged_kv_cache_340_b200.batch import ServingStep
    S, MB, NB, T, bs, Hq, Hkv, D = 4, 6, 40, 50, 16, 4, 2, 128
    ref = Reference(pa, S, MB, NB, bs, Hq, Hkv, D)
    gen = torch.Generator().manual_seed(8)
    k, v = (torch.randn((37, Hkv, D), generator=gen).half() for _ in range(2))
    ref.step([37, 0, 0, 0], np.zeros(S, bool), k, v)
    for s in (1, 2):
        ref.pool.fork(ref.tables[0], 37, ref.tables[s])
        ref.ctx[s] = 37
    sv = ServingStep(S, MB, NB, bs, Hq, Hkv, D, T, dtype=torch.float16,
                     pool=pa.DevicePool(NB, bs, pa.PA_POOL_FIFO, host_pool=ref.pool))
    sv.block_tables.copy_(torch.from_numpy(ref.tables))
    sv.context_lens.copy_(torch.from_numpy(ref.ctx))
    for got, x in zip(sv.cache(), ref.codes + ref.scales):
        got.copy_(torch.from_numpy(x))
    drive(pa, sv, ref, S, T, np.random.default_rng(9), 6,
          lambda new, fin, kk, vv, q: sv.step(dev(new), dev(fin), kk.cuda(), vv.cuda(), q.cuda()))


def test_tables_and_slots_serve_a_16_bit_cache(pa):
    """The append's slots (padding included), q_start, tables and pairs with
    the 16-bit slot write, counted block copy and prefill."""
    S, MB, NB, bs, Hq, Hkv, D, T = 3, 6, 30, 16, 4, 2, 128, 90
    pool = pa.DevicePool(NB, bs, pa.PA_POOL_LIFO)
    i32 = dict(dtype=torch.int32, device="cuda")
    tables, ctx = torch.full((S, MB), -1, **i32), torch.zeros(S, **i32)
    q_start, slots, num = torch.empty(S + 1, **i32), torch.empty(T, **i32), torch.empty(1, **i32)
    pairs = torch.empty((S, 2), dtype=torch.int64, device="cuda")
    kc, vc = (torch.zeros((NB, Hkv, bs, D), dtype=torch.float16, device="cuda") for _ in range(2))
    gen = torch.Generator().manual_seed(10)
    for new in ([30, 0, 41], [3, 17, 20]):
        k, v = (torch.randn((T, Hkv, D), generator=gen).half().cuda() for _ in range(2))
        q = torch.randn((T, Hq, D), generator=gen).half().cuda()
        out = torch.zeros((T, Hq, D), device="cuda")
        pa.pa_dpool_append(pool, tables, ctx, dev(new), q_start, slots, pairs, num)
        pa.pa_copy_blocks_counted(kc, vc, pairs, num)
        pa.pa_reshape_and_cache(k, v, kc, vc, slots)
        pa.pa_prefill(out, q, q_start, max(new), kc, vc, tables, ctx, D ** -0.5)
        torch.cuda.synchronize()
        assert pa.pa_read_device_errors() == 0
        want = oracle.paged_prefill(f64(q), q_start.cpu().numpy(), f64(kc), f64(vc), tables.cpu().numpy(), ctx.cpu().numpy(),
                                    D ** -0.5, bs)
        n = sum(new)
        # the acceptance bound of the prefill tests (fp16, fp32 output)
        assert np.abs(f64(out)[:n] - want[:n]).max() <= 4e-3
        assert (out[n:] == 0).all()


def test_layers_share_the_step(pa):
    """Two layers over one block table: forks' copies reach every layer's cache,
    each layer's write and attention only its own."""
    from paged_kv_cache_340_b200.batch import ServingStep
    S, MB, NB, T, bs, Hq, Hkv, D = 4, 6, 40, 60, 16, 4, 2, 64
    gen = torch.Generator().manual_seed(11)
    refs = [Reference(pa, S, MB, NB, bs, Hq, Hkv, D) for _ in range(2)]

    def rows(*shape):
        return [torch.randn(shape, generator=gen).half() for _ in refs]

    for ref, k, v in zip(refs, rows(21, Hkv, D), rows(21, Hkv, D)):
        ref.step([21, 0, 0, 0], np.zeros(S, bool), k, v)
        ref.pool.fork(ref.tables[0], 21, ref.tables[1])
        ref.ctx[1] = 21
    sv = ServingStep(S, MB, NB, bs, Hq, Hkv, D, T, dtype=torch.float16, num_layers=2,
                     pool=pa.DevicePool(NB, bs, pa.PA_POOL_FIFO, host_pool=refs[0].pool))
    sv.block_tables.copy_(torch.from_numpy(refs[0].tables))
    sv.context_lens.copy_(torch.from_numpy(refs[0].ctx))
    for i, ref in enumerate(refs):
        for got, x in zip(sv.cache(i), ref.codes + ref.scales):
            got.copy_(torch.from_numpy(x))
    for new in ([1, 1, 30, 0], [1, 0, 1, 5], [2, 14, 0, 1]):
        k, v, q = rows(T, Hkv, D), rows(T, Hkv, D), rows(S, Hq, D)
        sv.schedule(dev(new), dev(np.zeros(S)))
        outs = [sv.attend(k[i].cuda(), v[i].cuda(), q[i].cuda(), layer=i).clone() for i in range(2)]
        torch.cuda.synchronize()
        for i, ref in enumerate(refs):
            ref.step(new, np.zeros(S, bool), k[i], v[i])
            assert np.array_equal(sv.block_tables.cpu().numpy(), ref.tables)
            for got, want in zip(sv.cache(i), ref.codes + ref.scales):
                assert np.array_equal(got.cpu().numpy(), want)
            ref.check_out(outs[i], q[i], sv.scale)
    assert pa.pa_read_device_errors() == 0
    with pytest.raises(ValueError, match="attend for each"):
        sv.step(dev([0] * S), dev([0] * S), k[0].cuda(), v[0].cuda(), q[0].cuda())
