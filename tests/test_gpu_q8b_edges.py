"""pa_decode_q8b and pa_append_q8b where they are easily wrong: a wait that runs
out while further work has been claimed, softmaxes of one token, blocks that are
all bad."""
import math

import numpy as np
import pytest
import torch

from test_gpu_q8b import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_340_b200 import _build
    _build.build()
    import paged_kv_cache_340_b200 as pa
    return pa


@pytest.mark.parametrize("first,tile", [(100, 0), (900, 0), (900, 5)])
def test_wait_that_runs_out_among_claimed_items(pa, first, tile):
    """More items than CTAs, so the CTA whose K tile never comes has taken on
    others and may have asked for one more: it leaves after the answer, only
    those items are lost, and the calls after it are sound."""
    rng = np.random.default_rng(5)
    lens = rng.integers(1, 400, 300)
    lens[0] = first
    c = Case(3, 3, 128, 16, lens, seed=43)
    args = [c.q.half().cuda(), *[torch.from_numpy(a).cuda() for a in (c.kq, c.vq, c.ks, c.vs, c.tables, c.ctx)], c.scale,
            int(lens.max())]
    want, out = (torch.empty((300, 3, 128), device="cuda") for _ in range(2))
    pa.pa_decode_q8b(want, *args)
    for _ in range(3):
        out.fill_(float("nan"))
        pa.pa_decode_q8b_withhold_tile(out, *args, 0, 0, tile, 5_000_000)
        again = torch.empty_like(want)
        pa.pa_decode_q8b(again, *args)
        torch.cuda.synchronize()
        assert pa.pa_read_device_errors() == 0x8
        lost = (out != want).any(-1)
        assert lost[0, 0] and int(lost.sum()) <= 6  # four items are known at a time, one more is asked for
        assert torch.equal(again, want)
    assert pa.pa_read_device_errors() == 0


# A softmax of one token: out is that token's V whatever its score. Counted in units of V: its scale's logarithm (below
# 8 in magnitude, within one step of 2^-21: ln2 2^-21 relative) and two powers of two (2 steps, 2^-22 each), the weight's
# 23 bits (2^-24) and five roundings of fp32 (2^-24 each), 1.2e-6 together. The score's size is not in it. The other
# tokens, n - 1 with scores of 0, weigh exp(-target) each beside it: less than (n - 1) exp(-target) max|V| is theirs.
PEAKED = 2.0 ** -19


def peaked(D, Hq, Hkv, bs, n, at, target, seed):
    """n tokens a sequence, token `at` with a score of `target` for every head and the others with 0."""
    c = Case(Hq, Hkv, D, bs, [n] * 6, seed=seed, spread=0.2)
    G = Hq // Hkv
    sign = torch.sign(c.q.view(6, Hkv, G, D)[:, :, :1])
    q = c.q.abs().view(6, Hkv, G, D)
    c.q = (q / q.sum(-1, keepdim=True) * sign).view(6, Hq, D) * 50  # the heads of a group agree in their signs
    c.kq[:] = 0
    for s in range(6):
        b, o = c.tables[s, at // bs], at % bs
        c.kq[b, :, o] = 127 * sign[s, :, 0].numpy().astype(np.int8)
        c.ks[b] = target / (50 * 127 * c.scale)
    return c


def check_peaked(pa, c, at, target, qdt, **kw):
    got = c.run(pa, qdt, **kw).double().cpu().numpy()
    G = c.Hq // c.Hkv
    for s in range(6):
        b, o = c.tables[s, at // c.bs], at % c.bs
        v = np.repeat(c.vq[b, :, o].astype(np.float64) * c.vs[b].astype(np.float64)[:, None], G, 0)
        others = (int(c.ctx[s]) - 1) * math.exp(-max(target, 0)) * 127 * float(c.vs[c.tables[s]].max())
        assert (np.abs(got[s] - v) <= PEAKED * np.abs(v) + others).all(), (s, np.abs(got[s] - v).max(), kw)
    assert pa.pa_read_device_errors() == 0


@pytest.mark.parametrize("target", [-1000.0, 30.0, 100.0, 300.0, 1000.0])
@pytest.mark.parametrize("D,bs,Hq,Hkv", [(128, 16, 2, 2), (64, 16, 2, 2), (128, 32, 12, 3), (64, 32, 8, 1), (128, 16, 8, 1)])
def test_one_token_gives_its_values(pa, D, bs, Hq, Hkv, target):
    c = peaked(D, Hq, Hkv, bs, 1, 0, target, seed=51)
    check_peaked(pa, c, 0, target, torch.float16)
    check_peaked(pa, c, 0, target, torch.bfloat16, max_ctx=5000)  # as one of several partitions


@pytest.mark.parametrize("target", [60.0, 200.0, 1000.0, 4000.0])
@pytest.mark.parametrize("D,bs,Hq,Hkv", [(128, 16, 2, 2), (64, 16, 4, 2), (128, 32, 4, 1), (64, 32, 8, 1), (128, 16, 8, 1)])
@pytest.mark.parametrize("at", [0, 200, 899])
def test_a_dominating_token_gives_its_values(pa, D, bs, Hq, Hkv, target, at):
    """Its score is far above the others', in the first, an inner or the last tile; with and without partitions."""
    c = peaked(D, Hq, Hkv, bs, 900, at, target, seed=52)
    for ws in (True, False):
        check_peaked(pa, c, at, target, torch.float16, workspace=ws)


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 2, 2), (64, 8, 1), (128, 8, 1)])
def test_a_sequence_of_bad_blocks_alone_gives_zeros(pa, D, Hq, Hkv):
    c = Case(Hq, Hkv, D, 16, [300, 40, 5], seed=54)
    c.tables[1] = c.NB
    c.tables[0, 8:16] = -1  # a tile without a block between two others
    out = c.run(pa, torch.float16)
    assert pa.pa_read_device_errors() == 0x1
    assert (out[1] == 0).all() and torch.isfinite(out).all()
    d = Case(Hq, Hkv, D, 16, [300, 40, 5], seed=54)
    d.tables[0, 8:-8] = d.tables[0, 16:].copy()
    d.ctx[:] = [172, 0, 5]
    d.check(out, torch.float16)
