"""pa_decode_q8b and pa_append_q8b where they are easily wrong: a wait that runs
out while further work has been claimed, softmaxes of one token, blocks that are
all bad, queries with a few large elements, lengths that
are wrong where nothing is written."""
import math

import numpy as np
import pytest
import torch

from test_gpu_q8b import Case, WriteCase

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


def raised(D, Hq, Hkv, bs, lens, times, seed, qdt, heads=slice(None), spread=0.5, codes=0):
    """A case whose queries have four elements `times` the size of the others, over codes of at most `codes` in K."""
    rng = np.random.default_rng(seed)
    c = Case(Hq, Hkv, D, bs, lens, seed=seed, spread=spread)
    dims = rng.choice(D, 4, replace=False)
    for d in dims:
        c.q[:, heads, d] = c.q[:, heads, d].sign() * (0.5 + c.q[:, heads, d].abs() / 4) * times
    c.kq[..., dims] = rng.integers(-codes, codes + 1, c.kq[..., dims].shape)
    c.q = c.q.to(qdt).float()
    return c


@pytest.mark.parametrize("qdt,times", [(torch.float16, 1), (torch.float16, 30), (torch.float16, 100), (torch.float16, 1e3),
                                       (torch.float16, 3e4), (torch.bfloat16, 1e3), (torch.bfloat16, 1e6)])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 4, 4), (64, 4, 4), (128, 6, 3), (128, 6, 2), (64, 8, 2), (128, 16, 2), (64, 7, 1),
                                      (128, 11, 1)])
def test_scores_of_queries_with_few_large_elements(pa, qdt, times, D, Hq, Hkv):
    """Two tokens with V opposite: out = M tanh((s0 - s1) / 2), so its error shows the scores'. A score is within 2^-20
    of A = scale sum_d |q_d k_d|: a difference of two within 2^-19 A, half of which is the tanh's, at most; the powers of
    two, weights and fp32 steps as for one token (2^-19)."""
    S = 40
    c = raised(D, Hq, Hkv, 16, [2] * S, times, seed=53, qdt=qdt, spread=0.2)
    b = c.tables[:, 0]
    c.vq[b, :, 0], c.vq[b, :, 1] = 127, -127
    got = c.run(pa, qdt).double().cpu().numpy()
    G = Hq // Hkv
    k = c.kq[b][:, :, :2].astype(np.float64) * c.ks[b].astype(np.float64)[:, :, None, None]  # [S, Hkv, 2, D]
    k = np.repeat(k, G, 1)
    q = c.q.double().numpy()[:, :, None]
    s = (q * k).sum(-1) * c.scale
    A = (np.abs(q) * np.abs(k)).sum(-1).max(-1) * c.scale
    M = np.repeat(127 * c.vs[b].astype(np.float64), G, 1)
    err = np.abs(got - (M * np.tanh((s[..., 0] - s[..., 1]) / 2))[..., None]).max(-1)
    assert (err <= M * (2.0 ** -20 * A + 2.0 ** -19)).all(), float((err / (M * (2.0 ** -20 * A + 2.0 ** -19))).max())
    assert pa.pa_read_device_errors() == 0


@pytest.mark.parametrize("qdt,times", [(torch.float16, 1e3), (torch.bfloat16, 1e5)])
@pytest.mark.parametrize("D,bs,Hq,Hkv", [(128, 16, 2, 2), (64, 32, 2, 2), (128, 32, 10, 2), (64, 16, 8, 1), (128, 16, 6, 2),
                                         (128, 16, 17, 1), (64, 32, 12, 4)])
def test_decode_of_queries_with_few_large_elements(pa, qdt, times, D, bs, Hq, Hkv):
    """All heads such, or one of a group; short and long, split and not, and more of them than CTAs."""
    for heads in (slice(None), slice(Hq - 1, None), slice(0, None, 2)):
        c = raised(D, Hq, Hkv, bs, [1, 17, 129, 300, 0, 2500], times, 55, qdt, heads=heads)
        for kw in (dict(), dict(workspace=False), dict(max_ctx=9000)):
            c.check(c.run(pa, qdt, **kw), qdt, f"{heads} {kw}")
    lens = np.random.default_rng(56).integers(0, 300, 500)
    c = raised(D, Hq, Hkv, bs, lens, times, 57, qdt)
    c.q[::3] = torch.from_numpy(np.random.default_rng(58).normal(size=c.q[::3].shape)).to(qdt).float()
    a = c.run(pa, qdt)
    c.check(a, qdt, "many")
    assert torch.equal(a, c.run(pa, qdt, workspace=False, order=np.random.default_rng(59).permutation(500)))
    assert pa.pa_read_device_errors() == 0


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 2, 2), (64, 2, 2), (128, 4, 1), (64, 8, 1), (128, 8, 1)])
def test_non_finite_queries_beside_ones_with_few_large_elements(pa, D, Hq, Hkv):
    c = raised(D, Hq, Hkv, 16, [300, 40, 1], 1e3, 60, torch.float16)
    want = c.run(pa, torch.float16)
    c.check(want, torch.float16)
    c.q[0, 1, 3], c.q[2, 0, 0] = math.nan, math.inf
    got = c.run(pa, torch.float16)
    bad = torch.zeros(got.shape[:2], dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[2, 0] = True
    assert torch.isnan(got[bad]).all() and torch.isfinite(got[~bad]).all()
    d = Case.__new__(Case)
    d.__dict__.update(c.__dict__)
    d.q = torch.where(bad.cpu()[..., None], torch.zeros(()), c.q)
    ref, tol = d.ref(torch.float16)
    assert (np.abs(got.double().cpu().numpy() - ref) <= tol)[~bad.cpu().numpy()].all()
    assert pa.pa_read_device_errors() == 0


@pytest.mark.parametrize("pad", [0, 1, 40, 400])
def test_write_does_not_look_at_sequences_without_new_tokens(pa, pad):
    """Whether the work is dealt out by tokens or by blocks (as the padding has it): a length past the table row, or
    below 0, is no error of a sequence that gets nothing, and is one of a sequence that does."""
    old, new = [40, 3, 7, 30, 5, 9], [0, 2, 0, 1, 0, 0]
    c = WriteCase(2, 64, 16, torch.float16, old, new, seed=61, pad=pad)
    right = c.ctx.copy()
    c.ctx[[0, 2, 5]] = [100000, -3, 2 ** 31 - 1]
    d = c.run(pa)
    assert pa.pa_read_device_errors() == 0
    c.check(pa, d, ctx=right)
    c.ctx[3] = 100000
    c.run(pa)
    assert pa.pa_read_device_errors() == 0x4


@pytest.mark.parametrize("qdt,size", [(torch.float16, 2.0 ** -16), (torch.float16, 2.0 ** -22), (torch.bfloat16, 2.0 ** -60),
                                      (torch.bfloat16, 2.0 ** 90)])
@pytest.mark.parametrize("times", [1, 300])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 2, 2), (64, 8, 1), (128, 8, 2)])
def test_very_small_and_large_queries(pa, qdt, size, times, D, Hq, Hkv):
    """Subnormal elements and far exponents, the scale making up for them."""
    c = raised(D, Hq, Hkv, 16, [1, 40, 300], times, 62, torch.float32)
    c.q = (c.q * size).to(qdt).float()
    c.scale /= size
    c.check(c.run(pa, qdt), qdt)
    assert pa.pa_read_device_errors() == 0
