"""int8 cache with one scale per (block, kv head) on the GPU: pa_append_q8b,
pa_decode_q8b, pa_copy_blocks_q8b.

The write must give the codes and scales of its definition bit for bit (every
step is one IEEE fp32 operation, redone here in numpy). Decode is compared
with the oracle's attention in double precision over the dequantized cache.

Tolerance of decode, relative to the largest |V| row element M that a sequence
sees. A score is a sum of D products with q's elements rounded to 2^-22 of the
power of two of the head's largest one (most are exact), computed within 2^-20
of A = scale * log2(e) * sum_d |q_d k_d|, and exp2's own error is below 2^-20:
every weight is off by at most ln2 * A * 2^-20 + 2^-20, relative. A weighted
mean moves by at most twice the
largest relative error of its weights times M. Weights held in 23 bits of a
tile's largest one, 128 to a tile, lose another 2^-17 M; fp32 sums over L
terms, a few 2^-24 sqrt(L). So
  |out - ref| <= M * (2 * (A + 1) * 2^-20 + 2^-17 + 2^-24 * sqrt(L) * 8)
plus half a step of a 16-bit output's type."""
import math

import numpy as np
import pytest
import torch

import oracle
from _helpers import f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_340_b200 import _build
    _build.build()
    import paged_kv_cache_340_b200 as pa
    return pa


def cdiv(a, b):
    return -(-a // b)


def random_tables(lens, bs, rng, spare=3, MB=None):
    n = [cdiv(int(x), bs) for x in lens]
    NB = sum(n) + spare
    perm = rng.permutation(NB)
    tables = np.full((len(lens), MB or max(1, max(n))), -1, np.int32)
    at = 0
    for s, k in enumerate(n):
        tables[s, :k] = perm[at:at + k]
        at += k
    return tables, NB


# ------------------------------------------------------------------- write

F = np.float32


def quantize(x, inv):
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.rint((x * inv).astype(F))
        y = np.where(np.isnan(y), F(0), y)
    return np.clip(y, -127, 127).astype(np.int8)


def write_rows(cache, scale, x, q_start, tables, ctx, bs):
    """The definition, block by block: cache int8 [NB, H, bs, D], scale [NB, H], x float32 [T, H, D]; in place."""
    for s in range(len(ctx)):
        n = int(q_start[s + 1] - q_start[s])
        p0 = int(ctx[s]) - n
        for j in range(p0 // bs, cdiv(p0 + n, bs)) if n else ():
            a, e = max(p0, j * bs), min(p0 + n, (j + 1) * bs)
            rows = x[q_start[s] + a - p0:q_start[s] + e - p0]
            b, o0 = int(tables[s, j]), a - j * bs
            for h in range(scale.shape[1]):
                r = rows[:, h]
                finite = np.abs(r[np.isfinite(r)])
                amax = F(finite.max()) if finite.size else F(0)
                new = F(amax / F(127))
                if new < np.finfo(F).tiny:
                    new = F(0)
                old = scale[b, h] if o0 else F(0)
                now = max(old, new)
                cache[b, h, o0:o0 + e - a] = quantize(r, F(F(1) / now) if now > 0 else F(0))
                if o0 and now > old:
                    cache[b, h, :o0] = quantize(cache[b, h, :o0].astype(F), F(old / now))
                scale[b, h] = now


class WriteCase:
    def __init__(self, H, D, bs, dtype, old, new, seed, pad=3, spread=0.7):
        rng = np.random.default_rng(seed)
        old, new = np.array(old), np.array(new)
        self.ctx = (old + new).astype(np.int32)
        self.bs = bs
        self.tables, self.NB = random_tables(self.ctx, bs, rng)
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = int(new.sum()) + pad
        self.key, self.value = (torch.from_numpy((rng.normal(size=(T, H, D)) * np.exp(
            rng.normal(size=(T, H, 1)) * spread)).astype(np.float32)).to(dtype) for _ in range(2))
        self.codes = [rng.integers(-127, 128, (self.NB, H, bs, D)).astype(np.int8) for _ in range(2)]
        self.scales = [(rng.random((self.NB, H)) * 0.02).astype(F) for _ in range(2)]

    def run(self, pa, stream=None):
        d = [torch.from_numpy(a).cuda() for a in self.codes + self.scales]
        args = (self.key.cuda(), self.value.cuda(), torch.from_numpy(self.q_start).cuda(), *d,
                torch.from_numpy(self.tables).cuda(), torch.from_numpy(self.ctx).cuda())
        torch.cuda.synchronize()
        pa.pa_append_q8b(*args, stream=stream)
        torch.cuda.synchronize()
        return d

    def check(self, pa, d, ctx=None, q_start=None):
        q = self.q_start if q_start is None else q_start
        c = self.ctx if ctx is None else ctx
        for codes, scale, x, got, gots in zip(self.codes, self.scales, (self.key, self.value), d[:2], d[2:]):
            codes, scale = codes.copy(), scale.copy()
            write_rows(codes, scale, x.float().numpy(), q, self.tables, c, self.bs)
            assert np.array_equal(gots.cpu().numpy().view(np.int32), scale.view(np.int32))
            assert np.array_equal(got.cpu().numpy(), codes)


OLD_NEW = [
    ([0, 0, 0, 0, 0], [1, 16, 17, 33, 250]),            # from empty, around a block
    ([1, 15, 16, 31, 100, 0], [1, 1, 1, 1, 1, 1]),      # single tokens
    ([5, 0, 13, 40, 7], [0, 0, 3, 100, 9]),             # some sequences with none
    ([3], [1]),
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,D,bs", [(1, 128, 16), (3, 64, 16), (5, 128, 32), (8, 64, 32)])
@pytest.mark.parametrize("k", range(len(OLD_NEW)))
def test_write_is_bit_exact(pa, dtype, H, D, bs, k):
    c = WriteCase(H, D, bs, dtype, *OLD_NEW[k], seed=k * 10 + H)
    d = c.run(pa)
    assert pa.pa_read_device_errors() == 0
    c.check(pa, d)


@pytest.mark.parametrize("more", [-1, 0, 1])
@pytest.mark.parametrize("dtype,D,bs", [(torch.float16, 128, 32), (torch.float32, 64, 16), (torch.bfloat16, 64, 32)])
def test_write_few_and_many_tokens_a_sequence(pa, dtype, D, bs, more):
    """Work is dealt out by tokens or by blocks, whichever are fewer: both, on
    either side of the point where they are as many (by padding), with long,
    single-token and empty sequences in one batch and more than 128 of them."""
    rng = np.random.default_rng(77)
    S = 150
    new = rng.integers(0, 2, S)
    new[[3, 70, 149]] = [101, 2 * bs, bs + 1]
    old = rng.integers(0, 3 * bs, S)
    T = int(new.sum())
    pad = next(k for k in range(10000) if T + k >= (T + k) // bs + 2 * S + 1) + more
    c = WriteCase(2, D, bs, dtype, old, new, seed=78, pad=pad)
    d = c.run(pa)
    assert pa.pa_read_device_errors() == 0
    c.check(pa, d)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_write_extreme_values(pa, dtype):
    """Zero blocks, NaN and infinities (kept out of the scale), the type's
    largest and smallest values, ties, and a zero block that gets a value."""
    c = WriteCase(2, 64, 16, dtype, [0, 0, 0, 0, 16, 4, 4, 2], [16, 16, 3, 2, 1, 1, 1, 2], seed=5)
    big, small = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    q = c.q_start
    for x in (c.key, c.value):
        x[q[0]:q[1]] = 0
        x[q[1], 0, 0], x[q[1], 1, 3], x[q[1] + 2, 0, 1] = math.nan, math.inf, -math.inf
        x[q[2]:q[3], 0] = math.nan                 # nothing finite at all
        x[q[2], 1, 5] = -big
        x[q[3]:q[4]] *= small
        x[q[4], 0] = 0
        x[q[4], 0, :4] = torch.tensor([254.0, 1.0, -1.0, 3.0]).to(dtype)
        x[q[5]] = 0                                # the older rows' scale stays
        x[q[6], 0, 0] = big                        # the older rows' codes fall to zero
    for s in c.scales:
        s[c.tables[7, 0]] = 0                      # older rows of zeros
    for k in c.codes:
        k[c.tables[7, 0], :, :2] = 0
    d = c.run(pa)
    assert pa.pa_read_device_errors() == 0
    c.check(pa, d)


def test_write_again_changes_nothing(pa):
    """The same rows written twice give the same cache (a scale that grew stays)."""
    c = WriteCase(4, 128, 16, torch.bfloat16, [3, 20, 0], [1, 30, 16], seed=6)
    d = c.run(pa)
    first = [t.clone() for t in d]
    pa.pa_append_q8b(c.key.cuda(), c.value.cuda(), torch.from_numpy(c.q_start).cuda(), *d,
                     torch.from_numpy(c.tables).cuda(), torch.from_numpy(c.ctx).cuda())
    for t, w in zip(d, first):
        assert torch.equal(t, w)


def test_token_by_token_stays_within_its_bound(pa):
    """Rows appended one at a time: off by half a step of the last scale, and
    at most half a step more for each later token that raised it."""
    H, D, bs, n = 2, 128, 16, 16
    g = torch.Generator().manual_seed(7)
    x = torch.randn((n, H, D), generator=g)
    kc, vc = (torch.zeros((1, H, bs, D), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((1, H), device="cuda") for _ in range(2))
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    seen = []
    for t in range(n):
        pa.pa_append_q8b(x[t:t + 1].cuda(), x[t:t + 1].cuda(), torch.tensor([0, 1], dtype=torch.int32, device="cuda"), kc, vc,
                         ks, vs, table, torch.tensor([t + 1], dtype=torch.int32, device="cuda"))
        seen.append(ks[0].cpu().double())
    got = (kc[0].double() * ks[0].double()[:, None, None]).cpu().permute(1, 0, 2)
    for t in range(n):
        for h in range(H):
            raises = {float(seen[u][h]) for u in range(t, n)}  # the scales the row has lived under
            bound = sum(raises) / 2 * (1 + 2.0 ** -16)  # fp32 steps: 2^-22 of 127 steps is far below 2^-16 of half of one
            assert (got[t, h] - x[t, h].double()).abs().max() <= bound + 127 * 2.0 ** -22 * max(raises)
    assert torch.equal(kc, vc) and torch.equal(ks, vs)


def test_write_skips_bad_sequences(pa):
    c = WriteCase(3, 64, 16, torch.float16, [4, 0, 9, 30], [5, 20, 1, 20], seed=8)
    keep = c.tables[1, 1]
    c.tables[1, 1] = c.NB                # a bad block: its rows are skipped
    d = c.run(pa)
    assert pa.pa_read_device_errors() == 0x1
    want = WriteCase(3, 64, 16, torch.float16, [4, 0, 9, 30], [5, 20, 1, 20], seed=8)
    ok = [i for i in range(c.NB) if i != keep]
    for got, codes, scale, x, gots in zip(d[:2], want.codes, want.scales, (want.key, want.value), d[2:]):
        untouched = codes[keep].copy()
        write_rows(codes, scale, x.float().numpy(), want.q_start, want.tables, want.ctx, 16)
        assert np.array_equal(got.cpu().numpy()[ok], codes[ok])
        assert np.array_equal(got.cpu().numpy()[keep], untouched)
    c.tables[1, 1] = keep
    for bad in (4, 10_000):              # fewer tokens than new ones; past the table row
        c.ctx[0] = bad
        d = c.run(pa)
        assert pa.pa_read_device_errors() == 0x4
        ctx, q = c.ctx.copy(), c.q_start.copy()
        full = [a.copy() for a in c.codes]
        for codes, scale, x, got in zip(full, [s.copy() for s in c.scales], (c.key, c.value), d[:2]):
            x = x.float().numpy()
            write_rows(codes, scale, x[q[1]:], q[1:] - q[1], c.tables[1:], ctx[1:], 16)
            assert np.array_equal(got.cpu().numpy(), codes)


def test_write_more_new_tokens_than_rows_is_recorded(pa):
    c = WriteCase(1, 64, 16, torch.float16, [0], [8], seed=9, pad=0)
    c.q_start[1] = 9                     # past num_tokens
    c.ctx[0] = 9
    d = c.run(pa)
    assert pa.pa_read_device_errors() == 0x4
    assert np.array_equal(d[0].cpu().numpy(), c.codes[0])


# -------------------------------------------------------------------- copy

@pytest.mark.parametrize("H", [1, 3, 8])
@pytest.mark.parametrize("count", [None, 0, 2])
def test_copy_blocks(pa, H, count):
    g = torch.Generator().manual_seed(61 + H)
    kc, vc = (torch.randint(-127, 128, (12, H, 16, 64), generator=g, dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.rand((12, H), generator=g) for _ in range(2))
    pairs = np.array([[3, 7], [0, 11], [5, 2]], np.int64)
    d = [t.cuda() for t in (kc, vc, ks, vs)]
    num = None if count is None else torch.tensor([count], dtype=torch.int32, device="cuda")
    pa.pa_copy_blocks_q8b(*d, torch.from_numpy(pairs).cuda(), num)
    for got, w in zip(d, (kc, vc, ks, vs)):
        w = w.clone()
        for a, b in pairs[:3 if count is None else count]:
            w[b] = w[a]
        assert torch.equal(got.cpu(), w)
    assert pa.pa_read_device_errors() == 0
    bad = torch.tensor([[1, 12], [-1, 3]], dtype=torch.int64, device="cuda")
    before = [t.clone() for t in d]
    pa.pa_copy_blocks_q8b(*d, bad)
    assert pa.pa_read_device_errors() == 0x10
    assert all(torch.equal(a, b) for a, b in zip(d, before))


# ------------------------------------------------------------------ decode

class Case:
    """A random cache with NaN scales on every block no sequence uses and
    random codes in every slot past a sequence's end."""

    def __init__(self, Hq, Hkv, D, bs, ctx, seed, q_scale=1.0, MB=None, spread=0.5):
        rng = np.random.default_rng(seed)
        self.ctx = np.array(ctx, np.int32)
        self.bs, self.D, self.Hq, self.Hkv = bs, D, Hq, Hkv
        self.tables, self.NB = random_tables(self.ctx, bs, rng, MB=MB)
        self.kq, self.vq = (rng.integers(-127, 128, (self.NB, Hkv, bs, D)).astype(np.int8) for _ in range(2))
        self.ks, self.vs = ((np.exp(rng.normal(size=(self.NB, Hkv)) * spread) / 73).astype(F) for _ in range(2))
        unused = np.setdiff1d(np.arange(self.NB), self.tables[self.tables >= 0])
        self.ks[unused] = np.nan
        self.vs[unused] = np.nan
        self.q = torch.from_numpy((rng.normal(size=(len(ctx), Hq, D)) * q_scale).astype(F))
        self.scale = 1.0 / math.sqrt(D)

    def run(self, pa, qdt, out_dt=torch.float32, workspace=True, order=None, max_ctx=None, stream=None):
        S = len(self.ctx)
        out = torch.full((S, self.Hq, self.D), float("nan"), dtype=out_dt, device="cuda")
        L = int(self.ctx.max(initial=0)) if max_ctx is None else max_ctx
        ws = None
        if workspace:
            n = pa.pa_decode_q8b_workspace_bytes(S, self.Hq, self.Hkv, self.D, L)
            ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        d = [torch.from_numpy(a).cuda() for a in (self.kq, self.vq, self.ks, self.vs, self.tables, self.ctx)]
        o = None if order is None else torch.tensor(order, dtype=torch.int32, device="cuda")
        q = self.q.to(qdt).cuda()
        torch.cuda.synchronize()
        pa.pa_decode_q8b(out, q, *d, self.scale, L, ws, seq_order=o, stream=stream)
        torch.cuda.synchronize()
        return out

    def ref(self, qdt, seqs=None):
        """(expected [S, Hq, D], tolerance [S, 1, 1]) in double."""
        rows = [np.repeat(np.nan_to_num(a)[:, :, None], self.bs, 2) for a in (self.ks, self.vs)]
        q = f64(self.q.to(qdt))
        want = oracle.paged_decode_q8(q, self.kq, self.vq, *rows, self.tables, np.maximum(self.ctx, 0), self.scale, self.bs)
        tol = np.zeros((len(self.ctx), 1, 1))
        for s, L in enumerate(self.ctx):
            if L <= 0:
                continue
            ids = self.tables[s, :cdiv(int(L), self.bs)]
            k = np.abs(self.kq[ids].astype(np.float64)) * self.ks[ids][..., None, None]     # [n, H, bs, D]
            A = 0.0
            for h in range(self.Hkv):
                G = self.Hq // self.Hkv
                A = max(A, float((k[:, h].reshape(-1, self.D) @ np.abs(q[s, h * G:(h + 1) * G]).T).max()))
            A *= self.scale * math.log2(math.e)
            M = float((np.abs(self.vq[ids].astype(np.float64)) * self.vs[ids][..., None, None]).max())
            tol[s] = M * (2 * (A + 1) * 2.0 ** -20 + 2.0 ** -17 + 2.0 ** -24 * math.sqrt(L) * 8)
        return want, tol

    def check(self, out, qdt, what=""):
        want, tol = self.ref(qdt)
        got = f64(out)
        assert np.isfinite(got).all(), what
        err = np.abs(got - want) - np.abs(want) * (torch.finfo(out.dtype).eps / 2 if out.dtype != torch.float32 else 0)
        assert (err <= tol).all(), f"{what}: {float((err / np.maximum(tol, 1e-300)).max()):.3g} of the tolerance"


LENS = [1, 15, 16, 17, 33, 127, 128, 129, 255, 256, 257, 700]


@pytest.mark.parametrize("qdt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (4, 2), (3, 1), (8, 2), (10, 2), (6, 1), (16, 2), (12, 1), (17, 1)])
def test_decode_matches_oracle(pa, qdt, bs, D, Hq, Hkv):
    c = Case(Hq, Hkv, D, bs, LENS, seed=Hq * 100 + Hkv + D)
    for ws in (True, False):
        out = c.run(pa, qdt, workspace=ws)
        assert pa.pa_read_device_errors() == 0
        c.check(out, qdt, f"workspace {ws}")


@pytest.mark.parametrize("qdt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,bs,Hq,Hkv", [(128, 16, 4, 1), (64, 32, 2, 2), (128, 32, 8, 1)])
def test_decode_16bit_output_equals_the_rounded_fp32_one(pa, qdt, D, bs, Hq, Hkv):
    c = Case(Hq, Hkv, D, bs, [1, 40, 300, 0], seed=3)
    a, b = c.run(pa, qdt), c.run(pa, qdt, out_dt=qdt)
    assert torch.equal(a.to(qdt), b)
    c.check(b, qdt)
    assert (a[3] == 0).all()


@pytest.mark.parametrize("D,bs", [(128, 16), (64, 16), (128, 32), (64, 32)])
@pytest.mark.parametrize("S,L", [(1, 5000), (2, 20011), (3, 1025)])
def test_decode_few_long_sequences(pa, D, bs, S, L):
    """With a workspace few long sequences are split; lengths of 0 and 1 and a
    short one are in the same batch."""
    c = Case(4, 1, D, bs, ([L, 0, 1, 129] * 2)[:S + 1], seed=L)
    for ws in (True, False):
        c.check(c.run(pa, torch.bfloat16, workspace=ws), torch.bfloat16, f"workspace {ws}")
    # a bound of the lengths above the largest one
    c.check(c.run(pa, torch.bfloat16, max_ctx=L + 5000), torch.bfloat16)
    assert pa.pa_read_device_errors() == 0


def test_decode_is_deterministic_and_order_free(pa):
    c = Case(8, 2, 128, 16, [900, 3, 77, 0, 1400], seed=21)
    a = c.run(pa, torch.float16)
    for order in (None, [4, 0, 2, 1, 3], [3, 1, 2, 0, 4]):
        assert torch.equal(c.run(pa, torch.float16, order=order), a)


@pytest.mark.parametrize("D", [64, 128])
def test_decode_large_and_flat_scores(pa, D):
    """Scores of hundreds (a softmax of one token) and of zero (a mean)."""
    c = Case(4, 2, D, 16, [500, 129], seed=31, q_scale=60.0)
    c.check(c.run(pa, torch.bfloat16), torch.bfloat16, "large")
    c = Case(4, 2, D, 16, [500, 129], seed=32, q_scale=0.0)
    c.check(c.run(pa, torch.float16), torch.float16, "flat")


@pytest.mark.parametrize("D", [64, 128])
def test_decode_small_weights_are_not_lost(pa, D):
    """One token's weight is 2^20 times the others', whose sum still counts in
    other tiles; scales 2^24 apart between blocks of one tile."""
    c = Case(1, 1, D, 16, [4096], seed=33)
    q = c.q.half().float().numpy()[0, 0]
    c.kq[:] = 0
    first = c.tables[0, 0]
    c.kq[first, 0, 0] = np.sign(q) * 127
    c.ks[:] = 1e-6
    c.ks[first] = 20 * math.log(2) / (c.scale * np.abs(q).sum() * 127)
    c.check(c.run(pa, torch.float16), torch.float16, "one large weight")
    c = Case(2, 1, D, 16, [600], seed=34)
    c.vs[c.tables[0, ::2]] *= 2.0 ** -24
    c.check(c.run(pa, torch.float16), torch.float16, "V scales far apart")


def test_decode_zero_blocks(pa):
    """Blocks of scale 0 (all-zero rows) in K, V or both; all of V zero."""
    c = Case(4, 1, 128, 16, [200, 100], seed=35)
    c.ks[c.tables[0, 2]] = 0
    c.vs[c.tables[0, 3]] = 0
    c.vs[c.tables[1, :7]] = 0
    out = c.run(pa, torch.float16)
    c.check(out, torch.float16)
    assert (out[1] == 0).all()


def test_decode_bad_tables_and_lengths(pa):
    c = Case(4, 2, 128, 16, [100, 60, 300, 50], seed=36)
    c.tables[0, 2] = c.NB + 4               # tokens 32..47 of sequence 0 are skipped
    c.tables[1, 0] = -7
    out = c.run(pa, torch.float16)
    assert pa.pa_read_device_errors() == 0x1
    assert torch.isfinite(out).all()
    # the same as a sequence without those blocks
    d = Case(4, 2, 128, 16, [100, 60, 300, 50], seed=36)
    for s, j in ((0, 2), (1, 0)):
        d.tables[s, j:-1] = d.tables[s, j + 1:].copy()
        d.ctx[s] -= 16
    d.check(out, torch.float16)
    # a bound below a length clamps it; a negative length is 0; a bad schedule entry is skipped
    e = Case(4, 2, 128, 16, [100, 60, 300, 50], seed=36)
    out = e.run(pa, torch.float16, max_ctx=128)
    assert pa.pa_read_device_errors() == 0x4
    f = Case(4, 2, 128, 16, [100, 60, 300, 50], seed=36)
    f.ctx[2] = 128
    f.check(out, torch.float16)
    e.ctx[1] = -3
    out = e.run(pa, torch.float16, order=[0, 1, 9, 3])
    assert pa.pa_read_device_errors() == 0x4
    assert (out[1] == 0).all() and torch.isnan(out[2]).all() and torch.isfinite(out[[0, 3]]).all()
    assert not any(torch.isnan(x).any() for x in (out[0], out[3]))


@pytest.mark.parametrize("D,bs,Hq,Hkv", [(128, 16, 2, 2), (128, 32, 16, 2), (64, 16, 2, 2), (64, 32, 8, 1), (64, 16, 4, 1)])
def test_decode_more_items_than_ctas(pa, D, bs, Hq, Hkv):
    """More (sequence, kv head) pairs than fit the GPU at once, so each CTA
    works through several: lengths of 0, 1, a few tiles and around their ends."""
    rng = np.random.default_rng(D + Hq)
    lens = rng.integers(0, 400, 900)
    lens[rng.integers(0, 900, 200)] = rng.choice([0, 1, 16, 128, 129, 256, 257, 512, 513, 1000], 200)
    c = Case(Hq, Hkv, D, bs, lens, seed=77, MB=64)
    order = rng.permutation(900)
    a = c.run(pa, torch.bfloat16, order=order)
    assert pa.pa_read_device_errors() == 0
    c.check(a, torch.bfloat16)
    assert torch.equal(a, c.run(pa, torch.bfloat16, workspace=False))
    assert (a[torch.from_numpy(lens == 0).cuda()] == 0).all()


@pytest.mark.parametrize("D", [64, 128])
def test_decode_non_finite_query_gives_nan_rows_only_there(pa, D):
    c = Case(4, 2, D, 16, [300, 0, 40], seed=39)
    c.q[0, 1, 3], c.q[2, 2, 0], c.q[1, 0, 0] = math.nan, math.inf, math.nan
    for ws in (True, False):
        out = c.run(pa, torch.float16, workspace=ws)
        bad = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
        bad[0, 1] = bad[2, 2] = True
        assert torch.isnan(out[bad]).all() and torch.isfinite(out[~bad]).all()
        assert (out[1] == 0).all()


@pytest.mark.parametrize("tile", [0, 1, 3])
def test_decode_wait_that_runs_out_returns_and_reports(pa, tile):
    """One K tile's copy never issued: the launch ends, the error word says
    so, every other output is right, and the next call is sound."""
    c = Case(3, 3, 128, 16, [500, 40, 700], seed=41)
    args = [c.q.half().cuda(), *[torch.from_numpy(a).cuda() for a in (c.kq, c.vq, c.ks, c.vs, c.tables, c.ctx)], c.scale, 700]
    want = torch.empty((3, 3, 128), device="cuda")
    pa.pa_decode_q8b(want, *args)
    out = torch.empty_like(want)
    pa.pa_decode_q8b_withhold_tile(out, *args, 0, 1, tile, 20_000_000)
    torch.cuda.synchronize()
    assert pa.pa_read_device_errors() == 0x8
    others = torch.ones((3, 3), dtype=torch.bool, device="cuda")
    others[0, 1] = False
    assert torch.equal(out[others], want[others])
    again = torch.empty_like(want)
    pa.pa_decode_q8b(again, *args)
    pa.pa_decode_q8b_withhold_tile(out, *args, 1, 2, 5, 20_000_000)  # past that sequence's end: nothing withheld
    assert pa.pa_read_device_errors() == 0
    assert torch.equal(again, want) and torch.equal(out, want)


def test_decode_empty_batches(pa):
    c = Case(4, 2, 128, 16, [0, 0], seed=37)
    assert (c.run(pa, torch.float16) == 0).all()
    assert (c.run(pa, torch.float16, max_ctx=1000) == 0).all()
    z = torch.empty((0, 4, 128), dtype=torch.float16, device="cuda")
    d = [torch.from_numpy(a).cuda() for a in (c.kq, c.vq, c.ks, c.vs)]
    pa.pa_decode_q8b(torch.empty((0, 4, 128), device="cuda"), z, *d, torch.empty((0, 1), dtype=torch.int32, device="cuda"),
                     torch.empty(0, dtype=torch.int32, device="cuda"), 0.1, 0)
    assert pa.pa_read_device_errors() == 0


def test_decode_and_write_past_32_bit_offsets(pa):
    """Blocks whose byte offset in the cache is above 2^32."""
    H, D, bs = 16, 128, 16
    NB = (1 << 32) // (H * D * bs) + 40
    kc, vc = (torch.empty((NB, H, bs, D), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((NB, H), float("nan"), device="cuda") for _ in range(2))
    n = 300
    ids = np.concatenate([[5], np.arange(NB - 18, NB)]).astype(np.int32)
    tables = torch.from_numpy(ids[None]).cuda()
    ctx = torch.tensor([n], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(2)
    key, value = (torch.randn((n, H, D), generator=g).bfloat16() for _ in range(2))
    pa.pa_append_q8b(key.cuda(), value.cuda(), torch.tensor([0, n], dtype=torch.int32, device="cuda"), kc, vc, ks, vs, tables,
                     ctx)
    q = torch.randn((1, 2 * H, D), generator=g).half()
    out = torch.empty((1, 2 * H, D), device="cuda")
    pa.pa_decode_q8b(out, q.cuda(), kc, vc, ks, vs, tables, ctx, D ** -0.5, n)
    assert pa.pa_read_device_errors() == 0
    c = Case(2 * H, H, D, bs, [n], seed=1)
    use = torch.from_numpy(ids.astype(np.int64)).cuda()
    c.tables, c.NB, c.q = np.arange(19, dtype=np.int32)[None], 19, q.float()
    c.kq, c.vq, c.ks, c.vs = (t[use].cpu().numpy() for t in (kc, vc, ks, vs))
    for codes, scale, x in ((c.kq, c.ks, key), (c.vq, c.vs, value)):
        wc, wsc = np.zeros_like(codes), np.zeros_like(scale)
        write_rows(wc, wsc, x.float().numpy(), np.array([0, n]), c.tables, c.ctx, bs)
        assert np.array_equal(scale, wsc)
        wc[18, :, 12:] = codes[18, :, 12:]  # past the last token: left as it was
        assert np.array_equal(codes, wc)
    c.check(out, torch.float16)


def test_binding_refuses_wrong_types_and_shapes(pa):
    c = Case(4, 2, 128, 16, [20], seed=38)
    d = [torch.from_numpy(a).cuda() for a in (c.kq, c.vq, c.ks, c.vs, c.tables, c.ctx)]
    q = c.q.half().cuda()
    out = torch.empty_like(q)
    pa.pa_decode_q8b(out, q, *d, c.scale, 20)
    for i, bad in ((0, d[0].to(torch.uint8)), (2, d[2].double()), (2, d[2][:, :1].contiguous()), (4, d[4].long()),
                   (5, d[5].long()), (1, d[1][:, :, :, :64].contiguous())):
        e = list(d)
        e[i] = bad
        with pytest.raises(ValueError):
            pa.pa_decode_q8b(out, q, *e, c.scale, 20)
    with pytest.raises(ValueError):
        pa.pa_decode_q8b(out[:, :2], q, *d, c.scale, 20)
    with pytest.raises(ValueError):
        pa.pa_decode_q8b(out, q.transpose(0, 1).contiguous().transpose(0, 1).expand(1, 4, 128)[:, ::2], *d, c.scale, 20)
    with pytest.raises(pa.PagedAttentionError):
        pa.pa_decode_q8b(out, q, *d, c.scale, 20, torch.empty(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        pa.pa_append_q8b(q[:, :2], q[:, :2].float(), torch.tensor([0, 1], dtype=torch.int32, device="cuda"), *d)
    assert pa.pa_read_device_errors() == 0


def test_stream_as_object_handle_or_current(pa):
    """The three ways to give a stream, each behind work of that stream that the call has to wait for."""
    c = Case(4, 2, 128, 16, [70, 33], seed=39)
    d = [torch.from_numpy(a).cuda() for a in (c.kq, c.vq, c.ks, c.vs, c.tables, c.ctx)]
    q = c.q.half().cuda()
    want = torch.empty_like(q)
    pa.pa_decode_q8b(want, q, *d, c.scale, 70)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for give in (st, st.cuda_stream, None):
        late, out, nxt = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            torch.cuda._sleep(2_000_000)
            late.copy_(q)
            if give is None:
                pa.pa_decode_q8b(out, late, *d, c.scale, 70)
        if give is not None:
            pa.pa_decode_q8b(out, late, *d, c.scale, 70, stream=give)
        with torch.cuda.stream(st):
            nxt.copy_(out)
        torch.cuda.synchronize()
        assert torch.equal(nxt, want)
    assert pa.pa_read_device_errors() == 0


def test_binding_takes_numpy_numbers_and_refuses_the_rest(pa):
    c = Case(4, 2, 128, 16, [20], seed=40)
    d = [torch.from_numpy(a).cuda() for a in (c.kq, c.vq, c.ks, c.vs, c.tables, c.ctx)]
    q = c.q.half().cuda()
    out = torch.empty_like(q)
    pa.pa_decode_q8b(out, q, *d, np.float32(c.scale), np.int64(20))
    c.check(out, torch.float16)
    with pytest.raises(OverflowError):
        pa.pa_decode_q8b(out, q, *d, c.scale, 1 << 40)
    with pytest.raises(TypeError):
        pa.pa_decode_q8b(out, q, *d, c.scale, 20.5)
    with pytest.raises(TypeError):
        pa.pa_decode_q8b(out, q, *d, None, 20)
    with pytest.raises(TypeError):
        pa.pa_decode_q8b(out, q.cpu().numpy(), *d, c.scale, 20)
    with pytest.raises(ValueError):
        pa.pa_decode_q8b(out, q.cpu(), *d, c.scale, 20)
    with pytest.raises(ValueError):
        pa.pa_decode_q8b(out, q.to(torch.int16), *d, c.scale, 20)
    with pytest.raises(ValueError):
        pa.pa_copy_blocks_q8b(*d[:4], torch.zeros((1, 3), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        pa.pa_copy_blocks_q8b(*d[:4], torch.zeros((1, 2), dtype=torch.int64, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"))
    with pytest.raises(pa.PagedAttentionError):
        pa.pa_decode_q8b(out, q, *d, float("nan"), 20)
    assert pa.pa_read_device_errors() == 0
