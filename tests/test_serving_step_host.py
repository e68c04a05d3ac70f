"""Argument checks of the append, release, write and decode calls over a cache
with block scales: each returns its status before any device work (the fake
device addresses are never touched)."""
import pytest

A = 1 << 20  # a fake 16-byte aligned address


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_340_b200 import _build
    _build.build()
    import paged_kv_cache_340_b200 as pa
    return pa


@pytest.mark.parametrize("kw,code", [
    (dict(nb=0), -3), (dict(bs=0), -3), (dict(mb=0), -3), (dict(S=-1), -3), (dict(S=8193), -3), (dict(T=-1), -3),
    (dict(S=8192, mb=1 << 17), -3),              # flattened table index past 2^30
    (dict(nb=1 << 27, bs=16), -3),               # slots past int32
    (dict(state=None), -1), (dict(tables=None), -1), (dict(ctx=None), -1), (dict(new=None), -1),
    (dict(q_start=None), -1), (dict(slots=None), -1), (dict(pairs=None), -1), (dict(num=None), -1),
    (dict(state=A + 8), -7), (dict(pairs=A + 8), -7), (dict(tables=A + 2), -7), (dict(slots=A + 1), -7),
])
def test_dpool_append_host_checks(pa, kw, code):
    a = dict(state=A, nb=64, bs=16, tables=A, mb=8, ctx=A, new=A, S=4, q_start=A, slots=A, T=10, pairs=A, num=A)
    a.update(kw)
    assert pa._lib.pa_dpool_append(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(nb=0), -3), (dict(S=8193), -3), (dict(mb=-1), -3), (dict(state=None), -1), (dict(tables=None), -1),
    (dict(ctx=None), -1), (dict(fin=None), -1), (dict(fin=A + 2), -7), (dict(state=A + 4), -7),
    (dict(S=0, tables=None, ctx=None, fin=None), 0),
])
def test_dpool_release_host_checks(pa, kw, code):
    a = dict(state=A, nb=64, bs=16, tables=A, mb=8, ctx=A, fin=A, S=4)
    a.update(kw)
    assert pa._lib.pa_dpool_release(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), -2), (dict(D=96), -5), (dict(bs=64), -6), (dict(H=0), -3), (dict(T=-1), -3), (dict(S=-1), -3),
    (dict(S=65536), -3), (dict(nb=1 << 27, bs=32), -3), (dict(key=None), -1), (dict(vs=None), -1), (dict(ctx=None), -1),
    (dict(key=A + 8), -7), (dict(kc=A + 4), -7), (dict(ks=A + 4), -7), (dict(q=A + 2), -7),
    (dict(T=0, key=None), 0), (dict(S=0, q=None), 0),
])
def test_append_q8b_host_checks(pa, kw, code):
    a = dict(key=A, value=A, dt=1, q=A, T=9, kc=A, vc=A, ks=A, vs=A, tables=A, mb=8, ctx=A, S=3, nb=40, H=2, D=128, bs=16)
    a.update(kw)
    assert pa._lib.pa_append_q8b(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q_dt=0), -2), (dict(out_dt=2), -2), (dict(D=256), -5), (dict(bs=8), -6), (dict(Hq=7), -4), (dict(S=-1), -3),
    (dict(L=-1), -3), (dict(L=(1 << 30) + 1), -3), (dict(scale=float("nan")), -3), (dict(scale=float("inf")), -3),
    (dict(Hkv=65535, Hq=65535 * 9), -3),         # nine heads to a kv head: two CTAs each, past the grid's second axis
    (dict(nb=1 << 27, Hkv=8), -3),               # cache rows past int32
    (dict(out=None), -1), (dict(q=None), -1), (dict(ks=None), -1), (dict(tables=None), -1),
    (dict(out=A + 8), -7), (dict(vc=A + 8), -7), (dict(vs=A + 4), -7), (dict(order=A + 2), -7), (dict(ws=A + 8), -7),
    (dict(ws_bytes=0), -9), (dict(S=0, out=None, q=None), 0),
])
def test_decode_q8b_host_checks(pa, kw, code):
    a = dict(out=A, q=A, q_dt=1, kc=A, vc=A, ks=A, vs=A, tables=A, mb=4096, ctx=A, S=2, Hq=8, Hkv=2, D=128, scale=0.1,
             bs=16, nb=40, L=60000, out_dt=1, order=None, ws=A, ws_bytes=1 << 34)
    a.update(kw)
    assert pa._lib.pa_decode_q8b(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q_dt=2, out_dt=2), -2), (dict(D=64), -5), (dict(Hq=4), -4), (dict(seq=2), -3), (dict(seq=-1), -3), (dict(head=2), -3),
    (dict(tile=-1), -3), (dict(limit=99_999), -3), (dict(limit=1_000_000_001), -3), (dict(kc=None), -1), (dict(out=A + 8), -7),
])
def test_decode_q8b_withhold_tile_host_checks(pa, kw, code):
    a = dict(out=A, q=A, q_dt=1, kc=A, vc=A, ks=A, vs=A, tables=A, mb=4096, ctx=A, S=2, Hq=2, Hkv=2, D=128, scale=0.1,
             bs=16, nb=40, L=60000, out_dt=1, seq=1, head=1, tile=0, limit=1_000_000)
    a.update(kw)
    assert pa._lib.pa_decode_q8b_withhold_tile(*a.values(), None) == code


def test_decode_q8b_workspace_bytes(pa):
    f = pa.pa_decode_q8b_workspace_bytes
    assert f(-1, 8, 2, 128, 100) == 0 and f(1, 0, 2, 128, 100) == 0 and f(1, 8, 2, 128, -1) == 0
    assert f(1, 8, 3, 128, 100) == 0 and f(1, 8, 2, 96, 100) == 0 and f(1, 8, 2, 128, (1 << 30) + 1) == 0
    assert f(1, 8, 2, 128, 1 << 30) > 0
    for S, Hq, Hkv, D, L in [(0, 8, 8, 64, 0), (1, 8, 8, 128, 1), (8, 32, 8, 128, 131072), (256, 32, 8, 128, 4096)]:
        n = f(S, Hq, Hkv, D, L)
        assert 0 < n < 1 << 28


@pytest.mark.parametrize("kw,code", [
    (dict(D=96), -5), (dict(bs=8), -6), (dict(n=-1), -3), (dict(H=0), -3), (dict(pairs=None), -1), (dict(vs=None), -1),
    (dict(kc=A + 8), -7), (dict(pairs=A + 4), -7), (dict(count=A + 2), -7), (dict(n=0, pairs=None), 0),
])
def test_copy_blocks_q8b_host_checks(pa, kw, code):
    a = dict(kc=A, vc=A, ks=A, vs=A, pairs=A, count=None, n=3, nb=40, H=2, D=128, bs=16)
    a.update(kw)
    assert pa._lib.pa_copy_blocks_q8b(*a.values(), None) == code


@pytest.mark.parametrize("T", [(1 << 30) + 1, (1 << 31) - 1])
def test_dpool_append_refuses_more_slots_than_it_can_number(pa, T):
    assert pa._lib.pa_dpool_append(A, 64, 16, A, 8, A, A, 4, A, A, T, A, A, None) == -3


def test_append_q8b_refuses_tables_wider_than_its_positions(pa):
    """Positions are 32-bit: a row of 2^27 blocks of 16 would reach 2^31."""
    for mb, bs, code in ((1 << 27, 16, -3), (1 << 26, 32, -3), ((1 << 27) - 1, 16, 0), ((1 << 26) - 1, 32, 0)):
        # (without tokens nothing is launched; the sizes are checked first)
        assert pa._lib.pa_append_q8b(A, A, 1, A, 0, A, A, A, A, A, mb, A, 3, 40, 2, 128, bs, None) == code


@pytest.mark.parametrize("blocks,size", [(40, 32), (41, 16), (39, 16)])
def test_serving_step_refuses_a_pool_of_other_sizes(pa, blocks, size):
    """A pool of more blocks hands out ids that the caches do not have, one of other block size other slots."""
    from types import SimpleNamespace

    from paged_kv_cache_340_b200.batch import ServingStep
    with pytest.raises(ValueError, match="pool"):
        ServingStep(2, 4, 40, 16, 4, 2, 64, 10, device="cpu", pool=SimpleNamespace(num_blocks=blocks, block_size=size))
