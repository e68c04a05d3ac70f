"""pa_decode_q8b and pa_append_q8b where they are easily wrong: a wait that runs
out while further work has been claimed."""
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
