"""What a weight of a shared prefix's part may be off by (tests/_sparse.py says how the bounds on
results are derived)."""
import pytest
import torch

from _latent import assert_close
from _sparse import attend, rounded
from test_gpu_prefix import Batch

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _close(got, want, bound, what):
    assert bool(torch.isfinite(got).all()), what       # (a NaN compares as within any bound)
    assert_close(got, want, bound, what)


@pytest.mark.parametrize("kind", ["token", "tensor", "head", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_key_that_outweighs_the_rest(D, kind):
    """Two keys, the first with 2^30 times the other's weight and more: the row is its value.
    Under value scales of its own its weight is one f16 term, half a step of which is 2^-11 of
    it; else it is a power of two, but for what fp32 loses."""
    b = Batch(100, 2, [0] * 20, 8, 3, D, kind)
    c, blk = b.c, int(b.c.table[0, 0])
    c.k[blk, :, 0] = 0x7E if c.e4m3 else 4.0                    # 448
    c.k[blk, :, 1] = 0
    scale = 1.0 if not c.e4m3 else (c.kw["k_scale_cache"][blk, :, 0] if kind == "token"
                                    else c.kw["k_scale"].expand(8)).cpu().double().view(8, 1)
    c.val["k"][blk, :, 0] = (448.0 if c.e4m3 else 4.0) * scale
    c.val["k"][blk, :, 1] = 0.0
    b.q = b.q.abs() + 0.5
    b.dq = b.q.to(DEV)
    want, bound = torch.zeros(b.q.shape).double(), torch.zeros(b.q.shape).double()
    for s in range(b.B):
        for g in range(24):
            k, v = (c.rows(x, 0, g // 3, [0]) for x in "kv")
            assert float((k[0] - k[1]) @ b.q[s, g].double()) * D ** -0.5 * 1.4427 > 30
            want[s, g], bound[s, g] = attend(b.q[s, g].double(), k, v, D ** -0.5,
                                             2.0 ** -11 if kind == "token" else 0.0)
            bound[s, g] += 2.0 ** -30 * float(v.abs().max())
    _close(b.run().cpu(), want, rounded(bound, want, False), "outweighed")
    assert int(b.err) == 0
