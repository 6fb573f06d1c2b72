"""What a weight of a shared prefix's part may be off by, and references that move under one
scale for the cache or one a head (tests/_sparse.py says how the bounds on results are derived)."""
import pytest
import torch

from _latent import assert_close, codes_to_values
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


@pytest.mark.parametrize("kind", ["tensor", "head"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("grow", [1, -1])
def test_references_that_move_under_one_scale(D, kind, grow):
    """Keys that grow along the prefix (or shrink): the references of most rows pass by more than
    2^8 from tile to tile, up to hundreds of binades in all.  A weight is one f16 term (2^-11)."""
    b = Batch(200 + D, 1500, [i % 40 for i in range(37)], 16, 5, D, kind)     # 2 row tiles a head
    c = b.c
    k = codes_to_values(c.k.cpu())
    for p in range(b.npp):
        k[int(c.table[0, p])] *= 2.0 ** ((p // 12 if grow > 0 else (b.npp - 1 - p) // 12) - 6)
    code = k.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    c.k = code.to(DEV)
    c.kw["k_scale"] = c.kw["k_scale"] * 64
    c.val["k"] = codes_to_values(code) * c.kw["k_scale"].cpu().double().view(1, -1, 1, 1)
    keys = 64 if D == 256 else 128
    want, bound = torch.zeros(b.q.shape).double(), torch.zeros(b.q.shape).double()
    moves = torch.zeros(b.q.shape[:2])
    for h in range(c.Hkv):
        pp = range(b.npp)
        pk, pv = c.rows("k", 0, h, pp), c.rows("v", 0, h, pp)
        for s in range(b.B):
            tp = range(-(-c.lens[s + 1] // 16))
            kk = torch.cat((pk, c.rows("k", s + 1, h, tp)))
            vv = torch.cat((pv, c.rows("v", s + 1, h, tp)))
            for g in range(5 * h, 5 * h + 5):
                x = b.q[s, g].double()
                weight = 2.0 ** -11 + 2.0 ** -16 * float(x.abs().max() * pk.abs().sum(1).max()) * D ** -0.5
                want[s, g], bound[s, g] = attend(x, kk, vv, D ** -0.5, weight)
                bound[s, g] += len(vv) * 2.0 ** -30 * float(vv.abs().max())
                top = torch.stack([t.max() for t in (pk @ x * D ** -0.5 * 1.4426950408889634).split(keys)])
                moves[s, g] = (top.cummax(0).values.diff() > 8).sum()
    if grow > 0:
        assert float((moves >= 2).float().mean()) > 0.9      # the test tests what it says
    first = b.run()
    _close(first.cpu(), want, rounded(bound, want, False), "first")
    for _ in range(5):
        assert torch.equal(b.run(), first)
    assert int(b.err) == 0
