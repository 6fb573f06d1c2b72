"""How far a page's 8-bit score may lie from what it stands for, the sum over a group's query
heads of the largest q . x over keys x between the page's channels' extremes, and so what a page
left out can at most hold more than one taken.  Ordinary keys and keys with an outlier channel."""
import pytest
import torch

import fp8_kv_cache_write_gb300 as fk
from _sparse import Cache, query_codes

pytestmark = pytest.mark.gpu

DEV = "cuda"
HALF_CODE = 0.5 + 2.0 ** -16         # a code: half a step, and 127 of fp32's 2^-24 in the quotient


def _cache(kind, D, outlier):
    c = Cache(300 + D, [3001, 700], 2, D, kind)
    x = torch.randn(c.nb, 2, 16, D, generator=torch.Generator().manual_seed(301)) * 4
    x[..., 3] *= outlier
    if kind == "bf16":
        c.k = x.to(torch.bfloat16).to(DEV)
        c.val["k"] = c.k.cpu().double()
    else:
        code = x.clamp(-448, 448).to(torch.float8_e4m3fn)
        s = torch.rand(c.nb, 2, 16, generator=torch.Generator().manual_seed(302)) * 0.01 + 0.2
        c.k, c.kw["k_scale_cache"] = code.view(torch.uint8).to(DEV), s.to(DEV)
        c.val["k"] = code.double() * s[..., None].double()
    return c


@pytest.mark.parametrize("outlier", [1.0, 20.0])
@pytest.mark.parametrize("kind", ["token", "bf16"])
@pytest.mark.parametrize("D,G", [(64, 1), (128, 4), (256, 8)])
def test_scores_and_the_pages_taken(D, G, kind, outlier):
    c = _cache(kind, D, outlier)
    q = torch.randn(2, 2 * G, D, generator=torch.Generator().manual_seed(303)).to(torch.bfloat16)
    bounds = torch.zeros(c.nb, 2, 2, D, dtype=torch.int8, device=DEV)
    scale = torch.zeros(c.nb, 2, device=DEV)
    fk.kv_page_bounds(c.k, c.dtable, c.dlens, bounds, scale, **c.args(fk, "k"))
    pages, counts = fk.kv_page_select(q.to(DEV), bounds, scale, c.dtable, c.dlens, budget=20)
    bounds, scale, pages = bounds.cpu(), scale.cpu().double(), pages.cpu()
    assert counts.tolist() == [[20, 20], [20, 20]]
    for b, n in enumerate(c.lens):
        m = -(-n // 16)
        blk = c.table[b, :m].long()
        for h in range(2):
            x = torch.stack([torch.cat((r.amax(0), r.amin(0)))
                             for r in (c.rows("k", b, h, [p]) for p in range(m))])      # [m][2 D]
            qh = q[b, h * G:(h + 1) * G].double()
            u = torch.cat((qh.clamp(min=0).sum(0), qh.clamp(max=0).sum(0)))
            upper = x @ u
            per_head = sum((torch.maximum(x[:, :D] * g, x[:, D:] * g)).sum(1) for g in qh)
            assert torch.allclose(upper, per_head, rtol=1e-12, atol=1e-9)        # what it stands for
            sq = float((u.float().abs().max() / torch.tensor(127.0)).double())
            sp = scale[blk, h]
            score = (bounds[blk, h].reshape(m, -1).double() @ query_codes(q[b, h * G:(h + 1) * G]).double()) * sp * sq
            # c s is off by half a step of s from u, a bound by half a step of its scale from x
            off = (u.abs().sum() * sp + x.abs().sum(1) * sq + 2 * D * HALF_CODE * sp * sq) * HALF_CODE
            off = off + 2.0 ** -23 * (score.abs() + (x.abs() @ u.abs()))          # roundings of fp32
            assert bool(((score - upper).abs() <= off).all())
            taken = torch.zeros(m, dtype=torch.bool)
            taken[pages[b, h].long()] = True
            assert bool(taken[0]) and bool(taken[m - 1])                          # the forced ones
            chosen = taken.clone()
            chosen[0] = chosen[m - 1] = False
            assert float((upper - off)[~taken].max()) <= float((upper + off)[chosen].min())
