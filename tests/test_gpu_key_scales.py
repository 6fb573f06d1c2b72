"""Key scales of zero (a head of keys that are all zero) and below it, one for the cache or one a
head: every attention call takes them as it takes any other factor (tests/_sparse.py says how
the bounds on results are derived)."""
import pytest
import torch

import fp8_kv_cache_write_gb300 as fk
from _latent import assert_close, codes_to_values, latent_attention, latent_values
from _sparse import Cache, attend, bounds_of, rounded
from test_gpu_latent import _attend, _cache, _pages
from test_gpu_prefix import Batch

pytestmark = pytest.mark.gpu

DEV = "cuda"
SCALES = [[0.0], [-0.011], [0.01, 0.0, -0.02]]         # the last: a scale a head


def _kind(scales):
    return "tensor" if len(scales) == 1 else "head"


def _close(got, want, bound, what):
    assert bool(torch.isfinite(got).all()), what       # (a NaN compares as within any bound)
    assert_close(got, want, bound, what)


def _rescale(c, scales):
    """The keys of a cache under other scales."""
    s = torch.tensor(scales)
    c.kw["k_scale"] = s.to(DEV)
    c.val["k"] = codes_to_values(c.k.cpu()) * s.double().view(1, -1, 1, 1)


def _prefix_expect(b, softmax_scale, prefix_pages=None):
    """As Batch.expect, at any softmax scale.  A weight of the prefix's part is one f16 term at
    the least (2^-11 of it), a query's values are off by up to 2^-17 of its largest."""
    c = b.c
    want, bound = torch.zeros(b.q.shape).double(), torch.zeros(b.q.shape).double()
    for h in range(c.Hkv):
        pp = range(-(-c.lens[0] // 16)) if prefix_pages is None else prefix_pages
        pk, pv = c.rows("k", 0, h, pp), c.rows("v", 0, h, pp)
        for s in range(b.B):
            tp = range(-(-c.lens[s + 1] // 16))
            k = torch.cat((pk, c.rows("k", s + 1, h, tp)))
            v = torch.cat((pv, c.rows("v", s + 1, h, tp)))
            for g in range(h * b.G, (h + 1) * b.G):
                weight = 2.0 ** -11 + 2.0 ** -16 * float(
                    b.q[s, g].abs().max() * pk.abs().sum(1).max()) * softmax_scale
                want[s, g], bound[s, g] = attend(b.q[s, g].double(), k, v, softmax_scale, weight)
                bound[s, g] += len(v) * 2.0 ** -30 * float(v.abs().max())
    return want, rounded(bound, want, False)


@pytest.mark.parametrize("scales", SCALES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefix_attention(D, scales):
    """Tiles that are full, end early, and hold a page that is not there."""
    for prefix in (1, 127, 128, 300, 1024):
        b = Batch(100 + prefix, prefix, [0, 40], 3, 2, D, _kind(scales))
        _rescale(b.c, scales)
        want, bound = _prefix_expect(b, D ** -0.5)
        _close(b.run().cpu(), want, bound, f"prefix {prefix}")
        assert int(b.err) == 0
    b.prefix_table[3] = -1
    want, bound = _prefix_expect(b, D ** -0.5, [p for p in range(64) if p != 3])
    _close(b.run().cpu(), want, bound, "a page that is not there")
    assert int(b.err) == -6


def test_prefix_factors_that_vanish():
    """A softmax scale and a key scale whose product is no fp32 number but zero: every key weighs
    the same."""
    b = Batch(400, 100, [0, 20], 1, 4, 64, "tensor")
    _rescale(b.c, [1e-20])
    want, bound = _prefix_expect(b, 1e-30)
    _close(b.run(softmax_scale=1e-30).cpu(), want, bound, "vanishing factor")


@pytest.mark.parametrize("scales", SCALES)
def test_decode_sparse_and_bounds(scales):
    """The whole decode, the sparse one and the page bounds over the same cache."""
    D = 128
    c = Cache(500, [200, 33, 16], 3, D, _kind(scales))
    _rescale(c, scales)
    q = torch.randn(3, 6, D, generator=torch.Generator().manual_seed(501)).to(torch.bfloat16)
    want, bound = torch.zeros(q.shape).double(), torch.zeros(q.shape).double()
    for b, n in enumerate(c.lens):
        for g in range(6):
            pages = range(-(-n // 16))
            want[b, g], bound[b, g] = attend(q[b, g].double(), c.rows("k", b, g // 2, pages),
                                             c.rows("v", b, g // 2, pages), D ** -0.5)
    bound = rounded(bound, want, False)
    pages = torch.arange(c.mbs, dtype=torch.int32, device=DEV).expand(3, 3, -1).contiguous()
    out = fk.sparse_decode_attn(q.to(DEV), c.k, c.v, c.dtable, c.dlens, pages, **c.args(fk))
    _close(out.cpu(), want, bound, "sparse")
    out = fk.paged_decode_attn(q.to(DEV), c.k, c.v, c.dtable, c.dlens, **c.args(fk))
    _close(out.cpu(), want, torch.full_like(bound, 4e-3), "decode")
    bounds = torch.zeros(c.nb, 3, 2, D, dtype=torch.int8, device=DEV)
    scale = torch.zeros(c.nb, 3, device=DEV)
    fk.kv_page_bounds(c.k, c.dtable, c.dlens, bounds, scale, **c.args(fk, "k"))
    for b, n in enumerate(c.lens):
        for p in range(-(-n // 16)):
            for h in range(3):
                hi, lo, s = bounds_of(c.rows("k", b, h, [p]).float())
                blk = int(c.table[b, p])
                assert float(scale[blk, h]) == float(s)
                assert torch.equal(bounds[blk, h].cpu(), torch.stack((hi, lo)))


def _prefill_bound(z, v, single, weight):
    """Bound on a prefill row by its weights' rounding, from its logits z and its values v.  A
    weight is stored relative to a reference at most as large as the largest, in one e4m3
    term (off by 2^-4 of it or by half of the smallest step, 2^-10) or two with a lift of 2^8
    (2^-8, 2^-18); the sum it is divided by is of the stored weights.  So a row is off by
    sum_t d_t |v_t - o| over the stored weights' sum, d_t the rounding; `weight`: what fp32 adds."""
    eps, tiny = (2.0 ** -4, 2.0 ** -10) if single else (2.0 ** -8, 2.0 ** -18)
    p, l = torch.softmax(z, 0), float(torch.exp(z - z.max()).sum())
    d = eps * p + tiny / l
    return (d @ (v.abs() + (p @ v).abs())) / (1 - eps - len(z) * tiny / l) + weight


@pytest.mark.parametrize("two_level", [False, True])
@pytest.mark.parametrize("scales", SCALES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefill(D, scales, two_level):
    """Split operands (the short rows) and single ones (those of 8192 keys and more).  Keys like
    N(0, 1): within the prefill's stated 1e-2.  The head of keys like N(0, 4), for which that
    is not stated: of the query as it is stored, and within the bound by the weights' rounding."""
    lens, chunk, G = [8300, 70, 16], 9, 2
    c = Cache(600, lens, 3, D, _kind(scales))
    _rescale(c, scales)
    q = torch.randn(3 * chunk, 3 * G, D, generator=torch.Generator().manual_seed(601)).to(torch.bfloat16)
    cu = torch.arange(0, 4 * chunk, chunk, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = fk.prefill_attn(q.to(DEV), cu, chunk, c.k, c.v, c.dtable, c.dlens, two_level=two_level,
                          err_flag=err, **c.args(fk))
    want, bound = torch.zeros(q.shape).double(), torch.full(q.shape, 1e-2).double()
    for b, n in enumerate(lens):
        single = n - chunk >= 8192
        for h in range(3):
            k, v = (c.rows(x, b, h, range(-(-n // 16))) for x in "kv")
            far = abs(scales[h % len(scales)]) > 0.011
            for i in range(chunk):
                m = n - chunk + i + 1
                for g in range(h * G, (h + 1) * G):
                    x = q[b * chunk + i, g].double()
                    if far and single:
                        x = x.float().to(torch.float8_e4m3fn).double()
                    # (split: the query's two terms miss 2^-17 of its largest value at most)
                    weight = 0.0 if single else 2.0 ** -16 * float(x.abs().max() * k.abs().sum(1).max())
                    o, fp32 = attend(x, k[:m], v[:m], D ** -0.5, weight)
                    want[b * chunk + i, g] = o
                    if far:
                        bound[b * chunk + i, g] = _prefill_bound(k[:m] @ x * D ** -0.5, v[:m], single, fp32)
    _close(out.cpu(), want, bound, "prefill")
    assert int(err) == 0


@pytest.mark.parametrize("scale", [0.0, -0.011])
@pytest.mark.parametrize("H", [16, 64])
def test_latent(H, scale):
    """The latent attention, whose one scale is keys' and values' at once."""
    nb, L, lens = 40, 256, [300, 17]
    cache, _, _ = _cache(700, nb, L, "e4m3", False)
    bt = _pages(701, lens, 20, nb)
    q = torch.randn(2, 1, H, L + 64, generator=torch.Generator().manual_seed(702)).to(torch.bfloat16)
    got = _attend(q, cache, bt, lens, L, scale, None, "e4m3", 0.07).cpu()
    rows = latent_values(cache, True, scale, None)
    want, bound = latent_attention(q, rows, bt, lens, L, 0.07, True)
    _close(got, want, bound + 1e-30, "latent")
