"""GPU: what a latent call must not depend on or let through."""
import pytest
import torch

import fp8_kv_cache_write_gb300 as fk
from tests._latent import (HALF, assert_close, latent_attention, latent_values, rotate, table,
                           thetas)
from tests.test_gpu_latent import KINDS, _attend, _cache, _pages

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,token", KINDS)
@pytest.mark.parametrize("S,H,n", [(2, 16, 40), (3, 5, 129), (4, 32, 66), (2, 64, 300), (130, 1, 200)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_row_that_a_query_does_not_see_stays_out_of_it(value, kind, token, S, H, n):
    # the last token's latent holds NaN (or inf): the queries in front of it are what they
    # are without it
    if kind == "e4m3" and value == float("inf"):
        pytest.skip("no infinite code")
    nb, L = 24, 256
    cache, scale, sc = _cache(41, nb, L, kind, token)
    bt = _pages(41, [n], 20, nb)
    q = torch.randn(1, S, H, L + 64, generator=torch.Generator().manual_seed(42)).to(torch.bfloat16)
    clean = _attend(q, cache, bt, [n], L, scale, sc, kind, 0.07).cpu()
    for lost in (1, 2) if S > 2 else (1,):           # the last row, or the last two
        for t in range(n - lost, n):
            blk, off = int(bt[0, t // 16]), t % 16
            for dim in (0, 77, 200, L - 1):
                if kind == "bf16":
                    cache[blk, off, dim] = value
                else:
                    cache[blk, off, dim] = 0x7F if dim % 2 else 0xFF
        got = _attend(q, cache, bt, [n], L, scale, sc, kind, 0.07).cpu()
        assert torch.equal(got[0, :S - lost], clean[0, :S - lost])
        if value != value:                           # (an infinite logit may be -inf: no weight)
            assert bool(torch.isnan(got[0, S - lost:]).all())


@pytest.mark.parametrize("kind,token", KINDS)
@pytest.mark.parametrize("bad", [-1, -2, -3, -2 ** 31, 2 ** 31 - 1])
def test_every_id_outside_the_cache_is_reported(kind, token, bad):
    lens, nb, L = [300, 90], 40, 128
    cache, scale, sc = _cache(43, nb, L, kind, token)
    bt = _pages(43, lens, 20, nb - 1)                # the last block is nobody's
    q = torch.randn(2, 1, 16, L + 64, generator=torch.Generator().manual_seed(44)).to(torch.bfloat16)
    bt[0, 7] = bad
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _attend(q, cache, bt, lens, L, scale, sc, kind, 0.07, err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == -6
    rows = latent_values(cache, kind == "e4m3", scale, sc)
    safe = bt.clone()
    safe[0, 7] = nb - 1
    want, bound = latent_attention(q, rows, safe, lens, L, 0.07, kind == "e4m3",
                                   None if sc is None else sc.flatten(), skip=(nb - 1,))
    assert_close(got.cpu(), want, bound, "skipped page")


def test_the_same_call_gives_the_same_bits():
    # the sums' order is fixed: what a call gives does not depend on timing
    lens, nb, L = [2500, 700, 1300], 300, 512
    for kind, token in KINDS:
        cache, scale, sc = _cache(45, nb, L, kind, token)
        cache, sc = cache.cuda(), None if sc is None else sc.cuda()
        bt = _pages(45, lens, 160, nb)
        q = torch.randn(3, 1, 128, L + 64, generator=torch.Generator().manual_seed(46)).to(torch.bfloat16)
        q = (q * 3).cuda()
        first = _attend(q, cache, bt, lens, L, scale, sc, kind, 0.07)
        for _ in range(100):
            assert torch.equal(_attend(q, cache, bt, lens, L, scale, sc, kind, 0.07), first)


@pytest.mark.parametrize("T,H", [(1, 8), (5, 20), (33, 1), (40, 128)])
def test_queries_with_heads_outside_tokens(T, H):
    # q_pe and q_pe_out as [H][T][64] in memory, and one of them so
    L = 256
    g = torch.Generator().manual_seed(T + H)
    c = torch.randn(T, L, generator=g).to(torch.bfloat16).cuda()
    k_pe = torch.randn(T, 64, generator=g).to(torch.bfloat16).cuda()
    q_pe = torch.randn(T, H, 64, generator=g).to(torch.bfloat16)
    pos = torch.arange(T) + 900
    kw = dict(kv_dtype=fk.KV_BF16, positions=pos.cuda(), rope_freqs=table(thetas(64)).cuda())
    want = rotate(q_pe, pos, thetas(64), False)
    slots = torch.arange(T, device="cuda")
    cache = torch.zeros(-(-T // 16), 16, L + 64, dtype=torch.bfloat16, device="cuda")
    heads_first = lambda x: x.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    ref = fk.latent_cache_write(c, k_pe, slots, cache, q_pe=q_pe.cuda(), **kw)
    assert_close(ref.cpu(), want, HALF[torch.bfloat16] * want.abs() + 1e-4, "q_pe")
    for src in (q_pe.cuda(), heads_first(q_pe)):
        for dst in (None, heads_first(torch.zeros_like(q_pe)), heads_first(
                torch.zeros(T, H, L + 64, dtype=torch.bfloat16))[..., L:]):
            got = fk.latent_cache_write(c, k_pe, slots, cache, q_pe=src, q_pe_out=dst, **kw)
            assert torch.equal(got, ref)
    own = heads_first(q_pe)
    assert fk.latent_cache_write(c, k_pe, slots, cache, q_pe=own, q_pe_out=own, **kw) is own
    assert torch.equal(own, ref)
    if T * H > 1:                                    # outputs that overlap
        with pytest.raises(fk.Fp8kvError):
            fk.latent_cache_write(c, k_pe, slots, cache, q_pe=q_pe.cuda(), q_pe_out=torch.zeros(
                64, dtype=torch.bfloat16, device="cuda").expand(T, H, 64), **kw)
