"""GPU: rows whose offsets in a cache pass 32 bits, in the rotary, read and latent calls.
The caches are larger than 4 GiB; only the rows in use are ever written."""
import pytest
import torch

import fp8_kv_cache_write_gb300 as fk
from tests._latent import HALF, assert_close, latent_attention, rotate, table, thetas

pytestmark = pytest.mark.gpu


def test_rotary_write_and_read():
    T, Hkv, D = 40, 8, 256
    nb = (1 << 32) // (Hkv * 16 * D) + 500            # bytes of e4m3; values of bf16
    g = torch.Generator().manual_seed(1)
    slots = torch.cat((torch.arange(T // 2), nb * 16 - 1 - torch.arange(T - T // 2)))
    pos = torch.arange(T) + 77
    qkv = torch.randn(T, 3 * Hkv, D, generator=g).to(torch.bfloat16)
    want = rotate(qkv[:, Hkv:2 * Hkv], pos, thetas(D), False)
    d = qkv.cuda()
    for kv, dt in ((fk.KV_E4M3, torch.uint8), (fk.KV_BF16, torch.bfloat16)):
        kc = torch.empty(nb, Hkv, 16, D, dtype=dt, device="cuda")
        vc = torch.empty_like(kc)
        ks, vs = torch.empty(nb, Hkv, 16, device="cuda"), torch.empty(nb, Hkv, 16, device="cuda")
        kw = dict(kv_dtype=kv, scale_mode=fk.SCALE_PER_TOKEN_HEAD, k_scale_cache=ks, v_scale_cache=vs)
        fk.rope_kv_cache_write(d[:, :Hkv], d[:, Hkv:2 * Hkv], d[:, 2 * Hkv:], pos.cuda(), slots.cuda(),
                               table(thetas(D)).cuda(), kc, vc, **kw)
        k, v = fk.kv_cache_read(kc, vc, slots.cuda(), out_dtype=fk.OUT_F32, **kw)
        for got, x in ((k.cpu(), want), (v.cpu(), qkv[:, 2 * Hkv:].double())):
            # half a step of the cache's type (tiny codes: 2^-10 of the scale), and fp32's
            top = x.abs().amax(-1, keepdim=True)
            half = 2.0 ** -4 if kv == fk.KV_E4M3 else HALF[torch.bfloat16]
            tiny = top / 448 * 2.0 ** -10 if kv == fk.KV_E4M3 else 0.0
            assert_close(got, x, x.abs() * half * (1 + 2.0 ** -10) + tiny + top * 2.0 ** -18, "rows")
        del kc, vc, ks, vs


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
def test_latent_write_read_and_attention(kind):
    n, L, H = 200, 512, 16
    e4m3 = kind == "e4m3"
    nb = (1 << 32) // (16 * (L + 64) * (1 if e4m3 else 2)) + 500
    g = torch.Generator().manual_seed(2)
    x = torch.randn(n, L + 64, generator=g).to(torch.bfloat16)
    pages = torch.cat((torch.arange(6), nb - 1 - torch.arange(7)))       # first and last blocks
    slots = pages[torch.arange(n) // 16] * 16 + torch.arange(n) % 16
    cache = torch.empty(nb, 16, L + 64, dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda")
    sc = torch.empty(nb, 16, device="cuda")
    kw = dict(kv_dtype=fk.KV_E4M3 if e4m3 else fk.KV_BF16, scale_mode=fk.SCALE_PER_TOKEN_HEAD,
              scale_cache=sc)
    d = x.cuda()
    fk.latent_cache_write(d[:, :L], d[:, L:], slots.cuda(), cache, **kw)
    rows = fk.latent_cache_read(cache, slots.cuda(), out_dtype=fk.OUT_F32, **kw).double().cpu()
    top = x.double().abs().amax(-1, keepdim=True)
    bound = x.double().abs() * 2.0 ** -4 * (1 + 2.0 ** -10) + top / 448 * 2.0 ** -10 if e4m3 else 0 * x
    assert_close(rows, x.double(), bound, "rows")
    q = torch.randn(1, 1, H, L + 64, generator=g).to(torch.bfloat16)
    out = fk.latent_decode_attn(q.cuda(), cache, pages.to(torch.int32)[None].cuda(),
                                torch.tensor([n], dtype=torch.int32, device="cuda"), latent_dim=L,
                                softmax_scale=0.07, **kw)
    order = torch.arange(13, dtype=torch.int32)[None]                    # the rows read, in order
    padded = torch.cat((rows, torch.zeros(13 * 16 - n, L + 64, dtype=torch.float64)))
    scales = torch.cat((sc.view(-1)[slots.cuda()].cpu(), torch.ones(13 * 16 - n))) if e4m3 else None
    want, bound = latent_attention(q, padded, order, [n], L, 0.07, e4m3, scales)
    assert_close(out.cpu(), want, bound, "attention")
