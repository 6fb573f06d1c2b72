"""GPU: rotary positions fused with the cache write, and rows read back, against plain
64-bit formulas.  The bounds count the roundings: half a step of the output type, plus
the fp32 arithmetic of a rotation (two products and a sum of values up to |x| + |y|,
with sine and cosine of an angle good to 2^-24 turns)."""
import pytest
import torch

import fp8_kv_cache_write_gb300 as fk
from tests._latent import E4M3_HALF, E4M3_TINY, HALF, assert_close, codes_to_values, rotate, table, thetas

pytestmark = pytest.mark.gpu

MODES = [("e4m3", fk.SCALE_PER_TOKEN_HEAD), ("e4m3", fk.SCALE_PER_TENSOR),
         ("e4m3", fk.SCALE_PER_HEAD), ("bf16", fk.SCALE_PER_TENSOR)]


def _inputs(seed, T, Hq, Hkv, D, spare=4):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16)
    nb = (T + 15) // 16 + spare
    slots = torch.randperm(nb * 16, generator=g)[:T].to(torch.int64)
    return qkv, slots, nb


def _caches(nb, Hkv, D, kind, fill=0x3C):
    if kind == "e4m3":
        k = torch.full((nb, Hkv, 16, D), fill, dtype=torch.uint8, device="cuda")
    else:
        k = torch.full((nb, Hkv, 16, D), 1.5, dtype=torch.bfloat16, device="cuda")
    s = torch.full((nb, Hkv, 16), -2.0, device="cuda")
    return k, k.clone(), s, s.clone()


def _call(qkv, Hq, Hkv, positions, slots, freqs, kc, vc, ks, vs, kind, mode, **kw):
    hs = torch.linspace(0.01, 0.05, Hkv, device="cuda") if mode == fk.SCALE_PER_HEAD else \
        torch.full((1,), 0.02, device="cuda")
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    out = fk.rope_kv_cache_write(
        q if Hq else None, k, v, positions.cuda(), slots.cuda(), freqs.cuda(), kc, vc,
        kv_dtype=fk.KV_E4M3 if kind == "e4m3" else fk.KV_BF16, scale_mode=mode, k_scale=hs,
        v_scale=hs, k_scale_cache=ks, v_scale_cache=vs, **kw)
    return out, hs


def _check_keys(k, kc, ks, hs, slots, kind, mode, arith):
    """Stored keys (and scales) of slots against the rotated 64-bit keys k [T][Hkv][D]."""
    T, Hkv, D = k.shape
    blk, off = slots // 16, slots % 16
    if kind == "bf16":
        got = kc.cpu()[blk, :, off]
        assert_close(got, k, HALF[torch.bfloat16] * (k.abs() + arith) + arith, "bf16 keys")
        return
    codes = codes_to_values(kc.cpu()[blk, :, off])
    if mode == fk.SCALE_PER_TOKEN_HEAD:
        s = ks.cpu()[blk, :, off].double()
        want = k.abs().amax(-1) / 448
        assert_close(s, want, want * 2.0 ** -23 + arith.amax(-1) / 448, "scales")
    elif mode == fk.SCALE_PER_HEAD:
        s = hs.cpu().double()[None].expand(T, Hkv)
    else:
        s = hs.cpu().double()[0].expand(T, Hkv)
    want = torch.clamp(k / s[..., None], -448, 448)
    slack = arith / s[..., None] + want.abs() * 2.0 ** -22
    assert_close(codes, want, (want.abs() + slack) * E4M3_HALF + E4M3_TINY + slack, "key codes")


@pytest.mark.parametrize("kind,mode", MODES)
@pytest.mark.parametrize("D,rd,interleaved", [(64, 64, False), (64, 16, True), (128, 128, False),
                                              (128, 64, False), (128, 112, True), (256, 256, True),
                                              (256, 64, False), (256, 48, True)])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 4, 1), (17, 6, 3), (333, 0, 2)])
def test_rope_write_matches_the_formula(kind, mode, D, rd, interleaved, T, Hq, Hkv):
    qkv, slots, nb = _inputs(D + rd + T + mode, T, Hq, Hkv, D)
    g = torch.Generator().manual_seed(T)
    positions = torch.randint(-5, 1 << 20, (T,), generator=g)
    positions[0] = (1 << 31) + 12345               # far position
    theta = thetas(rd)
    kc, vc, ks, vs = _caches(nb, Hkv, D, kind)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref = [t.clone() for t in (kc, vc, ks, vs)]
    mscale = 1.25
    out, hs = _call(qkv.cuda(), Hq, Hkv, positions, slots, table(theta), kc, vc, ks, vs, kind, mode,
                    interleaved=interleaved, mscale=mscale, err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    # the angle: |position| * theta_i * 2^-53 turns of the table's double, 2^-24 of a
    # turn in fp32; sine and cosine 2 ulp; the rotation 3 roundings
    x = qkv[:, :Hq + Hkv].double()
    both = rotate(x, positions, theta, interleaved, mscale)
    mag = rotate(x.abs(), torch.zeros_like(positions), theta, interleaved, mscale)
    pair = torch.zeros_like(x)
    if interleaved:
        m = mag[..., 0:rd:2] + mag[..., 1:rd:2]
        pair[..., 0:rd:2], pair[..., 1:rd:2] = m, m
    else:
        m = mag[..., :rd // 2] + mag[..., rd // 2:rd]
        pair[..., :rd // 2], pair[..., rd // 2:rd] = m, m
    arith = pair * (2.0 ** -21 + 6.3 * float(positions.abs().max()) * 2.0 ** -53)
    if Hq:
        want = both[:, :Hq]
        assert_close(out.cpu(), want, HALF[torch.bfloat16] * (want.abs() + arith[:, :Hq]) +
                     arith[:, :Hq], "rotated q")
    else:
        assert out is None
    _check_keys(both[:, Hq:], kc, ks, hs, slots, kind, mode, arith[:, Hq:])
    # v, its scales, and every byte of other slots: exactly what kv_cache_write leaves
    v = qkv[:, Hq + Hkv:].contiguous().cuda()
    fk.kv_cache_write(v, v, slots.cuda(), ref[0], ref[1],
                      kv_dtype=fk.KV_E4M3 if kind == "e4m3" else fk.KV_BF16, scale_mode=mode,
                      k_scale=hs, v_scale=hs, k_scale_cache=ref[2], v_scale_cache=ref[3])
    assert torch.equal(vc.view(torch.uint8), ref[1].view(torch.uint8))
    assert torch.equal(vs, ref[3])
    rest = torch.ones(nb * 16, dtype=torch.bool)
    rest[slots] = False
    rest = rest.cuda()
    assert torch.equal(kc.transpose(1, 2).flatten(0, 1)[rest].view(torch.uint8),
                       ref[0].transpose(1, 2).flatten(0, 1)[rest].view(torch.uint8))
    assert torch.equal(ks.transpose(1, 2).flatten(0, 1)[rest],
                       ref[2].transpose(1, 2).flatten(0, 1)[rest])


def test_zero_angle_is_the_plain_write():
    # position 0 turns nothing: codes, scales and q are those of the unrotated rows
    qkv, slots, nb = _inputs(5, 100, 4, 2, 128)
    qkv[7] = 0                                     # zero rows: scale 0, codes 0
    kc, vc, ks, vs = _caches(nb, 2, 128, "e4m3")
    ref = [t.clone() for t in (kc, vc, ks, vs)]
    d = qkv.cuda()
    out, _ = _call(d, 4, 2, torch.zeros(100, dtype=torch.int64), slots, table(thetas(128)), kc, vc,
                   ks, vs, "e4m3", fk.SCALE_PER_TOKEN_HEAD)
    fk.kv_cache_write(d[:, 4:6].contiguous(), d[:, 6:].contiguous(), slots.cuda(), ref[0], ref[1],
                      kv_dtype=fk.KV_E4M3, scale_mode=fk.SCALE_PER_TOKEN_HEAD, k_scale_cache=ref[2],
                      v_scale_cache=ref[3])
    assert torch.equal(out, d[:, :4])
    for a, b in zip((kc, vc, ks, vs), ref):
        assert torch.equal(a, b)


def _every_bf16():
    return torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)


# ordinary, around the range in which quotients need no divide, subnormal, huge, negative, 0
SCALES = [0.02, 1.0, 448.0, 1.2345678e-3, 2.0 ** -89, 2.0 ** -90 * 1.75, 2.0 ** -91 * 1.75,
          2.0 ** 117 * 1.999, 2.0 ** 118, 3e38, 1e-40, -0.37, 0.0, float("inf"), float("nan"),
          0.1 / 3]


def test_codes_of_every_bf16_value():
    # v rows are stored as they are: the codes are those of kv_cache_write
    v = _every_bf16().view(512, 1, 128).expand(512, len(SCALES), 128).contiguous().cuda()
    slots = torch.arange(512, device="cuda")
    hs = torch.tensor(SCALES, device="cuda")
    kc, vc, _, _ = _caches(32, len(SCALES), 128, "e4m3")
    ref = [kc.clone(), vc.clone()]
    kw = dict(kv_dtype=fk.KV_E4M3, scale_mode=fk.SCALE_PER_HEAD, k_scale=hs, v_scale=hs)
    fk.rope_kv_cache_write(None, torch.zeros_like(v), v, slots, slots, table(thetas(128)).cuda(),
                           kc, vc, **kw)
    fk.kv_cache_write(torch.zeros_like(v), v, slots, *ref, **kw)
    for h, s in enumerate(SCALES):
        assert torch.equal(vc[:, h], ref[1][:, h]), s


def test_codes_of_rows_of_every_magnitude():
    # rows' own scales: every power of two, infinities, subnormal rows whose scale is 0
    g = torch.Generator().manual_seed(8)
    x = torch.randn(268, 1, 128, generator=g, dtype=torch.float64)
    x = (x * 2.0 ** (torch.arange(268, dtype=torch.float64) - 138)[:, None, None])
    x = x.clamp(-3.3e38, 3.3e38).to(torch.bfloat16)
    x[100, 0, 5] = float("inf")
    x[101, 0, 6] = float("-inf")
    v = x.cuda()
    slots = torch.arange(268, device="cuda")
    kc, vc, ks, vs = _caches(17, 1, 128, "e4m3")
    ref = [t.clone() for t in (kc, vc, ks, vs)]
    kw = dict(kv_dtype=fk.KV_E4M3, scale_mode=fk.SCALE_PER_TOKEN_HEAD)
    fk.rope_kv_cache_write(None, v, v, torch.zeros_like(slots), slots, table(thetas(128)).cuda(),
                           kc, vc, k_scale_cache=ks, v_scale_cache=vs, **kw)
    fk.kv_cache_write(v, v, slots, ref[0], ref[1], k_scale_cache=ref[2], v_scale_cache=ref[3], **kw)
    assert torch.equal(vs, ref[3])
    assert torch.equal(vc, ref[1])


@pytest.mark.parametrize("scale", SCALES)
def test_latent_codes_of_every_bf16_value(scale):
    # unrotated latent rows hold the codes kv_cache_write gives their 128- and 64-wide pieces
    T, L = 1024, 512
    c = _every_bf16().view(1, -1).expand(8, 65536).reshape(T, L).contiguous().cuda()
    kp = _every_bf16().view(T, 64).contiguous().cuda()
    slots = torch.arange(T, device="cuda")
    s = torch.full((1,), scale, device="cuda")
    cache = torch.full((64, 16, L + 64), 0x3C, dtype=torch.uint8, device="cuda")
    fk.latent_cache_write(c, kp, slots, cache, kv_dtype=fk.KV_E4M3, scale=s)
    for part, D in ((c, 128), (kp, 64)):
        rows = part.view(T, -1, D)
        ref = torch.zeros(64, rows.shape[1], 16, D, dtype=torch.uint8, device="cuda")
        fk.kv_cache_write(rows, rows, slots, ref, ref.clone(), kv_dtype=fk.KV_E4M3, k_scale=s,
                          v_scale=s)
        got = cache.view(T, L + 64)[:, :L] if D == 128 else cache.view(T, L + 64)[:, L:]
        assert torch.equal(got, ref.transpose(1, 2).reshape(T, -1))


def test_in_place_q_padding_and_bad_slots():
    T, Hq, Hkv, D = 40, 4, 2, 128
    qkv, slots, nb = _inputs(6, T, Hq, Hkv, D)
    slots[::5] = -1                                # padding
    slots[3] = nb * 16                             # outside
    positions = torch.arange(T) + 9
    kc, vc, ks, vs = _caches(nb, Hkv, D, "e4m3")
    before = [t.clone() for t in (kc, vc, ks, vs)]
    d = qkv.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, _ = _call(d, Hq, Hkv, positions, slots, table(thetas(D)), kc, vc, ks, vs, "e4m3",
                   fk.SCALE_PER_TOKEN_HEAD, q_out=d[:, :Hq], err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == -6
    assert out.data_ptr() == d.data_ptr()
    want = rotate(qkv[:, :Hq], positions, thetas(D), False)
    assert_close(d[:, :Hq].cpu(), want, HALF[torch.bfloat16] * want.abs() + 1e-5, "q in place")
    assert torch.equal(d[:, Hq:].cpu(), qkv[:, Hq:])
    ok = (slots >= 0) & (slots < nb * 16)
    written = torch.zeros(nb * 16, dtype=torch.bool)
    written[slots[ok]] = True
    for a, b in zip((kc, vc), before[:2]):
        same = (a == b).all(-1).transpose(1, 2).flatten(0, 1).all(-1).cpu()
        assert bool(same[~written].all()) and not bool(same[written].any())


@pytest.mark.parametrize("out_dtype", [fk.OUT_F32, fk.OUT_BF16])
@pytest.mark.parametrize("kind,mode", MODES)
@pytest.mark.parametrize("D,Hkv,T", [(64, 1, 1), (64, 5, 77), (128, 8, 300), (256, 3, 1000)])
def test_read_back_is_code_times_scale(kind, mode, D, Hkv, T, out_dtype):
    g = torch.Generator().manual_seed(D + Hkv + T)
    nb = 40
    if kind == "e4m3":
        kc = torch.randint(0, 256, (nb, Hkv, 16, D), generator=g, dtype=torch.uint8)
        kc[(kc & 0x7F) == 0x7F] = 0x7E             # no NaN codes
        vc = kc.flip(0).contiguous()
    else:
        kc = torch.randn(nb, Hkv, 16, D, generator=g).to(torch.bfloat16)
        vc = kc.flip(0).contiguous()
    ks, vs = torch.rand(nb, Hkv, 16, generator=g), torch.rand(nb, Hkv, 16, generator=g)
    hk, hv = torch.rand(Hkv, generator=g) + 0.1, torch.rand(Hkv, generator=g) + 0.1
    slots = torch.randint(0, nb * 16, (T,), generator=g)
    if T > 4:
        slots[2] = -1                              # a zero row
        slots[4] = slots[1]                        # the same row twice
    k, v = fk.kv_cache_read(kc.cuda(), vc.cuda(), slots.cuda(), kv_dtype=fk.KV_E4M3 if kind == "e4m3"
                            else fk.KV_BF16, scale_mode=mode, k_scale=hk.cuda(), v_scale=hv.cuda(),
                            k_scale_cache=ks.cuda(), v_scale_cache=vs.cuda(), out_dtype=out_dtype)
    blk, off = slots.clamp_min(0) // 16, slots.clamp_min(0) % 16
    for got, c, sc, hs in ((k, kc, ks, hk), (v, vc, vs, hv)):
        x = c[blk, :, off]
        if kind == "e4m3":
            x = x.view(torch.float8_e4m3fn).float()
            x = x * (sc[blk, :, off][..., None] if mode == fk.SCALE_PER_TOKEN_HEAD else
                     hs[None, :, None] if mode == fk.SCALE_PER_HEAD else hs[0])
        want = torch.where((slots >= 0)[:, None, None], x.float(), 0.0)
        want = want.to(torch.float32 if out_dtype == fk.OUT_F32 else torch.bfloat16)
        assert got.dtype == want.dtype and torch.equal(got.cpu(), want)


def test_read_outside_the_cache_sets_the_error_and_zeroes():
    kc = torch.full((2, 1, 16, 64), 0x38, dtype=torch.uint8, device="cuda")
    slots = torch.tensor([0, 32, 1 << 40, 31], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = fk.kv_cache_read(kc, kc, slots, kv_dtype=fk.KV_E4M3, k_scale=torch.ones(1, device="cuda"),
                            v_scale=torch.ones(1, device="cuda"), err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == -6
    assert torch.equal(k[:, 0, 0].cpu().float(), torch.tensor([1.0, 0.0, 0.0, 1.0]))


def test_large_rows_of_many_tokens():
    # enough tokens that a warp takes a whole token's rows
    T, Hq, Hkv, D = 5001, 10, 3, 64
    qkv, slots, nb = _inputs(8, T, Hq, Hkv, D)
    kc, vc, ks, vs = _caches(nb, Hkv, D, "e4m3")
    positions = torch.arange(T) + 100000
    out, hs = _call(qkv.cuda(), Hq, Hkv, positions, slots, table(thetas(D)), kc, vc, ks, vs, "e4m3",
                    fk.SCALE_PER_TOKEN_HEAD)
    x = rotate(qkv[:, :Hq + Hkv], positions, thetas(D), False)
    mag = qkv[:, :Hq + Hkv].double().abs()
    arith = (mag + mag.roll(D // 2, -1)) * 2.0 ** -21
    assert_close(out.cpu(), x[:, :Hq], HALF[torch.bfloat16] * (x[:, :Hq].abs() + arith[:, :Hq]) +
                 arith[:, :Hq], "rotated q")
    _check_keys(x[:, Hq:], kc, ks, hs, slots, "e4m3", fk.SCALE_PER_TOKEN_HEAD, arith[:, Hq:])
