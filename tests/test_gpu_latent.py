"""GPU: the latent cache (write, read) and its absorbed attention against plain 64-bit
formulas (tests/_latent.py derives the bounds)."""
import pytest
import torch

import fp8_kv_cache_write_gb300 as fk
from tests._latent import (E4M3_HALF, E4M3_TINY, HALF, assert_close, codes_to_values,
                           latent_attention, latent_values, rotate, table, thetas)

pytestmark = pytest.mark.gpu


def _cache(seed, nb, L, kind, token):
    """Random rows in the cache's own format, with a few strong channels."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(nb, 16, L + 64, generator=g)
    x[..., 3] *= 8
    if kind == "bf16":
        return x.to(torch.bfloat16), None, None
    scale = 0.02
    sc = (torch.rand(nb, 16, generator=g) * 0.03 + 0.005) if token else None
    s = sc[..., None] if token else scale
    return (x / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale, sc


def _pages(seed, lens, mbs, nb):
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    bt = torch.full((len(lens), mbs), -7, dtype=torch.int32)   # unread entries are no page
    at = 0
    for b, n in enumerate(lens):
        pages = min(-(-n // 16), mbs)
        bt[b, :pages] = perm[at:at + pages]
        at += pages
    return bt


def _attend(q, cache, bt, lens, L, scale, sc, kind, softmax_scale, out_dtype=fk.OUT_F32, **kw):
    token = sc is not None
    return fk.latent_decode_attn(
        q.cuda(), cache.cuda(), bt.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
        latent_dim=L, kv_dtype=fk.KV_E4M3 if kind == "e4m3" else fk.KV_BF16,
        scale_mode=fk.SCALE_PER_TOKEN_HEAD if token else fk.SCALE_PER_TENSOR,
        scale=None if scale is None else torch.tensor([scale], device="cuda"),
        scale_cache=None if sc is None else sc.cuda(), softmax_scale=softmax_scale,
        out_dtype=out_dtype, **kw)


def _check_attention(seed, lens, S, H, L, kind, token, out_dtype=fk.OUT_F32, softmax_scale=0.07,
                     num_splits=0, mbs=None):
    mbs = mbs or max(1, max(-(-n // 16) for n in lens) + 1)
    nb = sum(-(-n // 16) for n in lens) + 3
    cache, scale, sc = _cache(seed, nb, L, kind, token)
    bt = _pages(seed, lens, mbs, nb)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn(len(lens), S, H, L + 64, generator=g).to(torch.bfloat16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _attend(q, cache, bt, lens, L, scale, sc, kind, softmax_scale, out_dtype, err_flag=err,
                  num_splits=num_splits)
    torch.cuda.synchronize()
    assert int(err) == 0
    rows = latent_values(cache, kind == "e4m3", scale, sc)
    want, bound = latent_attention(q, rows, bt, lens, L, softmax_scale, kind == "e4m3",
                                   None if sc is None else sc.flatten())
    if out_dtype == fk.OUT_BF16:
        bound = bound + HALF[torch.bfloat16] * (want.abs() + bound)
    assert_close(got.cpu(), want, bound + 1e-30, f"attention {lens} S {S} H {H} L {L} {kind}")
    return got


KINDS = [("e4m3", False), ("e4m3", True), ("bf16", False)]


@pytest.mark.parametrize("kind,token", KINDS)
@pytest.mark.parametrize("H", [16, 64, 1])
def test_one_tile(kind, token, H):
    _check_attention(1, [64], 1, H, 512, kind, token)


@pytest.mark.parametrize("kind,token", KINDS)
@pytest.mark.parametrize("L", [128, 256, 512])
@pytest.mark.parametrize("lens", [[1], [127], [128], [129], [700], [16, 1, 0, 333, 2049]])
def test_lengths(kind, token, L, lens):
    _check_attention(2, lens, 1, 16, L, kind, token)


@pytest.mark.parametrize("kind,token", KINDS)
@pytest.mark.parametrize("H", [1, 3, 16, 20, 33, 64, 65, 128])
def test_heads(kind, token, H):
    _check_attention(3, [300, 77], 1, H, 512, kind, token)


@pytest.mark.parametrize("kind,token", KINDS)
@pytest.mark.parametrize("S,H", [(2, 16), (3, 5), (4, 64), (8, 8), (130, 1)])
def test_several_query_tokens_see_only_what_is_before_them(kind, token, S, H):
    # the 1- and 0-token sequences leave queries that see nothing: zero rows
    got = _check_attention(4, [300, S, 1, 0, 128], S, H, 256, kind, token)
    assert torch.all(got[3] == 0) and (S == 1 or torch.all(got[2, :S - 1] == 0))


@pytest.mark.parametrize("kind,token", KINDS)
def test_splits_agree(kind, token):
    # the same sums in another order: fp32 partials, weights against other references
    outs = [_check_attention(5, [5000, 100, 900], 1, 16, 512, kind, token, num_splits=n)
            for n in (1, 2, 7, 100, 0)]
    assert all(o.shape == outs[0].shape for o in outs)


@pytest.mark.parametrize("kind,token", KINDS)
def test_bf16_output_and_three_dimensional_q(kind, token):
    _check_attention(6, [400, 33], 1, 32, 512, kind, token, out_dtype=fk.OUT_BF16)
    cache, scale, sc = _cache(6, 4, 512, kind, token)
    bt = torch.tensor([[2, 1, 3]], dtype=torch.int32)
    q = torch.randn(1, 16, 576).to(torch.bfloat16)
    a = _attend(q, cache, bt, [40], 512, scale, sc, kind, 0.05)
    b = _attend(q[:, None], cache, bt, [40], 512, scale, sc, kind, 0.05)
    assert a.shape == (1, 16, 512) and torch.equal(a, b[:, 0])


@pytest.mark.parametrize("kind,token", KINDS)
def test_steep_softmax_moves_the_reference(kind, token):
    # logits that grow along the sequence by hundreds of binades: the running
    # reference has to follow
    L, n = 256, 900
    nb = 60
    g = torch.Generator().manual_seed(7)
    x = torch.randn(nb, 16, L + 64, generator=g) * 0.1
    bt = _pages(7, [n], 58, nb)
    ramp = torch.linspace(-3.0, 3.0, n)
    for t in range(n):
        x[bt[0, t // 16], t % 16, 0] = ramp[t]
    q = torch.zeros(1, 1, 16, L + 64)
    q[..., 0] = torch.linspace(-400, 400, 16)
    q = q.to(torch.bfloat16)
    if kind == "bf16":
        cache, scale, sc = x.to(torch.bfloat16), None, None
    else:
        scale, sc = 0.0078125, None
        if token:
            sc = torch.full((nb, 16), 0.0078125)
            sc[::3] *= 64
        s = sc[..., None] if token else scale
        cache = (x / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    got = _attend(q, cache, bt, [n], L, scale, sc, kind, 1.0, num_splits=1)
    rows = latent_values(cache, kind == "e4m3", scale, sc)
    want, bound = latent_attention(q, rows, bt, [n], L, 1.0, kind == "e4m3",
                                   None if sc is None else sc.flatten())
    assert_close(got.cpu(), want, bound, "steep")


@pytest.mark.parametrize("kind,token", KINDS)
@pytest.mark.parametrize("sink", [0, 130, 2999])
@pytest.mark.parametrize("share", [0.5, 0.999])
def test_a_key_that_dwarfs_the_others_leaves_them_their_weight(kind, token, sink, share):
    # one key takes `share` of the softmax, thousands of others split the rest: weights
    # 2^-13 and less of the largest, which e4m3 has no room for under one reference
    L, n, nb, H = 512, 3000, 190, 20
    cache, scale, sc = _cache(21, nb, L, kind, token)
    bt = _pages(21, [n], 189, nb)
    rows = latent_values(cache, kind == "e4m3", scale, sc)
    at = bt[0].long()[torch.arange(n) // 16] * 16 + torch.arange(n) % 16
    g = torch.Generator().manual_seed(22)
    q = torch.randn(1, 1, H, L + 64, generator=g) * 0.1
    x = rows[at]
    # steer q along the sink's row until its logit has the share asked for
    dirn = x[sink] / x[sink].norm() ** 2
    for h in range(H):
        lo, hi = 0.0, 4000.0
        for _ in range(60):
            mid = (lo + hi) / 2
            z = (x @ (q[0, 0, h].double() + mid * dirn)) * 0.07
            lo, hi = (mid, hi) if float(torch.softmax(z, -1)[sink]) < share else (lo, mid)
        q[0, 0, h] += (lo * dirn).float()
    q = q.to(torch.bfloat16)
    got = _attend(q, cache, bt, [n], L, scale, sc, kind, 0.07, num_splits=1).cpu()
    want, bound = latent_attention(q, rows, bt, [n], L, 0.07, kind == "e4m3",
                                   None if sc is None else sc.flatten())
    assert_close(got, want, bound, "sink")
    # the others' part of the result is there, not only the sink's
    p = torch.softmax((q[0, 0].double() @ x.T) * 0.07, -1)
    p[:, sink] = 0
    rest = p @ x[:, :L]
    have = got[0, 0].double() - (want[0, 0] - rest)
    off = (have - rest).norm(dim=-1) / rest.norm(dim=-1)
    if share == 0.5:
        assert float(off.max()) < 0.1, float(off.max())


@pytest.mark.parametrize("kind,token", KINDS)
def test_nan_behind_the_sequence_stays_out(kind, token):
    lens = [37, 150]
    nb, L = 16, 512
    cache, scale, sc = _cache(8, nb, L, kind, token)
    bt = _pages(8, lens, 10, nb)
    q = torch.randn(2, 1, 20, L + 64, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16)
    clean = _attend(q, cache, bt, lens, L, scale, sc, kind, 0.07)
    used = torch.zeros(nb, 16, dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(n):
            used[bt[b, t // 16], t % 16] = True
    if kind == "bf16":
        cache[~used] = float("nan")
    else:
        cache[~used] = 0x7F
        if token:
            sc[~used] = float("nan")
    got = _attend(q, cache, bt, lens, L, scale, sc, kind, 0.07)
    assert torch.equal(got, clean)


@pytest.mark.parametrize("kind,token", KINDS)
def test_bad_pages_are_reported_and_skipped(kind, token):
    lens = [300, 200]
    nb, L = 40, 256
    cache, scale, sc = _cache(9, nb, L, kind, token)
    bt = _pages(9, lens, 20, nb)
    q = torch.randn(2, 1, 16, L + 64, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16)
    bt[0, 0:9] = nb + 5                            # the first tile has no page at all
    bt[1, 5] = -3
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _attend(q, cache, bt, lens, L, scale, sc, kind, 0.07, err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == -6
    rows = latent_values(cache, kind == "e4m3", scale, sc)
    safe = bt.clone()
    safe[(bt < 0) | (bt >= nb)] = nb - 1           # a page of neither sequence's own
    assert not bool((bt == nb - 1).any())
    want, bound = latent_attention(q, rows, safe, lens, L, 0.07, kind == "e4m3",
                                   None if sc is None else sc.flatten(), skip=(nb - 1,))
    assert_close(got.cpu(), want, bound, "skipped pages")


@pytest.mark.parametrize("kind,token", KINDS)
def test_lengths_beyond_the_table_and_below_zero(kind, token):
    L, nb = 256, 12
    cache, scale, sc = _cache(30, nb, L, kind, token)
    bt = torch.randperm(nb, generator=torch.Generator().manual_seed(3))[:9].to(torch.int32).view(3, 3)
    q = torch.randn(3, 1, 16, L + 64, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    want = _attend(q, cache, bt, [48, 0, 17], L, scale, sc, kind, 0.07)
    got = _attend(q, cache, bt, [5000, -3, 17], L, scale, sc, kind, 0.07)
    assert torch.equal(got, want) and torch.all(got[1] == 0)


def test_many_more_sequences_than_workers():
    # shares of several whole sequences, and sequences without keys between them
    g = torch.Generator().manual_seed(31)
    lens = [int(x) for x in torch.randint(0, 70, (400,), generator=g)]
    for i in range(0, 400, 7):
        lens[i] = 0
    _check_attention(31, lens, 1, 16, 128, "e4m3", True)
    _check_attention(32, lens[:200], 1, 70, 128, "bf16", False)


def test_rows_of_zeros_have_scale_zero():
    lens, nb, L = [100, 40], 12, 512
    cache, scale, sc = _cache(10, nb, L, "e4m3", True)
    bt = _pages(10, lens, 8, nb)
    for t in (0, 5, 17, 99):
        cache[bt[0, t // 16], t % 16] = 0
        sc[bt[0, t // 16], t % 16] = 0
    for t in range(40):                            # a sequence of zeros alone
        cache[bt[1, t // 16], t % 16] = 0
        sc[bt[1, t // 16], t % 16] = 0
    q = torch.randn(2, 1, 16, L + 64, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    got = _attend(q, cache, bt, lens, L, scale, sc, "e4m3", 0.07).cpu()
    rows = latent_values(cache, True, scale, sc)
    want, _ = latent_attention(q, rows, bt, lens, L, 0.07, True, sc.flatten())
    # the bound of the other rows: zero rows add nothing to the numerator
    keep = sc.clone()
    keep[keep == 0] = 0.01
    _, bound = latent_attention(q, rows, bt, lens, L, 0.07, True, keep.flatten())
    assert_close(got, want, bound + 1e-30, "zero rows")
    assert torch.all(got[1] == 0)


def test_nan_and_inf_queries_stay_in_their_rows():
    for kind, token in KINDS:
        cache, scale, sc = _cache(11, 8, 512, kind, token)
        bt = _pages(11, [100], 7, 8)
        q = torch.randn(1, 1, 16, 576, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
        clean = _attend(q, cache, bt, [100], 512, scale, sc, kind, 0.07)
        q[0, 0, 3, 100] = float("nan")
        q[0, 0, 7, 0] = float("inf")
        got = _attend(q, cache, bt, [100], 512, scale, sc, kind, 0.07)
        assert torch.isnan(got[0, 0, 3]).all() and torch.isnan(got[0, 0, 7]).all()
        rest = [h for h in range(16) if h not in (3, 7)]
        assert torch.equal(got[0, 0, rest], clean[0, 0, rest])


def test_many_sequences_and_a_long_one():
    g = torch.Generator().manual_seed(12)
    lens = [int(x) for x in torch.randint(0, 200, (70,), generator=g)]
    _check_attention(12, lens, 1, 16, 512, "e4m3", True)
    _check_attention(13, [20011], 1, 64, 512, "e4m3", True)
    _check_attention(14, [9973], 1, 128, 512, "bf16", False)


# ---------------------------------------------------------------- write and read
@pytest.mark.parametrize("kind,token", KINDS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,L", [(1, 1, 128), (5, 20, 512), (65, 128, 256), (300, 0, 512)])
def test_latent_write_matches_the_formula(kind, token, interleaved, T, H, L):
    g = torch.Generator().manual_seed(T + H + L)
    ckr = torch.randn(T, L + 64, generator=g).to(torch.bfloat16)
    ckr[:, L + 2] *= 30                            # a strong rotary channel
    nb = T // 16 + 4
    slots = torch.randperm(nb * 16, generator=g)[:T]
    if T > 4:
        slots[1] = -1
    positions = torch.randint(0, 1 << 20, (T,), generator=g)
    theta = thetas(64)
    dt = torch.uint8 if kind == "e4m3" else torch.bfloat16
    cache = torch.full((nb, 16, L + 64), 9, dtype=dt, device="cuda")
    before = cache.clone()
    sc = torch.full((nb, 16), -1.0, device="cuda")
    scale = torch.full((1,), 0.05, device="cuda")
    d = ckr.cuda()
    q = torch.randn(T, max(H, 1), L + 64, generator=g).to(torch.bfloat16)
    dq = q.cuda()
    q_pe = torch.randn(T, max(H, 1), 64, generator=g).to(torch.bfloat16)
    out = fk.latent_cache_write(
        d[:, :L], d[:, L:], slots.cuda(), cache, kv_dtype=fk.KV_E4M3 if kind == "e4m3" else fk.KV_BF16,
        scale_mode=fk.SCALE_PER_TOKEN_HEAD if token else fk.SCALE_PER_TENSOR, scale=scale,
        scale_cache=sc, positions=positions.cuda(), rope_freqs=table(theta).cuda(),
        interleaved=interleaved, q_pe=q_pe.cuda() if H else None, q_pe_out=dq[..., L:] if H else None)
    torch.cuda.synchronize()
    if H:
        want = rotate(q_pe, positions, theta, interleaved)
        arith = 2.0 ** -20 * q_pe.double().abs().amax(-1, keepdim=True) * 2
        assert_close(dq[..., L:].cpu(), want, HALF[torch.bfloat16] * (want.abs() + arith) + arith,
                     "q_pe")
        assert out.data_ptr() == dq[..., L:].data_ptr()
    assert torch.equal(dq[..., :L].cpu(), q[..., :L])          # untouched
    k = rotate(ckr[:, None, L:], positions, theta, interleaved)[:, 0]
    x = torch.cat((ckr[:, :L].double(), k), -1)
    ok = slots >= 0
    x, at = x[ok], slots[ok]
    arith = torch.zeros_like(x)
    arith[:, L:] = 2.0 ** -20 * 2 * ckr[ok][:, L:].double().abs().amax(-1, keepdim=True)
    got = cache.flatten(0, 1).cpu()[at]
    if kind == "bf16":
        assert_close(got, x, HALF[torch.bfloat16] * (x.abs() + arith) + arith, "rows")
    else:
        if token:
            s = sc.flatten().cpu()[at].double()[:, None]
            want = x.abs().amax(-1, keepdim=True) / 448
            assert_close(s, want, want * 2.0 ** -23 + arith.amax(-1, keepdim=True) / 448, "scales")
        else:
            s = torch.full((x.shape[0], 1), float(scale), dtype=torch.float64)
        want = (x / s).clamp(-448, 448)
        slack = arith / s + want.abs() * 2.0 ** -22
        assert_close(codes_to_values(got), want, (want.abs() + slack) * E4M3_HALF + E4M3_TINY + slack,
                     "codes")
        # the latent part's codes are those of the fp32 quotient, exactly
        exact = (ckr[ok][:, :L].float() / s.float()).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(got[:, :L], exact.view(torch.uint8))
    rest = torch.ones(nb * 16, dtype=torch.bool)
    rest[at] = False
    assert torch.equal(cache.flatten(0, 1)[rest.cuda()], before.flatten(0, 1)[rest.cuda()])


def test_nan_and_inf_stay_in_their_row_and_out_of_its_scale():
    # as in kv_cache_write: the scale is that of the numbers, NaN keeps a NaN code
    T, L = 6, 512
    x = torch.randn(T, L + 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    x[1, 5], x[2, L + 3], x[3, 7] = float("nan"), float("nan"), float("inf")
    d, slots = x.cuda(), torch.arange(T, device="cuda")
    cache = torch.zeros(1, 16, L + 64, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(1, 16, device="cuda")
    fk.latent_cache_write(d[:, :L], d[:, L:], slots, cache, kv_dtype=fk.KV_E4M3,
                          scale_mode=fk.SCALE_PER_TOKEN_HEAD, scale_cache=sc)
    v = codes_to_values(cache.cpu())[0, :T]
    amax = torch.where(torch.isnan(x), 0.0, x.float()).abs().amax(-1)
    assert torch.equal(sc[0, :T].cpu(), amax / 448)
    assert torch.isnan(v[1, 5]) and torch.isnan(v[2, L + 3]) and int(torch.isnan(v[1]).sum()) == 1
    assert torch.equal(torch.isnan(v[[0, 4, 5]]).any(), torch.tensor(False))
    # rotated: the NaN reaches its partner only
    kc = torch.zeros(1, 1, 16, 64, dtype=torch.uint8, device="cuda")
    ks = torch.zeros(1, 1, 16, device="cuda")
    k = x[:, None, :64].clone()
    k[4, 0, 9] = float("nan")
    k = k.cuda()
    fk.rope_kv_cache_write(None, k, k, slots + 3, slots, table(thetas(64)).cuda(), kc, kc.clone(),
                           kv_dtype=fk.KV_E4M3, scale_mode=fk.SCALE_PER_TOKEN_HEAD, k_scale_cache=ks,
                           v_scale_cache=ks.clone())
    nan = torch.isnan(codes_to_values(kc.cpu())[0, 0, 4])
    assert nan.nonzero().flatten().tolist() == [9, 41] and torch.isfinite(ks[0, 0, 4])


def test_latent_write_without_positions_and_in_place():
    T, H, L = 33, 8, 512
    g = torch.Generator().manual_seed(1)
    c, kpe = (torch.randn(T, n, generator=g).to(torch.bfloat16).cuda() for n in (L, 64))
    slots = torch.arange(T, device="cuda") + 16
    cache = torch.zeros(4, 16, L + 64, dtype=torch.bfloat16, device="cuda")
    assert fk.latent_cache_write(c, kpe, slots, cache, kv_dtype=fk.KV_BF16) is None
    assert torch.equal(cache.flatten(0, 1)[slots], torch.cat((c, kpe), 1))
    q = torch.randn(T, H, 64, generator=g).to(torch.bfloat16).cuda()
    ref = rotate(q.cpu(), torch.arange(T), thetas(64), False)
    r = fk.latent_cache_write(c, kpe, slots, cache, kv_dtype=fk.KV_BF16,
                              positions=torch.arange(T, device="cuda"),
                              rope_freqs=table(thetas(64)).cuda(), q_pe=q, q_pe_out=q)
    assert r is q
    assert_close(q.cpu(), ref, HALF[torch.bfloat16] * ref.abs() + 1e-5, "q in place")


@pytest.mark.parametrize("out_dtype", [fk.OUT_F32, fk.OUT_BF16])
@pytest.mark.parametrize("kind,token", KINDS)
@pytest.mark.parametrize("L,T", [(128, 1), (256, 130), (512, 1001)])
def test_latent_read(kind, token, L, T, out_dtype):
    nb = 70
    cache, scale, sc = _cache(L + T, nb, L, kind, token)
    g = torch.Generator().manual_seed(T)
    slots = torch.randint(0, nb * 16, (T,), generator=g)
    if T > 3:
        slots[3] = -1
        slots[0] = nb * 16
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = fk.latent_cache_read(
        cache.cuda(), slots.cuda(), kv_dtype=fk.KV_E4M3 if kind == "e4m3" else fk.KV_BF16,
        scale_mode=fk.SCALE_PER_TOKEN_HEAD if token else fk.SCALE_PER_TENSOR,
        scale=None if scale is None else torch.tensor([scale], device="cuda"),
        scale_cache=None if sc is None else sc.cuda(), out_dtype=out_dtype, err_flag=err)
    ok = (slots >= 0) & (slots < nb * 16)
    at = torch.where(ok, slots, 0)
    x = cache.flatten(0, 1)[at]
    if kind == "e4m3":
        x = x.view(torch.float8_e4m3fn).float() * (sc.flatten()[at][:, None] if token else
                                                    torch.tensor(scale, dtype=torch.float32))
    want = torch.where(ok[:, None], x.float(), 0.0).to(got.dtype)
    assert torch.equal(got.cpu(), want)
    assert int(err) == (-6 if T > 3 else 0)
