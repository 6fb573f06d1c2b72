"""Refusals of the rotary, cache-read and latent calls: every one is decided on the
host before anything is launched, so none of this touches a GPU."""
import ctypes
import os
import re

import pytest
import torch

import fp8_kv_cache_write_gb300 as fk

N = ctypes.c_void_p(0)
A = ctypes.c_void_p(4096)              # aligned, never dereferenced: the call is refused
ODD = ctypes.c_void_p(4100)


@pytest.fixture(scope="module")
def lib():
    fk.build()
    return fk.lib()


def _constant(name):
    text = open(os.path.join(os.path.dirname(__file__), "..", "include", "fp8kv.h")).read()
    m = re.search(name + r"\s*=?\s*(\d+)", text)
    return int(m.group(1))


def test_constants_match_the_header():
    assert _constant("define FP8KV_LATENT_ROPE") == fk.LATENT_ROPE
    for n in ("NONE", "LINEAR", "NTK", "YARN", "BANDS"):
        assert _constant("FP8KV_ROPE_" + n) == getattr(fk, "ROPE_" + n)


def test_rope_write_refusals(lib):
    def call(**k):
        g = lambda n, d: k.get(n, d)
        return lib.fp8kv_rope_kv_cache_write(
            g("q", A), g("qs", 512), g("k", A), g("ks", 256), g("v", A), 256, g("pos", A),
            g("slots", A), g("freqs", A), g("rd", 128), 0, g("mscale", 1.0), g("T", 3), g("Hq", 4),
            g("Hkv", 2), g("D", 128), g("qo", A), g("qos", 512), g("kc", A), A, g("nb", 4),
            g("dtype", 0), g("mode", 2), N, N, g("ksc", A), A, N, N)

    assert call(T=0) == 0
    assert call(T=-1) == -1 and call(Hkv=0) == -1 and call(Hq=-1) == -1 and call(nb=-1) == -1
    assert call(D=96) == -2
    assert call(rd=0) == -1 and call(rd=144) == -1 and call(rd=24) == -2
    assert call(mscale=float("nan")) == -1
    assert call(dtype=2) == -1 and call(mode=3) == -1
    for n in ("q", "k", "v", "pos", "slots", "freqs", "qo", "kc", "ksc"):
        assert call(**{n: N}) == -1, n
    for n in ("q", "k", "v", "qo", "kc", "pos", "slots", "freqs"):
        assert call(**{n: ODD}) == -1, n
    assert call(mode=0) == -1                          # per tensor without scales
    assert call(qs=500) == -1 and call(qs=516) == -1   # rows overlap; rows not 16-byte aligned
    assert call(ks=248) == -1 and call(qos=8) == -1
    assert call(T=1 << 40) == -2 and call(Hq=70000) == -2


def test_read_refusals(lib):
    def call(**k):
        g = lambda n, d: k.get(n, d)
        return lib.fp8kv_kv_cache_read(g("kc", A), g("vc", A), g("nb", 4), g("dtype", 0),
                                       g("mode", 2), N, N, g("ksc", A), A, g("slots", A), g("T", 3),
                                       g("Hkv", 2), g("D", 128), g("ko", A), g("vo", A),
                                       g("od", 1), N, N)

    assert call(T=0) == 0
    assert call(T=-1) == -1 and call(Hkv=0) == -1 and call(nb=-1) == -1 and call(od=2) == -1
    assert call(D=80) == -2 and call(T=1 << 40) == -2
    assert call(dtype=3) == -1 and call(mode=-1) == -1 and call(mode=1) == -1
    for n in ("kc", "vc", "ksc", "slots", "ko", "vo"):
        assert call(**{n: N}) == -1, n
    for n in ("kc", "vc", "ko", "vo"):
        assert call(**{n: ODD}) == -1, n

    def latent(**k):
        g = lambda n, d: k.get(n, d)
        return lib.fp8kv_latent_cache_read(g("c", A), g("nb", 4), g("dtype", 0), g("mode", 2), N,
                                           g("sc", A), g("slots", A), g("T", 3), g("L", 512),
                                           g("out", A), g("od", 0), N, N)

    assert latent(T=0) == 0 and latent(L=192) == -2 and latent(T=-2) == -1
    for n in ("c", "sc", "slots", "out"):
        assert latent(**{n: N}) == -1, n
    assert latent(out=ODD) == -1 and latent(mode=0) == -1 and latent(od=7) == -1


def test_latent_write_refusals(lib):
    def call(**k):
        g = lambda n, d: k.get(n, d)
        return lib.fp8kv_latent_cache_write(
            g("c", A), g("cs", 576), g("kpe", A), g("kps", 576), g("pos", A), g("freqs", A), 0,
            g("mscale", 1.0), g("slots", A), g("T", 3), g("L", 512), g("cache", A), g("nb", 4),
            g("dtype", 0), g("mode", 2), N, g("sc", A), g("q", A), g("qs", 512), g("qh", 64),
            g("qo", A), g("qos", 4608), g("qoh", 576), g("H", 8), N, N)

    assert call(T=0) == 0
    assert call(L=500) == -2 and call(T=-1) == -1 and call(H=-1) == -1
    assert call(pos=N) == -1 and call(freqs=N) == -1   # both or neither
    assert call(q=N) == -1 and call(qo=N) == -1 and call(H=0) == -1
    for n in ("c", "kpe", "slots", "cache", "sc"):
        assert call(**{n: N}) == -1, n
    for n in ("c", "kpe", "cache", "q", "qo"):
        assert call(**{n: ODD}) == -1, n
    assert call(cs=504) == -1 and call(kps=56) == -1 and call(cs=580) == -1
    assert call(qh=60) == -1 and call(qs=100) == -1 and call(qoh=68) == -1
    assert call(mscale=float("nan")) == -1 and call(H=70000) == -2


def test_latent_attention_refusals(lib):
    def call(**k):
        g = lambda n, d: k.get(n, d)
        return lib.fp8kv_latent_decode_attn(
            g("q", A), g("cache", A), g("dtype", 0), g("mode", 2), N, g("sc", A), g("bt", A),
            g("mbs", 10), g("lens", A), g("B", 2), g("S", 1), g("H", 16), g("L", 512), g("nb", 40),
            g("scale", 0.1), g("splits", 0), g("ws", A), g("wsb", 0), g("out", A), g("od", 0), N, N)

    assert call(B=0) == 0
    assert call(B=-1) == -1 and call(S=0) == -1 and call(H=0) == -1 and call(splits=-1) == -1
    assert call(L=64) == -2 and call(L=384) == -2
    assert call(mbs=0) == -1 and call(nb=0) == -1
    for s in (0.0, -0.1, float("nan"), float("inf")):
        assert call(scale=s) == -1
    assert call(S=2000, H=128) == -2 and call(B=1 << 17) == -2 and call(nb=1 << 31) == -2
    assert call(mbs=1 << 28) == -2
    for n in ("q", "cache", "sc", "bt", "lens", "out"):
        assert call(**{n: N}) == -1, n
    for n in ("q", "cache", "out"):
        assert call(**{n: ODD}) == -1, n
    assert call() == -3                                # workspace too small
    assert call(ws=N, wsb=1 << 40) == -3
    assert call(ws=ODD, wsb=1 << 40) == -1


def test_latent_plan(lib):
    # workers fill the 152 SMs that a machine without a GPU plans for, one CTA per
    # group of at most 64 rows; the workspace holds two partials a CTA
    for B, S, H, L, mbs in [(8, 1, 128, 512, 1375), (1, 1, 16, 512, 64), (32, 2, 16, 256, 2048),
                            (1, 1, 1, 128, 1), (4, 3, 65, 512, 100)]:
        w, ws = fk.latent_attn_plan(B, S, H, L, mbs)
        groups = -(-S * H // 64)
        rows = -(-S * H // groups)
        cols = 16 if rows <= 16 else 32 if rows <= 32 else 64
        assert 1 <= w <= max(1, 152 // groups)
        assert w <= B * -(-mbs // 4)
        assert ws == 2 * w * groups * cols * (L + 2) * 4
        assert fk.latent_attn_plan(B, S, H, L, mbs, 3)[0] == min(3, B * -(-mbs // 4))
    for bad in [(-1, 1, 16, 512, 4), (1, 0, 16, 512, 4), (1, 1, 0, 512, 4), (1, 1, 16, 512, -1)]:
        with pytest.raises(fk.Fp8kvError):
            fk.latent_attn_plan(*bad)


def test_binding_checks_come_before_the_library():
    T, nb = 4, 2
    x = torch.zeros(T, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                    # host tensors
        fk.rope_kv_cache_write(x, x, x, torch.zeros(T, dtype=torch.int64),
                               torch.zeros(T, dtype=torch.int64), torch.zeros(64, dtype=torch.int64),
                               torch.zeros(nb, 2, 16, 128, dtype=torch.uint8),
                               torch.zeros(nb, 2, 16, 128, dtype=torch.uint8), kv_dtype=fk.KV_E4M3)
    with pytest.raises(TypeError):
        fk.latent_decode_attn(torch.zeros(1, 16, 576), torch.zeros(2, 16, 576, dtype=torch.uint8),
                              torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                              latent_dim=512, kv_dtype=fk.KV_E4M3, softmax_scale=0.1)
    with pytest.raises(ValueError):
        fk.kv_cache_read(torch.zeros(2, 2, 16, 128, dtype=torch.uint8),
                         torch.zeros(2, 2, 16, 128, dtype=torch.uint8),
                         torch.zeros(3, dtype=torch.int64), kv_dtype=fk.KV_E4M3)
    with pytest.raises(ValueError):
        fk.latent_cache_read(torch.zeros(2, 16, 576, dtype=torch.bfloat16),
                             torch.zeros(3, dtype=torch.int64), kv_dtype=fk.KV_BF16)
