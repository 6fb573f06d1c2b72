"""Refusals of the calls that read part of a cache: every one is decided on the host before
anything is launched, so none of this touches a GPU."""
import ctypes

import pytest
import torch

import fp8_kv_cache_write_gb300 as fk

N = ctypes.c_void_p(0)
A = ctypes.c_void_p(4096)              # aligned, never dereferenced: the call is refused
ODD = ctypes.c_void_p(4098)


@pytest.fixture(scope="module")
def lib():
    fk.build()
    return fk.lib()


def test_page_bounds_refusals(lib):
    def call(**k):
        g = lambda n, d: k.get(n, d)
        return lib.fp8kv_kv_page_bounds(g("kc", A), g("dtype", 0), g("mode", 2), N, g("ksc", A),
                                        g("bt", A), g("mbs", 4), g("lens", A), g("B", 2),
                                        g("Hkv", 2), g("D", 128), g("nb", 8), g("new", 1),
                                        g("bounds", A), g("scale", A), N, N)

    assert call(B=0) == 0
    for n in ("B", "mbs", "nb", "new"):
        assert call(**{n: -1}) == -1, n
    assert call(Hkv=0) == -1 and call(mbs=0) == -1 and call(nb=0) == -1
    assert call(D=96) == -2 and call(mbs=(1 << 27) - 31) == -2 and call(nb=1 << 31) == -2
    assert call(dtype=2) == -1 and call(mode=3) == -1 and call(mode=0) == -1   # no scales
    for n in ("kc", "ksc", "bt", "lens", "bounds", "scale"):
        assert call(**{n: N}) == -1, n
        assert call(**{n: ODD}) == -1, n
    # a grid of more than 2^31 warps
    assert call(B=1 << 20, Hkv=64, mbs=1 << 10, new=0) == -2


def test_page_select_refusals(lib):
    def call(**k):
        g = lambda n, d: k.get(n, d)
        return lib.fp8kv_kv_page_select(g("q", A), g("bounds", A), g("scale", A), g("bt", A),
                                        g("mbs", 4), g("lens", A), g("B", 2), g("Hq", 4),
                                        g("Hkv", 2), g("D", 128), g("nb", 8), g("budget", 3),
                                        g("sink", 1), g("recent", 1), g("ws", A),
                                        g("bytes", 64), g("pages", A), g("counts", A), N, N)

    assert call(B=0) == 0
    for n in ("B", "mbs", "nb", "budget", "sink", "recent"):
        assert call(**{n: -1}) == -1, n
    assert call(budget=0, sink=0, recent=0) == -1 and call(sink=2, recent=2) == -1
    assert call(sink=(1 << 31) - 1, recent=(1 << 31) - 1) == -1
    assert call(Hq=5) == -1 and call(Hkv=0) == -1 and call(mbs=0) == -1 and call(nb=0) == -1
    assert call(D=32) == -2 and call(Hq=34) == -2                        # 17 heads a group
    assert call(mbs=(1 << 27) - 31) == -2 and call(nb=1 << 31) == -2
    assert call(B=1 << 30, mbs=1 << 10) == -2
    assert call(bytes=63) == -3 and call(ws=N) == -3 and call(ws=ODD) == -1
    assert fk.kv_page_select_workspace_bytes(2, 2, 4) == 64
    size = ctypes.c_size_t(0)
    for bad, st in (((-1, 2, 4), -1), ((2, 0, 4), -1), ((2, 2, -1), -1), ((2, 2, 1 << 27), -2)):
        assert lib.fp8kv_kv_page_select_workspace_bytes(*bad, ctypes.byref(size)) == st
    assert lib.fp8kv_kv_page_select_workspace_bytes(2, 2, 4, None) == -1
    for n in ("q", "bounds", "scale", "bt", "lens", "pages", "counts"):
        assert call(**{n: N}) == -1, n
        assert call(**{n: ODD}) == -1, n


def test_sparse_attn_refusals(lib):
    def call(**k):
        g = lambda n, d: k.get(n, d)
        return lib.fp8kv_sparse_decode_attn(
            g("q", A), g("kc", A), g("vc", A), g("dtype", 0), g("mode", 2), N, N, g("ksc", A),
            g("vsc", A), g("bt", A), g("mbs", 4), g("lens", A), g("pages", A), g("counts", A),
            g("budget", 3), g("B", 2), g("Hq", 4), g("Hkv", 2), g("D", 128), g("nb", 8),
            g("scale", 0.1), g("out", A), g("od", 1), N, N)

    assert call(B=0) == 0
    for n in ("B", "mbs", "nb", "budget"):
        assert call(**{n: -1}) == -1, n
    assert call(budget=0) == -1 and call(Hq=5) == -1 and call(Hkv=0) == -1
    assert call(mbs=0) == -1 and call(nb=0) == -1
    assert call(D=96) == -2 and call(Hq=34) == -2 and call(nb=1 << 31) == -2
    assert call(mbs=1 << 27) == -2 and call(B=1 << 28) == -2 and call(budget=(1 << 30) + 1) == -2
    assert call(dtype=2) == -1 and call(mode=3) == -1 and call(mode=1) == -1 and call(od=2) == -1
    for bad in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert call(scale=bad) == -1, bad
    for n in ("q", "kc", "vc", "ksc", "vsc", "bt", "lens", "pages", "out"):
        assert call(**{n: N}) == -1, n
        assert call(**{n: ODD}) == -1, n
    assert call(counts=ODD) == -1


def test_prefix_attn_refusals(lib):
    def call(**k):
        g = lambda n, d: k.get(n, d)
        return lib.fp8kv_prefix_decode_attn(
            g("q", A), g("kc", A), g("vc", A), g("dtype", 0), g("mode", 2), N, N, g("ksc", A),
            g("vsc", A), g("pt", A), g("npp", 5), g("plen", A), g("bt", A), g("mbs", 4),
            g("lens", A), g("B", 2), g("Hq", 4), g("Hkv", 2), g("D", 128), g("nb", 8),
            g("scale", 0.1), g("ws", A), g("bytes", 1 << 30), g("out", A), g("od", 1), N, N)

    assert call(B=0) == 0
    for n in ("B", "mbs", "nb", "npp"):
        assert call(**{n: -1}) == -1, n
    assert call(npp=0) == -1 and call(Hq=5) == -1 and call(Hkv=0) == -1
    assert call(mbs=0) == -1 and call(nb=0) == -1
    assert call(D=96) == -2 and call(Hq=34) == -2 and call(nb=1 << 31) == -2
    assert call(mbs=1 << 27) == -2 and call(npp=1 << 27) == -2 and call(B=1 << 25) == -2
    assert call(dtype=2) == -1 and call(mode=3) == -1 and call(mode=1) == -1 and call(od=2) == -1
    for bad in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert call(scale=bad) == -1, bad
    for n in ("q", "kc", "vc", "ksc", "vsc", "pt", "plen", "bt", "lens", "out"):
        assert call(**{n: N}) == -1, n
        assert call(**{n: ODD}) == -1, n
    assert call(ws=N) == -3 and call(bytes=100) == -3 and call(ws=ODD) == -1


def test_prefix_plan(lib):
    """Every size that the call takes has a plan, whose slots hold the pieces that the
    partition can make of a row tile (the arithmetic of csrc/prefix.cuh)."""
    import random
    rng = random.Random(1)
    for _ in range(400):
        Hkv, G, D = rng.randint(1, 8), rng.choice([1, 3, 8, 16]), rng.choice([64, 128, 256])
        B, npp = rng.choice([1, 2, 9, 40, 300]), rng.choice([1, 7, 8, 9, 100, 2048, 9000])
        workers, ws = fk.prefix_attn_plan(B, Hkv * G, Hkv, D, npp)
        keys = 64 if D == 256 else 128
        units = Hkv * -(-B * G // 128)
        splits, rest = divmod(ws, B * G * Hkv * (D + 2) * 4)
        assert rest == 0 and 1 <= workers <= max(152, units)
        for length in {0, 1, 16 * npp // 3, 16 * npp}:
            T = -(-length // keys)
            W = T * units
            n = min(W, workers)
            share = [w * W // n for w in range(n + 1)] if n else [0]
            holder = lambda t: ((t + 1) * n - 1) // W
            seen = 0
            for u in range(units if T else 0):
                first, last = holder(u * T), holder((u + 1) * T - 1)
                assert share[first] <= u * T < share[first + 1]
                assert share[last] < (u + 1) * T <= share[last + 1]
                assert last - first + 1 <= splits
                seen += last - first + 1
            assert seen >= (units if T else 0)
    for bad in ((-1, 4, 2, 64, 1), (1, 5, 2, 64, 1), (1, 4, 0, 64, 1), (1, 4, 2, 64, -1)):
        assert lib.fp8kv_prefix_attn_plan(*bad, None, None) == -1
    assert lib.fp8kv_prefix_attn_plan(1, 4, 2, 32, 1, None, None) == -2
    assert lib.fp8kv_prefix_attn_plan(1, 34, 2, 64, 1, None, None) == -2


def test_limits_and_alignment(lib):
    """Scale caches are read 16 bytes at a time; lists and a CTA's share of the prefix are
    counted in 31 bits."""
    four = ctypes.c_void_p(4100)

    def bounds(ksc=A, mode=2):
        return lib.fp8kv_kv_page_bounds(A, 0, mode, four, ksc, A, 4, A, 2, 2, 128, 8, 0, N, A, N, N)

    def sparse(ksc=A, vsc=A, q=A):
        return lib.fp8kv_sparse_decode_attn(q, A, A, 0, 2, N, N, ksc, vsc, A, 4, A, A, A, 3, 2, 4, 2,
                                            128, 8, 0.1, A, 1, N, N)

    def prefix(ksc=A, vsc=A, B=2, Hq=4, Hkv=2, npp=5, ws=A, bytes=0):
        return lib.fp8kv_prefix_decode_attn(A, A, A, 0, 2, N, N, ksc, vsc, A, npp, A, A, 4, A, B, Hq,
                                            Hkv, 128, 8, 0.1, ws, bytes, A, 1, N, N)

    def select(budget):
        return lib.fp8kv_kv_page_select(A, A, A, A, 4, A, 2, 4, 2, 128, 8, budget, 1, 1, A, 0, A, A, N,
                                        N)

    assert bounds(ksc=four) == -1
    assert sparse(ksc=four) == -1 and sparse(vsc=four) == -1
    assert prefix(ksc=four) == -1 and prefix(vsc=four) == -1
    assert prefix(ws=ctypes.c_void_p(4112), bytes=1 << 30) == -1      # partials: 32 bytes at a time
    assert prefix() == -3 and select(1 << 30) == -3          # good but for the workspace
    assert select((1 << 30) + 1) == -2
    assert prefix(B=1 << 20, Hq=64, Hkv=64, npp=(1 << 27) - 32) == -2
    assert lib.fp8kv_prefix_attn_plan(1 << 20, 64, 64, 128, (1 << 27) - 32, None, None) == -2


def test_binding_refuses_what_it_can_see():
    """Wrong types, shapes and places name the argument (CPU tensors: no call goes out)."""
    i32 = dict(dtype=torch.int32)
    kc, vc = torch.zeros(8, 2, 16, 64, dtype=torch.uint8), torch.zeros(8, 2, 16, 64, dtype=torch.uint8)
    bt, lens = torch.zeros(3, 4, **i32), torch.zeros(3, **i32)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    bounds, scale = torch.zeros(8, 2, 2, 64, dtype=torch.int8), torch.zeros(8, 2)
    s = torch.ones(1)
    kw = dict(kv_dtype=fk.KV_E4M3, k_scale=s)
    with pytest.raises(ValueError, match="k_cache"):
        fk.kv_page_bounds(kc, bt, lens, bounds, scale, **kw)                # not on a GPU
    with pytest.raises(ValueError, match="q"):
        fk.kv_page_select(q, bounds, scale, bt, lens, budget=2)
    with pytest.raises(ValueError, match="q"):
        fk.sparse_decode_attn(q, kc, vc, bt, lens, torch.zeros(3, 2, 2, **i32), v_scale=s, **kw)
    with pytest.raises(ValueError, match="q"):
        fk.prefix_decode_attn(q, kc, vc, bt[0], lens[:1], bt, lens, v_scale=s, **kw)
