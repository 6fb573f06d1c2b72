"""Sizes that the latent attention refuses, on the host before anything is launched."""
import ctypes

import pytest

import fp8_kv_cache_write_gb300 as fk

N = ctypes.c_void_p(0)
A = ctypes.c_void_p(4096)              # aligned, never dereferenced: the call is refused


@pytest.fixture(scope="module")
def lib():
    fk.build()
    return fk.lib()


def attend(lib, **k):
    g = lambda n, d: k.get(n, d)
    return lib.fp8kv_latent_decode_attn(
        A, A, 0, 2, N, A, A, g("mbs", 10), A, g("B", 2), g("S", 1), g("H", 16), 512, 40,
        g("scale", 0.1), 0, A, 0, A, 0, N, N)


def test_tables_whose_positions_would_pass_32_bits(lib):
    # a length is taken up to max_blocks_per_seq pages and rounded up to whole tiles of 128,
    # two of which are looked ahead, in 32-bit arithmetic
    for mbs in ((1 << 27) - 1, (1 << 27) - 31, 1 << 27, 1 << 30):
        assert attend(lib, mbs=mbs) == -2, mbs
    assert attend(lib, mbs=(1 << 27) - 32) == -3       # goes on to the workspace's size


def test_a_plan_refuses_what_the_call_refuses(lib):
    # so that nobody allocates gigabytes for a call that cannot run
    for B, S, H, mbs in ((2, 2000, 128, 10), (2, 65535, 65535, 10), (65536, 1, 16, 10),
                         (2, 1, 16, (1 << 27) - 31)):
        assert attend(lib, B=B, S=S, H=H, mbs=mbs) == -2
        with pytest.raises(fk.Fp8kvError) as e:
            fk.latent_attn_plan(B, S, H, 512, mbs)
        assert e.value.status == -2
    assert fk.latent_attn_plan(65535, 1, 16, 512, 10)[1] > 0
    assert fk.latent_attn_plan(1, 512, 128, 512, (1 << 27) - 32)[1] > 0


def test_a_softmax_scale_that_overflows_in_binades(lib):
    # the kernel takes it times log2(e), in fp32
    assert attend(lib, scale=3e38) == -1
    assert attend(lib, scale=2.3e38) == -3
