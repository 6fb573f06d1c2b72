"""GPU: the calls together, as a decode loop uses them -- eagerly, captured in a graph and
replayed, on other streams, with outputs at odd offsets -- against plain 64-bit formulas."""
import math

import pytest
import torch

import fp8_kv_cache_write_gb300 as fk
from tests._latent import (HALF, assert_close, codes_to_values, latent_attention, latent_values,
                           rotate, table, thetas)

pytestmark = pytest.mark.gpu


def _pages(lens, mbs, nb, seed):
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    return perm[:len(lens) * mbs].reshape(len(lens), mbs)


class Latent:
    """A latent-attention layer's state: a prompt stored, then decode steps."""

    def __init__(self, kind, token, lens, H=16, L=512, steps=3, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.token, self.H, self.L = kind, token, H, L
        self.lens = list(lens)
        B = len(lens)
        mbs = max(-(-(n + steps) // 16) for n in lens)
        self.nb = B * mbs + 2
        self.bt = _pages(lens, mbs, self.nb, seed)
        dt = torch.uint8 if kind == "e4m3" else torch.bfloat16
        self.cache = torch.full((self.nb, 16, L + 64), 0x7F, dtype=torch.uint8).to(dt).cuda()
        if kind != "e4m3":
            self.cache.fill_(float("nan"))
        self.sc = torch.full((self.nb, 16), float("nan"), device="cuda")
        self.scale = torch.full((1,), 0.02, device="cuda")
        self.theta = thetas(64)
        self.freqs = table(self.theta).cuda()
        self.kw = dict(kv_dtype=fk.KV_E4M3 if kind == "e4m3" else fk.KV_BF16,
                       scale_mode=fk.SCALE_PER_TOKEN_HEAD if token else fk.SCALE_PER_TENSOR,
                       scale=self.scale, scale_cache=self.sc)
        rows = [(b, t) for b, n in enumerate(lens) for t in range(n)]
        self.store([b for b, _ in rows], [t for _, t in rows],
                   torch.randn(len(rows), L + 64, generator=g).to(torch.bfloat16))
        self.g = g
        self.ws = torch.empty(fk.latent_attn_plan(B, 1, H, L, mbs)[1], dtype=torch.uint8, device="cuda")

    def slot(self, b, t):
        return int(self.bt[b, t // 16]) * 16 + t % 16

    def store(self, bs, ts, x):
        slots = torch.tensor([self.slot(b, t) for b, t in zip(bs, ts)], device="cuda")
        d = x.cuda()
        fk.latent_cache_write(d[:, :self.L], d[:, self.L:], slots, self.cache,
                              positions=torch.tensor(ts, device="cuda"), rope_freqs=self.freqs, **self.kw)

    def check(self, q_out, lens, q_nope, q_pe, softmax_scale):
        B = len(lens)
        rows = latent_values(self.cache.cpu(), self.kind == "e4m3", 0.02 if not self.token else None,
                             self.sc.cpu() if self.token else None)
        pos = torch.tensor([n - 1 for n in lens])
        q = torch.cat((q_nope.double(), rotate(q_pe, pos, self.theta, False)), -1)
        q = q.to(torch.bfloat16)
        # q is rounded to bf16 either way; a rotation next to a rounding boundary may land
        # one bf16 step apart: half a step of z's terms, 2^-8 |q_pe . k|, twice in out
        want, bound = latent_attention(q[:, None], rows, self.bt, lens, self.L, softmax_scale,
                                       self.kind == "e4m3", self.sc.cpu().flatten() if self.token else None)
        live = torch.isfinite(rows[:, self.L:]).all(-1)
        k_pe = rows[live][:, self.L:].abs().amax(0)
        dz = 2.0 ** -8 * float((q_pe.double().abs().amax((0, 1)) @ k_pe)) * softmax_scale
        mags = rows[live][:, :self.L].abs().amax(0)
        assert_close(q_out.cpu(), want[:, 0], bound[:, 0] + 2 * dz * mags, "decode step")


@pytest.mark.parametrize("kind,token", [("e4m3", True), ("e4m3", False), ("bf16", False)])
def test_latent_decode_steps_eager_and_replayed(kind, token):
    lens = [37, 200, 16]
    B, scale = len(lens), 1 / math.sqrt(192)
    st = Latent(kind, token, lens)
    L, H = st.L, st.H
    static = {"x": torch.zeros(B, L + 64, dtype=torch.bfloat16, device="cuda"),
              "q": torch.zeros(B, H, L + 64, dtype=torch.bfloat16, device="cuda"),
              "q_pe": torch.zeros(B, H, 64, dtype=torch.bfloat16, device="cuda"),
              "pos": torch.zeros(B, dtype=torch.int64, device="cuda"),
              "slots": torch.full((B,), -1, dtype=torch.int64, device="cuda"),
              "lens": torch.zeros(B, dtype=torch.int32, device="cuda"),
              "out": torch.zeros(B, H, L, device="cuda"), "bt": st.bt.cuda()}

    def step():
        s = static
        fk.latent_cache_write(s["x"][:, :L], s["x"][:, L:], s["slots"], st.cache, positions=s["pos"],
                              rope_freqs=st.freqs, q_pe=s["q_pe"], q_pe_out=s["q"][..., L:], **st.kw)
        fk.latent_decode_attn(s["q"], st.cache, s["bt"], s["lens"], latent_dim=L, softmax_scale=scale,
                              workspace=st.ws, out=s["out"], **st.kw)

    graph = None
    for i in range(4):
        now = [n + 1 for n in st.lens] if i < 3 else st.lens
        x = torch.randn(B, L + 64, generator=st.g).to(torch.bfloat16)
        q_nope = torch.randn(B, H, L, generator=st.g).to(torch.bfloat16)
        q_pe = torch.randn(B, H, 64, generator=st.g).to(torch.bfloat16)
        static["x"].copy_(x)
        static["q"][..., :L].copy_(q_nope)
        static["q_pe"].copy_(q_pe)
        static["pos"].copy_(torch.tensor([n - 1 for n in now]))
        static["lens"].copy_(torch.tensor(now, dtype=torch.int32))
        static["slots"].copy_(torch.tensor([st.slot(b, n - 1) for b, n in enumerate(now)]))
        if i == 0:
            step()
        else:
            if graph is None:                  # captured with other contents than replayed
                saved = [t.clone() for t in (st.cache, st.sc)]
                side = torch.cuda.Stream()
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    step()
                torch.cuda.current_stream().wait_stream(side)
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
                st.cache.copy_(saved[0])
                st.sc.copy_(saved[1])
            graph.replay()
        torch.cuda.synchronize()
        st.lens = now
        st.check(static["out"], now, q_nope, q_pe, scale)
    # and back: the rows a fresh read gives are the cache's values, rounded once
    slots = torch.tensor([st.slot(b, t) for b, n in enumerate(st.lens) for t in range(n)], device="cuda")
    got = fk.latent_cache_read(st.cache, slots, out_dtype=fk.OUT_F32, **st.kw)
    rows = latent_values(st.cache.cpu(), kind == "e4m3", float(st.scale), st.sc.cpu() if token else None)
    want = rows[slots.cpu()]
    assert_close(got.cpu(), want, want.abs() * 2.0 ** -24, "read back")


def test_two_graphs_on_two_streams_with_their_own_workspaces():
    a, b = Latent("e4m3", True, [300, 21], seed=1), Latent("bf16", False, [77, 1000], seed=2)
    runs = []
    for st in (a, b):
        q = torch.randn(2, st.H, st.L + 64, generator=st.g).to(torch.bfloat16)
        lens = torch.tensor(st.lens, dtype=torch.int32, device="cuda")
        out = torch.zeros(2, st.H, st.L, device="cuda")
        args = (q.cuda(), st.cache, st.bt.cuda(), lens)
        call = lambda args=args, st=st, out=out: fk.latent_decode_attn(
            *args, latent_dim=st.L, softmax_scale=0.07, workspace=st.ws, out=out, **st.kw)
        want = call().clone()
        torch.cuda.synchronize()
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=stream):
            call()
        out.zero_()
        runs.append((stream, graph, out, want))
    torch.cuda.synchronize()
    for _ in range(20):
        for stream, graph, _, _ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, out, want in runs:
        assert torch.equal(out, want)


def test_another_stream_and_its_own_allocations():
    st = Latent("e4m3", True, [500, 90], seed=3)
    q = torch.randn(2, st.H, st.L + 64, generator=st.g).to(torch.bfloat16).cuda()
    lens = torch.tensor(st.lens, dtype=torch.int32, device="cuda")
    bt = st.bt.cuda()
    call = lambda **kw: fk.latent_decode_attn(q, st.cache, bt, lens, latent_dim=st.L,
                                              softmax_scale=0.07, **kw, **st.kw)
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        got = call(stream=side)                # output and workspace allocated for `side`
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]
        side.synchronize()
        assert torch.equal(got, want)
        del junk
    k = fk.latent_cache_read(st.cache, torch.arange(64, device="cuda"), stream=side, **st.kw)
    side.synchronize()
    assert torch.equal(k.nan_to_num(), fk.latent_cache_read(
        st.cache, torch.arange(64, device="cuda"), **st.kw).nan_to_num())


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
def test_rotary_write_then_paged_decode(kind):
    # a prompt stored through the rotary write, then one decode step over it: softmax over
    # the rotated, quantised keys
    lens, Hq, Hkv, D, rd = [40, 129], 8, 2, 128, 64
    g = torch.Generator().manual_seed(4)
    nb, mbs = 20, 9
    bt = _pages(lens, mbs, nb, 4)
    dt = torch.uint8 if kind == "e4m3" else torch.bfloat16
    kc = torch.zeros(nb, Hkv, 16, D, dtype=dt, device="cuda")
    vc = torch.zeros_like(kc)
    ks = torch.zeros(nb, Hkv, 16, device="cuda")
    vs = torch.zeros_like(ks)
    kw = dict(kv_dtype=fk.KV_E4M3 if kind == "e4m3" else fk.KV_BF16,
              scale_mode=fk.SCALE_PER_TOKEN_HEAD if kind == "e4m3" else fk.SCALE_PER_TENSOR,
              k_scale_cache=ks, v_scale_cache=vs)
    freqs, mscale = fk.rope_freqs(rd, 10000.0, scaling=fk.ROPE_YARN, factor=4.0, original_context=64,
                                  device="cuda")
    theta = [int(f) * 2 * math.pi / 2 ** 64 for f in freqs.tolist()]
    rows = [(b, t) for b, n in enumerate(lens) for t in range(n)]
    qkv = torch.randn(len(rows), Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16)
    slots = torch.tensor([int(bt[b, t // 16]) * 16 + t % 16 for b, t in rows])
    pos = torch.tensor([t for _, t in rows])
    d = qkv.cuda()
    q = fk.rope_kv_cache_write(d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], pos.cuda(), slots.cuda(),
                               freqs, kc, vc, mscale=mscale, **kw)
    last = [sum(lens[:b + 1]) - 1 for b in range(len(lens))]
    out = fk.paged_decode_attn(q[last].contiguous(), kc, vc, bt.cuda(),
                               torch.tensor(lens, dtype=torch.int32, device="cuda"), **kw)
    k, v = fk.kv_cache_read(kc, vc, slots.cuda(), out_dtype=fk.OUT_F32, **kw)
    k, v = k.double().cpu(), v.double().cpu()
    # keys are the rotated rows within e4m3's half step (2^-4; tiny ones 2^-10 of the scale)
    kr = rotate(qkv[:, Hq:Hq + Hkv], pos, theta, False, mscale)
    half = 2.0 ** -4 if kind == "e4m3" else 2.0 ** -8
    floor = kr.abs().amax(-1, keepdim=True) / 448 * 2.0 ** -10 * (kind == "e4m3")
    assert_close(k, kr, kr.abs() * half * (1 + 2.0 ** -10) + floor + 1e-5, "keys")
    for b, n in enumerate(lens):
        at = range(last[b] - n + 1, last[b] + 1)
        for h in range(Hq):
            kk, vv = k[at][:, h // (Hq // Hkv)], v[at][:, h // (Hq // Hkv)]
            p = torch.softmax(kk @ q[last[b], h].double().cpu() / math.sqrt(D), -1)
            # the decode's stated bound for its fp32 output on N(0,1) values
            assert_close(out[b, h].cpu(), p @ vv, torch.full((D,), 4e-3, dtype=torch.float64), "decode")


def test_outputs_at_odd_offsets():
    # outputs that start 16 but not 32 bytes aligned take the narrower stores
    g = torch.Generator().manual_seed(5)
    kc = torch.randint(0, 120, (6, 2, 16, 64), generator=g, dtype=torch.uint8).cuda()
    one = torch.ones(1, device="cuda")
    slots = torch.randperm(96, generator=g)[:50].cuda()
    want, _ = fk.kv_cache_read(kc, kc, slots, kv_dtype=fk.KV_E4M3, k_scale=one, v_scale=one)
    for off in (0, 8, 16, 24):
        buf = torch.zeros(2, 50 * 2 * 64 + 64, dtype=torch.bfloat16, device="cuda")
        k, v = (b[off:off + 50 * 2 * 64].view(50, 2, 64) for b in buf)
        fk.kv_cache_read(kc, kc, slots, kv_dtype=fk.KV_E4M3, k_scale=one, v_scale=one, k_out=k, v_out=v)
        assert torch.equal(k, want) and torch.equal(v, want)
        assert torch.all(buf[:, :off] == 0) and torch.all(buf[:, off + 50 * 2 * 64:] == 0)
    cb = torch.randn(3 * 16 * 192 + 32, generator=g).to(torch.bfloat16).cuda()
    cache = cb[8:8 + 3 * 16 * 192].view(3, 16, 192)        # a bf16 cache 16 bytes in
    at = torch.arange(48, device="cuda")
    assert torch.equal(fk.latent_cache_read(cache, at, kv_dtype=fk.KV_BF16), cache.flatten(0, 1))


def test_visible_nan_reaches_every_head_and_inf_too():
    # a key that IS seen spreads its NaN, as in the formula
    for kind in ("e4m3", "bf16"):
        st = Latent(kind, False, [50, 60], seed=6)
        q = torch.randn(2, st.H, st.L + 64, generator=st.g).to(torch.bfloat16).cuda()
        lens = torch.tensor(st.lens, dtype=torch.int32, device="cuda")
        blk, off = int(st.bt[0, 1]), 5
        st.cache[blk, off, 7] = 0x7F if kind == "e4m3" else float("nan")
        out = fk.latent_decode_attn(q, st.cache, st.bt.cuda(), lens, latent_dim=st.L,
                                    softmax_scale=0.07, **st.kw)
        assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()


def test_calls_with_nothing_to_do():
    dev = "cuda"
    e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device=dev)
    none = e(0, dt=torch.int64)
    kc = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device=dev)
    q = fk.rope_kv_cache_write(e(0, 4, 64), e(0, 2, 64), e(0, 2, 64), none, none,
                               table(thetas(64)).to(dev), kc, kc.clone(), kv_dtype=fk.KV_BF16)
    assert q.shape == (0, 4, 64)
    k, v = fk.kv_cache_read(kc, kc, none, kv_dtype=fk.KV_BF16)
    assert k.shape == v.shape == (0, 2, 64)
    lc = torch.zeros(2, 16, 192, dtype=torch.bfloat16, device=dev)
    assert fk.latent_cache_write(e(0, 128), e(0, 64), none, lc, kv_dtype=fk.KV_BF16) is None
    assert fk.latent_cache_read(lc, none, kv_dtype=fk.KV_BF16).shape == (0, 192)
    out = fk.latent_decode_attn(e(0, 1, 16, 192), lc, torch.zeros(0, 1, dtype=torch.int32, device=dev),
                                torch.zeros(0, dtype=torch.int32, device=dev), latent_dim=128,
                                kv_dtype=fk.KV_BF16, softmax_scale=0.1)
    assert out.shape == (0, 1, 16, 128)
