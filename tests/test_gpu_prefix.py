"""Decode attention behind a shared prefix on the GPU, against a plain 64-bit implementation
(tests/_sparse.py says how the bounds on results are derived)."""
import pytest
import torch

import fp8_kv_cache_write_gb300 as fk
from _latent import assert_close
from _sparse import Cache, attend, rounded

pytestmark = pytest.mark.gpu

DEV = "cuda"
KINDS = ["token", "tensor", "head", "bf16"]


class Batch:
    """A prefix (the cache's first sequence) and the tails behind it, with queries."""

    def __init__(self, seed, prefix, tails, Hkv, G, D, kind, **kw):
        self.c = c = Cache(seed, [prefix] + list(tails), Hkv, D, kind, **kw)
        self.B, self.G, self.D = len(tails), G, D
        self.npp = max(1, -(-prefix // 16))
        self.mbs = max(1, max(-(-n // 16) for n in tails))
        self.q = torch.randn(self.B, Hkv * G, D, generator=torch.Generator().manual_seed(seed + 1)).to(torch.bfloat16)
        self.dq = self.q.to(DEV)
        self.prefix_table = c.dtable[0, :self.npp].contiguous()
        self.prefix_len = torch.tensor([prefix], dtype=torch.int32, device=DEV)
        self.table = c.dtable[1:, :self.mbs].contiguous()
        self.lens = c.dlens[1:].contiguous()
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(self, **kw):
        return fk.prefix_decode_attn(self.dq, self.c.k, self.c.v, self.prefix_table, self.prefix_len,
                                     self.table, self.lens, err_flag=self.err,
                                     **{**self.c.args(fk), **kw})

    def expect(self, out_bf16=False, prefix_pages=None, tail_pages=None):
        c = self.c
        want, bound = torch.zeros(self.q.shape).double(), torch.zeros(self.q.shape).double()
        # a weight of the prefix's part: one f16 term (e4m3), two bf16 terms; f16's smallest
        # step, 2^-24 under a lift of 2^7 and of weights up to 2^8 under their largest, is
        # below the 2^-30 of the largest value that is added.  e4m3: the query's second term
        # is a multiple of 2^-9 where its largest value is at least 2^7, so a value is off by
        # 2^-17 of the largest, and a logit by that times the key's sum of magnitudes; twice,
        # for the weight and for the sum it is divided by
        for h in range(c.Hkv):
            pp = range(-(-c.lens[0] // 16)) if prefix_pages is None else prefix_pages
            pk, pv = c.rows("k", 0, h, pp), c.rows("v", 0, h, pp)
            for b in range(self.B):
                tp = range(-(-c.lens[b + 1] // 16)) if tail_pages is None else tail_pages[b]
                k = torch.cat((pk, c.rows("k", b + 1, h, tp)))
                v = torch.cat((pv, c.rows("v", b + 1, h, tp)))
                for g in range(h * self.G, (h + 1) * self.G):
                    weight = 2.0 ** -16
                    if c.e4m3 and len(pk):
                        weight = 2.0 ** -12 + 2.0 ** -16 * float(
                            self.q[b, g].abs().max() * pk.abs().sum(1).max()) * self.D ** -0.5
                    want[b, g], bound[b, g] = attend(self.q[b, g].double(), k, v, self.D ** -0.5, weight)
                    if len(v):
                        bound[b, g] += len(v) * 2.0 ** -30 * float(v.abs().max())
        return want, rounded(bound, want, out_bf16)

    def check(self, what, **kw):
        want, bound = self.expect()
        assert_close(self.run(**kw).cpu(), want, bound, what)
        assert int(self.err) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefix_lengths(D, kind):
    """Prefixes that end inside a page and inside a tile, none at all; empty tails."""
    for prefix in (0, 1, 16, 63, 64, 65, 127, 128, 129, 300):
        b = Batch(prefix, prefix, [0, 1, 40, 16, 17], 2, 3, D, kind)
        b.check(f"prefix {prefix}")


@pytest.mark.parametrize("G,B", [(1, 1), (1, 130), (3, 50), (8, 16), (8, 17), (16, 9), (12, 3)])
@pytest.mark.parametrize("kind", ["token", "bf16"])
def test_rows(G, B, kind):
    """One row to several row tiles, groups that do not divide a tile."""
    tails = [(7 * i) % 37 for i in range(B)]
    Batch(1000 + G, 333, tails, 2, G, 64, kind).check("rows")


@pytest.mark.parametrize("kind", ["token", "tensor", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_prefix_many_pieces(D, kind):
    """One head's prefix dealt to every SM, many tiles a CTA."""
    Batch(2000, 30001, [5, 100], 1, 4, D, kind).check("long prefix")


@pytest.mark.parametrize("kind", ["token", "bf16"])
@pytest.mark.parametrize("D", [64, 256])
def test_shares_across_row_tiles(D, kind):
    """More row tiles than SMs: a CTA goes from one row tile to the next."""
    tails = [i % 5 for i in range(48)]
    Batch(3000, 500, tails, 40, 16, D, kind).check("shares")     # 240 row tiles


def test_output_types_and_workspaces():
    b = Batch(4000, 1000, [9, 33, 0], 2, 4, 128, "token")
    want, bound = b.expect(out_bf16=True)
    out = torch.full((3, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    assert b.run(out=out, out_dtype=fk.OUT_BF16) is out
    assert_close(out.cpu(), want, bound, "bf16")
    _, need = fk.prefix_attn_plan(3, 8, 2, 128, b.npp)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device=DEV)     # NaN partials
    first = b.run(workspace=ws)
    assert bool((ws[need:] == 0xFF).all())
    again = b.run(workspace=ws)
    assert torch.equal(first, again)                          # the same split, the same sums
    assert torch.equal(first, b.run(workspace=ws[:100]))      # too small: one of the call's own


def test_bad_blocks_and_lengths_past_the_table():
    b = Batch(5000, 200, [40, 70], 2, 2, 128, "tensor")
    b.prefix_table[3], b.prefix_table[10] = -1, b.c.nb
    b.table[0, 1] = 1 << 30
    want, bound = b.expect(prefix_pages=[p for p in range(13) if p not in (3, 10)],
                           tail_pages=[[0, 2], [0, 1, 2, 3, 4]])
    assert_close(b.run().cpu(), want, bound, "bad blocks")
    assert int(b.err) == -6
    b = Batch(5100, 208, [48, 80], 1, 2, 64, "token")          # whole pages
    b.prefix_len += 1000
    b.lens += 1000
    want, bound = b.expect(tail_pages=[[0, 1, 2], [0, 1, 2, 3, 4]])
    b.lens[0] = 48
    assert_close(b.run().cpu(), want, bound, "past the end")
    assert int(b.err) == -6
    b = Batch(5200, 100, [20], 1, 2, 64, "token")
    b.prefix_len -= 200                                        # negative: none
    want, bound = b.expect(prefix_pages=[])
    assert_close(b.run().cpu(), want, bound, "negative length")


def test_every_block_bad():
    b = Batch(5300, 100, [20, 3], 1, 2, 64, "token")
    b.prefix_table[:] = -1
    want, bound = b.expect(prefix_pages=[])
    assert_close(b.run().cpu(), want, bound, "no prefix page")
    assert int(b.err) == -6


@pytest.mark.parametrize("low,high", [(-100, -60), (-20, 10), (-120, 20), (30, 60)])
def test_value_scales_of_any_size(low, high):
    b = Batch(6000, 700, [200, 33], 1, 4, 64, "token")
    c = b.c
    g = torch.Generator().manual_seed(61)
    s = torch.exp2(torch.randint(low, high + 1, (c.nb, 1, 16), generator=g).float())
    s[torch.rand(s.shape, generator=g) < 0.2] = 0.0
    c.kw["v_scale_cache"] = s.to(DEV)
    codes = (torch.randn(c.nb, 1, 16, 64, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    c.v, c.val["v"] = codes.view(torch.uint8).to(DEV), codes.double() * s[..., None].double()
    want, bound = b.expect()
    # a weight's smallest step, 2^-25 under a lift of 2^7, against the largest weight, which
    # is at least 1; values up to 448 / 1 of the largest weight's scale
    bound += 900 * 2.0 ** -22 * float(want.abs().max())
    assert_close(b.run().cpu(), want, bound, "value scales")


def test_strong_and_far_logits():
    """References that move with every tile, up and down."""
    b = Batch(7000, 3000, [50, 0], 1, 8, 128, "bf16", amplitude=30.0)
    b.q *= 8
    b.dq = b.q.to(DEV)
    b.check("far logits")


def test_not_a_number_stays_in_its_row():
    """A query with a NaN makes its own rows NaN; infinite keys those that see them."""
    b = Batch(8000, 400, [30, 30, 30], 2, 4, 64, "bf16")
    want, bound = b.expect()
    b.dq[1, 2, 5] = float("nan")
    out = b.run().cpu()
    assert bool(torch.isnan(out[1, 2]).all())
    ok = torch.ones(3, 8, dtype=torch.bool)
    ok[1, 2] = False
    assert_close(out[ok], want[ok], bound[ok], "other rows")


def test_the_same_as_one_table():
    """Whole pages of prefix and tail in one table: the decode attention's result."""
    b = Batch(9000, 160, [64, 33], 2, 4, 128, "token")
    table = torch.cat((b.prefix_table.expand(2, -1), b.table), dim=1).contiguous()
    whole = fk.paged_decode_attn(b.dq, b.c.k, b.c.v, table, b.lens + 160, **b.c.args(fk))
    _, bound = b.expect()
    assert_close(b.run().cpu(), whole.cpu().double(), 2 * bound, "one table")


def test_graphs_streams_and_shared_workspaces():
    """Captured and replayed with other queries, lengths and tails; two graphs on two streams
    with workspaces of their own; the same workspace for calls one after another."""
    a, b = Batch(10000, 900, [40, 17, 3], 2, 4, 128, "token"), Batch(10100, 2500, [0, 200], 1, 8, 64, "bf16")
    ws = [torch.empty(8 << 20, dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs, graphs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for x, w, s in zip((a, b), ws, streams):
        x.run(workspace=w)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            first = x.run(workspace=w)
            second = x.run(workspace=w)                 # behind it, in the same workspace
        outs.append((first, second))
        graphs.append(graph)
    for i in range(3):
        a.prefix_len.fill_(900 - 100 * i)
        a.c.lens[0] = 900 - 100 * i
        b.q = torch.randn(b.q.shape, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16)
        b.dq.copy_(b.q.to(DEV))
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for x, (first, second) in zip((a, b), outs):
            want, bound = x.expect()
            assert_close(first.cpu(), want, bound, f"replay {i}")
            assert torch.equal(first, second)
    side = torch.cuda.Stream()
    out = a.run(stream=side)
    side.synchronize()
    want, bound = a.expect()
    assert_close(out.cpu(), want, bound, "stream argument")


def test_rows_over_4_gib():
    D, Hkv, nb = 256, 8, 1 << 18                        # 8 GiB of keys
    b = Batch(11000, 70, [20], Hkv, 1, D, "tensor")
    c = b.c
    kc = torch.zeros(nb, Hkv, 16, D, dtype=torch.uint8, device=DEV)
    vc = torch.zeros(nb, Hkv, 16, D, dtype=torch.uint8, device=DEV)
    shift = nb - c.nb
    kc[shift:], vc[shift:] = c.k, c.v
    want, bound = b.expect()
    out = fk.prefix_decode_attn(b.dq, kc, vc, b.prefix_table + shift, b.prefix_len, b.table + shift,
                                b.lens, **c.args(fk))
    assert_close(out.cpu(), want, bound, "far blocks")


def test_refusals_on_the_device():
    b = Batch(12000, 40, [8, 8], 2, 2, 64, "token")
    kw = b.c.args(fk)
    call = lambda **k: fk.prefix_decode_attn(
        k.get("q", b.dq), b.c.k, k.get("v", b.c.v), k.get("pt", b.prefix_table), k.get("pl", b.prefix_len),
        k.get("bt", b.table), k.get("lens", b.lens), **{**kw, **k.get("kw", {})})
    for kind, what, args in (
            (TypeError, "q", dict(q=b.dq.float())), (ValueError, "prefix_table", dict(pt=b.prefix_table.cpu())),
            (TypeError, "prefix_len", dict(pl=b.prefix_len.long())),
            (ValueError, "prefix_len", dict(pl=b.lens)), (ValueError, "context_lens", dict(lens=b.prefix_len)),
            (ValueError, "v_cache", dict(v=b.c.v[1:])), (ValueError, "out", dict(kw=dict(out=torch.zeros(2, 4, 32, device=DEV)))),
            (fk.Fp8kvError, "INVALID", dict(kw=dict(softmax_scale=-1.0))),
            (fk.Fp8kvError, "INVALID", dict(pt=b.prefix_table[:0])),
            (ValueError, "v_scale_cache", dict(kw=dict(v_scale_cache=None)))):
        with pytest.raises(kind, match=what):
            call(**args)
