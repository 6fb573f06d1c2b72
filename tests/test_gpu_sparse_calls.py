"""Uses of the calls that read part of a cache which the tests beside this one do not make:
tables past a CTA's shared memory, workspaces and streams of the caller's, misaligned scales,
empty batches, lists of very different lengths, the same call over and over."""
import pytest
import torch

import fp8_kv_cache_write_gb300 as fk
from _latent import assert_close
from _sparse import Cache, attend, rounded, select
from test_gpu_prefix import Batch

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _random_bounds(g, nb, Hkv, D):
    return (torch.randint(-127, 128, (nb, Hkv, 2, D), generator=g).to(torch.int8),
            torch.rand(nb, Hkv, generator=g) * 0.01 + 0.001)


@pytest.mark.parametrize("mbs", [50000, 50001, 70000])
def test_selection_over_a_million_tokens(mbs):
    """Keys that just fit a CTA's shared memory, and more, which are read again; a NaN-filled
    workspace of the caller's, whose end stays as it was; one that is too small."""
    g = torch.Generator().manual_seed(mbs)
    nb, D = 900, 64                                    # sequences share blocks: scores repeat
    table = torch.randint(0, nb, (2, mbs), generator=g).to(torch.int32)
    lens = [16 * mbs, 16 * 50000 - 3]
    q = torch.randn(2, 2, D, generator=g).to(torch.bfloat16)
    bounds, scale = _random_bounds(g, nb, 1, D)
    args = (q.to(DEV), bounds.to(DEV), scale.to(DEV), table.to(DEV),
            torch.tensor(lens, dtype=torch.int32, device=DEV))
    need = fk.kv_page_select_workspace_bytes(2, 1, mbs)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
    got = [fk.kv_page_select(*args, budget=700, sink=2, recent=5, workspace=w)
           for w in (ws, None, ws[:100])]
    assert bool((ws[need:] == 0xFF).all())
    for b, ctx in enumerate(lens):
        n = -(-ctx // 16)
        t = table[b, :n].long()
        want = select(q[b], bounds[t, 0], scale[t, 0], n, 700, 2, 5)
        for pages, counts in got:
            assert pages[b, 0].tolist() == want and int(counts[b, 0]) == 700


def test_a_run_on_another_stream():
    """Bounds, selection and attention with `stream`, outputs of the calls' own: the same as on
    the current one."""
    c = Cache(200, [700, 90, 0, 331], 2, 128, "token")
    q = torch.randn(4, 8, 128, generator=torch.Generator().manual_seed(201)).to(torch.bfloat16).to(DEV)

    def run(**kw):
        bounds = torch.zeros(c.nb, 2, 2, 128, dtype=torch.int8, device=DEV)
        scale = torch.zeros(c.nb, 2, device=DEV)
        if "stream" in kw:
            kw["stream"].wait_stream(torch.cuda.current_stream())
        fk.kv_page_bounds(c.k, c.dtable, c.dlens, bounds, scale, **c.args(fk, "k"), **kw)
        pages, counts = fk.kv_page_select(q, bounds, scale, c.dtable, c.dlens, budget=9, **kw)
        out = fk.sparse_decode_attn(q, c.k, c.v, c.dtable, c.dlens, pages, counts, **c.args(fk), **kw)
        torch.cuda.synchronize()
        return bounds, scale, pages, counts, out

    for a, b in zip(run(), run(stream=torch.cuda.Stream())):
        assert torch.equal(a, b)


def test_two_graphs_at_once():
    """Two captured runs of selection and attention, replayed on two streams at once, with
    nothing shared but their inputs."""
    c = Cache(210, [16 * 300, 16 * 250 + 7], 2, 64, "bf16")
    g = torch.Generator().manual_seed(211)
    q = [torch.randn(2, 6, 64, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2)]
    bounds = torch.zeros(c.nb, 2, 2, 64, dtype=torch.int8, device=DEV)
    scale = torch.zeros(c.nb, 2, device=DEV)
    fk.kv_page_bounds(c.k, c.dtable, c.dlens, bounds, scale, **c.args(fk, "k"))

    def run(x):
        pages, counts = fk.kv_page_select(x, bounds, scale, c.dtable, c.dlens, budget=40, recent=3)
        return pages, fk.sparse_decode_attn(x, c.k, c.v, c.dtable, c.dlens, pages, counts, **c.args(fk))

    want = [run(x) for x in q]
    torch.cuda.synchronize()
    streams, graphs, got = [torch.cuda.Stream(), torch.cuda.Stream()], [], []
    for x, s in zip(q, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got.append(run(x))
        graphs.append(graph)
    for _ in range(5):
        for pages, out in got:
            pages.fill_(-7)
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_scales_and_workspaces_off_their_borders():
    """Views that start inside a 16-byte (32-byte) piece are refused before any launch."""
    c = Cache(220, [40, 40], 2, 64, "token")
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    bounds = torch.zeros(c.nb, 2, 2, 64, dtype=torch.int8, device=DEV)
    scale = torch.zeros(c.nb, 2, device=DEV)
    pages = torch.zeros(2, 2, 2, dtype=torch.int32, device=DEV)

    def off(t):
        x = torch.zeros(t.numel() + 1, device=DEV)[1:].view(t.shape)
        return x.copy_(t)

    for name in ("k_scale_cache", "v_scale_cache"):
        kw = {**c.args(fk), name: off(c.kw[name])}
        with pytest.raises(fk.Fp8kvError, match="INVALID"):
            fk.sparse_decode_attn(q, c.k, c.v, c.dtable, c.dlens, pages, **kw)
        with pytest.raises(fk.Fp8kvError, match="INVALID"):
            fk.prefix_decode_attn(q, c.k, c.v, c.dtable[0], c.dlens[:1], c.dtable, c.dlens, **kw)
    with pytest.raises(fk.Fp8kvError, match="INVALID"):
        fk.kv_page_bounds(c.k, c.dtable, c.dlens, bounds, scale,
                          **{**c.args(fk, "k"), "k_scale_cache": off(c.kw["k_scale_cache"])})
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)[16:]
    with pytest.raises(fk.Fp8kvError, match="INVALID"):
        fk.prefix_decode_attn(q, c.k, c.v, c.dtable[0], c.dlens[:1], c.dtable, c.dlens, workspace=ws,
                              **c.args(fk))


def test_counts_past_32_bits():
    """Whole numbers that would wrap on their way into the library."""
    c = Cache(225, [40, 33], 2, 64, "tensor")
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    bounds = [torch.zeros(c.nb, 2, 2, 64, dtype=torch.int8, device=DEV) for _ in range(2)]
    scale = torch.zeros(c.nb, 2, device=DEV)
    for b, new in zip(bounds, (None, (1 << 32) + 1)):
        fk.kv_page_bounds(c.k, c.dtable, c.dlens, b, scale, new_tokens=new, **c.args(fk, "k"))
    assert torch.equal(*bounds)
    for bad in (dict(budget=3, sink=1 << 32), dict(budget=3, recent=1 << 32),
                dict(budget=3, sink=-(1 << 32)), dict(budget=(1 << 32) + 3)):
        with pytest.raises(fk.Fp8kvError, match="INVALID"):
            fk.kv_page_select(q, bounds[0], scale, c.dtable, c.dlens, **bad)


def test_empty_batches():
    c = Cache(230, [40], 2, 64, "head")
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    bounds = torch.zeros(c.nb, 2, 2, 64, dtype=torch.int8, device=DEV)
    scale = torch.zeros(c.nb, 2, device=DEV)
    fk.kv_page_bounds(c.k, c.dtable[:0], c.dlens[:0], bounds, scale, **c.args(fk, "k"))
    pages, counts = fk.kv_page_select(q, bounds, scale, c.dtable[:0], c.dlens[:0], budget=3)
    assert pages.shape == (0, 2, 3) and counts.shape == (0, 2)
    assert fk.sparse_decode_attn(q, c.k, c.v, c.dtable[:0], c.dlens[:0], pages, counts,
                                 **c.args(fk)).shape == (0, 4, 64)
    assert fk.prefix_decode_attn(q, c.k, c.v, c.dtable[0], c.dlens[:1], c.dtable[:0], c.dlens[:0],
                                 **c.args(fk)).shape == (0, 4, 64)
    assert not bool(bounds.any()) and not bool(scale.any())


def test_budgets_past_the_table_and_uneven_lists():
    """A budget of more pages than any sequence has: all of them; then lists of one page, of
    none and of hundreds in one call."""
    c = Cache(240, [16 * 200, 50, 1, 0], 2, 128, "token")
    q = torch.randn(4, 6, 128, generator=torch.Generator().manual_seed(241)).to(torch.bfloat16)
    bounds = torch.zeros(c.nb, 2, 2, 128, dtype=torch.int8, device=DEV)
    scale = torch.zeros(c.nb, 2, device=DEV)
    fk.kv_page_bounds(c.k, c.dtable, c.dlens, bounds, scale, **c.args(fk, "k"))
    pages, counts = fk.kv_page_select(q.to(DEV), bounds, scale, c.dtable, c.dlens, budget=1000)
    for b, n in enumerate(c.lens):
        m = -(-n // 16)
        assert counts[b].tolist() == [m, m]
        for h in range(2):
            assert pages[b, h].tolist() == list(range(m)) + [-1] * (1000 - m)
    counts[0, 1], counts[1, 0] = 1, 0
    out = fk.sparse_decode_attn(q.to(DEV), c.k, c.v, c.dtable, c.dlens, pages, counts, **c.args(fk))
    want, bound = torch.zeros(q.shape).double(), torch.zeros(q.shape).double()
    for b in range(4):
        for h in range(2):
            rows = range(int(counts[b, h]))
            k, v = c.rows("k", b, h, rows), c.rows("v", b, h, rows)
            for g in range(3 * h, 3 * h + 3):
                want[b, g], bound[b, g] = attend(q[b, g].double(), k, v, 128 ** -0.5)
    assert_close(out.cpu(), want, rounded(bound, want, False), "uneven lists")
    assert not bool(out[1, :3].any()) and not bool(out[3].any())


@pytest.mark.parametrize("kind", ["token", "tensor", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_same_prefix_call_again(D, kind):
    """References that move all the time (keys that grow along the prefix), row tiles that
    leave warps idle, shares that cross them: twenty calls leave the same bits, the right ones."""
    b = Batch(12000 + D, 1500, [i % 40 for i in range(37)], 16, 5, D, kind)   # 2 row tiles a head
    grow = torch.ones(b.c.nb, 1, 1, 1)
    for p in range(b.npp):
        grow[int(b.c.table[0, p])] = 2.0 ** (p // 12)
    if kind == "bf16":
        b.c.val["k"] = b.c.val["k"] * grow.double() / 64
        b.c.k = b.c.val["k"].to(torch.bfloat16).to(DEV)
    elif kind == "token":
        s = b.c.kw["k_scale_cache"].cpu() * grow[..., 0] / 64
        b.c.val["k"] = b.c.val["k"] * grow.double() / 64
        b.c.kw["k_scale_cache"] = s.to(DEV)
    first = b.run()
    want, bound = b.expect()
    assert_close(first.cpu(), want, bound, "first")
    for _ in range(20):
        assert torch.equal(b.run(), first)
    assert int(b.err) == 0
