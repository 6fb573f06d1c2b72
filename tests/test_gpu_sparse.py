"""Page bounds, page selection and sparse decode attention on the GPU, against plain 64-bit
implementations (tests/_sparse.py says how the bounds on results are derived)."""
import pytest
import torch

import fp8_kv_cache_write_gb300 as fk
from _latent import assert_close
from _sparse import Cache, attend, bounds_of, rounded, select

pytestmark = pytest.mark.gpu

DEV = "cuda"
KINDS = ["token", "tensor", "head", "bf16"]


def _err():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _bounds(c, new_tokens=None, **kw):
    bounds = torch.full((c.nb, c.Hkv, 2, c.D), 77, dtype=torch.int8, device=DEV)
    scale = torch.full((c.nb, c.Hkv), -1.0, device=DEV)
    fk.kv_page_bounds(c.k, c.dtable, c.dlens, bounds, scale, new_tokens=new_tokens,
                      **c.args(fk, "k"), **kw)
    return bounds, scale


def _check_bounds(c, bounds, scale, new_tokens=None):
    want_b = torch.full((c.nb, c.Hkv, 2, c.D), 77, dtype=torch.int8)
    want_s = torch.full((c.nb, c.Hkv), -1.0)
    for b, n in enumerate(c.lens):
        first = max(0, n - new_tokens) // 16 if new_tokens else 0
        for p in range(first, -(-n // 16)):
            for h in range(c.Hkv):
                blk = int(c.table[b, p])
                # the products code * scale of the cache, in fp32 as the definition has them
                hi, lo, s = bounds_of(c.rows("k", b, h, [p]).float())
                want_b[blk, h, 0], want_b[blk, h, 1], want_s[blk, h] = hi, lo, s
    assert torch.equal(scale.cpu(), want_s)
    assert torch.equal(bounds.cpu(), want_b)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_bounds_of_all_pages(D, kind):
    c = Cache(1, [0, 1, 15, 16, 17, 130], 3, D, kind)
    err = _err()
    bounds, scale = _bounds(c, err_flag=err)
    _check_bounds(c, bounds, scale)
    assert int(err) == 0


@pytest.mark.parametrize("new", [1, 2, 15, 16, 17, 18, 33, 1000])
def test_bounds_of_the_pages_of_new_tokens(new):
    c = Cache(2, [0, 1, 15, 16, 17, 31, 32, 33, 64, 90], 2, 64, "token")
    _check_bounds(c, *_bounds(c, new), new)


def test_bounds_of_odd_values():
    """Zeros, NaN and infinities, subnormals, the largest numbers."""
    c = Cache(3, [16, 16, 16, 16, 16, 5], 1, 64, "bf16", extra=0)
    vals = torch.randn(c.nb, 1, 16, 64).to(torch.bfloat16)
    t = c.table[:, 0].long()
    vals[t[0]] = 0
    vals[t[1], 0, 3, 5] = float("nan")
    vals[t[1], 0, :, 7] = float("nan")
    vals[t[2], 0, 2, 0], vals[t[2], 0, 9, 1] = float("inf"), float("-inf")
    vals[t[3]] = (torch.randn(1, 16, 64) * 1e-38).to(torch.bfloat16)
    vals[t[4]] = (torch.randn(1, 16, 64).sign() * 3.38e38).to(torch.bfloat16)
    vals[t[5], 0, 5:] = float("nan")                                # behind the sequence
    c.k = vals.to(DEV)
    bounds, scale = _bounds(c)
    big = torch.finfo(torch.float32).max
    for b, n in enumerate(c.lens):
        x = vals[t[b], 0, :n].float()
        hi = torch.nan_to_num(x, nan=-float("inf"), posinf=float("inf")).amax(0)
        lo = torch.nan_to_num(x, nan=float("inf"), neginf=-float("inf")).amin(0)
        empty = torch.isnan(x).all(0)
        hi, lo = hi.masked_fill(empty, 0).clamp(-big, big), lo.masked_fill(empty, 0).clamp(-big, big)
        s = torch.maximum(hi.abs(), lo.abs()).max() / torch.tensor(127.0)
        assert float(scale[t[b], 0]) == float(s)
        for i, w in enumerate((hi, lo)):
            code = torch.zeros(64) if float(s) == 0 else torch.round(w / s).clamp(-127, 127)
            assert torch.equal(bounds[t[b], 0, i].cpu(), code.to(torch.int8)), (b, i)


def test_bounds_of_bad_blocks_and_lengths_past_the_table():
    c = Cache(4, [40, 33], 2, 128, "tensor")
    good = _bounds(c)
    c.dtable[0, 1], c.dtable[1, 0] = c.nb, -1
    c.dlens[1] = 1000
    err = _err()
    bounds, scale = _bounds(c, err_flag=err)
    assert int(err) == -6
    for b, p in ((0, 0), (0, 2), (1, 1)):
        blk = int(c.table[b, p])
        assert torch.equal(bounds[blk], good[0][blk])
    for b, p in ((0, 1), (1, 0)):
        assert bool((bounds[int(c.table[b, p])] == 77).all())


# ---------------------------------------------------------------- selection
def _random_bounds(seed, nb, Hkv, D):
    g = torch.Generator().manual_seed(seed)
    return (torch.randint(-127, 128, (nb, Hkv, 2, D), generator=g).to(torch.int8),
            torch.rand(nb, Hkv, generator=g) * 0.01 + 0.001)


def _check_select(q, bounds, scale, table, lens, budget, sink, recent, **kw):
    err = _err()
    pages, counts = fk.kv_page_select(
        q.to(DEV), bounds.to(DEV), scale.to(DEV), table.to(DEV),
        torch.tensor(lens, dtype=torch.int32, device=DEV), budget=budget, sink=sink, recent=recent,
        err_flag=err, **kw)
    pages, counts = pages.cpu(), counts.cpu()
    Hkv = scale.shape[1]
    G = q.shape[1] // Hkv
    for b, ctx in enumerate(lens):
        n = -(-ctx // 16)
        t = table[b, :n].long()
        for h in range(Hkv):
            want = select(q[b, h * G:(h + 1) * G], bounds[t, h], scale[t, h], n, budget, sink, recent)
            assert int(counts[b, h]) == len(want) == min(n, budget)
            assert pages[b, h].tolist() == want + [-1] * (budget - len(want)), (b, h)
    assert int(err) == 0


@pytest.mark.parametrize("D,G", [(64, 1), (128, 3), (128, 8), (256, 16)])
def test_selection(D, G):
    lens = [0, 1, 16, 17, 160, 161, 1000, 5000]
    Hkv, mbs = 2, 313
    nb = len(lens) * mbs + 3
    g = torch.Generator().manual_seed(5)
    table = torch.randperm(nb, generator=g)[:len(lens) * mbs].view(len(lens), mbs).to(torch.int32)
    q = torch.randn(len(lens), Hkv * G, D, generator=g).to(torch.bfloat16)
    bounds, scale = _random_bounds(6, nb, Hkv, D)
    for budget, sink, recent in ((10, 1, 1), (10, 0, 0), (10, 4, 6), (1, 0, 1), (37, 3, 0),
                                 (312, 1, 2), (400, 1, 1)):
        _check_select(q, bounds, scale, table, lens, budget, sink, recent)


@pytest.mark.parametrize("mbs,B", [(8200, 1), (40000, 1), (700, 70)])
def test_selection_over_cluster_sizes(mbs, B):
    """Many pages of one sequence (many CTAs score them, one takes them), many sequences."""
    g = torch.Generator().manual_seed(7)
    nb = 4000                                      # sequences share blocks: scores repeat
    table = torch.randint(0, nb, (B, mbs), generator=g).to(torch.int32)
    lens = torch.randint(16 * (mbs - 40), 16 * mbs + 1, (B,), generator=g).tolist()
    q = torch.randn(B, 4, 64, generator=g).to(torch.bfloat16)
    bounds, scale = _random_bounds(8, nb, 2, 64)
    _check_select(q, bounds, scale, table, lens, 100, 1, 4)


def test_selection_with_ties():
    """Equal scores everywhere, a few values only, zeros of both signs: the lower pages win."""
    mbs, D = 500, 64
    table = torch.arange(2 * mbs).view(2, mbs).to(torch.int32)
    g = torch.Generator().manual_seed(9)
    q = torch.randn(2, 2, D, generator=g).to(torch.bfloat16)
    lens = [16 * mbs, 16 * mbs - 5]
    few = torch.randint(-2, 3, (2 * mbs, 1, 2, 1), generator=g).expand(-1, -1, -1, D)
    for bounds in (torch.ones(2 * mbs, 1, 2, D), few, torch.zeros(2 * mbs, 1, 2, D)):
        for scale in (torch.ones(2 * mbs, 1), (torch.arange(2 * mbs) % 3).float().view(-1, 1)):
            _check_select(q, bounds.to(torch.int8).contiguous(), scale, table, lens, 60, 2, 3)
    # a query of zeros: every score is 0
    _check_select(torch.zeros_like(q), few.to(torch.int8).contiguous(), torch.ones(2 * mbs, 1), table,
                  lens, 60, 0, 1)


def test_selection_of_extreme_scores():
    """Scores of infinite and NaN scales, over the whole range of fp32."""
    mbs, D = 300, 128
    table = torch.arange(mbs).view(1, mbs).to(torch.int32)
    g = torch.Generator().manual_seed(10)
    q = torch.randn(1, 1, D, generator=g).to(torch.bfloat16)
    bounds, _ = _random_bounds(11, mbs, 1, D)
    scale = torch.exp2(torch.randint(-149, 128, (mbs, 1), generator=g).float())
    scale[::50] = float("inf")
    _check_select(q, bounds, scale, table, [16 * mbs], 40, 1, 1)
    scale[7], scale[200] = float("nan"), float("nan")
    pages, _ = fk.kv_page_select(q.to(DEV), bounds.to(DEV), scale.to(DEV), table.to(DEV),
                                 torch.tensor([16 * mbs], dtype=torch.int32, device=DEV), budget=4,
                                 sink=1, recent=1)
    assert pages[0, 0].tolist() == [0, 7, 200, mbs - 1]


def test_selection_of_bad_blocks_and_lengths():
    mbs, D = 100, 64
    table = torch.arange(mbs).view(1, mbs).to(torch.int32)
    g = torch.Generator().manual_seed(12)
    q = torch.randn(1, 2, D, generator=g).to(torch.bfloat16)
    bounds, scale = _random_bounds(13, mbs, 1, D)
    bad = table.clone()
    bad[0, 3::4] = torch.tensor([-1, mbs, 1 << 30])[torch.arange(25) % 3].to(torch.int32)
    good = [p for p in range(mbs) if p % 4 != 3]
    want = select(q[0], bounds[good, 0], scale[good, 0], len(good), 50, 1, 0)
    err = _err()
    pages, counts = fk.kv_page_select(q.to(DEV), bounds.to(DEV), scale.to(DEV), bad.to(DEV),
                                      torch.tensor([9999], dtype=torch.int32, device=DEV),
                                      budget=50, sink=1, recent=0, err_flag=err)
    assert int(err) == -6 and int(counts[0, 0]) == 50
    assert pages[0, 0].tolist() == [good[i] for i in want]


# ---------------------------------------------------------------- attention over a list
def _expect(c, q, lists, scale, out_bf16=False):
    B, Hq, D = q.shape
    G = Hq // c.Hkv
    want, bound = torch.zeros(B, Hq, D).double(), torch.zeros(B, Hq, D).double()
    for b in range(B):
        n = -(-c.lens[b] // 16)
        for h in range(c.Hkv):
            pages = [p for p in lists[b][h] if 0 <= p < n]
            k, v = c.rows("k", b, h, pages), c.rows("v", b, h, pages)
            for g in range(h * G, (h + 1) * G):
                want[b, g], bound[b, g] = attend(q[b, g].double().cpu(), k, v, scale)
    return want, rounded(bound, want, out_bf16)


def _lists(seed, c, budget):
    """Random page lists: of any order, with unused entries, some of them past the sequence."""
    g = torch.Generator().manual_seed(seed)
    B = len(c.lens)
    pages = torch.full((B, c.Hkv, budget), -1, dtype=torch.int32)
    counts = torch.zeros(B, c.Hkv, dtype=torch.int32)
    for b, n in enumerate(c.lens):
        for h in range(c.Hkv):
            order = torch.randperm(-(-n // 16), generator=g)[:budget]
            pages[b, h, :len(order)] = order
            counts[b, h] = len(order)
    return pages, counts


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 3, 8, 16])
def test_sparse_attention(D, kind, G):
    lens = [0, 1, 15, 16, 17, 100, 530]
    c = Cache(20 + G, lens, 2, D, kind)
    q = torch.randn(len(lens), 2 * G, D, generator=torch.Generator().manual_seed(21)).to(torch.bfloat16)
    for budget, out_dtype in ((7, fk.OUT_F32), (40, fk.OUT_BF16)):
        pages, counts = _lists(22, c, budget)
        err = _err()
        out = fk.sparse_decode_attn(q.to(DEV), c.k, c.v, c.dtable, c.dlens, pages.to(DEV),
                                    counts.to(DEV), out_dtype=out_dtype, err_flag=err, **c.args(fk))
        lists = [[pages[b, h, :int(counts[b, h])].tolist() for h in range(2)] for b in range(len(lens))]
        want, bound = _expect(c, q, lists, D ** -0.5, out_dtype == fk.OUT_BF16)
        assert_close(out.cpu(), want, bound, f"budget {budget}")
        assert int(err) == 0


@pytest.mark.parametrize("kind", ["token", "bf16"])
def test_sparse_attention_over_long_lists(kind):
    """One sequence, clusters of several CTAs, more than 32 pages a warp."""
    c = Cache(30, [60000], 1, 64, kind)
    q = torch.randn(1, 5, 64, generator=torch.Generator().manual_seed(31)).to(torch.bfloat16)
    pages = torch.arange(c.mbs, dtype=torch.int32).view(1, 1, -1)
    out = fk.sparse_decode_attn(q.to(DEV), c.k, c.v, c.dtable, c.dlens, pages.to(DEV), **c.args(fk))
    want, bound = _expect(c, q, [[pages[0, 0].tolist()]], 0.125)
    assert_close(out.cpu(), want, bound, "all pages")


def test_entries_that_say_nothing():
    """Negative entries, pages past the sequence, counts of zero, past the list and negative."""
    c = Cache(40, [100, 37, 16, 50], 2, 128, "token")
    q = torch.randn(4, 4, 128, generator=torch.Generator().manual_seed(41)).to(torch.bfloat16)
    pages = torch.tensor([[[3, -1, 0, 2000000000], [-5, -1, -1, -1]], [[7, 3, 2, 1], [0, 1, 2, 3]],
                          [[0, 1, 2, 3], [3, 2, 1, 0]], [[0, 1, 1, 3], [2, 2, 2, 2]]], dtype=torch.int32)
    counts = torch.tensor([[4, 4], [4, 0], [1000, -3], [4, 3]], dtype=torch.int32)
    err = _err()
    out = fk.sparse_decode_attn(q.to(DEV), c.k, c.v, c.dtable, c.dlens, pages.to(DEV), counts.to(DEV),
                                err_flag=err, **c.args(fk))
    lists = [[pages[b, h, :max(0, min(4, int(counts[b, h])))].tolist() for h in range(2)] for b in range(4)]
    want, bound = _expect(c, q, lists, 128 ** -0.5)         # a page listed twice counts twice
    assert_close(out.cpu(), want, bound, "odd entries")
    assert int(err) == 0 and float(out[0, 2:].abs().max()) == 0 and float(out[1, 2:].abs().max()) == 0


def test_bad_blocks_are_skipped():
    c = Cache(50, [100, 100], 1, 64, "tensor")
    q = torch.randn(2, 2, 64, generator=torch.Generator().manual_seed(51)).to(torch.bfloat16)
    c.dtable[0, 2], c.dtable[1, 0] = c.nb, -7
    pages = torch.arange(7, dtype=torch.int32).expand(2, 1, 7).contiguous()
    err = _err()
    out = fk.sparse_decode_attn(q.to(DEV), c.k, c.v, c.dtable, c.dlens, pages.to(DEV), err_flag=err,
                                **c.args(fk))
    want, bound = _expect(c, q, [[[0, 1, 3, 4, 5, 6]], [[1, 2, 3, 4, 5, 6]]], 0.125)
    assert_close(out.cpu(), want, bound, "bad blocks")
    assert int(err) == -6


@pytest.mark.parametrize("low,high", [(-100, -60), (-20, 10), (-120, 20), (30, 60)])
def test_value_scales_of_any_size(low, high):
    """Per-token value scales over many binades, zero among them: the weights keep their bits
    beside each other, and rows of zeros count in the sum."""
    c = Cache(60, [200, 33], 1, 64, "token")
    g = torch.Generator().manual_seed(61)
    s = torch.exp2(torch.randint(low, high + 1, (c.nb, 1, 16), generator=g).float())
    s[torch.rand(s.shape, generator=g) < 0.2] = 0.0
    c.kw["v_scale_cache"] = s.to(DEV)
    codes = (torch.randn(c.nb, 1, 16, 64, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    c.v, c.val["v"] = codes.view(torch.uint8).to(DEV), codes.double() * s[..., None].double()
    q = torch.randn(2, 4, 64, generator=g).to(torch.bfloat16)
    pages = torch.arange(c.mbs, dtype=torch.int32).expand(2, 1, c.mbs).contiguous()
    out = fk.sparse_decode_attn(q.to(DEV), c.k, c.v, c.dtable, c.dlens, pages.to(DEV), **c.args(fk))
    want, bound = _expect(c, q, [[pages[0, 0].tolist()]] * 2, 0.125)
    # weights lie below 2^4 (of the reference) and hold 2^-25 / 16 absolutely: 2^-33 of the
    # largest |weight * value| for each key
    bound += 233 * 2.0 ** -29 * float(want.abs().max())
    assert_close(out.cpu(), want, bound, "value scales")


def test_strong_and_far_logits():
    """Keys whose logits lie hundreds apart, in every order; the largest values."""
    c = Cache(70, [400], 1, 128, "bf16", amplitude=30.0)
    q = (torch.randn(1, 8, 128, generator=torch.Generator().manual_seed(71)) * 8).to(torch.bfloat16)
    for pages in (list(range(25)), list(range(24, -1, -1))):
        t = torch.tensor(pages, dtype=torch.int32, device=DEV).view(1, 1, -1)
        out = fk.sparse_decode_attn(q.to(DEV), c.k, c.v, c.dtable, c.dlens, t, **c.args(fk))
        want, bound = _expect(c, q, [[pages]], 128 ** -0.5)
        assert_close(out.cpu(), want, bound, "far logits")


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("kind", ["token", "head", "bf16"])
def test_a_decode_loop(kind):
    """Prompt, then steps: write, bounds of the last page, selection, attention; captured into
    a graph and replayed with other tokens, on a stream of its own."""
    B, Hkv, G, D, start, steps, budget = 3, 2, 4, 128, 200, 20, 6
    lens = [start, 90, 16]
    c = Cache(80, [n + steps for n in lens], Hkv, D, kind)
    g = torch.Generator().manual_seed(81)
    k_new = torch.randn(steps, B, Hkv, D, generator=g).to(torch.bfloat16).to(DEV)
    v_new = torch.randn(steps, B, Hkv, D, generator=g).to(torch.bfloat16).to(DEV)
    q_new = torch.randn(steps, B, Hkv * G, D, generator=g).to(torch.bfloat16).to(DEV)
    cur = torch.tensor(lens, dtype=torch.int32, device=DEV)
    kin, vin, qin = k_new[0].clone(), v_new[0].clone(), q_new[0].clone()
    bounds = torch.zeros(c.nb, Hkv, 2, D, dtype=torch.int8, device=DEV)
    scale = torch.zeros(c.nb, Hkv, device=DEV)
    pages = torch.zeros(B, Hkv, budget, dtype=torch.int32, device=DEV)
    counts = torch.zeros(B, Hkv, dtype=torch.int32, device=DEV)
    out = torch.zeros(B, Hkv * G, D, device=DEV)
    slots = torch.zeros(B, dtype=torch.int64, device=DEV)
    rows = torch.arange(B, device=DEV)
    err = _err()
    kw, kkw = c.args(fk), c.args(fk, "k")
    fk.kv_page_bounds(c.k, c.dtable, cur, bounds, scale, err_flag=err, **kkw)

    def step():
        cur.add_(1)
        pos = (cur - 1).long()
        slots.copy_(c.dtable[rows, pos // 16].long() * 16 + pos % 16)
        fk.kv_cache_write(kin, vin, slots, c.k, c.v, err_flag=err, **kw)
        fk.kv_page_bounds(c.k, c.dtable, cur, bounds, scale, new_tokens=1, err_flag=err, **kkw)
        fk.kv_page_select(qin, bounds, scale, c.dtable, cur, budget=budget, recent=2, pages=pages,
                          counts=counts, err_flag=err)
        fk.sparse_decode_attn(qin, c.k, c.v, c.dtable, cur, pages, counts, out=out, err_flag=err, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i in range(3):
            for dst, src in ((kin, k_new), (vin, v_new), (qin, q_new)):
                dst.copy_(src[i])
            step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()                                         # recorded, not run
    for i in range(3, steps):
        for dst, src in ((kin, k_new), (vin, v_new), (qin, q_new)):
            dst.copy_(src[i])
        graph.replay()
        # what the step left, against the definitions over the cache as it is now
        slot = torch.arange(c.nb * 16, device=DEV)
        k, v = fk.kv_cache_read(c.k, c.v, slot, out_dtype=fk.OUT_F32, **kw)
        for n, t in (("k", k), ("v", v)):
            c.val[n] = t.cpu().double().view(c.nb, 16, Hkv, D).transpose(1, 2)
        c.lens = cur.tolist()
        assert c.lens == [n + i + 1 for n in lens]
        lists = []
        for b, n in enumerate(c.lens):
            np_ = -(-n // 16)
            t = c.table[b, :np_].long()
            lists.append([])
            for h in range(Hkv):
                for p in range(np_):
                    hi, lo, s = bounds_of(c.rows("k", b, h, [p]).float())
                    assert float(scale[t[p], h]) == float(s)
                    assert torch.equal(bounds[t[p], h].cpu(), torch.stack((hi, lo)))
                want = select(qin[b, h * G:(h + 1) * G].cpu(), bounds.cpu()[t, h], scale.cpu()[t, h],
                              np_, budget, 1, 2)
                assert pages[b, h, :int(counts[b, h])].tolist() == want
                lists[-1].append(want)
        want, bound = _expect(c, qin, lists, D ** -0.5)
        assert_close(out.cpu(), want, bound, f"step {i}")
    assert int(err) == 0


def test_all_pages_selected_is_the_whole_decode():
    """With a budget of every page the sparse attention is the decode attention: both are
    within the decode's stated 4e-3 of exact, here held to what each may be off by."""
    c = Cache(90, [777, 300], 2, 128, "token")
    q = torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(91)).to(torch.bfloat16).to(DEV)
    bounds, scale = _bounds(c)
    pages, counts = fk.kv_page_select(q, bounds, scale, c.dtable, c.dlens, budget=c.mbs)
    out = fk.sparse_decode_attn(q, c.k, c.v, c.dtable, c.dlens, pages, counts, **c.args(fk))
    whole = fk.paged_decode_attn(q, c.k, c.v, c.dtable, c.dlens, **c.args(fk))
    _, bound = _expect(c, q.cpu(), [[list(range(-(-n // 16)))] * 2 for n in c.lens], 128 ** -0.5)
    assert_close(out.cpu(), whole.cpu().double(), 2 * bound, "all pages")


def test_rows_over_4_gib():
    """Blocks whose bytes lie past 32-bit offsets, in the cache and in its bounds."""
    D, Hkv, nb = 256, 8, 1 << 18                        # 8 GiB of keys, 1 GiB of bounds
    far = nb - 1 - torch.arange(4)
    kc = torch.zeros(nb, Hkv, 16, D, dtype=torch.uint8, device=DEV)
    vc = torch.zeros(nb, Hkv, 16, D, dtype=torch.uint8, device=DEV)
    c = Cache(100, [50], Hkv, D, "tensor", extra=0)
    kc[far], vc[far] = c.k[c.table[0].long()], c.v[c.table[0].long()]
    table = far.view(1, 4).to(torch.int32).to(DEV)
    bounds = torch.zeros(nb, Hkv, 2, D, dtype=torch.int8, device=DEV)
    scale = torch.zeros(nb, Hkv, device=DEV)
    kw = c.args(fk)
    fk.kv_page_bounds(kc, table, c.dlens, bounds, scale, **c.args(fk, "k"))
    q = torch.randn(1, Hkv, D, generator=torch.Generator().manual_seed(101)).to(torch.bfloat16)
    pages, counts = fk.kv_page_select(q.to(DEV), bounds, scale, table, c.dlens, budget=3)
    out = fk.sparse_decode_attn(q.to(DEV), kc, vc, table, c.dlens, pages, counts, **kw)
    lists = [[]]
    for h in range(Hkv):
        ref = [bounds_of(c.rows("k", 0, h, [p]).float()) for p in range(4)]
        b = torch.stack([torch.stack(r[:2]) for r in ref])
        s = torch.stack([r[2] for r in ref])
        assert torch.equal(bounds[far, h].cpu(), b) and torch.equal(scale[far, h].cpu(), s)
        lists[0].append(select(q[0, h:h + 1], b, s, 4, 3, 1, 1))
        assert pages[0, h].tolist() == lists[0][h]
    want, bound = _expect(c, q, lists, D ** -0.5)
    assert_close(out.cpu(), want, bound, "far blocks")


def test_refusals_on_the_device():
    """Arguments of wrong types, shapes and places name themselves and launch nothing."""
    c = Cache(110, [40, 40], 2, 64, "token")
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    bounds, scale = _bounds(c)
    pages = torch.zeros(2, 2, 3, dtype=torch.int32, device=DEV)
    kw = c.args(fk)
    bad = [
        (TypeError, "bounds", lambda: fk.kv_page_bounds(c.k, c.dtable, c.dlens, bounds.float(), scale, **c.args(fk, "k"))),
        (ValueError, "bounds_scale", lambda: fk.kv_page_bounds(c.k, c.dtable, c.dlens, bounds, scale[1:], **c.args(fk, "k"))),
        (ValueError, "new_tokens", lambda: fk.kv_page_bounds(c.k, c.dtable, c.dlens, bounds, scale, new_tokens=0, **c.args(fk, "k"))),
        (ValueError, "k_scale_cache", lambda: fk.kv_page_bounds(c.k, c.dtable, c.dlens, bounds, scale, kv_dtype=fk.KV_E4M3, scale_mode=fk.SCALE_PER_TOKEN_HEAD)),
        (TypeError, "q", lambda: fk.kv_page_select(q.float(), bounds, scale, c.dtable, c.dlens, budget=3)),
        (ValueError, "context_lens", lambda: fk.kv_page_select(q, bounds, scale, c.dtable, c.dlens[:1], budget=3)),
        (ValueError, "pages", lambda: fk.kv_page_select(q, bounds, scale, c.dtable, c.dlens, budget=3, pages=pages[:, :, :2])),
        (fk.Fp8kvError, "INVALID", lambda: fk.kv_page_select(q, bounds, scale, c.dtable, c.dlens, budget=3, sink=2, recent=2)),
        (fk.Fp8kvError, "INVALID", lambda: fk.kv_page_select(q, bounds, scale, c.dtable, c.dlens, budget=0)),
        (ValueError, "block_table", lambda: fk.kv_page_select(q, bounds, scale, c.dtable.cpu(), c.dlens, budget=3)),
        (TypeError, "pages", lambda: fk.sparse_decode_attn(q, c.k, c.v, c.dtable, c.dlens, pages.long(), **kw)),
        (ValueError, "counts", lambda: fk.sparse_decode_attn(q, c.k, c.v, c.dtable, c.dlens, pages, pages[..., 0].contiguous()[:1], **kw)),
        (ValueError, "q", lambda: fk.sparse_decode_attn(q.transpose(0, 1), c.k, c.v, c.dtable, c.dlens, pages, **kw)),
        (ValueError, "v_cache", lambda: fk.sparse_decode_attn(q, c.k, c.v[1:], c.dtable, c.dlens, pages, **kw)),
        (ValueError, "out", lambda: fk.sparse_decode_attn(q, c.k, c.v, c.dtable, c.dlens, pages, out=torch.zeros(2, 4, 32, device=DEV), **kw)),
    ]
    for kind, what, call in bad:
        with pytest.raises(kind, match=what):
            call()
