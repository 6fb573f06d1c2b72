"""More operators around the paged cache that perf measurements run: decode attention that
does not read every cached key for every sequence.  Bounds of each page's keys, the pages a
query takes by those bounds, attention over the pages taken, and attention of a batch whose
sequences share a long prefix.

Every operator has a plain form here (elementary torch operations, fp32 or fp64) and the
call a user makes of the library (`own` true).  The cases stand for decode steps and
prompts of the sizes this repository's workloads use.
"""
import math

import torch

own = False

PAGE = 16


def _api():
    import fp8_kv_cache_write_gb300 as fk
    return fk


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's new tokens: the last page of each of 32 sequences is summed up again
        {"name": "bounds step", "op": "bounds", "B": 32, "Hkv": 8, "D": 128, "lo": 1000, "hi": 32768, "new": 1,
         "cache": "e4m3", "mode": "token"},
        # a 128k-token prompt's pages after it was stored
        {"name": "bounds prompt", "op": "bounds", "B": 1, "Hkv": 8, "D": 128, "lo": 131072, "hi": 131072, "new": 0,
         "cache": "e4m3", "mode": "token"},
        # a ragged batch of short prompts, wide heads, bf16 cache
        {"name": "bounds ragged", "op": "bounds", "B": 5, "Hkv": 2, "D": 256, "lo": 77, "hi": 4099, "new": 0,
         "cache": "bf16", "mode": "tensor"},
        # one request over a 128k-token context: latency
        {"name": "select one", "op": "select", "B": 1, "Hq": 64, "Hkv": 8, "D": 128, "lo": 131072, "hi": 131072,
         "budget": 128, "sink": 1, "recent": 4},
        # a batch under load, a tenth of its pages
        {"name": "select load", "op": "select", "B": 8, "Hq": 32, "Hkv": 8, "D": 128, "lo": 18000, "hi": 22000,
         "budget": 128, "sink": 1, "recent": 4},
        # a ragged batch with long contexts, some shorter than the budget
        {"name": "select ragged", "op": "select", "B": 32, "Hq": 64, "Hkv": 8, "D": 64, "lo": 1000, "hi": 65000,
         "budget": 200, "sink": 2, "recent": 8},
        # one request, 128 pages of a 128k-token context: latency
        {"name": "sparse attn one", "op": "sparse", "B": 1, "Hq": 64, "Hkv": 8, "D": 128, "lo": 131072,
         "hi": 131072, "budget": 128, "cache": "e4m3", "mode": "token"},
        # a larger batch, 256 pages a head
        {"name": "sparse attn load", "op": "sparse", "B": 32, "Hq": 32, "Hkv": 8, "D": 128, "lo": 18000, "hi": 22000,
         "budget": 256, "cache": "e4m3", "mode": "token"},
        # wide heads in bf16, contexts shorter and longer than the budget, an odd one
        {"name": "sparse attn ragged", "op": "sparse", "B": 9, "Hq": 8, "Hkv": 1, "D": 256, "lo": 100, "hi": 9001,
         "budget": 301, "cache": "bf16", "mode": "tensor"},
        # a few sequences behind a short system prompt: latency
        {"name": "prefix attn few", "op": "prefix", "B": 4, "Hq": 32, "Hkv": 8, "D": 128, "prefix": 2000, "lo": 20,
         "hi": 300, "cache": "e4m3", "mode": "tensor"},
        # a batch that asks about one 32k-token document
        {"name": "prefix attn load", "op": "prefix", "B": 32, "Hq": 32, "Hkv": 8, "D": 128, "prefix": 32768,
         "lo": 100, "hi": 1000, "cache": "e4m3", "mode": "token"},
        # many samples of one prompt, eight query heads a key head, bf16 cache, an odd length
        {"name": "prefix attn samples", "op": "prefix", "B": 100, "Hq": 64, "Hkv": 8, "D": 64, "prefix": 8197,
         "lo": 1, "hi": 500, "cache": "bf16", "mode": "tensor"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["bounds", "select", "sparse", "sparse", "prefix", "prefix"])
    cache = rng.choice(["e4m3", "e4m3", "bf16"])
    mode = rng.choice(["token", "tensor"]) if cache == "e4m3" else "tensor"
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.randint(1, 8)
    G = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
    if op == "prefix":
        prefix = _log(rng, 16, 30000)
        most = max(1, min(100, 900_000_000 // (prefix * G * Hkv * D)))
        hi = _log(rng, 1, 1000)
        return {"op": op, "B": _log(rng, 1, most), "Hq": Hkv * G, "Hkv": Hkv, "D": D, "prefix": prefix,
                "lo": max(1, int(hi * rng.uniform(0.05, 1.0))), "hi": hi, "cache": cache, "mode": mode}
    hi = _log(rng, 16, 60000)
    lo = max(1, int(hi * rng.uniform(0.05, 1.0)))
    B = _log(rng, 1, max(1, min(32, 600_000_000 // (hi * Hkv * D * 8))))
    if op == "bounds":
        return {"op": op, "B": B, "Hkv": Hkv, "D": D, "lo": lo, "hi": hi, "new": rng.choice([0, 1, _log(rng, 1, hi)]),
                "cache": cache, "mode": mode}
    budget = _log(rng, 8, max(9, min(400, _pages(hi))))
    if op == "select":
        return {"op": op, "B": B, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "lo": lo, "hi": hi, "budget": budget,
                "sink": rng.randint(0, 3), "recent": rng.randint(1, 5)}
    return {"op": op, "B": B, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "lo": lo, "hi": hi, "budget": budget,
            "cache": cache, "mode": mode}


def _contexts(case):
    """Context lengths of the batch: log-spaced from lo to hi (a single sequence: hi)."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    if B == 1:
        return [hi]
    return [int(round(lo * (hi / lo) ** (i / (B - 1)))) for i in range(B)]


def _pages(n):
    return -(-n // PAGE)


def _first_page(case, ctx):
    """The first page that the last `new` tokens of a sequence touch (0 new: all pages)."""
    return max(0, ctx - case["new"]) // PAGE if case["new"] else 0


def work(case):
    op, Hkv, D = case["op"], case["Hkv"], case["D"]
    ctx = _contexts(case)
    if op == "select":
        out = case["B"] * Hkv * (case["budget"] + 1) * 4
        n = [_pages(c) for c in ctx if _pages(c) > case["budget"]]
        return {"bytes": sum(n) * (Hkv * (2 * D + 4) + 4) + 2 * len(n) * case["Hq"] * D + out + 4 * case["B"],
                "flops": sum(n) * Hkv * 4 * D}
    e = 1 if case["cache"] == "e4m3" else 2
    tok = 4 if case["mode"] == "token" else 0            # bytes of a stored scale
    if op == "bounds":
        first = [_first_page(case, c) for c in ctx]
        rows = sum(c - PAGE * f for c, f in zip(ctx, first))
        pages = sum(_pages(c) - f for c, f in zip(ctx, first))
        return {"bytes": rows * Hkv * (D * e + tok) + pages * (Hkv * (2 * D + 4) + 4), "flops": 3 * rows * Hkv * D}
    rows = 4 * case["B"] * case["Hq"] * D                # q read, the output written
    if op == "sparse":
        n = sum(min(c, PAGE * case["budget"]) for c in ctx) * Hkv
        ids = sum(min(_pages(c), case["budget"]) for c in ctx) * Hkv
        return {"bytes": n * 2 * (D * e + tok) + rows + 8 * ids, "flops": 4 * D * n * (case["Hq"] // Hkv)}
    n = case["prefix"] + sum(ctx)
    return {"bytes": n * Hkv * 2 * (D * e + tok) + rows + 4 * (_pages(case["prefix"]) + sum(_pages(c) for c in ctx)),
            "flops": 4 * D * case["Hq"] * (case["B"] * case["prefix"] + sum(ctx))}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _codes(g, shape, cache):
    """Cache contents: rounded normals, as codes or bf16."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    if cache == "bf16":
        return x
    return (x * 100.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    g = _gen(seed)
    op, B, Hkv, D = case["op"], case["B"], case["Hkv"], case["D"]
    s = {"case": case, "op": op}
    order = torch.randperm(B, generator=g, device="cuda").cpu().tolist()
    lens = [_contexts(case)[i] for i in order]
    mbs = _pages(max(lens))
    npre = _pages(case.get("prefix", 0))
    nb = B * mbs + npre + 3
    blocks = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    s["context_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["block_table"] = blocks[:B * mbs].view(B, mbs)
    s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    if op != "bounds":
        s["q"] = _randn(g, B, case["Hq"], D)
    if op == "select":
        # channels whose keys lie around a mean of their own, some pages far from it
        mid = torch.randn(Hkv, 1, D, generator=g, device="cuda")
        half = torch.randn(nb, Hkv, 1, D, generator=g, device="cuda").abs_().mul_(0.4).add_(1.2)
        centre = mid[None] + torch.randn(nb, Hkv, 1, D, generator=g, device="cuda") * 0.4
        x = torch.cat((centre + half, centre - half), dim=2)
        s["bounds_scale"] = x.abs().amax((2, 3)) / 127.0
        s["bounds"] = torch.round(x / s["bounds_scale"][..., None, None]).to(torch.int8)
        return s
    s["e4m3"], s["token"] = case["cache"] == "e4m3", case["mode"] == "token"
    s["k_cache"] = _codes(g, (nb, Hkv, PAGE, D), case["cache"])
    s["k_scale"] = torch.full((1,), 0.011, device="cuda")
    s["k_scale_cache"] = torch.rand(nb, Hkv, PAGE, generator=g, device="cuda") * 0.01 + 0.005
    if op == "bounds":
        s["bounds"] = torch.zeros(nb, Hkv, 2, D, dtype=torch.int8, device="cuda")
        s["bounds_scale"] = torch.zeros(nb, Hkv, device="cuda")
        return s
    s["v_cache"] = _codes(g, (nb, Hkv, PAGE, D), case["cache"])
    s["v_scale"] = torch.full((1,), 0.009, device="cuda")
    s["v_scale_cache"] = torch.rand(nb, Hkv, PAGE, generator=g, device="cuda") * 0.01 + 0.005
    s["softmax_scale"] = 1.0 / math.sqrt(D)
    if op == "prefix":
        s["prefix_table"] = blocks[B * mbs:B * mbs + npre]
        s["prefix_len"] = torch.full((1,), case["prefix"], dtype=torch.int32, device="cuda")
        return s
    # what a selection leaves: each head's pages in their order, the first and the last among
    # them, -1 behind the pages of a sequence that has fewer than the budget
    budget = case["budget"]
    n = _pages_of(s)[:, None]
    page = torch.arange(mbs, device="cuda")
    key = torch.rand(B, Hkv, mbs, generator=g, device="cuda")
    key = key.masked_fill((page == 0) | (page == n[..., None] - 1), -1.0).masked_fill(page >= n[..., None], 2.0)
    key = torch.nn.functional.pad(key, (0, max(0, budget - mbs)), value=2.0)
    best, at = torch.sort(key, dim=-1)
    at = torch.where(best[..., :budget] < 2.0, at[..., :budget], torch.full_like(at[..., :budget], 1 << 30))
    at = torch.sort(at, dim=-1).values
    s["pages"] = torch.where(at < (1 << 30), at, torch.full_like(at, -1)).to(torch.int32)
    s["counts"] = n.clamp(max=budget).expand(B, Hkv).to(torch.int32).contiguous()
    return s


# ---------------------------------------------------------------- the operators
def run(s):
    return _RUN[s["op"]](s)


def _f8(t):
    """A cache's bytes as the e4m3 values they are (bf16 caches as they are)."""
    return t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t


def _127():
    """127 as a divisor on the GPU: a division by a host number would be a product with its inverse."""
    return torch.full((1,), 127.0, device="cuda")


def _pages_of(s):
    return (s["context_lens"] + (PAGE - 1)) // PAGE


def _cache_kw(fk, s):
    return dict(kv_dtype=fk.KV_E4M3 if s["e4m3"] else fk.KV_BF16,
                scale_mode=fk.SCALE_PER_TOKEN_HEAD if s["token"] else fk.SCALE_PER_TENSOR)


def _kv_kw(fk, s):
    return dict(k_scale=s["k_scale"], v_scale=s["v_scale"], k_scale_cache=s["k_scale_cache"],
                v_scale_cache=s["v_scale_cache"], softmax_scale=s["softmax_scale"], out_dtype=fk.OUT_BF16,
                **_cache_kw(fk, s))


def _rows(s, name, at, dtype=torch.float32):
    """Cached rows at an index of (block, head) as values."""
    x = _f8(s[name + "_cache"])[at].to(dtype)
    if s["e4m3"]:
        x = x * (s[name + "_scale_cache"][at][..., None] if s["token"] else s[name + "_scale"]).to(dtype)
    return x


def _bounds(s):
    c = s["case"]
    if own:
        fk = _api()
        fk.kv_page_bounds(s["k_cache"], s["block_table"], s["context_lens"], s["bounds"], s["bounds_scale"],
                          new_tokens=c["new"] or None, k_scale=s["k_scale"], k_scale_cache=s["k_scale_cache"],
                          **_cache_kw(fk, s))
    else:
        B, mbs = s["block_table"].shape
        ctx = s["context_lens"][:, None]
        first = (ctx - c["new"]).clamp(min=0) // PAGE if c["new"] else torch.zeros_like(ctx)
        page = torch.arange(mbs, device="cuda")[None]
        b, p = torch.nonzero((page >= first) & (page < _pages_of(s)[:, None]), as_tuple=True)
        blk = s["block_table"][b, p].long()
        x = _rows(s, "k", blk)                                                    # [pages][Hkv][16][D]
        seen = (p[:, None] * PAGE + torch.arange(PAGE, device="cuda") < ctx[b])[:, None, :, None]
        hi = x.masked_fill(~seen, float("-inf")).amax(2)
        lo = x.masked_fill(~seen, float("inf")).amin(2)
        x = torch.stack((hi, lo), dim=2)
        scale = x.abs().amax((2, 3)) / _127()
        s["bounds"][blk] = torch.round(x / scale[..., None, None]).to(torch.int8)
        s["bounds_scale"][blk] = scale
    return {"bounds": s["bounds"], "scales": s["bounds_scale"]}


def _select(s):
    c = s["case"]
    B, Hkv, D, budget = c["B"], c["Hkv"], c["D"], c["budget"]
    if own:
        fk = _api()
        pages, counts = fk.kv_page_select(s["q"], s["bounds"], s["bounds_scale"], s["block_table"],
                                          s["context_lens"], budget=budget, sink=c["sink"], recent=c["recent"])
        return {"pages": pages, "counts": counts}
    q = s["q"].double().view(B, Hkv, -1, D)
    q = torch.cat((q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)), dim=-1).float()  # [B][Hkv][2 D]
    q = torch.round(q / (q.abs().amax(-1, keepdim=True) / _127()))
    at = s["block_table"].long()                                                  # [B][mbs]
    x = s["bounds"].flatten(2)[at].float()                                        # [B][mbs][Hkv][2 D]
    score = (x * q[:, None]).sum(-1) * s["bounds_scale"][at]                      # whole sums, one rounding
    score = score.transpose(1, 2)
    n = _pages_of(s)[:, None, None]
    page = torch.arange(at.shape[1], device="cuda")
    forced = (page < c["sink"]) | (page >= n - c["recent"])
    score = score.masked_fill(forced, float("inf")).masked_fill(page >= n, float("-inf"))
    score = torch.nn.functional.pad(score, (0, max(0, budget - score.shape[-1])), value=float("-inf"))
    best, at = torch.sort(score, dim=-1, descending=True, stable=True)
    at = at[..., :budget]
    at = torch.sort(torch.where(at < n, at, torch.full_like(at, 1 << 30)), dim=-1).values
    return {"pages": torch.where(at < (1 << 30), at, torch.full_like(at, -1)).to(torch.int32),
            "counts": n[..., 0].clamp(max=budget).expand(B, Hkv).to(torch.int32).contiguous()}


def _sparse(s):
    c = s["case"]
    if own:
        fk = _api()
        return fk.sparse_decode_attn(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["context_lens"],
                                     s["pages"], s["counts"], **_kv_kw(fk, s))
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    at = s["pages"].clamp(min=0).long()
    blk = s["block_table"].long().gather(1, at.view(B, -1)).view(at.shape)        # [B][Hkv][budget]
    head = torch.arange(Hkv, device="cuda")[None, :, None]
    k, v = _rows(s, "k", (blk, head)).flatten(2, 3), _rows(s, "v", (blk, head)).flatten(2, 3)
    pos = at[..., None] * PAGE + torch.arange(PAGE, device="cuda")
    seen = ((s["pages"][..., None] >= 0) & (pos < s["context_lens"][:, None, None, None])).flatten(2)
    z = torch.matmul(s["q"].float().view(B, Hkv, -1, D), k.transpose(2, 3)) * s["softmax_scale"]
    p = torch.exp((z := z.masked_fill(~seen[:, :, None], float("-inf"))) - z.amax(-1, keepdim=True).clamp_min(-1e30))
    return (torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp_min(1e-30)).view(B, Hkv * z.shape[2], D).to(
        torch.bfloat16)


def _prefix(s):
    c = s["case"]
    if own:
        fk = _api()
        return fk.prefix_decode_attn(s["q"], s["k_cache"], s["v_cache"], s["prefix_table"], s["prefix_len"],
                                     s["block_table"], s["context_lens"], workspace=s["workspace"],
                                     **_kv_kw(fk, s))
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    at = s["prefix_table"].long()
    pk, pv = (_rows(s, n, at).transpose(0, 1).flatten(1, 2) for n in ("k", "v"))  # [Hkv][keys][D]
    at = s["block_table"].long()
    k, v = (_rows(s, n, at).transpose(1, 2).flatten(2, 3) for n in ("k", "v"))    # [B][Hkv][keys][D]
    q = s["q"].float().view(B, Hkv, -1, D) * s["softmax_scale"]
    G = q.shape[2]
    zp = torch.matmul(q.transpose(0, 1).flatten(1, 2), pk.transpose(1, 2)).view(Hkv, B, G, -1).transpose(0, 1)
    zp = zp.masked_fill(torch.arange(zp.shape[-1], device="cuda") >= s["prefix_len"], float("-inf"))
    z = torch.matmul(q, k.transpose(2, 3))
    pos = torch.arange(z.shape[-1], device="cuda")
    z = z.masked_fill(pos >= s["context_lens"][:, None, None, None], float("-inf"))
    top = torch.maximum(z.amax(-1, keepdim=True), zp.amax(-1, keepdim=True)).clamp_min(-1e30)
    z, zp = torch.exp(z - top), torch.exp(zp - top)
    o = torch.matmul(zp.transpose(0, 1).flatten(1, 2), pv).view(Hkv, B, G, D).transpose(0, 1) + torch.matmul(z, v)
    o = o / (z.sum(-1, keepdim=True) + zp.sum(-1, keepdim=True)).clamp_min(1e-30)
    return o.reshape(B, Hkv * G, D).to(torch.bfloat16)


_RUN = {"bounds": _bounds, "select": _select, "sparse": _sparse, "prefix": _prefix}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"bounds": _bounds64, "select": _select64, "sparse": _sparse64, "prefix": _prefix64}[case["op"]](s, case)


def _cached64(s, name, blocks, head):
    """One head's rows of a list of blocks, [16 * blocks][D]."""
    x = s[name + "_cache"][blocks, head]
    x = (x.view(torch.float8_e4m3fn) if s["e4m3"] else x).double()
    if s["e4m3"]:
        x *= s[name + "_scale_cache"][blocks, head].double().unsqueeze(-1) if s["token"] else \
            s[name + "_scale"].double()
    return x.reshape(-1, x.shape[-1])


def _bounds64(s, case):
    # the codes are whole numbers by a rounding and have no value in 64 bits of their own
    scales = torch.zeros(s["bounds_scale"].shape, dtype=torch.float64, device="cuda")
    for b, ctx in enumerate(s["context_lens"].tolist()):
        first = _first_page(case, ctx)
        blocks = s["block_table"][b, first:_pages(ctx)].long()
        for h in range(case["Hkv"]):
            x = _cached64(s, "k", blocks, h)
            x[ctx - PAGE * first:] = 0
            scales[blocks, h] = x.abs().view(len(blocks), -1).max(1).values / 127
    return {"bounds": None, "scales": scales}


def _select64(s, case):
    B, Hkv, budget = case["B"], case["Hkv"], case["budget"]
    G = case["Hq"] // Hkv
    pages = torch.full((B, Hkv, budget), -1, dtype=torch.int64, device="cuda")
    counts = torch.zeros(B, Hkv, dtype=torch.int64, device="cuda")
    for b, ctx in enumerate(s["context_lens"].tolist()):
        n = _pages(ctx)
        blocks = s["block_table"][b, :n].long()
        for h in range(Hkv):
            q = s["q"][b, h * G:(h + 1) * G].double()
            w = torch.cat((torch.relu(q).sum(0), -torch.relu(-q).sum(0))).float()
            w = torch.round(w / torch.div(w.abs().max(), torch.full_like(w, 127))).long()
            code = s["bounds"][blocks, h].reshape(n, -1).long()
            score = (code * w).sum(1).float() * s["bounds_scale"][blocks, h]
            score[:case["sink"]] = math.inf
            score[max(0, n - case["recent"]):] = math.inf
            rank = torch.argsort(-score, stable=True)[:budget]
            counts[b, h] = len(rank)
            pages[b, h, :len(rank)] = rank.sort().values
    return {"pages": pages.to(torch.int32), "counts": counts.to(torch.int32)}


def _attend64(s, q, k, v):
    p = torch.softmax(q @ k.T * s["softmax_scale"], dim=-1)
    return p @ v


def _sparse64(s, case):
    G = case["Hq"] // case["Hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, ctx in enumerate(s["context_lens"].tolist()):
        for h in range(case["Hkv"]):
            page = s["pages"][b, h]
            page = page[page >= 0].long()
            blocks = s["block_table"][b].long()[page]
            seen = (page[:, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten() < ctx
            k, v = (_cached64(s, n, blocks, h)[seen] for n in ("k", "v"))
            out[b, h * G:(h + 1) * G] = _attend64(s, s["q"][b, h * G:(h + 1) * G].double(), k, v)
    return out


def _prefix64(s, case):
    if case["B"] * case["Hq"] * case["D"] * (case["prefix"] + case["hi"]) > 2e10:
        return None
    G, P = case["Hq"] // case["Hkv"], case["prefix"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for h in range(case["Hkv"]):
        pk, pv = (_cached64(s, n, s["prefix_table"].long(), h)[:P] for n in ("k", "v"))
        for b, ctx in enumerate(s["context_lens"].tolist()):
            k, v = (_cached64(s, n, s["block_table"][b].long(), h)[:ctx] for n in ("k", "v"))
            out[b, h * G:(h + 1) * G] = _attend64(s, s["q"][b, h * G:(h + 1) * G].double(), torch.cat((pk, k)),
                                                  torch.cat((pv, v)))
    return out
