"""The operators around the paged cache that perf measurements run: rotary positions fused
with the cache write, reading cached rows back, and the latent cache (one shared vector a
token) with its write, read and absorbed decode attention.

Every operator has a plain form here (elementary torch operations, fp32 or fp64) and the
call a user makes of the library (`own` true).  The cases stand for decode steps, prompt
chunks and whole prompts of the sizes this repository's workloads use.
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
        # one decode step of a small batch: latency of a single launch
        {"name": "rope write step", "op": "rope_write", "T": 8, "Hq": 32, "Hkv": 8, "D": 128, "rd": 128,
         "interleaved": False, "cache": "e4m3", "mode": "token", "start": 20000},
        # a long prompt's chunk stored at once, far positions, long-context frequencies
        {"name": "rope write prompt", "op": "rope_write", "T": 32768, "Hq": 32, "Hkv": 8, "D": 128, "rd": 128,
         "interleaved": False, "cache": "e4m3", "mode": "token", "start": 98304},
        # an odd prompt: wide heads, a quarter of each rotated, interleaved pairs, per-tensor scale
        {"name": "rope write odd", "op": "rope_write", "T": 4099, "Hq": 8, "Hkv": 1, "D": 256, "rd": 64,
         "interleaved": True, "cache": "e4m3", "mode": "tensor", "start": 77},
        # a short cached prefix read back
        {"name": "kv read prefix", "op": "kv_read", "T": 1000, "Hkv": 8, "D": 64, "cache": "e4m3", "mode": "token"},
        # a 128k-token context read back in bf16
        {"name": "kv read context", "op": "kv_read", "T": 131072, "Hkv": 8, "D": 128, "cache": "e4m3",
         "mode": "token"},
        # one decode step of 32 sequences, the query's rotary part turned in the same call
        {"name": "latent write step", "op": "latent_write", "T": 32, "H": 128, "L": 512, "rd": 64,
         "interleaved": True, "cache": "e4m3", "mode": "token", "start": 20000},
        # a prompt chunk of a rank that holds 16 heads
        {"name": "latent write prompt", "op": "latent_write", "T": 32768, "H": 16, "L": 512, "rd": 64,
         "interleaved": True, "cache": "e4m3", "mode": "token", "start": 4096},
        # a prefix read back for the up-projection; a bf16 cache of odd length
        {"name": "latent read prefix", "op": "latent_read", "T": 1001, "L": 512, "cache": "bf16", "mode": "tensor"},
        {"name": "latent read context", "op": "latent_read", "T": 131072, "L": 512, "cache": "e4m3",
         "mode": "token"},
        # one sequence, short context, few heads: latency
        {"name": "latent attn tiny", "op": "latent_attn", "B": 1, "S": 1, "H": 16, "L": 512, "lo": 1024, "hi": 1024,
         "cache": "e4m3", "mode": "tensor"},
        # a batch under load, all 128 heads on one GPU
        {"name": "latent attn load", "op": "latent_attn", "B": 8, "S": 1, "H": 128, "L": 512, "lo": 18000,
         "hi": 22000, "cache": "e4m3", "mode": "token"},
        # ragged contexts, two query tokens a sequence (one drafted), 16 heads, bf16 cache
        {"name": "latent attn ragged", "op": "latent_attn", "B": 32, "S": 2, "H": 16, "L": 512, "lo": 1000,
         "hi": 32768, "cache": "bf16", "mode": "tensor"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_write", "kv_read", "latent_write", "latent_read", "latent_attn", "latent_attn"])
    cache = rng.choice(["e4m3", "e4m3", "bf16"])
    mode = rng.choice(["token", "tensor"]) if cache == "e4m3" else "tensor"
    if op == "rope_write":
        D = rng.choice([64, 128, 256])
        Hkv = rng.randint(1, 8)
        return {"op": op, "T": _log(rng, 1, 16000), "Hq": Hkv * rng.randint(1, 4), "Hkv": Hkv, "D": D,
                "rd": rng.choice([D, D // 2, D // 4]), "interleaved": rng.random() < 0.5, "cache": cache,
                "mode": mode, "start": _log(rng, 1, 1 << 20)}
    if op == "kv_read":
        return {"op": op, "T": _log(rng, 1, 60000), "Hkv": rng.randint(1, 8), "D": rng.choice([64, 128, 256]),
                "cache": cache, "mode": mode}
    if op == "latent_write":
        return {"op": op, "T": _log(rng, 1, 5000), "H": rng.choice([1, 8, 16, 20, 32, 64, 128]),
                "L": rng.choice([128, 256, 512]), "rd": 64, "interleaved": rng.random() < 0.5, "cache": cache,
                "mode": mode, "start": _log(rng, 1, 1 << 20)}
    if op == "latent_read":
        return {"op": op, "T": _log(rng, 1, 90000), "L": rng.choice([128, 256, 512]), "cache": cache, "mode": mode}
    hi = _log(rng, 16, 24000)
    B = _log(rng, 1, max(1, min(64, 160000 // hi)))
    H = rng.choice([1, 8, 16, 20, 32, 64, 128])
    return {"op": op, "B": B, "S": rng.choice([1, 1, 1, 2, 3]) if H <= 32 else 1, "H": H,
            "L": rng.choice([128, 256, 512, 512]), "lo": max(1, int(hi * rng.uniform(0.05, 1.0))), "hi": hi,
            "cache": cache, "mode": mode}


def _contexts(case):
    """Context lengths of the batch: log-spaced from lo to hi (a single sequence: hi)."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    if B == 1:
        return [hi]
    return [int(round(lo * (hi / lo) ** (i / (B - 1)))) for i in range(B)]


def work(case):
    op = case["op"]
    e = 1 if case["cache"] == "e4m3" else 2
    tok = 4 if case["mode"] == "token" else 0            # bytes of a stored scale
    if op == "rope_write":
        T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
        return {"bytes": T * (4 * Hq * D + 2 * Hkv * (D * (2 + e) + tok) + 16),
                "flops": 3 * T * (Hq + Hkv) * case["rd"]}
    if op == "kv_read":
        T, Hkv, D = case["T"], case["Hkv"], case["D"]
        return {"bytes": T * (2 * Hkv * (D * (e + 2) + tok) + 8), "flops": 2 * T * Hkv * D}
    W = case["L"] + 64
    if op == "latent_write":
        return {"bytes": case["T"] * (W * (2 + e) + tok + 4 * case["H"] * 64 + 16),
                "flops": 3 * case["T"] * (case["H"] + 1) * 64}
    if op == "latent_read":
        return {"bytes": case["T"] * (W * (e + 2) + tok + 8), "flops": case["T"] * W}
    n = sum(_contexts(case))
    rows = case["B"] * case["S"] * case["H"]
    return {"bytes": n * (W * e + tok) + 2 * rows * (W + case["L"]) + 4 * sum(-(-c // PAGE) for c in _contexts(case)),
            "flops": 2 * n * case["S"] * case["H"] * (W + case["L"])}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _frequencies(rd):
    """Angles per position (radians) of the rotated pairs, in 64 bits, and the same in
    2^-64ths of a turn (the table the library's calls take)."""
    i = torch.arange(rd // 2, dtype=torch.float64)
    theta = 500000.0 ** (-2.0 * i / rd)
    table = torch.tensor([int(round(t / (2.0 * math.pi) * 2.0 ** 64)) for t in theta.tolist()], dtype=torch.int64)
    return theta.cuda(), table.cuda()


def _codes(g, shape, cache):
    """Cache contents: rounded normals with a few strong channels, as codes or bf16."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    if cache == "bf16":
        return x
    return (x * 100.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    e4m3, token = case["cache"] == "e4m3", case["mode"] == "token"
    s = {"case": case, "op": op, "e4m3": e4m3, "token": token}
    dt = torch.uint8 if e4m3 else torch.bfloat16
    if op == "latent_attn":
        B, W = case["B"], case["L"] + 64
        order = torch.randperm(B, generator=g, device="cuda").cpu().tolist()
        lens = [_contexts(case)[i] for i in order]
        mbs = -(-max(lens) // PAGE)
        nb = B * mbs + 3
        s["q"] = _randn(g, B, case["S"], case["H"], W)
        s["cache"] = _codes(g, (nb, PAGE, W), case["cache"])
        s["context_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["block_table"] = torch.randperm(nb, generator=g, device="cuda")[:B * mbs].view(B, mbs).to(torch.int32)
        s["scale"] = torch.full((1,), 0.01, device="cuda")
        s["scale_cache"] = torch.rand(nb, PAGE, generator=g, device="cuda") * 0.01 + 0.005
        s["softmax_scale"] = 1.0 / math.sqrt(192.0)
        s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
        return s
    T = case["T"]
    nb = -(-T // PAGE) + 5
    pages = torch.randperm(nb, generator=g, device="cuda")
    t = torch.arange(T, device="cuda")
    s["slots"] = pages[t // PAGE] * PAGE + t % PAGE
    s["positions"] = t + case.get("start", 0)
    if "rd" in case:
        s["theta"], s["table"] = _frequencies(case["rd"])
    if op in ("rope_write", "kv_read"):
        Hkv, D = case["Hkv"], case["D"]
        s["k_scale"] = torch.full((1,), 0.0625, device="cuda")
        s["v_scale"] = torch.full((1,), 0.03125, device="cuda")
        if op == "rope_write":
            Hq = case["Hq"]
            # q, k and v are views of one projection's output
            qkv = _randn(g, T, Hq + 2 * Hkv, D)
            qkv[:, Hq, 3] *= 20                            # a strong key channel
            s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
            s["k_cache"] = torch.zeros(nb, Hkv, PAGE, D, dtype=dt, device="cuda")
            s["v_cache"] = torch.zeros(nb, Hkv, PAGE, D, dtype=dt, device="cuda")
            s["k_scale_cache"] = torch.zeros(nb, Hkv, PAGE, device="cuda")
            s["v_scale_cache"] = torch.zeros(nb, Hkv, PAGE, device="cuda")
        else:
            s["k_cache"] = _codes(g, (nb, Hkv, PAGE, D), case["cache"])
            s["v_cache"] = _codes(g, (nb, Hkv, PAGE, D), case["cache"])
            s["k_scale_cache"] = torch.rand(nb, Hkv, PAGE, generator=g, device="cuda") * 0.01 + 0.005
            s["v_scale_cache"] = torch.rand(nb, Hkv, PAGE, generator=g, device="cuda") * 0.01 + 0.005
        return s
    L = case["L"]
    s["scale"] = torch.full((1,), 0.0625, device="cuda")
    if op == "latent_write":
        # the down-projection's output: the latent and the shared rotary key side by side
        ckr = _randn(g, T, L + 64)
        s["c"], s["k_pe"] = ckr[:, :L], ckr[:, L:]
        s["q"] = _randn(g, T, case["H"], L + 64)           # absorbed queries; the last 64 get turned
        s["q_pe"] = _randn(g, T, case["H"], 64)
        s["cache"] = torch.zeros(nb, PAGE, L + 64, dtype=dt, device="cuda")
        s["scale_cache"] = torch.zeros(nb, PAGE, device="cuda")
    else:
        s["cache"] = _codes(g, (nb, PAGE, L + 64), case["cache"])
        s["scale_cache"] = torch.rand(nb, PAGE, generator=g, device="cuda") * 0.01 + 0.005
    return s


# ---------------------------------------------------------------- the operators
def _f8(t):
    """A cache's bytes as the e4m3 values they are (bf16 caches as they are)."""
    return t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t


def run(s):
    return _RUN[s["op"]](s)


def _cos_sin(s):
    angle = s["positions"].to(torch.float64)[:, None, None] * s["theta"]      # [T][1][rd/2]
    return torch.cos(angle).float(), torch.sin(angle).float()


def _rotate(x, cos, sin, rd, interleaved):
    """x [T][H][D] fp32, its first rd dimensions turned."""
    if interleaved:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rd // 2], x[..., rd // 2:rd]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((turned, x[..., rd:]), dim=-1)


def _store(x, cache, at, e4m3, scale):
    """Rows x (fp32) into the cache at index `at`, as codes of x / scale or as bf16."""
    if e4m3:
        cache[at] = (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        cache[at] = x.to(torch.bfloat16)


def _rope_write(s):
    c = s["case"]
    if own:
        fk = _api()
        q = fk.rope_kv_cache_write(
            s["q"], s["k"], s["v"], s["positions"], s["slots"], s["table"], s["k_cache"], s["v_cache"],
            kv_dtype=fk.KV_E4M3 if s["e4m3"] else fk.KV_BF16,
            scale_mode=fk.SCALE_PER_TOKEN_HEAD if s["token"] else fk.SCALE_PER_TENSOR,
            interleaved=c["interleaved"], k_scale=s["k_scale"], v_scale=s["v_scale"],
            k_scale_cache=s["k_scale_cache"], v_scale_cache=s["v_scale_cache"])
    else:
        cos, sin = _cos_sin(s)
        q = _rotate(s["q"].float(), cos, sin, c["rd"], c["interleaved"]).to(torch.bfloat16)
        k, v = _rotate(s["k"].float(), cos, sin, c["rd"], c["interleaved"]), s["v"].float()
        blk, off = s["slots"] // PAGE, s["slots"] % PAGE
        ks, vs = s["k_scale"], s["v_scale"]
        if s["token"]:
            ks, vs = k.abs().amax(-1, keepdim=True) / 448.0, v.abs().amax(-1, keepdim=True) / 448.0
            s["k_scale_cache"][blk, :, off] = ks[..., 0]
            s["v_scale_cache"][blk, :, off] = vs[..., 0]
        at = (blk[:, None], torch.arange(c["Hkv"], device="cuda")[None, :], off[:, None])
        _store(k, s["k_cache"], at, s["e4m3"], ks)
        _store(v, s["v_cache"], at, s["e4m3"], vs)
    return {"q": q, "k_cache": _f8(s["k_cache"]), "v_cache": _f8(s["v_cache"]),
            "k_scales": s["k_scale_cache"], "v_scales": s["v_scale_cache"]}


def _kv_read(s):
    if own:
        fk = _api()
        k, v = fk.kv_cache_read(
            s["k_cache"], s["v_cache"], s["slots"], kv_dtype=fk.KV_E4M3 if s["e4m3"] else fk.KV_BF16,
            scale_mode=fk.SCALE_PER_TOKEN_HEAD if s["token"] else fk.SCALE_PER_TENSOR, k_scale=s["k_scale"],
            v_scale=s["v_scale"], k_scale_cache=s["k_scale_cache"], v_scale_cache=s["v_scale_cache"],
            out_dtype=fk.OUT_BF16)
        return {"k": k, "v": v}
    blk, off = s["slots"] // PAGE, s["slots"] % PAGE
    out = {}
    for n in ("k", "v"):
        x = _f8(s[n + "_cache"])[blk, :, off].float()
        if s["e4m3"]:
            x = x * (s[n + "_scale_cache"][blk, :, off][..., None] if s["token"] else s[n + "_scale"])
        out[n] = x.to(torch.bfloat16)
    return out


def _latent_write(s):
    c = s["case"]
    L = c["L"]
    if own:
        fk = _api()
        fk.latent_cache_write(
            s["c"], s["k_pe"], s["slots"], s["cache"], kv_dtype=fk.KV_E4M3 if s["e4m3"] else fk.KV_BF16,
            scale_mode=fk.SCALE_PER_TOKEN_HEAD if s["token"] else fk.SCALE_PER_TENSOR, scale=s["scale"],
            scale_cache=s["scale_cache"], positions=s["positions"], rope_freqs=s["table"],
            interleaved=c["interleaved"], q_pe=s["q_pe"], q_pe_out=s["q"][..., L:])
    else:
        cos, sin = _cos_sin(s)
        s["q"][..., L:] = _rotate(s["q_pe"].float(), cos, sin, 64, c["interleaved"]).to(torch.bfloat16)
        k_pe = _rotate(s["k_pe"].float()[:, None], cos, sin, 64, c["interleaved"])[:, 0]
        x = torch.cat((s["c"].float(), k_pe), dim=-1)
        blk, off = s["slots"] // PAGE, s["slots"] % PAGE
        scale = s["scale"]
        if s["token"]:
            scale = x.abs().amax(-1, keepdim=True) / 448.0
            s["scale_cache"][blk, off] = scale[:, 0]
        _store(x, s["cache"], (blk, off), s["e4m3"], scale)
    return {"q_pe": s["q"][..., L:], "cache": _f8(s["cache"]), "scales": s["scale_cache"]}


def _latent_read(s):
    if own:
        fk = _api()
        return fk.latent_cache_read(
            s["cache"], s["slots"], kv_dtype=fk.KV_E4M3 if s["e4m3"] else fk.KV_BF16,
            scale_mode=fk.SCALE_PER_TOKEN_HEAD if s["token"] else fk.SCALE_PER_TENSOR, scale=s["scale"],
            scale_cache=s["scale_cache"], out_dtype=fk.OUT_BF16)
    x = _f8(s["cache"]).flatten(0, 1)[s["slots"]].float()
    if s["e4m3"]:
        x = x * (s["scale_cache"].flatten()[s["slots"]][:, None] if s["token"] else s["scale"])
    return x.to(torch.bfloat16)


def _rows(s, dtype):
    """The batch's cached rows [B][padded length][L + 64] in `dtype`, and which keys each
    query token sees [B][S][padded length]."""
    x = _f8(s["cache"])[s["block_table"].long()].to(dtype)                  # [B][mbs][16][W]
    if s["e4m3"]:
        x = x * (s["scale_cache"][s["block_table"].long()][..., None] if s["token"] else s["scale"]).to(dtype)
    x = x.flatten(1, 2)
    S = s["case"]["S"]
    last = s["context_lens"][:, None] - S + torch.arange(S, device="cuda")  # a query's own position
    return x, torch.arange(x.shape[1], device="cuda") <= last[..., None]


def _latent_attn(s):
    c = s["case"]
    if own:
        fk = _api()
        return fk.latent_decode_attn(
            s["q"], s["cache"], s["block_table"], s["context_lens"], latent_dim=c["L"],
            kv_dtype=fk.KV_E4M3 if s["e4m3"] else fk.KV_BF16,
            scale_mode=fk.SCALE_PER_TOKEN_HEAD if s["token"] else fk.SCALE_PER_TENSOR, scale=s["scale"],
            scale_cache=s["scale_cache"], softmax_scale=s["softmax_scale"], workspace=s["workspace"],
            out_dtype=fk.OUT_BF16)
    return _attend(s, torch.float32).to(torch.bfloat16)


def _attend(s, dtype):
    c = s["case"]
    B, S, H = c["B"], c["S"], c["H"]
    x, seen = _rows(s, dtype)
    z = torch.matmul(s["q"].to(dtype).view(B, S * H, -1), x.transpose(1, 2)).mul_(s["softmax_scale"])
    z = z.view(B, S, H, -1).masked_fill_(~seen[:, :, None], float("-inf"))
    z = torch.exp(z - z.amax(-1, keepdim=True).clamp_min(-1e30))            # a row that sees nothing: zeros
    o = torch.matmul(z.view(B, S * H, -1), x[..., :c["L"]]).view(B, S, H, -1)
    return o / z.sum(-1, keepdim=True).clamp_min(1e-30)


_RUN = {"rope_write": _rope_write, "kv_read": _kv_read, "latent_write": _latent_write,
        "latent_read": _latent_read, "latent_attn": _latent_attn}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "latent_attn":
        x, seen = _rows64(s)
        return _softmax_rows64(s, x, seen)
    at = s["slots"]
    if op == "kv_read":
        out = {}
        for n in ("k", "v"):
            x = _cache64(s[n + "_cache"]).transpose(1, 2).flatten(0, 1)[at]
            if s["e4m3"]:
                sc = s[n + "_scale_cache"].double().transpose(1, 2).flatten(0, 1)[at][..., None]
                x *= sc if s["token"] else s[n + "_scale"].double()
            out[n] = x
        return out
    if op == "latent_read":
        x = _cache64(s["cache"]).flatten(0, 1)[at]
        if s["e4m3"]:
            x *= s["scale_cache"].double().flatten()[at][:, None] if s["token"] else s["scale"].double()
        return x
    if op == "latent_write":
        L = case["L"]
        q = _turn64(s["q_pe"].double(), s, case)
        x = torch.cat((s["c"].double(), _turn64(s["k_pe"].double()[:, None], s, case)[:, 0]), dim=1)
        rows, scales = _quantised64(x, s, s["scale"])
        n = s["cache"].shape[0] * PAGE
        cache = torch.zeros(n, L + 64, dtype=torch.float64, device="cuda")
        cache[at] = rows
        sc = torch.zeros(n, dtype=torch.float64, device="cuda")
        if s["token"]:
            sc[at] = scales[:, 0]
        return {"q_pe": q, "cache": cache.view(-1, PAGE, L + 64), "scales": sc.view(-1, PAGE)}
    nb, Hkv, _, D = s["k_cache"].shape
    out = {"q": _turn64(s["q"].double(), s, case)}
    for n, x in (("k", _turn64(s["k"].double(), s, case)), ("v", s["v"].double())):
        rows, scales = _quantised64(x, s, s[n + "_scale"])
        cache = torch.zeros(nb * PAGE, Hkv, D, dtype=torch.float64, device="cuda")
        cache[at] = rows
        sc = torch.zeros(nb * PAGE, Hkv, dtype=torch.float64, device="cuda")
        if s["token"]:
            sc[at] = scales[..., 0]
        out[n + "_cache"] = cache.view(nb, PAGE, Hkv, D).transpose(1, 2)
        out[n + "_scales"] = sc.view(nb, PAGE, Hkv).transpose(1, 2)
    return out


def _cache64(t):
    return (t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t).double()


def _quantised64(x, s, given):
    """(what the stored codes stand for before they are rounded, the scales)."""
    if not s["e4m3"]:
        return x, None
    scale = x.abs().max(-1, keepdim=True).values / 448 if s["token"] else given.double()
    return torch.clamp(x / scale, min=-448, max=448), scale


def _turn64(x, s, case):
    """x [T][H][D] as complex numbers times e^(i angle)."""
    rd = case["rd"]
    turn = torch.polar(torch.ones_like(s["theta"])[None].expand(x.shape[0], -1),
                       s["positions"].double()[:, None] * s["theta"])[:, None]
    y = x.clone()
    if case["interleaved"]:
        z = torch.view_as_complex(x[..., :rd].reshape(*x.shape[:-1], rd // 2, 2).contiguous()) * turn
        y[..., :rd] = torch.view_as_real(z).reshape(*x.shape[:-1], rd)
    else:
        z = torch.complex(x[..., :rd // 2].contiguous(), x[..., rd // 2:rd].contiguous()) * turn
        y[..., :rd // 2], y[..., rd // 2:rd] = z.real, z.imag
    return y


def _rows64(s):
    blocks = s["block_table"].long()
    x = _cache64(s["cache"])[blocks]
    if s["e4m3"]:
        x *= s["scale_cache"].double()[blocks].unsqueeze(-1) if s["token"] else s["scale"].double()
    x = x.reshape(x.shape[0], -1, x.shape[-1])
    S = s["case"]["S"]
    t = torch.arange(x.shape[1], device="cuda")
    own_pos = s["context_lens"].long().unsqueeze(1) - S + torch.arange(S, device="cuda")
    return x, t.view(1, 1, -1) <= own_pos.unsqueeze(-1)


def _softmax_rows64(s, x, seen):
    L = s["case"]["L"]
    out = []
    for b in range(x.shape[0]):
        z = torch.einsum("shw,tw->sht", s["q"][b].double(), x[b]) * s["softmax_scale"]
        z = torch.where(seen[b].unsqueeze(1), z, torch.full_like(z, float("-inf")))
        p = torch.nan_to_num(torch.softmax(z, dim=-1), nan=0.0)
        out.append(torch.einsum("sht,tl->shl", p, x[b][:, :L]))
    return torch.stack(out)
