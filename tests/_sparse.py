"""Plain 64-bit implementations that the tests of page bounds, page selection, sparse and
prefix decode attention compare with, the caches they run on, and the bounds that results
are held to.  Written from the definitions, with no code of the library."""
import torch

from _latent import HALF, codes_to_values

PAGE = 16


class Cache:
    """A paged cache of random rows: codes (every bit pattern but NaN's) or bf16, scales of
    its mode, and the values they stand for in 64 bits.  Blocks are handed out in a shuffled
    order; what no sequence holds is filled with NaN bytes."""

    def __init__(self, seed, lens, Hkv, D, kind, extra=3, dev="cuda", amplitude=1.0):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.Hkv, self.D, self.lens = kind, Hkv, D, list(lens)
        B = len(self.lens)
        self.mbs = max(1, max(-(-n // PAGE) for n in self.lens))
        self.nb = B * self.mbs + extra
        order = torch.randperm(self.nb, generator=g)
        self.table = order[:B * self.mbs].view(B, self.mbs).to(torch.int32)
        self.spare = order[B * self.mbs:].to(torch.int32)
        self.e4m3 = kind != "bf16"
        shape = (self.nb, Hkv, PAGE, D)
        x = {n: (torch.randn(shape, generator=g) * amplitude) for n in "kv"}
        self.kw, self.val, raw = {}, {}, {}
        for n in "kv":
            if not self.e4m3:
                raw[n] = x[n].to(torch.bfloat16)
                self.val[n] = raw[n].double()
                continue
            raw[n] = (x[n] * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            if kind == "tensor":
                s = torch.rand(1, generator=g) * 0.01 + 0.005
                full, self.kw[n + "_scale"] = s.view(1, 1, 1, 1), s
            elif kind == "head":
                s = torch.rand(Hkv, generator=g) * 0.01 + 0.005
                full, self.kw[n + "_scale"] = s.view(1, Hkv, 1, 1), s
            else:
                s = torch.rand(self.nb, Hkv, PAGE, generator=g) * 0.01 + 0.005
                full, self.kw[n + "_scale_cache"] = s[..., None], s
            self.val[n] = codes_to_values(raw[n]) * full.double()
        # rows that no sequence holds: NaN codes, NaN scales
        used = torch.zeros(self.nb, PAGE, dtype=torch.bool)
        for b, n in enumerate(self.lens):
            for p in range(-(-n // PAGE)):
                used[self.table[b, p], :min(PAGE, n - p * PAGE)] = True
        for n in "kv":
            junk = ~used[:, None, :].expand(self.nb, Hkv, PAGE)
            if self.e4m3:
                raw[n][junk] = 0x7F
                if kind == "token":
                    self.kw[n + "_scale_cache"][junk] = float("nan")
            else:
                raw[n][junk] = float("nan")
        self.k, self.v = raw["k"].to(dev), raw["v"].to(dev)
        self.kw = {n: t.to(dev) for n, t in self.kw.items()}
        self.dev = dev
        self.dtable = self.table.to(dev)
        self.dlens = torch.tensor(self.lens, dtype=torch.int32, device=dev)

    def args(self, fk, only=""):
        """Keyword arguments of the cache's type and scales (only "k": the keys' scales)."""
        mode = {"tensor": fk.SCALE_PER_TENSOR, "head": fk.SCALE_PER_HEAD,
                "token": fk.SCALE_PER_TOKEN_HEAD, "bf16": fk.SCALE_PER_TENSOR}[self.kind]
        return dict(kv_dtype=fk.KV_E4M3 if self.e4m3 else fk.KV_BF16, scale_mode=mode,
                    **{n: t for n, t in self.kw.items() if n.startswith(only)})

    def rows(self, name, b, h, pages):
        """Values of sequence b's tokens on those of its pages (in that order), masked at its
        length: ([n][D], positions [n])."""
        n = self.lens[b]
        x, pos = [], []
        for p in pages:
            t = min(PAGE, n - p * PAGE)
            if t > 0:
                x.append(self.val[name][int(self.table[b, p]), h, :t])
                pos += range(p * PAGE, p * PAGE + t)
        return torch.cat(x) if x else torch.zeros(0, self.D, dtype=torch.float64)


def attend(q, k, v, scale, weight=2.0 ** -16):
    """(softmax(q k^T scale) v, bound) in 64 bits for one query [D] and its keys.

    The bound is on an fp32 result.  A logit is a sum of D products in fp32: at most D / 16
    roundings (one a step of the tensor pipe, which may truncate: a whole unit, 2^-23, of the
    sum of magnitudes S), one for each factor: off by z <= (D / 16 + 4) 2^-23 S.  A weight is
    off by z relative to itself, and so is the sum it is divided by; exp2's approximation adds
    2^-21, the rounding of a weight `weight` (two bf16 terms: 2^-16, coarser than two f16 terms;
    one f16 term: 2^-12), the sums over n keys (n + 64) 2^-23."""
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    z = k @ q * scale
    p = torch.softmax(z, 0)
    S = float(((k.abs() @ q.abs()) * scale).max())
    D, n = q.shape[0], k.shape[0]
    rel = 2 * (D / 16 + 4) * 2.0 ** -23 * S + 2.0 ** -20 + weight + 2 * (n + 64) * 2.0 ** -23
    return p @ v, (p @ v.abs()) * rel + 1e-30


def rounded(bound, want, out_bf16):
    """The bound behind an output rounded to its type."""
    return bound + want.abs() * HALF[torch.bfloat16 if out_bf16 else torch.float32]


def bounds_of(x):
    """(hi codes, lo codes, scale) of one page's keys [tokens][D] (fp32): rounded as defined,
    every fp32 operation an IEEE one on the CPU."""
    x = torch.nan_to_num(x.float(), nan=0.0, posinf=torch.finfo(torch.float32).max,
                         neginf=torch.finfo(torch.float32).min)
    hi, lo = x.amax(0), x.amin(0)
    s = torch.maximum(hi.abs(), lo.abs()).max() / torch.tensor(127.0)
    if float(s) == 0.0:
        z = torch.zeros_like(hi, dtype=torch.int8)
        return z, z, s
    code = lambda t: torch.round(t / s).clamp(-127, 127).to(torch.int8)
    return code(hi), code(lo), s


def query_codes(q):
    """The 8-bit query [2 D] of one KV head's query heads q [G][D] (bf16)."""
    q = q.double()
    u = torch.cat((q.clamp(min=0).sum(0), q.clamp(max=0).sum(0))).float()
    s = u.abs().max() / torch.tensor(127.0)
    if float(s) == 0.0:
        return torch.zeros_like(u, dtype=torch.int64)
    return torch.round(u / s).long()


def select(q, bounds, scale, n, budget, sink, recent):
    """The page list of one (sequence, KV head): bounds [n][2][D] int8, scale [n] fp32."""
    if n <= budget:
        return list(range(n))
    c = query_codes(q)
    score = (bounds.reshape(n, -1).long() @ c).float() * scale
    forced = set(range(sink)) | set(range(n - recent, n))
    order = sorted((p for p in range(n) if p not in forced), key=lambda p: (-float(score[p]), p))
    return sorted(list(forced) + order[:budget - len(forced)])
