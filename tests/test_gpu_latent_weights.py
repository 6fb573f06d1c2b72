"""GPU: what the latent attention's weights keep.  Rows whose logits are set exactly, in
binades, through two values of the rotary key; a latent column of ones, whose output is
the share of the softmax's mass that reached the result.

The bound of an e4m3 result: a weight of a code enters the product within 2^-8 of itself
(two terms: e4m3, 4 significant bits, and e5m2, 3 more of what that misses) and 2^-11 (by
way of f16), or, where it is small, within 2^-15 of the largest weight among its tile of
128 keys (e5m2's half step 2^-17 and, under 2^-6, 2^-14 of a unit that the tile's largest
exceeds twice) or 2^-54 of the row's largest (the reference stays within 2^40 of its
highest).  The sum of the weights is fp32's."""
import math

import pytest
import torch

import fp8_kv_cache_write_gb300 as fk
from tests._latent import latent_values

pytestmark = pytest.mark.gpu

LN2 = math.log(2.0)


class Rows:
    """`n` keys of one sequence whose logits, in binades, are z [n] for a query along the
    rotary values 0 and 1 (value 1 holds sixteenths); latents are normals but for column
    0, which is 1.  Per-token scales are powers of two, so that every value is a code."""

    def __init__(self, z, L=256, token=False, seed=0, kind="e4m3"):
        g = torch.Generator().manual_seed(seed)
        self.n, self.L, self.kind, self.token = len(z), L, kind, token
        n = self.n
        pages = -(-n // 16)
        nb = pages + 3
        x = torch.randn(nb, 16, L + 64, generator=g)
        x[..., 0] = 1.0
        x[..., L:] = 0.0
        self.bt = torch.randperm(nb - 1, generator=g)[:pages].to(torch.int32)[None]
        t = torch.arange(n)
        blk, off = self.bt[0].long()[t // 16], t % 16
        z = torch.as_tensor(z, dtype=torch.float32)
        fine = z - torch.round(z * 4) / 4            # whole quarters (exact codes), the rest finer
        x[blk, off, L] = z - fine
        x[blk, off, L + 1] = 16 * fine
        self.at = blk * 16 + off
        self.scale, self.sc = None, None
        if kind == "bf16":
            self.cache = x.to(torch.bfloat16)
        elif token:
            self.sc = 2.0 ** torch.randint(-3, 0, (nb, 16), generator=g).float()
            self.cache = (x / self.sc[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            self.scale = 0.125
            self.cache = (x / self.scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

    def zero(self, keys):
        """Rows of zeros, as the write stores them: scale 0."""
        for k in keys:
            self.cache.view(-1, self.L + 64)[self.at[k]] = 0
            if self.sc is not None:
                self.sc.view(-1)[self.at[k]] = 0

    def queries(self, H, S=1):
        q = torch.zeros(1, S, H, self.L + 64)
        q[..., self.L] = 1.0
        q[..., self.L + 1] = torch.linspace(0.0625, 0.0, H)   # heads differ in the last binade
        return q.to(torch.bfloat16)

    def call(self, q, lens=None, bt=None, **kw):
        lens = [self.n] if lens is None else lens
        return fk.latent_decode_attn(
            q.cuda(), self.cache.cuda(), (self.bt if bt is None else bt).cuda(),
            torch.tensor(lens, dtype=torch.int32, device="cuda"), latent_dim=self.L,
            kv_dtype=fk.KV_BF16 if self.kind == "bf16" else fk.KV_E4M3,
            scale_mode=fk.SCALE_PER_TOKEN_HEAD if self.token else fk.SCALE_PER_TENSOR,
            scale=None if self.scale is None else torch.tensor([self.scale], device="cuda"),
            scale_cache=None if self.sc is None else self.sc.cuda(), softmax_scale=LN2, **kw)

    def exact(self, q, skip=()):
        """(out, bound of the library's error) of S 1 queries in 64 bits."""
        rows = latent_values(self.cache, self.kind == "e4m3", self.scale, self.sc)
        keep = torch.ones(self.n, dtype=torch.bool)
        for b in skip:
            keep &= self.at // 16 != b
        t = torch.arange(self.n)[keep]
        x = rows[self.at[keep]]
        z = q[0, 0].double() @ x.T * LN2
        p = torch.softmax(z, -1)
        s = torch.full((len(t),), 1.0, dtype=torch.float64) if self.sc is None else \
            self.sc.view(-1).double()[self.at[keep]].clamp_min(2.0 ** -100)
        c = x[:, :self.L]
        out = p @ c
        mags = p @ c.abs()
        if self.kind == "bf16":
            # two bf16 terms: 2^-16 of a weight
            err = p * 2.0 ** -16
        else:
            w = p * s
            most = torch.zeros(w.shape[0], int(t[-1]) // 128 + 1, dtype=torch.float64)
            most.scatter_reduce_(1, (t // 128).expand(w.shape[0], -1), w, "amax")
            err = w * (2.0 ** -8 + 2.0 ** -11) + most[:, t // 128] * 2.0 ** -15
            err = (err + w.amax(-1, keepdim=True) * 2.0 ** -54) / s
        # a logit: fp32 products and sums of values up to |z|, the exponential's 2^-22;
        # the products' fp32 sums, a step of 16 keys at a time (2^-23 if it cuts off)
        dz = 2.0 ** -21 * float((q[0, 0].double().abs() @ x.abs().T).max()) + 2.0 ** -20
        return out, err @ c.abs() + (2 * dz + self.n / 16 * 2.0 ** -23) * mags + 1e-300


def check(rows, got, q, skip=()):
    want, bound = rows.exact(q, skip)
    got = got[0, 0].cpu().double()
    off = (got - want).abs()
    assert bool((off <= bound).all()), (
        f"worst ratio to its bound {float((off / bound).max()):.3g}, mass "
        f"{float((got[:, 0] / want[:, 0]).min()):.4f} to {float((got[:, 0] / want[:, 0]).max()):.4f}")
    # what a caller needs of it: the mass of the softmax is there
    assert float((got[:, 0] / want[:, 0] - 1).abs().max()) < 2.0 ** -8


def far_below(n, token, seed=3):
    """One strong key, then keys 14 binades below it that hold most of the mass."""
    g = torch.Generator().manual_seed(seed)
    z = 10.0 + torch.rand(n, generator=g)
    z[0] = 24.0
    return z


DEEP = ["logits", "zeros", "pages"]


@pytest.mark.parametrize("H", [1, 16, 64])
@pytest.mark.parametrize("token", [False, True])
@pytest.mark.parametrize("deep", DEEP)
def test_keys_behind_a_tile_far_below_keep_their_weight(deep, token, H):
    # a strong key, a whole tile of keys that weigh nothing (far lower logits, rows of
    # zeros, pages outside the cache), then thousands of ordinary keys
    n = 200 * 128
    z = far_below(n, token)
    if deep == "logits":
        z[128:256] = -46.0                           # 70 binades under the first key
    rows = Rows(z, token=token, seed=1)
    skip = ()
    bt = rows.bt
    if deep == "zeros":
        rows.zero(range(128, 256))
    if deep == "pages":
        bt = rows.bt.clone()
        skip = tuple(int(b) for b in bt[0, 8:16])
        bt[0, 8:16] = rows.cache.shape[0] + 9
    q = rows.queries(H)
    check(rows, rows.call(q, bt=bt, num_splits=1), q, skip)


@pytest.mark.parametrize("H", [1, 16, 64])
@pytest.mark.parametrize("token", [False, True])
@pytest.mark.parametrize("peak,weak", [(-5.0, -13.0), (0.0, -8.25), (-2.0, -10.5), (-9.0, -14.0)])
def test_many_weak_keys_beside_a_strong_one_in_every_tile(peak, weak, token, H):
    # a tile's largest key `peak` binades from the row's first, the other 127 at `weak`
    n = 150 * 128
    g = torch.Generator().manual_seed(5)
    z = weak + 0.5 * torch.rand(n, generator=g)
    z[5::128] = peak
    z[0] = 0.0
    rows = Rows(z, token=token, seed=2)
    q = rows.queries(H)
    check(rows, rows.call(q, num_splits=1), q)


@pytest.mark.parametrize("H", [16, 32, 64])
@pytest.mark.parametrize("token", [False, True])
@pytest.mark.parametrize("shape", ["flat", "steps down", "steps up", "sawtooth"])
def test_slopes_and_steps(shape, token, H):
    # references that have to follow in either direction, and back
    n = 61 * 128 + 77
    t = torch.arange(n)
    g = torch.Generator().manual_seed(6)
    z = {"flat": torch.zeros(n), "steps down": -(t // 128).float(),
         "steps up": (t // 128).float() * 0.5 - 20,
         "sawtooth": -8.0 * (t // 128 % 4).float()}[shape] + torch.rand(n, generator=g) * 0.75
    rows = Rows(z, token=token, seed=4)
    q = rows.queries(H)
    check(rows, rows.call(q, num_splits=1), q)
    check(rows, rows.call(q), q)


@pytest.mark.parametrize("H", [1, 16, 32, 64, 128])
def test_bf16_weights_hold_sixteen_bits(H):
    # fp32 output, ordinary logits: the two bf16 terms of a weight are the whole error
    n = 1000
    z = torch.randn(n, generator=torch.Generator().manual_seed(7)) * 2.5
    rows = Rows(z, kind="bf16", seed=8)
    q = rows.queries(H)
    for splits in (1, 0):
        check(rows, rows.call(q, num_splits=splits), q)


@pytest.mark.parametrize("token", [False, True])
def test_scales_far_from_one(token):
    # rows 2^40 times smaller and larger than ordinary ones
    for k in (-40, 40):
        z = far_below(40 * 128, token)
        z[128:256] = -46.0
        rows = Rows(z, token=token, seed=9)
        if token:
            rows.sc *= 2.0 ** k
        else:
            rows.scale *= 2.0 ** k
        q = rows.queries(16)
        q = (q.float() * 2.0 ** -k).to(torch.bfloat16)
        check(rows, rows.call(q, num_splits=1), q)


@pytest.mark.parametrize("k,token", [(-88, True), (-64, True), (64, True), (90, True),
                                     (-110, False), (-64, False), (64, False), (90, False)])
@pytest.mark.parametrize("splits", [1, 0])
def test_scales_near_the_ends_of_their_range(k, token, splits):
    # the row sums hold weights divided by the scales, here times 2^88, with a reference
    # far under the strong key's
    z = far_below(60 * 128, token)
    z[128:256] = -46.0
    rows = Rows(z, token=token, seed=10)
    if token:
        rows.sc *= 2.0 ** k
    else:
        rows.scale *= 2.0 ** k
    q = (rows.queries(16).float() * 2.0 ** -k).to(torch.bfloat16)
    want, _ = rows.exact(q)
    got = rows.call(q, num_splits=splits)[0, 0].cpu().double()
    assert bool(torch.isfinite(got).all())
    assert float((got[:, 0] / want[:, 0] - 1).abs().max()) < 2.0 ** -8
    assert float(((got - want).norm(dim=1) / want.norm(dim=1)).max()) < 2.0 ** -8


@pytest.mark.parametrize("splits", [1, 2, 0])
def test_zero_rows_in_front_of_far_lower_keys(splits):
    # rows of zeros (logit 0), keys 150 binades below them, then ordinary keys
    n = 64 * 128
    z = torch.full((n,), -150.0) + torch.rand(n, generator=torch.Generator().manual_seed(11))
    z[n // 2 + 300:] = 1.0
    rows = Rows(z * 0.25, token=True, seed=12)       # values that the codes hold ...
    rows.zero(range(0, 128))
    q = (rows.queries(16).float() * 4).to(torch.bfloat16)     # ... times 4
    want, _ = rows.exact(q)
    got = rows.call(q, num_splits=splits)[0, 0].cpu().double()
    assert bool(torch.isfinite(got).all())
    assert float((got - want).norm(dim=1).max() / want.norm(dim=1).max()) < 2.0 ** -8
