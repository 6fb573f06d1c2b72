"""Plain 64-bit implementations that the rotary, cache-read and latent tests compare
with, and the bounds their results are held to.  Written from the definitions, with no
code of the library."""
import math

import torch

# half a step of a rounding, relative to the value (e4m3: also half of its smallest
# step, 2^-10, absolute)
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
E4M3_HALF, E4M3_TINY = 2.0 ** -4, 2.0 ** -10


def table(theta):
    """The library's frequency table from angles per position (radians, floats)."""
    return torch.tensor([int(round(t / (2 * math.pi) * 2.0 ** 64)) for t in theta],
                        dtype=torch.int64)


def thetas(rd, base=10000.0):
    return [base ** (-2.0 * i / rd) for i in range(rd // 2)]


def rotate(x, positions, theta, interleaved, mscale=1.0):
    """x [T][H][D] in 64 bits with its first 2 len(theta) values turned."""
    x = x.double().clone()
    rd = 2 * len(theta)
    ang = positions.double()[:, None] * torch.tensor(theta, dtype=torch.float64)[None]
    c, s = mscale * torch.cos(ang)[:, None], mscale * torch.sin(ang)[:, None]
    if interleaved:
        a, b = x[..., 0:rd:2].clone(), x[..., 1:rd:2].clone()
        x[..., 0:rd:2], x[..., 1:rd:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rd // 2].clone(), x[..., rd // 2:rd].clone()
        x[..., :rd // 2], x[..., rd // 2:rd] = a * c - b * s, b * c + a * s
    return x


def codes_to_values(codes):
    return codes.view(torch.float8_e4m3fn).double()


def assert_close(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = err > bound
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} values off, worst error "
        f"{float(err.max()):.3e}, worst ratio to its bound "
        f"{float((err / bound.clamp_min(1e-300)).max()):.3f}")


def latent_values(cache, e4m3, scale=None, scale_cache=None):
    """The cache's rows in 64 bits, [num_blocks * 16][W]."""
    x = (codes_to_values(cache) if e4m3 else cache.double()).flatten(0, 1)
    if e4m3:
        x = x * (scale_cache.double().reshape(-1, 1) if scale_cache is not None
                 else float(scale))
    return x


def latent_attention(q, rows, block_table, context_lens, L, softmax_scale, e4m3, scales=None,
                     skip=()):
    """(out, bound of the library's error) in 64 bits.  q [B][S][H][W]; rows
    [num_blocks * 16][W]; scales [num_blocks * 16] (per token) or None; skip: block ids
    whose keys do not exist.

    The bound, for out = sum w_t c_t / sum w_t (c_t the row's latent values, s_t its
    scale): a weight of a code is rounded to f16 (2^-11) and then to two e4m3 terms (half
    a step of the second: 2^-8 of the weight, or 2^-10 absolute in units where the largest
    weight of its tile of 128 keys is at least 2^-2, i.e. 2^-8 of that one; 2^-60 of a
    row's largest where a tile lies that far below) or to bf16 (2^-8); a logit is off by
    fp32 sums of the products and, for e4m3, by what two terms of q miss (2^-17 of the
    row's largest value).
    """
    B, S, H, W = q.shape
    out = torch.zeros(B, S, H, L, dtype=torch.float64)
    bound = torch.zeros_like(out)
    for b in range(B):
        ctx = max(0, min(int(context_lens[b]), block_table.shape[1] * 16))
        for s in range(S):
            n = ctx - S + s + 1
            if n <= 0:
                continue
            t = torch.arange(n)
            blocks = block_table[b].long()[t // 16]
            keep = torch.ones(n, dtype=torch.bool)
            for bad in skip:
                keep &= blocks != bad
            t, blocks = t[keep], blocks[keep]
            if t.numel() == 0:
                continue
            at = blocks * 16 + t % 16
            x = rows[at]
            qs = q[b, s].double()
            z = (qs @ x.T) * softmax_scale
            p = torch.softmax(z, -1)
            c = x[:, :L]
            out[b, s] = p @ c
            mags = p @ c.abs()
            dz = 2.0 ** -18 * float(((qs.abs() @ x.abs().T) * softmax_scale).max()) + 2.0 ** -20
            if e4m3:
                dz += 2.0 ** -17 * float(qs.abs().max()) * float(x.abs().sum(-1).max()) * softmax_scale
                sc = torch.ones(t.numel(), dtype=torch.float64) if scales is None else \
                    scales.double()[at].clamp_min(2.0 ** -100)
                w = p * sc                                  # weights of the codes
                code = c / sc[:, None]
                most = torch.zeros(H, int(t[-1]) // 128 + 1, dtype=torch.float64)
                most.scatter_reduce_(1, (t // 128).expand(H, -1), w, "amax")
                err = torch.maximum(w * (2.0 ** -8 + 2.0 ** -11), most[:, t // 128] * 2.0 ** -8)
                err += w.amax(-1, keepdim=True) * 2.0 ** -60
                bound[b, s] = err @ code.abs()
            else:
                bound[b, s] = mags * 2.0 ** -8
            bound[b, s] += 2 * dz * mags + 2.0 ** -20 * mags
    return out, bound
