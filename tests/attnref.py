"""Plain 64-bit implementations of the softmax-attention operators, written
from their formulas, and the error bounds the kernels' arithmetic allows."""
import math

import torch

# half a step relative to the value
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def table(rot, length, base=10000.0):
    """cos, sin rows (FP32) of the angles pos * base^(-2i/rot)."""
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = torch.arange(length, dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def norm_rotate(x, norm, eps, w, rot, adjacent, cs, pos):
    """x [T, H, D] (float64) -> (norm and rotation, the magnitude that bounds
    each channel's rounding errors)."""
    x = x.double()
    if norm:
        m = (x * x).sum(-1, keepdim=True)
        x = x / torch.sqrt((m / x.shape[-1] if norm == 2 else m) + eps)
    if w is not None:
        x = x * w.double()
    y, mag = x.clone(), x.abs()
    if rot:
        c = cs[pos, :rot // 2].double()[:, None]
        s = cs[pos, rot // 2:].double()[:, None]
        lo = slice(0, rot, 2) if adjacent else slice(0, rot // 2)
        hi = slice(1, rot, 2) if adjacent else slice(rot // 2, rot)
        a, b = x[..., lo], x[..., hi]
        y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
        mag[..., lo] = mag[..., hi] = a.abs() + b.abs()
    return y, mag


def rows_bound(y, mag, dtype):
    """One rounding to the io type; in FP32 before it the sum of squares (up
    to 8 + 5 additions and a product per lane: 16 steps), square root,
    reciprocal and four products and a sum per channel: 24 half steps of the
    channel pair's magnitude."""
    return HALF[dtype] * y.abs() + 24 * 2.0 ** -24 * mag + 1e-30


def attend(q, K, V, mask, scale, softcap):
    """q [R, D], K, V [L, D], mask [R, L] (all float64): (o, sum p|v| / sum p,
    bound on the FP32 error of a row's scores)."""
    s = q @ K.T * scale
    mag = (q.abs() @ K.abs().T) * abs(scale)
    s = s if softcap == 0 else softcap * torch.tanh(s / softcap)
    s = s.masked_fill(~mask, -math.inf)
    p = torch.softmax(s, -1)
    mag = mag.masked_fill(~mask, 0.0).amax(-1, keepdim=True)
    return p @ V, p @ V.abs(), mag


def attend_bound(o, av, mag, D, keys, dtype, softcap, split):
    """|o' - o| of a kernel that sums scores over D products in FP32 (error at
    most (D + 4) 2^-24 of the products' magnitude; a cap adds 8 steps of the
    cap), takes 2^x to 2^-21, rounds each weight to `split` relative, and sums
    `keys` weighted values and weights in FP32 (statistically sqrt, here a
    bound of keys / 16 + 64 half steps, as partial sums of 16 are joined), then
    rounds once.  An error e of every score moves the output by at most
    2 e sum p|v| / sum p."""
    e = (D + 4) * 2.0 ** -24 * mag + (8 * softcap * 2.0 ** -24)
    rel = 2 * e + 2.0 ** -20 + 2 * split + 2 * (keys / 16 + 64) * 2.0 ** -24
    return HALF[dtype] * o.abs() + rel * av + 1e-30


def paged(pages, ids, page, n):
    """The first n tokens, [Hkv, n, D] float64, of the pages ids."""
    g = pages[ids.long()].double()  # [W, H, P, D]
    return g.transpose(0, 1).reshape(g.shape[1], -1, g.shape[3])[:, :n]
