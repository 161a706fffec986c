"""FP8 rows of any code with MX-FP4 weights: inputs, bound, and what a single matrix instruction would
cut (no tests here).

A row's values lie in one or two of its 128-value blocks, all others are zero codes, so that the bound
does not grow with K and a cut shows in any tile.  Bound: a block's products are whole and go through
two instructions, each off by at most 2^-20 of its largest term (none above the sum M of the block's
magnitudes); multiplying by the row's scale and adding rounds to 2^-24, once a block.  Two blocks:
2 (2^-20 + 2^-24) M of each, blocks of zeros add nothing: 2^-19 (1 + 2^-4) of the sum of magnitudes.

The cut: among eight neighbours each product loses, towards zero, what is below 2^(E-13), E the largest sum
of two codes' exponents."""
import numpy as np
import torch

import more_reference as mref

BOUND = 2.0 ** -19 * (1 + 2.0 ** -4)

# one of each tile of FP8 rows: (16 x 64, K in four), 16 x 64, 64 x 128, 128 x 256 twice
CASES = [dict(tokens=12, experts=2, k=4096, f=128), dict(tokens=90, experts=16, k=1536, f=136),
         dict(tokens=400, experts=16, k=1536, f=520), dict(tokens=900, experts=2, k=256, f=4096),
         dict(tokens=700, experts=1, k=1920, f=8192)]


def tile(tokens, experts, k, f):
    """The tile that these sizes are given (top 1: a row a token)."""
    used = min(tokens, experts)

    def tiles(bi, bj):
        return (tokens + used * (bi - 1)) // bi * -(-f // bj)

    if k >= 2048 and tiles(16, 64) <= 512:
        return "16x64, K in four"
    rows = -(-tokens // used)
    if rows <= 12:
        return "16x64"
    return "128x256" if rows > 80 and tiles(128, 256) >= 128 else "64x128"


def inputs(c, rows):
    """(x, x_scales, w, w_scales) on the CPU; `rows` of the packed buffer."""
    g = torch.Generator().manual_seed(c["k"] + c["f"])

    def whole(low, high, *shape):
        return torch.randint(low, high, shape, generator=g, dtype=torch.int32).to(torch.uint8)

    k, f = c["k"], c["f"]
    x = whole(0, 256, rows, k)
    x = torch.where((x & 0x7F) == 0x7F, torch.zeros_like(x), x)
    blocks = k // 128
    kept = torch.zeros(rows, blocks, dtype=torch.bool)
    for _ in range(2):
        kept[torch.arange(rows), torch.randint(0, blocks, (rows,), generator=g)] = True
    x = torch.where(kept.repeat_interleave(128, 1), x, torch.zeros_like(x))
    xs = 0.5 + torch.rand(rows, blocks, generator=g)
    return x, xs, whole(0, 256, c["experts"], f, k // 2), whole(110, 118, c["experts"], f, k // 32)


def cut_error(x, xs, w, w_scales):
    """What single instructions would lose of row x [K] times weights w [n][K/2], and the sum of
    magnitudes, in 64 bits."""
    v = x.view(torch.float8_e4m3fn).float().double().numpy()
    u = mref.E2M1[np.stack([w & 15, w >> 4], -1).reshape(len(w), -1)]
    scale = np.repeat(np.exp2(w_scales.astype(np.float64) - 127), 32, 1) * np.repeat(xs.double().numpy(), 128)

    def exponent(a, least):
        with np.errstate(divide="ignore"):
            return np.where(a == 0, -99, np.maximum(np.floor(np.log2(np.abs(a))), least))

    p = v * u
    e = (exponent(v, -6)[None] + exponent(u, 0)).reshape(len(w), -1, 8).max(-1)
    unit = np.repeat(np.exp2(e - 13), 8, 1)
    cut = np.trunc(p / unit) * unit
    return np.abs(((p - cut) * scale).sum(1)), np.abs(p * scale).sum(1)
