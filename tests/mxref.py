"""MXFP4 in numpy, in 64 bits, from the format's definition: the nearest of the
sixteen E2M1 values by distance, ties to the even code, one power-of-two scale
per 32 values (the smallest with max|x| <= 6 * 2^e).  Shares no code with the
library."""
import numpy as np
import torch

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def row_bytes(d):
    return -(-(d // 2 + d // 32) // 16) * 16


def quantise(x):
    """x [..., K] float64 (bf16 values) -> (codes [..., K] uint8, scale bytes
    [..., K/32] uint8)."""
    x = np.asarray(x, np.float64)
    blk = x.reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(blk).all(-1)
    blk = np.where(bad[..., None], 0.0, blk)
    amax = np.abs(blk).max(-1)
    e = np.full(amax.shape, -127.0)
    todo = amax > 0
    e[todo] = np.ceil(np.log2(amax[todo] / 6.0))
    e = np.where(todo & (amax > 6.0 * np.exp2(e)), e + 1, e)
    e = np.where(todo & (amax <= 6.0 * np.exp2(e - 1)), e - 1, e)
    e = np.maximum(e, -127.0)
    a = np.abs(blk) / np.exp2(e)[..., None]
    dist = np.abs(a[..., None] - GRID)
    near = dist == dist.min(-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    codes = (pick + 8 * np.signbit(blk)).astype(np.uint8)
    codes = np.where(bad[..., None], 0, codes).reshape(x.shape).astype(np.uint8)
    return codes, np.where(bad, 255, e + 127).astype(np.uint8)


def values(codes, scale):
    """fp64 values (NaN for a NaN block)."""
    c = codes.astype(np.int64)
    v = np.where(c >= 8, -1.0, 1.0) * GRID[c % 8]
    s = np.where(scale == 255, np.nan, np.exp2(scale.astype(np.float64) - 127))
    return (v.reshape(*v.shape[:-1], -1, 32) * s[..., None]).reshape(v.shape)


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(b):
    return np.stack((b & 15, b >> 4), axis=-1).reshape(*b.shape[:-1], -1)


def cache_rows(x, pad=0):
    """Rows x [..., d] -> cache rows [..., row_bytes(d)] (padding bytes `pad`)."""
    d = x.shape[-1]
    codes, scale = quantise(x)
    out = np.full((*x.shape[:-1], row_bytes(d)), pad, np.uint8)
    out[..., : d // 2] = pack(codes)
    out[..., d // 2: d // 2 + d // 32] = scale
    return out


def cache_values(rows, d):
    return values(unpack(rows[..., : d // 2]), rows[..., d // 2: d // 2 + d // 32])


def scale_tiles(scale):
    """Scale bytes [rows, K/32] -> the operand layout, tiles of 128 rows x 4
    blocks (512 bytes, rows padded with zeros)."""
    rows, nb = scale.shape
    out = np.zeros((-(-rows // 128), nb // 4, 512), np.uint8)
    for r in range(rows):
        for c in range(nb):
            out[r // 128, c // 4, r % 32 * 16 + r % 128 // 32 * 4 + c % 4] = scale[r, c]
    return out


def bf16_values(t):
    """bf16 tensor -> float64 array (NaN and infinities kept)."""
    return t.detach().float().cpu().numpy().astype(np.float64)


def hard_rows(n, d, seed):
    """bf16 rows over the whole range of the type: magnitudes from subnormal to
    the largest, blocks of zeros, rounding ties, negative zeros, NaN and
    infinities."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, d, generator=g)
    ex = torch.randint(-133, 126, (n, d // 32), generator=g).float()
    kind = torch.randint(0, 8, (n, d // 32), generator=g)
    x = x.view(n, -1, 32)
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    tie = ties[torch.randint(0, 8, x.shape, generator=g)] * (1 - 2 * (x < 0).float())
    x = torch.where((kind == 1)[..., None], tie, x)
    x = torch.where((kind == 2)[..., None], torch.zeros(()), x)
    x = torch.where((kind == 3)[..., None], -torch.zeros(()), x)
    wide = torch.where(kind[..., None] <= 1, torch.exp2(ex)[..., None], torch.ones(()))
    x = (x.double() * wide.double()).clamp(-3.3e38, 3.3e38).float()
    x[..., 5] = torch.where(kind == 4, torch.tensor(float("nan")), x[..., 5])
    x[..., 31] = torch.where(kind == 5, torch.tensor(float("inf")), x[..., 31])
    return x.reshape(n, d).bfloat16()
