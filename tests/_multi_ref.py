"""Plain references of the many-tensor AdamW and its 8-bit states, on the CPU.

``adamw64`` is the update in binary64.  The 8-bit form is written out twice:
``encode_ref`` works on binary32 bit patterns (what the header documents, bit
for bit), ``nearest64`` searches the table of all code values in binary64."""
import math

import numpy as np
import torch

M32 = 0xFFFFFFFF
E4M3 = dict(dtype=torch.float8_e4m3fn, top=8, cut=20, floor=0.0)
E5M2 = dict(dtype=torch.float8_e5m2, top=15, cut=21, floor=2.0 ** -16)


def adamw64(p, m, v, g, *, lr, eps, wd, beta1, beta2, t, clip=1.0, scale=1.0):
    """(p, m, v, |update|, sum of |terms| of m) after step t, all binary64 tensors."""
    p, m, v, g = (x.double() for x in (p, m, v, g))
    g = g / scale * clip
    mag = (beta1 * m).abs() + ((1 - beta1) * g).abs()
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    den = v.sqrt() / math.sqrt(1 - beta2 ** t) + eps
    upd = lr / (1 - beta1 ** t) * m / den
    return p * (1 - lr * wd) - upd, m, v, upd.abs(), lr / (1 - beta1 ** t) * mag / den, mag


def mix(x):
    x = x & M32
    x ^= x >> 16
    x = (x * 0x9E3779B1) & M32
    x ^= x >> 15
    x = (x * 0xBB67AE85) & M32
    return x ^ (x >> 16)


def random_ints(n, seed, t, tensor):
    """(below 2^20 for m, below 2^21 for v) of the n elements of a tensor."""
    q = np.arange((n + 7) // 8, dtype=np.uint64)
    x = (np.uint64(mix((mix((seed ^ mix(t)) & M32) + tensor) & M32)) + q * np.uint64(0x9E3779B1)) & np.uint64(M32)
    x ^= x >> np.uint64(16)
    x = (x * np.uint64(0x9E3779B1)) & np.uint64(M32)
    x ^= x >> np.uint64(15)
    x = (x * np.uint64(0xBB67AE85)) & np.uint64(M32)
    x ^= x >> np.uint64(16)
    rm, rv = [], []
    for _ in range(8):
        x = (x * np.uint64(1664525) + np.uint64(1013904223)) & np.uint64(M32)
        rm.append(x >> np.uint64(12))
        x = (x * np.uint64(1664525) + np.uint64(1013904223)) & np.uint64(M32)
        rv.append(x >> np.uint64(11))
    f = lambda r: torch.from_numpy(np.stack(r, 1).reshape(-1)[:n].astype(np.int32))  # noqa: E731
    return f(rm), f(rv)


def encode_ref(x, kind, rnd=None):
    """(codes, scale bytes) of the fp32 tensor x; rnd: stochastic rounding's integers, or None (nearest)."""
    n = x.numel()
    nb = -(-n // 32)
    pad = torch.zeros(nb * 32, dtype=torch.float32)
    pad[:n] = x
    b = pad.view(nb, 32)
    top = b.abs().amax(1) if nb else torch.zeros(0)
    top = torch.where(torch.isnan(b).any(1), torch.full_like(top, math.nan), top) if nb else top
    byte = (((top.view(torch.int32) + 0x1FFFFF) >> 23).clamp(max=254) - kind["top"]).clamp(min=1)
    bad = ~torch.isfinite(top)
    byte = torch.where(bad, torch.full_like(byte, 255), byte)
    inv = torch.where(bad, torch.ones_like(byte), (254 - byte) << 23).view(torch.float32)
    y = b * inv[:, None]
    z = y
    if rnd is not None:
        r = torch.zeros(nb * 32, dtype=torch.int32)
        r[:n] = rnd
        z = ((y.view(torch.int32) + r.view(nb, 32)) & -(1 << kind["cut"])).view(torch.float32)
    if kind["floor"]:
        z = torch.where(y > 0, z.clamp(min=kind["floor"]), z)
    most = 1.75 * 2.0 ** kind["top"]
    z = z.clamp(min=-most, max=most)
    z = torch.where(bad[:, None], torch.full_like(z, math.nan), z)
    return z.to(kind["dtype"]).reshape(-1)[:n], byte.to(torch.uint8)


def decode_ref(codes, byte):
    """fp32 values."""
    n = codes.numel()
    s = torch.where(byte == 0, torch.full_like(byte, 64, dtype=torch.int32) << 16, byte.to(torch.int32) << 23).view(torch.float32)
    return codes.float() * s.repeat_interleave(32)[:n]


def code_table(kind):
    """All finite non-negative code values of the type, ascending, in binary64."""
    v = torch.arange(128, dtype=torch.uint8).view(kind["dtype"]).double()
    return v[torch.isfinite(v)].numpy()


def nearest64(x, kind):
    """Values that x (binary64 numpy) is stored as with nearest rounding, by search."""
    table = code_table(kind)
    out = np.zeros_like(x)
    for a in range(0, len(x), 32):
        b = x[a:a + 32]
        top = np.abs(b).max()
        e = -126
        while top > table[-1] * 2.0 ** e:       # the smallest power of two that holds the largest magnitude
            e += 1
        y = np.abs(b) / 2.0 ** e
        i = np.clip(np.searchsorted(table, y), 1, len(table) - 1)
        lo, hi = table[i - 1], table[i]
        up = (y - lo > hi - y) | ((y - lo == hi - y) & (i % 2 == 0))     # ties: the even code
        q = np.where(up, hi, lo)
        if kind["floor"]:
            q = np.where(y > 0, np.maximum(q, kind["floor"]), q)
        out[a:a + 32] = np.sign(b) * q * 2.0 ** e
    return out
