"""Plain implementations in 64 bits of the operators on head vectors, and the
pools the tests run them on.  Nothing here uses the library."""
from __future__ import annotations

import math

import numpy as np
import torch

GROUP = 32


# --------------------------------------------------------------- 4-bit format

def q4_bytes(dim: int) -> int:
    return (dim // 2 + dim // 8 + 15) // 16 * 16


def q4_encode(x: np.ndarray) -> np.ndarray:
    """float32 [..., D] -> uint8 [..., B], from the format's definition."""
    x = np.asarray(x, np.float32)
    d = x.shape[-1]
    g = x.reshape(-1, GROUP)
    ok = np.isfinite(g).all(1)
    g = np.where(ok[:, None], g, np.float32(0))
    lo, hi = np.minimum(g.min(1), np.float32(0)), np.maximum(g.max(1), np.float32(0))
    r15 = np.float32(1.0 / 15.0)
    s = (hi * r15 - lo * r15).astype(np.float32)
    bits = (s.view(np.uint32) + np.uint32(8)) & np.uint32(0xFFFFFFF0)
    bits = np.where(bits.view(np.float32) < np.float32(2.0 ** -100), np.uint32(0), bits)
    step = bits.view(np.float32).astype(np.float64)
    by = np.where(step > 0, step, 1.0)
    # the quotient in 64 bits decides every tie rightly: x has 24 bits and the step
    # 20, so x / step is never within 2^-53 of a half-way point without being on it
    z = np.clip(np.rint(-lo.astype(np.float64) / by), 0, 15)
    code = np.clip(np.rint(g.astype(np.float64) / by[:, None]) + z[:, None], 0, 15)
    live = ok & (step > 0)
    code = np.where(live[:, None], code, 0).astype(np.uint32)
    word = np.where(ok, np.where(live, bits | z.astype(np.uint32), np.uint32(0)),
                    np.uint32(0x7FC00000)).astype(np.uint32)
    n = x.size // d
    out = np.zeros((n, q4_bytes(d)), np.uint8)
    packed = (code.reshape(n, d // 8, 8) << (4 * np.arange(8, dtype=np.uint32))).sum(2, dtype=np.uint32)
    out[:, : d // 2] = packed.astype("<u4").view(np.uint8).reshape(n, d // 2)
    out[:, d // 2: d // 2 + d // 8] = word.astype("<u4").view(np.uint8).reshape(n, d // 8)
    return out.reshape(*x.shape[:-1], q4_bytes(d))


def q4_parts(raw: np.ndarray, dim: int):
    """uint8 [..., B] -> (codes, zero points, steps) as float64, each [..., D]."""
    lead = raw.shape[:-1]
    w = np.ascontiguousarray(raw[..., : dim // 2]).view("<u4").astype(np.uint32)
    code = (w[..., None] >> (4 * np.arange(8, dtype=np.uint32))) & 15
    word = np.ascontiguousarray(raw[..., dim // 2: dim // 2 + dim // 8]).view("<u4").astype(np.uint32)
    step = (word & np.uint32(0xFFFFFFF0)).view(np.float32).astype(np.float64)
    rep = lambda a: np.repeat(a, GROUP, -1)  # noqa: E731
    return code.reshape(*lead, dim).astype(np.float64), rep((word & 15).astype(np.float64)), rep(step)


def q4_decode(raw: np.ndarray, dim: int) -> np.ndarray:
    c, z, s = q4_parts(raw, dim)
    return (c - z) * s


# ----------------------------------------------------------------- rotation

def frequencies(rot: int, base=10000.0, scaling="plain", factor=1.0, original_len=0, slow=0.0, fast=0.0,
                gain=0.0):
    """(radians per position [rot/2] in float64, gain), from the formulas."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        at = lambda t: rot * math.log(original_len / (t * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(at(fast))), min(rot - 1, math.ceil(at(slow)))
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        f = f / factor * ramp + f * (1 - ramp)
        gain = gain or 0.1 * math.log(factor) + 1
    if scaling == "bands":
        k = np.clip((original_len * f / (2 * math.pi) - slow) / (fast - slow), 0, 1)
        f = f / factor * (1 - k) + f * k
    return f, gain or 1.0


def rows_of(freq, gain, positions) -> np.ndarray:
    """float64 [tokens, 2, R/2].  Positions times frequencies in extended precision, so that
    the angle keeps 2^-40 of a turn at positions of 2^40."""
    a = np.asarray(positions, np.longdouble)[:, None] * np.asarray(freq, np.longdouble)
    return np.stack((np.cos(a), np.sin(a)), 1).astype(np.float64) * gain


def turn(x: np.ndarray, rows: np.ndarray, style: str, inverse=False) -> np.ndarray:
    """[tokens, heads, D] turned, in the arithmetic of its type (float32: each product and sum
    rounded by itself)."""
    half = rows.shape[2]
    c, s = rows[:, 0, None].astype(x.dtype), rows[:, 1, None].astype(x.dtype)
    if inverse:
        s = -s
    y = x.copy()
    a_at, b_at = (slice(0, half), slice(half, 2 * half)) if style == "half" else \
        (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    a, b = x[..., a_at], x[..., b_at]
    y[..., a_at] = a * c - b * s
    y[..., b_at] = a * s + b * c
    return y


# -------------------------------------------------------------------- pools

def pool_view(raw, L, P, T, H, B, layer, comp, page_first, hnd):
    """[P, T, H, B] view of one layer and component of a C = 2 pool's bytes (numpy or torch)."""
    inner = (H, T, B) if hnd else (T, H, B)
    x = raw.reshape(P, L, 2, *inner)[:, layer, comp] if page_first else \
        raw.reshape(L, 2, P, *inner)[layer, comp]
    return (x.swapaxes(1, 2) if isinstance(x, np.ndarray) else x.transpose(1, 2)) if hnd else x


# ---------------------------------------------------------------- attention

def attend(q, k, v, scale, window=0):
    """One request in float64: q [n, Hq, D], k and v [len, H, D]; returns out, lse and the
    normalised weights [Hq, n, len]."""
    n, hq, d = q.shape
    length, h, _ = k.shape
    g = hq // h
    pos = length - n + np.arange(n)[:, None]
    t = np.arange(length)[None]
    seen = t <= pos
    if window:
        seen &= t > pos - window
    out, lse, ws = np.zeros((n, hq, d)), np.full((n, hq), -np.inf), np.zeros((hq, n, length))
    with np.errstate(all="ignore"):
        for j in range(hq):
            x = scale * (q[:, j] @ k[:, j // g].T)
            for i in range(n):
                at = seen[i]
                if not at.any():
                    continue
                top = x[i][at].max()
                p = np.exp(x[i][at] - top)
                ws[j, i, at] = p / p.sum()
                out[i, j] = (p / p.sum()) @ v[at, j // g]
                lse[i, j] = top + math.log(p.sum()) if np.isfinite(p.sum()) else np.nan
    return out, lse, ws


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2
