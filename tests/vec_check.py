"""A check of kv_attend whose tolerance follows each query's own weights: what a query does
not see, or gives no weight, leaves no room for error.  Plain numpy in 64 bits."""
from __future__ import annotations

import numpy as np
import torch

import vec_ref
from vec_ref import half_step


def attend(q, k, v, scale, window=0):
    """One request, one head, in 64 bits: out [n, D], lse [n], weights and scores [n, len]."""
    n, length = q.shape[0], k.shape[0]
    pos, t = length - n + np.arange(n)[:, None], np.arange(length)[None]
    seen = t <= pos
    if window:
        seen = seen & (t > pos - window)
    with np.errstate(all="ignore"):
        x = np.where(seen, scale * (q @ k.T), -np.inf)
        top = np.where(seen.any(1), x.max(1, initial=-np.inf), 0.0)[:, None]
        p = np.exp(x - top)
        total = p.sum(1, keepdims=True)
        w = p / np.where(total > 0, total, 1.0)
        lse = np.where(total[:, 0] > 0, top[:, 0] + np.log(total[:, 0]), -np.inf)
    return w @ v, lse, w, x


def check(b, out, lse=None, q=None, requests=None, many=None, key_parts=2):
    """Compares a batch's outputs (lse: None = not looked at) with 64 bits.  Roundings:

    * a score: float32 sums of exact products, 2^-20 of 24 times sum |q| x step (zero points
      cancel), and 2^-21 of 1 + |x| + |largest x| in the exponential.  With many rows a request
      (80 or more at heads of 128 or fewer) keys are fp16 too: 2^-11 of |q| |k|, 2^-18 in two
      parts; and queries, 2^-39 of the row's largest |q| x step, over D products of 15;
    * a weight (with its step) to fp16: 2^-11 of each |w v|, and as much again for the values
      with many rows; below fp16's normal range 2^-28 of the largest weight x step a token;
    * the sums: each of length / 16 additions is cut at 2^-23 of w x step x 15;
    * the output: half a step of its type."""
    q = (b.q if q is None else q).double().cpu().numpy()
    out = out.double().cpu().numpy()
    lse = None if lse is None else lse.double().cpu().numpy()
    if many is None:
        many = b.dim <= 128 and max(b.n_q) * b.group >= 80
    at, worst = 0, 0.0
    for i, n in enumerate(b.n_q):
        if (requests is None or i in requests) and n:
            length = b.lens[i]
            k, v = (vec_ref.q4_decode(x, b.dim) for x in b.kv[i])
            _, _, ks = vec_ref.q4_parts(b.kv[i][0], b.dim)
            _, _, vs = vec_ref.q4_parts(b.kv[i][1], b.dim)
            for j in range(b.H * b.group):
                h, qj, got = j // b.group, q[at:at + n, j], out[at:at + n, j]
                want, wl, w, x = attend(qj, k[:, h], v[:, h], b.scale, b.window)
                none = np.isneginf(wl)
                assert not got[none].any(), (i, j)
                if lse is not None:
                    assert np.all(np.isneginf(lse[at:at + n, j][none])), (i, j)
                if none.all():
                    continue
                size, av = abs(b.scale), np.abs(v[:, h])
                xs = np.where(w > 0, np.abs(np.where(np.isfinite(x), x, 0.0)), 0.0)
                dx = 2.0 ** -20 * 24 * size * (np.abs(qj) @ ks[:, h].T)
                dx = dx + 2.0 ** -21 * (1 + xs + xs.max(1, keepdims=True))
                if many:
                    dx = dx + (2.0 ** -18 if key_parts == 2 else 2.0 ** -11) * size * (np.abs(qj) @ np.abs(k[:, h]).T)
                    dx = dx + 2.0 ** -39 * 15 * b.dim * size * (np.abs(qj) * ks[:, h].max(0)).max(1)[:, None]
                by_w = w @ av
                tol = half_step(b.dt) * np.abs(want) * (1 + 2 ** -7) + 2.0 ** -10 * (1 if many else 0.55) * by_w
                tol = tol + (w * dx) @ av + (w * dx).sum(1, keepdims=True) * np.abs(want)
                ws = w[:, :, None] * vs[None, :, h, ::32]
                tol = tol + np.repeat(2.0 ** -23 * (length / 16 + 16) * 15 * ws.sum(1)
                                      + 2.0 ** -28 * 15 * length * ws.max(1), 32, -1)
                if many:
                    tol = tol + 2.0 ** -31 * w.max(1, keepdims=True) * ((w > 0) @ av)
                tol = tol + 2.0 ** -25 * (b.dt == torch.float16)
                err = np.abs(got - want)
                ok = none[:, None] | (err <= tol)
                worst = max(worst, float((err / np.maximum(tol, 1e-300))[~none].max()))
                assert ok.all(), (i, j, np.argwhere(~ok)[:4].tolist(), worst)
                if lse is not None:
                    el = np.abs(lse[at:at + n, j][~none] - wl[~none])
                    lim = ((w * dx).sum(1) + 2.0 ** -20 + 2.0 ** -21 * np.abs(np.where(none, 0, wl)))[~none]
                    assert np.all(el <= lim), (i, j, float((el / lim).max()))
        at += n
    return worst
