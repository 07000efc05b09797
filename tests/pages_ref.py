"""Plain implementations in 64 bits of attention over 16-bit and fp8 pages, bounds of pages and
selection, and the batches that the tests run them on.  Nothing here uses the library's kernels."""
from __future__ import annotations

import numpy as np
import torch

from vec_ref import half_step, pool_view

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def e4m3(raw: np.ndarray) -> np.ndarray:
    """uint8 codes as float64."""
    return torch.from_numpy(np.ascontiguousarray(raw)).view(torch.float8_e4m3fn).double().numpy()


# ------------------------------------------------------------------ attention

def softmax_rows(q, k, v, seen, scale):
    """q [n, D], k and v [m, D], seen [n, m], in 64 bits: out, lse, weights, scores."""
    with np.errstate(all="ignore"):
        x = np.where(seen, scale * (q @ k.T), -np.inf)
        some = seen.any(1)
        top = np.where(some, x.max(1, initial=-np.inf), 0.0)[:, None]
        p = np.where(seen, np.exp(x - top), 0.0)
        total = p.sum(1, keepdims=True)
        w = p / np.where(some[:, None], total, 1.0)
        lse = np.where(some, top[:, 0] + np.log(np.where(some, total[:, 0], 1.0)), -np.inf)
        out = np.einsum("nm,md->nd", w, np.where(seen.any(0)[:, None], v, 0.0))
    return out, lse, w, x


def tolerance(q, k, v, w, x, want, scale, dt, fp8, many):
    """Bounds on the roundings of one head's rows (out [n, D], lse [n]):

    * a score: float32 sums of exact products, at most D / 16 + 16 of them cut at 2^-23 of sum |q k| (2^-18
      in all); a bf16 query against fp8 keys 2^-38 of its largest |q| times |k|; and the exponential,
      2^-21 of 1 + |x| + |largest x|;
    * a weight, in two parts 2^-17 (bf16) or 2^-21 (fp16) of itself, in one half a step of its type, and
      2^-31 of the largest in fp16 (2^-25 with the largest at 2^7 or more);
    * the sums: each of m / 16 + 16 additions is cut at 2^-23 of sum |w v|;
    * the output: half a step."""
    m = k.shape[0]
    av = np.abs(np.where((w > 0).any(0)[:, None], v, 0.0))
    xs = np.where(w > 0, np.abs(np.where(np.isfinite(x), x, 0.0)), 0.0)
    dx = 2.0 ** -18 * abs(scale) * (np.abs(q) @ np.abs(k).T) + 2.0 ** -21 * (1 + xs + xs.max(1, keepdims=True, initial=0))
    bf = dt == torch.bfloat16
    if fp8 and bf:
        dx = dx + 2.0 ** -38 * abs(scale) * np.abs(q).max(1)[:, None] * np.abs(k).sum(1)[None]
    narrow = bf and not fp8                            # weights are bf16
    if many or (fp8 and bf):
        by = half_step(torch.bfloat16 if narrow else torch.float16)
    else:
        by = 2.0 ** -17 if narrow else 2.0 ** -21
    by_w = w @ av
    tol = half_step(dt) * np.abs(want) * (1 + 2 ** -7) + (by + 2.0 ** -23 * (m / 16 + 16)) * by_w
    tol = tol + (w * dx) @ av + (w * dx).sum(1, keepdims=True) * np.abs(want)
    if not narrow:
        tol = tol + 2.0 ** -31 * w.max(1, keepdims=True, initial=0) * ((w > 0) @ av)
    tol = tol + 2.0 ** -25 * (dt == torch.float16) + 2.0 ** -130
    return tol, (w * dx).sum(1) + 2.0 ** -20 + 2.0 ** -24 * m / 16


# --------------------------------------------------------------------- bounds

def step_of(m: np.ndarray) -> np.ndarray:
    """The least power of two s with m <= 127 s; 0 below 2^-100, infinity for what is not finite."""
    with np.errstate(all="ignore"):
        mant, exp = np.frexp(m / 127.0)
        s = np.ldexp(1.0, exp - (mant == 0.5))
        return np.where(np.isfinite(m), np.where(m < 2.0 ** -100, 0.0, s), np.inf)


def bounds_of(x: np.ndarray):
    """Keys [tokens, H, D] of one page in float64: codes of lo and hi [H, D] and steps [H, D / 32]."""
    h, d = x.shape[1:]
    lo, hi = x.min(0), x.max(0)
    m = np.abs(x).max(0).reshape(h, d // 32, 32).max(2)
    m = np.where(np.isfinite(x).all(0).reshape(h, d // 32, 32).all(2), m, np.inf)
    s = step_of(m)
    by = np.repeat(np.where((s > 0) & np.isfinite(s), s, np.inf), 32, 1)
    with np.errstate(all="ignore"):
        a, b = np.floor(lo / by), np.ceil(hi / by)
    live = np.isfinite(by)
    return np.where(live, a, 0).astype(np.int8), np.where(live, b, 0).astype(np.int8), s.astype(np.float32)


def record_bytes(d: int) -> int:
    return -(-(2 * d + d // 8) // 16) * 16


def record(lo, hi, s) -> np.ndarray:
    h, d = lo.shape
    out = np.zeros((h, record_bytes(d)), np.uint8)
    out[:, :d], out[:, d:2 * d] = lo.view(np.uint8), hi.view(np.uint8)
    out[:, 2 * d:2 * d + d // 8] = np.ascontiguousarray(s, "<f4").view(np.uint8).reshape(h, d // 8)
    return out


def parts(rec: np.ndarray, d: int):
    lead = rec.shape[:-1]
    c = np.ascontiguousarray
    return (c(rec[..., :d]).view(np.int8), c(rec[..., d:2 * d]).view(np.int8),
            c(rec[..., 2 * d:2 * d + d // 8]).view("<f4").reshape(*lead, d // 32))


def scores(q: np.ndarray, lo, hi, s) -> np.ndarray:
    """Query heads [group, D] (float64 of 16-bit values) against records [pages, D ...]: float32 [pages]."""
    g, d = q.shape
    q = q.reshape(g, d // 32, 32)
    t = step_of(np.where(np.isfinite(q).all(2), np.abs(q).max(2), np.inf))
    with np.errstate(all="ignore"):
        c = np.where(((t > 0) & np.isfinite(t))[..., None], np.rint(q / np.where(t > 0, t, 1.0)[..., None]), 0.0)
        a, b = lo.reshape(-1, d // 32, 32).astype(np.float64), hi.reshape(-1, d // 32, 32).astype(np.float64)
        dot = np.einsum("gik,pik->gpi", np.maximum(c, 0), b) + np.einsum("gik,pik->gpi", np.minimum(c, 0), a)
        w = s.astype(np.float32)[None] * t.astype(np.float32)[:, None]
        term = dot.astype(np.float32) * w
        total = term[..., 0]
        for i in range(1, d // 32):
            total = total + term[..., i]
        most = np.float32(np.finfo(np.float32).max)
        return np.where(np.isfinite(total), total, most).max(0)


def select(score: np.ndarray, budget, keep_first, keep_last) -> list:
    """The indices picked of pages with these scores, ascending, filled up with -1."""
    n = len(score)
    if n <= budget:
        return list(range(n)) + [-1] * (budget - n)
    kept = [j for j in range(n) if j < keep_first or j >= n - keep_last]
    rest = sorted((j for j in range(n) if keep_first <= j < n - keep_last), key=lambda j: (-score[j], j))
    return sorted(kept + rest[:budget - len(kept)])


# -------------------------------------------------------------------- batches

class Pages:
    """A pool of 16-bit or fp8 pages, its bytes random (stale) until something is put there."""

    def __init__(self, kvb, dim, fmt, dtype, T, H, P, L=2, page_first=False, hnd=False, offset=0, seed=0, device="cuda"):
        self.kvb, self.dim, self.fmt, self.T, self.H, self.P, self.L = kvb, dim, fmt, T, H, P, L
        self.page_first, self.hnd, self.offset = page_first, hnd, offset
        self.dt = DT[dtype]
        self.dtype = kvb.KV_BF16 if dtype == "bf16" else kvb.KV_FP16
        self.format = kvb.KV_CACHE_E4M3 if fmt == "e4m3" else kvb.KV_CACHE_SAME
        self.k_scale, self.v_scale = (0.0625, 0.03125) if fmt == "e4m3" else (1.0, 1.0)
        self.B = dim * (1 if fmt == "e4m3" else 2)
        self.bytes = L * 2 * P * T * H * self.B
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.alloc = torch.randint(0, 256, (offset + self.bytes,), generator=g, device="cuda", dtype=torch.uint8)
        lay = kvb.make_layout(L, 2, P, T, H, self.B, kvb.KV_PAGE_FIRST if page_first else kvb.KV_LAYER_FIRST,
                              kvb.KV_HND if hnd else kvb.KV_NHD, 1 if fmt == "e4m3" else 2)
        self.pool = kvb.kv_pool_register(lay, self.alloc.data_ptr(), offset)

    def view(self, comp, layer=1):
        return pool_view(self.alloc[self.offset:], self.L, self.P, self.T, self.H, self.B, layer % self.L, comp, self.page_first, self.hnd)

    def words(self, x):
        """Float values [..., D] on the GPU as the pool holds them, uint8 [..., B]."""
        x = x.clamp(-448, 448).to(torch.float8_e4m3fn) if self.fmt == "e4m3" else x.to(self.dt)
        return x.contiguous().view(torch.uint8).view(*x.shape[:-1], self.B)

    def put(self, table, x, comp, layer=1):
        """Values [tokens, H, D] (fp8: before the scale) to a row of a page table."""
        at = torch.arange(x.shape[0], device="cuda")
        self.view(comp, layer)[table.long()[at // self.T], at % self.T] = self.words(x)

    def held(self, table, n, comp, layer=1):
        """The first n tokens of a row of a page table in float64, scale included."""
        at = torch.arange(n, device="cuda")
        raw = self.view(comp, layer)[table.long()[at // self.T], at % self.T].contiguous()
        x = raw.view(torch.float8_e4m3fn) if self.fmt == "e4m3" else raw.view(self.dt)
        return x.double().cpu().numpy().reshape(n, self.H, self.dim) * (self.v_scale if comp else self.k_scale)

    def close(self):
        self.kvb.kv_pool_close(self.pool)


class Batch:
    """Requests with new tokens n_q and own lengths lens; groups: (first request, end, prefix length)."""

    def __init__(self, kvb, lens, n_q, groups=(), H=2, group=4, dim=128, fmt="same", dtype="bf16", T=16, seed=1, spare=3, loud=1.0, **page):
        self.kvb, self.lens, self.n_q, self.groups, self.H, self.group, self.dim = kvb, lens, n_q, list(groups), H, group, dim
        self.per, self.pre = max(1, -(-max(lens, default=0) // T)), max(1, -(-max([g[2] for g in groups], default=0) // T))
        P = len(lens) * self.per + len(self.groups) * self.pre + spare
        self.p = p = Pages(kvb, dim, fmt, dtype, T, H, P, seed=seed, **page)
        g = self.gen = torch.Generator(device="cuda")
        g.manual_seed(seed)
        order = torch.randperm(P, generator=g, device="cuda").int()
        self.table = order[:len(lens) * self.per].view(len(lens), self.per).contiguous()
        at = len(lens) * self.per
        self.prefix_table = order[at:at + len(self.groups) * self.pre].view(len(self.groups), self.pre).contiguous()
        normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        for row, n in [(self.table[i], n) for i, n in enumerate(lens)] + [(self.prefix_table[i], x[2]) for i, x in enumerate(self.groups)]:
            for comp in (0, 1):
                x = normal(n, H, dim) * (loud if comp == 0 else 1.0)
                p.put(row, x * (1.0 / (p.v_scale if comp else p.k_scale)), comp)
        self.tokens = sum(n_q)
        self.q = normal(max(1, self.tokens), H * group, dim).to(p.dt)
        self.out = torch.full_like(self.q, 7.0)
        self.lse = torch.full((max(1, self.tokens), H * group), 7.0, device="cuda")
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.q_start = i32([0] + list(np.cumsum(n_q)))
        self.d_lens = i32(lens)
        self.group_start = i32([x[0] for x in self.groups] + [self.groups[-1][1]] if self.groups else [0])
        self.prefix_lens = i32([x[2] for x in self.groups] or [0])
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.scale = dim ** -0.5
        self.works = []

    def __enter__(self):
        return self

    def __exit__(self, *a):
        torch.cuda.synchronize()
        self.p.close()
        for work, behind in self.works:                    # not a byte past the workspace
            assert torch.equal(work[work.numel() - 4096:], behind)

    def common(self, q=None, out=None):
        kvb, p = self.kvb, self.p
        q = self.q[:self.tokens] if q is None else q
        out = self.out[:self.tokens] if out is None else out
        return kvb.vecs(q), kvb.vecs(out), dict(
            lse=self.lse.data_ptr(), q_start=self.q_start.data_ptr(), lens=self.d_lens.data_ptr(), pages=self.table.data_ptr(),
            pages_stride=self.per, requests=len(self.lens), tokens=self.tokens, max_q=max(self.n_q, default=0), max_len=max(self.lens, default=0),
            q_heads=self.H * self.group, head_dim=self.dim, dtype=p.dtype, format=p.format, layer=1 % p.L, scale=self.scale,
            k_scale=p.k_scale, v_scale=p.v_scale, status=self.status.data_ptr())

    def space(self, a, need):
        work = torch.randint(0, 256, (need + 4096,), device="cuda", dtype=torch.uint8)   # whatever it held before
        self.works.append((work, work[need:].clone()))
        a.workspace, a.workspace_bytes = work.data_ptr(), need
        return a

    def max_group(self):
        at = np.cumsum([0] + list(self.n_q))
        return int(max([at[b] - at[a] for a, b, _ in self.groups], default=0))

    def shared_args(self, q=None, out=None, **kw):
        a, b, c = self.common(q, out)
        if self.groups:
            c.update(groups=len(self.groups), group_start=self.group_start.data_ptr(), prefix_lens=self.prefix_lens.data_ptr(),
                     prefix_pages=self.prefix_table.data_ptr(), prefix_stride=self.pre, max_group=self.max_group(),
                     max_prefix=max(x[2] for x in self.groups))
        c.update(kw)
        args = self.kvb.make_attend_shared_args(a, b, **c)
        return self.space(args, self.kvb.kv_attend_shared_workspace(self.p.pool, args))

    def selected_args(self, picks, q=None, out=None, **kw):
        a, b, c = self.common(q, out)
        c.update(picks=picks.data_ptr(), budget=picks.shape[2])
        c.update(kw)
        args = self.kvb.make_attend_selected_args(a, b, **c)
        return self.space(args, self.kvb.kv_attend_selected_workspace(self.p.pool, args))

    def run(self, stream=None, **kw):
        self.kvb.kv_attend_shared(self.p.pool, self.shared_args(**kw), stream)
        torch.cuda.synchronize()
        return self.out[:self.tokens], self.lse[:self.tokens]

    def rows(self):
        """(request, first query token, queries, prefix length and table or None) of each request."""
        at = np.cumsum([0] + list(self.n_q))
        for i, n in enumerate(self.n_q):
            g = [(x[2], self.prefix_table[k]) for k, x in enumerate(self.groups) if x[0] <= i < x[1]]
            yield i, int(at[i]), n, g[0] if g else (0, None)

    def many(self):
        return self.max_group() * self.group > 16 or max(self.n_q, default=0) * self.group > 16

    def check(self, requests=None, out=None, lse=None, q=None, nan_ok=False):
        """Outputs and logarithms against 64 bits; returns the largest part of a tolerance used."""
        q = (self.q if q is None else q).double().cpu().numpy()
        out = (self.out if out is None else out).double().cpu().numpy()
        lse = (self.lse if lse is None else lse).double().cpu().numpy()
        worst = 0.0
        for i, a, n, (pre, table) in self.rows():
            if n == 0 or (requests is not None and i not in requests):
                continue
            own = self.lens[i]
            k, v = (np.concatenate(([self.p.held(table, pre, c)] if pre else []) + [self.p.held(self.table[i], own, c)]) for c in (0, 1))
            pos = own - n + np.arange(n)
            seen = np.concatenate((np.ones((n, pre), bool), np.arange(own)[None] <= pos[:, None]), 1)
            worst = max(worst, self.check_rows(q[a:a + n], k, v, np.repeat(seen[:, None], self.H, 1), out[a:a + n], lse[a:a + n], self.many()))
        return worst

    def check_rows(self, q, k, v, seen, out, lse, many):
        """q [n, heads, D] over k and v [m, H, D]; seen [n, H, m]."""
        worst = 0.0
        for j in range(self.H * self.group):
            h = j // self.group
            want, wl, w, x = softmax_rows(q[:, j], k[:, h], v[:, h], seen[:, h], self.scale)
            none = ~seen[:, h].any(1)
            assert not out[none, j].any() and np.all(np.isneginf(lse[none, j])), j
            if none.all():
                continue
            tol, tl = tolerance(q[:, j], k[:, h], v[:, h], w, x, want, self.scale, self.p.dt, self.p.fmt == "e4m3", many)
            err = np.abs(out[:, j] - want)
            ok = none[:, None] | (err <= tol)
            worst = max(worst, float((err / tol)[~none].max()))
            assert ok.all(), (j, np.argwhere(~ok)[:4].tolist(), worst)
            el = np.abs(lse[~none, j] - wl[~none])
            assert np.all(el <= (tl + 2.0 ** -21 * np.abs(np.where(none, 0, wl)))[~none]), (j, float(el.max()))
        return worst
