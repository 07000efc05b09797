"""Cases that measure the operators on a paged KV pool: kv_rotate, kv_append with kv_fetch, kv_attend.

A case names one pass through one operator.  ``run`` computes it either in its
plain form (elementary torch operations in 32 bits, rounded once) or, where
``own`` is true, with the calls of include/kvb.h that a serving program makes
for it.  Pools are uint8 tensors in one of the four pool layouts.

A 4-bit head vector of D values is D/2 bytes of codes (value i in bits
4*(i%8).. of 32-bit word i/8), D/32 scale words, and zeros up to a multiple of
16 bytes.  A scale word is a float32 whose low four mantissa bits hold the zero
point z of its 32 values: value = (code - z) * s, s = float(word with those
bits 0).  With lo and hi the least and the largest of 0 and the 32 values, s is
hi * (1/15) - lo * (1/15) in float32, rounded to 20 significant bits;
z = round(-lo / s) and code = round(x / s) + z, kept in 0..15, are quotients
rounded exactly, ties to even.  A group with a value that is not finite is held
as NaN, one with s under 2^-100 as zeros.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
GROUP = 32


# ------------------------------------------------------------------- cases

def listed():
    """The calls of a serving program that keeps its KV pages in a pool of this framework."""
    return [
        # One token of one request before its attention: the smallest call, all latency.
        dict(name="rotate one token", kind="rotate", dtype="bf16", tokens=1, heads=40, head_dim=128,
             rot_dim=128, style="half", scaling="none", factor=1.0, far=4096, inverse=False),
        # A long prompt chunk at far positions, frequencies scaled for a long context.
        dict(name="rotate long prompt", kind="rotate", dtype="bf16", tokens=8192, heads=40,
             head_dim=128, rot_dim=128, style="half", scaling="yarn", factor=16.0, far=1000000,
             inverse=False),
        # Interleaved pairs on part of the head, an odd token count, turned back.
        dict(name="rotate part back", kind="rotate", dtype="fp16", tokens=1537, heads=16,
             head_dim=192, rot_dim=64, style="interleaved", scaling="bands", factor=8.0, far=131072,
             inverse=True),
        # A decode batch: one new token of each request into a 4-bit page-first HND pool.
        dict(name="append decode 4-bit", kind="append", dtype="bf16", format="q4", tokens=64,
             q_heads=32, heads=8, head_dim=128, rot_dim=128, style="half", page_tokens=32,
             page_first=True, hnd=True, far=131072),
        # A prompt chunk into a 4-bit layer-first NHD pool.
        dict(name="append prompt 4-bit", kind="append", dtype="bf16", format="q4", tokens=8192,
             q_heads=32, heads=8, head_dim=128, rot_dim=128, style="half", page_tokens=16,
             page_first=False, hnd=False, far=131072),
        # The same pages in 16 bits, at an odd token count.
        dict(name="append prompt 16-bit", kind="append", dtype="fp16", format="same", tokens=2049,
             q_heads=24, heads=6, head_dim=64, rot_dim=32, style="interleaved", page_tokens=16,
             page_first=False, hnd=False, far=8192),
        # 8-bit pages of 256 tokens.
        dict(name="append prompt 8-bit", kind="append", dtype="bf16", format="e4m3", tokens=5000,
             q_heads=16, heads=2, head_dim=256, rot_dim=128, style="half", page_tokens=256,
             page_first=False, hnd=True, far=32768),
        # One short request: the smallest attention call, all latency.
        dict(name="attend one short", kind="attend", dtype="bf16", requests=1, q_len=1, max_len=150,
             q_heads=32, heads=8, head_dim=128, page_tokens=16, page_first=False, hnd=False, window=0),
        # One request with a long cache: all the parallelism lies along the tokens.
        dict(name="attend one long", kind="attend", dtype="bf16", requests=1, q_len=1,
             max_len=131072, q_heads=32, heads=8, head_dim=128, page_tokens=32, page_first=True,
             hnd=True, window=0),
        # A decode batch of ragged lengths.
        dict(name="attend decode batch", kind="attend", dtype="bf16", requests=64, q_len=1,
             max_len=8192, q_heads=32, heads=8, head_dim=128, page_tokens=16, page_first=False,
             hnd=False, window=0),
        # A few drafted tokens of each request, checked at once, inside a sliding window.
        dict(name="attend drafts", kind="attend", dtype="fp16", requests=24, q_len=5, max_len=4500,
             q_heads=12, heads=4, head_dim=64, page_tokens=64, page_first=True, hnd=False,
             window=2000),
        # A prompt chunk behind a restored prefix.
        dict(name="attend prompt chunk", kind="attend", dtype="bf16", requests=2, q_len=1000,
             max_len=8192, q_heads=32, heads=8, head_dim=128, page_tokens=16, page_first=False,
             hnd=False, window=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the ranges above."""
    kind = rng.choice(("rotate", "append", "attend", "attend"))
    dtype = rng.choice(("bf16", "fp16"))
    style = rng.choice(("half", "interleaved"))
    page = dict(page_tokens=rng.choice((1, 16, 17, 32, 64, 256)), page_first=rng.random() < 0.5,
                hnd=rng.random() < 0.5)
    if kind == "rotate":
        dim = rng.choice((64, 96, 128, 192, 256))
        return dict(kind=kind, dtype=dtype, tokens=_log(rng, 1, 8192), heads=rng.randint(1, 40),
                    head_dim=dim, rot_dim=rng.choice((dim, dim // 2, 32)), style=style,
                    scaling=rng.choice(("none", "linear", "ntk", "yarn", "bands")),
                    factor=rng.choice((2.0, 8.0, 32.0)), far=_log(rng, 100, 4000000),
                    inverse=rng.random() < 0.3)
    heads = rng.choice((1, 2, 3, 4, 8, 10))
    if kind == "append":
        dim = rng.choice((64, 96, 128, 256))
        return dict(kind=kind, dtype=dtype, format=rng.choice(("q4", "q4", "same", "e4m3")),
                    tokens=_log(rng, 1, 8192), q_heads=heads * rng.randint(1, 4), heads=heads,
                    head_dim=dim, rot_dim=rng.choice((dim, dim // 2, 32)), style=style,
                    far=_log(rng, 100, 1000000), **page)
    dim = rng.choice((64, 96, 128, 128, 256))
    group, window = rng.choice((1, 2, 4, 5, 8)), rng.choice((0, 0, 0, _log(rng, 16, 8192)))
    q_len = rng.choice((1, 1, 1, rng.randint(2, 8), _log(rng, 9, 700)))
    cap = min(2 ** 28 // (heads * dim), 2 ** 35 // (heads * group * dim * q_len))  # tokens of all requests: cached values, products
    longest = _log(rng, max(q_len, 20), min(60000, cap))
    most = min(48, cap // longest)
    return dict(kind=kind, dtype=dtype, requests=rng.randint(1, most), q_len=q_len, max_len=longest,
                q_heads=heads * group, heads=heads, head_dim=dim, window=window, **page)


# -------------------------------------------------------- what a case is made of

def _frequencies(c):
    """Radians per position of each pair (float64, CPU) and the factor on cos and sin."""
    r = c["rot_dim"]
    base, scaling, factor = 10000.0, c.get("scaling", "none"), c.get("factor", 1.0)
    i = torch.arange(r // 2, dtype=torch.float64)
    if scaling == "ntk":
        base = base * factor ** (r / (r - 2))
    f = base ** (-2.0 * i / r)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        at = lambda turns: r * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(at(32.0))), min(r - 1, math.ceil(at(1.0)))
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    if scaling == "bands":
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return f / factor * (1 - keep) + f * keep, 1.0
    return f, 1.0


def _rows(c, positions):
    """[tokens, 2, rot_dim / 2] float32: the cosines, then the sines, of every pair's angle."""
    f, m = _frequencies(c)
    a = positions.double()[:, None] * f.to(positions.device)
    return torch.stack((torch.cos(a) * m, torch.sin(a) * m), 1).float()


def _shape(c):
    """(pages, head vector bytes) of a case's pool."""
    d = c["head_dim"]
    b = {"same": 2 * d, "e4m3": d, "q4": -(-(d // 2 + d // 8) // 16) * 16}[c.get("format", "q4")]
    t = c["page_tokens"]
    if c["kind"] == "append":
        return -(-c["tokens"] // t) + 3, b
    return c["requests"] * -(-c["max_len"] // t) + 3, b


LAYERS, LAYER = 2, 1


def _view(c, pool, comp):
    """One layer and component of the pool as [pages, page_tokens, heads, bytes]."""
    pages, b = _shape(c)
    t, h = c["page_tokens"], c["heads"]
    inner = (h, t, b) if c["hnd"] else (t, h, b)
    x = pool.view(pages, LAYERS, 2, *inner)[:, LAYER, comp] if c["page_first"] else pool.view(LAYERS, 2, pages, *inner)[LAYER, comp]
    return x.transpose(1, 2) if c["hnd"] else x


def _quantised(x):
    """Float32 vectors [..., D] as 4-bit head vectors [..., bytes]."""
    d = x.shape[-1]
    g = x.reshape(*x.shape[:-1], d // GROUP, GROUP)
    ok = torch.isfinite(g).all(-1)
    g = torch.where(ok[..., None], g, torch.zeros_like(g))
    lo, hi = g.amin(-1).clamp(max=0.0), g.amax(-1).clamp(min=0.0)
    s = hi * (1.0 / 15.0) - lo * (1.0 / 15.0)
    bits = (s.view(torch.int32) + 8) & -16
    bits = torch.where(bits.view(torch.float32) < 2.0 ** -100, torch.zeros_like(bits), bits)
    s = bits.view(torch.float32)
    by = torch.where(s > 0, s, torch.ones_like(s)).double()  # 16-bit inputs meet ties of x / s: divided in 64 bits
    z = torch.round(-lo.double() / by).clamp(0, 15)
    code = (torch.round(g.double() / by[..., None]) + z[..., None]).clamp(0, 15)
    live = ok & (s > 0)
    code = torch.where(live[..., None], code, torch.zeros_like(code)).to(torch.uint8).reshape(*x.shape[:-1], d // 2, 2)
    word = torch.where(ok, torch.where(s > 0, bits | z.to(torch.int32), torch.zeros_like(bits)), torch.full_like(bits, 0x7FC00000))
    out = torch.zeros(*x.shape[:-1], -(-(d // 2 + d // 8) // 16) * 16, dtype=torch.uint8, device=x.device)
    out[..., : d // 2] = code[..., 0] | (code[..., 1] << 4)
    out[..., d // 2 : d // 2 + d // 8] = word.contiguous().view(torch.uint8)
    return out


def _values(raw, d):
    """4-bit head vectors [..., bytes] as float32 values [..., D]."""
    code = torch.stack((raw[..., : d // 2] & 15, raw[..., : d // 2] >> 4), -1).reshape(*raw.shape[:-1], d // GROUP, GROUP)
    word = raw[..., d // 2 : d // 2 + d // 8].contiguous().view(torch.int32)
    z, s = (word & 15).float(), (word & -16).view(torch.float32)
    return ((code.float() - z[..., None]) * s[..., None]).reshape(*raw.shape[:-1], d)


class _Handles:
    """The framework's handles of one state, closed with it."""

    def __init__(self, kvb):
        self.kvb, self.pool, self.rotary = kvb, None, None

    def __del__(self):
        if self.pool is not None:
            self.kvb.kv_pool_close(self.pool)
        if self.rotary is not None:
            self.kvb.kv_rotary_close(self.rotary)


def _own(c, s):
    """What a program keeps for the framework's calls: handles and argument blocks over its buffers."""
    from hierarchical_kv_cache_backup_gb300 import kvb

    h = s["handles"] = _Handles(kvb)
    dt = {"bf16": kvb.KV_BF16, "fp16": kvb.KV_FP16}[c["dtype"]]
    if c["kind"] != "attend":
        sc = {"none": kvb.KV_ROTARY_PLAIN, "linear": kvb.KV_ROTARY_LINEAR, "ntk": kvb.KV_ROTARY_NTK,
              "yarn": kvb.KV_ROTARY_YARN, "bands": kvb.KV_ROTARY_BANDS}[c.get("scaling", "none")]
        slow, fast = (1.0, 32.0) if sc == kvb.KV_ROTARY_YARN else (1.0, 4.0)
        h.rotary = kvb.kv_rotary_create(c["rot_dim"], kvb.KV_ROTARY_HALF if c["style"] == "half" else kvb.KV_ROTARY_INTERLEAVED,
                                        base=10000.0, scaling=sc, factor=c.get("factor", 1.0), original_len=4096, slow=slow, fast=fast)
    if c["kind"] == "rotate":
        s["args"] = kvb.make_rotate_args(kvb.vecs(s["x"]), kvb.vecs(s["out"]), tokens=c["tokens"], heads=c["heads"], head_dim=c["head_dim"], dtype=dt,
                                         inverse=c["inverse"], positions=s["positions"].data_ptr(), rows_out=s["rows"].data_ptr())
        return
    pages, b = _shape(c)
    lay = kvb.make_layout(LAYERS, 2, pages, c["page_tokens"], c["heads"], b, kvb.KV_PAGE_FIRST if c["page_first"] else kvb.KV_LAYER_FIRST,
                          kvb.KV_HND if c["hnd"] else kvb.KV_NHD, {"same": 2, "e4m3": 1}.get(c.get("format"), 1))
    h.pool = kvb.kv_pool_register(lay, s["pool"].data_ptr())
    if c["kind"] == "append":
        fmt = {"same": kvb.KV_CACHE_SAME, "e4m3": kvb.KV_CACHE_E4M3, "q4": kvb.KV_CACHE_Q4}[c["format"]]
        s["args"] = kvb.make_append_args(kvb.vecs(s["k"]), kvb.vecs(s["v"]), kvb.vecs(s["q"]), kvb.vecs(s["q_out"]), tokens=c["tokens"],
                                         q_heads=c["q_heads"], head_dim=c["head_dim"], dtype=dt, format=fmt, layer=LAYER, k_scale=s["k_scale"],
                                         v_scale=s["v_scale"], rows=s["rows"].data_ptr(), slots=s["slots"].data_ptr(), status=s["status"].data_ptr())
        s["back"] = kvb.make_fetch_args(kvb.vecs(s["k_out"]), kvb.vecs(s["v_out"]), tokens=c["tokens"], head_dim=c["head_dim"], dtype=dt, format=fmt,
                                        layer=LAYER, k_scale=s["k_scale"], v_scale=s["v_scale"], slots=s["slots"].data_ptr(), status=s["status"].data_ptr())
        return
    s["args"] = kvb.make_attend_args(kvb.vecs(s["q"]), kvb.vecs(s["out"]), lse=s["lse"].data_ptr(), q_start=s["q_start"].data_ptr(),
                                     lens=s["lens"].data_ptr(), pages=s["table"].data_ptr(), pages_stride=s["table"].stride(0),
                                     requests=c["requests"], tokens=s["q"].shape[0], max_q=c["q_len"], max_len=c["max_len"], q_heads=c["q_heads"],
                                     head_dim=c["head_dim"], dtype=dt, layer=LAYER, window=c["window"], scale=s["scale"], status=s["status"].data_ptr())
    need = kvb.kv_attend_workspace(h.pool, s["args"])
    s["workspace"] = torch.zeros(max(1, need), dtype=torch.uint8, device="cuda")
    s["args"].workspace, s["args"].workspace_bytes = s["workspace"].data_ptr(), need


def prepare(case, seed):
    """The inputs of one pass, from the seed, and the buffers and handles that a program keeps."""
    c, s = case, {"case": case}
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, d = DTYPES[c["dtype"]], c["head_dim"]
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    whole = lambda hi, *shape: torch.randint(0, hi, shape, generator=g, device="cuda")  # noqa: E731
    stale = lambda n: torch.randint(0, 256, (n,), generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    if c["kind"] == "rotate":
        t, h = c["tokens"], c["heads"]
        s["x"] = normal(t, h + 4, d).to(dt)[:, :h]       # query and key heads of a fused projection
        s["positions"] = whole(c["far"], 1) + torch.arange(t, device="cuda")
        s["out"] = torch.empty(t, h, d, dtype=dt, device="cuda")
        s["rows"] = torch.empty(t, 2, c["rot_dim"] // 2, device="cuda")
    elif c["kind"] == "append":
        t, h, hq, pt = c["tokens"], c["heads"], c["q_heads"], c["page_tokens"]
        pages, b = _shape(c)
        x = normal(t, hq + 2 * h, d)
        x[:, hq : hq + h] = x[:, hq : hq + h] * torch.exp(0.7 * normal(h, d)) + 0.5 * normal(h, d)  # keys have louder and offset channels
        x = x.to(dt)
        s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq : hq + h], x[:, hq + h :]
        s["rows"] = _rows(c, whole(c["far"], t))
        order = torch.randperm(pages, generator=g, device="cuda")[: -(-t // pt)]
        s["slots"] = (order[:, None] * pt + torch.arange(pt, device="cuda")).reshape(-1)[:t].contiguous()
        s["pool"] = stale(LAYERS * 2 * pages * pt * h * b)
        s["k_scale"], s["v_scale"] = 0.0625, 0.03125
        s["q_out"] = torch.empty(t, hq, d, dtype=dt, device="cuda")
        s["k_out"], s["v_out"] = torch.empty(2, t, h, d, dtype=dt, device="cuda").unbind(0)
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    else:
        r, h, hq, pt, ql = c["requests"], c["heads"], c["q_heads"], c["page_tokens"], c["q_len"]
        pages, b = _shape(c)
        per = -(-c["max_len"] // pt)
        low = max(ql, c["max_len"] // 2)
        lens = low + whole(c["max_len"] - low + 1, r)
        lens[0] = c["max_len"]
        n_q = torch.tensor([ql - 5 * i % ql for i in range(r)], device="cuda")  # ragged new tokens
        s["lens"], s["q_len"] = lens.int(), n_q
        s["q_start"] = torch.cat((torch.zeros(1, device="cuda", dtype=torch.long), n_q.cumsum(0))).int()
        s["table"] = torch.randperm(pages, generator=g, device="cuda")[: r * per].view(r, per).int()
        s["q"] = normal(int(s["q_start"][-1]), hq, d).to(dt)
        s["pool"] = stale(LAYERS * 2 * pages * pt * h * b)  # what is past a request's length is stale
        for comp in (0, 1):
            for i in range(r):
                n = int(lens[i])
                x = normal(n, h, d)
                if comp == 0:
                    x = x * torch.exp(0.5 * normal(h, d)) + 0.5 * normal(h, d)
                at = torch.arange(n, device="cuda")
                _view(c, s["pool"], comp)[s["table"][i].long()[at // pt], at % pt] = _quantised(x)
        s["scale"] = 1.0 / math.sqrt(d)
        s["out"] = torch.empty(s["q"].shape, dtype=dt, device="cuda")
        s["lse"] = torch.empty(s["q"].shape[0], hq, device="cuda")
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own:
        _own(c, s)
    return s


# ----------------------------------------------------------------- one pass

def _rotated(c, x, rows, inverse=False):
    """Float32 vectors [tokens, heads, D], their first rot_dim values turned by the rows."""
    r = c["rot_dim"]
    cos, sin = rows[:, 0, None], rows[:, 1, None]
    if inverse:
        sin = -sin
    if c["style"] == "half":
        a, b = x[..., : r // 2], x[..., r // 2 : r]
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
    u, v = a * cos - b * sin, a * sin + b * cos
    y = torch.cat((u, v), -1) if c["style"] == "half" else torch.stack((u, v), -1).flatten(-2)
    return torch.cat((y, x[..., r:]), -1)


def _plain_rotate(c, s):
    rows = _rows(c, s["positions"])
    return {"out": _rotated(c, s["x"].float(), rows, c["inverse"]).to(s["x"].dtype), "rows": rows}


def _plain_append(c, s):
    dt, d, pt = s["k"].dtype, c["head_dim"], c["page_tokens"]
    k, v = _rotated(c, s["k"].float(), s["rows"]), s["v"].float()
    page, at = s["slots"] // pt, s["slots"] % pt
    q = _rotated(c, s["q"].float(), s["rows"]).to(dt)
    back = []
    for comp, x, scale in ((0, k, s["k_scale"]), (1, v, s["v_scale"])):
        view = _view(c, s["pool"], comp)
        if c["format"] == "same":
            view[page, at] = x.to(dt).contiguous().view(torch.uint8)
            back.append(view[page, at].view(dt))
        elif c["format"] == "e4m3":
            view[page, at] = (x * (1.0 / scale)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            back.append((view[page, at].view(torch.float8_e4m3fn).float() * scale).to(dt))
        else:
            view[page, at] = _quantised(x)
            back.append(_values(view[page, at], d).to(dt))
    return {"q": q, "k": back[0], "v": back[1]}


def _plain_attend(c, s):
    r, h, d, ql, n = c["requests"], c["heads"], c["head_dim"], c["q_len"], c["max_len"]
    g = c["q_heads"] // h
    at = torch.arange(ql, device="cuda")
    real = at < s["q_len"][:, None]                                             # [r, ql]
    row = (s["q_start"][:-1, None] + at).clamp(max=s["q"].shape[0] - 1).long()
    q = s["q"].float()[row].view(r, ql, h, g, d)
    k, v = (_values(_view(c, s["pool"], comp)[s["table"].long()].flatten(1, 2)[:, :n], d) for comp in (0, 1))
    tok = torch.arange(n, device="cuda")
    pos = (s["lens"][:, None] - s["q_len"][:, None] + at)[:, :, None]           # the place of each new token
    seen = (tok <= pos) & (tok < s["lens"][:, None, None])
    if c["window"]:
        seen &= tok > pos - c["window"]
    v = v.masked_fill((tok >= s["lens"][:, None])[:, :, None, None], 0.0)
    q, k, v = (x.permute(0, 2, 1, 3).contiguous() for x in (q.flatten(3, 4).view(r, ql, h, g * d), k, v))
    q = q.view(r, h, ql * g, d)
    seen = seen[:, None, :, None].expand(r, 1, ql, g, n).reshape(r, 1, ql * g, n)
    x = (q @ k.transpose(2, 3) * s["scale"]).masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total)).view(r, h, ql, g).permute(0, 2, 1, 3).reshape(r, ql, h * g)
    o = o.view(r, h, ql, g, d).permute(0, 2, 1, 3, 4).reshape(r, ql, h * g, d)
    return {"out": o[real].to(s["q"].dtype), "lse": lse[real]}


def run(state):
    """One pass."""
    s, c = state, state["case"]
    if not own:
        return {"rotate": _plain_rotate, "append": _plain_append, "attend": _plain_attend}[c["kind"]](c, s)
    h = s["handles"]
    if c["kind"] == "rotate":
        h.kvb.kv_rotate(h.rotary, s["args"])
        return {"out": s["out"], "rows": s["rows"]}
    if c["kind"] == "append":
        h.kvb.kv_append(h.pool, h.rotary, s["args"])
        h.kvb.kv_fetch(h.pool, s["back"])
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    h.kvb.kv_attend(h.pool, s["args"])
    return {"out": s["out"], "lse": s["lse"]}


def work(case):
    """Bytes (each input read once, each output written once) and operations of one pass."""
    c = case
    d = c["head_dim"]
    if c["kind"] == "rotate":
        n = c["tokens"] * c["heads"]
        return {"bytes": 4 * n * d + c["tokens"] * (8 + 4 * c["rot_dim"]), "flops": 3 * n * c["rot_dim"]}
    pages, b = _shape(c)
    if c["kind"] == "append":
        t, h, hq = c["tokens"], c["heads"], c["q_heads"]
        return {"bytes": t * (4 * hq * d + 4 * h * d + 2 * h * b + 4 * c["rot_dim"] + 8) + t * (2 * h * b + 4 * h * d + 8),
                "flops": t * (3 * (hq + h) * c["rot_dim"] + 6 * 2 * h * d)}
    # lengths lie evenly between half the longest and the longest
    r, n, ql, w = c["requests"], c["max_len"], c["q_len"], c["window"]
    length, new = (n + (r - 1) * (max(ql, n // 2) + n) / 2) / r, sum(ql - 5 * i % ql for i in range(r)) / r
    sees = min(length - (new - 1) / 2, w or length)
    reads = min(length, w + new - 1) if w else length
    return {"bytes": r * (reads * c["heads"] * 2 * b + new * c["q_heads"] * (4 * d + 4) + 4 * reads / c["page_tokens"]),
            "flops": 4 * r * new * sees * c["q_heads"] * d}


# ------------------------------------------------------------- in 64 bits

def _turned(c, x, a, m, inverse):
    """Vectors in 64 bits as complex numbers, multiplied by m * exp(i a)."""
    r, y = c["rot_dim"], x.clone()
    one, two = (slice(0, r // 2), slice(r // 2, r)) if c["style"] == "half" else (slice(0, r, 2), slice(1, r, 2))
    w = torch.complex(x[..., one].contiguous(), x[..., two].contiguous()) * torch.polar(torch.full_like(a, m), -a if inverse else a)[:, None]
    y[..., one], y[..., two] = w.real, w.imag
    return y


def _held(c, x, scale):
    """What the pool's format keeps of values in 64 bits."""
    if c["format"] == "same":
        return x
    if c["format"] == "e4m3":
        y = (x / scale).clamp(-448, 448)
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        return torch.round(y / step) * step * scale
    y = x.unflatten(-1, (-1, GROUP))
    lo, hi = y.amin(-1, keepdim=True).clamp(max=0), y.amax(-1, keepdim=True).clamp(min=0)
    part = hi.float() * (1 / 15) - lo.float() * (1 / 15)     # the format's step is a float32 of 20 bits by definition
    mant, exp = torch.frexp(part.double())
    s = torch.ldexp(torch.floor(mant * 2 ** 20 + 0.5), exp - 20)
    z = torch.round(-lo / s)
    return ((torch.round(y / s) + z).clamp(0, 15) - z).mul(s).flatten(-2)


def exact(case, seed):
    """The same outputs in 64 bits, from the definitions."""
    c, s = case, prepare(case, seed)
    if c["kind"] == "rotate":
        f, m = _frequencies(c)
        a = s["positions"].double()[:, None] * f.cuda()
        return {"out": _turned(c, s["x"].double(), a, m, c["inverse"]), "rows": torch.stack((a.cos(), a.sin()), 1) * m}
    if c["kind"] == "append":
        row = s["rows"].double()
        a = torch.atan2(row[:, 1], row[:, 0])
        turned = lambda x: _turned(c, x.double(), a, 1.0, False)  # noqa: E731
        return {"q": turned(s["q"]), "k": _held(c, turned(s["k"]), s["k_scale"]), "v": _held(c, s["v"].double(), s["v_scale"])}
    h, d, pt, g = c["heads"], c["head_dim"], c["page_tokens"], c["q_heads"] // c["heads"]
    shift = 4 * torch.arange(8, device="cuda")
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    for i in range(c["requests"]):
        a, e, n = int(s["q_start"][i]), int(s["q_start"][i + 1]), int(s["lens"][i])
        at = torch.arange(n, device="cuda")
        pos = torch.arange(n - (e - a), n, device="cuda")[:, None]
        hide = at > pos
        if c["window"]:
            hide = hide | (at <= pos - c["window"])
        both = []
        for comp in (0, 1):
            raw = _view(c, s["pool"], comp)[s["table"][i].long()[at // pt], at % pt].contiguous().view(torch.int32)
            code = (raw[..., : d // 8, None] >> shift) & 15
            word = raw[..., d // 8 : d // 8 + d // 32]
            step = (word - (word & 15)).view(torch.float32).double()
            both.append((code.reshape(n, h, d // 32, 32) - (word & 15)[..., None]).double().mul(step[..., None]).reshape(n, h, d))
        for j in range(c["q_heads"]):
            x = torch.mm(s["q"][a:e, j].double(), both[0][:, j // g].T).mul(s["scale"]).masked_fill(hide, -math.inf)
            lse[a:e, j] = torch.logsumexp(x, 1)
            out[a:e, j] = torch.mm(torch.softmax(x, 1), both[1][:, j // g])
    return {"out": out, "lse": lse}
