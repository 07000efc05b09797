"""Cases that measure attention over shared prefixes and over selected pages of a paged KV pool.

Four operators of a serving step whose pages hold keys and values in 16 bits or in fp8 (e4m3):
kv_attend_shared (requests of a group share a long prefix, attended once for all of them), kv_bound
(bounds of the keys of each page), kv_select (the pages whose bounds promise a query most) and
kv_attend_selected (attention over those pages alone).  A case names one pass through one of them.
``run`` computes it either in its plain form (elementary torch operations in 32 bits, rounded once) or,
where ``own`` is true, with the calls of include/kvb.h that a serving program makes for it.

Bounds of a page and KV head.  Group g is dims 32 g .. 32 g + 31; lo and hi are the least and the largest
value that the page's keys (fp8: before their scale) have in a dim.  With m the largest |lo|, |hi| of the
group, its step s is the least power of two with m <= 127 s; the codes are floor(lo / s) and ceil(hi / s).
m < 2^-100: s and codes are 0.  A value that is not finite: s is infinity, codes 0.  A record is D codes
of lo, D of hi (int8), D / 32 steps (float32), and zeros up to a multiple of 16 bytes.

Score of a page.  A query head's values are codes too: c = round(q / t) with t the step as above of the
group, ties to even.  With b = hi's code where c > 0 and lo's where c < 0, the group's term is
(sum of c b) x (s t), the page's score for the head the sum of the terms in the order of their groups, in
float32; one that is not finite counts as the largest float32.  A page's score for a KV head is the largest
over the query heads that read it.
"""
import functools
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
GROUP = 32
LAYERS, LAYER = 2, 1
MOST = 3.4028234663852886e38


# ------------------------------------------------------------------- cases

def listed():
    """The calls of a serving program that keeps its KV pages in 16 bits or in fp8."""
    return [
        # Two short requests behind a common system prompt: the smallest call, all latency.
        dict(name="shared two short", kind="shared", dtype="bf16", format="same", groups=1, members=2, q_len=1,
             prefix=150, own_len=30, q_heads=32, heads=8, head_dim=128, page_tokens=16, page_first=False, hnd=False),
        # A decode batch behind one long prompt.
        dict(name="shared decode batch", kind="shared", dtype="bf16", format="same", groups=1, members=64, q_len=1,
             prefix=8192, own_len=1000, q_heads=32, heads=8, head_dim=128, page_tokens=16, page_first=False, hnd=False),
        # A few drafted tokens of each request, in several groups of requests.
        dict(name="shared drafts", kind="shared", dtype="fp16", format="same", groups=5, members=6, q_len=5,
             prefix=2500, own_len=700, q_heads=12, heads=4, head_dim=64, page_tokens=64, page_first=True, hnd=False),
        # 8-bit pages of 256 tokens, wide heads, two long prompts.
        dict(name="shared decode 8-bit", kind="shared", dtype="bf16", format="e4m3", groups=2, members=24, q_len=1,
             prefix=20000, own_len=2000, q_heads=16, heads=2, head_dim=256, page_tokens=256, page_first=False, hnd=True),
        # Prompt chunks of four requests behind one prefix: bound by the products.
        dict(name="shared prompt chunks", kind="shared", dtype="bf16", format="same", groups=1, members=4, q_len=500,
             prefix=8192, own_len=1000, q_heads=32, heads=8, head_dim=128, page_tokens=16, page_first=False, hnd=False),
        # The pages that a decode step wrote to: one a request.
        dict(name="bound decode", kind="bound", dtype="bf16", format="same", requests=64, new=1, max_len=8192,
             heads=8, head_dim=128, page_tokens=16, page_first=False, hnd=False),
        # All pages of long prompts.
        dict(name="bound prompts", kind="bound", dtype="bf16", format="same", requests=4, new=32768, max_len=32768,
             heads=8, head_dim=128, page_tokens=32, page_first=True, hnd=True),
        # One request with a long cache.
        dict(name="select one long", kind="select", dtype="bf16", requests=1, q_len=1, max_len=131072, q_heads=32,
             heads=8, head_dim=128, page_tokens=16, budget=256, keep_first=1, keep_last=2),
        # A decode batch of ragged lengths.
        dict(name="select decode batch", kind="select", dtype="fp16", requests=32, q_len=1, max_len=32768, q_heads=32,
             heads=8, head_dim=128, page_tokens=32, budget=64, keep_first=1, keep_last=4),
        # Attention of one request over what was selected of its long cache: all latency.
        dict(name="selected one long", kind="selected", dtype="bf16", format="same", requests=1, q_len=1, max_len=131072,
             q_heads=32, heads=8, head_dim=128, page_tokens=16, page_first=True, hnd=True, budget=256),
        # A decode batch over 8-bit pages.
        dict(name="selected decode 8-bit", kind="selected", dtype="bf16", format="e4m3", requests=48, q_len=1, max_len=32768,
             q_heads=32, heads=8, head_dim=128, page_tokens=32, page_first=False, hnd=False, budget=64),
        # A prompt chunk, every query with pages of its own.
        dict(name="selected prompt chunk", kind="selected", dtype="fp16", format="same", requests=2, q_len=150, max_len=8192,
             q_heads=12, heads=4, head_dim=64, page_tokens=16, page_first=False, hnd=False, budget=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the ranges above."""
    kind = rng.choice(("shared", "shared", "bound", "select", "selected"))
    dim = rng.choice((64, 96, 128, 128, 192, 256))
    c = dict(kind=kind, dtype=rng.choice(("bf16", "fp16")), heads=rng.choice((1, 2, 3, 4, 8)), head_dim=dim)
    group = rng.choice((1, 2, 4, 5, 8))
    if kind != "select":
        c.update(format=rng.choice(("same", "same", "e4m3")), page_first=rng.random() < 0.5, hnd=rng.random() < 0.5)
    if kind != "bound":
        c["q_heads"] = c["heads"] * group
    if kind == "shared":
        c["page_tokens"] = rng.choice((1, 16, 17, 32, 64, 256))
        c["q_len"] = rng.choice((1, 1, 1, rng.randint(2, 8), _log(rng, 9, 400)))
        c["groups"], c["members"] = _log(rng, 1, 12), _log(rng, 1, 64)
        while c["groups"] * c["members"] * c["q_len"] > 2000 or c["groups"] * c["members"] > 400:
            c["members"], c["groups"] = max(1, c["members"] // 2), max(1, c["groups"] * 2 // 3)
        rows = c["groups"] * c["members"] * c["q_len"] * c["q_heads"]
        cap = min(2 ** 28 // (c["heads"] * dim * c["groups"]), 2 ** 35 * 3 // 2 // (rows * dim))   # cached values, products
        c["prefix"] = _log(rng, 16, max(16, min(40000, cap)))
        c["own_len"] = _log(rng, c["q_len"], max(c["q_len"], min(3000, cap // c["members"])))
        return c
    c["page_tokens"] = rng.choice((8, 16, 16, 17, 32, 64))
    if kind == "bound":
        c["requests"] = _log(rng, 1, 64)
        c["max_len"] = _log(rng, 20, max(20, min(100000, 2 ** 27 // (c["requests"] * c["heads"] * dim))))
        c["new"] = rng.choice((1, 1, _log(rng, 1, c["max_len"]), c["max_len"]))
        return c
    c["requests"], c["q_len"] = _log(rng, 1, 48), rng.choice((1, 1, 1, rng.randint(2, 8), _log(rng, 9, 100)))
    while c["requests"] * c["q_len"] > 300:
        c["requests"] = max(1, c["requests"] // 2)
    tokens = c["requests"] * c["q_len"]
    cap = 2 ** 30 // (c["requests"] * c["heads"] * dim)
    if kind == "select":
        cap = min(cap, 2 ** 27 // (tokens * c["q_heads"]) * c["page_tokens"])
    low = 40 * c["page_tokens"] if kind == "select" else 20                       # something is left to select
    c["max_len"] = _log(rng, max(low, c["q_len"]), max(low, c["q_len"], min(200000, cap)))
    most = max(8, min(512, 2 ** 28 // (tokens * c["heads"] * dim * c["page_tokens"])))
    if kind == "select":
        most = min(512, c["max_len"] // (4 * c["page_tokens"]))
        c["keep_first"], c["keep_last"] = rng.randint(0, 2), rng.randint(0, 4)
    c["budget"] = _log(rng, 8, most)
    return c


# -------------------------------------------------------- what a case is made of

def _step(m):
    """The least power of two s with m <= 127 s (float32), and 1 / s; 0 and 0 under 2^-100, infinity and 0 where m is not finite."""
    e = (m.view(torch.int32) + 0x1FFFF) >> 23
    s, inv = ((e - 6).clamp(min=1) << 23).view(torch.float32), ((260 - e).clamp(1, 254) << 23).view(torch.float32)
    none = torch.zeros_like(m)
    tiny, far = m < 2.0 ** -100, ~torch.isfinite(m)
    s = torch.where(tiny, none, torch.where(far, torch.full_like(m, math.inf), s))
    return s, torch.where(tiny | far, none, inv)


def _grouped(x):
    """[..., D] as [..., D / 32, 32]."""
    return x.unflatten(-1, (-1, GROUP))


def _record_bytes(d):
    return -(-(2 * d + d // 8) // 16) * 16


def _records(lo, hi):
    """Bounds (float32, [..., D]) as records [..., bytes]."""
    d = lo.shape[-1]
    a, b = _grouped(lo), _grouped(hi)
    m = torch.maximum(a.abs().amax(-1), b.abs().amax(-1))
    s, inv = _step(torch.where(torch.isnan(m), torch.full_like(m, math.inf), m))
    code = lambda x: torch.where(inv[..., None] > 0, x, torch.zeros_like(x)).to(torch.int8).flatten(-2).view(torch.uint8)  # noqa: E731
    out = torch.zeros(*lo.shape[:-1], _record_bytes(d), dtype=torch.uint8, device=lo.device)
    out[..., :d] = code(torch.floor(a * inv[..., None]))
    out[..., d : 2 * d] = code(torch.ceil(b * inv[..., None]))
    out[..., 2 * d : 2 * d + d // 8] = s.view(torch.uint8)
    return out


def _parts(rec, d):
    """Records as codes of lo and hi (int8) and steps (float32)."""
    return rec[..., :d].view(torch.int8), rec[..., d : 2 * d].view(torch.int8), rec[..., 2 * d : 2 * d + d // 8].view(torch.float32)


def _pages(c):
    """Pages of a case's pool."""
    t = c["page_tokens"]
    if c["kind"] == "shared":
        return c["groups"] * (-(-c["prefix"] // t) + c["members"] * -(-c["own_len"] // t)) + 3
    return c["requests"] * -(-c["max_len"] // t) + 3


def _view(c, pool, comp):
    """One layer and component of the pool as words [pages, page_tokens, heads, D]."""
    pages, t, h, d = _pages(c), c["page_tokens"], c["heads"], c["head_dim"]
    b = d * (1 if c["format"] == "e4m3" else 2)
    inner = (h, t, b) if c["hnd"] else (t, h, b)
    x = pool.view(pages, LAYERS, 2, *inner)[:, LAYER, comp] if c["page_first"] else pool.view(LAYERS, 2, pages, *inner)[LAYER, comp]
    if c["format"] != "e4m3":
        x = x.view(torch.int16)
    return x.transpose(1, 2) if c["hnd"] else x


def _typed(c, x):
    """Words of a pool as the values they are."""
    return x.view(torch.float8_e4m3fn if c["format"] == "e4m3" else DTYPES[c["dtype"]])


def _layout(c, kvb):
    b = c["head_dim"] * (1 if c.get("format") == "e4m3" else 2)
    return kvb.make_layout(LAYERS, 2, _pages(c), c["page_tokens"], c["heads"], b, kvb.KV_PAGE_FIRST if c.get("page_first") else kvb.KV_LAYER_FIRST,
                           kvb.KV_HND if c.get("hnd") else kvb.KV_NHD, 1 if c.get("format") == "e4m3" else 2)


class _Handles:
    """The framework's handles of one state, closed with it."""

    def __init__(self, kvb):
        self.kvb, self.pool = kvb, None

    def __del__(self):
        if self.pool is not None:
            self.kvb.kv_pool_close(self.pool)


def _own(c, s):
    """What a program keeps for the framework's calls: the pool's handle, argument blocks over its buffers, a workspace."""
    from hierarchical_kv_cache_backup_gb300 import kvb

    h = s["handles"] = _Handles(kvb)
    h.pool = kvb.kv_pool_register(_layout(c, kvb), s["pool"].data_ptr())
    kind = c["kind"]
    common = dict(lens=s["lens"].data_ptr(), pages=s["table"].data_ptr(), pages_stride=s["table"].stride(0), requests=s["lens"].shape[0],
                  head_dim=c["head_dim"], dtype={"bf16": kvb.KV_BF16, "fp16": kvb.KV_FP16}[c["dtype"]], status=s["status"].data_ptr())
    if kind != "select":
        common.update(format=kvb.KV_CACHE_E4M3 if c["format"] == "e4m3" else kvb.KV_CACHE_SAME, layer=LAYER)
    if kind != "bound":
        common.update(q_start=s["q_start"].data_ptr(), tokens=s["q"].shape[0], max_q=c["q_len"], q_heads=c["q_heads"])
    if kind == "bound":
        s["args"] = kvb.make_bound_args(s["bounds"].data_ptr(), first=s["first"].data_ptr(), max_len=c["max_len"], max_new=c["new"], **common)
    elif kind == "select":
        s["args"] = kvb.make_select_args(s["bounds"].data_ptr(), kvb.vecs(s["q"]), s["picks"].data_ptr(), max_len=c["max_len"], budget=c["budget"],
                                         keep_first=c["keep_first"], keep_last=c["keep_last"], **common)
    elif kind == "selected":
        s["args"] = kvb.make_attend_selected_args(kvb.vecs(s["q"]), kvb.vecs(s["out"]), lse=s["lse"].data_ptr(), picks=s["picks"].data_ptr(),
                                                  budget=c["budget"], max_len=c["max_len"], scale=s["scale"], k_scale=s["k_scale"],
                                                  v_scale=s["v_scale"], **common)
    else:
        s["args"] = kvb.make_attend_shared_args(kvb.vecs(s["q"]), kvb.vecs(s["out"]), lse=s["lse"].data_ptr(), max_len=c["own_len"],
                                                group_start=s["group_start"].data_ptr(), prefix_lens=s["prefix_lens"].data_ptr(),
                                                prefix_pages=s["prefix_table"].data_ptr(), prefix_stride=s["prefix_table"].stride(0),
                                                groups=c["groups"], max_group=c["members"] * c["q_len"], max_prefix=c["prefix"],
                                                scale=s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"], **common)
    size = {"select": kvb.kv_select_workspace, "selected": kvb.kv_attend_selected_workspace, "shared": kvb.kv_attend_shared_workspace}.get(kind)
    if size is not None:
        need = size(h.pool, s["args"])
        s["workspace"] = torch.zeros(max(1, need), dtype=torch.uint8, device="cuda")
        s["args"].workspace, s["args"].workspace_bytes = s["workspace"].data_ptr(), need


def prepare(case, seed):
    """The inputs of one pass, from the seed, and the buffers and handles that a program keeps."""
    c, s = case, {"case": case}
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, d, h, pt, kind = DTYPES[c["dtype"]], c["head_dim"], c["heads"], c["page_tokens"], c["kind"]
    pages = _pages(c)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    whole = lambda hi, *shape: torch.randint(0, hi, shape, generator=g, device="cuda")  # noqa: E731
    loud, offset = torch.exp(0.5 * normal(h, d)), 0.5 * normal(h, d)             # channels of keys differ
    keys = lambda n: normal(n, h, d) * loud + offset + 0.5 * normal(-(-n // 64), h, d).repeat_interleave(64, 0)[:n]  # noqa: E731
    ragged = lambda n, most, low: low + whole(most - low + 1, n)  # noqa: E731
    s["k_scale"], s["v_scale"], s["scale"] = (0.0625, 0.03125, 1.0 / math.sqrt(d)) if c.get("format") == "e4m3" else (1.0, 1.0, 1.0 / math.sqrt(d))
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = c["groups"] * c["members"] if kind == "shared" else c["requests"]
    longest = c["own_len"] if kind == "shared" else c["max_len"]
    per = -(-longest // pt)
    order = torch.randperm(pages, generator=g, device="cuda")
    s["table"] = order[: r * per].view(r, per).int()
    lens = ragged(r, longest, max(c.get("q_len", 1), longest // 2))
    lens[0] = longest
    s["lens"] = lens.int()
    if kind != "bound":
        ql = c["q_len"]
        n_q = torch.tensor([ql - 5 * i % ql for i in range(r)], device="cuda")   # ragged new tokens
        s["q_len"] = n_q
        s["q_start"] = torch.cat((torch.zeros(1, device="cuda", dtype=torch.long), n_q.cumsum(0))).int()
        tokens = sum(ql - 5 * i % ql for i in range(r))
        s["q"] = normal(tokens, c["q_heads"], d).to(dt)
    stale = lambda: torch.randint(0, 256, (LAYERS * 2 * pages * pt * h * d * (1 if c["format"] == "e4m3" else 2),), generator=g,  # noqa: E731
                                  device="cuda", dtype=torch.uint8)

    def fill(table, length):
        at = torch.arange(length, device="cuda")
        for comp, x in ((0, keys(length)), (1, normal(length, h, d))):
            view = _view(c, s["pool"], comp)
            x = x * (1.0 / (s["v_scale"] if comp else s["k_scale"]))
            x = x.clamp(-448, 448).to(torch.float8_e4m3fn) if c["format"] == "e4m3" else x.to(dt)
            view[table.long()[at // pt], at % pt] = x.view(view.dtype)

    if kind == "select":
        s["pool"] = torch.empty(LAYERS * 2 * pages * pt * h * d * 2, dtype=torch.uint8, device="cuda")   # not looked at
        s["bounds"] = torch.zeros(pages, h, _record_bytes(d), dtype=torch.uint8, device="cuda")
        for i in range(r):
            n = int(lens[i])
            x = keys(n).to(dt).float()
            x = torch.cat((x, x[-1:].expand(-n % pt, h, d))).view(-1, pt, h, d)
            s["bounds"][s["table"][i, : x.shape[0]].long()] = _records(x.amin(1), x.amax(1))
        s["picks"] = torch.empty(s["q"].shape[0], h, c["budget"], dtype=torch.int32, device="cuda")
    elif kind == "bound":
        s["pool"] = stale()
        for i in range(r):
            fill(s["table"][i], int(lens[i]))
        s["first"] = (lens - c["new"]).clamp(min=0).int()
        s["bounds"] = torch.zeros(pages, h, _record_bytes(d), dtype=torch.uint8, device="cuda")
    else:
        s["pool"] = stale()                                                      # what is past a request's length is stale
        for i in range(r):
            fill(s["table"][i], int(lens[i]))
        s["out"] = torch.empty(s["q"].shape, dtype=dt, device="cuda")
        s["lse"] = torch.empty(s["q"].shape[0], c["q_heads"], device="cuda")
        if kind == "shared":
            n = c["groups"]
            s["group_start"] = (torch.arange(n + 1, device="cuda") * c["members"]).int()
            s["prefix_lens"] = ragged(n, c["prefix"], c["prefix"] // 2).int()
            s["prefix_lens"][0] = c["prefix"]
            s["prefix_table"] = order[r * per : r * per + n * -(-c["prefix"] // pt)].view(n, -1).int()
            for i in range(n):
                fill(s["prefix_table"][i], int(s["prefix_lens"][i]))
        else:
            # pages in any spread over what a query sees, its own page among them, in their order
            req, pos = _places(c, s)
            seen = pos // pt + 1
            x = torch.rand(pos.shape[0], h, per, generator=g, device="cuda")
            at = torch.arange(per, device="cuda")
            x = torch.where(at < seen[:, None, None], x, torch.full_like(x, -1.0))
            x = torch.where(at == seen[:, None, None] - 1, torch.full_like(x, 2.0), x)
            top = x.topk(min(per, c["budget"]), -1)
            picks = torch.where(top.values < 0, torch.full_like(top.indices, per), top.indices).sort(-1).values
            picks = torch.where(picks == per, torch.full_like(picks, -1), picks)
            pad = torch.full((*picks.shape[:2], c["budget"] - picks.shape[2]), -1, device="cuda")
            s["picks"] = torch.cat((picks, pad), -1).int()
    if own:
        _own(c, s)
    return s


# ----------------------------------------------------------------- one pass

def _places(c, s):
    """Request and position of each query token."""
    tok = torch.arange(s["q"].shape[0], device="cuda")
    r = torch.searchsorted(s["q_start"][1:], tok, right=True)
    return r, (s["lens"] - s["q_len"] - s["q_start"][:-1]).long()[r] + tok


def _softmax_parts(q, k, v, seen, scale):
    """Largest score, sum of exp and weighted sum of values: q [b, H, rows, D], k and v [b, H, n, D], seen [b, 1 or H, rows, n]."""
    x = (q @ k.transpose(2, 3) * scale).masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    return top[..., 0], p.sum(-1), p @ v


def _cached(c, s, table, lens, n):
    """Keys and values [b, H, n, D] in float32 of the first n tokens of each row of a page table; zeros past its length."""
    keep = (torch.arange(n, device="cuda") < lens[:, None])[:, :, None, None]
    both = (_typed(c, _view(c, s["pool"], comp)[table.long()].flatten(1, 2)[:, :n]).float() for comp in (0, 1))
    k, v = (x.masked_fill(~keep, 0.0).transpose(1, 2).contiguous() for x in both)
    return k * s["k_scale"], v * s["v_scale"]


def _rows(c, q):
    """Queries [b, n, q_heads, D] as [b, H, n * group, D]."""
    b, n, d = q.shape[0], q.shape[1], c["head_dim"]
    h = c["heads"]
    return q.view(b, n, h, -1, d).transpose(1, 2).reshape(b, h, -1, d)


def _tokens(c, x, n):
    """[b, H, n * group, ...] as [b, n, q_heads, ...]."""
    return x.unflatten(2, (n, -1)).transpose(1, 2).flatten(2, 3)


def _plain_shared(c, s):
    ql, most, g = c["q_len"], c["members"] * c["q_len"], c["q_heads"] // c["heads"]
    q, last = s["q"].float(), s["q"].shape[0] - 1
    tok = torch.arange(last + 1, device="cuda")
    # the prefix of a group against all of its queries at once
    start = s["q_start"][s["group_start"].long()].long()
    row = (start[:-1, None] + torch.arange(most, device="cuda")).clamp(max=last)
    k, v = _cached(c, s, s["prefix_table"], s["prefix_lens"], c["prefix"])
    seen = (torch.arange(c["prefix"], device="cuda") < s["prefix_lens"][:, None])[:, None, None]
    one = [_tokens(c, x, most) for x in _softmax_parts(_rows(c, q[row]), k, v, seen, s["scale"])]
    at = torch.searchsorted(start[1:], tok, right=True)
    one = [x[at, tok - start[at]] for x in one]
    # a request's own tokens
    i = torch.arange(ql, device="cuda")
    row = (s["q_start"][:-1, None] + i).clamp(max=last).long()
    k, v = _cached(c, s, s["table"], s["lens"], c["own_len"])
    pos = (s["lens"] - s["q_len"])[:, None] + i
    seen = (torch.arange(c["own_len"], device="cuda") <= pos[:, :, None])[:, None, :, None].expand(-1, 1, -1, g, -1).flatten(2, 3)
    two = [_tokens(c, x, ql) for x in _softmax_parts(_rows(c, q[row]), k, v, seen, s["scale"])]
    at = torch.searchsorted(s["q_start"][1:], tok, right=True)
    two = [x[at, tok - s["q_start"][at]] for x in two]
    top = torch.maximum(one[0], two[0])
    base = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    a, b = torch.exp(one[0] - base), torch.exp(two[0] - base)
    total = one[1] * a + two[1] * b
    o = (one[2] * a[..., None] + two[2] * b[..., None]) / torch.where(total > 0, total, torch.ones_like(total))[..., None]
    return {"out": o.to(s["q"].dtype), "lse": base + torch.log(total)}


def _plain_bound(c, s):
    pt, lens, first = c["page_tokens"], s["lens"].long(), s["first"].long()
    last = (lens - 1) // pt
    n = (c["new"] + pt - 2) // pt + 1
    at = torch.minimum(first[:, None] // pt + torch.arange(n, device="cuda"), last[:, None])
    page = torch.gather(s["table"].long(), 1, at)
    x = _typed(c, _view(c, s["pool"], 0)[page]).float()                         # [r, n, pt, H, D]
    live = ((at[:, :, None] * pt + torch.arange(pt, device="cuda")) < lens[:, None, None])[..., None, None]
    lo, hi = x.masked_fill(~live, math.inf).amin(2), x.masked_fill(~live, -math.inf).amax(2)
    s["bounds"][page] = _records(lo, hi)
    lo, hi, step = _parts(s["bounds"], c["head_dim"])
    return {"lo": lo, "hi": hi, "step": step}


def _plain_select(c, s):
    d, h, pt, budget, n = c["head_dim"], c["heads"], c["page_tokens"], c["budget"], s["table"].shape[1]
    req, pos = _places(c, s)
    seen = (pos // pt + 1)[:, None, None]
    lo, hi, step = _parts(s["bounds"][s["table"].long()], d)                    # [r, n, H, ...]
    i = torch.arange(c["q_len"], device="cuda")
    row = (s["q_start"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1).long()
    q = _grouped(_rows(c, s["q"].float()[row]))                                 # [r, H, rows, D / 32, 32]
    t, inv = _step(q.abs().amax(-1))
    code = torch.round(torch.where(inv[..., None] > 0, q * inv[..., None], torch.zeros_like(q))).transpose(2, 3)
    both = [_grouped(x.float()).permute(0, 2, 3, 4, 1) for x in (lo, hi)]       # [r, H, D / 32, 32, n]
    dots = code.clamp(max=0) @ both[0] + code.clamp(min=0) @ both[1]            # whole numbers below 2^24: exact in any order
    weight = step.permute(0, 2, 3, 1)[:, :, :, None] * t.transpose(2, 3)[..., None]
    score = functools.reduce(torch.add, (dots * weight).unbind(2))              # [r, H, rows, n]
    score = torch.where(torch.isfinite(score), score, torch.full_like(score, MOST))
    score = _tokens(c, score, c["q_len"]).unflatten(2, (h, -1)).amax(3)         # [r, q_len, H, n]
    score = score[req, torch.arange(pos.shape[0], device="cuda") - s["q_start"][req]]
    at = torch.arange(n, device="cuda")
    score = torch.where((at < c["keep_first"]) | (at >= seen - c["keep_last"]), torch.full_like(score, math.inf), score)
    score = torch.where(at < seen, score, torch.full_like(score, -math.inf))
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., : min(n, budget)]
    best = torch.where(torch.arange(best.shape[-1], device="cuda") < seen, best, torch.full_like(best, n)).sort(-1).values
    s["picks"].fill_(-1)
    s["picks"][..., : best.shape[-1]] = torch.where(best == n, torch.full_like(best, -1), best)
    return {"picks": s["picks"]}


def _plain_selected(c, s):
    d, h, pt = c["head_dim"], c["heads"], c["page_tokens"]
    req, pos = _places(c, s)
    picks = s["picks"].long()                                                   # [tokens, H, budget]
    tok = (picks.clamp(min=0)[..., None] * pt + torch.arange(pt, device="cuda")).flatten(2)
    seen = (picks >= 0).repeat_interleave(pt, -1) & (tok <= pos[:, None, None])
    tok = torch.where(seen, tok, torch.zeros_like(tok))
    page = s["table"].long()[req[:, None, None], tok // pt]
    head = torch.arange(h, device="cuda")[:, None]
    k, v = (_typed(c, _view(c, s["pool"], comp)[page, tok % pt, head]).float() for comp in (0, 1))   # [tokens, H, n, D]
    q = s["q"].float().unflatten(1, (h, -1))
    top, total, o = _softmax_parts(q, k * s["k_scale"], (v * s["v_scale"]).masked_fill(~seen[..., None], 0.0), seen[:, :, None], s["scale"])
    o = o / torch.where(total > 0, total, torch.ones_like(total))[..., None]
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    return {"out": o.flatten(1, 2).to(s["q"].dtype), "lse": (top + torch.log(total)).flatten(1, 2)}


def run(state):
    """One pass."""
    s, c = state, state["case"]
    if not own:
        return {"shared": _plain_shared, "bound": _plain_bound, "select": _plain_select, "selected": _plain_selected}[c["kind"]](c, s)
    h = s["handles"]
    if c["kind"] == "bound":
        h.kvb.kv_bound(h.pool, s["args"])
        lo, hi, step = _parts(s["bounds"], c["head_dim"])
        return {"lo": lo, "hi": hi, "step": step}
    if c["kind"] == "select":
        h.kvb.kv_select(h.pool, s["args"])
        return {"picks": s["picks"]}
    if c["kind"] == "selected":
        h.kvb.kv_attend_selected(h.pool, s["args"])
    else:
        h.kvb.kv_attend_shared(h.pool, s["args"])
    return {"out": s["out"], "lse": s["lse"]}


def work(case):
    """Bytes (each input read once, each output written once) and operations of one pass."""
    c = case
    d, h, pt = c["head_dim"], c["heads"], c["page_tokens"]
    vec = d * (1 if c.get("format") == "e4m3" else 2)
    mean = lambda n, most, low: (most + (n - 1) * (low + most) / 2) / n  # noqa: E731  lengths lie evenly between low and most, the first is most
    if c["kind"] == "bound":
        r, n = c["requests"], mean(c["requests"], c["max_len"], max(1, c["max_len"] // 2))
        new = min(c["new"], n)
        read = min(n, new + (pt - 1) / 2 + (pt - 1) / 2 * (new < n))              # the pages of new tokens, up to the length
        pages = 1 + (new - 1) / pt
        return {"bytes": r * (read * h * vec + pages * (h * _record_bytes(d) + 4) + 8), "flops": 2 * r * read * h * d}
    ql = c["q_len"]
    r = c["groups"] * c["members"] if c["kind"] == "shared" else c["requests"]
    new = sum(ql - 5 * i % ql for i in range(r))
    if c["kind"] == "shared":
        n = mean(r, c["own_len"], max(ql, c["own_len"] // 2))
        p = mean(c["groups"], c["prefix"], c["prefix"] // 2)
        cached = r * n + c["groups"] * p
        return {"bytes": cached * (2 * h * vec + 4 / pt) + new * c["q_heads"] * (4 * d + 4),
                "flops": 4 * new * c["q_heads"] * d * (p + n - (new / r - 1) / 2)}
    n = mean(r, c["max_len"], max(ql, c["max_len"] // 2))
    sees = n - (new / r - 1) / 2
    if c["kind"] == "select":
        pages = n / pt
        return {"bytes": r * pages * (h * _record_bytes(d) + 4) + new * (c["q_heads"] * 2 * d + 4 * h * c["budget"]),
                "flops": 2 * new * c["q_heads"] * d * sees / pt}
    picked = min(sees, c["budget"] * pt - (pt - 1) / 2)
    # a page that several queries of a request select is read once: at most what the request holds
    read = min(n, new / r * picked)
    return {"bytes": r * read * 2 * h * vec + new * (c["q_heads"] * (4 * d + 4) + 4 * h * min(c["budget"], sees / pt)),
            "flops": 4 * new * c["q_heads"] * d * picked}


# ------------------------------------------------------------- in 64 bits

def _exact_rows(q, k, v, hide, scale):
    """Queries [n, D] over keys and values [m, D] in 64 bits."""
    x = torch.mm(q.double(), k.T).mul(scale)
    if hide is not None:
        x = x.masked_fill(hide, -math.inf)
    return torch.mm(torch.softmax(x, 1), v), torch.logsumexp(x, 1)


def exact(case, seed):
    """The same outputs in 64 bits, from the definitions; what is selected has no other value than its own."""
    c, s = case, prepare(case, seed)
    h, d, pt = c["heads"], c["head_dim"], c["page_tokens"]
    if c["kind"] == "select":
        return None
    if c["kind"] == "bound":
        if c["requests"] * (-(-c["new"] // pt) + 1) > 40000:
            return None
        x, steps = _view(c, s["pool"], 0), torch.zeros(_pages(c), h, d // GROUP, dtype=torch.float64, device="cuda")
        codes = [torch.zeros(_pages(c), h, d, dtype=torch.int8, device="cuda") for _ in range(2)]
        for i in range(c["requests"]):
            n = int(s["lens"][i])
            for j in range(int(s["first"][i]) // pt, (n - 1) // pt + 1):
                p = int(s["table"][i, j])
                y = _typed(c, x[p, : min(pt, n - j * pt)].contiguous()).double()
                m = y.abs().amax(0).view(h, -1, GROUP).amax(-1)
                mant, exp = torch.frexp(m / 127)
                steps[p] = torch.ldexp(torch.ones_like(m), exp - (mant == 0.5).int())
                by = steps[p].repeat_interleave(GROUP, 1)
                codes[0][p], codes[1][p] = torch.floor(y.amin(0) / by).to(torch.int8), torch.ceil(y.amax(0) / by).to(torch.int8)
        return {"lo": codes[0], "hi": codes[1], "step": steps}
    g = c["q_heads"] // h
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")

    def vectors(table, at, head):
        return [_typed(c, _view(c, s["pool"], comp)[table.long()[at // pt], at % pt, head]).double() * s["v_scale" if comp else "k_scale"]
                for comp in (0, 1)]

    if c["kind"] == "shared":
        for i in range(s["lens"].shape[0]):
            a, e, n, grp = int(s["q_start"][i]), int(s["q_start"][i + 1]), int(s["lens"][i]), i // c["members"]
            p = int(s["prefix_lens"][grp])
            hide = torch.arange(p + n, device="cuda") > p + torch.arange(n - (e - a), n, device="cuda")[:, None]
            for j in range(h):
                parts = zip(vectors(s["prefix_table"][grp], torch.arange(p, device="cuda"), j), vectors(s["table"][i], torch.arange(n, device="cuda"), j))
                k, v = (torch.cat(x) for x in parts)
                for m in range(j * g, j * g + g):
                    out[a:e, m], lse[a:e, m] = _exact_rows(s["q"][a:e, m], k, v, hide, s["scale"])
        return {"out": out, "lse": lse}
    for i in range(s["lens"].shape[0]):
        a, e, n = int(s["q_start"][i]), int(s["q_start"][i + 1]), int(s["lens"][i])
        for t in range(a, e):
            for j in range(h):
                p = s["picks"][t, j]
                at = (p[p >= 0].long()[:, None] * pt + torch.arange(pt, device="cuda")).flatten()
                at = at[at <= n - (e - t)]
                k, v = vectors(s["table"][i], at, j)
                out[t, j * g : j * g + g], lse[t, j * g : j * g + g] = _exact_rows(s["q"][t, j * g : j * g + g], k, v, None, s["scale"])
    return {"out": out, "lse": lse}
