"""Which kernel takes what of a call of attention over 16-bit and fp8 pages, and the room it has for that: the
library's own plan, compiled for the host."""
import ctypes
import random
import shutil
import subprocess

import numpy as np
import pytest

from hierarchical_kv_cache_backup_gb300 import build as kbuild

HARNESS = r"""
#include "kvb_pages_plan.h"
using namespace kvb;
// in: requests, tokens, max_q, max_len, groups, max_group, max_prefix, budget, T, q_heads, kv_heads, D, fp8, sms, per_sm
static PagePlan plan_of(const uint32_t *in) {
    return plan_pages(in[0], in[1], in[2], in[3], in[4], in[5], in[6], in[7], in[8], in[9], in[10], in[11], in[12] != 0, (int)in[13], in[14]);
}
extern "C" void h_plan(const uint32_t *in, uint64_t *out) {
    const PagePlan p = plan_of(in);
    for (const PageEngine *e : {&p.rows, &p.tc}) {
        const uint64_t v[] = {e->on, e->prefix, e->own, e->whole, e->unit_cost, e->row_tile, e->kv_shift, e->workers, e->slot_rows, e->team, e->units, e->small};
        for (uint64_t x : v) *out++ = x;
    }
    *out++ = p.joined;
    *out++ = p.bytes;
    *out++ = p.join_heads;
    *out++ = p.wide_join;
}
// Whether the kernels' 32-bit counts hold the call.
extern "C" int h_fits(const uint32_t *in) {
    return plan_counts_fit(plan_of(in), in[2], in[3], in[5], in[6], in[7], in[8], in[9], in[10]);
}
// Tiles and units of all segments, of the kernel for few rows and of that on tcgen05.
extern "C" void h_work(const uint32_t *in, const int *q_start, const int *lens, const int *group_start, const int *prefix_lens, uint64_t *out) {
    const PagePlan p = plan_of(in);
    PageAttendArgs a{};
    a.q_start = q_start; a.lens = lens; a.group_start = group_start; a.prefix_lens = prefix_lens;
    a.requests = in[0]; a.tokens = in[1]; a.max_q = in[2]; a.max_len = in[3]; a.groups = in[4]; a.max_group = in[5]; a.max_prefix = in[6];
    a.budget = in[7]; a.pool.T = in[8]; a.q_heads = in[9]; a.pool.H = in[10]; a.group = in[9] / in[10];
    int picked = 0;
    a.picks = in[7] ? &picked : nullptr;
    while ((1ull << a.pool.t_shift) < a.pool.T) ++a.pool.t_shift;             // division by T, as the library's
    a.pool.t_mul = (uint32_t)(((1ull << 32) * ((1ull << a.pool.t_shift) - a.pool.T)) / a.pool.T + 1);
    a.joined = p.joined; a.rows = p.rows; a.tc = p.tc;
    for (const PageEngine *e : {&a.rows, &a.tc}) {
        out[0] = out[1] = 0;
        for (uint32_t s = 0; e->on && s < seg_count(a, *e); ++s) {
            const PageSeg g = seg_at(a, *e, s);
            const uint64_t tiles = seg_tiles(a, *e, g);
            out[0] += tiles;
            out[1] += seg_units(a, *e, g, tiles);
        }
        out += 2;
    }
}
// The kernel for few rows: what a block's table sums up of `segs` segments of these tiles and units.
extern "C" uint64_t h_packed(const uint32_t *in, uint32_t segs, uint64_t tiles, uint64_t units) {
    const PagePlan p = plan_of(in);
    uint64_t sum = 0;
    for (uint32_t s = 0; s < segs; ++s) sum += pack_work(p.rows, tiles, units);
    return sum;
}
"""
ENGINE = ("on", "prefix", "own", "whole", "unit_cost", "row_tile", "kv_shift", "workers", "slot_rows", "team", "units", "small")
IN = ("requests", "tokens", "max_q", "max_len", "groups", "max_group", "max_prefix", "budget", "T", "q_heads", "kv_heads", "D", "fp8", "sms", "per_sm")
SHAPE = dict(groups=0, max_group=0, max_prefix=0, budget=0, T=16, q_heads=32, kv_heads=8, D=128, fp8=0, sms=152, per_sm=3)


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("plan")
    (d / "h.cpp").write_text(HARNESS)
    subprocess.run([cc, "-O1", "-std=c++17", "-shared", "-fPIC", "-I", kbuild.CSRC, str(d / "h.cpp"), "-o", str(d / "h.so")], check=True)
    return ctypes.CDLL(str(d / "h.so"))


class Plan:
    def __init__(self, host, **kw):
        shape = dict(SHAPE, **kw)
        self.args = np.array([shape[k] for k in IN], dtype=np.uint32)
        self.host, out = host, np.zeros(2 * len(ENGINE) + 4, dtype=np.uint64)
        host.h_plan(ctypes.c_void_p(self.args.ctypes.data), ctypes.c_void_p(out.ctypes.data))
        out = [int(x) for x in out]
        n = len(ENGINE)
        self.rows, self.tc = dict(zip(ENGINE, out[:n])), dict(zip(ENGINE, out[n:2 * n]))
        self.joined, self.bytes, self.join_heads, self.wide_join = out[2 * n:]

    def fits(self):
        return bool(self.host.h_fits(ctypes.c_void_p(self.args.ctypes.data)))

    def work(self, q_start, lens, group_start=(0,), prefix_lens=(0,)):
        """(tiles, units) of the kernel for few rows and of that on tcgen05."""
        at = [np.array(x, dtype=np.int32) for x in (q_start, lens, group_start, prefix_lens)]
        out = np.zeros(4, dtype=np.uint64)
        self.host.h_work(*(ctypes.c_void_p(x.ctypes.data) for x in (self.args, *at, out)))
        return [(int(out[0]), int(out[1])), (int(out[2]), int(out[3]))]


def test_plans(host):
    """A call of each kind: who takes the prefixes, who the requests' own tokens."""
    p = Plan(host, requests=2, tokens=2, max_q=1, max_len=30, groups=1, max_group=2, max_prefix=150)
    assert p.rows["on"] and p.rows["whole"] and p.joined and not p.tc["on"] and p.bytes == 0
    p = Plan(host, requests=64, tokens=64, max_q=1, max_len=1000, groups=1, max_group=64, max_prefix=8192)
    assert p.tc["prefix"] and not p.tc["own"] and p.rows["own"] and not p.rows["prefix"] and not p.joined
    p = Plan(host, requests=4, tokens=2000, max_q=500, max_len=1000, groups=1, max_group=2000, max_prefix=8192)
    assert p.tc["own"] and not p.tc["prefix"] and not p.rows["on"] and p.joined
    p = Plan(host, requests=2, tokens=100, max_q=50, max_len=1000, groups=1, max_group=100, max_prefix=8192)
    assert p.tc["own"] and p.tc["prefix"] and not p.rows["on"] and not p.joined
    p = Plan(host, requests=1, tokens=1, max_q=1, max_len=131072, budget=256)
    assert p.rows["own"] and not p.rows["whole"] and not p.tc["on"]


@pytest.mark.parametrize("seed", range(60))
def test_room_for_the_work(host, seed):
    """What valid ranges hold is never more than the plan has room for, and counts that are said to be small are."""
    rng = random.Random(seed)
    requests, q, length, prefix = rng.choice((1, 3, 60, 127)), rng.choice((1, 4, 30, 600)), rng.choice((0, 1, 90, 5000)), rng.choice((0, 40, 9000))
    picked = seed % 3 == 0
    groups = 0 if picked else rng.choice((0, 1, 4))
    n_q = [rng.choice((1, q, rng.randint(0, q))) for _ in range(requests)]
    q_start = np.cumsum([0] + n_q)
    marks = sorted(rng.randint(0, requests) for _ in range(groups + 1))
    max_group = max([int(q_start[b] - q_start[a]) for a, b in zip(marks, marks[1:])], default=0)
    kv_heads, group = rng.choice((1, 4, 8)), rng.choice((1, 4, 16, 40))
    p = Plan(host, requests=requests, tokens=max(1, sum(n_q)), max_q=max(1, max(n_q)), max_len=length, groups=groups, max_group=max_group, max_prefix=prefix if groups else 0,
             budget=rng.choice((1, 30, 2000)) if picked else 0, T=rng.choice((1, 16, 17, 256)), q_heads=kv_heads * group, kv_heads=kv_heads,
             D=rng.choice((64, 128, 256)))
    lens = [rng.choice((0, length, rng.randint(0, length))) for _ in range(requests)]
    for e, (tiles, units) in zip((p.rows, p.tc), p.work(q_start, lens, marks, [prefix] * max(1, groups))):
        if e["on"]:
            assert units <= e["units"] and (not e["small"] or tiles < 2 ** 31)


def test_lists_of_large_pages(host):
    """A list counts whole pages, of up to 2^20 tokens, however short the request is."""
    tokens = 6 * 54720
    p = Plan(host, requests=6, tokens=tokens, max_q=54720, max_len=64, budget=1, T=1 << 20, q_heads=1, kv_heads=1, D=64, per_sm=4)
    (tiles, units), _ = p.work([54720 * i for i in range(7)], [64] * 6)
    assert p.rows["on"] and units == p.rows["units"] == tokens
    assert tiles == tokens << 14 and not p.rows["small"]
    assert tiles + (units << 32) >> 32 != units                  # what a sum of 32-bit words would have said


@pytest.mark.parametrize("heads", [1, 255, 256, 1025])
def test_overlapping_ranges_do_not_wrap_the_tables_sums(host, heads):
    """64 requests of the same 65,535 query tokens (every other range out of order): more units than there is room for,
    whether a block's table sums them in 32 bits or a kernel of its own in 64."""
    n = 65535
    p = Plan(host, requests=127, tokens=n, max_q=n, max_len=16, budget=1, T=16, q_heads=heads, kv_heads=heads, D=64)
    (tiles, units), _ = p.work([n * (i % 2) for i in range(128)], [16] * 127)
    assert units == 64 * n * heads > p.rows["units"]
    if p.rows["small"]:
        host.h_packed.restype, host.h_packed.argtypes = ctypes.c_uint64, [ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_uint64]
        assert host.h_packed(p.args.ctypes.data, 64, tiles // 64, units // 64) >> 32 > p.rows["units"]
        assert host.h_packed(p.args.ctypes.data, 1, tiles // 64, units // 64) == tiles // 64 | (units // 64) << 32


@pytest.mark.parametrize("chunk,length,budget,T", [(4096, 1 << 20, 64, 16), (32768, 1 << 17, 64, 16), (65535, 1 << 20, 512, 32), (8192, 1 << 22, 2048, 1)])
def test_chunks_over_long_caches_count_their_lists(host, chunk, length, budget, T):
    """What a list stands for is the work, not all that the request has cached."""
    p = Plan(host, requests=1, tokens=chunk, max_q=chunk, max_len=length, budget=budget, T=T)
    (tiles, units), _ = p.work([0, chunk], [length])
    assert p.fits() and tiles < 2 ** 31 and units == chunk * 8
    assert p.rows["small"] and tiles <= units * ((budget * T >> p.rows["kv_shift"]) + 2 + p.rows["unit_cost"])


@pytest.mark.parametrize("kw", [dict(max_q=65535, max_len=1 << 24, budget=1 << 24), dict(max_q=65535, max_len=1 << 29, budget=1, kv_heads=64, q_heads=64),
                                dict(max_q=65535, max_len=1 << 29)])
def test_work_past_32_bits_does_not_fit(host, kw):
    assert not Plan(host, **dict(dict(requests=2, tokens=70000, T=1), **kw)).fits()


@pytest.mark.parametrize("seed", range(40))
def test_what_fits_is_counted_in_31_bits(host, seed):
    rng = random.Random(seed)
    picked = seed % 2
    q, kv_heads, group = rng.choice((1, 500, 65535)), rng.choice((1, 8, 64)), rng.choice((1, 5, 16, 17))
    length, prefix, groups = rng.choice((1, 5000, 1 << 20, 1 << 29)), rng.choice((0, 1 << 20, 1 << 29)), 0 if picked else rng.choice((0, 1))
    p = Plan(host, requests=1, tokens=q, max_q=q, max_len=length, groups=groups, max_group=q if groups else 0, max_prefix=prefix if groups else 0,
             budget=rng.choice((1, 64, 1 << 24)) if picked else 0, T=rng.choice((1, 16, 1 << 20)), q_heads=kv_heads * group, kv_heads=kv_heads)
    if p.fits():
        for tiles, _ in (p.work([0, q], [length], [0, 1], [prefix]) if length * q < 2 ** 45 else ()):
            assert tiles < 2 ** 32 if groups else tiles < 2 ** 31


@pytest.mark.parametrize("max_q", [1, 4, 10, 100])
@pytest.mark.parametrize("max_len", [50, 20000])
def test_groups_without_prefixes(host, max_q, max_len):
    """They are planned as no groups are: no kernel is launched, given SMs or room for prefixes of no tokens."""
    kw = dict(requests=6, tokens=6 * max_q, max_q=max_q, max_len=max_len)
    p, alone = Plan(host, groups=2, max_group=3 * max_q, **kw), Plan(host, **kw)
    assert p.joined and (p.rows, p.tc, p.bytes) == (alone.rows, alone.tc, alone.bytes)


def test_the_sms_go_where_the_work_is(host):
    """A few queries over a long prefix beside a chunk of another request, and the other way round."""
    kw = dict(requests=5, tokens=54, max_q=50, groups=1, max_group=4)
    far, near = Plan(host, max_len=100, max_prefix=100000, **kw), Plan(host, max_len=100000, max_prefix=100, **kw)
    for p in (far, near):
        assert p.rows["prefix"] and not p.rows["own"] and p.tc["own"] and not p.tc["prefix"]
    assert far.tc["workers"] < 20 and near.tc["workers"] > 130


@pytest.mark.parametrize("n_q,joined", [([500] * 4, 1), ([64] * 16, 1), ([500, 300, 200, 120], 1), ([512], 1), ([500] * 4 + [1], 1), ([2048] + [1] * 8, 1),
                                        ([1] * 63 + [512], 0), ([500] * 4 + [1] * 16, 0), ([2048] + [1] * 30, 0), ([1] * 7 + [64], 0), ([63] * 16, 0)])
def test_a_prefix_is_read_again_only_by_requests_that_fill_units(host, n_q, joined):
    """A chunk among single tokens leaves the prefix to be read for all of them together."""
    p = Plan(host, requests=len(n_q), tokens=sum(n_q), max_q=max(n_q), max_len=1000, groups=1, max_group=sum(n_q), max_prefix=8192)
    assert p.joined == joined and p.tc["prefix"] == 1 - joined
    q_start = np.cumsum([0] + n_q)
    _, (tiles, units) = p.work(q_start, [1000] * len(n_q), [0, len(n_q)], [8192])
    filled = -(-sum(n_q) * 4 // 256)
    assert tiles <= 8 * ((4 * filled // 3 if joined else filled) * (8192 // 64 + 10) + (filled + len(n_q)) * (1000 // 64 + 1 + 10))
