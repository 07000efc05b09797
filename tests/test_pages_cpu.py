"""Attention over 16-bit and fp8 pages, bounds and selection without a GPU: how a call's work is
cut and joined, compiled for the host, and refusals that need no device."""
import ctypes
import os
import random
import shutil
import subprocess

import numpy as np
import pytest

from hierarchical_kv_cache_backup_gb300 import build as kbuild

kbuild.build_library()
from hierarchical_kv_cache_backup_gb300 import kvb  # noqa: E402

HARNESS = r"""
#include <map>
#include <vector>
#include "kvb_pages.h"
using namespace kvb;
// Cuts a call among workers and takes every row's pieces back together.  Returns 0, or the number of
// the check that failed.  in: requests, tokens, max_q, max_len, groups, max_group, max_prefix, H, group,
// T, budget, row_tile, kv_tile, workers, prefix, own, joined, unit_cost, whole; units: room in the workspace.
extern "C" int h_cut(const int *in, const int *q_start, const int *lens, const int *group_start, const int *prefix_lens,
                     unsigned long long units, unsigned long long *total) {
    PageAttendArgs a{};
    a.q_start = q_start; a.lens = lens; a.group_start = group_start; a.prefix_lens = prefix_lens;
    a.requests = in[0]; a.tokens = in[1]; a.max_q = in[2]; a.max_len = in[3]; a.groups = in[4]; a.max_group = in[5];
    a.max_prefix = in[6]; a.pool.H = in[7]; a.group = in[8]; a.pool.T = in[9]; a.budget = in[10];
    int picked = 0;
    a.picks = in[10] ? &picked : nullptr;
    PageEngine &e = a.rows;
    while ((1ull << a.pool.t_shift) < (unsigned)in[9]) ++a.pool.t_shift;      // division by T, as the library's
    a.pool.t_mul = (uint32_t)(((1ull << 32) * ((1ull << a.pool.t_shift) - in[9])) / in[9] + 1);
    e.row_tile = in[11]; e.kv_shift = in[12] == 16 ? 4 : 6; e.workers = in[13]; e.prefix = in[14]; e.own = in[15]; a.joined = in[16]; e.unit_cost = in[17]; e.whole = in[18];
    const uint32_t n = seg_count(a, e);
    std::vector<uint64_t> st(n + 1), su(n + 1);
    uint64_t t = 0, u = 0;
    for (uint32_t s = 0; s < n; ++s) {
        st[s] = t; su[s] = u;
        const PageSeg g = seg_at(a, e, s);
        const uint64_t x = seg_tiles(a, e, g);
        t += x;
        u += seg_units(a, e, g, x);
    }
    st[n] = t; su[n] = u;
    e.seg_tiles = st.data(); e.seg_units = su.data();
    *total = t;
    if (u > units) return 1;
    if (e.whole) e.workers = (uint32_t)units;
    const uint64_t run = e.whole ? u : t, share = e.whole ? 1 : share_of(t, e.workers);
    const std::vector<uint64_t> &counts = e.whole ? su : st;
    std::map<std::vector<uint64_t>, int> alone;
    std::vector<int32_t> segs(n * kSegWords + 1);
    for (uint32_t s = 0; s < n; ++s) put_seg(segs.data() + s * kSegWords, seg_at(a, e, s));
    const PageTable table{st.data(), su.data(), segs.data()};
    std::map<uint64_t, PagePiece> slots;
    uint64_t done = 0;
    for (uint32_t w = 0; w < e.workers; ++w) {
        uint64_t x = w * share, x1 = x + share < run ? x + share : run;
        if (x >= x1) continue;
        uint32_t seg = find_segment(counts.data(), n, x);
        if (x < counts[seg] || x >= counts[seg + 1]) return 11;
        while (x < x1) {
            const PagePiece p = piece_of(a, e, table, &seg, x, x1, w);
            done += p.span;
            x += p.span;
            if (p.span == 0) return 12;
            if (e.whole) {
                if (p.k0 != 0 || p.k1 != p.n_tiles || (uint32_t)p.n_tiles != unit_tiles(a, e, p.s, p.rt) || p.rt >= row_tiles(a, e, p.s)) return 13;
                if (!alone.emplace(std::vector<uint64_t>{p.s.index, (uint64_t)p.rt, (uint64_t)p.head}, 1).second) return 14;
                continue;
            }
            if (p.k1 <= p.k0) continue;
            if ( p.k1 > p.n_tiles || p.head >= (int)a.pool.H || p.rt >= row_tiles(a, e, p.s)) return 2;
            if ((uint32_t)p.n_tiles != unit_tiles(a, e, p.s, p.rt)) return 3;
            if (p.slot >= units + e.workers || !slots.emplace(p.slot, p).second) return 4;
        }
    }
    if (done != run) return 5;
    if (e.whole) return 0;
    for (uint32_t s = 0; s < n; ++s) {
        const PageSeg g = seg_at(a, e, s);
        for (int i = 0; i < g.n; ++i)
            for (uint32_t h = 0; h < a.pool.H; ++h)
                for (uint32_t j = 0; j < a.group; ++j) {
                    int row;
                    const int rt = row_tile_of(a, e, i, j, &row);
                    const uint64_t from = st[s] + tiles_before(a, e, g, rt) * a.pool.H;
                    const RowPieces r = row_pieces(a, e, share_of(t, e.workers), from, su[s], unit_span(a, e, g, rt), rt, row, h);
                    int at = 0;
                    if (r.any)
                        for (uint64_t w = r.w0; w <= r.w1; ++w) {
                            auto f = slots.find(r.unit + w);
                            if (f == slots.end()) return 6;
                            const PagePiece &p = f->second;
                            if (p.s.prefix != g.prefix || p.s.index != g.index || p.head != (int)h || p.k0 != at) return 7;
                            const int per = (int)((a.group + e.row_tile - 1) / e.row_tile);
                            const int row = a.picks ? p.rt % per * (int)e.row_tile + r.row : p.rt * (int)e.row_tile + r.row;
                            if (a.picks ? p.rt / per != i || row != (int)j : row != i * (int)a.group + (int)j) return 8;
                            at = p.k1;
                            if (w == r.w1 && at != p.n_tiles) return 9;
                        }
                    // all that the row sees is in its pieces
                    const int sees = g.prefix ? g.len : a.picks ? 0 : g.len - g.n + i + 1, pre = a.joined && g.in >= 0 ? prefix_seg(a, g.in).len : 0;
                    if (((int64_t)(at - tiles_of(e, pre)) << e.kv_shift) < sees) return 10;
                }
    }
    return 0;
}
extern "C" int h_group(const int *in, const int *q_start, const int *group_start, const int *prefix_lens, int r, int q0, int n) {
    PageAttendArgs a{};
    a.q_start = q_start; a.group_start = group_start; a.prefix_lens = prefix_lens;
    a.requests = in[0]; a.tokens = in[1]; a.groups = in[2]; a.max_group = in[3]; a.max_prefix = in[4];
    return group_of(a, r, q0, n);
}
extern "C" float h_step(unsigned bits, float *inv) { return bound_step(bits, inv); }
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("pages")
    (d / "h.cpp").write_text(HARNESS)
    subprocess.run([cc, "-O1", "-std=c++17", "-shared", "-fPIC", "-I", kbuild.CSRC, str(d / "h.cpp"), "-o", str(d / "h.so")],
                   check=True)
    lib = ctypes.CDLL(str(d / "h.so"))
    lib.h_step.restype = ctypes.c_float
    lib.h_cut.argtypes = [ctypes.c_void_p] * 5 + [ctypes.c_uint64, ctypes.c_void_p]
    return lib


def i32(x):
    return np.ascontiguousarray(x, dtype=np.int32)


def most_units(segs, tokens, most, group, row_tile, picked):
    """The room that the workspace has, as the library counts it."""
    if picked:
        return tokens * -(-group // row_tile)
    return min(segs * -(-most * group // row_tile), tokens * group // row_tile + segs)


def cut(host, rng, requests, max_q, max_len, groups, max_prefix, H, group, T, budget, row_tile, kv_tile, workers, prefix, own, joined=0, cost=0, whole=0):
    n_q = [rng.choice((0, 1, max_q, rng.randint(0, max_q))) for _ in range(requests)]
    q_start = np.cumsum([0] + n_q)
    lens = [rng.choice((0, 1, max_len, rng.randint(0, max_len))) for _ in range(requests)]
    marks = sorted(rng.randint(0, requests) for _ in range(groups + 1))
    prefix_lens = [rng.choice((0, 1, max_prefix, rng.randint(0, max_prefix))) for _ in range(groups)]
    tokens = max(1, int(q_start[-1]))
    max_group = max([int(q_start[b] - q_start[a]) for a, b in zip(marks, marks[1:])], default=0)
    units = H * ((most_units(groups, tokens, max_group, group, row_tile, False) if prefix else 0) +
                 (most_units(requests, tokens, max_q, group, row_tile, budget > 0) if own else 0))
    arrays = [i32(x) for x in ([requests, tokens, max_q, max_len, groups, max_group, max_prefix, H, group, T, budget,
                                row_tile, kv_tile, workers, prefix, own, joined, cost, whole], q_start, lens, marks, prefix_lens or [0])]
    total = ctypes.c_uint64()
    got = host.h_cut(*(x.ctypes.data for x in arrays), units, ctypes.byref(total))
    assert got == 0, (got, n_q, lens, marks, prefix_lens)
    return total.value


@pytest.mark.parametrize("seed", range(90))
def test_pieces_cover_every_row_once(host, seed):
    rng = random.Random(seed)
    picked = seed % 3 == 0
    groups = 0 if picked else rng.choice((0, 1, 5))
    which = (0, 1) if picked or groups == 0 else rng.choice(((1, 1), (1, 0), (0, 1), (0, 1, 1)))
    cut(host, rng, rng.choice((1, 3, 40, 150)), rng.choice((1, 5, 33)), rng.choice((1, 17, 500)), groups, rng.choice((0, 1, 900)),
        rng.choice((1, 2, 8)), rng.choice((1, 4, 5, 16, 17, 40)), rng.choice((1, 16, 17, 64)),
        rng.choice((1, 3, 100)) if picked else 0, rng.choice((16, 128, 256)), rng.choice((16, 64)),
        rng.choice((1, 7, 152, 1216)), *which, cost=rng.choice((0, 1, 10)))


def test_nothing_to_do_is_nothing(host):
    rng = random.Random(0)
    assert cut(host, rng, 3, 0, 50, 2, 0, 4, 4, 16, 0, 16, 16, 9, 1, 1) == 0


def test_overlapping_queries_pass_the_room(host):
    """Ranges that overlap (every other one out of order) may hold more units than the workspace has room for."""
    requests, tokens = 64, 100
    q_start, lens = i32([100 * (i % 2) for i in range(requests + 1)]), i32([300] * requests)
    args = i32([requests, tokens, 100, 300, 0, 0, 0, 2, 4, 16, 0, 16, 16, 152, 0, 1, 0, 0, 0])
    none = i32([0, 0])
    room = 2 * most_units(requests, tokens, 100, 4, 16, False)
    got = host.h_cut(args.ctypes.data, q_start.ctypes.data, lens.ctypes.data, none.ctypes.data, none.ctypes.data, room,
                     ctypes.byref(ctypes.c_uint64()))
    assert got == 1


def test_group_of_a_request(host):
    q_start = i32([0, 2, 2, 5, 6, 9])
    marks, lens = i32([0, 2, 2, 4, 4]), i32([7, 7, 9, 9])          # groups 0: requests 0, 1; 2: 2, 3; 4 has none
    args = i32([5, 9, 4, 9, 100])
    at = lambda r, m=marks, a=args, k=lens: host.h_group(  # noqa: E731
        a.ctypes.data, q_start.ctypes.data, m.ctypes.data, k.ctypes.data, r, int(q_start[r]), int(q_start[r + 1] - q_start[r]))
    assert [at(r) for r in range(5)] == [0, 0, 2, 2, -1]
    assert at(0, k=i32([0, 7, 9, 9])) == -1                        # an empty prefix
    assert at(3, a=i32([5, 9, 4, 3, 100])) == -1                   # more queries than max_group
    assert at(0, m=i32([3, 1, 4, 9, 0])) == -1                     # out of order
    assert at(1, m=i32([3, 1, 4, 9, 0])) == 1
    assert at(4, m=i32([0, 2, 2, 4, 7])) == -1


@pytest.mark.parametrize("m", [0.0, 1e-45, 2.0 ** -101, 2.0 ** -100, 0.01, 1.0, 1.984375, 1.984375 * (1 + 2 ** -23), 1.99, 127.0,
                               127.5, 1e30, 3.4028235e38, np.inf, np.nan])
def test_step_of_bounds(host, m):
    inv = ctypes.c_float()
    s = host.h_step(int(np.float32(m).view(np.uint32)), ctypes.byref(inv))
    if not np.isfinite(m):
        assert s == np.inf and inv.value == 0
    elif m < 2.0 ** -100:
        assert s == 0 and inv.value == 0
    else:
        assert np.frexp(s)[0] == 0.5 and s * inv.value == 1
        assert float(np.float32(m)) <= 127 * s and float(np.float32(m)) > 63.5 * s


V16 = kvb.kv_vecs(1 << 20, 128, 64)


@pytest.mark.parametrize("pool,status", [(None, kvb.KV_ERR_INVALID_ARG), (987654321, kvb.KV_ERR_CLOSED)])
def test_calls_without_a_pool(pool, status):
    at = dict(q_start=1 << 21, lens=1 << 21, pages=1 << 21, pages_stride=1, requests=1, tokens=1, max_q=1, max_len=1, q_heads=1, head_dim=64, dtype=0)
    sh = kvb.make_attend_shared_args(V16, V16, format=0, layer=0, scale=1.0, **at)
    se = kvb.make_select_args(1 << 22, V16, 1 << 23, budget=1, **at)
    sd = kvb.make_attend_selected_args(V16, V16, picks=1 << 23, budget=1, format=0, layer=0, scale=1.0, **at)
    bo = kvb.make_bound_args(1 << 22, lens=1 << 21, pages=1 << 21, pages_stride=1, requests=1, max_len=1, max_new=1, head_dim=64, dtype=0, format=0, layer=0)
    for call in (lambda: kvb.kv_attend_shared(pool, sh), lambda: kvb.kv_attend_shared_workspace(pool, sh), lambda: kvb.kv_select(pool, se),
                 lambda: kvb.kv_select_workspace(pool, se), lambda: kvb.kv_attend_selected(pool, sd),
                 lambda: kvb.kv_attend_selected_workspace(pool, sd), lambda: kvb.kv_bound(pool, bo)):
        with pytest.raises(kvb.KvError) as e:
            call()
        assert e.value.status == status


def test_null_blocks():
    lib, out = kvb.library(), ctypes.c_uint64()
    for call in (lambda: lib.kv_attend_shared(None, None, None), lambda: lib.kv_attend_shared_workspace(None, None, out),
                 lambda: lib.kv_attend_selected(None, None, None), lambda: lib.kv_attend_selected_workspace(None, None, out),
                 lambda: lib.kv_select(None, None, None), lambda: lib.kv_select_workspace(None, None, out), lambda: lib.kv_bound(None, None, None),
                 lambda: lib.kv_bound_bytes(128, None)):
        assert call() == kvb.KV_ERR_INVALID_ARG


@pytest.mark.parametrize("dim,want", [(64, 144), (96, 208), (128, 272), (192, 416), (256, 544)])
def test_record_sizes(dim, want):
    assert kvb.kv_bound_bytes(dim) == want


@pytest.mark.parametrize("dim", [0, 8, 32, 80, 160, 320])
def test_record_sizes_refused(dim):
    with pytest.raises(kvb.KvError) as e:
        kvb.kv_bound_bytes(dim)
    assert e.value.status == kvb.KV_ERR_LAYOUT


def test_block_sizes_match_the_header():
    """sizeof of every argument block, from the C compiler."""
    names = ["kv_attend_shared_args", "kv_bound_args", "kv_select_args", "kv_attend_selected_args"]
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    src = '#include "kvb.h"\n#include <stdio.h>\nint main(void) {' + \
        "".join('printf("%%zu\\n", sizeof(%s));' % n for n in names) + "return 0;}"
    exe = os.path.join(kbuild.BUILD, "page_block_sizes")
    os.makedirs(kbuild.BUILD, exist_ok=True)
    subprocess.run([cc, "-std=c99", "-x", "c", "-I", kbuild.INCLUDE, "-o", exe, "-"], input=src.encode(), check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(getattr(kvb, n)) for n in names]


@pytest.mark.parametrize("seed", range(30))
def test_whole_units_are_taken_once(host, seed):
    rng = random.Random(1000 + seed)
    picked = seed % 2
    cut(host, rng, rng.choice((1, 7, 60)), rng.choice((1, 3)), rng.choice((0, 1, 90)), 0 if picked else rng.choice((0, 3)), 70, rng.choice((1, 8)),
        rng.choice((1, 4, 5)), rng.choice((1, 16, 17)), rng.choice((1, 9)) if picked else 0, 16, 64, 1, 0, 1, joined=0 if picked else 1, whole=1)
