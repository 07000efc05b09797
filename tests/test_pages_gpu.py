"""kv_attend_shared, kv_bound, kv_select and kv_attend_selected against plain implementations in 64 bits
(pages_ref.py, where the tolerances are derived)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import pages_ref as ref  # noqa: E402
from hierarchical_kv_cache_backup_gb300 import kvb  # noqa: E402
from pages_ref import Batch  # noqa: E402

NHD, HND = dict(T=16), dict(T=17, page_first=True, hnd=True, offset=48)


def no_status(b):
    assert int(b.status) == 0


# ------------------------------------------------------------ shared prefixes

@pytest.mark.parametrize("fmt,dtype", [("same", "bf16"), ("same", "fp16"), ("e4m3", "bf16"), ("e4m3", "fp16")])
@pytest.mark.parametrize("dim,H,group", [(128, 2, 4), (64, 3, 1), (96, 1, 8), (192, 2, 3), (256, 2, 5)])
@pytest.mark.parametrize("page", [NHD, HND, dict(T=1, hnd=True), dict(T=64, page_first=True)])
def test_few_rows(fmt, dtype, dim, H, group, page):
    """Two requests of a group, one alone, lengths of 0 and 1 among them."""
    with Batch(kvb, [33, 1, 0, 150], [1, 1, 1, 1], [(0, 2, 70)], H, group, dim, fmt, dtype, **page) as b:
        b.run()
        b.check()
        no_status(b)


@pytest.mark.parametrize("fmt,dtype", [("same", "bf16"), ("same", "fp16"), ("e4m3", "bf16"), ("e4m3", "fp16")])
@pytest.mark.parametrize("dim,H,group", [(128, 2, 4), (64, 1, 3), (96, 2, 8), (192, 1, 4), (256, 1, 8)])
@pytest.mark.parametrize("page", [NHD, HND])
def test_many_rows(fmt, dtype, dim, H, group, page):
    """Groups of many query rows, one past a tile of 128 and one past 256; empty requests, groups and prefixes."""
    lens = [5, 0, 40, 1, 100, 63, 64, 65, 2, 30] + [3] * 30
    n_q = [5, 0, 7, 2, 9, 1, 1, 3, 1, 2] + [1] * 30
    with Batch(kvb, lens, n_q, [(0, 5, 130), (5, 5, 40), (5, 8, 0), (8, 40, 301)], H, group, dim, fmt, dtype, **page) as b:
        b.run()
        b.check()
        no_status(b)


@pytest.mark.parametrize("fmt,dtype", [("same", "bf16"), ("same", "fp16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("groups", [(), ((0, 2, 200),), ((0, 1, 64), (1, 3, 130))])
def test_prompt_chunks(fmt, dtype, groups):
    """Requests that fill units on their own: the prefix goes in front of their own tokens."""
    with Batch(kvb, [100, 64, 333], [100, 1, 70], groups, 2, 4, 128, fmt, dtype, **HND) as b:
        b.run()
        b.check()
        no_status(b)


@pytest.mark.parametrize("n_q,lens", [([3, 4], [2, 40]), ([40, 30], [10, 64]), ([80, 90], [3, 200])])
def test_more_new_tokens_than_own(n_q, lens):
    """The first queries of a request that is shorter than they are many see the prefix alone, or nothing."""
    for groups in ((), ((0, 2, 21),)):
        with Batch(kvb, lens, n_q, groups, 1, 4, 64) as b:
            b.run()
            b.check()
            no_status(b)


@pytest.mark.parametrize("dim,dtype,group", [(128, "bf16", 2), (64, "fp16", 8), (256, "bf16", 1)])
def test_long(dim, dtype, group):
    """Long prefixes and requests: all the parallelism lies along the tokens."""
    with Batch(kvb, [9001, 20], [1, 1], [(0, 2, 12345)], 2, group, dim, "same", dtype, T=64) as b:
        b.run()
        b.check()
    with Batch(kvb, [9001], [20], [(0, 1, 5000)], 2, group, dim, "same", dtype, T=64) as b:
        b.run()
        b.check()


@pytest.mark.parametrize("n", [1, 5])
@pytest.mark.parametrize("groups", [(), ((0, 100, 50), (100, 140, 33))])
def test_more_segments_than_a_table(n, groups):
    """What comes before each request is then summed by a kernel of its own."""
    lens = [7 + 3 * (i % 20) for i in range(150)]
    with Batch(kvb, lens, [1 + i % n for i in range(150)], groups, 1, 4, 64, T=8) as b:
        b.run()
        b.check()
        no_status(b)


@pytest.mark.parametrize("fmt,dtype,dim", [("same", "bf16", 64), ("same", "fp16", 96), ("same", "bf16", 128), ("e4m3", "bf16", 192), ("e4m3", "fp16", 256)])
@pytest.mark.parametrize("lens,n_q,groups,H,group", [
    ([400, 350], [300, 280], (), 4, 9), ([400, 350], [300, 280], ((0, 2, 150),), 4, 9),          # a token's rows in two row tiles
    ([5 + 3 * i for i in range(40)], [20] * 40, ((0, 25, 200), (25, 40, 90)), 8, 5),             # prefix and own tokens apart
    ([7 + i % 40 for i in range(300)], [3] * 300, ((0, 300, 2000),), 8, 4),                      # few own rows, many requests
    ([30, 90], [90, 110], ((0, 1, 100),), 1, 150)])                                              # a token of more rows than a tile
def test_more_rows_than_places(fmt, dtype, dim, lens, n_q, groups, H, group):
    """So many rows that a warp of the join takes several."""
    with Batch(kvb, lens, n_q, groups, H, group, dim, fmt, dtype, T=16) as b:
        b.run()
        b.check()
        no_status(b)


@pytest.mark.parametrize("sign", [-1.0, 0.0])
@pytest.mark.parametrize("n_q", [1, 40])
def test_scale_signs(sign, n_q):
    with Batch(kvb, [60, 70], [n_q, n_q], [(0, 2, 50)], 1, 4, 128) as b:
        b.scale *= sign
        b.run()
        b.check()


@pytest.mark.parametrize("n_q", [1, 40])
@pytest.mark.parametrize("loud", [30.0, 1e-4])
def test_score_ranges(n_q, loud):
    for fmt, dtype in (("same", "bf16"), ("same", "fp16"), ("e4m3", "bf16")):
        if fmt == "e4m3" and loud > 1:
            continue                     # past what fp8 holds
        with Batch(kvb, [600, 70], [n_q, n_q], [(0, 2, 500)], 1, 4, 128, fmt, dtype, loud=loud) as b:
            b.run()
            b.check()


@pytest.mark.parametrize("mul", [1e-20, 1e20, 1e-37])
def test_query_ranges_of_fp8_pages(mul):
    """A bf16 query is scaled by rows before it meets fp8 keys."""
    for n_q in (1, 20):
        with Batch(kvb, [60], [n_q], [(0, 1, 90)], 1, 4, 64, "e4m3") as b:
            b.q = (b.q.float() * mul).to(torch.bfloat16)
            b.scale = 0.1 / mul if mul != 1e-37 else 1e36
            b.run()
            b.check()


@pytest.mark.parametrize("n_q", [1, 3, 40])
def test_maxima_that_rise_late(n_q):
    """Scores that grow along the tokens: the running maximum moves again and again."""
    with Batch(kvb, [700], [n_q], [(0, 1, 900)], 1, 4, 128) as b:
        for table, n, start in ((b.prefix_table[0], 900, 0), (b.table[0], 700, 900)):
            x = b.q[:1, :1].float() * (0.002 * (start + torch.arange(n, device="cuda")[:, None, None]))
            b.p.put(table, x.expand(n, 1, 128), 0)
        b.run()
        b.check()


# ----------------------------------------------------- values that are not finite

BAD = {"same": [float("inf"), -float("inf"), float("nan")], "e4m3": [float("nan")]}


@pytest.mark.parametrize("fmt,dtype", [("same", "bf16"), ("same", "fp16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("n_q", [3, 20, 90])
@pytest.mark.parametrize("comp", [0, 1])
@pytest.mark.parametrize("dim", [64, 96, 128])
def test_not_finite_behind_the_mask(fmt, dtype, n_q, comp, dim):
    """A key or value that is not finite reaches the queries that see it, a value its own dim alone."""
    for bad in BAD[fmt]:
        with Batch(kvb, [150], [n_q], [(0, 1, 30)], 2, 4, dim, fmt, dtype, T=16) as b:
            b.run()
            want, wl = b.out.clone(), b.lse.clone()
            at, h, d = 150 - n_q + n_q // 2, 1, 37                   # query n_q // 2 is the first that sees it
            page = b.table[0, at // 16].long()
            words = torch.tensor([bad], device="cuda", dtype=torch.float32)
            word = words.to(torch.float8_e4m3fn) if fmt == "e4m3" else words.to(b.p.dt)
            size = b.p.B // dim
            b.p.view(comp)[page, at % 16, h, d * size:(d + 1) * size] = word.view(torch.uint8)
            b.run()
            got, gl = b.out[:n_q], b.lse[:n_q]
            first, heads = n_q // 2, slice(4, 8)
            clean = torch.ones_like(got, dtype=torch.bool)
            clean[first:, heads] = False
            assert torch.equal(got[clean], want[:n_q][clean])
            assert torch.equal(gl[:first], wl[:first]) and torch.equal(gl[:, :4], wl[:n_q, :4])
            hit = got[first:, heads]
            if comp == 1:
                assert not torch.isfinite(hit[..., d]).any()
                rest = [x for x in range(dim) if x != d]
                assert torch.equal(hit[..., rest], want[first:n_q, heads][..., rest])
                assert torch.equal(gl, wl[:n_q])
            elif np.isnan(bad):
                assert torch.isnan(hit).all() and torch.isnan(gl[first:, heads]).all()


@pytest.mark.parametrize("n_q", [1, 3, 20])
def test_stale_bytes_past_the_length(n_q):
    """All that lies past a length, in the last page and in the others, may hold anything."""
    with Batch(kvb, [21], [n_q], [(0, 1, 37)], 1, 2, 64, T=16) as b:
        for comp in (0, 1):
            held = [(b.p.held(t, n, comp), t, n) for t, n in ((b.table[0], 21), (b.prefix_table[0], 37))]
            b.p.view(comp).copy_(torch.full((1, 1, 1, 1), 255, dtype=torch.uint8, device="cuda").expand(b.p.view(comp).shape))   # NaN
            for x, t, n in held:
                b.p.put(t, torch.from_numpy(x).cuda().float(), comp)
        b.run()
        b.check()


@pytest.mark.parametrize("n_q", [3, 40])
def test_a_query_of_nan_stays_in_its_row(n_q):
    with Batch(kvb, [90], [n_q], [(0, 1, 70)], 1, 4, 128) as b:
        b.run()
        want = b.out.clone()
        b.q[1, 2, 5] = float("nan")
        b.run()
        assert torch.isnan(b.out[1, 2]).all() and torch.isnan(b.lse[1, 2])
        clean = torch.ones_like(b.out, dtype=torch.bool)
        clean[1, 2] = False
        assert torch.equal(b.out[clean], want[clean])


# -------------------------------------------------- what only the GPU sees

@pytest.mark.parametrize("fmt", ["same", "e4m3"])
@pytest.mark.parametrize("n_q", [1, 20, 90])
def test_bad_pages(fmt, n_q):
    """Queries that see a page outside the pool get NaN, the others what they would."""
    for where in ("own", "prefix"):
        with Batch(kvb, [100, 100], [n_q, n_q], [(0, 1, 60), (1, 2, 60)], 1, 4, 128, fmt, T=16) as b:
            b.run()
            want = b.out.clone()
            if where == "own":
                b.table[0, 6] = b.p.P                    # its tokens 96..99
            else:
                b.prefix_table[0, 1] = -1
            b.run()
            assert int(b.status) == kvb.KV_STATUS_BAD_PAGE
            first = max(0, 96 - (100 - n_q)) if where == "own" else 0
            assert torch.isnan(b.out[first:n_q]).all()
            assert torch.equal(b.out[:first], want[:first]) and torch.equal(b.out[n_q:2 * n_q], want[n_q:2 * n_q])


def test_pages_outside_a_length_are_not_looked_at():
    with Batch(kvb, [20, 90], [1, 1], [(0, 2, 30)], 1, 4, 64, T=16) as b:
        b.table[0, 2:] = 10 ** 9
        b.run()
        b.check()
        no_status(b)


@pytest.mark.parametrize("n_q", [1, 20, 70])
def test_bad_lengths_and_groups(n_q):
    def batch():
        return Batch(kvb, [40, 50, 60, 70], [n_q] * 4, [(0, 2, 33), (2, 4, 44)], 1, 4, 64, T=16)

    with batch() as b:
        b.run()
        want = b.out.clone()
    # a length past max_len is taken as that; a request out of order is left out
    with batch() as b:
        a = b.shared_args()
        b.d_lens[3] = 10 ** 6
        b.q_start[1] = 3 * n_q                           # requests 0 (too many) and 1 (backwards)
        kvb.kv_attend_shared(b.p.pool, a)
        torch.cuda.synchronize()
        assert int(b.status) == kvb.KV_STATUS_BAD_LENGTH
        assert torch.equal(b.out[2 * n_q:], want[2 * n_q:]) and (b.out[:2 * n_q] == 7).all()
    with batch() as b:
        a = b.shared_args()
        b.prefix_lens[1] = -5                            # as 0
        kvb.kv_attend_shared(b.p.pool, a)
        torch.cuda.synchronize()
        assert int(b.status) == kvb.KV_STATUS_BAD_LENGTH and torch.equal(b.out[:2 * n_q], want[:2 * n_q])
        b.groups[1] = (2, 4, 0)
        b.check()
    for starts in ([0, 9, 4], [0, 2, 70], [-1, 2, 4]):   # a group out of order has no prefix
        with batch() as b:
            a = b.shared_args()
            b.group_start.copy_(torch.tensor(starts, dtype=torch.int32))
            kvb.kv_attend_shared(b.p.pool, a)
            torch.cuda.synchronize()
            assert int(b.status) == kvb.KV_STATUS_BAD_LENGTH
            keep = {(0, 2, 70): [(0, 2, 33)], (-1, 2, 4): [(2, 4, 44)]}.get(tuple(starts), [])
            table = b.prefix_table
            if keep == [(2, 4, 44)]:
                b.prefix_table = table[1:]
            b.groups = keep
            b.check()
            b.prefix_table = table


def test_requests_that_share_query_tokens():
    """More work than valid ranges can make: nothing is done, and said so."""
    with Batch(kvb, [200] * 40, [1] * 40, (), 1, 4, 64) as b:
        b.q_start.copy_(torch.tensor([40 * (i % 2) for i in range(41)], dtype=torch.int32))
        a = b.shared_args(max_q=40)
        kvb.kv_attend_shared(b.p.pool, a)
        torch.cuda.synchronize()
        assert int(b.status) & kvb.KV_STATUS_BAD_LENGTH


# ------------------------------------------------ strides, streams, graphs

def test_strides_and_streams():
    with Batch(kvb, [100, 90], [3, 20], [(0, 2, 80)], 2, 4, 128) as b:
        b.run()
        want = b.out[:b.tokens].clone()
        wide, out = torch.zeros(b.tokens, 20, 128, dtype=torch.bfloat16, device="cuda"), torch.full((b.tokens, 12, 160), 3.0, dtype=torch.bfloat16, device="cuda")
        wide[:, 4:12] = b.q
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        b.run(stream.cuda_stream, q=wide[:, 4:12], out=out[:, 2:10, :128])
        assert torch.equal(out[:, 2:10, :128], want)
        out[:, 2:10, :128] = 3.0
        assert (out == 3.0).all()


def test_without_logarithms_and_status():
    for n_q in (1, 30):
        with Batch(kvb, [100], [n_q], [(0, 1, 80)], 1, 4, 128) as b:
            b.run()
            want = b.out.clone()
            b.lse.fill_(7.0)
            b.run(lse=None, status=None)
            assert torch.equal(b.out, want) and (b.lse == 7.0).all()


@pytest.mark.parametrize("n", [1, 200])
def test_calls_of_whole_units(n):
    """Short calls: a block a request and head, which needs no workspace where the requests are few; rows that see nothing too."""
    lens = [3 * (i % 9) for i in range(n)]
    with Batch(kvb, lens, [1 + i % 2 for i in range(n)], [(0, n, 40)], 2, 4, 128) as b:
        assert (b.shared_args().workspace_bytes == 0) == (n <= 100)
        b.run()
        b.check()
    with Batch(kvb, lens, [1 + i % 2 for i in range(n)], (), 2, 4, 64, "e4m3") as b:
        b.run()
        b.check()


def test_two_graphs_on_one_workspace():
    """Captured calls read their inputs again, and leave nothing in the workspace that the next would trip over."""
    with Batch(kvb, [100, 20, 60], [1, 1, 1], [(0, 3, 300)], 2, 8, 128) as b, Batch(kvb, [70], [30], (), 2, 4, 128, seed=9) as c:
        args = [(b, b.shared_args()), (c, c.shared_args())]
        work = torch.randint(0, 256, (max(x.workspace_bytes for _, x in args),), dtype=torch.uint8, device="cuda")
        side, graphs = torch.cuda.Stream(), []
        for z, x in args:
            x.workspace, x.workspace_bytes = work.data_ptr(), work.numel()
            kvb.kv_attend_shared(z.p.pool, x)
            torch.cuda.synchronize()
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=side):
                kvb.kv_attend_shared(z.p.pool, x, side.cuda_stream)
        for k in range(4):
            for (z, _), graph in zip(args, graphs):
                z.q.copy_(torch.randn(z.q.shape, generator=z.gen, device="cuda"))
                z.out.fill_(7.0)
                graph.replay()
            torch.cuda.synchronize()
            for z, _ in args:
                z.check()


def test_far_offsets():
    """A pool past 4 GiB, and pages at its end."""
    for fmt, n_q in (("same", 1), ("same", 20), ("e4m3", 20)):
        H, T, dim = 8, 64, 128
        P = (5 << 30) // (2 * T * H * dim * (1 if fmt == "e4m3" else 2)) + 1
        with Batch(kvb, [130], [n_q], [(0, 1, 100)], H, 2, dim, fmt, T=T, spare=P - 5, L=1, page_first=n_q == 1) as b:
            for table in (b.table, b.prefix_table):
                old = [[b.p.held(t, n, c, 0) for c in (0, 1)] for t, n in ((table[0], 130 if table is b.table else 100),)]
                table[0] = torch.tensor([P - 1, P // 2, P - 2] if table is b.table else [P - 3, P // 2 + 1], device="cuda")
                for c in (0, 1):
                    b.p.put(table[0], torch.from_numpy(old[0][c]).cuda().float() / (b.p.v_scale if c else b.p.k_scale), c, 0)
            b.run()
            b.check()


def refused(status, call, args, **kw):
    args = type(args).from_buffer_copy(args)
    for name, val in kw.items():
        setattr(args, name, val)
    with pytest.raises(kvb.KvError) as e:
        call(args)
    assert e.value.status == status, (kw, e.value)


INV, LAY, OOR, ALI = kvb.KV_ERR_INVALID_ARG, kvb.KV_ERR_LAYOUT, kvb.KV_ERR_OUT_OF_RANGE, kvb.KV_ERR_ALIGNMENT


def test_shared_refusals():
    with Batch(kvb, [100, 64], [2, 1], [(0, 2, 50)], 2, 2, 64) as b:
        a, call = b.shared_args(), lambda x: kvb.kv_attend_shared(b.p.pool, x)
        cpu = torch.zeros(64, dtype=torch.int32)
        for kw, status in [(dict(layer=2), OOR), (dict(head_dim=32), LAY), (dict(head_dim=96), LAY), (dict(head_dim=60), INV),
                           (dict(dtype=2), INV), (dict(format=kvb.KV_CACHE_Q4), INV), (dict(format=kvb.KV_CACHE_E4M3), LAY), (dict(q_heads=3), INV), (dict(q_heads=0), INV),
                           (dict(max_q=9), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
                           (dict(max_len=2 ** 29 + 1, pages_stride=2 ** 31), INV), (dict(max_prefix=2 ** 29 + 1, prefix_stride=2 ** 31), INV),
                           (dict(groups=65536), INV), (dict(requests=65536), INV), (dict(lens=None), INV), (dict(q_start=None), INV), (dict(pages=None), INV),
                           (dict(group_start=None), INV), (dict(prefix_lens=None), INV), (dict(prefix_pages=None), INV),
                           (dict(pages_stride=6), INV), (dict(q=kvb.kv_vecs(0, 128, 64)), INV), (dict(reserved=1), INV),
                           (dict(out=kvb.kv_vecs(b.out.data_ptr() + 2, 256, 64)), ALI), (dict(lse=b.lse.data_ptr() + 2), ALI),
                           (dict(pages=cpu.data_ptr()), INV), (dict(lens=cpu.data_ptr()), INV), (dict(prefix_pages=cpu.data_ptr()), INV),
                           (dict(workspace=a.workspace + 8), ALI)]:
            refused(status, call, a, **kw)
        torch.cuda.synchronize()
        assert (b.out == 7).all()
        for kw in (dict(requests=0), dict(tokens=0, max_q=0), dict(max_q=0)):
            n0 = kvb.kv_launch_count()
            kvb.kv_attend_shared(b.p.pool, b.shared_args(**kw))
            assert kvb.kv_launch_count() == n0
    for n_q in (1, 20):
        with Batch(kvb, [9000], [n_q], [(0, 1, 9000)], 1, 2, 64) as b:
            a, call = b.shared_args(), lambda x: kvb.kv_attend_shared(b.p.pool, x)
            assert a.workspace_bytes > 0
            refused(INV, call, a, workspace=None)
            refused(OOR, call, a, workspace_bytes=a.workspace_bytes - 1)
    with Batch(kvb, [0, 0], [2, 1], (), 1, 2, 64) as b:          # no cached token anywhere, no page table
        kvb.kv_attend_shared(b.p.pool, b.shared_args(max_len=0, pages=None))
        torch.cuda.synchronize()
        assert not b.out.any() and torch.isneginf(b.lse).all()
        no_status(b)


# --------------------------------------------------------------------- bounds

def bound(b, first=None, max_new=None, buffer=None, layer=1, **kw):
    buffer = torch.full((b.p.P, b.H, ref.record_bytes(b.dim)), 99, dtype=torch.uint8, device="cuda") if buffer is None else buffer
    f = torch.tensor(first, dtype=torch.int32, device="cuda") if first is not None else None
    a = kvb.make_bound_args(buffer.data_ptr(), lens=b.d_lens.data_ptr(), first=f.data_ptr() if f is not None else None, pages=b.table.data_ptr(),
                            pages_stride=b.per, requests=len(b.lens), max_len=max(b.lens), max_new=max(b.lens) if max_new is None else max_new,
                            head_dim=b.dim, dtype=b.p.dtype, format=b.p.format, layer=layer, status=b.status.data_ptr())
    for name, val in kw.items():
        setattr(a, name, val)
    kvb.kv_bound(b.p.pool, a)
    torch.cuda.synchronize()
    return buffer


def check_bounds(b, buffer, first):
    """All records, bit for bit: those of touched pages from their keys, the others as they were."""
    got, touched = buffer.cpu().numpy(), set()
    for i, n in enumerate(b.lens):
        x = b.p.held(b.table[i], n, 0) / b.p.k_scale
        for j in range(first[i] // b.p.T, -(-n // b.p.T)) if first[i] < n else ():
            page = int(b.table[i, j])
            touched.add(page)
            assert np.array_equal(got[page], ref.record(*ref.bounds_of(x[j * b.p.T:(j + 1) * b.p.T]))), (i, j)
    rest = [p for p in range(b.p.P) if p not in touched]
    assert (got[rest] == 99).all()


@pytest.mark.parametrize("fmt,dtype", [("same", "bf16"), ("same", "fp16"), ("e4m3", "bf16"), ("e4m3", "fp16")])
@pytest.mark.parametrize("dim,H", [(64, 3), (96, 2), (128, 8), (192, 1), (256, 2)])
@pytest.mark.parametrize("page", [NHD, HND, dict(T=1), dict(T=64, hnd=True)])
def test_bounds(fmt, dtype, dim, H, page):
    lens = [33, 0, 1, 150, 64]
    with Batch(kvb, lens, [1] * 5, (), H, 1, dim, fmt, dtype, loud=3.0, **page) as b:
        check_bounds(b, bound(b), [0] * 5)
        first = [32, 0, 1, 17, 63]
        check_bounds(b, bound(b, first, max_new=133), first)
        no_status(b)


def test_bounds_of_special_values():
    with Batch(kvb, [16, 16, 16, 16], [1] * 4, (), 1, 1, 64, T=16) as b:
        x = torch.randn(16, 1, 64, generator=b.gen, device="cuda")
        special = [x.clone() for _ in range(4)]
        special[0][3, 0, 5] = float("nan")
        special[0][3, 0, 40] = -float("inf")
        special[1][:] = 0.0
        special[1][2, 0, 33] = 2.0 ** -101
        special[2][:] = 127.0 * 2.0 ** -9                 # codes of 127 exactly
        special[2][1] = -127.0 * 2.0 ** -9
        special[3][:, :, :32] *= 1e38 / 4
        special[3][:, :, 32:] *= 1e-30
        for i in range(4):
            b.p.put(b.table[i], special[i], 0)
        got = bound(b)
        check_bounds(b, got, [0] * 4)
        lo, hi, s = ref.parts(got[b.table[:, 0].long()].cpu().numpy(), 64)
        assert np.isinf(s[0]).all() and not lo[0].any() and not s[1].any()
        assert (hi[2] == 127).all() and (lo[2] == -127).all()


def test_bounds_left_out():
    with Batch(kvb, [40, 50, 60, 70], [1] * 4, (), 1, 1, 64, T=16) as b:
        b.d_lens[1] = 71                                   # past max_len
        got = bound(b, [0, 0, 61, 0])                      # behind its length
        assert int(b.status) == kvb.KV_STATUS_BAD_LENGTH
        assert (got[b.table[1].long()] == 99).all() and (got[b.table[2].long()] == 99).all()
        b.status.zero_()
        b.d_lens[1] = 50
        got = bound(b, [0, 0, 0, 5], max_new=64)           # request 3 has 65 new tokens
        assert int(b.status) == kvb.KV_STATUS_BAD_LENGTH and (got[b.table[3].long()] == 99).all()
        b.status.zero_()
        b.table[0, 1] = b.p.P
        b.table[2, 0] = -7
        bound(b)
        assert int(b.status) == kvb.KV_STATUS_BAD_PAGE


def test_bound_refusals():
    with Batch(kvb, [40], [1], (), 1, 1, 64, T=16) as b:
        for kw, status in [(dict(layer=2), OOR), (dict(head_dim=32), LAY), (dict(head_dim=128), LAY), (dict(format=2), INV), (dict(dtype=2), INV),
                           (dict(max_new=41), INV), (dict(lens=None), INV), (dict(bounds=None), INV), (dict(pages=None), INV), (dict(reserved=1), INV),
                           (dict(bounds=b.out.data_ptr() + 8), ALI), (dict(requests=65536), INV)]:
            with pytest.raises(kvb.KvError) as e:
                bound(b, **kw)
            assert e.value.status == status, kw
        n0 = kvb.kv_launch_count()
        bound(b, requests=0)
        bound(b, max_new=0)
        assert kvb.kv_launch_count() == n0
    with pytest.raises(kvb.KvError):
        kvb.kv_bound_bytes(32)
    assert [kvb.kv_bound_bytes(d) for d in (64, 96, 128, 192, 256)] == [ref.record_bytes(d) for d in (64, 96, 128, 192, 256)]


def test_sizes_whose_products_pass_64_bits():
    """Counts that are in range one by one, and whose blocks or bytes are not."""
    with Batch(kvb, [4], [1], (), 64, 1, 64, T=1) as b:
        bounds, picks = bound(b), torch.zeros(1, 64, 1, dtype=torch.int32, device="cuda")
        big = dict(tokens=2 ** 30, max_len=2 ** 29, pages_stride=2 ** 29)
        a = select_args(b, bounds, picks, 1)
        for call in (lambda x: kvb.kv_select(b.p.pool, x), lambda x: kvb.kv_select_workspace(b.p.pool, x)):
            refused(INV, call, a, **big)
        a, s = b.shared_args(), b.selected_args(picks)
        for call, x in ((kvb.kv_attend_shared_workspace, a), (kvb.kv_attend_shared, a), (kvb.kv_attend_selected_workspace, s)):
            refused(INV, lambda y: call(b.p.pool, y), x, tokens=2 ** 30, max_q=65535, max_len=2 ** 29, pages_stride=2 ** 29)
        s.tokens = 2 ** 30                              # more units than a launch has blocks: cut in shares
        assert kvb.kv_attend_selected_workspace(b.p.pool, s) > 2 ** 36
        for kw in (dict(tokens=65535, max_q=65535, max_len=131072), dict(tokens=1 << 20, max_q=1, max_len=1 << 20, requests=65535)):
            for key, value in kw.items():
                setattr(a, key, value)
            assert kvb.kv_attend_shared_workspace(b.p.pool, a) >= 0


# ------------------------------------------------------------------ selection

def select_args(b, bounds, picks, budget, **kw):
    a = kvb.make_select_args(bounds.data_ptr(), kvb.vecs(b.q[:b.tokens]), picks.data_ptr(), q_start=b.q_start.data_ptr(), lens=b.d_lens.data_ptr(),
                             pages=b.table.data_ptr(), pages_stride=b.per, requests=len(b.lens), tokens=b.tokens, max_q=max(b.n_q), max_len=max(b.lens),
                             q_heads=b.H * b.group, head_dim=b.dim, dtype=b.p.dtype, budget=budget, status=b.status.data_ptr(), **kw)
    return b.space(a, kvb.kv_select_workspace(b.p.pool, a))


def select(b, bounds, budget, **kw):
    picks = torch.full((b.tokens, b.H, budget), 77, dtype=torch.int32, device="cuda")
    kvb.kv_select(b.p.pool, select_args(b, bounds, picks, budget, **kw))
    torch.cuda.synchronize()
    return picks


def check_picks(b, bounds, picks, budget, keep_first=0, keep_last=0):
    lo, hi, s = ref.parts(bounds.cpu().numpy(), b.dim)
    q, got = b.q.double().cpu().numpy(), picks.cpu().numpy()
    for i, a, n, _ in b.rows():
        for k in range(n):
            pos = b.lens[i] - n + k
            seen = pos // b.p.T + 1 if pos >= 0 else 0
            pages = b.table[i, :seen].cpu().numpy()
            for h in range(b.H):
                score = ref.scores(q[a + k, h * b.group:(h + 1) * b.group], lo[pages, h], hi[pages, h], s[pages, h]) if seen else []
                want = ref.select(score, budget, keep_first, keep_last)
                assert got[a + k, h].tolist() == want, (i, k, h)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,H,group", [(64, 2, 4), (96, 1, 5), (128, 3, 1), (192, 2, 8), (256, 1, 9)])
def test_select(dtype, dim, H, group):
    lens, n_q = [300, 0, 1, 77, 40, 500], [1, 1, 1, 3, 0, 2]
    with Batch(kvb, lens, n_q, (), H, group, dim, "same", dtype, T=4) as b:
        bounds = bound(b)
        for budget, first, last in ((7, 0, 0), (20, 1, 2), (5, 2, 3), (1, 0, 1), (200, 3, 1)):
            check_picks(b, bounds, select(b, bounds, budget, keep_first=first, keep_last=last), budget, first, last)
        no_status(b)


@pytest.mark.parametrize("pages", [2049, 9000, 40000])
def test_select_of_many_pages(pages):
    """Rows that 1,024 threads take, some longer than their registers hold."""
    with Batch(kvb, [pages, pages // 3], [1, 1], (), 1, 2, 64, T=1) as b:
        bounds = bound(b)
        for budget in (1, 64, 1500):
            check_picks(b, bounds, select(b, bounds, budget, keep_first=1), budget, 1)


@pytest.mark.parametrize("kinds", [1, 2, 40])
@pytest.mark.parametrize("pages", [300, 3000])
def test_select_ties(kinds, pages):
    """Pages that are copies of a few: ties go to the lowest index."""
    with Batch(kvb, [pages], [1], (), 2, 2, 64, T=1) as b:
        bounds = bound(b)
        few = bounds[b.table[0, :kinds].long()]
        bounds[b.table[0].long()] = few[torch.randint(0, kinds, (pages,), generator=b.gen, device="cuda")]
        for budget in (1, 33, 299):
            check_picks(b, bounds, select(b, bounds, budget, keep_first=2 if budget > 5 else 0), budget, 2 if budget > 5 else 0)


def test_select_not_finite():
    """A page whose score is not finite counts as the largest; a query of NaN leaves the first pages."""
    with Batch(kvb, [64], [1], (), 2, 2, 64, T=1) as b:
        x = torch.randn(64, 2, 64, generator=b.gen, device="cuda")
        x[50, 0, 3], x[60, 0, 40], x[20, 1, 0] = float("nan"), float("inf"), -float("inf")
        b.p.put(b.table[0], x, 0)
        bounds = bound(b)
        picks = select(b, bounds, 2)
        check_picks(b, bounds, picks, 2)
        assert picks[0, 0].tolist() == [50, 60] and 20 in picks[0, 1].tolist()
        b.q[0, 0, 0] = float("nan")
        picks = select(b, bounds, 5)
        check_picks(b, bounds, picks, 5)
        assert picks[0, 0].tolist() == [0, 1, 2, 3, 4]


def test_select_left_out():
    with Batch(kvb, [100, 100, 100], [2, 2, 2], (), 1, 2, 64, T=4) as b:
        bounds = bound(b)
        want = select(b, bounds, 6)
        picks = torch.full_like(want, 77)
        a = select_args(b, bounds, picks, 6)
        b.d_lens[1] = 101
        kvb.kv_select(b.p.pool, a)
        torch.cuda.synchronize()
        assert int(b.status) == kvb.KV_STATUS_BAD_LENGTH
        assert (picks[2:4] == 77).all() and torch.equal(picks[[0, 1, 4, 5]], want[[0, 1, 4, 5]])
        b.status.zero_()
        b.d_lens[1] = 100
        b.table[0, 3] = b.p.P                              # the page is picked last
        got = select(b, bounds, 24)
        assert int(b.status) == kvb.KV_STATUS_BAD_PAGE and not (got[:2] == 3).any() and torch.equal(got[2:], select(b, bounds, 24)[2:])


def test_select_refusals():
    with Batch(kvb, [100], [1], (), 1, 2, 64, T=4) as b:
        bounds = bound(b)
        picks = torch.full((1, 1, 5), 77, dtype=torch.int32, device="cuda")
        a, call = select_args(b, bounds, picks, 5), lambda x: kvb.kv_select(b.p.pool, x)
        for kw, status in [(dict(head_dim=32), LAY), (dict(head_dim=60), INV), (dict(dtype=2), INV), (dict(q_heads=0), INV), (dict(budget=0), INV),
                           (dict(budget=2 ** 24 + 1), INV), (dict(keep_first=6), INV), (dict(keep_first=3, keep_last=3), INV), (dict(keep_last=2 ** 32 - 1, keep_first=3), INV),
                           (dict(max_q=2), INV), (dict(picks=None), INV), (dict(bounds=None), INV), (dict(lens=None), INV), (dict(pages=None), INV), (dict(bounds=a.bounds + 8), ALI),
                           (dict(workspace=None), INV), (dict(workspace_bytes=a.workspace_bytes - 1), OOR), (dict(max_len=2 ** 29 + 1, pages_stride=2 ** 31), INV)]:
            refused(status, call, a, **kw)
        torch.cuda.synchronize()
        assert (picks == 77).all()


# ------------------------------------------------- attention over what is selected

def run_selected(b, picks, **kw):
    kvb.kv_attend_selected(b.p.pool, b.selected_args(picks, **kw))
    torch.cuda.synchronize()


def check_selected(b, picks):
    q, out, lse = (x.double().cpu().numpy() for x in (b.q, b.out, b.lse))
    T = b.p.T
    for i, a, n, _ in b.rows():
        k, v = (b.p.held(b.table[i], b.lens[i], c) for c in (0, 1))
        for r in range(n):
            pos = b.lens[i] - n + r
            seen_pages = pos // T + 1 if pos >= 0 else 0
            for h in range(b.H):
                at = [p * T + t for p in picks[a + r, h].tolist() if 0 <= p < seen_pages for t in range(T) if p * T + t <= pos]
                one = np.ones((1, 1, len(at)), bool)
                heads = slice(h * b.group, (h + 1) * b.group)
                sub = Batch.__new__(Batch)
                sub.H, sub.group, sub.scale, sub.p = 1, b.group, b.scale, b.p
                sub.check_rows(q[a + r:a + r + 1, heads], k[at, h:h + 1], v[at, h:h + 1], one, out[a + r:a + r + 1, heads], lse[a + r:a + r + 1, heads], False)


def some_picks(b, budget, holes=True):
    picks = torch.full((b.tokens, b.H, budget), -1, dtype=torch.int32)
    for i, a, n, _ in b.rows():
        for r in range(n):
            seen = max(0, (b.lens[i] - n + r) // b.p.T + 1)
            for h in range(b.H):
                some = torch.randperm(seen)[:budget].sort().values.int()
                picks[a + r, h, :len(some)] = some
                if holes and len(some) > 2:
                    picks[a + r, h, 1] = -1
    return picks.cuda()


@pytest.mark.parametrize("dim,H,group,budget", [(128, 2, 17, 20), (64, 1, 40, 90)])
def test_selected_more_rows_than_places(dim, H, group, budget):
    """So many rows that a warp of the join takes several; heads of a group in two and three row tiles."""
    with Batch(kvb, [900, 700], [310, 290], (), H, group, dim, T=8) as b:
        picks = some_picks(b, budget)
        run_selected(b, picks)
        check_selected(b, picks)
        no_status(b)


@pytest.mark.parametrize("fmt,dtype", [("same", "bf16"), ("same", "fp16"), ("e4m3", "bf16"), ("e4m3", "fp16")])
@pytest.mark.parametrize("dim,H,group", [(128, 2, 4), (64, 3, 1), (96, 1, 8), (192, 1, 16), (256, 2, 17), (64, 1, 40)])
@pytest.mark.parametrize("page", [NHD, HND, dict(T=1, page_first=True), dict(T=64, hnd=True)])
def test_selected(fmt, dtype, dim, H, group, page):
    with Batch(kvb, [150, 1, 0, 333], [1, 1, 1, 4], (), H, group, dim, fmt, dtype, **page) as b:
        for budget in (1, 3, 9):
            torch.manual_seed(budget)
            picks = some_picks(b, budget)
            b.out.fill_(7.0)
            run_selected(b, picks)
            check_selected(b, picks)
        no_status(b)


def test_selected_long():
    """Long lists of one request, and many requests: pieces joined, more segments than a table holds."""
    with Batch(kvb, [20000], [1], (), 2, 4, 128, T=16) as b:
        picks = some_picks(b, 700)
        run_selected(b, picks)
        check_selected(b, picks)
    with Batch(kvb, [90 + i % 50 for i in range(140)], [1] * 140, (), 1, 4, 64, T=16) as b:
        picks = some_picks(b, 4)
        run_selected(b, picks)
        check_selected(b, picks)


def test_selected_entries():
    """-1 is skipped, an index outside what the query sees too and said so, one that stands twice counts twice."""
    with Batch(kvb, [100], [1], (), 1, 2, 64, T=16) as b:
        picks = torch.tensor([[[2, -1, 2, 5]]], dtype=torch.int32, device="cuda")
        run_selected(b, picks)
        check_selected(b, picks)
        no_status(b)
        want = b.out.clone()
        for bad in (7, -2, 2 ** 31 - 1, -2 ** 31):
            picks[0, 0, 1] = bad
            run_selected(b, picks)
            assert int(b.status) == kvb.KV_STATUS_BAD_PAGE and torch.equal(b.out, want), bad
            b.status.zero_()
        picks.fill_(-1)
        run_selected(b, picks)
        assert not b.out.any() and torch.isneginf(b.lse).all()
        b.table[0, 2] = b.p.P
        picks[0, 0, 0] = 2
        run_selected(b, picks)
        assert int(b.status) == kvb.KV_STATUS_BAD_PAGE and torch.isnan(b.out).all()


def test_selected_stale_bytes():
    """Tokens of a picked page that the query does not see may hold anything."""
    for n_q in (1, 3):
        with Batch(kvb, [40], [n_q], (), 1, 2, 64, T=16) as b:
            picks = torch.tensor([[[0, 2]]] * n_q, dtype=torch.int32, device="cuda")
            run_selected(b, picks)
            want = b.out.clone()
            for comp in (0, 1):
                b.p.view(comp)[b.table[0, 2].long(), 8:] = 255
            run_selected(b, picks)
            assert torch.equal(b.out, want)


def test_selected_refusals():
    with Batch(kvb, [9000], [2], (), 1, 2, 64) as b:
        picks = some_picks(b, 500)
        a, call = b.selected_args(picks), lambda x: kvb.kv_attend_selected(b.p.pool, x)
        for kw, status in [(dict(layer=2), OOR), (dict(budget=0), INV), (dict(budget=2 ** 24 + 1), INV), (dict(picks=None), INV), (dict(picks=a.picks + 2), ALI),
                           (dict(head_dim=128), LAY), (dict(scale=float("inf")), INV), (dict(format=kvb.KV_CACHE_Q4), INV), (dict(pages=None), INV),
                           (dict(workspace=None), INV), (dict(workspace_bytes=a.workspace_bytes - 1), OOR), (dict(reserved=1), INV)]:
            refused(status, call, a, **kw)
        torch.cuda.synchronize()
        assert (b.out == 7).all()


# ------------------------------------------------------------ as they are used

@pytest.mark.parametrize("fmt", ["same", "e4m3"])
def test_a_decode_loop_over_selected_pages(fmt):
    """Append, bounds, selection and attention of a step in one graph, over a cache that grows by a token a
    step; with a budget of all pages it is attention over all of them (kv_attend_shared)."""
    H, group, dim, T, n, start, steps = 2, 4, 128, 8, 3, 50, 20
    with Batch(kvb, [start + steps] * n, [1] * n, (), H, group, dim, fmt, T=T) as b:
        p = b.p
        kv = torch.zeros(n, 2, H, dim, dtype=torch.bfloat16, device="cuda")
        slots = torch.zeros(n, dtype=torch.int64, device="cuda")
        first = torch.zeros(n, dtype=torch.int32, device="cuda")
        bounds = torch.zeros(p.P, H, ref.record_bytes(dim), dtype=torch.uint8, device="cuda")
        b.d_lens.fill_(start)
        shape = dict(lens=b.d_lens.data_ptr(), pages=b.table.data_ptr(), pages_stride=b.per, requests=n, max_len=start + steps, head_dim=dim,
                     dtype=p.dtype, format=p.format, layer=1)
        whole = kvb.make_bound_args(bounds.data_ptr(), max_new=start + steps, **shape)
        kvb.kv_bound(p.pool, whole)
        add = kvb.make_append_args(kvb.vecs(kv[:, 0]), kvb.vecs(kv[:, 1]), tokens=n, head_dim=dim, dtype=p.dtype, format=p.format, layer=1,
                                   slots=slots.data_ptr(), k_scale=p.k_scale, v_scale=p.v_scale)
        new = kvb.make_bound_args(bounds.data_ptr(), first=first.data_ptr(), max_new=1, **shape)
        budget = 4
        picks = torch.zeros(n, H, budget, dtype=torch.int32, device="cuda")
        sel = select_args(b, bounds, picks, budget, keep_first=1, keep_last=1)
        att = b.selected_args(picks)

        def step(stream):
            kvb.kv_append(p.pool, None, add, stream)
            kvb.kv_bound(p.pool, new, stream)
            kvb.kv_select(p.pool, sel, stream)
            kvb.kv_attend_selected(p.pool, att, stream)

        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step(side.cuda_stream)
        for t in range(start, start + steps):
            kv.copy_(torch.randn(kv.shape, generator=b.gen, device="cuda"))
            b.q.copy_(torch.randn(b.q.shape, generator=b.gen, device="cuda"))
            slots.copy_(b.table[:, t // T].long() * T + t % T)
            first.fill_(t)
            b.d_lens.fill_(t + 1)
            graph.replay()
            torch.cuda.synchronize()
            b.lens = [t + 1] * n
            check_picks(b, bounds, picks, budget, 1, 1)
            check_selected(b, picks)
        no_status(b)
        everything = torch.arange(b.per, dtype=torch.int32, device="cuda").expand(n, H, b.per).contiguous()
        run_selected(b, everything)
        check_selected(b, everything)
        b.run()
        b.check()


def test_a_branched_conversation():
    """Branches of one conversation: their shared prefix was another request's own pages, and all answers agree
    with attention of each branch by itself."""
    with Batch(kvb, [20, 9, 33], [1, 1, 1], [(0, 3, 130)], 2, 4, 128, T=16) as b:
        b.run()
        shared = b.out.clone()
        worst = b.check()
        assert worst <= 1.0
        # the same tokens as three requests without a prefix
        with Batch(kvb, [150, 139, 163], [1, 1, 1], (), 2, 4, 128, T=16, seed=5) as c:
            for i, n in enumerate(b.lens):
                for comp in (0, 1):
                    x = np.concatenate((b.p.held(b.prefix_table[0], 130, comp), b.p.held(b.table[i], n, comp)))
                    c.p.put(c.table[i], torch.from_numpy(x).cuda().float(), comp)
            c.q.copy_(b.q)
            c.run()
            c.check()
            # 2^-8 each of their roundings of a value under 4
            assert (c.out.float() - shared.float()).abs().max() <= 2 * 4 * 2.0 ** -8
