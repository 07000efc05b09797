"""Corners of kv_attend_shared, kv_bound, kv_select and kv_attend_selected, against plain implementations in 64
bits (pages_ref.py, where the tolerances are derived)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from hierarchical_kv_cache_backup_gb300 import kvb  # noqa: E402
from pages_ref import Batch, softmax_rows, tolerance  # noqa: E402
from vec_ref import half_step  # noqa: E402
from test_pages_gpu import bound, check_picks, check_selected, no_status, run_selected, select, some_picks  # noqa: E402


def test_a_chunk_over_a_long_cache_counts_its_lists():
    """Many query tokens of a request that may be very long are as much work as their lists of pages."""
    with Batch(kvb, [500], [300], (), 2, 4, 64, T=64) as b:
        b.table = torch.cat((b.table, torch.full((1, (1 << 26) // 64 - b.per), -1, dtype=torch.int32, device="cuda")), 1)
        picks = some_picks(b, 3)
        run_selected(b, picks, max_len=1 << 26, pages_stride=b.table.shape[1])
        check_selected(b, picks)
        no_status(b)
        a = b.selected_args(picks)
        for chunk, length in ((32768, 1 << 20), (65535, 1 << 24)):
            a.tokens, a.max_q, a.max_len, a.pages_stride = chunk, chunk, length, 1 << 24
            assert kvb.kv_attend_selected_workspace(b.p.pool, a) >= 0            # taken


@pytest.mark.parametrize("pages", [40, 300, 3000])
def test_zeros_of_both_signs_tie(pages):
    """Steps whose product underflows make every score a zero, of its sum's sign: the first pages are picked."""
    with Batch(kvb, [pages], [1], (), 2, 1, 64, T=1) as b:
        sign = torch.where(torch.rand(pages, 2, 1, generator=b.gen, device="cuda") < 0.5, -1.0, 1.0)
        b.p.put(b.table[0], sign.expand(pages, 2, 64) * 2.0 ** -90, 0)
        b.q.fill_(2.0 ** -90)
        bounds = bound(b)
        for budget, first, last in ((1, 0, 0), (9, 0, 0), (30, 2, 3)):
            picks = select(b, bounds, budget, keep_first=first, keep_last=last)
            check_picks(b, bounds, picks, budget, first, last)
            want = list(range(budget - last)) + list(range(pages - last, pages))
            assert picks[0].tolist() == [want, want]


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("fp16", 64), ("bf16", 96), ("fp16", 256)])
@pytest.mark.parametrize("n_q,groups", [(1, ()), (3, ((0, 1, 30),)), (20, ((0, 1, 30),)), (90, ())])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinite_keys(dtype, dim, n_q, groups, bad, sign):
    """A score of -infinity has weight 0, one of +infinity makes the query's outputs NaN, and nobody else's."""
    H, group, own, h, d = 2, 4, 150, 1, 37
    with Batch(kvb, [own], [n_q], groups, H, group, dim, "same", dtype, T=16) as b:
        b.scale *= sign
        at = own - n_q + n_q // 2                              # query n_q // 2 is the first that sees it
        b.run()
        clean, clean_lse = b.out.clone(), b.lse.clone()
        x = torch.from_numpy(b.p.held(b.table[0], own, 0)).cuda().float()
        x[at, h, d] = bad
        b.p.put(b.table[0], x, 0)
        b.run()
        no_status(b)
        pre = groups[0][2] if groups else 0
        k, v = (np.concatenate(([b.p.held(b.prefix_table[0], pre, c)] if pre else []) + [b.p.held(b.table[0], own, c)]) for c in (0, 1))
        k[pre + at, h, d] = 0.0                                # not looked at below
        q, out, lse = (y.double().cpu().numpy() for y in (b.q, b.out, b.lse))
        pos = own - n_q + np.arange(n_q)
        seen = np.concatenate((np.ones((n_q, pre), bool), np.arange(own)[None] <= pos[:, None]), 1)
        hit = np.arange(n_q) >= n_q // 2
        for j in range(H * group):
            if j // group != h:
                assert torch.equal(b.out[:, j], clean[:, j]) and torch.equal(b.lse[:, j], clean_lse[:, j])
                continue
            up = hit & (sign * bad * q[:, j, d] > 0)
            low = hit & (sign * bad * q[:, j, d] < 0)
            assert np.isnan(out[up, j]).all() and np.isnan(lse[up, j]).all()
            assert torch.equal(b.out[~torch.from_numpy(hit).cuda(), j], clean[~torch.from_numpy(hit).cuda(), j])
            if low.any():
                sees = seen[low].copy()
                sees[:, pre + at] = False
                want, wl, w, s = softmax_rows(q[low, j], k[:, h], v[:, h], sees, b.scale)
                tol, tl = tolerance(q[low, j], k[:, h], v[:, h], w, s, want, b.scale, b.p.dt, False, b.many())
                assert (np.abs(out[low, j] - want) <= tol).all() and (np.abs(lse[low, j] - wl) <= tl + 2.0 ** -21 * np.abs(wl)).all()


@pytest.mark.parametrize("n_q", [1, 20])
def test_scores_of_minus_infinity_alone(n_q):
    """Such a query gets what one that sees nothing gets."""
    with Batch(kvb, [40], [n_q], [(0, 1, 70)], 1, 4, 64) as b:
        b.q[:, 1] = 1.0
        b.q[:, 0] = b.q[:, 2:] = 0.0
        for table, n in ((b.table[0], 40), (b.prefix_table[0], 70)):
            x = torch.zeros(n, 1, 64, device="cuda")
            x[..., 5] = -float("inf")
            b.p.put(table, x, 0)
        b.run()
        assert not b.out[:, 1].any() and torch.isneginf(b.lse[:, 1]).all()
        assert torch.isnan(b.out[:, [0, 2, 3]]).all() and torch.isnan(b.lse[:, [0, 2, 3]]).all()       # 0 x infinity


@pytest.mark.parametrize("fmt,bad", [("same", float("nan")), ("same", -float("inf")), ("e4m3", float("nan"))])
@pytest.mark.parametrize("requests,n_q,H,prefix", [(1, 1, 2, 9000), (8, 1, 2, 9000), (2, 40, 2, 3000), (300, 3, 8, 1000)])
def test_values_of_no_weight(fmt, bad, requests, n_q, H, prefix):
    """A value that is not finite reaches the queries that see it, even where its piece of the tokens weighs nothing in the end."""
    with Batch(kvb, [60] * requests, [n_q] * requests, [(0, requests, prefix)], H, 4, 128, fmt, T=16) as b:
        b.q.fill_(1.0)
        b.p.put(b.prefix_table[0], torch.full((prefix, H, 128), -20.0 if fmt == "same" else -300.0, device="cuda"), 0)     # scores under -200
        for i in range(requests):
            b.p.put(b.table[i], torch.zeros(60, H, 128, device="cuda"), 0)
        b.run()
        b.check()
        clean, lse = b.out.clone(), b.lse.clone()
        size = b.p.B // 128
        word = torch.tensor([bad], device="cuda").to(torch.float8_e4m3fn if fmt == "e4m3" else b.p.dt).view(torch.uint8)
        b.p.view(1)[b.prefix_table[0, 700 // 16].long(), 700 % 16, 1, 5 * size:6 * size] = word
        b.run()
        assert not torch.isfinite(b.out[:, 4:8, 5]).any() and torch.equal(b.lse, lse)
        b.out[:, 4:8, 5] = clean[:, 4:8, 5]
        assert torch.equal(b.out, clean)


@pytest.mark.parametrize("n_q", [1, 3, 10, 70])
@pytest.mark.parametrize("own", [60, 6000])
def test_groups_without_prefixes(n_q, own):
    """No launch is made for them, and groups or lengths that are wrong are still said to be."""
    with Batch(kvb, [own, 30, own], [n_q] * 3, [(0, 2, 0), (2, 3, 0)], 2, 4, 64, T=16) as b:
        a, alone = b.shared_args(), b.shared_args(groups=0)
        n = kvb.kv_launch_count()
        kvb.kv_attend_shared(b.p.pool, alone)
        n, m = kvb.kv_launch_count(), kvb.kv_launch_count() - n
        torch.cuda.synchronize()
        want = b.out.clone()
        b.out.fill_(7.0)
        kvb.kv_attend_shared(b.p.pool, a)
        assert kvb.kv_launch_count() - n == m and a.workspace_bytes == alone.workspace_bytes
        torch.cuda.synchronize()
        b.check()
        no_status(b)
        assert torch.equal(b.out, want)
        for wrong in (b.prefix_lens, b.group_start):
            wrong[1] = 5
            kvb.kv_attend_shared(b.p.pool, a)
            torch.cuda.synchronize()
            assert int(b.status) == kvb.KV_STATUS_BAD_LENGTH and torch.equal(b.out, want)
            wrong[1] = 0 if wrong is b.prefix_lens else 2
            b.status.zero_()


@pytest.mark.parametrize("fmt,dtype,dim,H", [("same", "bf16", 128, 2), ("same", "fp16", 64, 3), ("e4m3", "bf16", 256, 1)])
@pytest.mark.parametrize("n_q", [[1] * 20 + [130], [130] + [1] * 20, [200] * 3 + [1], [1, 0, 90, 1, 70, 2]])
def test_a_chunk_among_single_tokens(fmt, dtype, dim, H, n_q):
    """Continuous batching: a prompt chunk beside requests of one token, behind one prefix, behind two, and behind none."""
    lens, n = [max(q, 37 + 9 * i) for i, q in enumerate(n_q)], len(n_q)
    for groups in ([(0, n, 300)], [(0, n // 2, 300), (n // 2, n, 90)], [(0, n - 1, 333)], ()):
        with Batch(kvb, lens, n_q, groups, H, 4, dim, fmt, dtype, T=16) as b:
            b.run()
            b.check()
            no_status(b)


@pytest.mark.parametrize("own", [500, 20000])
@pytest.mark.parametrize("selected", [False, True])
def test_requests_that_share_query_tokens_are_left_out(selected, own):
    """More units than valid ranges can make: not an output is written, by calls that are cut, of whole units, and on
    tcgen05.  (The ranges between, out of order, are said to be wrong as well: fewer requests of the same ranges are answered.)"""
    n, q = 40, 400
    with Batch(kvb, [own] * n, [q // n] * n, (), 1, 4, 64, T=64) as b:
        b.q_start.copy_(torch.tensor([q * (i % 2) for i in range(n + 1)], dtype=torch.int32))
        picks = torch.arange(200 if own > 500 else 1, dtype=torch.int32, device="cuda").expand(q, 1, -1).contiguous()
        for requests in (2, n):
            kw = dict(max_q=q, requests=requests)
            a = b.selected_args(picks, **kw) if selected else b.shared_args(**kw)
            assert (a.workspace_bytes == 0) == (selected and own == 500)         # whole units
            b.out.fill_(7.0)
            b.lse.fill_(7.0)
            b.status.zero_()
            (kvb.kv_attend_selected if selected else kvb.kv_attend_shared)(b.p.pool, a)
            torch.cuda.synchronize()
            assert int(b.status) == kvb.KV_STATUS_BAD_LENGTH
            left = (b.out == 7.0).all() and (b.lse == 7.0).all()
            assert left if requests == n else not (b.lse == 7.0).any()


@pytest.mark.parametrize("fmt,dtype", [("same", "bf16"), ("same", "fp16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("requests,n_q,prefix", [(1, 1, 30), (1, 1, 9000), (12, 1, 3000), (2, 40, 3000), (200, 3, 900)])
def test_two_runs_give_the_same_bits(fmt, dtype, requests, n_q, prefix):
    """Nothing that is written depends on which block ends first."""
    with Batch(kvb, [70 + 7 * (i % 9) for i in range(requests)], [n_q] * requests, [(0, requests, prefix)], 4, 4, 128, fmt, dtype) as b:
        b.run()
        out, lse = b.out.clone(), b.lse.clone()
        for _ in range(3):
            b.out.fill_(7.0)
            b.run()
            assert torch.equal(b.out, out) and torch.equal(b.lse, lse)
        picks = some_picks(b, 3)
        run_selected(b, picks)
        out = b.out.clone()
        run_selected(b, picks)
        assert torch.equal(b.out, out)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("power", [22, 25, 28, 40, 125])
@pytest.mark.parametrize("n_q,own,prefix", [(1, 60, 50), (1, 60, 9000), (40, 60, 900), (90, 100, 300)])
def test_scores_as_far_as_float32_goes(dtype, sign, power, n_q, own, prefix):
    """Scores of up to 2^125: the largest alone has weight, and its value comes out."""
    with Batch(kvb, [own], [n_q], [(0, 1, prefix)], 1, 4, 64, "same", dtype) as b:
        q = b.q.double().cpu().numpy()
        k, v = (np.concatenate((b.p.held(b.prefix_table[0], prefix, c), b.p.held(b.table[0], own, c)))[:, 0] for c in (0, 1))
        x = np.einsum("ijd,kd->ijk", q, k) * sign
        b.scale = float(sign * 2.0 ** (power - 1) / np.abs(x).max())                 # times log2(e): under 2^power
        b.run()
        out, lse = b.out.double().cpu().numpy(), b.lse.double().cpu().numpy()
        for i in range(n_q):
            x[i, :, prefix + own - n_q + i + 1:] = -np.inf
        two = np.sort(x, -1)[..., -2:]
        # far past the scores' roundings, and 2^32 or more apart in weight (n 2^-32 is under half a step of fp16)
        gap = (two[..., 1] - two[..., 0]) * abs(b.scale)
        clear = (gap > 2.0 ** -16 * np.abs(two[..., 1]) * abs(b.scale)) & (gap > 23)
        assert clear.mean() > 0.9
        top = x.argmax(-1)
        # With few rows weights have 2^-17 and the sums 2^-20: rounded, the value itself.  With many rows the largest
        # weight is 2^r, r the rounding of its score, and goes in rounded once (half a step) over a sum that is not;
        # then the output's own half a step, of a value up to that much larger.
        h = half_step(b.p.dt) if b.many() else 0.0
        assert (np.abs(out[clear] - v[top[clear]]) <= (2 * h + h * h) * np.abs(v[top[clear]])).all()
        assert np.allclose(lse, two[..., 1] * abs(b.scale), rtol=2.0 ** -18, atol=0)


@pytest.mark.parametrize("dim,H", [(64, 4), (128, 2)])
def test_two_calls_at_once(dim, H):
    """Calls on two streams, each with a workspace of its own, among them two that want all tensor memory of an SM."""
    made = [([70, 200, 90], [40, 60, 3], [(0, 3, 700)]), ([300] * 3, [100] * 3, ()), ([90] * 30, [1] * 30, [(0, 30, 2000)]), ([4000], [1], ())]
    batches = [Batch(kvb, lens, n_q, groups, H, 4, dim, seed=20 + i) for i, (lens, n_q, groups) in enumerate(made)]
    picks = [some_picks(b, 4) for b in batches]
    args = [(b.shared_args(), b.selected_args(p)) for b, p in zip(batches, picks)]
    want = []
    for b, (shared, selected) in zip(batches, args):
        kvb.kv_attend_selected(b.p.pool, selected)
        torch.cuda.synchronize()
        one = b.out.clone()
        kvb.kv_attend_shared(b.p.pool, shared)
        torch.cuda.synchronize()
        b.check()
        want.append((b.out.clone(), one))
    streams = [torch.cuda.Stream() for _ in batches]
    for k in range(40):
        for b, (shared, selected), stream in zip(batches, args, streams):
            if k % 3:
                kvb.kv_attend_shared(b.p.pool, shared, stream.cuda_stream)
            else:
                kvb.kv_attend_selected(b.p.pool, selected, stream.cuda_stream)
        if k % 3 != 1:
            torch.cuda.synchronize()
            for b, (shared, selected) in zip(batches, want):
                assert torch.equal(b.out, shared if k % 3 else selected)
    for b in batches:
        no_status(b)
        b.__exit__()


def test_rows_of_tables_apart():
    """Page tables inside wider ones, whose other entries are anything."""
    with Batch(kvb, [90, 33, 150], [1, 20, 3], [(0, 2, 100), (2, 3, 60)], 2, 4, 64, T=16) as b:
        b.run()
        want, picks = b.out.clone(), some_picks(b, 4)
        run_selected(b, picks)
        chosen = b.out.clone()
        own, pre = (torch.full((3, 40), 2 ** 31 - 1, dtype=torch.int32, device="cuda"), torch.full((2, 30), -9, dtype=torch.int32, device="cuda"))
        own[:, 7:7 + b.per], pre[:, 3:3 + b.pre] = b.table, b.prefix_table
        at = dict(pages=own.data_ptr() + 28, pages_stride=40)
        b.run(**at, prefix_pages=pre.data_ptr() + 12, prefix_stride=30)
        assert torch.equal(b.out, want)
        run_selected(b, picks, **at)
        assert torch.equal(b.out, chosen)
        bounds = bound(b)
        assert torch.equal(bound(b, pages=at["pages"], pages_stride=40), bounds)
        assert torch.equal(select(b, bounds, 3), select(b, bounds, 3, keep_first=0))
        no_status(b)
