"""kv_attend where a window's prompt chunk spans more tokens than one tile of queries sees,
where a group of a value is not finite, and where steps of the 4-bit format differ widely from
token to token: a query's result must not depend on what it does not see.  Few-row calls of
several tokens, cut and in windows, and long requests whose every tile shows."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import vec_check  # noqa: E402
import vec_ref  # noqa: E402
from hierarchical_kv_cache_backup_gb300 import kvb  # noqa: E402
from test_vectors_gpu import Batch, b_without, poke  # noqa: E402


def put(b, i, comp, tokens, x):
    """Float32 values of some tokens as request i's keys (comp 0) or values (comp 1); the other
    tokens keep their bytes."""
    raw, tab = b.pool.alloc.cpu().numpy(), b.table.cpu().numpy()[i]
    at = np.atleast_1d(np.arange(b.lens[i])[tokens])
    new = vec_ref.q4_encode(np.broadcast_to(np.asarray(x, np.float32), (len(at), b.H, b.dim)))
    b.kv[i][comp][at] = new
    b.pool.view(raw, b.layer, comp)[tab[at // b.T], at % b.T] = new
    b.pool.alloc.copy_(torch.from_numpy(raw))


def values(b, i, comp, tokens=slice(None)):
    """Request i's values as [tokens, H, D] float32."""
    at = np.atleast_1d(np.arange(b.lens[i])[tokens])
    return vec_ref.q4_decode(b.kv[i][comp][at], b.dim).astype(np.float32)


def grow(b, i, comp, tokens, power, groups=None, heads=slice(None)):
    """Multiplies tokens' values (of some groups and heads) by 2^power."""
    x = values(b, i, comp, tokens)
    cols = np.isin(np.arange(b.dim) // 32, range(b.dim // 32) if groups is None else groups)
    x[:, heads] = np.where(cols, x[:, heads] * np.float32(2.0) ** power, x[:, heads])
    put(b, i, comp, tokens, x)


# ----------------------------------------- windows over more than 1,024 tokens

def late_large_steps(dtype, dim, with_lse, comp, power):
    """1,400 new tokens in a window of 256: together they see 1,655, more than one tile of
    queries does.  The last 300 tokens' steps are 2^power times the others'."""
    with Batch([1700], [1400], 1, 1, dim, 16, dtype, window=256) as b:
        grow(b, 0, comp, slice(1400, 1700), power)
        if comp == 0:
            b.scale *= 2.0 ** -power          # scores of the large keys stay ordinary
        elif dtype == "fp16":                 # and the outputs in range
            grow(b, 0, comp, slice(None), -(power // 2))
        out, lse, status = b.run(**({} if with_lse else dict(lse=None)))
        assert status == 0 and torch.isfinite(out.float()).all()
        vec_check.check(b, out, lse if with_lse else None, key_parts=2 if with_lse else 1)


@pytest.mark.parametrize("dtype,dim,with_lse,comp,power", [
    ("bf16", 128, True, 1, 13), ("bf16", 64, False, 1, 13), ("fp16", 128, False, 1, 13), ("fp16", 96, True, 1, 13),
    ("bf16", 64, False, 0, 13), ("fp16", 128, False, 0, 13)])
def test_window_prompt_with_late_large_steps(dtype, dim, with_lse, comp, power):
    late_large_steps(dtype, dim, with_lse, comp, power)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("comp", [0, 1])
def test_window_prompt_with_zeros_first(dtype, comp):
    """Nothing but zeros, whose step is 0, before the tokens that matter; those are small."""
    with Batch([1800], [1500], 1, 1, 128, 16, dtype, window=300) as b:
        if comp:                              # 2^-30 is below fp16 outputs: 2^-6 will do
            grow(b, 0, comp, slice(None), -30 if dtype == "bf16" else -6)
        put(b, 0, comp, slice(0, 1100), 0.0)
        out, lse, status = b.run()
        assert status == 0
        vec_check.check(b, out, lse)


# -------------------------------------------------- a group that is not finite

def not_finite(dim, groups):
    x = np.zeros((1, dim), np.float32)
    for g in groups:
        x[:, 32 * g:32 * g + 32] = np.nan
    return vec_ref.q4_encode(x)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group,n_q", [(128, 4, 1), (128, 2, 6), (128, 4, 19), (64, 4, 1), (64, 4, 19), (96, 3, 1),
                                           (96, 2, 6), (256, 2, 1), (256, 2, 40), (192, 1, 6)])
@pytest.mark.parametrize("groups", [[0], [1], [0, 1]])
def test_few_rows_a_value_group_that_is_not_finite(dtype, dim, group, n_q, groups):
    """Only that group's dims are NaN, and only for the queries that see the token."""
    with Batch([90, 90], [n_q, n_q], 1, group, dim, 16, dtype, window=60) as b:
        late = 90 - 1 - n_q // 3                        # seen from its own position on
        early = 90 - n_q - 60 + 1 + n_q // 3            # seen as long as the window holds it
        poke(b, 0, late, 1, not_finite(dim, groups))
        poke(b, 1, early, 1, not_finite(dim, groups))
        out, lse, _ = b.run()
        out, lse = out.clone(), lse.clone()
        pos = 90 - n_q + np.arange(n_q)
        sees = np.concatenate(((pos >= late) & (pos - 60 < late), (pos >= early) & (pos - 60 < early)))
        want_nan = torch.zeros(out.shape, dtype=torch.bool)
        cols = [32 * g + e for g in groups for e in range(32)]
        want_nan[torch.from_numpy(sees)] = torch.isin(torch.arange(dim), torch.tensor(cols))
        nan = torch.isnan(out.float()).cpu()
        assert torch.equal(nan, want_nan)
        want, _, _ = b_without(b)
        assert torch.equal(out[torch.from_numpy(~sees).cuda()], want[torch.from_numpy(~sees).cuda()])
        # the other dims of the queries that see it: as if that token's values were zeros there
        for i, t in ((0, late), (1, early)):
            put(b, i, 1, t, 0.0)
        out = torch.where(want_nan.cuda(), 0.0, out.float())
        zeroed, lse0, _ = b.run()
        assert torch.equal(out, torch.where(want_nan.cuda(), 0.0, zeroed.float())) and torch.equal(lse, lse0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n_q", [1, 3])
def test_few_rows_a_group_that_is_not_finite_joined_over_chunks(dtype, n_q):
    with Batch([9000, 5000], [n_q, n_q], 1, 4, 128, 32, dtype) as b:
        assert b.args().workspace_bytes > 0
        poke(b, 0, 4321, 1, not_finite(128, [2]))
        out, _, _ = b.run()
        nan = torch.isnan(out.float())
        want_nan = torch.zeros_like(nan)
        want_nan[:n_q, :, 64:96] = True
        assert torch.equal(nan, want_nan)


# ------------------------------------------- steps that differ between tokens

FEW = [(128, 2, 6), (64, 4, 19), (96, 1, 6), (128, 4, 19), (256, 2, 40), (192, 1, 6)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group,n_q", FEW)
@pytest.mark.parametrize("power,groups", [(20, None), (45, [0]), (45, [1]), (90, None)])
def test_few_rows_do_not_feel_large_values_they_do_not_see(dtype, dim, group, n_q, power, groups):
    """A later new token's values are 2^power times the others': the queries before it get the
    bytes that they get without it."""
    with Batch([150], [n_q], 1, group, dim, 16, dtype) as b:
        want, wl, _ = b.run()
        want, wl, t = want.clone(), wl.clone(), 150 - n_q // 3 - 1
        grow(b, 0, 1, t, power, groups)
        out, lse, status = b.run()
        before = t - (150 - n_q)
        assert before > 0 and status == 0
        assert torch.equal(out[:before], want[:before]) and torch.equal(lse, wl)
        if dtype == "bf16":                              # fp16 outputs overflow
            vec_check.check(b, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group,n_q", [(128, 4, 1), (64, 2, 1), (256, 2, 1), (96, 3, 1)] + FEW)
@pytest.mark.parametrize("power,groups", [(20, None), (45, [0]), (45, [1])])
@pytest.mark.parametrize("at", [3, 140])
def test_few_rows_large_values_without_weight(dtype, dim, group, n_q, power, groups, at):
    """A token with large values whose key points away from every query: weight 0 or nearly so."""
    if at == 140 and n_q > 10:
        at = 100
    with Batch([150], [n_q], 1, group, dim, 16, dtype) as b:
        away(b, 0, at)
        grow(b, 0, 1, at, power, groups)
        out, lse, status = b.run()
        assert status == 0
        vec_check.check(b, out, lse)


def away(b, i, t, by=-12.0):
    """All queries nearly the same, and request i's key t against them: a weight of about e^-130."""
    g = torch.Generator(device="cuda")
    g.manual_seed(77)
    one = torch.randn(1, 1, b.dim, generator=g, device="cuda")
    b.q = (one + 0.1 * torch.randn(b.q.shape, generator=g, device="cuda")).to(b.dt)
    put(b, i, 0, t, by * one[0].cpu().numpy() * (128 / b.dim) ** 0.5)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group,n_q", [(128, 4, 1), (64, 4, 5)])
def test_few_rows_maximum_that_rises_far(dtype, dim, group, n_q):
    """Scores that rise by hundreds after tokens with large values: the large ones end with no
    weight and must not keep the scale that they brought."""
    with Batch([1000], [n_q], 1, group, dim, 16, dtype) as b:
        away(b, 0, slice(0, 400), by=-14.0)
        grow(b, 0, 1, slice(0, 400), 30)
        out, lse, status = b.run()
        assert status == 0
        vec_check.check(b, out, lse)


@pytest.mark.parametrize("dtype,dim,with_lse,comp,power", [
    (d, n, e, c, p) for d, n, e in (("bf16", 128, True), ("bf16", 64, False), ("fp16", 128, False), ("fp16", 96, True))
    for c in (0, 1) for p in (13, 15, 17)])
def test_window_prompt_with_steps_far_apart(dtype, dim, with_lse, comp, power):
    late_large_steps(dtype, dim, with_lse, comp, power)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group,n_q", [(128, 4, 40), (64, 1, 90), (96, 8, 11), (128, 1, 300)])
@pytest.mark.parametrize("comp,power,groups", [(1, 13, None), (1, 20, None), (1, 45, [0]), (1, 90, [1]), (0, 20, None),
                                               (0, 45, [1])])
def test_many_rows_do_not_feel_large_steps_they_do_not_see(dtype, dim, group, n_q, comp, power, groups):
    """The last new token's keys or values are 2^power times the others'."""
    with Batch([400, 350], [n_q, n_q], 2, group, dim, 16, dtype) as b:
        want, wl, _ = b.run()
        want, wl = want.clone(), wl.clone()
        grow(b, 0, comp, 399, power, groups, heads=1)
        for with_lse in (True, False):
            out, lse, status = b.run(**({} if with_lse else dict(lse=None)))
            assert status == 0
            if with_lse:                                  # the other head and request: as before
                assert torch.equal(out[:n_q, :group], want[:n_q, :group]) and torch.equal(out[n_q:], want[n_q:])
                assert torch.equal(lse[:n_q, :group], wl[:n_q, :group]) and torch.equal(lse[n_q:], wl[n_q:])
            o, c, l = out.clone(), b.n_q, lse.clone()
            # the queries before the last token, as a batch of their own
            b.n_q = [n_q - 1, 0]
            lens, kv, b.lens = b.lens, b.kv, [399, 350]
            b.kv = [[x[:399] for x in kv[0]], kv[1]]
            vec_check.check(b, o, l if with_lse else None, many=True, key_parts=2 if with_lse else 1)
            b.lens, b.kv, b.n_q = lens, kv, c


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("power,groups", [(13, None), (20, None), (45, [0])])
@pytest.mark.parametrize("at", [3, 360])
def test_many_rows_large_values_without_weight(dtype, power, groups, at):
    with Batch([400], [30], 1, 4, 128, 16, dtype) as b:
        away(b, 0, at)
        grow(b, 0, 1, at, power, groups)
        out, lse, status = b.run()
        assert status == 0
        vec_check.check(b, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("window", [0, 500])
def test_many_rows_uneven_steps_cut_and_windowed(dtype, window):
    """Requests long enough to be cut along their tokens, one of them with uneven steps."""
    with Batch([6000, 100, 5500], [40, 3, 40], 1, 4, 128, 32, dtype, window) as b:
        assert b.args().workspace_bytes > 0
        want, wl, _ = b.run()
        want, wl = want.clone(), wl.clone()
        grow(b, 0, 1, slice(5500, 6000, 97), 18, [1])
        grow(b, 0, 0, slice(5400, 6000, 89), -25, [0])
        out, lse, status = b.run()
        assert status == 0
        assert torch.equal(out[40:], want[40:]) and torch.equal(lse[40:], wl[40:])
        if dtype == "bf16":
            vec_check.check(b, out, lse)
        first = out.clone()
        out, _, _ = b.run()
        assert torch.equal(out, first)


def test_many_rows_uneven_steps_with_bad_pages_and_not_finite_groups():
    with Batch([200, 200], [40, 40], 1, 2, 64, 16, "bf16", window=60) as b:
        for i in (0, 1):
            grow(b, i, 1, 199, 40)
        poke(b, 0, 170, 1, not_finite(64, [1]))      # seen by the new tokens at 170..199
        b.table[1, 9] = -1                           # tokens 144..159: all but none of 160..199 see some
        out, lse, status = b.run()
        assert status == kvb.KV_STATUS_BAD_PAGE
        assert torch.isnan(out[40:].float()).all() and torch.isnan(lse[40:]).all()
        nan = torch.isnan(out[:40].float())
        want_nan = torch.zeros_like(nan)
        want_nan[10:, :, 32:] = True
        assert torch.equal(nan, want_nan)


# ------------------------------------- branches that small cases do not reach

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,H,group,n_q", [(64, 2, 4, 2), (64, 1, 3, 5), (64, 1, 8, 9), (96, 2, 2, 8), (96, 1, 5, 3),
                                             (128, 2, 4, 5), (128, 1, 8, 8), (128, 1, 1, 79), (64, 1, 1, 79), (96, 1, 3, 26)])
@pytest.mark.parametrize("window", [0, 1, 37, 300])
def test_few_rows_several_tokens(dtype, dim, H, group, n_q, window):
    """9 to 79 query rows at heads of 128 and fewer, ragged, more new tokens than cached ones."""
    with Batch([500, n_q, max(1, n_q - 2), 0, 33], [n_q, n_q, n_q, 2, 1], H, group, dim, 17, dtype, window, hnd=True) as b:
        assert max(b.n_q) * group < 80
        out, lse, status = b.run()
        assert status == 0
        vec_check.check(b, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group,n_q", [(64, 4, 5), (96, 8, 2), (128, 8, 6), (128, 1, 40), (256, 2, 5)])
@pytest.mark.parametrize("window", [0, 2500])
def test_few_rows_several_tokens_joined(dtype, dim, group, n_q, window):
    with Batch([5200, 3900, 10], [n_q, n_q, 1], 1, group, dim, 32, dtype, window) as b:
        assert b.args().workspace_bytes > 0
        out, lse, status = b.run()
        assert status == 0
        vec_check.check(b, out, lse)
        first = out.clone()
        out, _, _ = b.run()
        assert torch.equal(out, first)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group,n_q", [(128, 4, 1), (64, 4, 5), (256, 2, 1), (128, 4, 30)])
def test_long_requests_lose_no_tile(dtype, dim, group, n_q):
    """Values of every 32 tokens lie around +3 or -3: one tile left out, or taken twice, moves the
    outputs by several times the tolerance, without any logarithm to tell."""
    with Batch([9000], [n_q], 1, group, dim, 16, dtype) as b:
        sign = np.random.default_rng(3).choice([-3.0, 3.0], 282).repeat(32)[:9000, None, None]
        put(b, 0, 1, slice(None), values(b, 0, 1) * 0.1 + sign)
        put(b, 0, 0, slice(None), values(b, 0, 0) * 0.1)
        out, _, status = b.run(lse=None)
        assert status == 0
        vec_check.check(b, out, key_parts=1)


@pytest.mark.parametrize("dim,group,n_q,window", [(128, 4, 40, 0), (64, 1, 90, 0), (96, 8, 11, 200), (128, 1, 300, 0),
                                                  (128, 4, 1, 0), (64, 4, 5, 0)])
def test_logarithms_change_no_bit_of_fp16_outputs(dim, group, n_q, window):
    with Batch([900, 350], [n_q, n_q], 2, group, dim, 16, "fp16", window) as b:
        out, lse, _ = b.run()
        want, wl = out.clone(), lse.clone()
        out, lse, status = b.run(lse=None)
        assert torch.equal(out, want) and (lse == 7).all() and status == 0
        vec_check.check(b, out, wl)


def test_many_rows_in_a_graph_that_meets_uneven_steps_later():
    """One captured call, replayed over even and uneven steps and over other lengths."""
    with Batch([6000, 5500], [40, 40], 1, 4, 128, 32, "bf16") as b:
        a = b.args()
        assert a.workspace_bytes > 0
        kvb.kv_attend(b.pool.pool, a)
        torch.cuda.synchronize()
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=side):
            kvb.kv_attend(b.pool.pool, a, side.cuda_stream)
        out, lse, lens_d, status = b.out, b.lse, b.lens_d, b.status
        for step in range(4):
            if step == 1:
                grow(b, 1, 1, 5400, 20)
            if step == 2:
                grow(b, 1, 1, 5400, -20)
            if step == 3:
                b.lens = [3000, 41]
                b.kv = [[x[:n] for x in kv] for kv, n in zip(b.kv, b.lens)]
                lens_d.copy_(torch.tensor(b.lens, device="cuda"))
            out.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            vec_check.check(b, out, lse)
            assert int(status) == 0
