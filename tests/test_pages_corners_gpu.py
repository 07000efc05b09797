"""Corners of kv_attend_shared, kv_bound, kv_select and kv_attend_selected, against plain implementations in 64
bits (pages_ref.py, where the tolerances are derived)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from hierarchical_kv_cache_backup_gb300 import kvb  # noqa: E402
from pages_ref import Batch  # noqa: E402
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
            assert kvb.kv_attend_selected_workspace(b.p.pool, a) > 0


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
