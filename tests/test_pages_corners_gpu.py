"""Corners of kv_attend_shared, kv_bound, kv_select and kv_attend_selected, against plain implementations in 64
bits (pages_ref.py, where the tolerances are derived)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from hierarchical_kv_cache_backup_gb300 import kvb  # noqa: E402
from pages_ref import Batch  # noqa: E402
from test_pages_gpu import check_selected, no_status, run_selected, some_picks  # noqa: E402


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
