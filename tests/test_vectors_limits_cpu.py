"""Refusals of the operators on head vectors that need no device."""
import pytest

from hierarchical_kv_cache_backup_gb300 import build as kbuild

kbuild.build_library()
from hierarchical_kv_cache_backup_gb300 import kvb  # noqa: E402


@pytest.mark.parametrize("gain", [3.5e38, 1e39, 1e300])
def test_a_gain_past_float32_is_refused(gain):
    """Cosines and sines would be infinite, and 0 x infinity NaN."""
    with pytest.raises(kvb.KvError) as e:
        kvb.kv_rotary_create(64, gain=gain)
    assert e.value.status == kvb.KV_ERR_INVALID_ARG
    kvb.kv_rotary_close(kvb.kv_rotary_create(64, gain=3e38))
