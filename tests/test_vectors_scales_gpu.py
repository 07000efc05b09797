"""Scales of e4m3 pools that have no finite inverse are refused: zeros would be held as NaN."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from hierarchical_kv_cache_backup_gb300 import kvb  # noqa: E402
from test_vectors_gpu import FMT, Pool  # noqa: E402


def calls(p, x, slots, **scales):
    args = dict(tokens=2, head_dim=48, dtype=0, format=FMT["e4m3"], layer=0, slots=slots.data_ptr(), **scales)
    return (lambda: kvb.kv_append(p.pool, None, kvb.make_append_args(kvb.vecs(x), kvb.vecs(x), **args)),
            lambda: kvb.kv_fetch(p.pool, kvb.make_fetch_args(kvb.vecs(x), kvb.vecs(x), **args)))


@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
@pytest.mark.parametrize("scale", [1e-39, 1e-45, 2.0 ** -128])
def test_scales_without_an_inverse(which, scale):
    with Pool(48, "e4m3", T=4, H=2, P=3) as p:
        x, slots = torch.zeros(2, 2, 48, device="cuda", dtype=torch.bfloat16), torch.arange(2, device="cuda")
        before = p.alloc.clone()
        for call in calls(p, x, slots, **{which: scale}):
            with pytest.raises(kvb.KvError) as e:
                call()
            assert e.value.status == kvb.KV_ERR_INVALID_ARG
        torch.cuda.synchronize()
        assert torch.equal(p.alloc, before)


@pytest.mark.parametrize("scale", [2.0 ** -126, 1.5 * 2.0 ** -127, 3e38])
def test_least_and_largest_scales(scale):
    with Pool(48, "e4m3", T=4, H=2, P=3) as p:
        x = torch.zeros(2, 2, 48, device="cuda", dtype=torch.bfloat16)
        x[1, :, ::3] = 8 * scale if scale < 1 else 3e38
        want, slots = x.clone(), torch.arange(2, device="cuda")
        append, fetch = calls(p, x, slots, k_scale=scale, v_scale=scale)
        append()
        x.fill_(7.0)
        fetch()
        torch.cuda.synchronize()
        # e4m3 keeps 3 bits behind the point (2^-4 of a value), bf16 7; their sum, and bf16's least step
        err = (x.double() - want.double()).abs()
        assert bool((err <= want.double().abs() * (2.0 ** -4 + 2.0 ** -7) + 2.0 ** -133).all())
        assert not x[0].any()
