"""kv_rotate, kv_append and kv_fetch with so many tokens that a warp takes one by itself: the
same bytes as the definitions give, at counts that end inside a block."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import vec_ref  # noqa: E402
from hierarchical_kv_cache_backup_gb300 import kvb  # noqa: E402
from test_vectors_gpu import DT, FMT, STYLE, Pool, bits, check_rotation, decode, encode, gen, rotated  # noqa: E402


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,heads,dim,rot", [(4095, 3, 64, 64), (4096, 3, 64, 64), (4097, 5, 128, 128),
                                                  (5001, 1, 192, 64), (4097, 2, 80, 24), (4099, 3, 192, 90), (4096, 9, 8, 2)])
def test_rotate_many_tokens(dtype, style, tokens, heads, dim, rot):
    g = gen(tokens + dim)
    x = torch.randn(tokens, heads, dim, generator=g, device="cuda").to(DT[dtype][0])
    pos = torch.randint(0, 40000, (tokens,), generator=g, device="cuda")
    got, rows = rotated(x, rot, style, pos, want_rows=True)
    f, gain = vec_ref.frequencies(rot)
    rows64 = vec_ref.rows_of(f, gain, pos.cpu().numpy())
    assert np.abs(rows.double().cpu().numpy() - rows64).max() <= 2.0 ** -21
    check_rotation(x, got, rows64, style, False, gain)
    again, _ = rotated(x, rot, style, rows_in=rows)
    assert np.array_equal(bits(again), bits(got))
    # a token's bytes do not depend on how many others there are
    few, _ = rotated(x[:7].contiguous(), rot, style, pos[:7].contiguous())
    assert np.array_equal(bits(few), bits(got[:7]))
    rotated(x, rot, style, pos, out=x)
    assert np.array_equal(bits(x), bits(got))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt,dim,rot,style,H,Hq", [
    ("q4", 128, 128, "half", 2, 5), ("q4", 64, 32, "half", 3, 3), ("q4", 96, 96, "interleaved", 1, 2),
    ("q4", 160, 40, "half", 1, 1), ("q4", 192, 0, "half", 2, 0), ("same", 128, 64, "interleaved", 3, 4),
    ("same", 80, 80, "half", 2, 3), ("same", 8, 0, "half", 5, 0), ("e4m3", 128, 128, "half", 2, 7),
    ("e4m3", 48, 16, "interleaved", 3, 1), ("e4m3", 256, 0, "half", 1, 0)])
@pytest.mark.parametrize("tokens,page", [(4096, dict(T=16, page_first=False, hnd=False)),
                                         (4097, dict(T=17, page_first=True, hnd=True, offset=48)),
                                         (5001, dict(T=64, page_first=False, hnd=True, split=True))])
def test_append_and_fetch_many_tokens(dtype, fmt, dim, rot, style, H, Hq, tokens, page):
    dt, code = DT[dtype]
    g, n = gen(dim + rot + tokens), tokens
    with Pool(dim, fmt, H=H, P=-(-n // page["T"]) + 5, **page) as p:
        qkv = torch.randn(n, Hq + 2 * H, dim, generator=g, device="cuda")
        qkv[:, -1] *= 30.0
        qkv = qkv.to(dt)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        slots = torch.randperm(p.P * p.T, generator=g, device="cuda")[:n]
        slots[[0, 5, 777, n - 2]] = -1
        slots[[6, 4095]] = torch.tensor([p.P * p.T, -7], device="cuda")      # outside the pool
        ks, vs = 0.11, 0.02
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        rotary = rows = q_out = None
        if rot:
            f, gain = vec_ref.frequencies(rot)
            rows = torch.from_numpy(vec_ref.rows_of(f, gain, np.arange(n) * 31)).float().cuda()
            rotary = kvb.kv_rotary_create(rot, STYLE[style])
            q_out = torch.empty(n, Hq, dim, dtype=dt, device="cuda")
        want = p.alloc.cpu().numpy().copy()
        kvb.kv_append(p.pool, rotary, kvb.make_append_args(
            kvb.vecs(k), kvb.vecs(v), kvb.vecs(q) if rot else None, kvb.vecs(q_out) if rot else None, tokens=n,
            head_dim=dim, dtype=code, format=FMT[fmt], layer=1, slots=slots.data_ptr(), q_heads=Hq if rot else 0,
            k_scale=ks, v_scale=vs, rows=rows.data_ptr() if rot else None, status=status.data_ptr()))
        torch.cuda.synchronize()
        assert int(status) == kvb.KV_STATUS_BAD_SLOT
        k32, v32 = k.float().cpu().numpy(), v.float().cpu().numpy()
        if rot:
            rows32 = rows.cpu().numpy()
            k32 = vec_ref.turn(k32, rows32, style)
            q32 = vec_ref.turn(q.float().cpu().numpy(), rows32, style)
            assert np.array_equal(bits(q_out), torch.from_numpy(q32).to(dt).contiguous().view(torch.uint8).numpy())
            kvb.kv_rotary_close(rotary)
        at = slots.cpu().numpy()
        live = (at >= 0) & (at < p.P * p.T)
        for comp, x, s in ((0, k32, ks), (1, v32, vs)):
            p.view(want, 1, comp)[at[live] // p.T, at[live] % p.T] = encode(x, fmt, dt, s)[live]
        got = p.alloc.cpu().numpy()
        assert np.array_equal(got, want), np.flatnonzero(got != want)[:5]

        back = torch.full((2, n, H, dim), 7.0, dtype=dt, device="cuda")
        status.zero_()
        kvb.kv_fetch(p.pool, kvb.make_fetch_args(kvb.vecs(back[0]), kvb.vecs(back[1]), tokens=n, head_dim=dim,
                                                 dtype=code, format=FMT[fmt], layer=1, slots=slots.data_ptr(),
                                                 k_scale=ks, v_scale=vs, status=status.data_ptr()))
        torch.cuda.synchronize()
        assert int(status) == kvb.KV_STATUS_BAD_SLOT
        where = np.where(live, at, 0)
        for comp, s in ((0, ks), (1, vs)):
            held = decode(p.view(want, 1, comp)[where // p.T, where % p.T], fmt, dt, s, dim)
            held = torch.where(torch.from_numpy(live)[:, None, None], held, torch.zeros_like(held))
            assert torch.equal(back[comp].cpu(), held)
