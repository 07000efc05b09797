"""kv_rotate, kv_append, kv_fetch and kv_attend against plain implementations in
64 bits (vec_ref.py).  Every tolerance is a bound on rounding, stated where it
is used."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import vec_ref  # noqa: E402
from hierarchical_kv_cache_backup_gb300 import kvb  # noqa: E402
from vec_ref import half_step  # noqa: E402

DT = {"bf16": (torch.bfloat16, kvb.KV_BF16), "fp16": (torch.float16, kvb.KV_FP16)}
FMT = {"same": kvb.KV_CACHE_SAME, "e4m3": kvb.KV_CACHE_E4M3, "q4": kvb.KV_CACHE_Q4}
STYLE = {"half": kvb.KV_ROTARY_HALF, "interleaved": kvb.KV_ROTARY_INTERLEAVED}
SCALING = {"plain": kvb.KV_ROTARY_PLAIN, "linear": kvb.KV_ROTARY_LINEAR, "ntk": kvb.KV_ROTARY_NTK,
           "yarn": kvb.KV_ROTARY_YARN, "bands": kvb.KV_ROTARY_BANDS}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


# ------------------------------------------------------------------- rotate

def rotated(x, rot, style, positions=None, rows_in=None, inverse=False, out=None, want_rows=False, stream=None,
            **kw):
    r = kvb.kv_rotary_create(rot, STYLE[style], **kw)
    try:
        t, h, d = x.shape
        out = torch.empty(t, h, d, dtype=x.dtype, device="cuda") if out is None else out
        rows = torch.full((t, 2, rot // 2), float("nan"), device="cuda") if want_rows else None
        kvb.kv_rotate(r, kvb.make_rotate_args(
            kvb.vecs(x), kvb.vecs(out), t, h, d, kvb.KV_BF16 if x.dtype == torch.bfloat16 else kvb.KV_FP16,
            positions.data_ptr() if positions is not None else None,
            rows_in.data_ptr() if rows_in is not None else None,
            rows.data_ptr() if want_rows else None, inverse), stream)
        torch.cuda.synchronize()
        return out, rows
    finally:
        kvb.kv_rotary_close(r)


def check_rotation(x, got, rows64, style, inverse, gain):
    """One rounding to 16 bits, and the float32 part: cosines and sines off by at most 2^-21
    (rounding of the phase, 2 units of sincospi, the gain), three roundings of 2^-24."""
    x64 = x.double().cpu().numpy()
    want = vec_ref.turn(x64, rows64, style, inverse)
    half = rows64.shape[2]
    part = np.abs(x64)
    both = part.copy()
    if style == "half":
        both[..., :half] += part[..., half:2 * half]
        both[..., half:2 * half] += part[..., :half]
    else:
        both[..., 0:2 * half:2] += part[..., 1:2 * half:2]
        both[..., 1:2 * half:2] += part[..., 0:2 * half:2]
    tol = half_step(x.dtype) * np.abs(want) * (1 + 2 ** -7) + gain * 2.0 ** -20 * both + 2.0 ** -24
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), float((err / tol).max())
    passed = bits(got[..., 2 * half:]) == bits(x[..., 2 * half:])
    assert passed.all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,heads,dim,rot", [(1, 1, 8, 2), (1, 40, 128, 128), (3, 5, 64, 32), (7, 3, 96, 96),
                                                  (33, 9, 80, 24), (5, 2, 256, 256), (2, 6, 192, 90),
                                                  (700, 13, 128, 64), (2, 1, 40, 40)])
def test_rotate(dtype, style, tokens, heads, dim, rot):
    g = gen(tokens + dim)
    x = torch.randn(tokens, heads, dim, generator=g, device="cuda").to(DT[dtype][0])
    pos = torch.randint(0, 40000, (tokens,), generator=g, device="cuda")
    got, rows = rotated(x, rot, style, pos, want_rows=True)
    f, gain = vec_ref.frequencies(rot)
    rows64 = vec_ref.rows_of(f, gain, pos.cpu().numpy())
    assert np.abs(rows.double().cpu().numpy() - rows64).max() <= 2.0 ** -21
    check_rotation(x, got, rows64, style, False, gain)
    # from the stored rows: the same bytes; and back again
    again, _ = rotated(x, rot, style, rows_in=rows)
    assert np.array_equal(bits(again), bits(got))
    back, _ = rotated(got, rot, style, pos, inverse=True)
    check_rotation(got, back, rows64, style, True, gain)


@pytest.mark.parametrize("scaling,kw", [
    ("linear", dict(factor=8.0)), ("ntk", dict(factor=4.0, base=500000.0)),
    ("yarn", dict(factor=16.0, original_len=4096, slow=1.0, fast=32.0)),
    ("yarn", dict(factor=40.0, original_len=4096, slow=1.0, fast=32.0, gain=1.25)),
    ("bands", dict(factor=8.0, original_len=8192, slow=1.0, fast=4.0, base=500000.0)),
    ("plain", dict(gain=0.5))])
@pytest.mark.parametrize("far", [0, 131072, 2 ** 31 + 12345, 2 ** 40 + 1, -5])
def test_rotate_far_positions_and_scalings(scaling, kw, far):
    """Phases are 64-bit fractions of a turn, so an angle's error does not grow with the
    position but for the frequency's own 53 bits: 2^-53 x f x position radians."""
    g = gen(3)
    x = torch.randn(40, 2, 128, generator=g, device="cuda").to(torch.bfloat16)
    pos = far + torch.arange(40, device="cuda") * 37
    got, rows = rotated(x, 128, "half", pos, want_rows=True, scaling=SCALING[scaling], **kw)
    f, gain = vec_ref.frequencies(128, scaling=scaling, **kw)
    rows64 = vec_ref.rows_of(f, gain, pos.cpu().numpy())
    drift = abs(far) * 2.0 ** -51
    err = np.abs(rows.double().cpu().numpy() - rows64).max()
    assert err <= gain * (2.0 ** -21 + drift), err
    if drift < 2.0 ** -22:
        check_rotation(x, got, rows64, "half", False, gain)


def test_rotate_rows_alone():
    pos = torch.tensor([5, 1 << 33, 0], device="cuda")
    x = torch.zeros(3, 0, 64, device="cuda", dtype=torch.float16)
    _, rows = rotated(x, 48, "half", pos, out=x, want_rows=True)
    f, gain = vec_ref.frequencies(48)
    assert np.abs(rows.double().cpu().numpy() - vec_ref.rows_of(f, gain, pos.cpu().numpy())).max() <= 2.0 ** -21 + 2.0 ** -18


def test_rotate_in_place_strided_and_on_a_stream():
    g = gen(5)
    qkv = torch.randn(130, 12, 128, generator=g, device="cuda").to(torch.bfloat16)
    before = qkv.clone()
    pos = torch.arange(130, device="cuda") + 9
    want, _ = rotated(qkv[:, :10].contiguous(), 64, "half", pos)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    rotated(qkv[:, :10], 64, "half", pos, out=qkv[:, :10], stream=stream.cuda_stream)
    assert np.array_equal(bits(qkv[:, :10]), bits(want))
    assert np.array_equal(bits(qkv[:, 10:]), bits(before[:, 10:]))
    # heads ahead of tokens: any strides
    y = before.permute(1, 0, 2).contiguous().permute(1, 0, 2)[:, :10]
    got, _ = rotated(y, 64, "half", pos)
    assert np.array_equal(bits(got), bits(want))


def test_rotate_gradient():
    """The rotation is linear: its gradient, the inverse call, against central differences of
    sum(w y) in 64 bits (exact for a linear map but for rounding)."""
    g = gen(6)
    w = torch.randn(3, 2, 64, generator=g, device="cuda").to(torch.float16)
    pos = torch.tensor([0, 7, 5000], device="cuda")
    for style in ("half", "interleaved"):
        grad, _ = rotated(w, 48, style, pos, inverse=True, gain=1.5)
        f, gain = vec_ref.frequencies(48, gain=1.5)
        rows = vec_ref.rows_of(f, gain, pos.cpu().numpy())
        w64, x = w.double().cpu().numpy(), np.random.default_rng(1).standard_normal((3, 2, 64))
        num, e = np.zeros_like(x), 2.0 ** -10
        for t in range(3):
            for h in range(2):
                for d in range(64):
                    up, dn = x.copy(), x.copy()
                    up[t, h, d] += e
                    dn[t, h, d] -= e
                    num[t, h, d] = ((vec_ref.turn(up, rows, style) - vec_ref.turn(dn, rows, style)) * w64).sum() / (2 * e)
        tol = half_step(torch.float16) * np.abs(num) + 1.5 * 2.0 ** -19 * np.abs(w64).max() + 1e-9
        assert np.all(np.abs(grad.double().cpu().numpy() - num) <= tol)


def test_rotate_keeps_nan_and_infinity_to_their_pairs():
    x = torch.randn(1, 2, 64, device="cuda").to(torch.bfloat16)
    x[0, 0, 3], x[0, 1, 60] = float("nan"), float("inf")
    pos = torch.tensor([11], device="cuda")
    got, _ = rotated(x, 32, "half", pos)
    nan = torch.isnan(got)
    assert nan[0, 0, 3] and nan[0, 0, 19] and int(nan.sum()) == 2
    assert got[0, 1, 60] == float("inf")


# ----------------------------------------------------------- append and fetch

class Pool:
    def __init__(self, dim, fmt, T, H, P, L=2, page_first=False, hnd=False, offset=0, split=False, seed=1):
        self.dim, self.fmt, self.T, self.H, self.P, self.L = dim, fmt, T, H, P, L
        self.page_first, self.hnd = page_first, hnd
        self.B = kvb.kv_cache_head_bytes(FMT[fmt], dim)
        self.bytes = L * 2 * P * T * H * self.B
        lay = kvb.make_layout(L, 2, P, T, H, self.B, kvb.KV_PAGE_FIRST if page_first else kvb.KV_LAYER_FIRST,
                              kvb.KV_HND if hnd else kvb.KV_NHD, 1)
        self.offset = offset
        self.alloc = torch.randint(0, 256, (offset + self.bytes + 64,), generator=gen(seed), device="cuda",
                                   dtype=torch.uint8)
        if split:
            n = self.bytes // (2 * L)
            self.pool = kvb.kv_pool_register_split(lay, [self.alloc.data_ptr() + offset + i * n for i in range(2 * L)])
        else:
            self.pool = kvb.kv_pool_register(lay, self.alloc.data_ptr(), offset)

    def view(self, raw, layer, comp):
        raw = raw[self.offset:self.offset + self.bytes]
        return vec_ref.pool_view(raw, self.L, self.P, self.T, self.H, self.B, layer, comp, self.page_first, self.hnd)

    def __enter__(self):
        return self

    def __exit__(self, *a):
        torch.cuda.synchronize()
        kvb.kv_pool_close(self.pool)


def encode(x32, fmt, dtype, scale):
    """float32 numpy vectors as the pool's bytes (numpy uint8)."""
    if fmt == "q4":
        return vec_ref.q4_encode(x32)
    t = torch.from_numpy(x32)
    if fmt == "same":
        return t.to(dtype).contiguous().view(torch.uint8).numpy()
    inv = np.float32(1.0) / np.float32(scale)
    return torch.from_numpy(x32 * inv).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def decode(raw, fmt, dtype, scale, dim):
    raw = np.ascontiguousarray(raw)
    if fmt == "q4":
        return torch.from_numpy(vec_ref.q4_decode(raw, dim)).to(torch.float32).to(dtype)
    t = torch.from_numpy(raw)
    if fmt == "same":
        return t.view(dtype)
    return (t.view(torch.float8_e4m3fn).float() * np.float32(scale)).to(dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt,dim,rot,style", [
    ("q4", 128, 128, "half"), ("q4", 64, 32, "half"), ("q4", 96, 96, "interleaved"), ("q4", 32, 32, "half"),
    ("q4", 160, 40, "half"), ("q4", 256, 128, "half"), ("q4", 192, 0, "half"), ("same", 128, 64, "interleaved"),
    ("same", 80, 80, "half"), ("same", 8, 0, "half"), ("e4m3", 128, 128, "half"), ("e4m3", 48, 16, "interleaved"),
    ("e4m3", 256, 0, "half")])
@pytest.mark.parametrize("page", [dict(T=16, page_first=False, hnd=False), dict(T=1, page_first=True, hnd=True),
                                  dict(T=17, page_first=True, hnd=False, offset=48),
                                  dict(T=64, page_first=False, hnd=True, split=True)])
def test_append_and_fetch(dtype, fmt, dim, rot, style, page):
    """Pool bytes are the definition's, bit for bit, and no other byte of the allocation changes;
    fetch gives the held values rounded once."""
    dt, code = DT[dtype]
    H, Hq, n = 3, 7, 37
    g = gen(dim + rot)
    with Pool(dim, fmt, H=H, P=-(-n // page["T"]) + 5, **page) as p:
        qkv = torch.randn(n, Hq + 2 * H, dim, generator=g, device="cuda")
        qkv[:, Hq] *= 30.0                         # one head is loud
        qkv = qkv.to(dt)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        slots = torch.randperm(p.P * p.T, generator=g, device="cuda")[:n]
        slots[5] = -1
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
        k32, v32 = k.float().cpu().numpy(), v.float().cpu().numpy()
        if rot:
            rows32 = rows.cpu().numpy()
            k32 = vec_ref.turn(k32, rows32, style)
            q32 = vec_ref.turn(q.float().cpu().numpy(), rows32, style)
            assert np.array_equal(bits(q_out), torch.from_numpy(q32).to(dt).contiguous().view(torch.uint8).numpy())
            kvb.kv_rotary_close(rotary)
        at = slots.cpu().numpy()
        live = at >= 0
        for comp, x, s in ((0, k32, ks), (1, v32, vs)):
            p.view(want, 1, comp)[at[live] // p.T, at[live] % p.T] = encode(x, fmt, dt, s)[live]
        got = p.alloc.cpu().numpy()
        assert np.array_equal(got, want), np.flatnonzero(got != want)[:5]
        assert int(status) == 0

        back = torch.full((2, n, H, dim), 7.0, dtype=dt, device="cuda")
        kvb.kv_fetch(p.pool, kvb.make_fetch_args(kvb.vecs(back[0]), kvb.vecs(back[1]), tokens=n, head_dim=dim,
                                                 dtype=code, format=FMT[fmt], layer=1, slots=slots.data_ptr(),
                                                 k_scale=ks, v_scale=vs, status=status.data_ptr()))
        torch.cuda.synchronize()
        for comp, s in ((0, ks), (1, vs)):
            held = decode(p.view(want, 1, comp)[np.maximum(at, 0) // p.T, np.maximum(at, 0) % p.T], fmt, dt, s, dim)
            held = torch.where(torch.from_numpy(live)[:, None, None], held, torch.zeros_like(held))
            # -0 and 0 are the same value
            assert torch.equal(back[comp].cpu(), held)
        assert int(status) == 0


def test_append_special_values():
    """Groups with NaN or infinity, of zeros, of one sign, of the type's largest and least values."""
    x = torch.randn(8, 2, 64, generator=gen(2), device="cuda")
    x[0, 0, 3], x[1, 0, 40], x[1, 1, 5] = float("nan"), float("inf"), -float("inf")
    x[2] = 0.0
    x[3] = x[3].abs() + 3
    x[4] = -x[4].abs() - 3
    x[5], x[5, :, ::2] = torch.finfo(torch.bfloat16).max, torch.finfo(torch.bfloat16).min
    x[6] = 1e-38
    x[7, 0, :32], x[7, 0, 7] = 0.0, -2.5
    x = x.to(torch.bfloat16)
    with Pool(64, "q4", T=4, H=2, P=3) as p:
        slots = torch.arange(8, device="cuda")
        want = p.alloc.cpu().numpy().copy()
        for comp in (0, 1):
            p.view(want, 0, comp)[np.arange(8) // 4, np.arange(8) % 4] = vec_ref.q4_encode(x.float().cpu().numpy())
        kvb.kv_append(p.pool, None, kvb.make_append_args(kvb.vecs(x), kvb.vecs(x), tokens=8, head_dim=64, dtype=0,
                                                         format=FMT["q4"], layer=0, slots=slots.data_ptr()))
        back = torch.empty_like(x)
        kvb.kv_fetch(p.pool, kvb.make_fetch_args(kvb.vecs(back), None, tokens=8, head_dim=64, dtype=0,
                                                 format=FMT["q4"], layer=0, slots=slots.data_ptr()))
        torch.cuda.synchronize()
        assert np.array_equal(p.alloc.cpu().numpy(), want)
        nan = torch.isnan(back).view(8, 2, 2, 32).all(-1)
        assert nan[0, 0, 0] and nan[1, 0, 1] and nan[1, 1, 0] and int(nan.sum()) == 3
        assert int(torch.isnan(back).sum()) == 96
        assert not back[2].any() and not back[6].any()
        # -max / s = -7.5 rounds to -8, and -8 s is past bfloat16: the held value, rounded
        held = torch.from_numpy(vec_ref.q4_decode(vec_ref.q4_encode(x[5].float().cpu().numpy()), 64)).float()
        assert torch.equal(back[5].cpu(), held.to(torch.bfloat16))


def test_slots_outside_the_pool():
    """Left out and reported; nothing else is touched (the address code is tested on the CPU)."""
    with Pool(64, "q4", T=4, H=2, P=3) as p:
        x = torch.randn(5, 2, 64, device="cuda").to(torch.float16)
        slots = torch.tensor([12, -2, 2 ** 40, -1, 3], device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        want = p.alloc.cpu().numpy().copy()
        for comp in (0, 1):
            p.view(want, 0, comp)[0, 3] = vec_ref.q4_encode(x[4].float().cpu().numpy())
        args = dict(tokens=5, head_dim=64, dtype=1, format=FMT["q4"], layer=0, slots=slots.data_ptr())
        kvb.kv_append(p.pool, None, kvb.make_append_args(kvb.vecs(x), kvb.vecs(x), **args))
        back = torch.full_like(x, 3.0)
        kvb.kv_fetch(p.pool, kvb.make_fetch_args(None, kvb.vecs(back), status=status.data_ptr(), **args))
        torch.cuda.synchronize()
        assert np.array_equal(p.alloc.cpu().numpy(), want)
        assert int(status) == kvb.KV_STATUS_BAD_SLOT
        assert not back[:4].any() and back[4].any()
        status.zero_()
        kvb.kv_append(p.pool, None, kvb.make_append_args(kvb.vecs(x), kvb.vecs(x), status=status.data_ptr(), **args))
        torch.cuda.synchronize()
        assert int(status) == kvb.KV_STATUS_BAD_SLOT
        slots.copy_(torch.tensor([-1, -1, 1, -1, 3]))
        status.zero_()
        kvb.kv_append(p.pool, None, kvb.make_append_args(kvb.vecs(x), kvb.vecs(x), status=status.data_ptr(), **args))
        torch.cuda.synchronize()
        assert int(status) == 0


def test_append_in_place_queries():
    with Pool(128, "same", T=8, H=2, P=4) as p:
        x = torch.randn(9, 12, 128, generator=gen(4), device="cuda").to(torch.bfloat16)
        f, gain = vec_ref.frequencies(128)
        rows = torch.from_numpy(vec_ref.rows_of(f, gain, np.arange(9))).float().cuda()
        want = vec_ref.turn(x[:, :8].float().cpu().numpy(), rows.cpu().numpy(), "half")
        rotary = kvb.kv_rotary_create(128)
        q = kvb.vecs(x[:, :8])
        slots = torch.arange(9, device="cuda")
        kvb.kv_append(p.pool, rotary, kvb.make_append_args(
            kvb.vecs(x[:, 8:10]), kvb.vecs(x[:, 10:]), q, q, tokens=9, head_dim=128, dtype=0, format=0, layer=0,
            slots=slots.data_ptr(), q_heads=8, rows=rows.data_ptr()))
        torch.cuda.synchronize()
        kvb.kv_rotary_close(rotary)
        assert torch.equal(x[:, :8].cpu(), torch.from_numpy(want).to(torch.bfloat16))


def test_append_refusals():
    with Pool(64, "q4", T=4, H=2, P=3) as p:
        x = torch.zeros(2, 2, 64, device="cuda", dtype=torch.float16)
        slots = torch.arange(2, device="cuda")
        base = dict(tokens=2, head_dim=64, dtype=1, format=FMT["q4"], layer=0, slots=slots.data_ptr())
        before = p.alloc.clone()
        cpu = torch.zeros(2, dtype=torch.int64)
        rot, rows = kvb.kv_rotary_create(32), torch.zeros(2, 2, 16, device="cuda")
        cases = [
            (dict(layer=2), None, kvb.KV_ERR_OUT_OF_RANGE), (dict(format=0), None, kvb.KV_ERR_LAYOUT),
            (dict(head_dim=96), None, kvb.KV_ERR_LAYOUT), (dict(head_dim=72), None, kvb.KV_ERR_LAYOUT),
            (dict(format=9), None, kvb.KV_ERR_INVALID_ARG), (dict(dtype=2), None, kvb.KV_ERR_INVALID_ARG),
            (dict(slots=None), None, kvb.KV_ERR_INVALID_ARG), (dict(slots=cpu.data_ptr()), None, kvb.KV_ERR_INVALID_ARG),
            (dict(slots=slots.data_ptr() + 4), None, kvb.KV_ERR_ALIGNMENT),
            (dict(rows=rows.data_ptr()), None, kvb.KV_ERR_INVALID_ARG), (dict(), rot, kvb.KV_ERR_INVALID_ARG),
            (dict(q=kvb.vecs(x), q_out=kvb.vecs(x), q_heads=2), None, kvb.KV_ERR_INVALID_ARG),
        ]
        for kw, r, status in cases:
            with pytest.raises(kvb.KvError) as e:
                kvb.kv_append(p.pool, r, kvb.make_append_args(kvb.vecs(x), kvb.vecs(x), **{**base, **kw}))
            assert e.value.status == status, (kw, e.value)
        for fmt, dim in (("e4m3", 48),):
            with Pool(dim, fmt, T=4, H=2, P=3) as p8:
                y = torch.zeros(2, 2, dim, device="cuda", dtype=torch.float16)
                for s in (0.0, -1.0, float("nan"), float("inf")):
                    with pytest.raises(kvb.KvError) as e:
                        kvb.kv_append(p8.pool, None, kvb.make_append_args(
                            kvb.vecs(y), kvb.vecs(y), tokens=2, head_dim=dim, dtype=1, format=FMT[fmt], layer=0,
                            slots=slots.data_ptr(), k_scale=s))
                    assert e.value.status == kvb.KV_ERR_INVALID_ARG
        kvb.kv_rotary_close(rot)
        lay = kvb.make_layout(1, 1, 3, 4, 2, 48, 0, 0, 1)
        latent = kvb.kv_pool_register(lay, p.alloc.data_ptr())
        with pytest.raises(kvb.KvError) as e:
            kvb.kv_append(latent, None, kvb.make_append_args(kvb.vecs(x), kvb.vecs(x), **base))
        assert e.value.status == kvb.KV_ERR_LAYOUT
        kvb.kv_pool_close(latent)
        stale = kvb.kv_pool_register(kvb.kv_pool_info(p.pool)[0], p.alloc.data_ptr(), 0, 7001, 1)
        kvb.kv_pool_retire(7001, 2)
        with pytest.raises(kvb.KvError) as e:
            kvb.kv_append(stale, None, kvb.make_append_args(kvb.vecs(x), kvb.vecs(x), **base))
        assert e.value.status == kvb.KV_ERR_STALE
        kvb.kv_pool_close(stale)
        torch.cuda.synchronize()
        assert torch.equal(p.alloc, before)


# ------------------------------------------------------------------- attend

class Batch:
    """Requests with their pages; what is past a request's length is stale bytes."""

    def __init__(self, lens, n_q, H, group, dim, T, dtype, window=0, seed=1, page_first=False, hnd=False, offset=0,
                 split=False, k_mul=1.0, v_mul=None, layer=1):
        self.dt, self.code = DT[dtype]
        g = gen(seed)
        self.lens, self.n_q, self.H, self.group, self.dim, self.T = lens, n_q, H, group, dim, T
        self.window, self.layer = window, layer
        r, per = len(lens), max(1, -(-max(lens) // T))
        self.pool = Pool(dim, "q4", T, H, r * per + 3, 2, page_first, hnd, offset, split, seed)
        self.table = torch.randperm(self.pool.P, generator=g, device="cuda")[:r * per].view(r, per).int()
        self.kv = []
        tab = self.table.cpu().numpy()
        raw = self.pool.alloc.cpu().numpy()
        for i, n in enumerate(lens):
            both = []
            for comp in (0, 1):
                x = torch.randn(n, H, dim, generator=g, device="cuda")
                if comp == 0:
                    x = (x * torch.exp(0.5 * torch.randn(H, dim, generator=g, device="cuda")) + 0.3) * k_mul
                elif v_mul is not None:
                    x = x * torch.tensor(v_mul, device="cuda").repeat_interleave(32)[:dim]
                both.append(vec_ref.q4_encode(x.cpu().numpy()))
                at = np.arange(n)
                self.pool.view(raw, layer, comp)[tab[i][at // T], at % T] = both[-1]
            self.kv.append(both)
        self.pool.alloc.copy_(torch.from_numpy(raw))
        self.q = torch.randn(sum(n_q), H * group, dim, generator=g, device="cuda").to(self.dt)
        self.scale = 1.0 / dim ** 0.5

    def args(self, q=None, **kw):
        q = self.q if q is None else q
        self.out = torch.full((max(1, q.shape[0]), self.H * self.group, self.dim), 7.0, dtype=self.dt, device="cuda")
        self.lse = torch.full((max(1, q.shape[0]), self.H * self.group), 7.0, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.q_start = torch.tensor([0] + list(np.cumsum(self.n_q)), dtype=torch.int32, device="cuda")
        self.lens_d = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        d = dict(q_start=self.q_start.data_ptr(), lens=self.lens_d.data_ptr(), pages=self.table.data_ptr(),
                 pages_stride=self.table.stride(0), requests=len(self.lens), tokens=q.shape[0], max_q=max(self.n_q),
                 max_len=max(self.lens), q_heads=self.H * self.group, head_dim=self.dim, dtype=self.code,
                 layer=self.layer, scale=self.scale, window=self.window, lse=self.lse.data_ptr(),
                 status=self.status.data_ptr())
        a = kvb.make_attend_args(kvb.vecs(q), kvb.vecs(self.out), **{**d, **kw})
        need = kvb.kv_attend_workspace(self.pool.pool, a)
        self.work = torch.full((need // 4 + 4,), float("nan"), device="cuda")    # whatever it held
        a.workspace, a.workspace_bytes = self.work.data_ptr(), need
        return a

    def run(self, stream=None, q=None, **kw):
        kvb.kv_attend(self.pool.pool, self.args(q, **kw), stream)
        torch.cuda.synchronize()
        return self.out, self.lse, int(self.status)

    def check(self, out, lse, q=None, requests=None):
        """Rounding bounds.  Scores: products of exact codes summed in float32 (2^-20 of the sum
        of absolute products leaves room for truncating adders), the argument and the result of
        exp2 2^-22 of |x| and of 1; so a weight is off by dx and out by 2 dx max|v|.  Weights times
        steps rounded to fp16: 2^-11 of each |p step (code - 8)|, and 2^-24 of the largest step a
        token for those below fp16's normal range.  Then one rounding to the output's type.
        With many query rows a request the tensor-core kernel runs, which also rounds every key
        and value to fp16 (2^-11 each), and a query to 2^-22 of the row's largest |q| x step."""
        q = (self.q if q is None else q).double().cpu().numpy()
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        at = 0
        for i, n in enumerate(self.n_q):
            if requests is None or i in requests:
                k, v = (vec_ref.q4_decode(x, self.dim) for x in self.kv[i])
                qi = q[at:at + n]
                want, wl, w = vec_ref.attend(qi, k, v, self.scale, self.window)
                c, _, s = vec_ref.q4_parts(self.kv[i][1], self.dim)
                _, _, ks = vec_ref.q4_parts(self.kv[i][0], self.dim)
                for j in range(self.H * self.group):
                    h = j // self.group
                    seen = w[j].any(1)
                    if self.lens[i] == 0 or not seen.any():
                        assert not out[at:at + n, j].any() and np.all(np.isneginf(lse[at:at + n, j]))
                        continue
                    dx = 2.0 ** -20 * self.scale * 24 * (np.abs(qi[:, j])[:, None] * ks[None, :, h]).sum(2).max(1)
                    dx += 2.0 ** -21 * (1 + np.abs(wl[:, j]).clip(max=1e30))
                    vmax = np.abs(v[:, h]).max(0)
                    tol = half_step(self.dt) * np.abs(want[:, j]) * (1 + 2 ** -7)
                    tol = tol + 2.0 ** -11 * (w[j] @ (s[:, h] * np.abs(c[:, h] - 8)))
                    tol = tol + 2.0 ** -24 * 8 * self.lens[i] * s[:, h].max(0)[None] / np.maximum(1, 1)
                    if self.dim <= 128 and max(self.n_q) * self.group >= 64:
                        both = np.abs(qi[:, j])[:, None] * np.abs(k[None, :, h])
                        dx = dx + self.scale * 2.0 ** -11 * both.sum(2).max(1)
                        dx = dx + self.scale * 2.0 ** -22 * 16 * self.dim * (np.abs(qi[:, j])[:, None] * ks[None, :, h]).max((1, 2))
                        tol = tol + 2.0 ** -11 * (w[j] @ np.abs(v[:, h]))
                    tol = tol + 2 * dx[:, None] * vmax[None] + (2.0 ** -24 if self.dt == torch.float16 else 0)
                    err = np.abs(out[at:at + n, j] - want[:, j])
                    ok = ~seen | (err <= tol).all(1)
                    assert ok.all(), (i, j, float((err / tol).max()))
                    assert not out[at:at + n, j][~seen].any()
                    el = np.abs(lse[at:at + n, j][seen] - wl[:, j][seen])
                    assert np.all(el <= dx[seen] + 2.0 ** -22 * np.abs(wl[:, j][seen])), float(el.max())
                    assert np.all(np.isneginf(lse[at:at + n, j][~seen]))
            at += n

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.pool.__exit__()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,H,group", [(128, 2, 4), (64, 3, 1), (96, 1, 8), (128, 1, 12), (192, 2, 3), (256, 2, 5),
                                         (64, 2, 16)])
@pytest.mark.parametrize("page", [dict(T=16, page_first=False, hnd=False), dict(T=17, page_first=True, hnd=True),
                                  dict(T=1, page_first=True, hnd=False, offset=48),
                                  dict(T=64, page_first=False, hnd=True, split=True)])
def test_attend_one_token(dtype, dim, H, group, page):
    lens = [1, 0, 31, 32, 33, 257, 600]
    with Batch(lens, [1] * len(lens), H, group, dim, dtype=dtype, **page) as b:
        out, lse, status = b.run()
        b.check(out, lse)
        assert status == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("window", [0, 1, 20, 100])
@pytest.mark.parametrize("dim,H,group", [(128, 2, 4), (64, 1, 3), (256, 1, 2)])
def test_attend_several_tokens(dtype, window, dim, H, group):
    """Ragged counts of new tokens, one more than the cached tokens hold, none at all."""
    with Batch([300, 5, 64, 40, 0, 129, 7], [5, 5, 0, 33, 2, 1, 9], H, group, dim, 16, dtype, window) as b:
        out, lse, status = b.run()
        b.check(out, lse)
        assert status == 0


@pytest.mark.parametrize("dim,n", [(128, 90), (64, 200), (128, 257), (96, 70)])
@pytest.mark.parametrize("window", [0, 150])
def test_attend_prompt_chunk(dim, n, window):
    with Batch([700, n, 300], [n, n, 64], 2, 4, dim, 16, "bf16", window) as b:
        out, lse, status = b.run()
        b.check(out, lse)
        assert status == 0


@pytest.mark.parametrize("dim,dtype", [(128, "bf16"), (64, "fp16"), (256, "bf16")])
def test_attend_long(dim, dtype):
    """Long enough to be cut along the tokens and joined."""
    with Batch([9000, 100, 5001], [1, 1, 2], 1, 4, dim, 32, dtype, hnd=True, page_first=True) as b:
        a = b.args()
        assert a.workspace_bytes > 0
        out, lse, status = b.run()
        b.check(out, lse)
        assert status == 0
        first = out.clone()
        out, _, _ = b.run()
        assert torch.equal(out, first)      # no order of arrival in the result


@pytest.mark.parametrize("k_mul,v_mul", [(40.0, None), (1e-6, None), (1.0, [1e-20, 1.0, 1e20, 1e4]),
                                         (1.0, [1e-25, 1e-25, 3e-20, 1e30])])
def test_attend_ranges(k_mul, v_mul):
    """Sharp and flat softmax; values whose groups differ by powers of 10^20."""
    with Batch([257, 40, 1000], [1, 3, 1], 1, 4, 128, 16, "bf16", k_mul=k_mul, v_mul=v_mul) as b:
        out, lse, status = b.run()
        b.check(out, lse)


@pytest.mark.parametrize("mul", [1e-20, 1e20, 1e-30])
def test_attend_query_ranges(mul):
    with Batch([257, 40], [1, 3], 1, 4, 128, 16, "bf16", k_mul=1.0) as b:
        b.scale = float(np.float32(0.088 / mul))
        q = (b.q.float() * mul).to(torch.bfloat16)
        out, lse, _ = b.run(q=q)
        b.check(out, lse, q=q)


def test_attend_step_sizes_that_rise_late():
    """A group whose steps grow by 10^6 after the first tokens."""
    with Batch([400], [1], 1, 2, 64, 16, "bf16") as b:
        raw = b.pool.alloc.cpu().numpy()
        x = vec_ref.q4_decode(b.kv[0][1], 64).astype(np.float32)
        x[300:] *= 1e6
        b.kv[0][1] = vec_ref.q4_encode(x)
        at, tab = np.arange(400), b.table.cpu().numpy()[0]
        b.pool.view(raw, 1, 1)[tab[at // 16], at % 16] = b.kv[0][1]
        b.pool.alloc.copy_(torch.from_numpy(raw))
        out, lse, _ = b.run()
        b.check(out, lse)


# The kernel for many query rows: 256 rows a block, 64 cached tokens at a time.

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,H,group,n_q,lens", [
    (128, 1, 4, [64], [64]), (128, 2, 1, [128, 65, 0], [128, 129, 5]), (64, 3, 8, [33, 8], [500, 8]),
    (96, 1, 5, [40, 13], [257, 13]), (128, 1, 16, [8, 8, 8], [300, 127, 4]), (64, 1, 2, [300], [1100]),
    (128, 1, 3, [43], [129])])
@pytest.mark.parametrize("page", [dict(T=16, page_first=False, hnd=False), dict(T=17, page_first=True, hnd=True, offset=48),
                                  dict(T=64, page_first=False, hnd=True, split=True)])
def test_attend_many_rows(dtype, dim, H, group, n_q, lens, page):
    with Batch(lens, n_q, H, group, dim, dtype=dtype, **page) as b:
        out, lse, status = b.run()
        b.check(out, lse)
        assert status == 0


@pytest.mark.parametrize("window", [1, 5, 100, 129])
@pytest.mark.parametrize("dim", [64, 128])
def test_attend_many_rows_window(window, dim):
    with Batch([400, 70, 0], [90, 70, 20], 1, 4, dim, 16, "bf16", window) as b:
        out, lse, status = b.run()
        b.check(out, lse)
        assert status == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n_q,lens", [([64, 65], [64, 300]), ([20, 3, 20], [6000, 100, 5500])])
def test_attend_many_rows_without_lse(dtype, n_q, lens):
    """Where no logarithms are wanted the keys are rounded to fp16 (as `check` allows)."""
    with Batch(lens, n_q, 1, 4, 128, 16, dtype) as b:
        out, lse, status = b.run()
        exact = lse.clone()
        out, lse, status = b.run(lse=None)
        assert (lse == 7).all() and status == 0
        b.check(out, exact)


def test_attend_many_rows_lse_of_few_terms():
    """Sums of few terms: 2^-18 of the sizes of the products, with keys in two parts."""
    with Batch([8, 3], [8, 3], 1, 16, 64, 16, "fp16", k_mul=3.0) as b:
        _, lse, _ = b.run()
        at = 0
        for i, n in enumerate(b.n_q):
            k, v = (vec_ref.q4_decode(x, 64) for x in b.kv[i])
            q = b.q[at:at + n].double().cpu().numpy()
            _, want, _ = vec_ref.attend(q, k, v, b.scale)
            size = b.scale * np.abs(q).max() * np.abs(k).max() * 64
            assert np.abs(lse[at:at + n].double().cpu().numpy() - want).max() <= 2.0 ** -18 * size
            at += n


def test_attend_many_rows_cut_and_joined():
    with Batch([6000, 100, 5500], [20, 3, 20], 1, 4, 128, 32, "bf16") as b:
        assert b.args().workspace_bytes > 0
        out, lse, status = b.run()
        b.check(out, lse)
        first = out.clone()
        out, _, _ = b.run()
        assert torch.equal(out, first)


@pytest.mark.parametrize("k_mul,v_mul", [(40.0, None), (1e-6, None), (1.0, [1e-20, 1.0, 1e20, 1e4]),
                                         (1.0, [1e-25, 1e-25, 3e-20, 1e30])])
def test_attend_many_rows_ranges(k_mul, v_mul):
    with Batch([257, 70], [30, 20], 1, 4, 128, 16, "bf16", k_mul=k_mul, v_mul=v_mul) as b:
        out, lse, status = b.run()
        b.check(out, lse)


@pytest.mark.parametrize("sign", [-1.0, 0.0])
@pytest.mark.parametrize("n_q", [2, 40])
def test_attend_scale_signs(sign, n_q):
    with Batch([257], [n_q], 1, 4, 128, 16, "bf16") as b:
        b.scale *= sign
        out, lse, _ = b.run()
        b.scale = abs(b.scale)             # the tolerances go by its size; 0 is a plain mean
        if sign:
            q = -b.q
            want, _, _ = b.run(q=q)
            assert torch.equal(out, want)
        else:
            v = vec_ref.q4_decode(b.kv[0][1], 128)
            pos = 257 - n_q + np.arange(n_q)
            want = np.stack([v[:p + 1, 0].mean(0) for p in pos])[:, None]
            # rounding: 2^-8 of the result, 2^-10 of the mean size of a value
            assert np.all(np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * np.abs(v).mean())


@pytest.mark.parametrize("comp,groups", [(0, [0]), (1, [0]), (1, [1, 3]), (1, [0, 1, 2, 3])])
def test_attend_many_rows_nan_behind_the_mask(comp, groups):
    """A NaN among the keys makes every value NaN of the queries that see it; a NaN group among
    the values, those of that group."""
    with Batch([60, 60], [40, 40], 1, 2, 128, 16, "bf16", window=30) as b:
        x = np.zeros((1, 128), np.float32)
        for g in groups:
            x[:, 32 * g:32 * g + 32] = np.nan
        poke(b, 0, 57, comp, vec_ref.q4_encode(x))     # new token 37: seen by 37, 38, 39
        poke(b, 1, 5, comp, vec_ref.q4_encode(x))      # seen up to position 34: new tokens 0..14
        out, _, _ = b.run()
        out = out.clone()
        nan = torch.isnan(out.float())
        seen = torch.zeros(80, dtype=torch.bool, device="cuda")
        seen[37:40], seen[40:55] = True, True
        want_nan = torch.zeros_like(nan)
        cols = range(128) if comp == 0 else [32 * g + e for g in groups for e in range(32)]
        want_nan[:, :, list(cols)] = seen[:, None, None]
        assert torch.equal(nan, want_nan)
        want, _, _ = b_without(b)
        assert torch.equal(out[~seen], want[~seen])


def test_attend_many_rows_query_nan_stays_in_its_row():
    with Batch([300], [70], 1, 2, 128, 16, "bf16") as b:
        out, _, _ = b.run()
        want = out.clone()
        q = b.q.clone()
        q[1, 1, 5], q[69, 0, 9] = float("nan"), float("inf")
        out, _, _ = b.run(q=q)
        bad = torch.isnan(out.float()).all(-1)
        assert bad.nonzero().tolist() == [[1, 1], [69, 0]]
        assert torch.equal(out[~bad], want[~bad])


def test_attend_many_rows_bad_pages():
    with Batch([200, 200, 50], [40, 40, 10], 1, 2, 64, 16, "bf16", window=60) as b:
        b.table[0, 1] = b.pool.P            # tokens 16..31: outside every window
        b.table[1, 9] = -1                  # tokens 144..159: positions 144..218, all but none of 160..199
        b.table[2, 9] = 2 ** 31 - 1         # past its length
        out, lse, status = b.run()
        assert status == kvb.KV_STATUS_BAD_PAGE
        assert torch.isnan(out[40:80].float()).all() and torch.isnan(lse[40:80]).all()
        b.check(out, lse, requests=(0, 2))


def poke(b, i, token, comp, raw_vec):
    tab = b.table.cpu().numpy()[i]
    raw = b.pool.alloc.cpu().numpy()
    b.pool.view(raw, b.layer, comp)[tab[token // b.T], token % b.T] = raw_vec
    b.pool.alloc.copy_(torch.from_numpy(raw))


@pytest.mark.parametrize("comp", [0, 1])
@pytest.mark.parametrize("dim", [64, 128])
def test_attend_nan_behind_the_mask(comp, dim):
    """A cached NaN reaches the queries that see it and no other: not those before it, not
    those whose window has passed it."""
    with Batch([60, 60], [6, 6], 1, 2, dim, 16, "bf16", window=30) as b:
        nan = np.full((1, b.pool.B), 0, np.uint8)
        nan[:, :] = vec_ref.q4_encode(np.full((1, dim), np.nan, np.float32))
        poke(b, 0, 57, comp, nan)          # the place of new token 3: tokens 0..2 do not see it
        poke(b, 1, 27, comp, nan)          # left the window of new tokens 3.. (54 + 3 - 30 = 27)
        out, lse, status = b.run()
        seen = torch.isnan(out.float()).all(-1).all(-1)
        assert seen.tolist() == [False] * 3 + [True] * 3 + [True] * 3 + [False] * 3
        # the others are what they are without it
        want, _, _ = b_without(b)
        keep = ~seen
        assert torch.equal(out[keep], want[keep])


def b_without(b):
    """The same batch with its own values everywhere."""
    raw = b.pool.alloc.cpu().numpy()
    tab = b.table.cpu().numpy()
    for i, n in enumerate(b.lens):
        at = np.arange(n)
        for comp in (0, 1):
            b.pool.view(raw, b.layer, comp)[tab[i][at // b.T], at % b.T] = b.kv[i][comp]
    b.pool.alloc.copy_(torch.from_numpy(raw))
    out, lse, status = b.run()
    return out.clone(), lse, status


def test_attend_query_nan_stays_in_its_row():
    with Batch([100], [4], 1, 2, 128, 16, "bf16") as b:
        out, _, _ = b.run()
        want = out.clone()
        q = b.q.clone()
        q[1, 1, 5], q[3, 0, 9] = float("nan"), float("inf")
        out, _, _ = b.run(q=q)
        bad = torch.isnan(out.float()).all(-1)
        assert bad.nonzero().tolist() == [[1, 1], [3, 0]]
        assert torch.equal(out[~bad], want[~bad])


def test_attend_bad_pages():
    """Page ids outside the pool: reported, NaN for the queries that see them, the others right.
    (The kernels' own check of page ids is tested on the CPU first.)"""
    with Batch([100, 100, 50], [2, 1, 1], 1, 2, 64, 16, "bf16", window=40) as b:
        b.table[0, 1] = b.pool.P            # tokens 16..31: outside every window
        b.table[1, 4] = -1                  # tokens 64..79: seen
        b.table[2, 6] = 2 ** 31 - 1         # past its length
        out, lse, status = b.run()
        assert status == kvb.KV_STATUS_BAD_PAGE
        assert torch.isnan(out[2].float()).all() and torch.isnan(lse[2]).all()
        b.check(out, lse, requests=(0, 2))
        b.table[1, 4] = 0
        _, _, status = b.run()
        assert status == 0


def test_attend_bad_lengths():
    with Batch([100, 64, 50, 30], [2, 1, 1, 3], 1, 2, 64, 16, "bf16") as b:
        a = b.args()
        b.lens_d[1] = -4                    # taken as 0: sees nothing
        b.q_start[3] = 1                    # request 2 out of order (3..1), request 3 too long (1..7)
        kvb.kv_attend(b.pool.pool, a)
        torch.cuda.synchronize()
        assert int(b.status) == kvb.KV_STATUS_BAD_LENGTH
        b.check(b.out, b.lse, requests=(0,))
        assert not b.out[2].any() and torch.isneginf(b.lse[2]).all()
        assert (b.out[3:] == 7).all() and (b.lse[3:] == 7).all()      # left out
        b.lens_d[0] = 101                   # taken as max_len
        b.status.zero_()
        kvb.kv_attend(b.pool.pool, a)
        torch.cuda.synchronize()
        assert int(b.status) == kvb.KV_STATUS_BAD_LENGTH
        b.check(b.out, b.lse, requests=(0,))


def test_attend_strided_queries_and_streams():
    with Batch([300, 90], [3, 2], 2, 4, 128, 16, "bf16") as b:
        out, _, _ = b.run()
        want = out.clone()
        wide = torch.zeros(5, 20, 128, dtype=torch.bfloat16, device="cuda")
        wide[:, 4:12] = b.q
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        out, _, _ = b.run(stream.cuda_stream, q=wide[:, 4:12])
        assert torch.equal(out, want)


def test_attend_far_offsets():
    """A pool past 4 GiB, and pages at its end."""
    H, T, dim = 8, 64, 128
    B = vec_ref.q4_bytes(dim)
    P = (5 << 30) // (2 * T * H * B) + 1
    for page_first in (False, True):
        with Pool(dim, "q4", T, H, P, L=1, page_first=page_first) as p:
            x = torch.randn(130, H, dim, generator=gen(8), device="cuda").to(torch.bfloat16)
            table = torch.tensor([[P - 1, P // 2, P - 2]], dtype=torch.int32, device="cuda")
            slots = table[0].long()[torch.arange(130, device="cuda") // T] * T + torch.arange(130, device="cuda") % T
            kvb.kv_append(p.pool, None, kvb.make_append_args(kvb.vecs(x), kvb.vecs(x), tokens=130, head_dim=dim,
                                                             dtype=0, format=FMT["q4"], layer=0, slots=slots.data_ptr()))
            held = torch.empty_like(x)
            kvb.kv_fetch(p.pool, kvb.make_fetch_args(None, kvb.vecs(held), tokens=130, head_dim=dim, dtype=0,
                                                     format=FMT["q4"], layer=0, slots=slots.data_ptr()))
            q = torch.randn(1, H, dim, generator=gen(9), device="cuda").to(torch.bfloat16)
            out = torch.empty_like(q)
            qs, lens = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([130], dtype=torch.int32, device="cuda")
            a = kvb.make_attend_args(kvb.vecs(q), kvb.vecs(out), q_start=qs.data_ptr(), lens=lens.data_ptr(),
                                     pages=table.data_ptr(), pages_stride=3, requests=1, tokens=1, max_q=1, max_len=130,
                                     q_heads=H, head_dim=dim, dtype=0, layer=0, scale=0.1)
            work = torch.empty(max(1, kvb.kv_attend_workspace(p.pool, a)), dtype=torch.uint8, device="cuda")
            a.workspace, a.workspace_bytes = work.data_ptr(), work.numel()
            kvb.kv_attend(p.pool, a)
            torch.cuda.synchronize()
            kv = vec_ref.q4_decode(vec_ref.q4_encode(x.float().cpu().numpy()), dim)
            assert torch.equal(held.cpu(), torch.from_numpy(kv).float().to(torch.bfloat16))
            want, _, _ = vec_ref.attend(q.double().cpu().numpy(), kv, kv, 0.1)
            # 2^-8 of the result, 2^-11 of the weights' products (at most 8 steps of ~0.4), scores 2^-10
            assert np.abs(out.double().cpu().numpy() - want).max() <= 2.0 ** -8 * np.abs(want).max() + 2.0 ** -11 * 4 + 2.0 ** -10


def test_attend_refusals():
    with Batch([100, 64], [2, 1], 2, 2, 64, 16, "bf16") as b:
        a = b.args()
        before = b.out.clone()

        def refused(status, **kw):
            a = b.args()
            for name, val in kw.items():
                setattr(a, name, val)
            with pytest.raises(kvb.KvError) as e:
                kvb.kv_attend(b.pool.pool, a)
            assert e.value.status == status, (kw, e.value)

        INV, LAY, OOR, ALI = kvb.KV_ERR_INVALID_ARG, kvb.KV_ERR_LAYOUT, kvb.KV_ERR_OUT_OF_RANGE, kvb.KV_ERR_ALIGNMENT
        refused(OOR, layer=2)
        refused(LAY, head_dim=32)
        refused(LAY, head_dim=96)
        refused(INV, head_dim=60)
        refused(INV, dtype=2)
        refused(INV, q_heads=3)
        refused(INV, q_heads=0)
        refused(INV, max_q=9)
        refused(INV, scale=float("nan"))
        refused(INV, scale=float("inf"))
        refused(INV, max_len=2 ** 30 + 1, pages_stride=2 ** 31)
        refused(INV, lens=None)
        refused(INV, q_start=None)
        refused(INV, pages=None)
        refused(INV, pages_stride=6)
        refused(INV, q=kvb.kv_vecs(0, 128, 64))
        refused(ALI, out=kvb.kv_vecs(b.out.data_ptr() + 2, 256, 64))
        refused(ALI, lse=b.lse.data_ptr() + 2)
        cpu = torch.zeros(64, dtype=torch.int32)
        refused(INV, pages=cpu.data_ptr())
        refused(INV, lens=cpu.data_ptr())
        a = b.args()
        a.reserved[1] = 1
        with pytest.raises(kvb.KvError):
            kvb.kv_attend(b.pool.pool, a)
        torch.cuda.synchronize()
        assert torch.equal(b.out, before)
    with Batch([9000], [1], 1, 2, 64, 16, "bf16") as b:
        a = b.args()
        assert a.workspace_bytes > 0
        a.workspace_bytes -= 1
        with pytest.raises(kvb.KvError) as e:
            kvb.kv_attend(b.pool.pool, a)
        assert e.value.status == kvb.KV_ERR_OUT_OF_RANGE
        a.workspace_bytes, a.workspace = a.workspace_bytes + 1, None
        with pytest.raises(kvb.KvError) as e:
            kvb.kv_attend(b.pool.pool, a)
        assert e.value.status == kvb.KV_ERR_INVALID_ARG


def test_attend_of_empty_requests_and_wide_windows():
    """No cached token anywhere (no page table either); a window past every length."""
    with Batch([0, 0], [2, 1], 1, 2, 64, 16, "bf16") as b:
        a = b.args(max_len=0, pages=None)
        kvb.kv_attend(b.pool.pool, a)
        torch.cuda.synchronize()
        assert not b.out.any() and torch.isneginf(b.lse).all() and int(b.status) == 0
    with Batch([0], [40], 1, 2, 128, 16, "bf16") as b:          # the kernel for many rows
        kvb.kv_attend(b.pool.pool, b.args(max_len=0, pages=None))
        torch.cuda.synchronize()
        assert not b.out.any() and torch.isneginf(b.lse).all()
    for n_q in ([3], [60]):
        with Batch([300], n_q, 1, 2, 128, 16, "bf16") as b:
            out, lse, _ = b.run()
            want = out.clone()
            out, _, _ = b.run(window=2 ** 32 - 1)
            assert torch.equal(out, want)


def test_e4m3_saturates():
    x = torch.tensor([1e6, -1e6, float("inf"), -float("inf"), float("nan"), 448.0, 0.001, 0.0] * 6, device="cuda")
    x = x.view(1, 1, 48).to(torch.bfloat16)
    with Pool(48, "e4m3", T=2, H=1, P=2) as p:
        slots = torch.tensor([3], device="cuda")
        args = dict(tokens=1, head_dim=48, dtype=0, format=FMT["e4m3"], layer=1, slots=slots.data_ptr(), k_scale=1.0, v_scale=2.0)
        kvb.kv_append(p.pool, None, kvb.make_append_args(kvb.vecs(x), kvb.vecs(x), **args))
        k, v = torch.empty_like(x), torch.empty_like(x)
        kvb.kv_fetch(p.pool, kvb.make_fetch_args(kvb.vecs(k), kvb.vecs(v), **args))
        torch.cuda.synchronize()
        for got, top in ((k, 448.0), (v, 896.0)):
            got = got.float().view(6, 8)
            assert (got[:, 0] == top).all() and (got[:, 1] == -top).all() and (got[:, 2] == top).all()
            assert (got[:, 3] == -top).all() and torch.isnan(got[:, 4]).all() and (got[:, 7] == 0).all()
            assert (got[:, 5] == 448.0).all()


def test_nothing_to_do():
    n0 = kvb.kv_launch_count()
    with Batch([100], [1], 1, 2, 64, 16, "bf16") as b:
        for kw in (dict(requests=0), dict(tokens=0, max_q=0), dict(max_q=0)):
            kvb.kv_attend(b.pool.pool, b.args(**kw))
        x = torch.zeros(1, 1, 64, device="cuda", dtype=torch.bfloat16)
        d = dict(tokens=0, head_dim=64, dtype=0, format=FMT["q4"], layer=0, slots=None)
        kvb.kv_append(b.pool.pool, None, kvb.make_append_args(kvb.vecs(x), kvb.vecs(x), **d))
        kvb.kv_fetch(b.pool.pool, kvb.make_fetch_args(kvb.vecs(x), None, **d))
    assert kvb.kv_launch_count() == n0


def test_a_step_in_a_graph():
    """Rotate, append and attend captured once and replayed over new inputs in the same buffers."""
    H, group, dim, T = 2, 4, 128, 16
    with Pool(dim, "q4", T, H, 8) as p:
        rotary = kvb.kv_rotary_create(dim)
        n = 3                                                  # three requests, a token a step
        qkv = torch.zeros(n, H * group + 2 * H, dim, device="cuda", dtype=torch.bfloat16)
        q, k, v = qkv[:, :H * group], qkv[:, H * group:H * group + H], qkv[:, H * group + H:]
        q_out, out = torch.empty(n, H * group, dim, device="cuda", dtype=torch.bfloat16), torch.empty(n, H * group, dim, device="cuda", dtype=torch.bfloat16)
        rows = torch.empty(n, 2, dim // 2, device="cuda")
        pos = torch.zeros(n, dtype=torch.int64, device="cuda")
        slots, lens = torch.zeros_like(pos), torch.zeros(n, dtype=torch.int32, device="cuda")
        table = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=torch.int32, device="cuda")
        q_start = torch.arange(n + 1, dtype=torch.int32, device="cuda")
        turn = kvb.make_rotate_args(kvb.kv_vecs(), kvb.kv_vecs(), n, 0, dim, 0, pos.data_ptr(), rows_out=rows.data_ptr())
        add = kvb.make_append_args(kvb.vecs(k), kvb.vecs(v), kvb.vecs(q), kvb.vecs(q_out), tokens=n, head_dim=dim, dtype=0,
                                   format=FMT["q4"], layer=0, slots=slots.data_ptr(), q_heads=H * group, rows=rows.data_ptr())
        att = kvb.make_attend_args(kvb.vecs(q_out), kvb.vecs(out), q_start=q_start.data_ptr(), lens=lens.data_ptr(),
                                   pages=table.data_ptr(), pages_stride=2, requests=n, tokens=n, max_q=1, max_len=2 * T,
                                   q_heads=H * group, head_dim=dim, dtype=0, layer=0, scale=dim ** -0.5)
        assert kvb.kv_attend_workspace(p.pool, att) == 0

        def step(stream):
            kvb.kv_rotate(rotary, turn, stream)
            kvb.kv_append(p.pool, rotary, add, stream)
            kvb.kv_attend(p.pool, att, stream)

        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=side):
            step(side.cuda_stream)
        g, keys, vals = gen(12), [], []
        f, gain = vec_ref.frequencies(dim)
        for t in range(20):
            qkv.copy_(torch.randn(qkv.shape, generator=g, device="cuda"))
            pos.fill_(t)
            slots.copy_(table[:, t // T].long() * T + t % T)
            lens.fill_(t + 1)
            graph.replay()
            torch.cuda.synchronize()
            r32 = rows.cpu().numpy()
            turned = vec_ref.turn(k.float().cpu().numpy(), r32, "half")
            keys.append(vec_ref.q4_decode(vec_ref.q4_encode(turned), dim))
            vals.append(vec_ref.q4_decode(vec_ref.q4_encode(v.float().cpu().numpy()), dim))
            q64 = q_out.double().cpu().numpy()
            for i in range(n):
                want, _, _ = vec_ref.attend(q64[i:i + 1], np.stack([x[i] for x in keys]), np.stack([x[i] for x in vals]), dim ** -0.5)
                # 2^-8 of the result; weights' products 2^-11 x 8 steps of < 0.6; scores 2^-12 x values < 5
                err = np.abs(out[i:i + 1].double().cpu().numpy() - want).max()
                assert err <= 2.0 ** -8 * np.abs(want).max() + 2.0 ** -11 * 5 + 2.0 ** -9, (t, i, err)
        kvb.kv_rotary_close(rotary)
