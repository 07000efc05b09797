"""Operators on head vectors without a GPU: refusals that need no device, and the
address and rounding code of the kernels compiled for the host."""
import ctypes
import os
import shutil
import subprocess
from fractions import Fraction

import numpy as np
import pytest

from hierarchical_kv_cache_backup_gb300 import build as kbuild

kbuild.build_library()
from hierarchical_kv_cache_backup_gb300 import kvb  # noqa: E402

import vec_ref  # noqa: E402

HARNESS = r"""
#include "kvb_vec.h"
using namespace kvb;
extern "C" {
static PoolLayer layer(const uint64_t *g) {   // s_page, s_tok, T, P, mul, shift
    PoolLayer p{};
    p.s_page = g[0]; p.s_tok = (uint32_t)g[1]; p.T = (uint32_t)g[2]; p.P = (uint32_t)g[3];
    p.t_mul = (uint32_t)g[4]; p.t_shift = (uint32_t)g[5];
    return p;
}
int64_t h_slot(const uint64_t *g, int64_t slot) { return slot_offset(layer(g), slot); }
int64_t h_token(const uint64_t *g, const int32_t *table, uint32_t t, int *wrong) {
    bool w = false;
    const int64_t r = token_offset(layer(g), table, t, &w);
    *wrong = w;
    return r;
}
void h_span(const int *in, int *out) {
    bool bad = false;
    const Span s = row_span(in[0], in[1], in[2], in[3], in[4], in[5], in[6], in[7], in[8], in[9], &bad);
    out[0] = s.n; out[1] = s.len; out[2] = s.q0; out[3] = s.lo; out[4] = s.hi; out[5] = bad;
}
int h_vector(const uint64_t *g, uint32_t B, uint32_t page, uint32_t t, uint32_t *out) {
    PoolLayer p = layer(g);
    p.B = B; p.v_page = (uint32_t)(p.s_page / B); p.v_tok = p.s_tok / B;
    *out = vector_index(p, page, t);
    return vector_index_fits(p);
}
float h_round(float x, float s) { return q4_round(x, s, 1.0f / s); }
uint32_t h_step(float lo, float hi) { return q4_step_bits(lo, hi); }
void h_encode(const float *x, uint32_t *word, uint32_t *code) {   // 32 finite values
    float lo = 0, hi = 0;
    for (int i = 0; i < 32; ++i) { lo = fminf(lo, x[i]); hi = fmaxf(hi, x[i]); }
    *word = q4_step_bits(lo, hi);
    for (int i = 0; i < 32; ++i) code[i] = 0;
    if (*word == 0) return;
    const float s = f_bits(*word), inv = 1.0f / s, z = q4_zero(lo, s, inv);
    float c[32];
    for (int i = 0; i < 32; ++i) c[i] = q4_code(x[i], s, inv, z);
    for (int i = 0; i < 32; ++i) code[i] = q4_pack(c + i / 4 * 4) >> (4 * (i % 4)) & 15u;
    *word |= (uint32_t)z;
}
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    d = tmp_path_factory.mktemp("vec")
    src, so = d / "h.cpp", d / "h.so"
    src.write_text(HARNESS)
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no C++ compiler")
    subprocess.run([cc, "-O1", "-std=c++17", "-shared", "-fPIC", "-ffp-contract=off", "-I", kbuild.CSRC,
                    str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.h_slot.restype = lib.h_token.restype = ctypes.c_int64
    lib.h_slot.argtypes = [ctypes.c_void_p, ctypes.c_int64]
    lib.h_token.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint32, ctypes.c_void_p]
    lib.h_round.restype = ctypes.c_float
    lib.h_round.argtypes = [ctypes.c_float, ctypes.c_float]
    lib.h_step.restype = ctypes.c_uint32
    lib.h_step.argtypes = [ctypes.c_float, ctypes.c_float]
    lib.h_vector.argtypes = [ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint32, ctypes.c_uint32, ctypes.c_void_p]
    lib.h_span.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    lib.h_encode.argtypes = [ctypes.c_void_p] * 3
    return lib


def geom(s_page, s_tok, T, P):
    sh = 0
    while (1 << sh) < T:
        sh += 1
    return np.array([s_page, s_tok, T, P, ((1 << 32) * ((1 << sh) - T)) // T + 1, sh], np.uint64)


@pytest.mark.parametrize("T", [1, 3, 16, 17, 256])
@pytest.mark.parametrize("P", [1, 5, 4096, 2 ** 31 - 1])
def test_slot_addresses(host, T, P):
    s_page, s_tok = 40 * T * 640 + 48, 640
    g = geom(s_page, s_tok, T, P)
    for s in {0, 1, T - 1, T, P * T - 1, P * T // 2, 2 ** 32 - 1, 2 ** 32, 2 ** 32 + 5}:
        if s >= P * T:
            continue
        assert host.h_slot(g.ctypes.data, s) == (s // T) * s_page + (s % T) * s_tok
    for s in (-1, -2, P * T, P * T + 7, -2 ** 63, 2 ** 63 - 1):
        assert host.h_slot(g.ctypes.data, s) == -1


def test_token_addresses_and_bad_pages(host):
    T, P = 17, 1000
    s_page, s_tok = 70000 * 80, 80          # offsets pass 32 bits at page 768
    g = geom(s_page, s_tok, T, P)
    table = np.array([999, 0, 1000, -1, 5, 2 ** 31 - 1, -2 ** 31], np.int32)
    wrong = ctypes.c_int()
    for t in range(table.size * T):
        off = host.h_token(g.ctypes.data, table.ctypes.data, t, ctypes.byref(wrong))
        page = int(table[t // T])
        if 0 <= page < P:
            assert (off, wrong.value) == (page * s_page + (t % T) * s_tok, 0)
        else:
            assert (off, wrong.value) == (-1, 1)


@pytest.mark.parametrize("T,s_page,P,fits", [(17, 70000 * 80, 60000, True), (16, 8 * 16 * 80, 2 ** 25 - 1, True),
                                             (16, 8 * 16 * 80, 2 ** 25, False), (1, 80, 2 ** 31 - 1, True)])
def test_vector_indexes(host, T, s_page, P, fits):
    """Counts of vectors stay below 2^32, or the host refuses the pool."""
    g, out = geom(s_page, 80, T, P), ctypes.c_uint32()
    for page in (0, 1, P // 2, P - 1):
        for t in (0, T - 1, 5 * T + T // 2):
            assert host.h_vector(g.ctypes.data, 80, page, t, ctypes.byref(out)) == fits
            if fits:
                assert out.value * 80 == page * s_page + (t % T) * 80


@pytest.mark.parametrize("group,rows", [(1, 8), (4, 8), (5, 8), (8, 8), (12, 16), (3, 16), (4, 128)])
@pytest.mark.parametrize("window", [0, 1, 7, 100])
def test_spans(host, group, rows, window):
    """lo and hi of a row tile against the tokens that its rows see, one by one."""
    for n in (0, 1, 2, 5, 40):
        for length in (0, 1, 4, 40, 41, 300):
            for rt in range(-(-max(n, 1) * group // rows) + 1):
                out = (ctypes.c_int * 6)()
                host.h_span((ctypes.c_int * 10)(3, 3 + n, length, 100, 60, 500, group, window, rt, rows), out)
                assert list(out[:3]) == [n, length, 3] and out[5] == 0
                seen = set()
                for row in range(rt * rows, min((rt + 1) * rows, n * group)):
                    pos = length - n + row // group
                    first = max(0, pos - window + 1) if window else 0
                    seen |= set(range(first, pos + 1))
                lo, hi = out[3], out[4]
                assert 0 <= lo <= hi <= length
                assert seen <= set(range(lo, hi))
                if seen:
                    assert (lo, hi) == (min(seen), max(seen) + 1)


@pytest.mark.parametrize("q0,q1,length,n,kept", [
    (-1, 4, 10, 0, 10), (5, 4, 10, 0, 10), (0, 101, 10, 0, 10), (0, 61, 10, 0, 10),
    (0, 4, -3, 4, 0), (0, 4, 501, 4, 500), (2 ** 31 - 1, -2 ** 31, 10, 0, 10),
    (-2 ** 31, 2 ** 31 - 1, 2 ** 31 - 1, 0, 500)])
def test_bad_lengths_are_brought_into_range(host, q0, q1, length, n, kept):
    out = (ctypes.c_int * 6)()
    host.h_span((ctypes.c_int * 10)(q0, q1, length, 100, 60, 500, 4, 0, 0, 8), out)
    assert out[5] == 1 and out[0] == n and out[1] == kept
    assert 0 <= out[3] <= out[4] <= 500 and 0 <= out[2] <= 100


def test_quotients_round_exactly(host):
    """Next to and on half-way points, against rational arithmetic."""
    r = np.random.default_rng(1)
    for _ in range(4000):
        s = np.uint32((r.integers(30, 250) << 23) | (r.integers(0, 1 << 19) << 4)).view(np.float32)
        k = int(r.integers(-15, 16))
        near = np.float32((k + 0.5) * float(s))
        for x in (near, np.nextafter(near, np.float32(np.inf)), np.nextafter(near, np.float32(-np.inf)),
                  np.float32(k * float(s)), np.float32(r.uniform(-15, 15) * float(s))):
            want = round(Fraction(float(x)) / Fraction(float(s)))     # ties to even
            assert host.h_round(x, s) == want, (x, s)


@pytest.mark.parametrize("kind", ["normal", "bf16", "tiny", "huge", "positive", "negative", "zeros", "one"])
def test_group_encoding(host, kind):
    r = np.random.default_rng(7)
    for _ in range(300):
        x = r.standard_normal(32).astype(np.float32)
        if kind == "bf16":
            x = (x.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
        x = {"tiny": x * np.float32(1e-31), "huge": np.clip(x, -1, 1) * np.float32(3e38),
             "positive": np.abs(x) + 5, "negative": -np.abs(x) - 5, "zeros": x * 0,
             "one": np.eye(1, 32, 9, dtype=np.float32)[0]}.get(kind, x).astype(np.float32)
        word, code = ctypes.c_uint32(), (ctypes.c_uint32 * 32)()
        host.h_encode(x.ctypes.data, ctypes.byref(word), code)
        raw = vec_ref.q4_encode(x)
        want_word = raw[16:20].view("<u4")[0]
        c, z, s = vec_ref.q4_parts(raw, 32)
        assert word.value == want_word
        assert list(code) == list(c.astype(int))
        if s[0] > 0:      # half a step, and what the step's own rounding (2^-20) and the clamp leave
            assert np.all(np.abs((c - z) * s - x) <= s * (0.5 + 16 * 2.0 ** -19) + np.abs(x) * 2.0 ** -18)


@pytest.mark.parametrize("fmt,dim,want", [(kvb.KV_CACHE_SAME, 128, 256), (kvb.KV_CACHE_SAME, 8, 16),
                                          (kvb.KV_CACHE_E4M3, 48, 48), (kvb.KV_CACHE_Q4, 128, 80),
                                          (kvb.KV_CACHE_Q4, 64, 48), (kvb.KV_CACHE_Q4, 96, 64),
                                          (kvb.KV_CACHE_Q4, 256, 160), (kvb.KV_CACHE_Q4, 32, 32)])
def test_head_bytes(fmt, dim, want):
    assert kvb.kv_cache_head_bytes(fmt, dim) == want


@pytest.mark.parametrize("fmt,dim,status", [
    (3, 128, kvb.KV_ERR_INVALID_ARG), (kvb.KV_CACHE_Q4, 80, kvb.KV_ERR_LAYOUT),
    (kvb.KV_CACHE_Q4, 0, kvb.KV_ERR_LAYOUT), (kvb.KV_CACHE_E4M3, 72, kvb.KV_ERR_LAYOUT),
    (kvb.KV_CACHE_SAME, 4, kvb.KV_ERR_LAYOUT), (kvb.KV_CACHE_SAME, 264, kvb.KV_ERR_LAYOUT)])
def test_head_bytes_refusals(fmt, dim, status):
    with pytest.raises(kvb.KvError) as e:
        kvb.kv_cache_head_bytes(fmt, dim)
    assert e.value.status == status


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=63), dict(rot_dim=258), dict(style=2), dict(scaling=5),
    dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")), dict(gain=-1.0),
    dict(gain=float("nan")), dict(scaling=kvb.KV_ROTARY_LINEAR, factor=0.5),
    dict(scaling=kvb.KV_ROTARY_LINEAR, factor=float("inf")),
    dict(scaling=kvb.KV_ROTARY_NTK, factor=2.0, rot_dim=2),
    dict(scaling=kvb.KV_ROTARY_YARN, factor=2.0, slow=1.0, fast=32.0),
    dict(scaling=kvb.KV_ROTARY_YARN, factor=2.0, slow=32.0, fast=1.0, original_len=4096),
    dict(scaling=kvb.KV_ROTARY_BANDS, factor=2.0, slow=0.0, fast=4.0, original_len=4096)])
def test_rotary_refusals(kw):
    with pytest.raises(kvb.KvError) as e:
        kvb.kv_rotary_create(**{"rot_dim": 64, **kw})
    assert e.value.status == kvb.KV_ERR_INVALID_ARG


def test_rotary_handles():
    r = kvb.kv_rotary_create(64)
    kvb.kv_rotary_close(r)
    with pytest.raises(kvb.KvError) as e:
        kvb.kv_rotary_close(r)
    assert e.value.status == kvb.KV_ERR_CLOSED
    with pytest.raises(kvb.KvError) as e:
        kvb.kv_rotate(r, kvb.make_rotate_args(kvb.kv_vecs(), kvb.kv_vecs(), 1, 1, 64, 0))
    assert e.value.status == kvb.KV_ERR_CLOSED


V16 = kvb.kv_vecs(1 << 20, 128, 64)


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=12), kvb.KV_ERR_INVALID_ARG), (dict(head_dim=264), kvb.KV_ERR_INVALID_ARG),
    (dict(head_dim=32), kvb.KV_ERR_INVALID_ARG),              # less than rot_dim
    (dict(dtype=2), kvb.KV_ERR_INVALID_ARG), (dict(x=kvb.kv_vecs(0, 128, 64)), kvb.KV_ERR_INVALID_ARG),
    (dict(x=kvb.kv_vecs((1 << 20) + 8, 128, 64)), kvb.KV_ERR_ALIGNMENT),
    (dict(x=kvb.kv_vecs(1 << 20, 100, 64)), kvb.KV_ERR_ALIGNMENT),
    (dict(out=kvb.kv_vecs(1 << 20, 128, -64)), kvb.KV_ERR_INVALID_ARG),
    (dict(out=kvb.kv_vecs(1 << 20, 256, 64)), kvb.KV_ERR_INVALID_ARG),   # x itself with other strides
    (dict(positions=None), kvb.KV_ERR_INVALID_ARG), (dict(rows_in=1 << 21), kvb.KV_ERR_INVALID_ARG),
    (dict(positions=None, rows_in=(1 << 21) + 4), kvb.KV_ERR_ALIGNMENT),
    (dict(positions=None, rows_in=1 << 21, rows_out=1 << 22), kvb.KV_ERR_INVALID_ARG),
    (dict(rows_out=(1 << 21) + 4), kvb.KV_ERR_ALIGNMENT),
    (dict(positions=(1 << 21) + 4), kvb.KV_ERR_ALIGNMENT)])
def test_rotate_refusals(kw, status):
    r = kvb.kv_rotary_create(64)
    try:
        d = dict(x=V16, out=V16, tokens=3, heads=2, head_dim=64, dtype=0, positions=1 << 21)
        with pytest.raises(kvb.KvError) as e:
            kvb.kv_rotate(r, kvb.make_rotate_args(**{**d, **kw}))
        assert e.value.status == status
        assert kvb.kv_last_error()
    finally:
        kvb.kv_rotary_close(r)


def test_rotate_of_nothing_and_unknown_flags():
    r = kvb.kv_rotary_create(64)
    try:
        kvb.kv_rotate(r, kvb.make_rotate_args(kvb.kv_vecs(), kvb.kv_vecs(), 0, 2, 64, 0))
        a = kvb.make_rotate_args(V16, V16, 3, 2, 64, 0, positions=1 << 21)
        a.flags = 2
        with pytest.raises(kvb.KvError) as e:
            kvb.kv_rotate(r, a)
        assert e.value.status == kvb.KV_ERR_INVALID_ARG
        for call in (lambda: kvb.library().kv_rotate(r, None, None), lambda: kvb.library().kv_rotate(None, a, None),
                     lambda: kvb.library().kv_rotary_create(None, None),
                     lambda: kvb.library().kv_append(None, None, None, None),
                     lambda: kvb.library().kv_fetch(None, None, None),
                     lambda: kvb.library().kv_attend(None, None, None),
                     lambda: kvb.library().kv_attend_workspace(None, None, None)):
            assert call() == kvb.KV_ERR_INVALID_ARG
    finally:
        kvb.kv_rotary_close(r)


@pytest.mark.parametrize("pool,status", [(None, kvb.KV_ERR_INVALID_ARG), (987654321, kvb.KV_ERR_CLOSED)])
def test_pool_calls_without_a_pool(pool, status):
    ap = kvb.make_append_args(V16, V16, tokens=1, head_dim=64, dtype=0, format=0, layer=0, slots=1 << 21)
    fe = kvb.make_fetch_args(V16, V16, tokens=1, head_dim=64, dtype=0, format=0, layer=0, slots=1 << 21)
    at = kvb.make_attend_args(V16, V16, q_start=1 << 21, lens=1 << 21, pages=1 << 21, pages_stride=1, requests=1,
                              tokens=1, max_q=1, max_len=1, q_heads=1, head_dim=64, dtype=0, layer=0, scale=1.0)
    for call in (lambda: kvb.kv_append(pool, None, ap), lambda: kvb.kv_fetch(pool, fe),
                 lambda: kvb.kv_attend(pool, at), lambda: kvb.kv_attend_workspace(pool, at)):
        with pytest.raises(kvb.KvError) as e:
            call()
        assert e.value.status == status


def test_block_sizes_match_the_header():
    """sizeof of every argument block, from the C compiler."""
    names = ["kv_vecs", "kv_rotary_desc", "kv_rotate_args", "kv_append_args", "kv_fetch_args", "kv_attend_args"]
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    src = '#include "kvb.h"\n#include <stdio.h>\nint main(void) {' + \
        "".join('printf("%%zu\\n", sizeof(%s));' % n for n in names) + "return 0;}"
    exe = os.path.join(kbuild.BUILD, "block_sizes")
    os.makedirs(kbuild.BUILD, exist_ok=True)
    subprocess.run([cc, "-std=c99", "-x", "c", "-I", kbuild.INCLUDE, "-o", exe, "-"], input=src.encode(), check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(getattr(kvb, n)) for n in names]
