"""What the kernels for many query rows look over before they scale a request's steps, compiled
for the host: every token that a row sees has to be in it."""
import ctypes
import shutil
import subprocess

import pytest

from hierarchical_kv_cache_backup_gb300 import build as kbuild

HARNESS = r"""
#include "kvb_vec.h"
using namespace kvb;
extern "C" int h_seen(int n, int len, int max_q, int max_len, int group, int window, unsigned *parts) {
    bool bad = false;
    const Span s = row_span(0, n, len, n, max_q, max_len, group, window, 0, max_q * group, &bad);
    *parts = step_parts_of((unsigned)max_len, (unsigned)window, (unsigned)max_q);
    return bad ? -1 : s.hi - s.lo;
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("spans")
    (d / "h.cpp").write_text(HARNESS)
    subprocess.run([cc, "-O1", "-std=c++17", "-shared", "-fPIC", "-I", kbuild.CSRC, str(d / "h.cpp"), "-o", str(d / "h.so")],
                   check=True)
    return ctypes.CDLL(str(d / "h.so"))


@pytest.mark.parametrize("window", [0, 1, 256, 700, 1024, 4096, 2 ** 30])
@pytest.mark.parametrize("max_q,max_len", [(1, 1), (700, 1400), (1024, 1025), (2000, 8192), (4096, 4096), (8192, 16384),
                                           (65535, 2 ** 30), (8, 0)])
def test_step_parts_cover_what_all_rows_see(host, window, max_q, max_len):
    parts, widest = ctypes.c_uint(), 0
    for n in {1, max_q // 2, max_q}:
        for length in {0, min(n, max_len), max_len // 2, max_len}:
            seen = host.h_seen(n, length, max_q, max_len, 1 if max_q > 10000 else 4, window, ctypes.byref(parts))
            assert 0 <= seen <= 1024 * parts.value, (n, length)
            widest = max(widest, seen)
    assert parts.value == max(1, -(-widest // 1024))       # and not more than the fullest request needs
