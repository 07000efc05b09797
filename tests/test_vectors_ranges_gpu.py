"""kv_attend where a window's prompt chunk spans more tokens than one tile of queries sees, and
other ranges of steps and values."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import vec_check  # noqa: E402
import vec_ref  # noqa: E402
from test_vectors_gpu import Batch  # noqa: E402


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
