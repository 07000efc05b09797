"""The example that runs the operators together, against a plain stack in 32 bits."""
import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import vec_ref  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("four_bit_pages", os.path.join(ROOT, "examples", "four_bit_pages.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("prompt,decode", [(200, 12), (17, 3), (1, 2)])
def test_restored_pages_decode_the_same(example, prompt, decode):
    r = example.main(prompt, decode)
    assert r["status"] == 0
    assert torch.equal(r["from_home"], r["from_restored"])
    assert torch.isfinite(r["from_home"].float()).all()
    assert r["bytes_in_16_bits"] / r["bytes_moved"] == 3.2


def test_layer_0_holds_the_prompt(example):
    """Keys and values of the first layer, from a projection in float32: half a step of the format
    (the group's range over 30), and bf16 roundings of the projection (2^-8), of the value
    held (2^-8) and of the rotation's inputs."""
    r = example.main(40, 1)
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    m = example
    n = m.Q_HEADS + 2 * m.HEADS
    w = torch.randn(m.WIDTH, n * m.DIM, generator=g, device="cuda").mul(m.WIDTH ** -0.5).bfloat16()
    g.manual_seed(1)
    pages = 3 * 3 + 1
    torch.randperm(pages, generator=g, device="cuda")
    x = torch.randn(41, m.WIDTH, generator=g, device="cuda").bfloat16()[:40]
    qkv = (x.float() @ w.float()).view(40, n, m.DIM).cpu().numpy().astype(np.float64)
    f, gain = vec_ref.frequencies(m.DIM, scaling="yarn", factor=4.0, original_len=4096, slow=1.0, fast=32.0)
    k = vec_ref.turn(qkv[:, m.Q_HEADS:m.Q_HEADS + m.HEADS], vec_ref.rows_of(f, gain, np.arange(40)), "half")
    v = qkv[:, m.Q_HEADS + m.HEADS:]
    for want, got in ((k, r["keys"]), (v, r["values"])):
        grp = want.reshape(40, m.HEADS, m.DIM // 32, 32)
        span = np.maximum(grp.max(-1), 0) - np.minimum(grp.min(-1), 0)
        size = np.abs(grp).max(-1)
        tol = np.repeat(span / 30 + size * (3 * 2.0 ** -8) + 2.0 ** -8 * np.abs(qkv).max(), 32, -1).reshape(want.shape)
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)
