"""Long sums of the norm: rows up to the limit of 2^24 elements, and the weight gradient over many rows."""
import numpy as np
import pytest
import torch

from dynamic_short_convolution_amd import dynconv_norm_bwd, dynconv_norm_fwd
from oracle import norm_bwd, norm_fwd
from tests.parity import to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [2**24, 2**24 - 3, 1_000_003])
def test_longest_rows(D, dtype):
    """Elements near one another, as in a row whose mean is far from zero: sums of 2^24 squares and of
    dn n. A lane sums its elements in 64 bits, the sum is rounded to 32 (2^-24) and goes through
    eight additions of sums of one sign (2^-24 each), the product with 1 / D (two roundings), eps, root,
    division: 15 roundings, of the sum half count: 2^-24 * 10. n, y and dx add four each: 14 * 2^-24,
    of dx relative to dn, which dx = dn - n mean(dn n) takes the most of away. sigmoid adds a
    few steps of 2^-23 from its exponential and reciprocal: in all 32 * 2^-24."""
    tol = 32 * 2.0**-24 + (0 if dtype == torch.float32 else 2.0**-8)
    gen = torch.Generator().manual_seed(D)
    x = (1.1 + 0.01 * torch.rand(1, D, generator=gen)).to(dtype)
    w, z = (0.9 + 0.1 * torch.rand(D, generator=gen)).to(dtype), (1.0 + torch.rand(1, D, generator=gen)).to(dtype)
    dy = (0.5 + torch.rand(1, D, generator=gen)).to(dtype)
    x64, w64, z64, dy64 = (to64(t) for t in (x, w, z, dy))
    x, w, z, dy = (t.cuda() for t in (x, w, z, dy))
    y = dynconv_norm_fwd(x, w, gate=z)
    ref = norm_fwd(x64, w64, z64)
    assert np.max(np.abs(to64(y) / ref - 1)) <= tol
    dx, _, dw, dz = dynconv_norm_bwd(x, w, dy, gate=z)
    rx, rw, rz = norm_bwd(x64, w64, z64, dy64)
    dn = dy64 * w64 * z64 / (1 + np.exp(-z64)) / np.sqrt(np.mean(x64 * x64) + 1e-6)
    assert np.max(np.abs(to64(dx) - rx) / (np.abs(dn) + np.max(np.abs(dn)))) <= tol
    assert np.max(np.abs(to64(dw) / rw - 1)) <= 32 * 2.0**-24  # one row: dy silu(z) n, float32 in both types
    assert np.max(np.abs(to64(dz) / rz - 1)) <= tol


def test_weight_gradient_of_many_rows():
    """2^27 equal rows of one element: a float32 sum of equal terms can be off by half a step of 2^-24 at
    each addition, all the same way: for n terms by n / 2 * 2^-24 of it. A lane adds at most 512
    (256 * 2^-24), its workgroup 16 lanes (16), the rest is in 64 bits; a term has at most 16
    roundings."""
    rows = 2**27
    x = torch.ones(rows, 1, dtype=torch.bfloat16, device="cuda")
    dy = torch.full((rows, 1), 0.8984375, dtype=torch.bfloat16, device="cuda")
    dw = dynconv_norm_bwd(x, torch.ones(1, dtype=torch.bfloat16, device="cuda"), dy, eps=0.1)[2]
    assert abs(float(dw) / (rows * 0.8984375 / 1.1**0.5) - 1) <= (256 + 16 + 16) * 2.0**-24
