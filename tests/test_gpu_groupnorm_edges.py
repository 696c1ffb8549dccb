"""GPU edges of the group norm: column sums of long sequences, statistics of sequences without tokens, groups without
deviation. Tolerances as in tests/test_gpu_groupnorm.py.
"""
import numpy as np
import pytest
import torch

import dynamic_short_convolution_amd as dc
from dynamic_short_convolution_amd import _lib
from tests.parity import to64
from tests.test_gpu_groupnorm import TD, U, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    yield
    torch.cuda.synchronize()


def test_column_sums_of_many_long_sequences():
    """1024 workgroups' worth of sequences: a lane's float32 sums still end after 512 tokens. Terms that a sum of
    2048 and more rounds the same way every time: 4096 of them in one sum would be off by 1000 u of it, more than the
    48 + 512 u that sums of 512 are good for."""
    B, T, C = 1024, 4096, 256
    c = 1.0 + 3 * 2.0**-13
    x = rand(1, 1, T, C).expand(B, T, C)
    dy = torch.full((1, 1, C), c, device="cuda").expand(B, T, C)
    dbias = dc.dynconv_groupnorm_bwd(x, C, dy, weight=torch.ones(C, device="cuda"), bias=torch.zeros(C, device="cuda"), over="sequence")[2]
    assert (np.abs(to64(dbias) - B * T * c) <= (48 + 512) * U * B * T * c).all()


def test_statistics_without_tokens_from_the_entry_point():
    """T of 0: mean 0 and factor 0 of every sequence and group."""
    x = torch.zeros(1, dtype=torch.bfloat16, device="cuda")
    for B, C, groups in ((3, 64, 4), (2, 0, 5)):
        stats = torch.full((B, groups, 2), float("nan"), device="cuda")
        s = _lib.strides((64, 64, 1))
        st = _lib.load().dynconv_groupnorm_fwd(x.data_ptr(), s, None, None, None, None, None, x.data_ptr(), s, stats.data_ptr(), B, 0, C, groups,
                                               1, 0, 1e-5, 1, None, 0, torch.cuda.current_stream().cuda_stream)
        assert st == 0 and float(stats.abs().max()) == 0.0


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("width", [3, 57, 64, 100, 515, 1100, 2050, 4100, 9000])
@pytest.mark.parametrize("over", ["token", "sequence"])
def test_groups_without_deviation(width, over, dtype):
    """n is (x - mean) / sqrt(eps): a mean off by one rounding of 1000 makes it 0.02. The first mean may be off by 48 u of
    1000, the mean of the deviations from it by 48 u of that. The variance over 64-bit sums is off by some 2^-53 of
    1000^2, eight of which are (1000^2 / eps) 2^-50 / 2 of its root."""
    td = TD[dtype]
    x = torch.full((2, 3, 2 * width), 1000.0, dtype=td, device="cuda")
    if dtype == "f32":
        x += 0.1
    dy = rand(2, 2, 3, 2 * width, dtype=td)
    allowed = 50 * U * (50 * U * 1000.1) / np.sqrt(1e-5)
    y = dc.dynconv_groupnorm_fwd(x, 2, over=over)
    assert float(y.abs().max()) <= allowed
    # dx is then (dy - mean(dy)) / sqrt(eps)
    dx = to64(dc.dynconv_groupnorm_bwd(x, 2, dy, over=over)[0])
    d = to64(dy).reshape(2, 3, 2, width)
    m = d.mean(-1 if over == "token" else (1, 3), keepdims=True)
    ref = ((d - m) / np.sqrt(1e-5)).reshape(dx.shape)
    size = np.abs(d).max() / np.sqrt(1e-5)
    half = {"f32": U, "bf16": 2.0**-8, "f16": 2.0**-11}[dtype]
    assert (np.abs(dx - ref) <= (200 * U + 1000.1**2 / 1e-5 * 2.0**-51) * size + 1.01 * half * np.abs(ref)).all()


@pytest.mark.parametrize("width", [57, 64, 515, 2050])
def test_squares_past_float32(width):
    """Per token the variance of such values is infinite in float32: n is 0, not NaN, whatever the mean is off by."""
    x = rand(3, 2, 3, 2 * width) * 1e33 + 1e33
    w, b = rand(4, 2 * width), rand(5, 2 * width)
    assert torch.equal(dc.dynconv_groupnorm_fwd(x, 2, w, b), b.expand(2, 3, 2 * width))
    dx, dw, db, _ = dc.dynconv_groupnorm_bwd(x, 2, torch.ones_like(x), w, b)
    assert float(dx.abs().max()) == 0.0 == float(dw.abs().max()) and bool((db == 6.0).all())
