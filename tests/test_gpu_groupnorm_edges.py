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
