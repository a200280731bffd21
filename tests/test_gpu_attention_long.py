"""attention over a very long sequence: the tensor core's fp32 sums.

A product adds 16 keys to O and cuts the sum off at fp32's last place (it does
not round): less than 2^-23 of O a step, all in one direction, n / 16 steps."""

import pytest
import torch

import block_ref as R
import gpu_helpers as H

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_quantized_smooth_b200 import build
    build.build()
    torch.cuda.init()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T", [65536, 262144])
def test_positive_values(T, dtype):
    """Values of one sign, so that nothing cancels."""
    s = H.svdq()
    g = torch.Generator(device=DEV).manual_seed(T)
    q, k = (torch.randn(T, 1, 64, generator=g, device=DEV).to(dtype) for _ in range(2))
    v = (torch.rand(T, 1, 64, generator=g, device=DEV) + 0.5).to(dtype)
    got = s.attention(q, k, v)
    s.check_device_error()
    rows = torch.randint(0, T, (64,), generator=g, device=DEV)
    qd, kd, vd = q[rows, 0].double(), k[:, 0].double(), v[:, 0].double()
    want = torch.softmax(qd @ kd.T / 8, -1) @ vd
    size = (qd.abs() @ kd.abs().T / 8).amax(-1, keepdim=True)
    u = R.half_step(dtype)
    R.assert_within(got[rows, 0], want, (2 * u + 2.0 ** -16 * size + 2.0 ** -13 + T / 16 * 2.0 ** -23) * want)
