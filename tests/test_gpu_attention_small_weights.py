"""attention in fp16 where most weights are far below the row's largest: the
mass that many weak keys have beside a strong one, and weak keys with large
values.

Weights go to the tensor core as fp16 relative to the row's reference weight,
which stands at 2^7: a weight is off by half a step (u of it), or below
2^-14 by at most 2^-25, which is 2^-32 of the reference weight.  The sum of
the weights is at least the reference weight, so a key adds at most
2^-32 |v| to the error of the result."""

import math

import pytest
import torch

import block_ref as R
import gpu_helpers as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16
FLOOR = {HF: 2.0 ** -32, BF: 0.0}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_quantized_smooth_b200 import build
    build.build()
    torch.cuda.init()


def check(got, q, k, v, rows, causal, scale, what=""):
    """The given rows of one sequence and head against float64, all with the
    tolerance of block_ref.attention_ref and the floor."""
    dtype, T = q.dtype, k.shape[0]
    qd, kd, vd = q[rows, 0].double(), k[:, 0].double(), v[:, 0].double()
    s = qd @ kd.T * scale
    size = qd.abs() @ kd.abs().T * scale
    if causal:
        keep = torch.arange(T, device=DEV) <= rows[:, None]
        s, size = s.masked_fill(~keep, -math.inf), size.masked_fill(~keep, 0.0)
        mass = keep.double() @ vd.abs()
    else:
        mass = vd.abs().sum(0).expand(len(rows), -1)
    w = torch.softmax(s, -1)
    o, spread = w @ vd, w @ vd.abs()
    u = R.half_step(dtype)
    exponent = 2.0 ** -17 * size.amax(-1, keepdim=True)
    tol = u * o.abs() + (u + 2 * exponent + 2.0 ** -13) * spread + FLOOR[dtype] * mass + R.tiny(dtype)
    R.assert_within(got[rows, 0], o, tol, what)
    return o


@pytest.mark.parametrize("dtype", [HF, BF])
@pytest.mark.parametrize("gap", [0, 8, 13, 15, 17, 20, 24, 25, 26, 28, 30])
def test_two_keys(gap, dtype):
    """Keys `gap` log2 units apart, zero at the strong one: the result is the
    weak one's weight times its value."""
    s = H.svdq()
    q, k, v = (torch.zeros(2, 1, 64, dtype=dtype, device=DEV) for _ in range(3))
    q[:, 0, 0] = 1.0
    for strong in (0, 1):
        k.zero_(), v.zero_()
        k[strong, 0, 0] = gap
        v[1 - strong] = 60000.0
        scale = math.log(2.0)
        for causal in (False, True):
            got = s.attention(q, k, v, causal=causal, scale=scale)
            s.check_device_error()
            check(got, q, k, v, torch.arange(2, device=DEV), causal, scale, f"gap {gap}")


@pytest.mark.parametrize("dtype", [HF, BF])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("T,D", [(300, 128), (5000, 128), (20000, 64), (40000, 64)])
def test_a_strong_key_beside_many_weak_ones(T, D, causal, dtype):
    """The first key some 16 to 27 log2 units over all others, nothing as its
    value: what is left is the weak keys' share."""
    s = H.svdq()
    g = torch.Generator(device=DEV).manual_seed(T)
    q = torch.randn(T, 1, D, generator=g, device=DEV) * 0.1
    k = torch.randn(T, 1, D, generator=g, device=DEV)
    v = torch.rand(T, 1, D, generator=g, device=DEV) * 2000 + 1000
    q[:, 0, 0] = 1.0 - 0.05 * (torch.arange(T, device=DEV) % 9)
    k[0], v[0], k[1:, 0, 0] = 0.0, 0.0, 0.0
    k[0, 0, 0] = 27.0
    q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    scale = math.log(2.0)
    got = s.attention(q, k, v, causal=causal, scale=scale)
    s.check_device_error()
    rows = torch.unique(torch.cat([torch.arange(40, device=DEV), torch.arange(T - 40, T, device=DEV),
                                   torch.randint(0, T, (100,), generator=g, device=DEV)]))
    check(got, q, k, v, rows, causal, scale, f"{T} keys")


@pytest.mark.parametrize("at", [0, 100, 2000, 3999])
def test_strong_key_anywhere(at):
    """The strong key in any tile: in front of it the reference is a weak
    key's, behind it its own; divided among the blocks as well."""
    s = H.svdq()
    for T in (4000, 2000):
        if at >= T:
            continue
        g = torch.Generator(device=DEV).manual_seed(at)
        q = (torch.randn(T, 1, 128, generator=g, device=DEV) * 0.1).to(HF)
        k = torch.randn(T, 1, 128, generator=g, device=DEV).to(HF)
        v = (torch.rand(T, 1, 128, generator=g, device=DEV) * 2000 + 1000).to(HF)
        q[:, 0, 0], k[:, 0, 0] = 1.0, 0.0
        k[at], v[at] = 0.0, 0.0
        k[at, 0, 0] = 25.0
        for causal in (False, True):
            got = s.attention(q, k, v, causal=causal, scale=math.log(2.0))
            s.check_device_error()
            check(got, q, k, v, torch.arange(0, T, 7, device=DEV), causal, math.log(2.0), f"at {at} of {T}")


def test_the_largest_weights_stay_finite():
    """Scores that keep growing by just under the rescale step: weights of 2^8
    times the reference, times the largest values."""
    s = H.svdq()
    T, D = 1024, 64
    q, k, v = (torch.zeros(T, 1, D, dtype=HF, device=DEV) for _ in range(3))
    q[:, 0, 0] = 1.0
    k[:, 0, 0] = (torch.arange(T, device=DEV) // 128).to(HF) * 7.9375
    v[:] = 60000.0
    scale = math.log(2.0)
    for causal in (False, True):
        got = s.attention(q, k, v, causal=causal, scale=scale)
        s.check_device_error()
        check(got, q, k, v, torch.arange(0, T, 5, device=DEV), causal, scale)
