"""A padded batch through a whole block: rows in front of the first and behind
the last sequence, and the uninitialized memory that stands for them between
the steps, do not show in the sequences' rows."""

import pytest
import torch

import gpu_helpers as H
from test_gpu_dit_block import HEADS, HIDDEN, make_block

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_quantized_smooth_b200 import build
    build.build()
    torch.cuda.init()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("T,cu", [(300, [0, 200]), (300, [30, 100, 230]), (40, [5, 30]), (600, [0, 10, 500])])
def test_padded(T, cu, causal):
    s = H.svdq()
    w, _, g = make_block(40)
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    x = torch.randn(T, HIDDEN, generator=g, device=DEV).to(BF)
    mod = (torch.randn(len(cu) - 1, 4 * HIDDEN, generator=g, device=DEV) * 0.5).to(BF).chunk(4, 1)
    pos = torch.randint(0, 64, (T, 3), generator=g, device=DEV, dtype=torch.int32)
    plan = s.RopePlan((32, 48, 48), 256.0, HIDDEN // HEADS)
    inside = slice(cu[0], cu[-1])
    want = s.dit_block(x, w, mod, pos, plan, cut, causal)[inside]
    assert torch.isfinite(want).all()
    for bad in (float("nan"), float("inf"), 1e30):
        x2 = x.clone()
        x2[:cu[0]] = bad
        x2[cu[-1]:] = bad
        junk = [torch.full((T, n * HIDDEN), bad, device=DEV, dtype=BF) for n in (1, 1, 2, 3, 3)]
        del junk                     # what the allocator hands out next
        got = s.dit_block(x2, w, mod, pos, plan, cut, causal)
        s.check_device_error()
        assert torch.equal(got[inside], want)
