"""attention with its key tiles divided among the SMs, over several sequences:
long ones beside short and empty ones, offsets that fall or leave the tensors,
two calls at once, a replayed graph whose offsets change.  Every case asserts
that the call is divided."""

import pytest
import torch

import block_ref as R
import gpu_helpers as H
from test_block_args import items as walked
from test_divided_walk import DIVIDED
from test_gpu_attention import check, cu_of, make

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_quantized_smooth_b200 import build
    build.build()
    torch.cuda.init()


def is_divided(T, S, Hq, D, causal):
    return H.svdq()._lib.svdq_attention_workspace_bytes(T, S, Hq, D, int(causal)) > 0


@pytest.mark.parametrize("lens,Hq,causal", DIVIDED, ids=range(len(DIVIDED)))
def test_several_sequences(lens, Hq, causal):
    cu = cu_of(lens)
    for D, dtype in ((128, BF), (72, HF)):
        assert is_divided(cu[-1], len(lens), Hq, D, causal)
        check(*make(cu[-1], Hq, 1, D, dtype, seed=Hq), cu, causal, rel=False)


@pytest.mark.parametrize("causal", [False, True])
def test_rows_around_the_sequences(causal):
    """NaN and infinities in front of, between and behind them reach nothing;
    the output rows there stay as they were."""
    T, D = 12000, 128
    cu = cu_of([5500, 3, 6000], 101)
    assert is_divided(T, 3, 1, D, causal)
    q, k, v = make(T, 1, 1, D, seed=1)
    for t, bad in ((q, "nan"), (k, "nan"), (v, "inf")):
        t[:101] = float(bad)
        t[cu[-1]:] = float(bad)
    out = torch.full((T, 1, D), 3.0, dtype=BF, device=DEV)
    check(q, k, v, cu, causal, out=out, rel=False)
    assert (out[:101] == 3).all() and (out[cu[-1]:] == 3).all()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("cu", [[-5, 4000, 2 ** 31 - 1], [6000, 3000, 9001], [-2 ** 31, -1, 8000], [9001, 9500, 20000],
                                [0, 9000, 100], [50, 50, 50], [8999, 9000, 9001]])
def test_offsets_that_fall_or_leave_the_tensors(cu, causal):
    """The same sequences as the whole items' walk takes them for, and nothing
    outside the output."""
    T, D = 9001, 64
    assert is_divided(T, 2, 1, D, causal)
    q, k, v = make(T, 1, 1, D, seed=2)
    wide = torch.full((3 * T, 1, D), 7.0, dtype=BF, device=DEV)
    got = H.svdq().attention(q, k, v, torch.tensor(cu, dtype=torch.int32, device=DEV), causal, out=wide[T:2 * T])
    H.svdq().check_device_error()
    assert (wide[:T] == 7).all() and (wide[2 * T:] == 7).all()
    left = torch.ones(T, dtype=torch.bool, device=DEV)
    for begin, n in sorted({(b, n) for b, n, _, _ in walked(cu, T, 1, causal)}):
        left[begin:begin + n] = False
        ref, tol = R.attention_ref(q[begin:begin + n], k[begin:begin + n], v[begin:begin + n], None, causal, D ** -0.5)
        R.assert_within(got[begin:begin + n], ref, tol)
    assert (got[left] == 7).all()


@pytest.mark.parametrize("causal", [False, True])
def test_calls_at_once_and_graphs(causal):
    """Bit for bit: again, two divided calls at once on two streams, captured
    and replayed with other offsets in the same tensor."""
    s = H.svdq()
    T = 9001
    q, k, v = make(T, 1, 1, 128, seed=3)
    a_cu, b_cu, c_cu = (torch.tensor(c, dtype=torch.int32, device=DEV)
                        for c in ([0, 6000, 9001], [10, 10, 8990], [0, 1, 4500]))
    assert is_divided(T, 2, 1, 128, causal)

    def fresh(cu):
        return s.attention(q, k, v, cu, causal, out=torch.zeros_like(q))

    want = {id(c): fresh(c) for c in (a_cu, b_cu, c_cu)}
    st = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got, outs = [], [torch.zeros_like(q) for _ in st]
        for x, c, o in zip(st, (a_cu, b_cu), outs):
            x.wait_stream(torch.cuda.current_stream())
            got.append(s.attention(q, k, v, c, causal, out=o, stream=x))
        for x in st:
            torch.cuda.current_stream().wait_stream(x)
        assert torch.equal(got[0], want[id(a_cu)]) and torch.equal(got[1], want[id(b_cu)])
    moving, out = a_cu.clone(), torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.attention(q, k, v, moving, causal, out=out)
    for c in (a_cu, b_cu, c_cu, a_cu):
        moving.copy_(c)
        out.zero_()
        graph.replay()
        assert torch.equal(out, want[id(c)])
    s.check_device_error()
