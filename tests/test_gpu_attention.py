"""attention against float64: lengths from one row to long ones, packed
sequences, causal and full, grouped heads, head widths, strides, rows in no
sequence, non-finite values where a row does not attend."""

import pytest
import torch

import block_ref as R
import gpu_helpers as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_quantized_smooth_b200 import build
    build.build()
    torch.cuda.init()


def cu_of(lens, first=0):
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def make(T, Hq, Hk, D, dtype=BF, seed=0, by=1.4, views=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    out = []
    for i, n in enumerate((Hq, Hk, Hk)):
        t = torch.randn(T, n, D, generator=g, device=DEV) * (by if i < 2 else 1.0)
        out.append(t.to(dtype) if views is None else views[i].copy_(t))
    return out


def check(q, k, v, cu, causal, scale=None, out=None, rel=True, what=""):
    s = H.svdq()
    D = q.shape[-1]
    cut = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    got = s.attention(q, k, v, cut, causal, scale, out)
    s.check_device_error()
    ref, tol = R.attention_ref(q, k, v, cu, causal, scale or D ** -0.5)
    rows = torch.zeros(q.shape[0], dtype=torch.bool, device=DEV)
    for b, e in R.spans(q.shape[0], cu):
        rows[b:e] = True
    R.assert_within(got[rows], ref[rows], tol[rows], what)
    if rel and rows.any():
        err = (got[rows].double() - ref[rows]).norm() / ref[rows].norm()
        assert err <= R.attention_rel(q.dtype), f"{what}: relative error {err:.3e}"
    return got


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 33, 64, 100, 127, 128, 129, 200, 255, 256, 257, 383, 384,
                               385, 511, 513, 640, 1000])
def test_lengths(L, causal):
    check(*make(L, 2, 1, 128, seed=L), None, causal, rel=L >= 64)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [8, 16, 24, 40, 56, 64, 72, 80, 96, 104, 120, 128])
def test_head_widths(D, causal, dtype):
    check(*make(300, 2, 2, D, dtype, seed=D), cu_of([171, 129]), causal)


LENS = [[1], [0, 1, 0], [1, 1, 1, 1], [300, 0, 17, 128, 1], [128, 128], [256, 256, 256], [257, 255, 1, 383],
        [3] * 70, [0] * 40 + [5] + [0] * 30 + [130], [700, 40]]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens", LENS, ids=range(len(LENS)))
def test_packed_sequences(lens, causal):
    cu = cu_of(lens)
    check(*make(cu[-1], 3, 1, 128, seed=len(lens)), cu, causal, rel=False)
    check(*make(cu[-1], 2, 2, 64, HF, seed=len(lens)), cu, causal, rel=False)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (8, 8), (8, 2), (6, 2), (7, 1), (160, 5)])
def test_grouped_heads(Hq, Hk):
    check(*make(140, Hq, Hk, 128, seed=Hq), cu_of([100, 40]), True, rel=False)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D,dtype", [(128, BF), (64, HF)])
def test_long(causal, D, dtype):
    check(*make(4500, 2, 1, D, dtype, seed=3), cu_of([4352, 148]), causal)


def test_more_items_than_blocks():
    """Every block takes several items of different lengths in turn."""
    lens = [(37 * i * i) % 700 for i in range(40)]
    for causal in (False, True):
        check(*make(sum(lens), 8, 4, 128, seed=4), cu_of(lens), causal)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_growing_maxima(causal, dtype):
    """Scores that rise by more than the rescale step from tile to tile, fall
    again, and rows of very different sizes."""
    T = 900
    q, k, v = make(T, 2, 2, 128, dtype, seed=5, by=1.0)
    ramp = torch.linspace(0, 12, T, device=DEV)
    k += ramp[:, None, None].to(dtype) * torch.sign(q[0:1])
    q[::3] *= 6
    q[1::3] *= -3
    check(q, k, v, cu_of([T]), causal, rel=False)
    check(q, k.flip(0).contiguous(), v, cu_of([T]), causal, rel=False)


def test_equal_scores_average_the_values():
    """q = 0: every key weighs the same; exact in the weights."""
    q, k, v = make(1000, 1, 1, 128, seed=6)
    q.zero_()
    check(q, k, v, None, False, rel=False)
    check(q, k, v, None, True, rel=False)


def test_scales():
    q, k, v = make(260, 2, 2, 128, seed=7)
    for scale in (1e-6, 0.01, 1.0, 5.0):
        check(q, k, v, None, True, scale=scale, rel=False)


def test_a_very_low_score_is_not_a_mask():
    """Rows whose scores are all near the type's lowest: the softmax of their
    differences (k is one-hot, so the scores are exact)."""
    T = 200
    q, k, v = make(T, 1, 1, 64, seed=8)
    q.zero_(), k.zero_()
    q[:, 0, 0] = -3.0e38
    k[:, 0, 0] = 1.0
    check(q, k, v, None, False, scale=0.125, rel=False)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D,dtype", [(128, BF), (80, HF), (64, BF)])
def test_rows_in_no_sequence(causal, D, dtype):
    """NaN and infinities around and between the sequences reach nothing, and
    the output rows there stay as they were."""
    for lens, first, behind in (([100, 30], 9, 70), ([1], 0, 300), ([129, 0, 255], 3, 1), ([16, 112], 40, 200)):
        cu = cu_of(lens, first)
        T = cu[-1] + behind
        q, k, v = make(T, 2, 1, D, dtype, seed=9)
        for t, bad in ((q, "nan"), (k, "nan"), (v, "inf")):
            t[:first] = float(bad)
            t[cu[-1]:] = float(bad)
        v[cu[-1]:, :, ::2] = float("nan")
        out = torch.full((T, 2, D), 3.0, dtype=dtype, device=DEV)
        check(q, k, v, cu, causal, out=out, rel=False)
        assert (out[:first] == 3).all() and (out[cu[-1]:] == 3).all()


@pytest.mark.parametrize("causal", [False, True])
def test_a_sequence_of_nan_stays_alone(causal):
    cu = cu_of([130, 50, 77])
    q, k, v = make(257, 2, 2, 128, seed=10)
    for t in (q, k, v):
        t[130:180] = float("nan")
    check(q, k, v, cu, causal, rel=False)


@pytest.mark.parametrize("bad", ["inf", "-inf", "nan"])
@pytest.mark.parametrize("at", [0, 1, 100, 127, 128, 200, 255, 256, 300, 511, 700])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_causal_rows_in_front_of_a_bad_key_or_value(at, bad, dtype):
    """A non-finite key or value at one row leaves every row before it as it
    is; from that row on a value gives what the sum gives."""
    T = 800
    q, k, v = make(T, 2, 1, 128, dtype, seed=11, by=0.5)
    clean = H.svdq().attention(q, k, v, causal=True)
    v2 = v.clone()
    v2[at, 0, 5] = float(bad)
    v2[at, 0, 127] = float(bad)
    got = check(q, k, v2, None, True, rel=False)
    assert torch.equal(got[:at], clean[:at])
    rest = [c for c in range(128) if c not in (5, 127)]
    assert torch.equal(got[..., rest], clean[..., rest])
    k2 = k.clone()
    k2[at, 0, 9] = float("nan")
    got = H.svdq().attention(q, k2, v, causal=True)
    assert torch.equal(got[:at], clean[:at]) and torch.isnan(got[at:]).all()


def test_causal_opposite_infinities_meet():
    T = 300
    q, k, v = make(T, 1, 1, 64, seed=12, by=0.5)
    v[260, 0, 3], v[270, 0, 3], v[280, 0, 4] = float("inf"), float("-inf"), float("nan")
    check(q, k, v, None, True, rel=False)


def test_an_infinite_query_is_nan_in_its_row_alone():
    q, k, v = make(300, 2, 2, 128, seed=13)
    clean = H.svdq().attention(q, k, v)
    q[77, 1, 4] = float("inf")
    got = H.svdq().attention(q, k, v)
    assert torch.isnan(got[77, 1]).all()
    got[77, 1] = clean[77, 1]
    assert torch.equal(got, clean)


def test_views_of_one_buffer():
    """q, k, v and out side by side in the rows of one buffer, and with the
    heads in front."""
    T, Hq, Hk, D = 333, 4, 2, 72
    wide = torch.zeros(T, (2 * Hq + 2 * Hk) * D + 8, dtype=BF, device=DEV)
    cols = [0, Hq * D, (Hq + Hk) * D, (Hq + 2 * Hk) * D, (2 * Hq + 2 * Hk) * D]
    views = [wide[:, a:b].view(T, -1, D) for a, b in zip(cols, cols[1:])]
    check(*make(T, Hq, Hk, D, views=views), cu_of([300, 33]), True, out=views[3])
    assert (wide[:, cols[4]:] == 0).all()
    heads = [torch.empty(h, T, D, dtype=BF, device=DEV).transpose(0, 1) for h in (Hq, Hk, Hk, Hq)]
    check(*make(T, Hq, Hk, D, views=heads), cu_of([300, 33]), False, out=heads[3])


def test_offsets_over_32_bits():
    T, D, st = 300, 64, 1 << 23
    wide = torch.empty((T - 1) * st + 8 * D, dtype=BF, device=DEV)
    views = [wide.as_strided((T, h, D), (st, D, 1), at * D) for h, at in ((2, 0), (1, 2), (1, 3), (2, 4))]
    check(*make(T, 2, 1, D, views=views[:3]), cu_of([290, 10]), True, out=views[3])


def test_many_rows():
    """70 001 rows, rows sampled."""
    T = 70001
    q, k, v = make(T, 1, 1, 64, seed=14)
    got = H.svdq().attention(q, k, v, causal=True)
    H.svdq().check_device_error()
    for i in (0, 1, 127, 128, 33333, 65535, 65536, 69999, 70000):
        ref, tol = R.attention_ref(q[i:i + 1], k[i:i + 1], v[i:i + 1], None, False, 0.125)   # shapes
        w = torch.softmax(k[:i + 1, 0].double() @ q[i, 0].double() * 0.125, 0)
        o = w @ v[:i + 1, 0].double()
        spread = w @ v[:i + 1, 0].double().abs()
        u = R.half_step(BF)
        assert ((got[i, 0].double() - o).abs() <= u * o.abs() + (u + 2.0 ** -12) * spread).all(), i


def test_bad_offsets_stay_inside():
    T = 300
    q, k, v = make(T, 2, 1, 64, seed=15)
    wide = torch.full((3 * T, 2, 64), 7.0, dtype=BF, device=DEV)
    for cu in ([-5, 100, 2 ** 31 - 1], [200, 50, 300], [-2 ** 31, -1, 1000], [301, 400, 500], [0, 300] * 40):
        for causal in (False, True):
            H.svdq().attention(q, k, v, torch.tensor(cu, dtype=torch.int32, device=DEV), causal, out=wide[T:2 * T])
            H.svdq().check_device_error()
            assert (wide[:T] == 7).all() and (wide[2 * T:] == 7).all()


def test_repeats_on_streams_and_in_graphs():
    """Bit for bit: again, two calls at once on two streams, captured and
    replayed with other offsets in the same tensor."""
    s = H.svdq()
    q, k, v = make(2000, 8, 2, 128, seed=16)
    cu = torch.tensor(cu_of([700, 1300]), dtype=torch.int32, device=DEV)
    other = torch.tensor(cu_of([1500, 500]), dtype=torch.int32, device=DEV)
    a, b = s.attention(q, k, v, cu, True), s.attention(q, k, v, other, True)
    st = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for x, c in zip(st, (cu, other)):
            x.wait_stream(torch.cuda.current_stream())
            got.append(s.attention(q, k, v, c, True, stream=x))
        for x in st:
            torch.cuda.current_stream().wait_stream(x)
        assert torch.equal(got[0], a) and torch.equal(got[1], b)
    moving = cu.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g1 = s.attention(q, k, v, moving, True)
        g2 = s.attention(q, k, g1[:, :2], moving, True)
    want2 = [s.attention(q, k, w[:, :2], c, True) for w, c in ((a, cu), (b, other))]
    for c, w, w2 in ((cu, a, want2[0]), (other, b, want2[1]), (cu, a, want2[0])):
        moving.copy_(c)
        graph.replay()
        assert torch.equal(g1, w) and torch.equal(g2, w2)


def test_binding_refuses():
    s = H.svdq()
    q, k, v = make(8, 4, 2, 64)
    cu = torch.tensor([0, 8], dtype=torch.int32, device=DEV)
    for a in ((q, k.half(), v), (q, k, v[:, :1]), (q, k[:4], v), (q, k, v, cu.long()), (q, k, v, cu.cpu()),
              (q[..., :32], k, v), (q.float(), k.float(), v.float()), (q, k[:, 0], v), (q[0], k, v)):
        with pytest.raises(ValueError):
            s.attention(*a)
    with pytest.raises(s.SvdqError):                      # 3 heads on 2
        s.attention(q[:, :3], k, v)
    for out in (q, k.expand(8, 2, 64).repeat(1, 2, 1)[:, :, :32]):
        with pytest.raises((s.SvdqError, ValueError)):
            s.attention(q, k, v, out=out)
    for scale in (0.0, -1.0, float("nan")):
        with pytest.raises(s.SvdqError):
            s.attention(q, k, v, scale=scale)
    with pytest.raises(s.SvdqError):
        s.attention(q, k[:, :1].expand(8, 2, 64), v)      # one head standing for two
    assert s.attention(q[:0], k[:0], v[:0]).shape == (0, 4, 64)


def test_slots_that_sit_items_out():
    """Causal items of which one half of the rows has nothing to do, beside
    ones that keep it busy, many to a block: neither half runs ahead of the
    other (short sequences have no second half; the last key tile of a divided
    item has none for the first)."""
    s = H.svdq()
    for lens in ([700] + [100] * 60 + [2000] + [90] * 60, [128, 1500] * 6, [257] * 50):
        cu = cu_of(lens)
        q, k, v = make(cu[-1], 8, 2, 128, seed=17)
        cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
        first = check(q, k, v, cu, True)
        for _ in range(20):
            got = s.attention(q, k, v, cut, True)
            s.check_device_error()
            assert torch.equal(got, first)


def test_workspace_is_optional_and_checked():
    """The C ABI with and without workspace: both within the tolerance; too
    small a one is refused; the size query knows when none is of use."""
    import ctypes
    s = H.svdq()
    lib = s._lib
    T, D = 4000, 128
    q, k, v = make(T, 2, 1, D, seed=18)
    need = lib.svdq_attention_workspace_bytes(T, 1, 2, D, 0)
    assert need > 0
    for args in ((512, 1, 2, D, 1), (4352, 1, 1 << 12, D, 0), (4000, 40, 2, D, 1), (0, 1, 2, D, 0), (T, 1, 0, D, 0),
                 (T, 1, 2, 0, 0), (T, 1, 2, 136, 0), (T, 1, 2, 60, 0), (T, 0, 2, D, 0)):
        assert lib.svdq_attention_workspace_bytes(*args) == 0
    ws = torch.empty(need + 16, dtype=torch.uint8, device=DEV)
    P = ctypes.c_void_p
    for causal in (0, 1):
        ref, tol = R.attention_ref(q, k, v, None, bool(causal), D ** -0.5)
        for w, n, want in ((None, 0, s.SVDQ_OK), (ws, need, s.SVDQ_OK), (ws, need + 16, s.SVDQ_OK),
                           (ws, need - 1, s.SVDQ_ERR_INVALID_ARG)):
            out = torch.zeros_like(q)
            st = lib.svdq_attention(s.BF16, P(q.data_ptr()), 2 * D, D, P(k.data_ptr()), D, D, P(v.data_ptr()), D, D, T,
                                    2, 1, D, None, 1, causal, D ** -0.5, P(out.data_ptr()), 2 * D, D,
                                    None if w is None else P(w.data_ptr()), n,
                                    P(torch.cuda.current_stream().cuda_stream))
            assert st == want
            s.check_device_error()
            if want == s.SVDQ_OK:
                R.assert_within(out, ref, tol)
            else:
                assert (out == 0).all()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("T,Hq,Hk", [(2600, 1, 1), (3000, 1, 1), (3333, 2, 1), (9001, 1, 1), (5000, 3, 1)])
def test_divided_items(T, Hq, Hk, causal):
    """Few rows: their key tiles are divided among the blocks and joined."""
    assert H.svdq()._lib.svdq_attention_workspace_bytes(T, 1, Hq, 128, int(causal)) > 0
    check(*make(T, Hq, Hk, 128, seed=T), None, causal)
    check(*make(T, Hq, Hk, 72, HF, seed=T), cu_of([T - 100], 50), causal)
    many = cu_of([T // 2, 0, 1, T - T // 2 - 1])     # short ones beside: if it is divided at all
    check(*make(T, Hq, Hk, 128, seed=T), many, causal)


@pytest.mark.parametrize("bad", ["inf", "nan"])
def test_divided_items_keep_bad_keys_and_values_apart(bad):
    T = 4000
    q, k, v = make(T, 1, 1, 128, seed=19, by=0.5)
    clean = H.svdq().attention(q, k, v, causal=True)
    for at in (0, 640, 1100, 2900, 3999):
        v2 = v.clone()
        v2[at, 0, 5] = float(bad)
        got = check(q, k, v2, None, True, rel=False)
        assert torch.equal(got[:at], clean[:at])
        k2 = k.clone()
        k2[at, 0, 9] = float("nan")
        got = H.svdq().attention(q, k2, v, causal=True)
        assert torch.equal(got[:at], clean[:at]) and torch.isnan(got[at:]).all()


@pytest.mark.parametrize("what", ["norm", "rope", "attention", "divided"])
def test_first_call_of_a_process_may_be_captured(what):
    """A fresh process whose first call of the operator is under capture."""
    import os
    import subprocess
    import sys
    code = """
import torch
from nvfp4_w4a4_quantized_smooth_b200 import svdq as s
T = 4000
x = torch.randn(T, 256, device="cuda").bfloat16()
q = x.view(T, 2, 128)
pos = torch.zeros(T, 3, dtype=torch.int32, device="cuda")
calls = dict(norm=lambda: s.norm_gate_residual(x, x)[0], rope=lambda: s.rope_qk(q, None, pos, s.RopePlan((32, 48, 48), 256.0, 128))[0],
             attention=lambda: s.attention(q[:300], q[:300], q[:300]), divided=lambda: s.attention(q, q, q))
f = calls["%s"]
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = f()
g.replay()
s.check_device_error()
assert torch.equal(got, f())
""" % what
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
