"""norm_gate_residual against float64: every combination of its parts, odd
widths and row counts, strides, sequences, in-place outputs."""

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


def operands(T, C, S, dtype, seed, mean=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rnd(*shape, by=1.0, add=0.0):
        return (torch.randn(*shape, generator=g, device=DEV) * by + add).to(dtype)

    mod = rnd(S, 3 * C, by=0.7)
    return dict(x=rnd(T, C, by=2.0, add=mean), y=rnd(T, C, add=mean), gate=mod[:, :C], scale=mod[:, C:2 * C],
                shift=mod[:, 2 * C:], post_weight=rnd(C, by=0.3, add=1.0), pre_weight=rnd(C, by=0.3, add=1.0))


def run(o, cu, want_h=True, what="", **kw):
    """Call the operator on the operands and compare; returns (h, n)."""
    s = H.svdq()
    x, y = o["x"], o.get("y")
    args = {k: o.get(k) for k in ("gate", "scale", "shift", "post_weight", "pre_weight")}
    opts = dict(post=kw.get("post"), pre=kw.get("pre", "rms"), eps=kw.get("eps", 1e-6),
                gate_tanh=kw.get("gate_tanh", False), residual_scale=kw.get("a", 1.0))
    x0, y0 = x.clone(), None if y is None else y.clone()
    h0, n0 = kw.get("h"), kw.get("n")
    h, n = s.norm_gate_residual(x, y, **args, **opts, h=h0, n=n0,
                                cu_seqlens=None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV))
    hr, ht, nr, nt = R.norm_gate_ref(x0, y0, args["gate"], args["scale"], args["shift"], args["post_weight"],
                                     args["pre_weight"], opts["post"], opts["pre"], opts["eps"],
                                     opts["gate_tanh"], opts["residual_scale"], cu)
    rows = ~torch.isnan(nr).all(-1)
    if y is not None:
        R.assert_within(h[rows], hr[rows], ht[rows], what + " h")
    else:
        assert h is x
    if n is not None:
        R.assert_within(n[rows], nr[rows], nt[rows], what + " n")
    return h, n


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("post", [None, "rms", "layer"])
@pytest.mark.parametrize("pre", ["rms", "layer", None])
@pytest.mark.parametrize("gate", ["", "linear", "tanh"])
def test_every_combination(dtype, post, pre, gate):
    T, C = 37, 200
    o = operands(T, C, 3, dtype, 1)
    if not gate:
        o["gate"] = None
    if post is None:
        o["post_weight"] = None
    if pre is None:
        o["pre_weight"] = None
    run(o, cu_of([20, 0, 17]), post=post, pre=pre, gate_tanh=gate == "tanh", a=0.75)
    for drop in (("shift",), ("scale", "shift"), ("post_weight", "pre_weight")):
        run({**o, **{k: None for k in drop}}, cu_of([20, 0, 17]), post=post, pre=pre, gate_tanh=gate == "tanh")


@pytest.mark.parametrize("C", [8, 16, 72, 248, 256, 264, 1000, 3840, 4088, 4096, 4104, 5128, 8192])
@pytest.mark.parametrize("T", [1, 2, 5, 150])
def test_widths(C, T):
    run(operands(T, C, 1, BF, C + T), None, post="rms", pre="layer", gate_tanh=True)


@pytest.mark.parametrize("T", [295, 296, 297, 1185, 4352])
def test_row_counts(T):
    o = operands(T, 264, 2, BF, T)
    run(o, cu_of([T // 3, T - T // 3]), post="rms", pre="rms")
    o = operands(T, 3840, 1, BF, T)
    run(o, None, post="layer", pre="layer")


def test_first_norm_of_a_stack():
    o = operands(77, 3840, 1, BF, 5)
    for drop in (("gate", "post_weight", "y", "shift"), ("gate", "post_weight", "y", "scale", "shift")):
        run({**o, **{k: None for k in drop}}, None)


def test_only_the_residual():
    o = operands(50, 520, 1, HF, 6)
    o.update(scale=None, shift=None, pre_weight=None)
    h, n = run(o, None, post="rms", pre=None)
    assert n is None


@pytest.mark.parametrize("lens", [[3] * 100, [0] * 33 + [5] + [0] * 40 + [7], [1, 0, 0, 64, 200]])
def test_many_sequences(lens):
    S, T = len(lens), sum(lens)
    run(operands(T, 136, S, BF, T), cu_of(lens), post="rms", pre="rms", gate_tanh=True)


@pytest.mark.parametrize("C", [72, 3840])
def test_rows_in_no_sequence_stay_and_do_not_matter(C):
    """Rows in front of the first and behind the last sequence: NaN inputs,
    outputs untouched."""
    T, cu = 60, [7, 20, 20, 50]
    o = operands(T, C, 3, BF, 8)
    out = [torch.randn(T, C, device=DEV).to(BF) for _ in range(2)]
    keep = [t.clone() for t in out]
    for t in (o["x"], o["y"]):
        t[:7] = float("nan")
        t[50:] = float("inf")
    run(o, cu, post="rms", pre="layer", h=out[0], n=out[1])
    for t, k in zip(out, keep):
        assert torch.equal(t[:7], k[:7]) and torch.equal(t[50:], k[50:])


def test_no_sequence_has_rows():
    o = operands(9, 64, 2, BF, 8)
    h = torch.ones(9, 64, device=DEV, dtype=BF)
    n = torch.ones(9, 64, device=DEV, dtype=BF)
    for cu in ([0, 0, 0], [9, 9, 9]):
        run(o, cu, post="rms", h=h, n=n)
        assert (h == 1).all() and (n == 1).all()


def test_a_row_that_is_not_finite_stays_in_its_row():
    o = operands(64, 264, 1, BF, 9)
    o["x"][10, 3] = float("nan")
    o["y"][20, 100] = float("inf")
    h, n = H.svdq().norm_gate_residual(o["x"], o["y"], gate=o["gate"], post="rms", pre="rms")
    clean = torch.ones(64, dtype=torch.bool)
    clean[[10, 20]] = False
    assert torch.isfinite(h[clean.cuda()]).all() and torch.isfinite(n[clean.cuda()]).all()
    assert torch.isnan(n[10]).all()


def test_large_mean_layer_norm_keeps_its_digits():
    """mean 500, deviation 1 (2 for x): the statistics are of the deviations."""
    o = operands(33, 1024, 1, HF, 10, mean=500.0)
    o.update(gate=None, scale=None, shift=None, pre_weight=None, post_weight=None)
    run(o, None, post="layer", pre="layer")


@pytest.mark.parametrize("how", ["h=x", "h=y", "n=x", "n=y", "h=x,n=y", "h=y,n=x"])
def test_in_place(how):
    o = operands(311, 3840, 2, BF, 11)
    names = dict(p.split("=") for p in how.split(","))
    h, n = run(o, cu_of([100, 211]), post="rms", pre="rms", gate_tanh=True,
               h=o[names["h"]] if "h" in names else None, n=o[names["n"]] if "n" in names else None)


def test_strided_rows():
    """x, y, h and n as columns of one wider buffer, one gate for all sequences."""
    T, C = 130, 264
    wide = torch.randn(T, 4 * C + 8, device=DEV).to(BF)
    o = operands(T, C, 2, BF, 12)
    o["x"], o["y"] = wide[:, :C], wide[:, C:2 * C]
    o["gate"] = o["gate"][:1].expand(2, C)
    rest = wide[:, 4 * C:].clone()
    run(o, cu_of([60, 70]), post="rms", pre="rms", h=wide[:, 2 * C:3 * C], n=wide[:, 3 * C:4 * C])
    assert torch.equal(wide[:, 4 * C:], rest)


def test_offsets_over_32_bits():
    """Rows 2^23 elements apart: the last ones lie behind 2^31 elements."""
    T, C, ld = 300, 64, 1 << 23
    wide = torch.empty((T - 1) * ld + 4 * C, dtype=BF, device=DEV)
    o = operands(T, C, 1, BF, 13)
    v = [wide.as_strided((T, C), (ld, 1), i * C) for i in range(4)]
    v[0].copy_(o["x"]), v[1].copy_(o["y"])
    o["x"], o["y"] = v[0], v[1]
    run(o, None, post="rms", h=v[2], n=v[3])


def test_bad_offsets_stay_inside():
    """Offsets outside [0, T] or falling: no row outside the tensors is touched."""
    s = H.svdq()
    T, C = 40, 72
    wide = torch.full((3 * T, C), 7.0, dtype=BF, device=DEV)
    o = operands(T, C, 3, BF, 14)
    for cu in ([-5, 10, 100, 2 ** 31 - 1], [30, 5, 2, 40], [-2 ** 31, -1, -1, -1], [50, 60, 70, 80]):
        s.norm_gate_residual(o["x"], o["y"], gate=o["gate"], h=wide[T:2 * T],
                             cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV))
        assert (wide[:T] == 7).all() and (wide[2 * T:] == 7).all()


def test_repeats_bit_for_bit_on_another_stream_and_captured():
    s = H.svdq()
    o = operands(500, 3840, 2, BF, 15)
    cu = torch.tensor([0, 200, 500], dtype=torch.int32, device=DEV)
    call = lambda **kw: s.norm_gate_residual(o["x"], o["y"], gate=o["gate"], scale=o["scale"], post="rms",  # noqa: E731
                                             gate_tanh=True, cu_seqlens=cu, **kw)
    h, n = call()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    h2, n2 = call(stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(h, h2) and torch.equal(n, n2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h3, n3 = call()
    for _ in range(3):
        h3.zero_(), n3.zero_()
        graph.replay()
        assert torch.equal(h, h3) and torch.equal(n, n3)


def test_binding_refuses():
    s = H.svdq()
    x = torch.zeros(4, 64, dtype=BF, device=DEV)
    cu = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    for kw in (dict(y=x.half()), dict(y=x[:3]), dict(y=x, gate=x[:2]), dict(y=x, post_weight=x[0, :32]),
               dict(y=x, post="batch"), dict(y=x.cpu()), dict(cu_seqlens=cu.long()), dict(cu_seqlens=cu.cpu()),
               dict(cu_seqlens=cu[:1]), dict(cu_seqlens=torch.zeros(4, dtype=torch.int32, device=DEV)[::2]),
               dict(h=x), dict(y=x, h=x.float()), dict(y=x.t().contiguous().t()), dict(y=x, n=x[:, :32])):
        with pytest.raises(ValueError):
            s.norm_gate_residual(x, **kw)
    with pytest.raises(ValueError):
        s.norm_gate_residual(x.float())
    with pytest.raises(s.SvdqError):
        s.norm_gate_residual(x, x.clone(), h=x, n=x)
    with pytest.raises(s.SvdqError):
        s.norm_gate_residual(torch.zeros(4, 68, dtype=BF, device=DEV))
    h, n = s.norm_gate_residual(x[:0], x[:0])
    assert h.shape == n.shape == (0, 64)
