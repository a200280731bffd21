"""rope_qk against float64: axes, both pairings, the norm, head widths,
strided views, in place, far positions."""

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


def check(T, Hq, Hk, D, axes, pairs=True, norm=True, dtype=BF, far=1000, theta=256.0, seed=0, views=None, inplace=False):
    """views: (q, k) to fill and use; else columns of one qkv buffer."""
    s = H.svdq()
    g = torch.Generator(device=DEV).manual_seed(seed)
    if views is None:
        qkv = torch.empty(T, (Hq + 2 * Hk) * D, dtype=dtype, device=DEV)
        q, k = qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        qkv.normal_(generator=g)
        rest = qkv[:, (Hq + Hk) * D:].clone()
    else:
        q, k = views
        for t in views:
            t.copy_(torch.randn(t.shape, generator=g, device=DEV))
    w = [(torch.rand(D, generator=g, device=DEV) + 0.5).to(dtype) if norm else None for _ in range(2)]
    pos = torch.randint(-far, far, (T, len(axes)), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    plan = s.RopePlan(axes, theta, D, pairs)
    want = [R.rope_ref(t, wt, pos, axes, theta, pairs, 1e-6) for t, wt in zip((q, k), w)]
    q0, k0 = q.clone(), k.clone()
    out = dict(q_out=q, k_out=k) if inplace else {}
    got = s.rope_qk(q, k, pos, plan, w[0], w[1], **out)
    for name, o, (ref, tol) in zip("qk", got, want):
        R.assert_within(o, ref, tol, name)
    if not inplace:
        assert torch.equal(q, q0) and torch.equal(k, k0)
    if views is None:
        assert torch.equal(qkv[:, (Hq + Hk) * D:], rest)
    return got


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("pairs", [True, False])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("D,axes", [(128, (32, 48, 48)), (64, (16, 24, 24)), (128, (16, 16)), (8, (4, 4)),
                                    (96, (32, 32, 32)), (80, (16, 32, 16)), (256, (64, 64, 128)), (16, (16,)),
                                    (136, (32, 96)), (128, (32, 32, 32, 32)), (64, (8, 24, 24)), (64, (16, 24)),
                                    (24, (8,)), (88, (40, 48))])
def test_axes_and_widths(dtype, pairs, norm, D, axes):
    if not pairs and sum(axes) % 8:
        pytest.skip("halves need 8 | R")
    check(33, 3, 2, D, axes, pairs, norm, dtype)


@pytest.mark.parametrize("axes", [(2,), (2, 4, 4), (6, 10, 14), (10, 30)])
def test_a_rotated_part_that_is_no_multiple_of_eight(axes):
    check(21, 2, 1, 64, axes)


@pytest.mark.parametrize("T", [1, 2, 3, 5, 591, 593, 1183, 2371, 4352])
def test_token_counts(T):
    check(T, 30, 30, 128, (32, 48, 48), seed=T)
    check(T, 7, 1, 64, (16, 24, 24), pairs=False, norm=False, seed=T)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (32, 8), (17, 1), (64, 64)])
def test_heads(Hq, Hk):
    check(10, Hq, Hk, 128, (32, 48, 48))


def test_far_positions():
    """Any int32 position, frequencies from 1 down: the angle keeps its digits."""
    for theta in (256.0, 10000.0, 1e6):
        check(100, 2, 2, 128, (32, 48, 48), far=2 ** 31 - 1, theta=theta)


@pytest.mark.parametrize("pairs", [True, False])
@pytest.mark.parametrize("D", [128, 80])
def test_in_place(pairs, D):
    check(700, 5, 3, D, (16, 32, 16), pairs, inplace=True)


def test_one_of_the_two():
    s = H.svdq()
    q = torch.randn(9, 2, 64, device=DEV).to(BF)
    pos = torch.arange(9, device=DEV, dtype=torch.int32)[:, None].expand(9, 3).contiguous()
    plan = s.RopePlan((16, 24, 24), 256.0, 64)
    both = s.rope_qk(q, q.clone(), pos, plan)
    a, none = s.rope_qk(q, None, pos, plan)
    none2, b = s.rope_qk(None, q, pos, plan)
    assert none is None and none2 is None
    assert torch.equal(a, both[0]) and torch.equal(b, both[1])


def test_heads_in_front_of_tokens():
    """[H, T, D] memory: head stride over token stride."""
    q = torch.empty(4, 50, 64, dtype=BF, device=DEV).transpose(0, 1)
    k = torch.empty(2, 50, 64, dtype=BF, device=DEV).transpose(0, 1)
    check(50, 4, 2, 64, (16, 24, 24), views=(q, k))
    check(50, 4, 2, 64, (16, 24, 24), views=(q, k), inplace=True)


def test_offsets_over_32_bits():
    T, st = 300, 1 << 23
    wide = torch.empty((T - 1) * st + 4 * 64, dtype=BF, device=DEV)
    q = wide.as_strided((T, 2, 64), (st, 64, 1), 0)
    k = wide.as_strided((T, 2, 64), (st, 64, 1), 128)
    check(T, 2, 2, 64, (16, 24, 24), views=(q, k), inplace=True)


def test_elements_outside_the_rotation_pass_whatever_they_hold():
    s = H.svdq()
    q = torch.randn(6, 1, 64, device=DEV).to(BF)
    q[2, 0, 10] = float("inf")        # next to the rotated ten
    q[3, 0, 40] = float("nan")
    pos = torch.full((6, 3), 5, device=DEV, dtype=torch.int32)
    o, _ = s.rope_qk(q, None, pos, s.RopePlan((2, 4, 4), 256.0, 64))
    # as values: a NaN's payload is not one
    assert torch.equal(torch.nan_to_num(o[..., 10:], 7.0), torch.nan_to_num(q[..., 10:], 7.0))
    assert torch.equal(torch.isnan(o), torch.isnan(q))
    assert torch.isfinite(o[..., :10]).all()


def test_length_and_inverse():
    """A rotation keeps each pair's length, and position 0 changes nothing."""
    s = H.svdq()
    q = torch.randn(40, 3, 128, device=DEV).to(HF)
    plan = s.RopePlan((32, 48, 48), 256.0, 128)
    zero = torch.zeros(40, 3, device=DEV, dtype=torch.int32)
    assert torch.equal(s.rope_qk(q, None, zero, plan)[0], q)
    o, _ = s.rope_qk(q, None, zero + 77, plan)
    back, _ = s.rope_qk(o, None, zero - 77, plan)
    # two roundings of a pair, each u of its length
    u = R.half_step(HF)
    length = q.double().unflatten(-1, (64, 2)).norm(dim=-1).repeat_interleave(2, -1)
    assert ((back.double() - q.double()).abs() <= 2 * (2 * u + 2 * R.ROPE_SLACK) * length + 2 * R.tiny(HF)).all()


def test_streams_and_graphs():
    s = H.svdq()
    q = torch.randn(300, 8, 128, device=DEV).to(BF)
    k = torch.randn(300, 2, 128, device=DEV).to(BF)
    pos = torch.randint(0, 64, (300, 3), device=DEV, dtype=torch.int32)
    plan = s.RopePlan((32, 48, 48), 256.0, 128)
    a = s.rope_qk(q, k, pos, plan)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    b = s.rope_qk(q, k, pos, plan, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = s.rope_qk(q, k, pos, plan)
    del plan               # the graph keeps the frequencies it was captured with
    graph.replay()
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_binding_refuses():
    s = H.svdq()
    q = torch.zeros(4, 2, 64, dtype=BF, device=DEV)
    pos = torch.zeros(4, 3, dtype=torch.int32, device=DEV)
    plan = s.RopePlan((16, 24, 24), 256.0, 64)
    for a in ((q, q.half(), pos, plan), (q, q[:3], pos, plan), (q, q[:, 0], pos, plan), (q, q[..., :32], pos, plan),
              (q, None, pos.long(), plan), (q, None, pos[:, :2], plan), (q, None, pos.cpu(), plan),
              (q, None, pos[:3], plan), (q.float(), None, pos, plan),
              (q, None, pos, s.RopePlan((16, 24, 24), 256.0, 128)), (q, None, pos, plan, q[0, 0, :32])):
        with pytest.raises(ValueError):
            s.rope_qk(*a)
    with pytest.raises(ValueError):
        s.rope_qk(q, None, pos, plan, k_out=q)
    with pytest.raises(s.SvdqError):
        s.rope_qk(q, None, pos, plan, q_out=torch.zeros(4, 2, 68, dtype=BF, device=DEV)[..., 4:])
    with pytest.raises(s.SvdqError):           # q and k one tensor, both in place
        s.rope_qk(q, q, pos, plan, q_out=q, k_out=q)
    o, _ = s.rope_qk(q[:0], None, pos[:0], plan)
    assert o.shape == (0, 2, 64)
