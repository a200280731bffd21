"""A whole block: the norms, rotary positions and attention run together with
the linears between them.  Each step is checked against float64 (the linears
against the oracle) on the GPU's own inputs to it, and dit_block gives the same
bits as the steps."""

import numpy as np
import pytest
import torch

from nvfp4_w4a4_quantized_smooth_b200 import synth

import block_ref as R
import gpu_helpers as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
HIDDEN, HEADS, FFN = 512, 4, 1024
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_quantized_smooth_b200 import build
    build.build()
    torch.cuda.init()


def make_block(seed):
    s = H.svdq()
    host, dev = {}, {}
    for i, (name, K, N) in enumerate((("qkv", HIDDEN, 3 * HIDDEN), ("out", HIDDEN, HIDDEN), ("w1", HIDDEN, FFN),
                                      ("w3", HIDDEN, FFN), ("w2", FFN, HIDDEN))):
        g = torch.Generator().manual_seed(seed + i)
        L = synth.LayerOperands(None, *synth.make_weights(K, N, 128, g))
        host[name] = L
        dev[name] = s.PreparedWeights(L.qweight.cuda(), L.wscales.cuda(), L.wcscales.cuda(), L.wtscale.cuda(),
                                      L.smooth.cuda(), L.proj_down.cuda(), L.proj_up.cuda(), L.bias.cuda())
    g = torch.Generator(device=DEV).manual_seed(seed)
    vec = lambda n: (torch.rand(n, generator=g, device=DEV) + 0.5).to(BF)  # noqa: E731
    d = HIDDEN // HEADS
    w = s.DitBlock(dev["qkv"], dev["out"], dev["w1"], dev["w3"], dev["w2"], heads=HEADS, attn_pre=vec(HIDDEN),
                   attn_post=vec(HIDDEN), ffn_pre=vec(HIDDEN), ffn_post=vec(HIDDEN), q_norm=vec(d), k_norm=vec(d), eps=EPS)
    return w, host, g


def check_linear(L, x, y, what):
    rows = H.sample_rows(x.shape[0], 16)
    at = torch.from_numpy(rows).cuda()
    ref = H.oracle_y(L, x=x[at].cpu())[0]
    H.assert_y_close(y[at].cpu(), ref, what)


@pytest.mark.parametrize("lens,causal", [([1], False), ([200], False), ([130, 1, 0, 169], False), ([77, 300], True)])
def test_dit_block(lens, causal):
    s = H.svdq()
    w, host, g = make_block(40)
    T, S = sum(lens), len(lens)
    cu = [0] + np.cumsum(lens).tolist()
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    x = torch.randn(T, HIDDEN, generator=g, device=DEV).to(BF)
    mod = (torch.randn(S, 4 * HIDDEN, generator=g, device=DEV) * 0.5).to(BF).chunk(4, 1)
    pos = torch.randint(0, 64, (T, 3), generator=g, device=DEV, dtype=torch.int32)
    plan = s.RopePlan((32, 48, 48), 256.0, HIDDEN // HEADS)
    scale_a, gate_a, scale_f, gate_f = mod

    # step by step
    _, n = s.norm_gate_residual(x, scale=scale_a, pre_weight=w.attn_pre, eps=EPS, cu_seqlens=cut)
    ref = R.norm_gate_ref(x, None, None, scale_a, None, None, w.attn_pre, None, "rms", EPS, False, 1.0, cu)
    R.assert_within(n, ref[2], ref[3], "first norm")
    qkv = s.svdq_linear(n, w.qkv)
    check_linear(host["qkv"], n, qkv, "qkv")
    q, k, v = qkv.view(T, 3, HEADS, -1).unbind(1)
    want = [R.rope_ref(t, wt, pos, plan.axes, 256.0, True, EPS) for t, wt in ((q, w.q_norm), (k, w.k_norm))]
    s.rope_qk(q, k, pos, plan, w.q_norm, w.k_norm, EPS, q_out=q, k_out=k)
    for t, (o, tol) in zip((q, k), want):
        R.assert_within(t, o, tol, "rope")
    a = s.attention(q, k, v, cut, causal)
    o, tol = R.attention_ref(q, k, v, cu, causal, (HIDDEN // HEADS) ** -0.5)
    R.assert_within(a, o, tol, "attention")
    a = a.view(T, HIDDEN)
    y = s.svdq_linear(a, w.out)
    check_linear(host["out"], a, y, "out")
    h, n = s.norm_gate_residual(x, y, gate=gate_a, gate_tanh=True, post="rms", post_weight=w.attn_post,
                                pre_weight=w.ffn_pre, scale=scale_f, eps=EPS, cu_seqlens=cut)
    ref = R.norm_gate_ref(x, y, gate_a, scale_f, None, w.attn_post, w.ffn_pre, "rms", "rms", EPS, True, 1.0, cu)
    R.assert_within(h, ref[0], ref[1], "residual")
    R.assert_within(n, ref[2], ref[3], "second norm")
    y1, y3 = s.svdq_linear(n, w.w1), s.svdq_linear(n, w.w3)
    qa, asc, lr = s.silu_mul_quantize_act(y1, y3, w.w2.smooth, w.w2.proj_down)
    y = s.w4a4_linear(qa, asc, lr, w.w2.qweight, w.w2.wscales_tiled, w.w2.wcscales, w.w2.wtscale, w.w2.proj_up,
                      w.w2.bias, proj_up_folded=w.w2.proj_up_folded)
    x2, none = s.norm_gate_residual(h, y, gate=gate_f, gate_tanh=True, post="rms", post_weight=w.ffn_post, pre=None,
                                    eps=EPS, cu_seqlens=cut)
    assert none is None
    ref = R.norm_gate_ref(h, y, gate_f, None, None, w.ffn_post, None, "rms", None, EPS, True, 1.0, cu)
    R.assert_within(x2, ref[0], ref[1], "last residual")
    s.check_device_error()

    got = s.dit_block(x, w, mod, pos, plan, cut, causal)
    assert torch.equal(got, x2)

    # captured: two blocks in a row, replayed on new inputs
    graph = torch.cuda.CUDAGraph()
    xin = x.clone()
    with torch.cuda.graph(graph):
        out = s.dit_block(s.dit_block(xin, w, mod, pos, plan, cut, causal), w, mod, pos, plan, cut, causal)
    for t in (x, x.flip(0).contiguous()):
        xin.copy_(t)
        graph.replay()
        one = s.dit_block(t, w, mod, pos, plan, cut, causal)
        assert torch.equal(out, s.dit_block(one, w, mod, pos, plan, cut, causal))
    s.check_device_error()


def test_dit_block_enters_the_device_of_its_input(monkeypatch):
    """Called while another device is the current one: on its input's."""
    s = H.svdq()
    w, _, g = make_block(60)
    x = torch.randn(40, HIDDEN, generator=g, device=DEV).to(BF)
    mod = torch.zeros(1, 4 * HIDDEN, device=DEV, dtype=BF).chunk(4, 1)
    pos = torch.zeros(40, 3, device=DEV, dtype=torch.int32)
    plan = s.RopePlan((32, 48, 48), 256.0, HIDDEN // HEADS)
    want = s.dit_block(x, w, mod, pos, plan)
    seen, entered = [x.get_device() + 1], []
    real, on = s._current_device, s._on
    monkeypatch.setattr(s, "_current_device", lambda: seen.pop() if seen else real())
    monkeypatch.setattr(s, "_on", lambda i, stream: entered.append((i, stream)) or on(i, stream))
    assert torch.equal(s.dit_block(x, w, mod, pos, plan), want)
    assert entered == [(x.get_device(), None)] and not seen
    s.check_device_error()


def test_dit_block_refuses_other_widths():
    s = H.svdq()
    w, _, _ = make_block(50)
    with pytest.raises(ValueError):
        s.DitBlock(w.qkv, w.w1, w.w1, w.w3, w.w2, heads=HEADS, attn_pre=None, attn_post=None, ffn_pre=None,
                   ffn_post=None, q_norm=None, k_norm=None)
    with pytest.raises(ValueError):
        s.DitBlock(w.qkv, w.out, w.w1, w.w3, w.w2, heads=5, attn_pre=None, attn_post=None, ffn_pre=None,
                   ffn_post=None, q_norm=None, k_norm=None)
