"""Float64 references of the operators between a block's linears, and the
tolerances their arithmetic gives.

u = torch.finfo(type).eps / 2 is the relative error of one rounding to the
tensors' type (bf16 2^-8, fp16 2^-11); results below the smallest normal are
off by at most half the smallest step (TINY).  fp32 steps are 2^-24 each.
"""

import math

import torch

F64 = torch.float64


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    f = torch.finfo(dtype)
    return f.smallest_normal * f.eps / 2 * 2


def spans(T, cu):
    return [(0, T)] if cu is None else list(zip(cu[:-1], cu[1:]))


# ---- norm_gate_residual ------------------------------------------------------

def _norm(v, kind, w, eps):
    """(normed rows, size of the terms an fp32 evaluation rounds)."""
    size = v.abs()
    if kind == "layer":
        mean = v.mean(-1, keepdim=True)
        size = size + size.mean(-1, keepdim=True)
        v = v - mean
    if kind is not None:
        r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
        v, size = v * r, size * r
    if w is not None:
        v, size = v * w.to(F64), size * w.to(F64).abs()
    return v, size


# fp32 evaluation of a row: the sums of squares and the mean run over at most
# 16 terms per thread, 5 shuffles and 16 warps (under 40 roundings, and half
# of that in the square root), the other steps are under 10 roundings or
# function results of 2 ulp: below 64 steps of 2^-24 of the terms' size.
ROW_SLACK = 2.0 ** -18


def norm_gate_ref(x, y, gate, scale, shift, post_w, pre_w, post, pre, eps, gate_tanh, a, cu):
    """(h, h's tolerance, n, n's tolerance), float64; rows in no sequence NaN."""
    T, C = x.shape
    u = half_step(x.dtype)
    nan = torch.full((T, C), math.nan, dtype=F64, device=x.device)
    h, ht, n, nt = nan.clone(), nan.clone(), nan.clone(), nan.clone()
    for s, (b, e) in enumerate(spans(T, cu)):
        if e <= b:
            continue
        hv = x[b:e].to(F64)
        hs = hv.abs()
        if y is not None:
            v, vs = _norm(y[b:e].to(F64), post, post_w, eps)
            if gate is not None:
                g = gate[s].to(F64)
                g = torch.tanh(g) if gate_tanh else g
                v, vs = v * g, vs * g.abs()
            hv = a * hv + v
            hs = abs(a) * hs + vs
        h[b:e] = hv
        ht[b:e] = u * hv.abs() + ROW_SLACK * hs + tiny(x.dtype)
        # h's own fp32 error passes through the norm: relative to its terms
        w, ws = _norm(hv, pre, pre_w, eps)
        grow = torch.ones_like(hs) if pre is None else \
            1 / torch.sqrt((hv * hv).mean(-1, keepdim=True) + eps)
        err = ws + grow * (hs + hs.mean(-1, keepdim=True)) * (1 if pre_w is None else pre_w.to(F64).abs())
        if scale is not None:
            f = 1 + scale[s].to(F64)
            w, err = w * f, err * f.abs()
        if shift is not None:
            w, err = w + shift[s].to(F64), err + shift[s].to(F64).abs()
        n[b:e] = w
        nt[b:e] = u * w.abs() + ROW_SLACK * err + tiny(x.dtype)
    return h, ht, n, nt


# ---- rope_qk --------------------------------------------------------------------

# Angle: the 64-bit product of an int32 position and turns <= 0.16 is off by
# under 2^-24 turns, its fraction rounds to fp32 within 2^-25 turns: under
# 2^-20 radians together; sine and cosine 2 ulp, two products and a sum; the
# norm as a row of 256: below 2^-18 of |e0| + |e1|.
ROPE_SLACK = 2.0 ** -18


def rope_ref(v, w, pos, axes, theta, pairs, eps):
    """(rotated, tolerance) of [T, H, D]."""
    u = half_step(v.dtype)
    dt = v.dtype
    v = v.to(F64)
    if w is not None:
        v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) * w.to(F64)
    out, tol = v.clone(), ROPE_SLACK * v.abs()
    R, first = sum(axes), 0
    for a, d in enumerate(axes):
        i = torch.arange(d // 2, device=v.device)
        phi = pos[:, a:a + 1].to(F64) * theta ** (-2.0 * i.to(F64) / d)
        c, s = torch.cos(phi)[:, None], torch.sin(phi)[:, None]
        p = first + i
        lo, hi = (2 * p, 2 * p + 1) if pairs else (p, p + R // 2)
        e0, e1 = v[..., lo], v[..., hi]
        out[..., lo], out[..., hi] = e0 * c - e1 * s, e0 * s + e1 * c
        both = ROPE_SLACK * (e0.abs() + e1.abs())
        tol[..., lo], tol[..., hi] = both, both
        first += d // 2
    return out, tol + u * out.abs() + tiny(dt)


# ---- attention ------------------------------------------------------------------

# Each weight is rounded once to the tensors' type (u), the result once (u).
# fp32: products of 16-bit numbers are exact; their sum over D <= 128 and the
# tensor core's alignment stay below 2^-17 of the sum of absolute products,
# which times scale * log2(e) is an absolute error of the exponent; the
# exponent's fma is off by 2^-24 of its size, ex2 by 2^-22, the sums of
# weights and of weighted values by under 2^-14.
def attention_ref(q, k, v, cu, causal, scale):
    """(out, tolerance) of [T, Hq, D]; rows in no sequence NaN.  Keys and
    values a row does not attend are left out by selection."""
    T, Hq, D = q.shape
    g = Hq // k.shape[1]
    u = half_step(q.dtype)
    out = torch.full((T, Hq, D), math.nan, dtype=F64, device=q.device)
    tol = out.clone()
    for b, e in spans(T, cu):
        n = e - b
        if n <= 0:
            continue
        at = torch.arange(n, device=q.device)
        for h in range(Hq):
            qh, kh, vh = (t[b:e, i].to(F64) for t, i in ((q, h), (k, h // g), (v, h // g)))
            s = qh @ kh.T * scale
            size = (qh.abs() @ kh.abs().T * scale)
            if causal:
                keep = at[:, None] >= at
                s = s.masked_fill(~keep, -math.inf)
                size = size.masked_fill(~keep, 0.0)
            w = torch.softmax(s, -1)
            finite = torch.isfinite(vh)
            o = w @ torch.where(finite, vh, 0.0)
            spread = w @ torch.where(finite, vh, 0.0).abs()
            for j in torch.nonzero(~finite.all(-1)).flatten().tolist():   # rare: in by hand
                rows = at >= j if causal else at >= 0
                bad = torch.where(finite[j], 0.0, vh[j])
                o[rows] += bad
            exponent = 2.0 ** -17 * torch.nan_to_num(size, 0.0, 0.0, 0.0).amax(-1, keepdim=True)
            out[b:e, h] = o
            tol[b:e, h] = u * o.abs() + (u + 2 * exponent + 2.0 ** -13) * spread + tiny(q.dtype)
    return out, tol


def attention_rel(dtype):
    """Relative Frobenius error for independent values of mean zero: a
    rounding is u / sqrt(3) rms; the weights' roundings add up like the
    weighted values themselves, the result's is one more: sqrt(2 / 3) u, with
    half as much again for the fp32 steps and small samples."""
    return 1.25 * half_step(dtype)


def assert_within(got, want, tol, what=""):
    """Elementwise; infinities and NaN have to be the same ones."""
    got = got.to(F64)
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN at other places"
    inf = ~fin & ~torch.isnan(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    assert torch.isfinite(got[fin]).all(), f"{what}: non-finite results"
    over = (got - want).abs()[fin] - tol[fin]
    assert over.numel() == 0 or over.max() <= 0, \
        f"{what}: {int((over > 0).sum())} of {over.numel()} off, worst by {over.max().item():.3e}"
