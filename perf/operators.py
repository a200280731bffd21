"""Cases of the operators between the linears of a diffusion transformer block:

* norm    norms before and after a block, fused with its gate and residual scale
* rope    rotary positions with several axes on q and k, with their per-head RMS norm
* attn    attention over whole packed sequences, full or causal, grouped heads

`run` computes them in plain torch operations (32 bits, rounded once at the
end) or, with `own` set, by the calls a user makes of this package.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}

# Sizes of this repository's block: 4352 tokens (64 x 64 latent patches and
# 256 of text), hidden 3840 = 30 heads of 128; 17408 tokens are four of them.


def listed():
    full = "4352"
    four = "4352,4352,4352,4352"
    ragged = "1291,77,1,640,0,2343"
    return [
        # one token of a serving step: latency
        dict(name="norm_1", op="norm", type="bf16", lens="1", C=3840, post="rms", pre="rms", y=True, gate=True, tanh=True, shift=False),
        # a chunk of new text tokens through the entry norm only (no branch yet)
        dict(name="norm_77_entry", op="norm", type="bf16", lens="77", C=3840, post="", pre="rms", y=False, gate=False, tanh=False, shift=False),
        # between the attention and the feed-forward of one block, one image
        dict(name="norm_4352", op="norm", type="bf16", lens=full, C=3840, post="rms", pre="rms", y=True, gate=True, tanh=True, shift=False),
        # four images a batch, layer norm with shift and scale, no norm after the branch, fp16
        dict(name="norm_17408_layer", op="norm", type="fp16", lens=four, C=3840, post="", pre="layer", y=True, gate=True, tanh=False, shift=True),
        # one token: latency
        dict(name="rope_1", op="rope", type="bf16", T=1, Hq=30, Hk=30, D=128, axes="32,48,48", theta=256.0, pairs=True, norm=True, far=64),
        # q and k of one image, normed and turned by (time, height, width)
        dict(name="rope_4352", op="rope", type="bf16", T=4352, Hq=30, Hk=30, D=128, axes="32,48,48", theta=256.0, pairs=True, norm=True, far=512),
        # an odd number of tokens, grouped heads, halves, no norm, far positions (long videos)
        dict(name="rope_9973_halves", op="rope", type="bf16", T=9973, Hq=32, Hk=8, D=128, axes="32,48,48", theta=10000.0, pairs=False, norm=False, far=1 << 24),
        # a short text prompt, causal, grouped heads: latency
        dict(name="attn_77_causal", op="attn", type="bf16", lens="77", Hq=32, Hk=8, D=128, causal=True),
        # prompts of different lengths packed, causal, grouped heads, an empty one and one of one token
        dict(name="attn_ragged_causal", op="attn", type="bf16", lens=ragged, Hq=32, Hk=8, D=128, causal=True),
        # narrower heads, fp16, two images
        dict(name="attn_2304_d64", op="attn", type="fp16", lens="1280,1024", Hq=24, Hk=24, D=64, causal=False),
        # one image: the attention of the block whose linears this package has
        dict(name="attn_4352", op="attn", type="bf16", lens=full, Hq=30, Hk=30, D=128, causal=False),
        # four images
        dict(name="attn_17408", op="attn", type="bf16", lens=four, Hq=30, Hk=30, D=128, causal=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _split(rng, T, most):
    """T tokens in up to `most` sequences of different lengths, an empty one now and then."""
    cuts = sorted(rng.randint(0, T) for _ in range(rng.randint(1, most) - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [T])]


def draw(rng):
    op = rng.choice(["norm", "rope", "attn", "attn"])
    kind = rng.choice(["bf16", "bf16", "fp16"])
    if op == "norm":
        C = 8 * _log(rng, 8, 768)
        T = _log(rng, 1, min(17408, 17408 * 3840 // C))
        y = rng.random() < 0.8
        gate = y and rng.random() < 0.8
        return dict(op=op, type=kind, lens=",".join(map(str, _split(rng, T, 8))), C=C, post=rng.choice(["", "rms", "layer"]) if y else "",
                    pre=rng.choice(["rms", "layer"]), y=y, gate=gate, tanh=gate and rng.random() < 0.5, shift=rng.random() < 0.5)
    if op == "rope":
        D = rng.choice([64, 128, 128, 96, 80])
        Hk = rng.choice([1, 2, 4, 8, 30])
        Hq = Hk * rng.choice([1, 1, 2, 4])
        axes = rng.choice({64: ["16,24,24", "64", "8,24,24"], 128: ["32,48,48", "16,56,56", "64,64", "32,32,32"],
                           96: ["32,32,32", "24,36,36"], 80: ["16,32,32", "16,24,24"]}[D])
        T = _log(rng, 1, min(17408, 4352 * 60 * 128 // ((Hq + Hk) * D)))
        return dict(op=op, type=kind, T=T, Hq=Hq, Hk=Hk, D=D, axes=axes, theta=rng.choice([256.0, 10000.0]), pairs=rng.random() < 0.5,
                    norm=rng.random() < 0.6, far=_log(rng, 64, 1 << 24))
    D = rng.choice([64, 128, 128, 128, 96, 80, 72, 40])
    Hk = rng.choice([1, 2, 4, 8, 30])
    Hq = Hk * rng.choice([1, 1, 2, 4])
    T = _log(rng, 1, min(8192, round(math.sqrt(4 * 4352 ** 2 * 30 / Hq / 2))))
    lens = _split(rng, T, 6)
    return dict(op=op, type=kind, lens=",".join(map(str, lens)), Hq=Hq, Hk=Hk, D=D, causal=rng.random() < 0.6)


def _lens(case):
    return [int(n) for n in case["lens"].split(",")]


def _cu(case):
    cu = [0]
    for n in _lens(case):
        cu.append(cu[-1] + n)
    return cu


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    t = TYPES[case["type"]]

    def normal(*shape, by=1.0, to=None):
        return (torch.randn(*shape, generator=g, device=DEV) * by).to(to or t)

    def weight(n):
        return (torch.rand(n, generator=g, device=DEV) * 1.5 + 0.5).to(t)

    s = dict(case)
    if case["op"] == "norm":
        C, S = case["C"], len(_lens(case))
        T = sum(_lens(case))
        s["cu"] = torch.tensor(_cu(case), dtype=torch.int32, device=DEV)
        s["x"] = normal(T, C, by=2.0)
        s["y"] = normal(T, C) if case["y"] else None
        mod = normal(S, 3 * C, by=0.5)          # one product of the conditioning, cut in three
        s["gate"] = mod[:, :C] if case["gate"] else None
        s["scale"] = mod[:, C:2 * C]
        s["shift"] = mod[:, 2 * C:] if case["shift"] else None
        s["post_weight"] = weight(C) if case["post"] == "rms" else None
        s["pre_weight"] = weight(C) if case["pre"] == "rms" else None
        s["a"] = 1.0 if not case["y"] else 0.875
    elif case["op"] == "rope":
        T, Hq, Hk, D = (case[k] for k in ("T", "Hq", "Hk", "D"))
        axes = [int(n) for n in case["axes"].split(",")]
        qkv = normal(T, (Hq + 2 * Hk) * D)      # the output of one linear; v is left as it is
        s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        s["axes"] = axes
        s["pos"] = torch.randint(0, case["far"], (T, len(axes)), generator=g, device=DEV, dtype=torch.int32)
        s["q_weight"] = weight(D) if case["norm"] else None
        s["k_weight"] = weight(D) if case["norm"] else None
        if own:
            s["plan"] = svdq_module().RopePlan(axes, theta=case["theta"], head_dim=D, interleaved=case["pairs"])
    else:
        T, Hq, Hk, D = sum(_lens(case)), case["Hq"], case["Hk"], case["D"]
        s["lens"] = _lens(case)
        s["cu"] = torch.tensor(_cu(case), dtype=torch.int32, device=DEV)
        s["q"] = normal(T, Hq, D, by=1.4)       # as after a norm with its weight
        s["k"] = normal(T, Hk, D, by=1.4)
        s["v"] = normal(T, Hk, D)
    return s


def svdq_module():
    from nvfp4_w4a4_quantized_smooth_b200 import svdq
    return svdq


EPS = 1e-6


def _norm(v, kind, w):
    """The norm of each row in 32 bits."""
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    if kind:
        v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    return v if w is None else v * w.float()


def _norm_plain(s):
    t = s["x"].dtype
    x = s["x"].float()
    row = torch.bucketize(torch.arange(x.shape[0], device=DEV, dtype=torch.int32), s["cu"][1:], right=True)
    h = x
    if s["y"] is not None:
        u = _norm(s["y"].float(), s["post"], s["post_weight"])
        if s["gate"] is not None:
            g = s["gate"].float()
            u = (torch.tanh(g) if s["tanh"] else g)[row] * u
        h = s["a"] * x + u
    n = _norm(h, s["pre"], s["pre_weight"]) * (1.0 + s["scale"].float())[row]
    if s["shift"] is not None:
        n = n + s["shift"].float()[row]
    return dict(h=h.to(t) if s["y"] is not None else None, n=n.to(t))


def _turn(v, w, cos, sin, R, pairs):
    t = v.dtype
    v = v.float()
    if w is not None:
        v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w.float()
    if pairs:
        a, b = v[..., 0:R:2], v[..., 1:R:2]
        r = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = v[..., :R // 2], v[..., R // 2:R]
        r = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((r, v[..., R:]), -1).to(t)


def _rope_plain(s):
    pos = s["pos"].double()     # angles of far positions need 64 bits
    axis = torch.cat([torch.full((d // 2,), a, device=DEV) for a, d in enumerate(s["axes"])])
    power = torch.cat([torch.arange(0, d, 2, device=DEV, dtype=torch.float64) / d for d in s["axes"]])
    phi = pos[:, axis] * (s["theta"] ** -power)
    cos, sin = torch.cos(phi).float()[:, None], torch.sin(phi).float()[:, None]
    R = sum(s["axes"])
    return dict(q=_turn(s["q"], s["q_weight"], cos, sin, R, s["pairs"]), k=_turn(s["k"], s["k_weight"], cos, sin, R, s["pairs"]))


def _attn_plain(s):
    """Sequences padded to the longest, all of them in one product."""
    q, k, v = s["q"], s["k"], s["v"]
    T, Hq, D = q.shape
    Hk = k.shape[1]
    most = max(s["lens"])
    at = torch.arange(most, device=DEV)
    start, count = s["cu"][:-1].long()[:, None], (s["cu"][1:] - s["cu"][:-1]).long()[:, None]
    there = at < count                                     # [S, most]
    row = torch.where(there, start + at, torch.zeros_like(at))
    Q = q.float()[row].view(-1, most, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4).reshape(-1, Hk, Hq // Hk * most, D)
    K = k.float()[row].permute(0, 2, 3, 1)
    V = v.float()[row].permute(0, 2, 1, 3)
    w = torch.matmul(Q, K).view(-1, Hk, Hq // Hk, most, most).mul_(D ** -0.5)
    keep = there[:, None, None, None, :]
    if s["causal"]:
        keep = keep & (at[:, None] >= at)
    w.masked_fill_(~keep, -math.inf)
    w = w.sub_(w.amax(-1, keepdim=True).clamp_min_(-3e38)).exp_()
    o = torch.matmul(w.view(-1, Hk, Hq // Hk * most, most), V)
    o = o.view(-1, Hk, Hq // Hk, most, D) / w.sum(-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(-1, most, Hq, D)
    return o[there].to(q.dtype)


def run(s):
    if own:
        svdq = svdq_module()
        if s["op"] == "norm":
            h, n = svdq.norm_gate_residual(s["x"], s["y"], gate=s["gate"], scale=s["scale"], shift=s["shift"], post_weight=s["post_weight"],
                                           pre_weight=s["pre_weight"], post=s["post"] or None, pre=s["pre"], eps=EPS, gate_tanh=s["tanh"],
                                           residual_scale=s["a"], cu_seqlens=s["cu"])
            return dict(h=h if s["y"] is not None else None, n=n)
        if s["op"] == "rope":
            q, k = svdq.rope_qk(s["q"], s["k"], s["pos"], s["plan"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
            return dict(q=q, k=k)
        return svdq.attention(s["q"], s["k"], s["v"], cu_seqlens=s["cu"], causal=s["causal"])
    if s["op"] == "norm":
        return _norm_plain(s)
    if s["op"] == "rope":
        return _rope_plain(s)
    return _attn_plain(s)


def work(case):
    if case["op"] == "norm":
        T, C, S = sum(_lens(case)), case["C"], len(_lens(case))
        rows = 2 + (2 if case["y"] else 0)                          # x, n, and y, h
        mods = S * C * (1 + case["gate"] + case["shift"])
        ws = C * ((case["post"] == "rms") + (case["pre"] == "rms"))
        return {"bytes": 2 * (rows * T * C + mods + ws) + 4 * (S + 1), "flops": T * C * (4 + 4 * case["y"] + 4 * bool(case["post"]))}
    if case["op"] == "rope":
        n = case["T"] * (case["Hq"] + case["Hk"]) * case["D"]
        A = case["axes"].count(",") + 1
        return {"bytes": 4 * n + 4 * case["T"] * A + (4 * case["D"] if case["norm"] else 0), "flops": n * (3 + 4 * case["norm"])}
    T, Hq, Hk, D = sum(_lens(case)), case["Hq"], case["Hk"], case["D"]
    pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in _lens(case))
    return {"bytes": 2 * T * D * (2 * Hq + 2 * Hk) + 4 * (len(_lens(case)) + 1), "flops": 4 * D * Hq * pairs}


def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence."""
    s = prepare(case, seed)

    def wide(v):
        return v.to(torch.float64)

    def unit(v, kind):
        if kind == "rms":
            return v / torch.sqrt(torch.sum(v ** 2, -1, keepdim=True) / v.shape[-1] + EPS)
        if kind == "layer":
            var, mean = torch.var_mean(v, dim=-1, keepdim=True, correction=0)
            return (v - mean) / torch.sqrt(var + EPS)
        return v

    if case["op"] == "norm":
        cu, hs, ns = _cu(case), [], []
        for i, (b, e) in enumerate(zip(cu, cu[1:])):
            h = wide(s["x"][b:e])
            if s["y"] is not None:
                u = unit(wide(s["y"][b:e]), case["post"])
                u = u if s["post_weight"] is None else u * wide(s["post_weight"])
                if s["gate"] is not None:
                    g = wide(s["gate"][i])
                    if case["tanh"]:
                        g = 1 - 2 / (torch.exp(2 * g) + 1)
                    u = u * g
                h = h * s["a"] + u
            n = unit(h, case["pre"])
            n = n if s["pre_weight"] is None else n * wide(s["pre_weight"])
            n = n + n * wide(s["scale"][i])
            if s["shift"] is not None:
                n = n + wide(s["shift"][i])
            hs.append(h)
            ns.append(n)
        return dict(h=torch.cat(hs) if s["y"] is not None else None, n=torch.cat(ns))
    if case["op"] == "rope":
        out = {}
        for name in ("q", "k"):
            v = wide(s[name])
            if case["norm"]:
                v = unit(v, "rms") * wide(s[name + "_weight"])
            r, first, R = v.clone(), 0, sum(s["axes"])
            for a, d in enumerate(s["axes"]):
                i = torch.arange(d // 2, device=DEV)
                p = first // 2 + i
                lo, hi = (2 * p, 2 * p + 1) if case["pairs"] else (p, p + R // 2)
                z = torch.complex(v[..., lo], v[..., hi])
                phi = wide(s["pos"][:, a:a + 1]) * torch.exp(-2.0 * math.log(case["theta"]) / d * wide(i))
                z = z * torch.polar(torch.ones_like(phi), phi)[:, None]
                r[..., lo], r[..., hi] = z.real, z.imag
                first += d
            out[name] = r
        return out
    g = case["Hq"] // case["Hk"]
    cu, parts = _cu(case), []
    for b, e in zip(cu, cu[1:]):
        q = wide(s["q"][b:e]).transpose(0, 1) / math.sqrt(case["D"])
        k = wide(s["k"][b:e]).transpose(0, 1).repeat_interleave(g, 0)
        v = wide(s["v"][b:e]).transpose(0, 1).repeat_interleave(g, 0)
        w = torch.bmm(q, k.transpose(1, 2))
        if case["causal"]:
            w += torch.triu(torch.full((e - b, e - b), -math.inf, dtype=torch.float64, device=DEV), 1)
        parts.append(torch.bmm(torch.softmax(w, -1), v).transpose(0, 1))
        del w
    return torch.cat(parts)
