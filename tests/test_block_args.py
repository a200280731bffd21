"""Refusals of the operators between a block's linears, and the attention
kernel's walk over its work items, without a GPU."""

import ctypes
import itertools

import pytest
import torch

P = ctypes.c_void_p
FAKE, ODD = 0x100000, 0x100002


@pytest.fixture(scope="module")
def svdq():
    from nvfp4_w4a4_quantized_smooth_b200 import build
    build.build()
    from nvfp4_w4a4_quantized_smooth_b200 import svdq as mod
    return mod


MB = 1 << 20


def norm_args(**kw):
    a = dict(dtype=0, x=1 * MB, ldx=64, y=2 * MB, ldy=64, T=16, C=64, cu=None, S=1, post=1, post_w=None,
             gate_kind=1, gate=3 * MB, ldg=64, a=1.0, pre=1, pre_w=None, scale=4 * MB, lds=64,
             shift=None, ldb=0, eps=1e-6, h=5 * MB, ldh=64, n=6 * MB, ldn=64, stream=None)
    a.update(kw)
    return list(a.values())


NORM_BAD = [
    ("INVALID_ARG", dict(dtype=2)), ("INVALID_ARG", dict(dtype=-1)),
    ("INVALID_ARG", dict(post=3)), ("INVALID_ARG", dict(pre=-1)),
    ("INVALID_ARG", dict(gate_kind=3)), ("INVALID_ARG", dict(gate=None)),
    ("INVALID_ARG", dict(gate_kind=0)), ("INVALID_ARG", dict(eps=-1.0)),
    ("INVALID_ARG", dict(eps=float("nan"))), ("INVALID_ARG", dict(a=float("inf"))),
    ("INVALID_ARG", dict(x=None)), ("INVALID_ARG", dict(h=None)),
    ("INVALID_ARG", dict(y=None)),                                   # h without y
    ("INVALID_ARG", dict(y=None, h=None)),                           # post, gate without y
    ("INVALID_ARG", dict(y=None, h=None, post=0, gate_kind=0, gate=None, a=0.5)),
    ("INVALID_ARG", dict(y=None, h=None, post=0, gate_kind=0, gate=None, n=None, pre=0, scale=None)),
    ("INVALID_ARG", dict(n=None)),                                   # pre without n
    ("INVALID_ARG", dict(post=0, post_w=7 * MB)),
    ("INVALID_ARG", dict(h=1 * MB + 16)), ("INVALID_ARG", dict(n=5 * MB)),
    ("INVALID_ARG", dict(n=2 * MB + 128)), ("INVALID_ARG", dict(n=4 * MB)),
    ("INVALID_ARG", dict(h=1 * MB, ldh=72)),                         # other rows of x
    ("SHAPE", dict(T=-1)), ("SHAPE", dict(C=0)), ("SHAPE", dict(S=0)), ("SHAPE", dict(S=2)),
    ("SHAPE", dict(ldx=56)), ("SHAPE", dict(ldn=32)), ("SHAPE", dict(ldg=-8, cu=7 * MB, S=2)),
    ("UNSUPPORTED", dict(C=60)), ("UNSUPPORTED", dict(C=8200, ldx=8200, ldy=8200, ldh=8200, ldn=8200)),
    ("ALIGNMENT", dict(x=MB + 2)), ("ALIGNMENT", dict(ldy=68)), ("ALIGNMENT", dict(scale=4 * MB + 8)),
    ("ALIGNMENT", dict(lds=68, cu=7 * MB, S=2)), ("ALIGNMENT", dict(cu=MB + 2)),
    ("INVALID_ARG", dict(cu=5 * MB + 64)), ("INVALID_ARG", dict(cu=6 * MB - 4)),   # over h, into n
    ("UNSUPPORTED", dict(T=1 << 30)),
]


@pytest.mark.parametrize("status,kw", NORM_BAD, ids=[f"{s}-{i}" for i, (s, _) in enumerate(NORM_BAD)])
def test_norm_gate_refuses(svdq, status, kw):
    got = svdq._lib.svdq_norm_gate_residual(*norm_args(**kw))
    assert got == getattr(svdq, "SVDQ_ERR_" + status)


def on_device(svdq, status):
    """A call whose arguments pass gets as far as the device (none here)."""
    return torch.cuda.is_available() or status in (svdq.SVDQ_ERR_CUDA, svdq.SVDQ_ERR_ARCH)


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")

NORM_GOOD = [
    dict(), dict(h=1 * MB), dict(n=1 * MB), dict(h=2 * MB, n=1 * MB), dict(ldg=0, lds=0),
    dict(n=None, pre=0, scale=None), dict(y=None, h=None, post=0, gate_kind=0, gate=None),
    # x, h and n side by side in the rows of one buffer
    dict(ldx=192, h=1 * MB + 128, ldh=192, n=1 * MB + 256, ldn=192),
    # strides that step over nothing
    dict(T=1, ldx=0, ldy=-4, ldh=3, ldn=0), dict(ldg=-8, lds=68), dict(cu=6 * MB - 8),
]


@needs_no_gpu
@pytest.mark.parametrize("kw", NORM_GOOD, ids=range(len(NORM_GOOD)))
def test_norm_gate_takes(svdq, kw):
    assert on_device(svdq, svdq._lib.svdq_norm_gate_residual(*norm_args(**kw)))


def rope_args(svdq, axes=(16, 24, 24), **kw):
    ax = (ctypes.c_int * max(1, len(axes)))(*axes)
    turns = (ctypes.c_double * 256)()
    a = dict(dtype=0, q=1 * MB, qst=192, qsh=64, Hq=2, k=1 * MB + 256, kst=192, ksh=64, Hk=1, T=16,
             D=64, pos=3 * MB, ldp=max(1, len(axes)), axes=ax, n_axes=len(axes), turns=turns, il=1, qw=None, kw=None,
             eps=1e-6, qo=4 * MB, qost=128, qosh=64, ko=5 * MB, kost=64, kosh=64, stream=None)
    a.update(kw)
    return list(a.values())


ROPE_BAD = [
    ("INVALID_ARG", dict(dtype=7)), ("INVALID_ARG", dict(axes=())), ("INVALID_ARG", dict(axes=(2,) * 5)),
    ("INVALID_ARG", dict(eps=-1.0)), ("INVALID_ARG", dict(q=None)), ("INVALID_ARG", dict(ko=None)),
    ("INVALID_ARG", dict(pos=None)), ("INVALID_ARG", dict(turns=None)),
    ("INVALID_ARG", dict(Hq=0)),                         # q given, no heads
    ("INVALID_ARG", dict(qo=1 * MB + 16, qost=192)),     # shifted inside its input
    ("INVALID_ARG", dict(qo=1 * MB + 256, qost=192)),    # over k
    ("INVALID_ARG", dict(ko=4 * MB)),                    # over q_out
    ("INVALID_ARG", dict(qo=3 * MB)),                    # over the positions
    ("INVALID_ARG", dict(qost=64)),                      # its own heads meet
    ("SHAPE", dict(axes=(16, 24, 32))), ("SHAPE", dict(axes=(15, 24))), ("SHAPE", dict(axes=(0, 24))),
    ("SHAPE", dict(T=-1)), ("SHAPE", dict(Hq=-1)), ("SHAPE", dict(D=0)), ("SHAPE", dict(ldp=2)),
    ("SHAPE", dict(qst=32)), ("SHAPE", dict(qosh=32)),
    ("UNSUPPORTED", dict(D=68)), ("UNSUPPORTED", dict(D=264, qst=1024, qsh=264)),
    ("UNSUPPORTED", dict(axes=(16, 20), il=0)),          # R = 36 in halves
    ("ALIGNMENT", dict(q=MB + 2)), ("ALIGNMENT", dict(qst=196)), ("ALIGNMENT", dict(qosh=68, qost=136)),
    ("ALIGNMENT", dict(qw=8 * MB + 2)),
    ("UNSUPPORTED", dict(T=1 << 30)),
]


@pytest.mark.parametrize("status,kw", ROPE_BAD, ids=[f"{s}-{i}" for i, (s, _) in enumerate(ROPE_BAD)])
def test_rope_refuses(svdq, status, kw):
    assert svdq._lib.svdq_rope_qk(*rope_args(svdq, **kw)) == getattr(svdq, "SVDQ_ERR_" + status)


@needs_no_gpu
@pytest.mark.parametrize("kw", [
    dict(), dict(qo=1 * MB, qost=192, ko=1 * MB + 256, kost=192),            # both in place
    dict(k=None, Hk=0, ko=None), dict(q=None, Hq=0, qo=None), dict(T=1, qst=0, kst=0, qost=8),
    dict(axes=(16, 24, 24), il=0), dict(axes=(2, 4)), dict(T=1, ldp=0),
], ids=range(8))
def test_rope_takes(svdq, kw):
    assert on_device(svdq, svdq._lib.svdq_rope_qk(*rope_args(svdq, **kw)))


def test_rope_plan(svdq):
    import math
    plan = svdq.RopePlan((16, 24, 24), theta=256.0, head_dim=128)
    want = [256.0 ** (-2 * i / d) / (2 * math.pi) for d in (16, 24, 24) for i in range(d // 2)]
    assert list(plan._turns) == pytest.approx(want, rel=1e-15)
    for bad in ((), (2,) * 5, (3, 4), (0, 2), (-2, 4)):
        with pytest.raises((svdq.SvdqError, ValueError)):
            svdq.RopePlan(bad, theta=256.0, head_dim=128)
    with pytest.raises(ValueError):
        svdq.RopePlan((64, 80), theta=256.0, head_dim=128)
    for theta in (0.0, -1.0, 0.999, 1e-310, math.nan, math.inf):
        with pytest.raises(svdq.SvdqError):
            svdq.RopePlan((64,), theta=theta, head_dim=128)


def attn_args(**kw):
    # q | k | v in the rows of one buffer, out apart
    a = dict(dtype=0, q=1 * MB, qst=512, qsh=64, k=1 * MB + 512, kst=512, ksh=64, v=1 * MB + 768,
             vst=512, vsh=64, T=16, Hq=4, Hk=2, D=64, cu=None, S=1, causal=0, scale=0.125, out=3 * MB,
             ost=256, osh=64, ws=None, ws_bytes=0, stream=None)
    a.update(kw)
    return list(a.values())


ATTN_BAD = [
    ("INVALID_ARG", dict(dtype=2)), ("INVALID_ARG", dict(scale=0.0)), ("INVALID_ARG", dict(scale=-1.0)),
    ("INVALID_ARG", dict(scale=float("nan"))), ("INVALID_ARG", dict(scale=float("inf"))),
    ("INVALID_ARG", dict(q=None)), ("INVALID_ARG", dict(out=None)),
    ("INVALID_ARG", dict(out=1 * MB, ost=512)), ("INVALID_ARG", dict(out=1 * MB + 512, ost=512)),
    ("INVALID_ARG", dict(out=1 * MB + 896, ost=512)),
    ("SHAPE", dict(T=-1)), ("SHAPE", dict(Hq=0)), ("SHAPE", dict(Hk=0)), ("SHAPE", dict(Hq=3)),
    ("SHAPE", dict(D=0)), ("SHAPE", dict(S=0)), ("SHAPE", dict(S=2)), ("SHAPE", dict(qst=32)),
    ("SHAPE", dict(ksh=56)), ("SHAPE", dict(vst=-512)),
    ("UNSUPPORTED", dict(D=60)), ("UNSUPPORTED", dict(D=136, qsh=136, ksh=136, vsh=136, osh=136)),
    ("UNSUPPORTED", dict(Hq=1 << 20, Hk=1 << 20, T=1 << 20)), ("UNSUPPORTED", dict(T=1 << 30)),
    ("UNSUPPORTED", dict(cu=MB, S=1 << 29)),
    ("INVALID_ARG", dict(ost=64, osh=64)), ("INVALID_ARG", dict(ost=128, osh=64)),     # out's own rows meet
    ("UNSUPPORTED", dict(qst=1 << 39)),
    ("ALIGNMENT", dict(k=MB + 520)), ("ALIGNMENT", dict(vst=516)), ("ALIGNMENT", dict(osh=68)),
    ("ALIGNMENT", dict(cu=MB + 1)), ("ALIGNMENT", dict(ws=5 * MB + 8, ws_bytes=1 << 30)),
    ("INVALID_ARG", dict(ws=3 * MB - 16, ws_bytes=32)),      # over out
    ("INVALID_ARG", dict(scale=3e38)), ("INVALID_ARG", dict(cu=3 * MB + 16)),
    ("INVALID_ARG", dict(ws=5 * MB, ws_bytes=1 << 10, cu=5 * MB + 64)),
]


@pytest.mark.parametrize("status,kw", ATTN_BAD, ids=[f"{s}-{i}" for i, (s, _) in enumerate(ATTN_BAD)])
def test_attention_refuses(svdq, status, kw):
    assert svdq._lib.svdq_attention(*attn_args(**kw)) == getattr(svdq, "SVDQ_ERR_" + status)


@needs_no_gpu
@pytest.mark.parametrize("kw", [dict(),
                                # q, k, v and out side by side in one buffer
                                dict(out=1 * MB + 1024, qst=768, kst=768, vst=768, ost=768),
                                dict(T=1, qst=0, kst=0, vst=0, ost=0), dict(Hq=1, Hk=1, qsh=0, osh=3)],
                         ids=range(4))
def test_attention_takes(svdq, kw):
    assert on_device(svdq, svdq._lib.svdq_attention(*attn_args(**kw)))


def test_empty_calls_return_ok(svdq):
    assert svdq._lib.svdq_norm_gate_residual(*norm_args(T=0, x=None, y=None, h=None, n=None)) == svdq.SVDQ_OK
    assert svdq._lib.svdq_rope_qk(*rope_args(svdq, T=0)) == svdq.SVDQ_OK
    assert svdq._lib.svdq_attention(*attn_args(T=0, q=None)) == svdq.SVDQ_OK


def test_binding_refuses_host_tensors_and_wrong_types(svdq):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    plan = svdq.RopePlan((16, 24, 24), 256.0, 64)
    pos = torch.zeros(4, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        svdq.norm_gate_residual(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        svdq.rope_qk(q, q, pos, plan)
    with pytest.raises(ValueError, match="needs q or k"):
        svdq.rope_qk(None, None, pos, plan)
    with pytest.raises(ValueError, match="CUDA"):
        svdq.attention(q, q, q)


# ---- the divided walk: places of a line, cut into runs ----------------------------

def place_items(lens, Hq, causal):
    """(first place, item) of every item in order; an item takes a place more
    than its key tiles."""
    at, begin, out = 0, 0, []
    for n in lens:
        for head in range(Hq):
            for q0 in range(0, n, ITEM):
                k = max(tiles(n, q0, 0, causal), tiles(n, q0, 1, causal))
                out.append((at, begin, n, q0, head, k))
                at += k + 1
        begin += n
    return out, at


def causal_index(r2):
    import math
    i = int(math.sqrt(r2 + 1.0)) - 1
    while i > 0 and i * (i + 2) > r2:
        i -= 1
    while (i + 1) * (i + 3) <= r2:
        i += 1
    return i


def locate(lens, Hq, causal, w):
    """The kernel's closed form: (begin, n, q0, head), place in the item."""
    begin = 0
    for n in lens:
        nt, nk = (n + ITEM - 1) // ITEM, (n + ROWS - 1) // ROWS
        per = nt * (nt + 2) - (2 * nt - nk) if causal else nt * (nk + 1)
        if w < per * Hq:
            head, r2 = divmod(w, per)
            if causal:
                i = causal_index(r2)
                return (begin, n, i * ITEM, head), r2 - i * (i + 2)
            return (begin, n, r2 // (nk + 1) * ITEM, head), r2 % (nk + 1)
        w -= per * Hq
        begin += n
    return None, -1


def run_edge(lens, Hq, causal, w, total, run):
    if w >= total:
        return total
    (begin, n, q0, head), r = locate(lens, Hq, causal, w)
    k = max(tiles(n, q0, 0, causal), tiles(n, q0, 1, causal)) + 1
    near = 1 + max(1, run // 16)
    return w - r if r <= near else w + k - r if k - r < near else w


@pytest.mark.parametrize("lens,Hq", [([16384], 1), ([8192], 2), ([2600], 1), ([5000, 1, 0, 4000], 3), ([700], 2)])
@pytest.mark.parametrize("causal", [False, True])
def test_divided_runs_cover_every_key_tile_once(lens, Hq, causal):
    line, total = place_items(lens, Hq, causal)
    for at, begin, n, q0, head, k in line:
        for r in range(k + 1):
            assert locate(lens, Hq, causal, at + r) == ((begin, n, q0, head), r)
    G = 148
    run = max(6, (total + G - 1) // G)
    seen, ends = set(), []
    for b in range(G):
        at = run_edge(lens, Hq, causal, min(b * run, total), total, run)
        end = run_edge(lens, Hq, causal, min((b + 1) * run, total), total, run)
        first = True
        while at < end:
            (begin, n, q0, head), r = locate(lens, Hq, causal, at)
            k = max(tiles(n, q0, 0, causal), tiles(n, q0, 1, causal))
            ka, kb = max(0, r - 1), min(k, end - at + r - 1)
            assert 0 <= ka < kb <= k
            assert ka == 0 or first          # only a run's first item may have begun in front of it
            assert kb == k or at + 1 + kb - r >= end
            for j in range(ka, kb):
                assert (begin, q0, head, j) not in seen
                seen.add((begin, q0, head, j))
            at += 1 + kb - r
            first = False
    assert len(seen) == sum(k for *_, k in line)


# ---- the attention kernel's work items -------------------------------------------

ROWS, ITEM = 128, 256


def items(cu, T, Hq, causal):
    """The line of items that the kernel deals out: groups of 32 sequences;
    causal: item i of every sequence that has one, then i - 1; full: longest
    sequence first."""
    S, front = len(cu) - 1, 0
    for s0 in range(0, S, 32):
        seqs = []
        for s in range(s0, min(s0 + 32, S)):
            begin = max(min(max(cu[s], 0), T), front)
            front = max(min(max(cu[s + 1], 0), T), begin)
            seqs.append((begin, front - begin))
        if causal:
            for i in range(max((n + ITEM - 1) // ITEM for _, n in seqs) - 1, -1, -1):
                yield from ((b, n, i * ITEM, h) for b, n in seqs if n > i * ITEM for h in range(Hq))
        else:
            for b, n in sorted(seqs, key=lambda x: -x[1]):
                yield from ((b, n, q0, h) for h in range(Hq) for q0 in range(0, n, ITEM))


def dealt(line, blocks):
    """The items of each block: rounds, every other one turned."""
    out = [[] for _ in range(blocks)]
    for k, at in enumerate(range(0, len(line), blocks)):
        for b in range(blocks):
            w = at + (blocks - 1 - b if k % 2 else b)
            if w < len(line):
                out[b].append(line[w])
    return out


@pytest.mark.parametrize("blocks", [1, 7, 148])
def test_items_are_dealt_once_and_evenly(blocks):
    line = list(items([0, 5000, 5100, 9000], 9000, 8, True))
    got = dealt(line, blocks)
    assert sorted(x for b in got for x in b) == sorted(line)
    load = [sum(max(tiles(n, q0, 0, True), tiles(n, q0, 1, True)) for _, n, q0, _ in b) for b in got]
    assert max(load) <= 1.25 * sum(load) / blocks + 2


def tiles(n, q0, s, causal):
    if q0 + s * ROWS >= n:
        return 0
    t = (n + ROWS - 1) // ROWS
    return min(t, q0 // ROWS + s + 1) if causal else t


LENGTHS = [[1], [128], [129], [256], [257], [0, 5, 0], [300, 1, 0, 700], [3] * 70, [0] * 40 + [260], []]


@pytest.mark.parametrize("lens,causal", list(itertools.product(LENGTHS, (False, True))))
def test_items_cover_every_row_and_head_once(lens, causal):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    T, Hq = cu[-1], 3
    if len(cu) == 1:
        cu.append(0)
    seen = {}
    got = list(items(cu, T, Hq, causal))
    assert len(got) <= (T // ITEM + len(cu) - 1) * Hq        # the grid's bound
    for begin, n, q0, head in got:
        for s in range(2):
            t = tiles(n, q0, s, causal)
            for i in range(q0 + s * ROWS, min(n, q0 + (s + 1) * ROWS)):
                # the tiles cover exactly the keys the row attends
                assert t * ROWS > i if causal else t * ROWS >= n
                key = (begin + i, head)
                assert key not in seen
                seen[key] = True
        assert tiles(n, q0, 0, causal) >= 1
        # slot 1 never reads fewer tiles than slot 0, unless it has no rows
        assert tiles(n, q0, 1, causal) in (0, tiles(n, q0, 0, causal)) or causal
    assert len(seen) == T * Hq


@pytest.mark.parametrize("cu", [[5, 2, 900, 300], [-7, 10, 2000, 2 ** 31 - 1], [-2 ** 31, 2 ** 31 - 1], [3, 3, 3],
                                [0, 777] * 40])
def test_items_of_bad_offsets_stay_inside(cu):
    T = 777
    # no row twice, so at most T rows together
    seen = [(b + r, h) for b, n, q0, h in items(cu, T, 2, False) for r in range(q0, min(n, q0 + ITEM))]
    assert len(seen) == len(set(seen)) <= 2 * T
    for begin, n, q0, head in items(cu, T, 2, True):
        assert 0 <= begin and begin + n <= T and 0 <= q0 < n and 0 <= head < 2


def find_sequence(cu, S, row):
    """The warp's search: ends <= row, 32 probes a step."""
    lo, hi = 0, S
    while lo < hi:
        step = (hi - lo + 31) // 32
        yes = 0
        for lane in range(32):
            at = lo + (lane + 1) * step
            if at <= hi:
                assert 0 <= at <= S
                yes += cu[at] <= row
        lo += yes * step
        hi = min(hi, lo + step - 1)
    return lo


@pytest.mark.parametrize("S", [1, 2, 31, 32, 33, 100, 1025])
def test_find_sequence(S):
    g = torch.Generator().manual_seed(S)
    cu = [0] + torch.randint(0, 4, (S,), generator=g).cumsum(0).tolist()
    for row in range(cu[-1] + 2):
        assert find_sequence(cu, S, row) == sum(c <= row for c in cu[1:])
    bad = torch.randint(-5, 5, (S + 1,), generator=g).tolist()
    for row in range(5):
        assert 0 <= find_sequence(bad, S, row) <= S
