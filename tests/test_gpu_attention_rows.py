"""attention, row by row: what a row gets depends on its own query and on the
keys and values it attends, bit for bit.  Nothing of the rows that share its
warp, of the keys behind it (causal) or of the rows behind its sequence shows,
however large they are."""

import pytest
import torch

import gpu_helpers as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16
# Finite and large (scores past the rescale step and past 2^12 log2 units), and not finite.
BAD = {BF: [300.0, 3e4, 1e30, float("inf"), float("-inf")], HF: [300.0, 3e4, float("inf"), float("-inf")]}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_quantized_smooth_b200 import build
    build.build()
    torch.cuda.init()


def make(T, Hq, Hk, D, dtype, seed, by=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [(torch.randn(T, n, D, generator=g, device=DEV) * s).to(dtype)
            for n, s in ((Hq, by), (Hk, by), (Hk, 1.0))]


def offsets(*cu):
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_take_their_results_with_them(D, dtype):
    """Queries of very different sizes, in another order: the same results in
    that order."""
    s = H.svdq()
    T = 900
    q, k, v = make(T, 2, 1, D, dtype, seed=1)
    # maxima that grow by about the rescale step along the keys, more in some rows than in others
    k += (torch.linspace(0, 6, T, device=DEV)[:, None, None] * torch.sign(k[:1].float()) / D ** 0.5).to(dtype)
    size = 2.0 ** torch.randint(-2, 7, (T, 1, 1), device=DEV, generator=torch.Generator(device=DEV).manual_seed(2))
    q = (q.float() * size).to(dtype)
    clean = s.attention(q, k, v)
    for seed in range(4):
        at = torch.randperm(T, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed))
        got = s.attention(q[at], k, v)
        s.check_device_error()
        assert torch.equal(got, clean[at])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("at", [1, 20, 100, 127, 140, 159, 200, 255, 300, 511, 700])
def test_causal_rows_in_front_of_a_large_key(at, dtype):
    s = H.svdq()
    q, k, v = make(800, 2, 1, 128, dtype, seed=3)
    clean = s.attention(q, k, v, causal=True)
    for bad in BAD[dtype]:
        k2, v2 = k.clone(), v.clone()
        k2[at, 0, 9] = bad
        v2[at, 0, 5] = bad
        for a in ((k2, v), (k, v2), (k2, v2)):
            got = s.attention(q, *a, causal=True)
            s.check_device_error()
            assert torch.equal(got[:at], clean[:at]), (at, bad)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("causal", [False, True])
def test_rows_behind_a_sequence(causal, dtype):
    """A sequence alone, and with others packed behind it whose queries, keys
    and values are large."""
    s = H.svdq()
    for L in (1, 40, 150, 300, 390):
        q, k, v = make(800, 2, 1, 128, dtype, seed=L)
        alone = s.attention(q[:L], k[:L], v[:L], causal=causal)
        for bad in [1.0] + BAD[dtype]:
            q2, k2, v2 = (t.clone() for t in (q, k, v))
            for t in (q2, k2, v2):
                t[L:] *= bad
            for cu in (offsets(0, L, 800), offsets(0, L)):
                got = s.attention(q2, k2, v2, cu, causal)
                s.check_device_error()
                assert torch.equal(got[:L], alone), (L, bad)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_causal_prefixes(dtype):
    """The first rows of a causal sequence do not depend on its length."""
    s = H.svdq()
    q, k, v = make(1500, 2, 1, 128, dtype, seed=4, by=2.0)
    whole = s.attention(q, k, v, causal=True)
    for L in (1, 17, 129, 500, 777, 1499):
        assert torch.equal(s.attention(q[:L], k[:L], v[:L], causal=True), whole[:L])


@pytest.mark.parametrize("dtype", [BF, HF])
def test_divided_rows_in_front_of_a_large_key(dtype):
    s = H.svdq()
    T = 4000
    assert s._lib.svdq_attention_workspace_bytes(T, 1, 1, 128, 1) > 0
    q, k, v = make(T, 1, 1, 128, dtype, seed=5)
    clean = s.attention(q, k, v, causal=True)
    for at in (20, 700, 1111, 2900, 3999):
        for bad in BAD[dtype]:
            k2 = k.clone()
            k2[at, 0, 9] = bad
            got = s.attention(q, k2, v, causal=True)
            s.check_device_error()
            assert torch.equal(got[:at], clean[:at]), (at, bad)
