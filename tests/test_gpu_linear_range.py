"""Linear attention on the GPU where magnitudes differ from token to token: fp16, whose
operands are scaled into their range by powers of two, against the definition in 64 bits."""
import pytest

import linear_harness as H

pytestmark = pytest.mark.gpu

W = [(64, 64), (128, 128), (64, 128), (128, 64)]


def end_state(t, s0, b=0):
    """The state after request b's tokens, and the sum of magnitudes behind it, in float64:
    lam^n S + sum_j lam^(n-1-j) k_j^T v_j."""
    import torch
    lo, hi = t["row_offsets"][b:b + 2].tolist()
    k, v = t["k"][lo:hi].double(), t["v"][lo:hi].double()
    lam = torch.exp(t["log_decay"].double().clamp(max=0.0))
    w = lam[None] ** torch.arange(hi - lo - 1, -1, -1)[:, None]                    # [n, h]
    S = torch.einsum("nh,nhd,nhe->hde", w, k, v)
    A = torch.einsum("nh,nhd,nhe->hde", w, k.abs(), v.abs())
    if s0 is not None:
        past = lam[:, None, None] ** (hi - lo) * s0[b].double()
        S, A = S + past, A + past.abs()
    return S, A


@pytest.mark.parametrize("dk,dv", W)
@pytest.mark.parametrize("with_state", [False, True])
def test_segments_with_columns_that_change_by_chunk(dk, dv, with_state):
    # Four chunks to a segment, the columns of V larger by 2^8 in every second chunk, by other
    # powers in every fourth: a scale of the wrong chunk is wrong by a power of two.  The
    # bound is the harness's: every decayed value enters with 22 bits.
    import torch
    n, heads = 2000, 38
    t, s0 = H.make([n], heads, dk, dv, "fp16", seed=41, state=with_state,
                   decay=None if with_state else -2.0 ** -11)
    g = torch.Generator().manual_seed(42)
    p = torch.randint(-3, 4, (4, heads, dv), generator=g) + torch.tensor([0, 8, 0, 8])[:, None, None] - 4
    t["v"] = (t["v"].float() * torch.exp2(p[torch.arange(n) // H.C % 4].float())).half()
    out, state, bits = H.run(t, s0, 0.1)
    assert bits == 0
    S, A = end_state(t, s0)
    err = (state[0].double() - S).abs()
    chunks = -(-n // H.C)
    assert bool((err <= A * 2.0 ** -23 * (48 + 4 * chunks) + 1e-37).all()), (err / A).max()
    assert torch.isfinite(out.float()).all()


def two_terms(t, b=0):
    """What the fp16 operands of the state's update cost, per value of S: sum over chunks c
    of lam^(tokens behind c) 2^-39 M sum_j |k_j|, M the largest lam^(m-1-j) |v_j| of a column
    in the chunk.

    A decayed value x is split into two fp16 terms after a scaling by a power of two that takes
    M into [2^14, 2^15).  The first is off by at most 2^-11 |x|, which the second holds to
    2^-11 of itself, or to half of fp16's smallest step, 2^-25, where it is below
    2^-14: 2^-22 |x| (22 bits, in the harness's bound) or 2^-25 <= 2^-39 M.
    """
    import torch
    lo, hi = t["row_offsets"][b:b + 2].tolist()
    k, v = t["k"][lo:hi].double().abs(), t["v"][lo:hi].double().abs()
    lam = torch.exp(t["log_decay"].double().clamp(max=0.0))
    n = hi - lo
    extra = torch.zeros(k.shape[1], k.shape[2], v.shape[2], dtype=torch.float64)
    for c in range(0, n, H.C):
        m = min(H.C, n - c)
        w = lam[None] ** torch.arange(m - 1, -1, -1)[:, None]
        M = (w[..., None] * v[c:c + m]).amax(dim=0)
        extra += (lam ** (n - c - m))[:, None, None] * 2.0 ** -39 * k[c:c + m].sum(dim=0)[..., None] * M[:, None]
    return extra


@pytest.mark.parametrize("dk,dv", W)
@pytest.mark.parametrize("n,heads", [(300, 2), (2000, 38)])
def test_an_early_outlier_that_is_forgotten(dk, dv, n, heads):
    # The first token of every chunk has the largest fp16 values, the others are about 2^-26 of
    # them, and fast heads forget it within the chunk: the others are the state, and enter it
    # with as many bits as ever.  In one walk (300 tokens) and in segments of four chunks.
    import torch
    t, s0 = H.make([n], heads, dk, dv, "fp16", seed=43, amp=1e-3)
    t["k"] = torch.randn(n, heads, dk, generator=torch.Generator().manual_seed(44)).half()
    t["v"][::H.C] = torch.where(t["v"][::H.C] < 0, -6e4, 6e4).half()
    t["log_decay"] = torch.linspace(-1.5, -0.2, heads)
    out, state, bits = H.run(t, s0, 0.1)
    assert bits == 0
    S, A = end_state(t, s0)
    err = (state[0].double() - S).abs()
    chunks = -(-n // H.C)
    bound = A * 2.0 ** -23 * (48 + 4 * chunks) + two_terms(t) + 1e-37
    assert bool((err <= bound).all()), f"state off by {(err / bound).max():.3g} x its bound"


def output_bound(t, s0, scale, out):
    """How far an fp16 output may be off (one request): the harness's bound with the two terms
    of fp16's range taken from what is rounded.  A row of P = lam^(i-j) q_i . k_j and a
    column of the state are scaled so that their largest lies in [2^14, 2^15), and rounded to
    11 bits (u of each), or by half of fp16's smallest step, 2^-25 <= 2^-39 of the largest."""
    import torch
    u, C = 2.0 ** -11, H.C
    q, k, v = (t[x].double() for x in "qkv")
    lam = torch.exp(t["log_decay"].double().clamp(max=0.0))
    n = q.shape[0]
    S = s0[0].double() if s0 is not None else torch.zeros(*q.shape[1:], v.shape[2], dtype=torch.float64)
    bound = 1.01 * u * out.abs() + 2.0 ** -25
    for c in range(0, n, C):
        m, x = min(C, n - c), slice(c, min(c + C, n))
        w = torch.arange(m)[:, None] - torch.arange(m)[None]
        D = torch.where(w >= 0, lam[:, None, None] ** w.clamp(min=0), torch.zeros((), dtype=torch.float64))
        s = D * torch.einsum("ihd,jhd->hij", q[x], k[x]).abs()
        sa = D * torch.einsum("ihd,jhd->hij", q[x].abs(), k[x].abs())
        low = 2.0 ** -39 * s.amax(dim=2, keepdim=True) * (w >= 0)
        bound[x] += abs(scale) * torch.einsum("hij,jhe->ihe", 1.01 * u * s + 2.0 ** -17 * sa + low, v[x].abs())
        reach = lam[None] ** (torch.arange(m)[:, None] + 1)
        col = 1.01 * (u + 2.0 ** -15) * S.abs() + 2.0 ** -39 * S.abs().amax(dim=1, keepdim=True)
        bound[x] += abs(scale) * reach[..., None] * torch.einsum("ihd,hde->ihe", q[x].abs(), col)
        dec = lam[:, None] ** (m - 1 - torch.arange(m))[None]
        S = lam[:, None, None] ** m * S + torch.einsum("hj,jhd,jhe->hde", dec, k[x], v[x])
    return bound


@pytest.mark.parametrize("dk,dv", W)
@pytest.mark.parametrize("scale", [100.0, -3e4, 1e-25])
@pytest.mark.parametrize("with_state", [False, True])
def test_an_early_key_that_is_forgotten(dk, dv, scale, with_state):
    # The first key of every chunk is about 2^31 times the others, and the heads forget it in a few
    # tokens to a few dozen: later rows' weights are the others', in full precision.  Some keys are zero,
    # so that a row's largest weight may lie anywhere.
    import torch
    n, heads = 300, 6
    t, s0 = H.make([n], heads, dk, dv, "fp16", seed=45, state=with_state)
    g = torch.Generator().manual_seed(46)
    t["k"] = (torch.randn(n, heads, dk, generator=g) * 2e-5).half()
    t["k"][::H.C] = torch.where(t["k"][::H.C] < 0, -6e4, 6e4).half()
    t["k"][torch.rand(n, generator=g) < 0.3] = 0.0
    if s0 is not None:
        s0 = s0 * 1e-4
    t["log_decay"] = torch.tensor([-20.0, -3.0, -1.5, -1.0, -0.7, -0.5])
    out, state, bits = H.run(t, s0, scale)
    assert bits == 0
    ref = H.reference(t, s0, scale)[0][0]
    fits = ref.abs() < 6e4                         # (behind an outlier, outputs overflow fp16)
    bound = output_bound(t, s0, scale, ref)
    err = (out.double() - ref).abs()
    assert bool((err <= bound)[fits].all()), f"output off by {(err / bound)[fits].max():.3g} x its bound"
