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
